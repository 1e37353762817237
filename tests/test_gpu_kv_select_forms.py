"""kv_cache_select around the row widths where it takes other forms, and in rows with far more room than keys."""
import numpy as np
import pytest

from test_gpu_kv_select import run, weights

pytestmark = pytest.mark.gpu


# Registers of 8 CTAs, of 16; ranks in the shared memory of 16; keys read again.
@pytest.mark.parametrize("width", [131072, 131073, 262144, 262145, 786432, 786433])
def test_widths_where_the_form_changes(width):
    run(weights(1, width, 21, "odd"), [width], width // 5, 4, 512, carry=3)
    run(weights(1, width, 22, "few"), [width - 1], width // 2, 0, 100)


@pytest.mark.parametrize("width", [131072, 200000, 500000, 900001])
def test_rows_with_room_for_more_keys(width):
    """Most CTAs of a cluster, or all but one warp of each, have no key."""
    w = weights(5, width, 23, "odd")
    w[:, 4000:] = np.nan    # never read: NaN would be the first to be kept
    run(w, [4000, 1, 17, 0, 3999], 600, 2, 30)
    run(w, [4000, 599, 600, 601, 8], 600, 0, 0)
