"""How kv_cache_select spreads a sequence over CTAs and where its keys are held, on the CPU."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_prologue_kv_gb300", "csrc")
PROGRAM = """
#include <stdio.h>
#include "select_plan.cuh"
int main() {
    long long len, n; int sms, most;
    while (scanf("%lld %lld %d %d", &len, &n, &sms, &most) == 4) {
        const kvr::SelectForm f = kvr::select_form(len, n, sms, most);
        printf("%d %lld %d\\n", f.ctas, (long long)f.each, f.form);
    }
}
"""
SHARED, AGAIN = -1, 0


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    src = tmp_path_factory.mktemp("select") / "plan.cpp"
    exe = src.with_suffix("")
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-x", "c++", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def ask(cases):
        out = subprocess.run([str(exe)], input="".join("%d %d %d %d\n" % c for c in cases), check=True, capture_output=True, text=True)
        return [tuple(map(int, line.split())) for line in out.stdout.splitlines()]
    return ask


# (weights of a row, rows, most CTAs of a cluster): (CTAs, keys of a CTA, form)
@pytest.mark.parametrize("length,n,most,want", [
    (1, 1, 16, (1, 1, 1)), (1025, 500, 16, (1, 1025, 2)), (4095, 64, 16, (1, 4095, 4)), (16384, 500, 16, (1, 16384, 16)),
    (16385, 500, 16, (2, 8193, 16)), (131072, 1, 16, (8, 16384, 16)), (131073, 1, 16, (16, 8193, 16)),
    (262144, 1, 16, (16, 16384, 16)), (262145, 1, 16, (16, 16385, SHARED)), (786432, 1, 16, (16, 49152, SHARED)),
    (786433, 1, 16, (16, 49153, AGAIN)), (1 << 30, 1, 16, (16, 1 << 26, AGAIN)),
    # a device without clusters of 16
    (131072, 1, 8, (8, 16384, 16)), (131073, 1, 8, (8, 16385, SHARED)), (393216, 1, 8, (8, 49152, SHARED)),
    (393217, 1, 8, (8, 49153, AGAIN)), (1 << 30, 1, 8, (8, 1 << 27, AGAIN))])
def test_forms(forms, length, n, most, want):
    assert forms([(length, n, 152, most)]) == [want]


def test_every_key_has_a_place(forms):
    cases = [(length, n, sms, most) for length in list(range(0, 3000, 37)) + [2 ** k + d for k in range(11, 30) for d in (-1, 0, 1)]
             for n in (1, 7, 64, 1000) for sms in (148, 152) for most in (8, 16)]
    for (length, n, sms, most), (ctas, each, form) in zip(cases, forms(cases)):
        assert 1 <= ctas <= most and ctas * each >= length and (ctas - 1) * each < max(length, 1)
        assert each <= (1024 * form if form > 0 else 49152 if form == SHARED else 1 << 30)
