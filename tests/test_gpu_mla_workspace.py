"""The workspace that mla_attention takes from PyTorch's allocator: whose memory it is, on which stream, under capture."""
import numpy as np
import pytest
import torch

import attention_prologue_kv_gb300 as kvr
from attention_prologue_kv_gb300 import api
from attention_helpers import mla_case, run_mla

pytestmark = pytest.mark.gpu


def tensors(c):
    d = lambda t: t.cuda().contiguous()  # noqa: E731
    return [d(t) for t in (c.q_nope, c.q_rope, c.ckv, c.k, c.table, c.query_start, c.key_length)]


def keep_busy():
    """The current stream sleeps for some 0.2 s; what follows on it finds its kernels loaded and no free block cached."""
    torch.empty(8, dtype=torch.uint8, device="cuda").fill_(1)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(400_000_000)


@pytest.fixture
def workspaces(monkeypatch):
    """Addresses of the workspaces that calls take."""
    found, launch = [], api.BoundCall.__call__

    def note(call, *a, **kw):
        found.append(call.workspace.data_ptr())
        return launch(call, *a, **kw)

    monkeypatch.setattr(api.BoundCall, "__call__", note)
    return found


CASES = [([3, 1], [900, 1500], 24, 20), ([2] * 9, [700] * 9, 16, 21)]


def cases():
    return [mla_case(new, keys, H, block_size=64, seed=seed) for new, keys, H, seed in CASES]


def test_two_calls_captured_on_branches_of_a_graph(workspaces):
    """Two calls on streams forked inside a capture can run at the same time in a replay: they share no workspace."""
    both = cases()
    alone = [run_mla(c) for c in both]
    del workspaces[:]
    args, outs = [tensors(c) for c in both], [torch.zeros(c.q_nope.shape, device="cuda", dtype=c.q_nope.dtype) for c in both]
    sides = [torch.cuda.Stream() for _ in both]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for side in sides:
            side.wait_stream(main)
        for a, out, c, side in zip(args, outs, both, sides):
            kvr.mla_attention(*a, out, softmax_scale=c.scale, stream=side)
        for side in sides:
            main.wait_stream(side)
    assert len(set(workspaces)) == 2
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    for out, ref in zip(outs, alone):
        assert np.array_equal(out.double().cpu().numpy(), ref[0])


@pytest.mark.parametrize("raw", [False, True])
def test_a_call_on_another_stream_takes_no_memory_that_the_current_one_still_uses(workspaces, raw):
    """A block that was given back while the current stream's work on it waits goes to calls of that stream alone."""
    c = cases()[0]
    ref = run_mla(c)
    args = tensors(c)
    out = torch.zeros_like(args[0])
    size = kvr.prepare_mla_attention(*args, out, softmax_scale=c.scale).workspace.numel()
    side = torch.cuda.Stream()
    keep_busy()
    used = torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
    at = used.data_ptr()
    del used
    del workspaces[:]
    kvr.mla_attention(*args, out, softmax_scale=c.scale, stream=side.cuda_stream if raw else side)
    assert not torch.cuda.current_stream().query(), "the stream was done too early for this test"
    assert workspaces != [at]
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), ref[0])


@pytest.mark.parametrize("given", [True, False])
def test_a_bound_call_on_another_stream_waits_for_its_memory(given):
    """A workspace taken on the current stream, whose block that stream still writes, is not used before that is done."""
    c = cases()[0]
    ref = run_mla(c)
    args = tensors(c)
    out = torch.zeros_like(args[0])
    size = kvr.prepare_mla_attention(*args, out, softmax_scale=c.scale).workspace.numel()
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    keep_busy()
    used = torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
    filled = torch.cuda.Event()
    filled.record()
    at = used.data_ptr()
    del used
    call = kvr.prepare_mla_attention(*args, out, softmax_scale=c.scale)
    assert call.workspace.data_ptr() == at, "another block: nothing to wait for in this test"
    if given:
        call(side)
    else:
        with torch.cuda.stream(side):
            call()
    done.record(side)
    while not done.query():
        pass
    assert filled.query(), "the call did not wait for what the current stream did to its memory"
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), ref[0])


def test_calls_on_the_default_stream_by_its_handle():
    c = cases()[0]
    ref = run_mla(c)
    args = tensors(c)
    for handle in (0, torch.cuda.default_stream().cuda_stream):
        out = torch.zeros_like(args[0])
        with torch.cuda.stream(torch.cuda.Stream()):
            torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
            call = kvr.prepare_mla_attention(*args, out, softmax_scale=c.scale)
            kvr.mla_attention(*args, out, softmax_scale=c.scale, stream=handle)
            torch.cuda.synchronize()
            assert np.array_equal(out.double().cpu().numpy(), ref[0])
            out.zero_()
            torch.cuda.synchronize()
            call(handle)
            torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), ref[0])


def test_a_bound_call_made_and_captured_in_a_graph():
    """Made inside the capture, called on its stream and on one forked behind it."""
    c = cases()[1]
    ref = run_mla(c)
    args = tensors(c)
    outs = [torch.zeros_like(args[0]) for _ in range(2)]
    side, graph, calls = torch.cuda.Stream(), torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for out in outs:
            calls.append(kvr.prepare_mla_attention(*args, out, softmax_scale=c.scale))
        side.wait_stream(main)
        calls[0]()
        calls[1](side)
        main.wait_stream(side)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert np.array_equal(out.double().cpu().numpy(), ref[0])
