"""Calls on a stream other than the current one: the binding's own scratch and
outputs are neither taken from under other work nor handed out under theirs."""
import math

import pytest
import torch

from rope_frequency_chunk_b200 import fasa as F
from tests import span_util as S

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HOLD = 40_000_000  # cycles that a stream is kept busy, about 20 ms


@pytest.fixture(autouse=True)
def _clean_status():
    F.fasa_device_status(clear=True)
    yield
    assert F.fasa_device_status(clear=True) == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=S.DEV)


def scribble(sizes):
    """Takes and fills blocks of these bytes on the current stream, several
    times each: what the allocator has free there is handed out."""
    for n in sizes:
        for x in [torch.empty(n, dtype=torch.uint8, device=S.DEV) for _ in range(4)]:
            x.fill_(255)


def beside(call):
    """call(stream) on a side stream that is still busy when the current one
    has already taken and filled the memory that is free to it."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
    got = call(side)
    return side, got


@pytest.mark.parametrize("raw", [False, True])
def test_scratch_of_a_call_on_a_side_stream(raw):
    f = S.Filled([1200, 333], 8, 2, BF, 16)
    q = (S.randn(f.g, 2, 8, 128) * 1.5).to(BF)
    qp = (S.randn(f.g, 2, 5, 8, 128) * 1.5).to(BF)
    m0 = torch.rand(2, 2, f.cache.max_len, generator=f.g, device=S.DEV)

    m_ref = m0.clone()
    ref = [F.fasa_attend_decode(f.cache, f.seq_len, q, 1200, mass=m_ref),
           F.fasa_attend_prompt(f.cache, f.seq_len, qp, 1200)]
    ws = [F.fasa_attend_decode_workspace(f.cache, 1200, mass=True).numel(),
          F.fasa_attend_prompt_workspace(f.cache, 5, 1200).numel(), q.numel() * 2, qp.numel() * 2]
    m = m0.clone()
    torch.cuda.synchronize()

    def call(side):
        s = side.cuda_stream if raw else side
        a = F.fasa_attend_decode(f.cache, f.seq_len, q, 1200, mass=m, stream=s)
        b = F.fasa_attend_prompt(f.cache, f.seq_len, qp, 1200, stream=s)
        return a, b

    _, (a, b) = beside(call)
    scribble(ws)
    torch.cuda.synchronize()
    assert torch.equal(a, ref[0]) and torch.equal(b, ref[1]) and torch.equal(m, m_ref)


def test_eviction_on_a_side_stream():
    fs = [S.Filled([3000, 2500], 8, 4, BF, 16, seed=5) for _ in range(2)]
    m = [torch.rand(2, 4, f.cache.max_len, generator=torch.Generator(S.DEV).manual_seed(1), device=S.DEV) for f in fs]
    pos = [torch.arange(f.cache.max_len, device=S.DEV).int().expand(2, 4, -1).contiguous() for f in fs]
    cur = i32([2999, 2499])
    args = dict(max_seq_len=3000, budget=1400, n_sink=4, n_recent=50)
    n_ref = F.fasa_evict(fs[0].cache, fs[0].seq_len, cur, m[0], pos[0], **args)
    ws = F.fasa_evict_workspace(fs[1].cache, 3000, 1400).numel()
    torch.cuda.synchronize()
    _, n = beside(lambda side: F.fasa_evict(fs[1].cache, fs[1].seq_len, cur, m[1], pos[1], stream=side, **args))
    scribble([ws, 8])
    torch.cuda.synchronize()
    assert torch.equal(n, n_ref) and torch.equal(m[0], m[1]) and torch.equal(pos[0], pos[1])
    a, b = fs[0].cache, fs[1].cache
    for x, y in ((a.k, b.k), (a.v, b.v), (a.sketch, b.sketch)):
        assert torch.equal(x.nan_to_num(9.0), y.nan_to_num(9.0))


def test_two_streams_with_a_workspace_each():
    """Both workspaces live through all calls, and every call has queries of
    its own."""
    f = S.Filled([1200, 333], 8, 2, BF, 16)
    qs = [(S.randn(f.g, 2, 8, 128) * 1.5).to(BF) for _ in range(8)]
    ref = [F.fasa_attend_decode(f.cache, f.seq_len, q, 1200) for q in qs]
    side = torch.cuda.Stream()
    ws = [F.fasa_attend_decode_workspace(f.cache, 1200) for _ in range(2)]
    assert ws[0].data_ptr() != ws[1].data_ptr()
    outs = [torch.full_like(q, math.nan) for q in qs]
    torch.cuda.synchronize()
    for i, q in enumerate(qs):
        F.fasa_attend_decode(f.cache, f.seq_len, q, 1200, workspace=ws[i % 2], out=outs[i],
                             stream=side if i % 2 else None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_fasa_decode_on_a_side_stream():
    """The sparse decode's scratch has to be zero before its first launch."""
    f = S.Filled([1500], 8, 2, BF, cap=1500)
    q = (S.randn(f.g, 1, 8, 128) * 1.5).to(BF)
    ref = F.fasa_decode(f.cache, 1500, q, 1500, 64)
    torch.cuda.synchronize()
    scribble([F.fasa_decode_workspace_bytes(f.cache, 1500, 64), q.numel() * 2])  # dirty memory is free
    torch.cuda.synchronize()
    _, out = beside(lambda side: F.fasa_decode(f.cache, 1500, q, 1500, 64, stream=side))
    scribble([F.fasa_decode_workspace_bytes(f.cache, 1500, 64), q.numel() * 2])
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


def test_a_side_stream_inside_a_capture():
    """Calls on a forked stream of a captured graph: their scratch belongs to
    the graph, and replays give the eager results."""
    f = S.Filled([1200, 333], 8, 2, BF, 16)
    q = (S.randn(f.g, 2, 8, 128) * 1.5).to(BF)
    qp = (S.randn(f.g, 2, 5, 8, 128) * 1.5).to(BF)
    ref = [F.fasa_attend_decode(f.cache, f.seq_len, q, 1200), F.fasa_attend_prompt(f.cache, f.seq_len, qp, 1200)]
    outs = [torch.zeros_like(x) for x in ref]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        outs[1].copy_(F.fasa_attend_prompt(f.cache, f.seq_len, qp, 1200))
        a = F.fasa_attend_decode(f.cache, f.seq_len, q, 1200, stream=side)
        main.wait_stream(side)
        outs[0].copy_(a)
    del a
    for _ in range(3):
        for x in outs:
            x.zero_()
        scribble([1 << 20, 1 << 24])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], ref[0]) and torch.equal(outs[1], ref[1])
