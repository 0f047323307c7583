"""The prompt attention's workspace: what is sized for the longest call serves
the shorter ones (host side, no GPU needed)."""
import ctypes

import pytest

from tests.test_abi import L, _fake_cache  # noqa: F401  (L: fixture)
from tests.test_span_abi import span

NQ = (1, 2, 5, 8, 31, 32, 33, 64, 100, 255, 256, 257, 1000, 4096, 8191, 8192, 100000)


@pytest.mark.parametrize("batch,hq,hkv", [(1, 32, 8), (1, 8, 8), (1, 1, 1), (2, 28, 4), (1, 16, 1), (9, 32, 8),
                                          (40, 32, 8), (1, 9, 3)])
@pytest.mark.parametrize("max_len", [100, 1024, 8192, 1 << 20])
def test_a_workspace_for_many_queries_serves_few(L, batch, hq, hkv, max_len):
    c = ctypes.byref(_fake_cache(batch=batch, n_q_heads=hq, n_kv_heads=hkv, max_len=max_len))
    ws = L.fasa_attend_prompt_workspace_bytes
    whole = span(max_seq_len=max_len)
    sizes = [ws(c, whole, n) for n in NQ]
    assert all(a > 0 for a in sizes) and sizes == sorted(sizes)
    # shorter lengths and any window within it too
    for n in NQ:
        assert all(ws(c, span(max_seq_len=min(m, max_len), window=w, n_sink=k), n) <= sizes[NQ.index(n)]
                   for m in (1, 257, 1000, 5000, max_len) for w in (0, 1, 300, 4096) for k in (0, 70))


def test_a_call_asks_for_no_more_than_it_uses(L):
    """Many queries are not cut into parts: 256 bytes serve them, and not few."""
    c = ctypes.byref(_fake_cache(batch=1, n_q_heads=32, n_kv_heads=8, max_len=8192))
    run, ws = L.fasa_attend_prompt, L.fasa_attend_prompt_workspace_bytes
    sp = span(max_seq_len=8192)
    need = ws(c, sp, 5)
    assert need > 1 << 20 and ws(c, sp, 8192) >= need
    assert run(c, None, sp, 0x50000, 5, 0x70000, 0x80000, 256, None) == 4
    assert run(c, None, sp, 0x50000, 5, 0x70000, 0x80000, need - 1, None) == 4
    # refused for its size, or past that check (here, without a device, by the next)
    assert run(c, None, sp, 0x50000, 8192, 0x70000, 0x80000, 255, None) == 4
    import torch
    if not torch.cuda.is_available():
        assert run(c, None, sp, 0x50000, 8192, 0x70000, 0x80000, 256, None) == 5
