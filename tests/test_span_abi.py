"""Host-side checks of the span attention, eviction and slot appends: bad
arguments are refused before anything is launched (no GPU needed)."""
import ctypes

import pytest

from rope_frequency_chunk_b200 import fasa as F
from tests.test_abi import L, _fake_cache  # noqa: F401  (L: fixture)


def span(**kw):
    d = dict(seq_len=0x90000, q_pos=None, q_len=None, max_seq_len=100, window=0, n_sink=0, q_prerotated=0)
    d.update(kw)
    return ctypes.byref(F.fasa_span(**d))


def paged(**kw):
    d = dict(block_table=0xA0000, block_size=16, max_blocks=64, n_pages=100, reserved=0)
    d.update(kw)
    return ctypes.byref(F.fasa_paged(**d))


BAD_SPANS = [(dict(seq_len=None), 1), (dict(seq_len=0x90002), 1), (dict(q_pos=0x90001), 1), (dict(q_len=0x90003), 1),
             (dict(max_seq_len=0), 1), (dict(max_seq_len=-5), 1), (dict(window=-1), 1), (dict(n_sink=-1), 1),
             (dict(q_prerotated=2), 1), (dict(max_seq_len=1025), 3)]


def test_attend_decode_refusals(L):
    c = ctypes.byref(_fake_cache())
    ws = L.fasa_attend_decode_workspace_bytes
    run = L.fasa_attend_decode
    need = ws(c, span(), 0)
    assert 0 < need < ws(c, span(), 1)
    # a workspace for every length up to the cache's serves each window at it
    whole = ws(c, span(max_seq_len=1024), 1)
    assert all(ws(c, span(max_seq_len=n, window=w, n_sink=k), m) <= whole
               for n in (1, 64, 257, 1000) for w in (0, 1, 300) for k in (0, 70) for m in (0, 1))
    ok = (0x50000, 0x70000, None, 0x80000, need, None)
    for bad, status in BAD_SPANS:
        assert run(c, None, span(**bad), *ok) == status, bad
        assert ws(c, span(**bad), 0) == 0
    assert run(c, None, None, *ok) == 1 and ws(c, None, 0) == 0 and ws(None, span(), 0) == 0
    assert run(None, None, span(), *ok) == 1
    assert run(c, None, span(), 0x50008, 0x70000, None, 0x80000, need, None) == 1      # misaligned q
    assert run(c, None, span(), 0x50000, None, None, 0x80000, need, None) == 1         # no output
    assert run(c, None, span(), 0x50000, 0x70000, 0x60002, 0x80000, need, None) == 1   # misaligned weights
    assert run(c, None, span(), 0x50000, 0x70000, None, None, need, None) == 4
    assert run(c, None, span(), 0x50000, 0x70000, None, 0x80010, need, None) == 4
    assert run(c, None, span(), 0x50000, 0x70000, None, 0x80000, need - 1, None) == 4
    assert run(c, None, span(), 0x50000, 0x70000, 0x60000, 0x80000, need, None) == 4   # weights need more
    for bad in (dict(block_table=None), dict(block_size=24), dict(max_blocks=63), dict(n_pages=0)):
        assert run(c, paged(**bad), span(), *ok) == 1, bad
    assert run(ctypes.byref(_fake_cache(head_dim=64)), None, span(), *ok) == 2


def test_attend_prompt_refusals(L):
    c = ctypes.byref(_fake_cache())
    ws = L.fasa_attend_prompt_workspace_bytes
    run = L.fasa_attend_prompt
    need = ws(c, span(), 7)
    assert need > 0 and ws(c, span(), 0) == 0
    tail = (0x70000, 0x80000, need, None)
    for bad, status in BAD_SPANS:
        assert run(c, None, span(**bad), 0x50000, 7, *tail) == status, bad
    assert run(c, None, span(), 0x50000, 0, *tail) == 1
    assert run(c, None, span(), 0x50000, (1 << 19) + 1, 0x70000, 0x80000, 1 << 60, None) == 2
    assert run(c, None, span(), 0x50004, 7, *tail) == 1
    assert run(c, None, span(), 0x50000, 7, 0x70004, 0x80000, need, None) == 1
    assert run(c, None, span(), 0x50000, 7, 0x70000, 0x80000, need - 1, None) == 4
    assert run(c, None, span(), 0x50000, 7, 0x70000, None, need, None) == 4
    assert run(c, paged(block_size=48), span(), 0x50000, 7, *tail) == 1


def test_evict_refusals(L):
    c = ctypes.byref(_fake_cache())

    def desc(**kw):
        d = dict(seq_len=0x90000, cur_pos=0x91000, max_seq_len=1000, budget=100, n_sink=4, n_recent=10)
        d.update(kw)
        return ctypes.byref(F.fasa_evict_desc(**d))

    ws, run = L.fasa_evict_workspace_bytes, L.fasa_evict
    need = ws(c, desc())
    assert need >= 2 * 2 * 100 * 4
    arr = (0x50000, 0x60000, 0x50000, 0x60000, 0x92000)
    bad = [(dict(seq_len=None), 1), (dict(cur_pos=None), 1), (dict(cur_pos=0x91001), 1), (dict(max_seq_len=0), 1),
           (dict(budget=0), 1), (dict(n_sink=-1), 1), (dict(n_recent=-1), 1), (dict(n_sink=95, n_recent=6), 1),
           (dict(n_recent=2 ** 31 - 1), 1), (dict(max_seq_len=1025), 3)]
    for b, status in bad:
        assert run(c, None, desc(**b), *arr, 0x80000, need, None) == status, b
        assert ws(c, desc(**b)) == 0
    big = ctypes.byref(_fake_cache(max_len=1 << 20))
    assert run(big, None, desc(max_seq_len=(1 << 19) + 1), *arr, 0x80000, 1 << 40, None) == 2
    for i in range(5):
        a = list(arr)
        a[i] = None
        assert run(c, None, desc(), *a, 0x80000, need, None) == 1, i
        a[i] = arr[i] + 2
        assert run(c, None, desc(), *a, 0x80000, need, None) == 1, i
    assert run(c, None, desc(), *arr[:4], 0x90000, 0x80000, need, None) == 1   # len_out is seq_len
    assert run(c, None, desc(), *arr, 0x80000, need - 1, None) == 4
    assert run(c, None, desc(), *arr, None, need, None) == 4
    assert run(c, paged(max_blocks=63), desc(), *arr, 0x80000, need, None) == 1


def test_append_at_refusals(L):
    c = ctypes.byref(_fake_cache())
    run = L.fasa_append_kv_at
    ok = dict(k=0x50000, v=0x60000, n=4, s=0x90000, p=0x91000, sp=None, m=None)

    def call(pg=None, **kw):
        a = dict(ok, **kw)
        return run(c, pg, a["k"], a["v"], a["n"], a["s"], a["p"], a["sp"], a["m"], None)

    assert call(n=0) == 0
    assert call(n=-1) == 1 and call(n=1025) == 3
    assert call(s=None) == 1 and call(p=None) == 1 and call(s=0x90001) == 1 and call(p=0x91002) == 1
    assert call(k=0x50008) == 1 and call(v=None) == 1 and call(sp=0x70001) == 1 and call(m=0x70002) == 1
    assert call(pg=paged(block_size=8)) == 1


def test_binding_checks_its_tensors():
    import torch
    class C:  # the attributes the checks read
        batch, n_q_heads, n_kv_heads, max_len, dtype = 2, 4, 2, 8, torch.bfloat16
    with pytest.raises(TypeError):
        F._per_seq(C, torch.zeros(2, dtype=torch.int32), "seq_len")      # not on the device
    with pytest.raises(TypeError):
        F._per_slot(C, torch.zeros(2, 2, 8), "mass", torch.float32)
    with pytest.raises(TypeError):
        F._span(C, None, 8, 0, 0, None, None, False)
    with pytest.raises(TypeError):
        F._evict_desc(C, None, None, 8, 4, 0, 0)
    with pytest.raises(ValueError):
        F._same(torch.zeros(2, 3), torch.zeros(2, 4))
