"""GPU parity of the eviction and the appends to slots, and a serving run of
the operators together: append, prompt, decode with weights, evict, append,
decode again, FASA decode over what is left."""
import math

import pytest
import torch

from rope_frequency_chunk_b200 import fasa as F
from tests import span_util as S

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clean_status():
    F.fasa_device_status(clear=True)
    yield
    assert F.fasa_device_status(clear=True) == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=S.DEV)


def evict_case(lens, budget, n_sink, n_recent, dtype=BF, hkv=2, block=0, inplace=True, values="random", cur=None,
               cap=None, seed=0, n_dom=4):
    f = S.Filled(lens, 2 * hkv, hkv, dtype, block, seed, cap, n_dom)
    c = f.cache
    B, cap = len(lens), c.max_len
    if values == "random":
        m = torch.rand(B, hkv, cap, generator=f.g, device=S.DEV).pow_(6)
    elif values == "few":  # many equal weights, zeros of both signs
        m = torch.randint(0, 3, (B, hkv, cap), generator=f.g, device=S.DEV).float()
        m[:, :, ::7] = -0.0
    else:
        m = torch.full((B, hkv, cap), 0.5, device=S.DEV)
    pos = torch.stack([torch.stack([torch.randperm(cap, generator=f.g, device=S.DEV) for _ in range(hkv)])
                       for _ in range(B)]).int()
    cur = [L - 1 for L in lens] if cur is None else cur
    m0, pos0 = m.clone(), pos.clone()
    old = [[f.rows(x, b, L).clone() for x in (c.k, c.v, c.sketch)] for b, L in enumerate(lens)]
    mo = m if inplace else torch.full_like(m, 5.0)
    po = pos if inplace else torch.full_like(pos, 5)
    n = F.fasa_evict(c, f.seq_len, i32(cur), m, pos, max(lens), budget, n_sink=n_sink, n_recent=n_recent,
                     mass_out=None if inplace else mo, slot_pos_out=None if inplace else po)
    assert n.tolist() == [min(L, budget) for L in lens]
    assert f.seq_len.tolist() == list(lens)
    for b, L in enumerate(lens):
        for g in range(hkv):
            src = S.evict_plain(m0[b, g].tolist(), pos0[b, g].tolist(), L, cur[b], budget, n_sink, n_recent)
            k = len(src)
            assert mo[b, g, :k].tolist() == m0[b, g, src].tolist()
            assert po[b, g, :k].tolist() == pos0[b, g, src].tolist()
            for x, was in zip((c.k, c.v, c.sketch), old[b]):
                assert torch.equal(f.rows(x, b, max(L, 1))[g, :k] if k else was[g, :0], was[g, src])
            tail = slice(k, None)
            assert torch.equal(mo[b, g, tail], m0[b, g, tail] if inplace else torch.full_like(m0[b, g, tail], 5.0))


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("values", ["random", "few", "equal"])
@pytest.mark.parametrize("lens,budget,n_sink,n_recent", [
    ([1], 1, 0, 0), ([2], 1, 0, 0), ([2, 1, 5], 2, 1, 1), ([100, 33, 0], 64, 4, 8), ([544, 512, 513], 512, 4, 64),
    ([1000], 999, 0, 0), ([1000], 1, 1, 0), ([3001, 40], 700, 0, 700), ([777], 300, 300, 0)])
def test_evict_rows(lens, budget, n_sink, n_recent, values, inplace):
    evict_case(lens, budget, n_sink, n_recent, values=values, inplace=inplace)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [0, 16, 64])
@pytest.mark.parametrize("n_dom", [1, 16, 64])
def test_evict_types_pages_sketches(dtype, block, n_dom):
    evict_case([300, 120, 257], 128, 3, 20, dtype, hkv=3, block=block, n_dom=n_dom)


@pytest.mark.parametrize("values", ["random", "few"])
def test_evict_long_rows(values):
    """Rows of several CTAs (a cluster), the largest share of one CTA, and
    budgets above and below half."""
    evict_case([40000], 3001, 4, 512, hkv=1, values=values)
    evict_case([33001, 20000], 30000, 4, 100, hkv=2, values=values, inplace=False)
    evict_case([150001], 140000, 0, 1000, hkv=1, values=values)


def test_evict_many_rows():
    evict_case([200 + b for b in range(60)], 210, 4, 30, hkv=3)


def test_evict_positions():
    evict_case([200, 200], 100, 0, 50, cur=[10 ** 9, -5])    # nobody recent, everybody recent
    evict_case([200], 100, 50, 0, cur=[-2 ** 31])


def test_evict_flags_bad_lengths_and_pages():
    f = S.Filled([100, 60], 4, 2, BF, 16)
    m = torch.rand(2, 2, f.cache.max_len, generator=f.g, device=S.DEV)
    pos = torch.arange(f.cache.max_len, device=S.DEV).int().expand(2, 2, -1).contiguous()
    n = F.fasa_evict(f.cache, i32([101, -1]), i32([99, 59]), m.clone(), pos.clone(), 100, 50)
    assert F.fasa_device_status(clear=True) == 7 and n.tolist() == [50, 0]
    f.cache.block_table[0, 5] = -1
    before = f.cache.k.clone()
    F.fasa_evict(f.cache, f.seq_len, i32([99, 59]), m, pos, 100, 50, n_recent=30)
    assert F.fasa_device_status(clear=True) == 7
    assert f.cache.k.shape == before.shape


def test_evict_in_a_host_resident_cache():
    f = S.Filled([300], 4, 2, BF, cap=320)
    c = F.KVCache(1, 4, 2, 4, 320, BF, S.BASE, [[0, 1, 2, 3], [1, 2, 3, 4]], kv_on_host=True)
    c.k.copy_(f.cache.k), c.v.copy_(f.cache.v), c.sketch.copy_(f.cache.sketch)
    torch.cuda.synchronize()
    m = torch.rand(1, 2, 320, generator=f.g, device=S.DEV)
    pos = torch.arange(320, device=S.DEV).int().expand(1, 2, -1).contiguous()
    m2, pos2 = m.clone(), pos.clone()
    for x, a, b in ((f.cache, m, pos), (c, m2, pos2)):
        F.fasa_evict(x, f.seq_len, i32([299]), a, b, 300, 100, n_sink=4, n_recent=20)
    torch.cuda.synchronize()
    assert torch.equal(m, m2) and torch.equal(pos, pos2)
    for x, y in ((f.cache.k, c.k), (f.cache.v, c.v), (f.cache.sketch, c.sketch)):
        assert torch.equal(x[:, :, :100].cpu(), y[:, :, :100].cpu())


def test_evict_captured_and_replayed():
    f = S.Filled([700, 600], 4, 2, BF, 16)
    c = f.cache
    m = torch.rand(2, 2, c.max_len, generator=f.g, device=S.DEV)
    pos = torch.arange(c.max_len, device=S.DEV).int().expand(2, 2, -1).contiguous()
    k0, mo, po = c.k.clone(), torch.zeros_like(m), torch.zeros_like(pos)
    cur, n = i32([699, 599]), i32([0, 0])
    args = dict(n_sink=4, n_recent=50, mass_out=mo, slot_pos_out=po, len_out=n,
                workspace=F.fasa_evict_workspace(c, 700, 300))
    F.fasa_evict(c, f.seq_len, cur, m, pos, 700, 300, **args)
    ref = [x.clone() for x in (c.k, mo, po, n)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fasa_evict(c, f.seq_len, cur, m, pos, 700, 300, **args)
    for _ in range(2):
        c.k.copy_(k0)
        mo.zero_(), po.zero_(), n.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x.nan_to_num(9.0) if x.is_floating_point() else x,
                               y.nan_to_num(9.0) if y.is_floating_point() else y)
                   for x, y in zip((c.k, mo, po, n), ref))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [0, 16])
def test_append_at(dtype, block):
    """The rows of fasa_append_kv for the positions, in the slots' places."""
    f = S.Filled([200, 200, 200], 4, 2, dtype, block)
    c = f.cache
    n = 13
    kn, vn = S.randn(f.g, 3, 2, n, 128).to(dtype), S.randn(f.g, 3, 2, n, 128).to(dtype)
    slot0, pos0 = [0, 187, 50], [5, 187, 90]
    ref = F.KVCache(3, 4, 2, 4, 400, dtype, S.BASE, [[0, 1, 2, 3], [1, 2, 3, 4]])
    pos = torch.full((3, 2, c.max_len), -7, dtype=torch.int32, device=S.DEV)
    m = torch.ones(3, 2, c.max_len, device=S.DEV)
    old = [c.k.clone(), c.v.clone(), c.sketch.clone()]
    F.fasa_append_kv_at(c, kn, vn, i32(slot0), i32(pos0), slot_pos=pos, mass=m)
    for b in range(3):
        F.fasa_append_kv(ref, kn, vn, pos0[b])
        for new, was, x in ((c.k, old[0], ref.k), (c.v, old[1], ref.v), (c.sketch, old[2], ref.sketch)):
            got, had = f.rows(new, b, 200), f.rows(was, b, 200)
            s = slice(slot0[b], slot0[b] + n)
            assert torch.equal(got[:, s], x[b, :, pos0[b]:pos0[b] + n])
            keep = torch.ones(200, dtype=torch.bool, device=S.DEV)
            keep[s] = False
            assert torch.equal(got[:, keep], had[:, keep])
        want = torch.full((c.max_len,), -7, dtype=torch.int32, device=S.DEV)
        want[s] = torch.arange(pos0[b], pos0[b] + n, dtype=torch.int32, device=S.DEV)
        assert (pos[b] == want).all()
        assert (m[b] == (want < 0).float()).all()


def test_append_at_refuses_ranges():
    f = S.Filled([64, 64, 64], 4, 2, BF, 16)
    kn = S.randn(f.g, 3, 2, 2, 128).to(BF)
    before = f.cache.k.clone()
    F.fasa_append_kv_at(f.cache, kn, kn, i32([63, -1, 0]), i32([5, 5, 2 ** 31 - 2]))
    assert F.fasa_device_status(clear=True) == 7
    assert torch.equal(f.cache.k.nan_to_num(9.0), before.nan_to_num(9.0))


def test_append_behind_a_skipped_sequence():
    """A sequence out of range comes first; the others' angles are theirs."""
    f = S.Filled([64, 64, 64], 4, 2, BF, 16)
    kn, vn = (S.randn(f.g, 3, 2, 3, 128).to(BF) for _ in range(2))
    F.fasa_append_kv_at(f.cache, kn, vn, i32([-1, 0, 7]), i32([5, 0, 0]))
    assert F.fasa_device_status(clear=True) == 7
    ref = F.KVCache(3, 4, 2, 4, 64, BF, S.BASE, [[0, 1, 2, 3], [1, 2, 3, 4]])
    F.fasa_append_kv(ref, kn, vn, 0)
    for b, s0 in ((1, 0), (2, 7)):
        assert torch.equal(f.rows(f.cache.k, b, 64)[:, s0:s0 + 3], ref.k[b, :, :3])
        assert torch.equal(f.rows(f.cache.sketch, b, 64)[:, s0:s0 + 3], ref.sketch[b, :, :3])


@pytest.mark.parametrize("block", [0, 16])
def test_serving_run(block):
    """The operators as a serving loop uses them, checked step by step: a
    prompt, tokens decoded with their weights, evictions back to the budget,
    appends into the freed slots, and a FASA decode over what is left."""
    B, hq, hkv, cap, budget = 2, 8, 2, 272, 96
    g = torch.Generator(S.DEV).manual_seed(3)
    lens = [240, 150]
    f = S.Filled([0] * B, hq, hkv, BF, 0, cap=cap)
    if block:
        c = F.PagedKVCache(B, hq, hkv, 4, B * cap // block, block, cap // block, BF, S.BASE,
                           [[0, 1, 2, 3], [1, 2, 3, 4]])
        c.block_table.copy_(torch.randperm(B * cap // block, generator=torch.Generator().manual_seed(1))
                            .int().reshape(B, -1))
        f.cache, f.block = c, block
    c = f.cache
    mass = torch.zeros(B, hkv, cap, device=S.DEV)
    pos = torch.full((B, hkv, cap), -1, dtype=torch.int32, device=S.DEV)
    k, v = (S.randn(g, B, hkv, 240, 128).to(BF) for _ in range(2))
    F.fasa_append_kv_at(c, k, v, i32([0, 0]), i32([0, 0]), slot_pos=pos, mass=mass)
    f.lens, f.seq_len = list(lens), i32(lens)
    q = (S.randn(g, B, 150, hq, 128) * 1.5).to(BF)
    out = F.fasa_attend_prompt(c, f.seq_len, q, cap, window=64, n_sink=4)
    for b in range(B):
        ref, _, size, z = S.attend64(f, b, q[b], list(range(lens[b] - 150, lens[b])), 64, 4, False)
        S.check_out(out[b], ref, size, z, lens[b], p_rel=2.0 ** -8)
    at = list(lens)  # the next position of every sequence
    for step in range(12):
        q = (S.randn(g, B, hq, 128) * 1.5).to(BF)
        m0 = mass.clone()
        out = F.fasa_attend_decode(c, f.seq_len, q, cap, q_pos=i32(at), mass=mass)
        for b in range(B):
            ref, w, size, z = S.attend64(f, b, q[b:b + 1], [at[b]], 0, 0, False)
            S.check_out(out[b], ref[0], size[0], z, f.lens[b])
            assert (mass[b, :, :f.lens[b]].double() - m0[b, :, :f.lens[b]].double() - w).abs().max() < 1e-3
        kn, vn = (S.randn(g, B, hkv, 1, 128).to(BF) for _ in range(2))
        F.fasa_append_kv_at(c, kn, vn, f.seq_len, i32(at), slot_pos=pos, mass=mass)
        f.seq_len = f.seq_len + 1
        f.lens = [n + 1 for n in f.lens]
        at = [p + 1 for p in at]
        if step % 4 == 3:
            m0, p0 = mass.clone(), pos.clone()
            rows = [[f.rows(x, b, f.lens[b]).clone() for x in (c.k, c.v)] for b in range(B)]
            f.seq_len = F.fasa_evict(c, f.seq_len, i32([p - 1 for p in at]), mass, pos, cap, budget, n_sink=4,
                                     n_recent=16)
            for b in range(B):
                for h in range(hkv):
                    src = S.evict_plain(m0[b, h].tolist(), p0[b, h].tolist(), f.lens[b], at[b] - 1, budget, 4, 16)
                    assert pos[b, h, :len(src)].tolist() == p0[b, h, src].tolist()
                    for x, was in zip((c.k, c.v), rows[b]):
                        assert torch.equal(f.rows(x, b, len(src))[h], was[h, src])
            f.lens = f.seq_len.tolist()
            assert f.lens == [budget] * B
    # FASA over the evicted cache, every slot kept: the dense result
    q = (S.randn(g, B, hq, 128) * 1.5).to(BF)
    a = F.fasa_attend_decode(c, f.seq_len, q, cap, q_prerotated=True)
    if block:
        b = F.fasa_decode_paged(c, f.seq_len, q, cap, budget, q_prerotated=True)
    else:
        b = F.fasa_decode_varlen(c, f.seq_len, q, cap, budget, q_prerotated=True)
    assert (a.double() - b.double()).abs().max() < 0.03 and math.isfinite(float(a.float().sum()))
