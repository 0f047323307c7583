"""Evictions at their edges: pages outside the pool, the largest share of one
CTA, few and many moves."""

import numpy as np
import pytest
import torch

from rope_frequency_chunk_b200 import fasa as F
from tests import span_util as S

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _clean_status():
    F.fasa_device_status(clear=True)
    yield
    assert F.fasa_device_status(clear=True) == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=S.DEV)


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("L,budget,block,lost", [(300, 100, 16, "source"), (300, 100, 16, "target"),
                                                 (300, 100, 16, "both"), (9000, 4400, 64, "source"),
                                                 (9000, 4400, 64, "target")])
def test_moves_of_lost_pages_are_left_out_whole(L, budget, block, lost, inplace):
    """K, V, sketch, weights and positions against the plain form without
    exactly the moves that touch a lost page (few moves in one launch, many in
    two)."""
    hkv = 3
    f = S.Filled([L, L - 7], 2 * hkv, hkv, BF, block)
    c = f.cache
    m = torch.rand(2, hkv, c.max_len, generator=f.g, device=S.DEV)
    pos = torch.stack([torch.stack([torch.randperm(c.max_len, generator=f.g, device=S.DEV) for _ in range(hkv)])
                       for _ in range(2)]).int()
    gone = {"source": [budget // block + 2], "target": [1], "both": [1, 4, budget // block + 2]}[lost]
    for i, blk in enumerate(gone):
        c.block_table[0, blk] = [-1, c.n_pages, 2 ** 31 - 1][i]
    want = [x.clone() for x in (c.k, c.v, c.sketch)]
    mo = m if inplace else torch.full_like(m, 5.0)
    po = pos if inplace else torch.full_like(pos, 5)
    want_m, want_p = mo.clone(), po.clone()
    for b, n in enumerate(f.lens):
        for g in range(hkv):
            src = np.array(S.evict_plain(m[b, g].tolist(), pos[b, g].tolist(), n, n - 1, budget, 4, 20))
            dst = np.arange(len(src))
            if b == 0:
                bad = (src != dst) & (np.isin(src // block, gone) | np.isin(dst // block, gone))
                assert bad.any() and (bad.sum() < (src != dst).sum())
                src = np.where(bad, dst, src)  # a slot whose move is left out keeps its own
            s, d = torch.from_numpy(src).to(S.DEV), torch.from_numpy(dst).to(S.DEV)
            want_m[b, g, :budget], want_p[b, g, :budget] = m[b, g, s], pos[b, g, s]
            mv = s != d
            ps, pd = c.block_table[b, s[mv] // block].long(), c.block_table[b, d[mv] // block].long()
            for w, x in zip(want, (c.k, c.v, c.sketch)):
                w[pd, g, d[mv] % block] = x[ps, g, s[mv] % block]
    n = F.fasa_evict(c, f.seq_len, f.seq_len - 1, m, pos, L, budget, n_sink=4, n_recent=20,
                     mass_out=None if inplace else mo, slot_pos_out=None if inplace else po)
    assert F.fasa_device_status(clear=True) == 7 and n.tolist() == [budget, budget]
    assert torch.equal(mo, want_m) and torch.equal(po, want_p)
    for w, x in zip(want, (c.k, c.v, c.sketch)):
        assert torch.equal(w.nan_to_num(9.0), x.nan_to_num(9.0))


def kept_order(mass, pos, L, cur, budget, n_sink, n_recent):
    """evict_plain, sorted by numpy (long rows)."""
    t = np.arange(L)
    held = (pos[:L] < n_sink) | (pos[:L] > cur - n_recent)
    order = np.lexsort((t, np.where(held, 0.0, -mass[:L].astype(np.float64)), ~held))
    n = min(L, budget)
    kept = np.zeros(L, bool)
    kept[order[:n]] = True
    src = np.arange(n)
    src[~kept[:n]] = t[n:][kept[n:]]
    return src


def test_the_two_plain_forms_agree():
    g = torch.Generator(S.DEV).manual_seed(0)
    for L, budget in ((50, 20), (50, 50), (50, 49), (7, 1)):
        m = torch.randint(0, 4, (L,), generator=g, device=S.DEV).float().cpu().numpy()
        p = torch.randperm(L, generator=g, device=S.DEV).cpu().numpy()
        rest = (L, L - 1, budget, min(2, budget - 1), min(5, budget // 2))
        assert kept_order(m, p, *rest).tolist() == S.evict_plain(m.tolist(), p.tolist(), *rest)


@pytest.mark.parametrize("values", ["heavy", "few", "equal"])
@pytest.mark.parametrize("B,hkv,L", [(25, 3, 32768), (19, 2, 65536), (19, 2, 32801)])
def test_the_largest_share_of_one_block(B, hkv, L, values):
    """Rows enough that a row has as few CTAs as can hold it: one of 32768
    slots, two of 32768 each, two just above one's share."""
    lens = [L - 37 * b for b in range(B)]
    f = S.Filled(lens, hkv, hkv, BF, cap=L, n_dom=1)
    c = f.cache
    if values == "heavy":  # attention weights: most tiny, a few large
        m = torch.rand(B, hkv, L, generator=f.g, device=S.DEV).pow_(30)
    elif values == "few":
        m = torch.randint(0, 3, (B, hkv, L), generator=f.g, device=S.DEV).float()
    else:
        m = torch.full((B, hkv, L), 0.25, device=S.DEV)
    pos = torch.argsort(torch.rand(B, hkv, L, generator=f.g, device=S.DEV), -1).int()
    for budget in (L - 1, L // 2, 1):  # each from the rows that the last one kept
        n_sink, n_recent = min(4, budget - 1), min(200, budget // 2)
        old = [x.clone() for x in (c.k, c.v, c.sketch)]
        m0, p0 = m.clone(), pos.clone()
        n = F.fasa_evict(c, f.seq_len, i32([L - 1] * B), m, pos, L, budget, n_sink=n_sink, n_recent=n_recent)
        mc, pc = m0.cpu().numpy(), p0.cpu().numpy()
        for b in range(B):
            for g in range(hkv):
                src = kept_order(mc[b, g], pc[b, g], f.lens[b], L - 1, budget, n_sink, n_recent)
                s = torch.from_numpy(src).to(S.DEV)
                k = len(src)
                assert torch.equal(m[b, g, :k], m0[b, g, s]) and torch.equal(pos[b, g, :k], p0[b, g, s])
                for x, was in zip((c.k, c.v, c.sketch), old):
                    assert torch.equal(x[b, g, :k], was[b, g, s])
        assert n.tolist() == [min(x, budget) for x in f.lens]
        f.lens, f.seq_len = n.tolist(), n


@pytest.mark.parametrize("B,hkv,L,budget", [(42, 8, 70, 64), (38, 4, 400, 272), (38, 4, 401, 272)])
def test_rows_and_moves_at_the_limits_of_one_launch(B, hkv, L, budget):
    """Few moves of more rows than run at once; 128 and 129 moves a row."""
    lens = [L] * B
    f = S.Filled(lens, hkv, hkv, BF, 16)
    c = f.cache
    m = torch.rand(B, hkv, c.max_len, generator=f.g, device=S.DEV)
    m[:, :, budget:] += 2.0  # every slot behind the budget stays: as many moves as there can be
    pos = torch.argsort(torch.rand(B, hkv, c.max_len, generator=f.g, device=S.DEV), -1).int()
    m0, p0 = m.clone(), pos.clone()
    old = [[f.rows(x, b, L).clone() for x in (c.k, c.v, c.sketch)] for b in range(B)]
    F.fasa_evict(c, f.seq_len, i32([L - 1] * B), m, pos, L, budget)
    for b in range(B):
        for g in range(hkv):
            src = kept_order(m0[b, g].cpu().numpy(), p0[b, g].cpu().numpy(), L, L - 1, budget, 0, 0)
            assert (src >= budget).sum() == L - budget
            s = torch.from_numpy(src).to(S.DEV)
            assert torch.equal(m[b, g, :budget], m0[b, g, s]) and torch.equal(pos[b, g, :budget], p0[b, g, s])
            for x, was in zip((c.k, c.v, c.sketch), old[b]):
                assert torch.equal(f.rows(x, b, budget)[g], was[g, s])


@pytest.mark.parametrize("budget", [8192, 300000])
def test_the_longest_row(budget):
    """524288 slots, sixteen CTAs of 32768 each."""
    L = 1 << 19
    f = S.Filled([L, L - 5], 1, 1, BF, cap=L, n_dom=1)
    c = f.cache
    m = torch.rand(2, 1, L, generator=f.g, device=S.DEV).pow_(20)
    m[1] = (m[1] * 4).floor()  # ties
    pos = torch.argsort(torch.rand(2, 1, L, generator=f.g, device=S.DEV), -1).int()
    old = [x.clone() for x in (c.k, c.v, c.sketch)]
    m0, p0 = m.clone(), pos.clone()
    F.fasa_evict(c, f.seq_len, f.seq_len - 1, m, pos, L, budget, n_sink=4, n_recent=256)
    for b in range(2):
        src = kept_order(m0[b, 0].cpu().numpy(), p0[b, 0].cpu().numpy(), f.lens[b], f.lens[b] - 1, budget, 4, 256)
        s = torch.from_numpy(src).to(S.DEV)
        assert torch.equal(m[b, 0, :budget], m0[b, 0, s]) and torch.equal(pos[b, 0, :budget], p0[b, 0, s])
        for x, was in zip((c.k, c.v, c.sketch), old):
            assert torch.equal(x[b, 0, :budget], was[b, 0, s])
