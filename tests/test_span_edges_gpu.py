"""The span attention at its edges: workspaces made for other calls, lost
pages, values that are not finite."""

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


def test_one_prompt_workspace_for_every_chunk():
    """Sized once for the longest chunk, used for shorter ones and windows."""
    f = S.Filled([3000], 8, 2, BF, 16)
    ws = F.fasa_attend_prompt_workspace(f.cache, 1024, 3000)
    for n_q, window in ((1024, 0), (300, 0), (17, 0), (1, 0), (17, 900), (300, 64)):
        q = (S.randn(f.g, 1, n_q, 8, 128) * 1.5).to(BF)
        ws.fill_(255)
        out = F.fasa_attend_prompt(f.cache, f.seq_len, q, 3000, window=window, n_sink=3, workspace=ws)
        ref, _, size, z = S.attend64(f, 0, q[0], list(range(3000 - n_q, 3000)), window, 3, False)
        S.check_out(out[0], ref, size, z, 3000, p_rel=2.0 ** -8)


def not_finite(f, run, n_q, hq):
    """NaN in one query head (of one token), then in the only key that a row
    sees: NaN in exactly the outputs that depend on it."""
    B = len(f.lens)
    q = (S.randn(f.g, B, n_q, hq, 128) * 1.5).to(f.cache.dtype)
    good = run(f.seq_len, q)
    assert torch.isfinite(good).all()
    q[0, n_q // 2, 1, 5] = math.nan
    out = run(f.seq_len, q)
    bad = torch.zeros(B, n_q, hq, dtype=torch.bool, device=S.DEV)
    bad[0, n_q // 2, 1] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], good[~bad])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[40, 7], [1, 3], [900, 300]])
def test_nan_queries_stay_nan_in_the_decode(lens, dtype):
    f = S.Filled(lens, 8, 2, dtype, 16)
    not_finite(f, lambda n, q: F.fasa_attend_decode(f.cache, n, q[:, 0].contiguous(), max(lens))[:, None], 1, 8)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n_q", [1, 9, 600])
def test_nan_queries_stay_nan_in_prompts(n_q, dtype):
    f = S.Filled([700, 650], 8, 2, dtype, 16)
    not_finite(f, lambda n, q: F.fasa_attend_prompt(f.cache, n, q, 700), n_q, 8)


def test_nan_queries_stay_nan_on_host_resident_caches():
    c = F.KVCache(1, 8, 2, 4, 400, BF, S.BASE, [[0, 1, 2, 3]] * 2, kv_on_host=True)
    f = S.Filled([390], 8, 2, BF, cap=400)
    c.k.copy_(f.cache.k)
    c.v.copy_(f.cache.v)
    torch.cuda.synchronize()
    not_finite(f, lambda n, q: F.fasa_attend_decode(c, n, q[:, 0].contiguous(), 400)[:, None], 1, 8)
    not_finite(f, lambda n, q: F.fasa_attend_prompt(c, n, q, 400), 9, 8)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_nan_key_that_is_all_a_row_sees(dtype):
    f = S.Filled([1, 300], 4, 2, dtype, 16)
    f.put(f.cache.k, 0, torch.tensor([0], device=S.DEV), torch.full((2, 1, 128), math.nan, device=S.DEV).to(dtype))
    q = (S.randn(f.g, 2, 4, 128) * 1.5).to(dtype)
    m = torch.zeros(2, 2, f.cache.max_len, device=S.DEV)
    out = F.fasa_attend_decode(f.cache, f.seq_len, q, 300, mass=m)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()
    assert torch.isnan(m[0, :, 0]).all() and torch.isfinite(m[1]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block,gone", [(16, [2]), (16, [8, 9, 10, 11, 12, 13, 14, 15]), (64, [1, 6]), (256, [1]),
                                        (128, [0]), (16, [43])])
@pytest.mark.parametrize("n_q,window", [(1, 0), (40, 0), (640, 0), (300, 260)])
def test_lost_pages_are_left_out_of_prompts(block, gone, n_q, window, dtype):
    """Against float64 over the slots that are left: pages of a part of a block
    of slots, whole blocks, the first and the last page."""
    L = 700
    f = S.Filled([L, 90], 8, 2, dtype, block)
    q = (S.randn(f.g, 2, n_q, 8, 128) * 1.5).to(dtype)
    n = [n_q, min(n_q, 90)]
    keep = torch.ones(L, dtype=torch.bool, device=S.DEV)
    for pg in gone:
        keep[pg * block:(pg + 1) * block] = False
    k, v = f.rows(f.cache.k, 0, L).double(), f.rows(f.cache.v, 0, L).double()
    for i, pg in enumerate(gone):
        f.cache.block_table[0, pg] = [-1, f.cache.n_pages, -2 ** 31, 2 ** 31 - 1][i % 4]
    out = F.fasa_attend_prompt(f.cache, f.seq_len, q, L, window=window, n_sink=3, q_len=torch.tensor(
        n, dtype=torch.int32, device=S.DEV))
    p = torch.arange(L - n_q, L, device=S.DEV)
    see = S.visible(L, p, window, 3)
    # a page that no query sees is not looked up, and so not flagged
    assert F.fasa_device_status(clear=True) == (7 if (see & ~keep).any() else 0)
    see &= keep
    x = S.rotate64(q[0].double(), p)
    ref = torch.zeros(n_q, 8, 128, dtype=torch.float64, device=S.DEV)
    size, z_max = torch.zeros_like(ref), 0.0
    for h in range(8):
        z = (x[:, h] @ k[h // 4].T / math.sqrt(128)).masked_fill(~see, -math.inf)
        w = torch.softmax(z, 1).nan_to_num(0.0)
        ref[:, h], size[:, h] = w @ v[h // 4], w @ v[h // 4].abs()
        z_max = max(z_max, float((x[:, h].abs() @ k[h // 4].abs().T).max()) / math.sqrt(128))
    S.check_out(out[0], ref, size, z_max, L, p_rel=2.0 ** -8)
    r1, _, s1, z1 = S.attend64(f, 1, q[1, :n[1]], list(range(90 - n[1], 90)), window, 3, False)
    S.check_out(out[1, :n[1]], r1, s1, z1, 90, p_rel=2.0 ** -8)


def test_weights_that_are_not_16_byte_aligned():
    f = S.Filled([1000, 260], 8, 2, BF, 16)
    q = (S.randn(f.g, 2, 8, 128) * 1.5).to(BF)
    a = torch.zeros(2, 2, f.cache.max_len, device=S.DEV)
    b = torch.zeros(a.numel() + 1, device=S.DEV)[1:].view_as(a)
    assert b.data_ptr() % 16 == 4
    for m in (a, b):
        F.fasa_attend_decode(f.cache, f.seq_len, q, 1000, window=500, n_sink=3, mass=m)
    assert torch.equal(a, b) and (a.sum(-1) - 4).abs().max() < 1e-3


@pytest.mark.parametrize("n_q", [3, 700])
def test_f32_prompts_on_host_resident_caches(n_q):
    c = F.KVCache(1, 8, 2, 4, 800, F32, S.BASE, [[0, 1, 2, 3]] * 2, kv_on_host=True)
    f = S.Filled([790], 8, 2, F32, cap=800)
    c.k.copy_(f.cache.k)
    c.v.copy_(f.cache.v)
    torch.cuda.synchronize()
    q = S.randn(f.g, 1, n_q, 8, 128) * 1.5
    out = F.fasa_attend_prompt(c, f.seq_len, q, 800, window=300, n_sink=3)
    ref, _, size, z = S.attend64(f, 0, q[0], list(range(790 - n_q, 790)), 300, 3, False)
    S.check_out(out[0], ref, size, z, 790)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("prerot", [False, True])
def test_outputs_may_take_the_queries_place(dtype, prerot):
    """A row's queries are read before its output is written, whichever kernel
    and however many blocks share it."""
    f = S.Filled([3000, 70, 900], 8, 2, dtype, 16)
    for n_q in (0, 1, 5, 60, 400):  # 0: the decode
        q = (S.randn(f.g, 3, n_q, 8, 128) * 1.5 if n_q else S.randn(f.g, 3, 8, 128)).to(dtype)
        call = F.fasa_attend_prompt if n_q else F.fasa_attend_decode
        ref = call(f.cache, f.seq_len, q, 3000, q_prerotated=prerot)
        assert torch.equal(call(f.cache, f.seq_len, q, 3000, q_prerotated=prerot, out=q), ref)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_most_rows(dtype):
    """8191 sequences of 8 KV heads, the largest batch there is: append,
    decode with weights, a prompt, an eviction, against float64."""
    B, hkv, L, n = 8191, 8, 12, 3
    g = torch.Generator(S.DEV).manual_seed(2)
    c = F.KVCache(B, 2 * hkv, hkv, 1, L, dtype, S.BASE, [[i] for i in range(hkv)])
    lens = torch.randint(0, L - n + 1, (B,), generator=g, device=S.DEV).int()
    pos = torch.zeros(B, hkv, L, dtype=torch.int32, device=S.DEV)
    mass = torch.zeros(B, hkv, L, device=S.DEV)
    k, v = (S.randn(g, B, hkv, L - n, 128).to(dtype) for _ in range(2))
    F.fasa_append_kv_at(c, k, v, torch.zeros_like(lens), torch.zeros_like(lens), slot_pos=pos, mass=mass)
    k, v = (S.randn(g, B, hkv, n, 128).to(dtype) for _ in range(2))
    F.fasa_append_kv_at(c, k, v, lens, lens, slot_pos=pos, mass=mass)
    seq_len = lens + n
    q = (S.randn(g, B, 2 * hkv, 128) * 1.5).to(dtype)
    out = F.fasa_attend_decode(c, seq_len, q, L, mass=mass)
    outp = F.fasa_attend_prompt(c, seq_len, q[:, None].contiguous(), L, q_pos=seq_len)
    p = seq_len.double()[:, None, None] * S.BASE ** (-2.0 * torch.arange(64, dtype=torch.float64, device=S.DEV) / 128)
    x0, x1 = q.double().split(64, -1)
    x = torch.cat([x0 * p.cos() - x1 * p.sin(), x1 * p.cos() + x0 * p.sin()], -1).view(B, hkv, 2, 128)
    kk, vv = c.k.double(), c.v.double()
    see = (torch.arange(L, device=S.DEV) < seq_len[:, None])[:, None, None]
    kk, vv = (torch.where(see[:, :, 0, :, None], t, 0.0) for t in (kk, vv))
    z = (x @ kk.transpose(-1, -2) / math.sqrt(128)).masked_fill(~see, -math.inf)
    z_max = float((x.abs() @ kk.abs().transpose(-1, -2)).max()) / math.sqrt(128)
    w = torch.softmax(z, -1)
    ref, size = (w @ vv).view(B, 2 * hkv, 128), (w @ vv.abs()).view(B, 2 * hkv, 128)
    S.check_out(out, ref, size, z_max, L)
    S.check_out(outp[:, 0], ref, size, z_max, L, p_rel=2.0 ** -8)
    want = w.sum(2)
    rel = 2.0 * S.logit_error(dtype, z_max) + (L / 4 + 64) * 2.0 ** -24
    assert ((mass.double() - want).abs() <= rel * want + 2.0 ** -24 * 3).all()
    m0, k0 = mass.clone(), c.k.clone()
    n_new = F.fasa_evict(c, seq_len, seq_len - 1, mass, pos, L, 4, n_recent=1)
    assert torch.equal(n_new, seq_len.clamp(max=4))
    # the kept weights: the newest slot's and the three largest others
    last = (torch.arange(L, device=S.DEV) == seq_len[:, None] - 1)[:, None]
    top = m0.masked_fill(last, -1.0).masked_fill(~see[:, :, 0], -1.0).sort(-1, descending=True).values[..., :3]
    for L0 in (4, 9, 12):  # sequences of these lengths: their multisets of weights
        b = seq_len == L0
        got = mass[b][..., :4].sort(-1).values
        want = torch.cat([top[b], m0[b][..., L0 - 1:L0]], -1).sort(-1).values
        assert b.any() and torch.equal(got, want)
    for i in range(4):  # and their keys went with them
        t = pos[..., i].clamp(min=0).long()
        moved = torch.gather(k0, 2, t[..., None, None].expand(-1, -1, 1, 128))[:, :, 0]
        on = (i < n_new)[:, None].expand(-1, hkv)
        assert torch.equal(c.k[:, :, i][on], moved[on])
