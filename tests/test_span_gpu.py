"""GPU parity of the span attention (fasa_attend_decode, fasa_attend_prompt)
against float64, over lengths, windows, sinks, head groups, types and page
sizes, with NaN in every slot that no query sees."""
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


def decode_case(lens, hq, hkv, dtype, window=0, n_sink=0, block=0, prerot=False, mass=True, q_pos=None, seed=0,
                cap=None, max_len=None):
    f = S.Filled(lens, hq, hkv, dtype, block, seed, cap)
    pos = lens if q_pos is None else q_pos
    f.blind([S.visible(L, [p], window, n_sink)[0] for L, p in zip(lens, pos)])
    q = (S.randn(f.g, len(lens), hq, 128) * 1.5).to(dtype)
    m0 = torch.rand(len(lens), hkv, f.cache.max_len, generator=f.g, device=S.DEV)
    m = m0.clone() if mass else None
    out = torch.full_like(q, math.nan)
    F.fasa_attend_decode(f.cache, f.seq_len, q, max_len or max(max(lens), 1), window=window, n_sink=n_sink,
                         q_pos=None if q_pos is None else i32(q_pos), q_prerotated=prerot, mass=m, out=out)
    check_decode(f, q, out, m, m0, pos, window, n_sink, prerot)
    return f, q, out, m


def check_decode(f, q, out, m, m0, pos, window, n_sink, prerot):
    for b, L in enumerate(f.lens):
        ref, w, size, z = S.attend64(f, b, q[b:b + 1], [pos[b]], window, n_sink, prerot)
        S.check_out(out[b], ref[0], size[0], z, L)
        if m is not None:
            G = f.hq // f.hkv
            rel = 2.0 * S.logit_error(f.cache.dtype, z) + (L / 4 + 64) * 2.0 ** -24
            got, was = m[b, :, :L].double(), m0[b, :, :L].double()
            tol = rel * w + 2.0 ** -24 * (was + G + 1)
            assert ((got - was - w).abs() <= tol).all()
            assert torch.equal(m[b, :, L:], m0[b, :, L:])
            see = S.visible(L, [pos[b]], window, n_sink)[0]
            assert torch.equal(m[b, :, :L][:, ~see], m0[b, :, :L][:, ~see])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [0, 16, 128])
@pytest.mark.parametrize("lens", [[1], [0], [33, 0, 70], [256, 255, 1], [257], [2049, 1, 0, 640, 5], [4100, 4099]])
def test_decode_lengths(lens, block, dtype):
    decode_case(lens, 8, 2, dtype, block=block)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (9, 3), (7, 1), (8, 1), (9, 1), (16, 1), (32, 2), (28, 4)])
def test_decode_head_groups(hq, hkv, dtype):
    decode_case([530, 17], hq, hkv, dtype, block=32)
    decode_case([90, 1], hq, hkv, dtype, mass=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 4), (2, 0), (64, 4), (65, 64), (100, 130), (700, 3),
                                           (5000, 4), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_decode_windows(window, n_sink, dtype):
    decode_case([1500, 3, 0, 64, 777], 8, 2, dtype, window, n_sink, block=16)
    decode_case([1500, 3, 129], 8, 2, dtype, window, n_sink, mass=False)


def test_decode_positions():
    # behind, inside and before the cached slots; a negative one sees nothing
    decode_case([300, 300, 300, 300, 300], 8, 2, BF, 0, 0, 16, q_pos=[10 ** 9, 299, 120, 0, -1])
    decode_case([300, 300, 300, 300, 300], 8, 2, F32, 50, 4, 0, q_pos=[320, 299, 120, 0, -7])
    decode_case([300], 8, 2, BF, 40, 8, 0, q_pos=[2 ** 31 - 1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_prerotated_and_many_rows(dtype):
    decode_case([5 * b % 97 for b in range(150)], 8, 2, dtype, block=16, prerot=True)
    decode_case([3 * b % 401 for b in range(150)], 4, 1, dtype, prerot=True, window=100, n_sink=2)


def test_decode_long_row_is_split_and_joined():
    decode_case([70001], 8, 1, BF, cap=70016)
    decode_case([30011, 12], 4, 1, F32, block=256)
    decode_case([40000, 7], 8, 2, BF, window=20000, n_sink=300, block=64)


def test_decode_large_and_equal_logits():
    """Logits of thousands (one slot takes all) and all equal (a plain mean)."""
    f = S.Filled([700], 4, 2, BF, 0)
    q = (S.randn(f.g, 1, 4, 128) * 400).to(BF)
    out = F.fasa_attend_decode(f.cache, f.seq_len, q, 700, q_prerotated=True)
    ref, _, size, z = S.attend64(f, 0, q, [700], 0, 0, True)
    S.check_out(out[0], ref[0], size[0], z, 700)
    out = F.fasa_attend_decode(f.cache, f.seq_len, torch.zeros_like(q), 700)
    ref, _, size, z = S.attend64(f, 0, torch.zeros_like(q), [700], 0, 0, True)
    S.check_out(out[0], ref[0], size[0], z, 700)


def test_decode_offsets_past_32_bits():
    """Planes whose last rows lie behind 2^31 elements (and 2^32 bytes)."""
    for block in (0, 4096):
        f = S.Filled([5, 900], 8, 8, BF, 0, cap=1 << 20) if not block else None
        if block:  # a pool of which the sequences use the last pages
            hkv, n = 8, 520
            f = S.Filled([5, 900], 8, hkv, BF, block, cap=4096)
            c = F.PagedKVCache(2, 8, hkv, 4, n, block, 1, BF, S.BASE, [list(range(4))] * hkv)
            c.block_table.copy_(i32([[n - 1], [n - 2]]))
            for x, y in ((c.k, f.cache.k), (c.v, f.cache.v)):
                x[n - 1], x[n - 2] = y[f.cache.block_table[0, 0]], y[f.cache.block_table[1, 0]]
            f.cache = c
            assert c.k.numel() > 2 ** 31
        else:
            assert f.cache.k.numel() >= 2 ** 31
        q = (S.randn(f.g, 2, 8, 128) * 1.5).to(BF)
        m0 = torch.zeros(2, 8, f.cache.max_len, device=S.DEV)
        m = m0.clone()
        out = F.fasa_attend_decode(f.cache, f.seq_len, q, 1000, mass=m)
        check_decode(f, q, out, m, m0, f.lens, 0, 0, False)
        qp = (S.randn(f.g, 2, 3, 8, 128) * 1.5).to(BF)
        outp = F.fasa_attend_prompt(f.cache, f.seq_len, qp, 1000)
        for b in range(2):
            p = [f.lens[b] - 3 + j for j in range(3)]
            ref, _, size, z = S.attend64(f, b, qp[b], p, 0, 0, False)
            S.check_out(outp[b], ref, size, z, f.lens[b], p_rel=2.0 ** -8)
        del f, m, m0
        torch.cuda.empty_cache()


def test_clamped_lengths_and_bad_pages_are_flagged():
    f = S.Filled([40, 100], 4, 2, BF, 16)
    q = (S.randn(f.g, 2, 4, 128)).to(BF)
    good = F.fasa_attend_decode(f.cache, f.seq_len, q, 100)
    over = F.fasa_attend_decode(f.cache, i32([40, 1000]), q, 100)
    assert F.fasa_device_status(clear=True) == 7 and torch.equal(over, good)
    none = F.fasa_attend_decode(f.cache, i32([40, -3]), q, 100)
    assert F.fasa_device_status(clear=True) == 7
    assert torch.equal(none[0], good[0]) and (none[1] == 0).all()
    # a lost page's slots are left out: the rest of the sequence stays
    m = torch.zeros(2, 2, f.cache.max_len, device=S.DEV)
    f.cache.block_table[1, 2] = 1 << 20
    lost = F.fasa_attend_decode(f.cache, f.seq_len, q, 100, mass=m)
    assert F.fasa_device_status(clear=True) == 7 and torch.equal(lost[0], good[0])
    keep = torch.ones(100, dtype=torch.bool, device=S.DEV)
    keep[32:48] = False
    pg = f.cache.block_table[1, torch.arange(100, device=S.DEV) // 16].long()
    pg[32:48] = 0
    k = f.cache.k[pg, :, torch.arange(100, device=S.DEV) % 16].transpose(0, 1).double()[:, keep]
    v = f.cache.v[pg, :, torch.arange(100, device=S.DEV) % 16].transpose(0, 1).double()[:, keep]
    x = S.rotate64(q[1:].double(), [100])[0]
    for h in range(4):
        w = torch.softmax(k[h // 2] @ x[h] / math.sqrt(128), 0)
        assert (lost[1, h].double() - w @ v[h // 2]).abs().max() < 0.02
    assert (m[1, :, 32:48] == 0).all() and (m[1].sum(1) - 2.0).abs().max() < 1e-3
    qp = S.randn(f.g, 2, 5, 4, 128).to(BF)
    o = F.fasa_attend_prompt(f.cache, f.seq_len, qp, 100)
    assert F.fasa_device_status(clear=True) == 7 and torch.isfinite(o).all()


def test_pages_behind_the_window_may_be_gone():
    """Pages that hold only unseen slots need not exist (a windowed layer frees
    them): their entries are neither used nor flagged."""
    for bs, L, w in ((16, 900, 200), (64, 900, 200), (256, 1500, 300)):
        f = S.Filled([L], 8, 2, BF, bs)
        q = (S.randn(f.g, 1, 40, 8, 128) * 1.5).to(BF)
        a = F.fasa_attend_decode(f.cache, f.seq_len, q[:, 0].contiguous(), L, window=w, n_sink=4)
        b = F.fasa_attend_prompt(f.cache, f.seq_len, q, L, window=w, n_sink=4)
        last = (L - 40 - w + 1) // bs  # first page that a query's window reaches
        f.cache.block_table[0, 1:last] = -1
        assert torch.equal(F.fasa_attend_decode(f.cache, f.seq_len, q[:, 0].contiguous(), L, window=w, n_sink=4), a)
        assert torch.equal(F.fasa_attend_prompt(f.cache, f.seq_len, q, L, window=w, n_sink=4), b)
        assert F.fasa_device_status(clear=True) == 0


def test_captured_replayed_streams_and_out_of_order_workspaces():
    f = S.Filled([1200, 333], 8, 2, BF, 16)
    q = (S.randn(f.g, 2, 8, 128) * 1.5).to(BF)
    ref = F.fasa_attend_decode(f.cache, f.seq_len, q, 1200)
    ws = F.fasa_attend_decode_workspace(f.cache, 1200, mass=True)
    ws.fill_(255)  # nothing in it is read before it is written
    m = torch.zeros(2, 2, f.cache.max_len, device=S.DEV)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fasa_attend_decode(f.cache, f.seq_len, q, 1200, mass=m, out=out, workspace=ws)
        F.fasa_attend_decode(f.cache, f.seq_len, q, 1200, mass=m, out=out, workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    assert (m.sum(-1) - 6 * 4).abs().max() < 1e-3  # six calls, four heads a group, weights of one head sum to 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for st in (side, None) * 3:  # two streams, a workspace each
        outs.append(F.fasa_attend_decode(f.cache, f.seq_len, q, 1200, stream=st,
                                         workspace=F.fasa_attend_decode_workspace(f.cache, 1200)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_decode_on_host_resident_caches():
    c = F.KVCache(1, 8, 2, 4, 400, BF, S.BASE, [[0, 1, 2, 3]] * 2, kv_on_host=True)
    f = S.Filled([390], 8, 2, BF, cap=400)
    c.k.copy_(f.cache.k)
    c.v.copy_(f.cache.v)
    torch.cuda.synchronize()
    q = (S.randn(f.g, 1, 8, 128) * 1.5).to(BF)
    out = F.fasa_attend_decode(c, f.seq_len, q, 400)
    ref, _, size, z = S.attend64(f, 0, q, [390], 0, 0, False)
    S.check_out(out[0], ref[0], size[0], z, 390)
    qp = (S.randn(f.g, 1, 9, 8, 128) * 1.5).to(BF)
    out = F.fasa_attend_prompt(c, f.seq_len, qp, 400, window=50, n_sink=3)
    ref, _, size, z = S.attend64(f, 0, qp[0], list(range(381, 390)), 50, 3, False)
    S.check_out(out[0], ref, size, z, 390, p_rel=2.0 ** -8)


# ----------------------------------------------------------------- prompts

def prompt_case(lens, nq, hq, hkv, dtype, window=0, n_sink=0, block=0, prerot=False, q_pos=None, seed=0, n_q=None,
                cap=None, scale=1.5):
    f = S.Filled(lens, hq, hkv, dtype, block, seed, cap)
    B, n_q = len(lens), n_q or max(nq)
    first = [L - n for L, n in zip(lens, nq)] if q_pos is None else q_pos
    # slots that none of a sequence's queries sees
    f.blind([S.visible(L, [p + j for j in range(n)], window, n_sink).any(0) if n else
             torch.zeros(L, dtype=torch.bool, device=S.DEV) for L, p, n in zip(lens, first, nq)])
    q = (S.randn(f.g, B, n_q, hq, 128) * scale).to(dtype)
    for b in range(B):
        q[b, nq[b]:] = math.nan
    out = torch.full_like(q, 7.0)
    F.fasa_attend_prompt(f.cache, f.seq_len, q, max(max(lens), 1), window=window, n_sink=n_sink,
                         q_pos=None if q_pos is None else i32(q_pos),
                         q_len=None if all(n == n_q for n in nq) else i32(nq), q_prerotated=prerot, out=out)
    for b in range(B):
        assert (out[b, nq[b]:] == 7.0).all()  # rows behind a sequence's queries stay
        if nq[b]:
            p = [first[b] + j for j in range(nq[b])]
            ref, _, size, z = S.attend64(f, b, q[b, :nq[b]], p, window, n_sink, prerot)
            S.check_out(out[b, :nq[b]], ref, size, z, lens[b], p_rel=2.0 ** -8)
    return f, q, out


@pytest.mark.parametrize("prerot", [False, True])
@pytest.mark.parametrize("block", [0, 16, 64, 256])
@pytest.mark.parametrize("lens,nq", [([1], [1]), ([130], [130]), ([64, 0, 7], [3, 0, 7]), ([257, 300], [257, 1]),
                                     ([1000, 512], [129, 64]), ([700], [700])])
def test_prompt_lengths(lens, nq, block, prerot):
    prompt_case(lens, nq, 8, 2, BF, block=block, prerot=prerot)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (9, 3), (5, 1), (7, 1), (8, 1), (9, 1), (16, 1), (28, 4)])
def test_prompt_head_groups(hq, hkv):
    prompt_case([300, 77], [150, 77], hq, hkv, BF, block=32)
    prompt_case([200], [200], hq, hkv, BF, window=40, n_sink=5, prerot=True)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 4), (3, 0), (64, 4), (127, 128), (128, 129), (300, 3),
                                           (5000, 4), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_prompt_windows(window, n_sink):
    prompt_case([900, 70, 0], [900, 20, 0], 8, 2, BF, window, n_sink, block=16)
    prompt_case([1500], [333], 4, 1, BF, window, n_sink, prerot=True)


def test_prompt_positions():
    # positions before the cached end (later slots are not seen), behind it, and before the start
    prompt_case([400] * 5, [50] * 5, 8, 2, BF, 0, 0, 16, q_pos=[0, 100, 390, 5000, -25])
    prompt_case([400] * 4, [50] * 4, 8, 2, BF, 60, 4, 0, q_pos=[0, 100, 390, -25])
    prompt_case([400], [50], 8, 2, BF, 60, 4, 0, q_pos=[2 ** 31 - 50])
    prompt_case([5, 20], [9, 20], 8, 2, BF)  # more queries than slots: the first have nothing to see


def test_prompt_few_queries_long_cache():
    prompt_case([20000, 300], [4, 2], 8, 1, BF, block=64)
    prompt_case([33000], [17], 8, 2, BF, prerot=True)
    prompt_case([20000], [40], 8, 2, BF, window=9000, n_sink=100)


def test_prompt_long():
    prompt_case([2900], [2900], 8, 1, BF, block=64)
    prompt_case([2900], [2900], 8, 1, BF, window=512, n_sink=4, prerot=True)


def test_prompt_large_logits():
    prompt_case([600], [600], 4, 2, BF, prerot=True, scale=300.0)


@pytest.mark.parametrize("lens,nq,window", [([1], [1], 0), ([130, 5, 0], [130, 2, 0], 0), ([300], [77], 50)])
def test_prompt_f32(lens, nq, window):
    prompt_case(lens, nq, 8, 2, F32, window=window, n_sink=3, block=16)
    prompt_case(lens, nq, 3, 1, F32, window=window, n_sink=3)


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (9, 3), (8, 2), (10, 2)])
def test_prompt_f32_tokens_sharing_a_block(hq, hkv):
    """Enough tokens that up to eight share a CTA; windows end between them."""
    prompt_case([900, 300], [900, 77], hq, hkv, F32, window=37, n_sink=5, block=32)
    prompt_case([1300], [1201], hq, hkv, F32)
    prompt_case([700], [700], hq, hkv, F32, q_pos=[-9], window=64, n_sink=3, prerot=True)


@pytest.mark.parametrize("hq,hkv,nq", [(2, 2, 900), (1, 1, 1200), (6, 2, 590), (16, 1, 200), (16, 1, 250), (14, 2, 300),
                                       (32, 2, 130)])
def test_prompt_f32_few_and_many_rows(hq, hkv, nq):
    """Query rows below and above one tile's worth per SM; lengths inside a page, ragged batches, a row of none."""
    prompt_case([nq + 33, 0, 40], [nq, 5, 40], hq, hkv, F32, window=0, block=16)
    prompt_case([nq + 33], [nq], hq, hkv, F32, window=70, n_sink=130, block=64)
    prompt_case([nq], [nq], hq, hkv, F32, q_pos=[150], window=100, n_sink=3)


def test_prompt_one_query_is_the_decode():
    f = S.Filled([900, 65], 8, 2, BF, 16)
    q = (S.randn(f.g, 2, 8, 128) * 1.5).to(BF)
    a = F.fasa_attend_decode(f.cache, f.seq_len, q, 900, window=300, n_sink=4, q_pos=f.seq_len)
    b = F.fasa_attend_prompt(f.cache, f.seq_len, q[:, None], 900, window=300, n_sink=4, q_pos=f.seq_len)[:, 0]
    assert (a.double() - b.double()).abs().max() < 0.02


def test_prompt_captured_and_replayed():
    f = S.Filled([1500, 800], 8, 2, BF, 64)
    for nq in (600, 5):
        q = (S.randn(f.g, 2, nq, 8, 128) * 1.5).to(BF)
        ref = F.fasa_attend_prompt(f.cache, f.seq_len, q, 1500)
        ws = F.fasa_attend_prompt_workspace(f.cache, nq, 1500)
        ws.fill_(255)
        out = torch.empty_like(q)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            F.fasa_attend_prompt(f.cache, f.seq_len, q, 1500, out=out, workspace=ws)
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
