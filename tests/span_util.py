"""Plain float64 forms of the span attention and the eviction, and caches
filled for their tests: every slot that no query sees holds NaN."""
import math

import numpy as np
import torch

from rope_frequency_chunk_b200 import fasa as F

BASE = 1e4
DEV = "cuda"


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


class Filled:
    """A cache (contiguous, or paged with `block`) whose slots 0 .. lens[b]-1
    hold random rows and the others NaN; `table` entries behind a sequence's
    last page are out of range."""

    def __init__(self, lens, hq, hkv, dtype, block=0, seed=0, cap=None, n_dom=4):
        g = torch.Generator(DEV).manual_seed(seed)
        self.g, self.lens, self.hq, self.hkv, self.block = g, lens, hq, hkv, block
        B = len(lens)
        cap = cap or max(max(lens), 1)
        dom = [[(i + j) % 64 for j in range(n_dom)] for i in range(hkv)]
        if block:
            blocks = -(-cap // block)
            need = [-(-L // block) for L in lens]
            pages = sum(need) + 2
            perm = np.random.default_rng(seed).permutation(pages)
            table = np.full((B, blocks), pages + 7, np.int32)
            o = 0
            for b, n in enumerate(need):
                table[b, :n] = perm[o:o + n]
                o += n
            self.cache = F.PagedKVCache(B, hq, hkv, n_dom, pages, block, blocks, dtype, BASE, dom)
            self.cache.block_table.copy_(torch.from_numpy(table))
        else:
            self.cache = F.KVCache(B, hq, hkv, n_dom, cap, dtype, BASE, dom)
        c = self.cache
        for x in (c.k, c.v, c.sketch):
            x.fill_(math.nan)
        for b, L in enumerate(lens):
            if L:
                t = torch.arange(L, device=DEV)
                for x in (c.k, c.v, c.sketch):
                    self.put(x, b, t, randn(g, hkv, L, x.shape[-1]).to(x.dtype))
        self.seq_len = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def put(self, pool, b, t, rows):
        """rows [Hkv, n, .] into slots t of sequence b."""
        if self.block:
            pg = self.cache.block_table[b, t // self.block].long()
            pool[pg, :, t % self.block] = rows.transpose(0, 1)
        else:
            pool[b, :, t] = rows

    def rows(self, pool, b, n):
        """Slots 0 .. n-1 of sequence b, [Hkv, n, .]."""
        if self.block:
            t = torch.arange(n, device=DEV)
            pg = self.cache.block_table[b, t // self.block].long()
            return pool[pg, :, t % self.block].transpose(0, 1)
        return pool[b, :, :n]

    def blind(self, see):
        """NaN into slots that see[b] (bool [L]) says nobody sees."""
        for b, s in enumerate(see):
            t = torch.nonzero(~s).flatten()
            if len(t):
                for x in (self.cache.k, self.cache.v):
                    self.put(x, b, t, torch.full((self.hkv, len(t), 128), math.nan, device=DEV).to(x.dtype))


def visible(L, p, window, n_sink):
    """bool [len(p), L]: which slots the queries at positions p see."""
    t, p = torch.arange(L, device=DEV), torch.as_tensor(p, device=DEV).reshape(-1, 1)
    v = t <= p
    if window:
        v &= (t > p - window) | (t < n_sink)
    return v


def rotate64(x, p):
    """x [n, H, 128] float64, rows rotated at positions p [n]."""
    th = BASE ** (-2.0 * torch.arange(64, dtype=torch.float64, device=DEV) / 128)
    a = torch.as_tensor(p, device=DEV).double()[:, None, None] * th
    c, s = a.cos(), a.sin()
    x0, x1 = x[..., :64], x[..., 64:]
    return torch.cat([x0 * c - x1 * s, x1 * c + x0 * s], -1)


def attend64(f, b, q, p, window, n_sink, prerot):
    """The float64 attention of q [n, Hq, 128] at positions p over sequence b
    of a Filled cache: (out [n, Hq, 128], weights summed over heads and
    queries [Hkv, L], sum_t w |v|, the largest sum_d |q_d k_d| / sqrt(128))."""
    L = f.lens[b]
    n, hq = q.shape[0], q.shape[1]
    G = hq // f.hkv
    x = q.double() if prerot else rotate64(q.double(), p)
    out = torch.zeros(n, hq, 128, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(out)
    mass = torch.zeros(f.hkv, L, dtype=torch.float64, device=DEV)
    z_max = 0.0
    if L == 0:
        return out, mass, size, z_max
    see = visible(L, p, window, n_sink)
    k, v = f.rows(f.cache.k, b, L).double(), f.rows(f.cache.v, b, L).double()
    k, v = k.nan_to_num(0.0), v.nan_to_num(0.0)
    for g in range(f.hkv):
        for h in range(g * G, (g + 1) * G):
            z = (x[:, h] @ k[g].T / math.sqrt(128)).masked_fill(~see, -math.inf)
            w = torch.softmax(z, 1).nan_to_num(0.0)
            out[:, h] = w @ v[g]
            size[:, h] = w @ v[g].abs()
            mass[g] += w.sum(0)
            z_max = max(z_max, float((x[:, h].abs() @ k[g].abs().T).max()) / math.sqrt(128))
    return out, mass, size, z_max


def logit_error(dtype, z_max):
    """Bound on a logit's error, natural units: the rotated queries keep 16
    bits in bf16 caches' products (two bf16 terms: 2^-16), float32 sums of 128
    products (2^-17 of the sum of magnitudes), the rotation 2^-20."""
    return z_max * ((2.0 ** -16 if dtype == torch.bfloat16 else 0.0) + 2.0 ** -17 + 2.0 ** -20)


def check_out(got, ref, size, z_max, L, p_rel=2.0 ** -16):
    """got against the float64 result: a weight is off by at most twice the
    logits' error, its own rounding p_rel and the float32 sum over L slots
    (2^-24 each step of the longest chain, at most L / 4 + 64), and the output
    by one rounding to its type (half a step)."""
    dt = got.dtype
    w = 2.0 * logit_error(dt, z_max) + (p_rel if dt == torch.bfloat16 else 0.0) + (L / 4 + 64) * 2.0 ** -24
    e = w * (size + ref.abs())
    tol = e + torch.finfo(dt).eps / 2 * (ref.abs() + e) + 1e-30
    bad = (got.double() - ref).abs() > tol
    assert not bad.any() and torch.isfinite(got).all(), (
        f"{int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - ref).abs() / tol).nan_to_num(1e9).max()):.2f}"
        " of the tolerance")


def evict_plain(mass, pos, L, cur, budget, n_sink, n_recent):
    """(source slot of every kept slot 0 .. n-1) of one row, from the rules."""
    held = [(x < n_sink or x > cur - n_recent) for x in pos[:L]]
    n = min(L, budget)
    order = sorted(range(L), key=lambda t: (0, 0.0, t) if held[t] else (1, -mass[t], t))
    kept = set(order[:n])
    src = list(range(n))
    for dst, s in zip([t for t in range(n) if t not in kept], sorted(t for t in kept if t >= n)):
        src[dst] = s
    return src
