"""Cases of the cache operators beside the FASA decode: attention of one new
token over contiguous and paged caches (with a sliding window and sink tokens,
accumulating the attention weight of every slot), the same attention for
prompts, eviction from a cache by accumulated weight, and appends to slots
that are not their tokens' positions.

With ``own`` false, ``run`` computes each operator with elementary torch
operations in float32 (angles in float64), rounded once at the end; with
``own`` true it makes the library's calls. ``exact`` restates the definitions
in float64.
"""
import math
import random

import torch

own = False

D = 128
BASE = 5e5
N_DOM = 16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a chat's first tokens: one short sequence in 16-token pages
        dict(name="decode short paged", op="decode", batch=1, hq=32, hkv=8, dtype="bf16", max_len=70, min_len=33,
             block=16, window=0, n_sink=0, prerot=False, mass=False),
        # a serving batch of sequences of very different ages, each slot's weight accumulated for a later eviction
        dict(name="decode ragged weights", op="decode", batch=64, hq=32, hkv=8, dtype="bf16", max_len=16384,
             min_len=1, block=64, window=0, n_sink=0, prerot=False, mass=True),
        # windowed layers over full-precision caches
        dict(name="decode window f32", op="decode", batch=16, hq=8, hkv=2, dtype="f32", max_len=16000,
             min_len=3000, block=0, window=2048, n_sink=4, prerot=False, mass=False),
        # dense layers of a long-context batch
        dict(name="decode long paged", op="decode", batch=8, hq=32, hkv=8, dtype="bf16", max_len=65536,
             min_len=40000, block=128, window=0, n_sink=0, prerot=True, mass=False),
        # short questions, two at once, padded to the longer
        dict(name="prompt short", op="prompt", batch=2, hq=32, hkv=8, dtype="bf16", n_q=99, before=0, block=16,
             window=0, n_sink=0, prerot=False, ragged=True),
        # a whole long prompt, causal
        dict(name="prompt causal 8K", op="prompt", batch=1, hq=32, hkv=8, dtype="bf16", n_q=8192, before=0, block=0,
             window=0, n_sink=0, prerot=True, ragged=False),
        # the same through a windowed layer with sinks
        dict(name="prompt window 8K", op="prompt", batch=1, hq=28, hkv=4, dtype="bf16", n_q=8192, before=0, block=64,
             window=1024, n_sink=4, prerot=True, ragged=False),
        # a chunk of four prompts of their own lengths on top of what is cached
        dict(name="prompt chunk ragged", op="prompt", batch=4, hq=32, hkv=8, dtype="bf16", n_q=1024, before=5000,
             block=16, window=2048, n_sink=16, prerot=False, ragged=True),
        # a full cache makes room for the next 32 tokens
        dict(name="evict 32 of 544", op="evict", batch=8, hq=32, hkv=8, dtype="bf16", max_len=544, budget=512,
             block=64, n_sink=4, n_recent=64, ragged=False),
        # a long prompt cut down to its budget
        dict(name="evict 128K to 8K", op="evict", batch=1, hq=32, hkv=8, dtype="bf16", max_len=131072, budget=8192,
             block=0, n_sink=4, n_recent=512, ragged=False),
        # one new token for each of 64 sequences after an eviction
        dict(name="append one each", op="append", batch=64, hq=32, hkv=8, dtype="bf16", n_new=1, max_len=256,
             block=64),
        # a chunk of a prompt behind an evicted prefix
        dict(name="append 4096", op="append", batch=1, hq=32, hkv=8, dtype="bf16", n_new=4096, max_len=8192,
             block=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv = rng.choice([(32, 8), (32, 8), (28, 4), (8, 2), (8, 8), (16, 1), (27, 3)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    block = rng.choice([0, 16, 32, 64, 128, 256])
    op = rng.choice(["decode", "decode", "prompt", "prompt", "evict", "append"])
    if op == "decode":
        batch = _log(rng, 1, 64)
        most = min(65536, (1 << (21 if dtype == "bf16" else 20)) // (batch * hkv))
        max_len = _log(rng, 1, most)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, dtype=dtype, max_len=max_len,
                    min_len=rng.randint(1, max_len), block=block,
                    window=rng.choice([0, _log(rng, 2, max_len + 1)]), n_sink=rng.choice([0, 4, rng.randint(0, 64)]),
                    prerot=rng.random() < 0.5, mass=rng.random() < 0.4)
    if op == "prompt":
        batch = _log(rng, 1, 6)
        # full-precision prompts are small models' work
        n_q = _log(rng, 1, 4096 if dtype == "bf16" else 512)
        before = rng.choice([0, _log(rng, 1, 6000)])
        while batch > 1 and batch * hq * n_q * (n_q + before) > 1 << 30:
            batch -= 1
        if batch * hq * n_q * (n_q + before) > 1 << 30:
            before = 0
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, dtype=dtype, n_q=n_q, before=before, block=block,
                    window=rng.choice([0, _log(rng, 1, n_q + before)]),
                    n_sink=rng.choice([0, 4, rng.randint(0, 64)]), prerot=rng.random() < 0.5,
                    ragged=rng.random() < 0.6)
    if op == "evict":
        batch = _log(rng, 1, 32)
        max_len = _log(rng, 16, min(1 << 19, (1 << 20) // (batch * hkv)))
        budget = rng.randint(max(2, max_len // 20), max_len)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, dtype=dtype, max_len=max_len, budget=budget, block=block,
                    n_sink=rng.randint(0, min(8, budget // 2)), n_recent=rng.randint(0, budget // 2),
                    ragged=rng.random() < 0.5)
    batch = _log(rng, 1, 64)
    n_new = _log(rng, 1, max(1, 4096 // batch))
    return dict(op=op, batch=batch, hq=hq, hkv=hkv, dtype=dtype, n_new=n_new, max_len=n_new + rng.randint(8, 300),
                block=block)


# ------------------------------------------------------- shapes of a case

def _spread(n, lo, hi):
    """n lengths spread over lo .. hi by their logarithm, the largest first."""
    if n == 1 or lo >= hi:
        return [hi] * n
    lens = [hi]
    for i in range(1, n):
        f = (i * 0.6180339887498949) % 1.0
        lens.append(int(round(math.exp(math.log(lo) + f * (math.log(hi) - math.log(lo))))))
    return lens


def _lens(c):
    """Cached tokens of every sequence, and its queries (prompts)."""
    B = c["batch"]
    if c["op"] == "decode":
        return _spread(B, c["min_len"], c["max_len"]), [1] * B
    if c["op"] == "prompt":
        nq = _spread(B, max(1, c["n_q"] // 3), c["n_q"]) if c["ragged"] else [c["n_q"]] * B
        before = [c["before"] // (1 + b) if c["ragged"] else c["before"] for b in range(B)]
        return [n + o for n, o in zip(nq, before)], nq
    if c["op"] == "evict":
        return (_spread(B, max(1, c["budget"] // 2), c["max_len"]) if c["ragged"] else [c["max_len"]] * B), None
    return [c["max_len"]] * B, None


def _n_dom(c):
    return N_DOM


def _stride(c):
    chunks = -(-2 * _n_dom(c) * (4 if c["dtype"] == "f32" else 2) // 16)
    return (1 << (chunks - 1).bit_length()) * 16 // (4 if c["dtype"] == "f32" else 2)


def _visible(L, p, window, n_sink):
    """How many slots t < L with t <= p, t < n_sink or t > p - window."""
    hi = min(L, p + 1)
    lo = max(0, p - window + 1) if window else 0
    return max(0, hi - lo) + max(0, min(n_sink, lo, hi))


def work(case):
    c, es = case, 4 if case["dtype"] == "f32" else 2
    G, row = c["hq"] // c["hkv"], D * es
    lens, nq = _lens(c)
    if c["op"] == "decode":
        vis = sum(_visible(L, L, c["window"], c["n_sink"]) for L in lens)
        b = vis * c["hkv"] * (2 * row + (8 if c["mass"] else 0)) + 2 * c["batch"] * c["hq"] * row
        return {"bytes": b, "flops": 4 * D * c["hq"] * vis}
    if c["op"] == "prompt":
        pairs = sum(_visible(L, L - n + j, c["window"], c["n_sink"]) for L, n in zip(lens, nq) for j in range(n))
        seen = [L if not c["window"] else min(L, n + c["window"] - 1 + c["n_sink"]) for L, n in zip(lens, nq)]
        return {"bytes": sum(seen) * c["hkv"] * 2 * row + 2 * sum(nq) * c["hq"] * row,
                "flops": 4 * D * c["hq"] * pairs}
    if c["op"] == "evict":
        b = 0.0
        for L in lens:
            kept = min(L, c["budget"])
            b += 16 * kept + 8 * (L - kept)  # weights and positions read, the kept ones written
            tail = L - kept
            if tail:  # kept tokens behind the budget move into holes: the recent ones and their share of the rest
                rec = min(c["n_recent"], tail)
                rest = L - c["n_sink"] - c["n_recent"]
                share = (kept - c["n_sink"] - c["n_recent"]) / rest if rest > 0 else 0.0
                b += (rec + (tail - rec) * share) * 2 * (2 * row + _stride(c) * es)
        return {"bytes": b * c["hkv"], "flops": 0}
    n = c["batch"] * c["hkv"] * c["n_new"]
    return {"bytes": n * (4 * row + _stride(c) * es + 8), "flops": 6 * n * D // 2}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    r = random.Random(seed)
    B, hq, hkv, block = c["batch"], c["hq"], c["hkv"], c["block"]
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    lens, nq = _lens(c)
    cap = max(max(lens), c.get("max_len", 0))
    dom = [r.sample(range(D // 2), _n_dom(c)) for _ in range(hkv)]
    s = {"case": dict(c), "lens": lens}
    if block:
        blocks = -(-cap // block)
        need = [-(-L // block) for L in lens]
        pages = sum(need) + 3
        order = list(range(pages))
        r.shuffle(order)
        table, o = [], 0
        for n in need:  # blocks behind a sequence's last keep a spare page
            table.append(order[o:o + n] + [order[-1]] * (blocks - n))
            o += n
        shape, cap = (pages, hkv, block), blocks * block
    else:
        shape = (B, hkv, cap)
    if own:  # the handle that a serving program keeps
        from rope_frequency_chunk_b200 import fasa as F
        if block:
            h = F.PagedKVCache(B, hq, hkv, _n_dom(c), pages, block, blocks, dt, BASE, dom)
        else:
            h = F.KVCache(B, hq, hkv, _n_dom(c), cap, dt, BASE, dom)
        s["cache"], s["k"], s["v"], s["sketch"] = h, h.k, h.v, h.sketch
    else:
        s["k"] = torch.empty(*shape, D, dtype=dt, device=dev)
        s["v"] = torch.empty_like(s["k"])
        s["sketch"] = torch.empty(*shape, _stride(c), dtype=dt, device=dev)
    s["k"].normal_(generator=g)
    s["v"].normal_(generator=g)
    s["sketch"].normal_(generator=g)
    if block:
        t = torch.tensor(table, dtype=torch.int32, device=dev)
        s["table"] = h.block_table.copy_(t) if own else t
    s["cap"], s["dom"] = cap, torch.tensor(dom, device=dev)
    s["len"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if c["op"] in ("decode", "prompt"):
        shape = (B, hq, D) if c["op"] == "decode" else (B, c["n_q"], hq, D)
        s["q"] = (torch.randn(shape, generator=g, device=dev) * 1.5).to(dt)
        s["out"] = torch.zeros(shape, dtype=dt, device=dev)
    if c["op"] == "decode":
        s["mass"] = torch.rand(B, hkv, cap, generator=g, device=dev) if c["mass"] else None
        if own:
            s["ws"] = F.fasa_attend_decode_workspace(h, c["max_len"], mass=c["mass"])
    if c["op"] == "prompt":
        s["q_len"] = torch.tensor(nq, dtype=torch.int32, device=dev) if c["ragged"] else None
        if own:
            s["ws"] = F.fasa_attend_prompt_workspace(h, c["n_q"], max(lens))
    if c["op"] == "evict":
        # accumulated weights of a heavy-tailed law; the slots hold their positions in order, as after a prompt
        s["mass"] = torch.rand(B, hkv, cap, generator=g, device=dev).pow_(8) * 10
        pos = torch.arange(cap, dtype=torch.int32, device=dev).expand(B, hkv, cap)
        s["pos"] = pos.contiguous()
        s["cur"] = s["len"] - 1
        s["mass_out"], s["pos_out"] = torch.zeros_like(s["mass"]), torch.zeros_like(s["pos"])
        s["len_out"] = torch.zeros_like(s["len"])
        if own:
            s["ws"] = F.fasa_evict_workspace(h, c["max_len"], c["budget"])
    if c["op"] == "append":
        n = c["n_new"]
        s["k_new"] = torch.randn(B, hkv, n, D, generator=g, device=dev).to(dt)
        s["v_new"] = torch.randn(B, hkv, n, D, generator=g, device=dev).to(dt)
        s["slot0"] = torch.tensor([r.randint(0, c["max_len"] - n) for _ in range(B)], dtype=torch.int32, device=dev)
        s["pos0"] = s["slot0"] + torch.tensor([r.randint(0, 100000) for _ in range(B)], dtype=torch.int32, device=dev)
        s["pos"] = torch.zeros(B, hkv, cap, dtype=torch.int32, device=dev)
        s["mass"] = torch.ones(B, hkv, cap, device=dev)
    return s


# ------------------------------------------------------------- plain forms

def _theta():
    return BASE ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device="cuda") / D)


def _rotate(x, pos):
    """x [..., H, 128] at positions pos [...], angles in float64."""
    a = pos.double()[..., None, None] * _theta()
    co, si = a.cos().float(), a.sin().float()
    x0, x1 = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([x0 * co - x1 * si, x1 * co + x0 * si], -1)


def _rows(s, pool, n):
    """Slots 0 .. n-1 of a cache plane as [B, Hkv, n, .]."""
    if not s["case"]["block"]:
        return pool[:, :, :n]
    t = torch.arange(n, device="cuda")
    pages = s["table"].long()[:, t // s["case"]["block"]]
    return pool[pages, :, t % s["case"]["block"]].permute(0, 2, 1, 3)


def _attend(s, q, pos, mass):
    """q [B, n, Hq, 128] at positions pos [B, n] over the cached slots."""
    c = s["case"]
    B, n = pos.shape
    hkv, G, L = c["hkv"], c["hq"] // c["hkv"], max(s["lens"])
    q = q.float()
    if not c["prerot"]:
        q = _rotate(q, pos)
    q = q.reshape(B, n, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * G, D)
    t = torch.arange(L, device="cuda")
    p = pos[:, :, None]
    see = (t < s["len"][:, None, None]) & (t <= p)
    if c["window"]:
        see &= (t > p - c["window"]) | (t < c["n_sink"])
    see = see[:, None, :, None].expand(B, 1, n, G, L).reshape(B, 1, n * G, L)
    x = q @ _rows(s, s["k"], L).float().transpose(2, 3)
    x = (x * (1 / math.sqrt(D))).masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = x.sum(-1, keepdim=True)
    total = total.masked_fill(total == 0, 1.0)
    if mass is not None:
        mass[:, :, :L] += (x / total).sum(2)
    o = (x @ _rows(s, s["v"], L).float()) / total
    return o.reshape(B, hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, c["hq"], D).to(s["out"].dtype)


def _put(s, pool, b, g, t, rows):
    """Writes rows to slots t of (b, g) (index tensors of one length)."""
    if s["case"]["block"]:
        pool[s["table"].long()[b, t // s["case"]["block"]], g, t % s["case"]["block"]] = rows
    else:
        pool[b, g, t] = rows


def _get(s, pool, b, g, t):
    if s["case"]["block"]:
        return pool[s["table"].long()[b, t // s["case"]["block"]], g, t % s["case"]["block"]]
    return pool[b, g, t]


def _evict(s):
    c = s["case"]
    L, budget = max(s["lens"]), c["budget"]
    t = torch.arange(L, device="cuda")
    live = (t < s["len"][:, None]).unsqueeze(1)
    mass, pos = s["mass"][:, :, :L], s["pos"][:, :, :L]
    held = (pos < c["n_sink"]) | (pos > (s["cur"] - c["n_recent"])[:, None, None])
    rank = mass.masked_fill(held, math.inf).masked_fill(~live, -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    keep = torch.zeros_like(held).scatter_(-1, order, True) & live
    hole, move = ~keep & live & (t < budget), keep & (t >= budget)
    b, g, src = move.nonzero(as_tuple=True)  # both lists go by (b, g), then by slot, with as many of each
    dst = hole & (hole.cumsum(-1) <= move.sum(-1, keepdim=True))
    dst = dst.nonzero(as_tuple=True)[2]
    for pool in (s["k"], s["v"], s["sketch"]):
        _put(s, pool, b, g, dst, _get(s, pool, b, g, src))
    n = min(L, budget)
    kept = (t[:n] < s["len"][:, None]).unsqueeze(1)
    for x, y in ((s["mass"], s["mass_out"]), (s["pos"], s["pos_out"])):
        x = x.clone()
        x[b, g, dst] = x[b, g, src]
        y[:, :, :n] = torch.where(kept, x[:, :, :n], y[:, :, :n])
    torch.clamp(s["len"], max=budget, out=s["len_out"])


def _append(s):
    c = s["case"]
    B, hkv, n = c["batch"], c["hkv"], c["n_new"]
    i = torch.arange(n, device="cuda")
    pos = s["pos0"].long()[:, None] + i
    k = _rotate(s["k_new"].float().transpose(1, 2), pos).transpose(1, 2).to(s["k"].dtype)
    b, g, j = (x.reshape(-1) for x in torch.meshgrid(torch.arange(B, device="cuda"),
                                                     torch.arange(hkv, device="cuda"), i, indexing="ij"))
    t = s["slot0"].long()[b] + j
    k = k.reshape(-1, D)
    _put(s, s["k"], b, g, t, k)
    _put(s, s["v"], b, g, t, s["v_new"].reshape(-1, D))
    d = s["dom"][g]
    sk = torch.zeros(len(t), _stride(c), dtype=k.dtype, device="cuda")
    sk[:, 0:2 * _n_dom(c):2] = k.gather(1, d)
    sk[:, 1:2 * _n_dom(c):2] = k.gather(1, d + D // 2)
    _put(s, s["sketch"], b, g, t, sk)
    s["pos"][b, g, t] = (s["pos0"].long()[b] + j).int()
    s["mass"][b, g, t] = 0.0


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if own:
        from rope_frequency_chunk_b200 import fasa as F
        h = s["cache"]
    if op == "decode":
        if own:
            F.fasa_attend_decode(h, s["len"], s["q"], c["max_len"], window=c["window"], n_sink=c["n_sink"],
                                 q_prerotated=c["prerot"], mass=s["mass"], out=s["out"], workspace=s["ws"])
        else:
            s["out"] = _attend(s, s["q"][:, None], s["len"][:, None], s["mass"])[:, 0]
        return (s["out"], s["mass"]) if c["mass"] else (s["out"],)
    if op == "prompt":
        if own:
            F.fasa_attend_prompt(h, s["len"], s["q"], max(s["lens"]), window=c["window"], n_sink=c["n_sink"],
                                 q_len=s["q_len"], q_prerotated=c["prerot"], out=s["out"], workspace=s["ws"])
        else:
            n = s["q_len"] if s["q_len"] is not None else torch.full_like(s["len"], c["n_q"])
            j = torch.arange(c["n_q"], device="cuda")
            o = _attend(s, s["q"], (s["len"] - n)[:, None] + j, None)
            s["out"] = torch.where((j < n[:, None])[:, :, None, None], o, s["out"])
        return (s["out"],)
    if op == "evict":
        if own:
            F.fasa_evict(h, s["len"], s["cur"], s["mass"], s["pos"], c["max_len"], c["budget"], n_sink=c["n_sink"],
                         n_recent=c["n_recent"], mass_out=s["mass_out"], slot_pos_out=s["pos_out"],
                         len_out=s["len_out"], workspace=s["ws"])
        else:
            _evict(s)
        return s["k"], s["v"], s["sketch"], s["mass_out"], s["pos_out"], s["len_out"]
    if own:
        F.fasa_append_kv_at(h, s["k_new"], s["v_new"], s["slot0"], s["pos0"], slot_pos=s["pos"], mass=s["mass"])
    else:
        _append(s)
    return s["k"], s["v"], s["sketch"], s["pos"], s["mass"]


# ------------------------------------------------------------- definitions

def _plane(s, pool, b, g, n):
    """Slots 0 .. n-1 of (b, g)."""
    bs = s["case"]["block"]
    if not bs:
        return pool[b, g, :n]
    return torch.cat([pool[int(p), g] for p in s["table"][b, :-(-n // bs)].tolist()])[:n]


def _turn(x, pos):
    """Rows x [n, 128] as complex pairs, each turned by its position's angles."""
    f = torch.tensor([BASE ** (-i / (D // 2)) for i in range(D // 2)], dtype=torch.float64, device=x.device)
    a = pos.double()[:, None] * f
    z = torch.complex(x[:, :D // 2], x[:, D // 2:]) * torch.polar(torch.ones_like(a), a)
    return torch.cat([z.real, z.imag], 1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    B, hq, hkv = c["batch"], c["hq"], c["hkv"]
    G = hq // hkv
    lens, nq = _lens(c)
    if c["op"] in ("decode", "prompt"):
        one = c["op"] == "decode"
        q = s["q"][:, None] if one else s["q"]
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        mass = s["mass"].double() if one and c["mass"] else None
        for b in range(B):
            L = lens[b]
            first = L if one else L - nq[b]
            slot = torch.arange(L, device="cuda")
            for g in range(hkv):
                k, v = _plane(s, s["k"], b, g, L).double(), _plane(s, s["v"], b, g, L).double()
                for h in range(g * G, (g + 1) * G):
                    p = first + torch.arange(nq[b], device="cuda")
                    x = q[b, :nq[b], h].double()
                    if not c["prerot"]:
                        x = _turn(x, p)
                    w = (x @ k.T).div_(math.sqrt(D))
                    far = slot[None, :] - p[:, None]  # how far behind its query a slot lies, negated
                    out_of_sight = far > 0
                    if c["window"]:
                        out_of_sight |= (far <= -c["window"]) & (slot >= c["n_sink"])
                    w[out_of_sight] = -math.inf
                    w = torch.softmax(w, 1).nan_to_num_(0.0)
                    out[b, :nq[b], h] = w @ v
                    if mass is not None:
                        mass[b, g, :L] += w[0]
        out = out[:, 0] if one else out
        return (out, mass) if mass is not None else (out,)
    if c["op"] == "evict":
        k, v, sk, mo, po = (s[n].clone() for n in ("k", "v", "sketch", "mass_out", "pos_out"))
        mass, pos = s["mass"].cpu().numpy(), s["pos"].cpu().numpy()
        if B * hkv * max(lens) > 1 << 21:
            return None
        for b in range(B):
            L, budget = lens[b], min(lens[b], c["budget"])
            for g in range(hkv):
                m, p = mass[b, g, :L].tolist(), pos[b, g, :L].tolist()
                cur = L - 1
                safe = [x < c["n_sink"] or x > cur - c["n_recent"] for x in p]
                best = sorted(range(L), key=lambda t: (not safe[t], 0.0 if safe[t] else -m[t], t))[:budget]
                kept = set(best)
                moves = list(zip([t for t in range(budget) if t not in kept], sorted(t for t in best if t >= budget)))
                frm = list(range(budget))
                for dst, src in moves:
                    frm[dst] = src
                mo[b, g, :budget] = s["mass"][b, g, frm]
                po[b, g, :budget] = s["pos"][b, g, frm]
                if moves:
                    dst, src = (torch.tensor(x, device="cuda") for x in zip(*moves))
                    for pool, old in ((k, s["k"]), (v, s["v"]), (sk, s["sketch"])):
                        _put(s, pool, torch.full_like(dst, b), torch.full_like(dst, g), dst,
                             _plane(s, old, b, g, L)[src])
        return k, v, sk, mo, po, s["len"].clamp(max=c["budget"])
    k, v, sk, po, mo = (s[n].double() if n in ("k", "v", "sketch") else s[n].clone()
                        for n in ("k", "v", "sketch", "pos", "mass"))
    n = c["n_new"]
    for b in range(B):
        t0, p0 = int(s["slot0"][b]), int(s["pos0"][b])
        t = torch.arange(t0, t0 + n, device="cuda")
        for g in range(hkv):
            at = torch.full_like(t, b), torch.full_like(t, g), t
            x = _turn(s["k_new"][b, g].double(), p0 + torch.arange(n, device="cuda"))
            _put(s, k, *at, x)
            _put(s, v, *at, s["v_new"][b, g].double())
            y = torch.zeros(n, _stride(c), dtype=torch.float64, device="cuda")
            for i, d in enumerate(s["dom"][g].tolist()):
                y[:, 2 * i], y[:, 2 * i + 1] = x[:, d], x[:, d + D // 2]
            _put(s, sk, *at, y)
            po[b, g, t0:t0 + n] = p0 + torch.arange(n, dtype=torch.int32, device="cuda")
            mo[b, g, t0:t0 + n] = 0.0
    return k, v, sk, po, mo
