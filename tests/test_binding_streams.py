"""Which stream the binding's own tensors (scratch, outputs) belong to: the
one that the call launches on. Checked on the CPU with a stand-in for the
library and for torch's streams."""
import contextlib

import pytest
import torch

from rope_frequency_chunk_b200 import fasa as F

BF = torch.bfloat16
B, HQ, HKV, N = 2, 4, 2, 64


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class FakeLib:
    """Every call succeeds; sizes are 4096 bytes."""

    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("_bytes") else 0


class Cache:
    batch, n_q_heads, n_kv_heads, max_len, dtype = B, HQ, HKV, N, BF
    k = sketch = torch.zeros(1)

    def ref(self):
        return None

    pref = ref


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def q(*shape):
    return torch.zeros(*shape, 128, dtype=BF)


def win():
    return q(B, 1, HQ)


C = Cache()
PLANES = torch.zeros(B, HKV, 1, F.CAL_PLANES, N)
CALLS = {
    "attend_decode": lambda s: F.fasa_attend_decode(C, i32(B), q(B, HQ), N, stream=s),
    "attend_decode_mass": lambda s: F.fasa_attend_decode(C, i32(B), q(B, HQ), N, mass=torch.zeros(B, HKV, N), stream=s),
    "attend_prompt": lambda s: F.fasa_attend_prompt(C, i32(B), q(B, 3, HQ), N, stream=s),
    "evict": lambda s: F.fasa_evict(C, i32(B), i32(B), torch.zeros(B, HKV, N), i32(B, HKV, N), N, 8, stream=s),
    "score": lambda s: F.fasa_score(C, N, q(B, HQ), 0, stream=s),
    "select_topk": lambda s: F.fasa_select_topk(torch.zeros(B, HKV, N), 4, stream=s),
    "sparse_attend": lambda s: F.fasa_sparse_attend(C, N, q(B, HQ), 0, i32(B, HKV, 4), stream=s),
    "decode": lambda s: F.fasa_decode(C, N, q(B, HQ), 0, 4, stream=s),
    "decode_varlen": lambda s: F.fasa_decode_varlen(C, i32(B), q(B, HQ), N, 4, stream=s),
    "decode_paged": lambda s: F.fasa_decode_paged(C, i32(B), q(B, HQ), N, 4, stream=s),
    "decode_multi": lambda s: F.fasa_decode_multi(C, N, q(B, 2, HQ), 0, 4, stream=s),
    "dense_decode": lambda s: F.fasa_dense_decode(C, N, q(B, HQ), 0, stream=s),
    "calibrate_scores": lambda s: F.fasa_calibrate_scores(C, N, win(), 0, stream=s),
    "calibrate_counts": lambda s: F.fasa_calibrate_counts(PLANES, HKV, 4, stream=s),
    "calibrate_dominant": lambda s: F.fasa_calibrate_dominant(i32(HKV, 64), 4, stream=s),
    "calibrate": lambda s: F.fasa_calibrate(C, N, win(), 0, 4, 4, stream=s),
}


@pytest.fixture
def made(monkeypatch):
    """The (stream, shape) of every tensor that a call makes; the current
    stream is 7 outside torch.cuda.stream."""
    now, made, kept = [7], [], []

    @contextlib.contextmanager
    def use(stream):
        now.append(stream.cuda_stream)
        yield
        now.pop()

    def spy(f):
        def g(*a, **kw):
            made.append((now[-1], f.__name__))
            return f(*a, **kw)
        return g

    monkeypatch.setattr(F, "_lib", FakeLib())
    monkeypatch.setattr(F, "_dev", lambda t, name, dtype=None, home=None: t)
    monkeypatch.setattr(F, "_stream", lambda s: now[-1] if s is None else getattr(s, "cuda_stream", s))
    monkeypatch.setattr(F, "_launch", lambda *a: None, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(now[-1]))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append(s.cuda_stream))
    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, spy(getattr(torch, name)))
    return made, kept


@pytest.mark.parametrize("name", list(CALLS))
def test_own_tensors_belong_to_the_launch_stream(made, name):
    """The test's own inputs are torch.zeros on the current stream; everything
    else that is made is the binding's."""
    made, kept = made
    plain = {}
    for s in (None, Stream(7)):  # the current stream: nothing special
        del made[:], kept[:]
        CALLS[name](s)
        plain[s is None] = list(made)
        assert {x for x, _ in made} == {7} and not kept
    assert plain[True] == plain[False]
    for s, handle in ((Stream(99), 99), (99, 99), (0, 0), (1, 0)):
        del made[:], kept[:]
        CALLS[name](s)
        assert [f for _, f in made] == [f for _, f in plain[True]]  # the same tensors
        assert handle in {x for x, _ in made} <= {7, handle}
        assert all(f == "zeros" for x, f in made if x == 7)
        assert set(kept) == {7}  # what is returned stays until the caller's stream is done with it
