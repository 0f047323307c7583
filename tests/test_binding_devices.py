"""Tensors on another device than the cache are refused by the cache operators
(checked on the CPU: a stand-in for a tensor elsewhere)."""
import pytest
import torch

from rope_frequency_chunk_b200 import fasa as F
from tests.test_binding_streams import B, HKV, HQ, N, Cache, FakeLib, i32, q

U8 = torch.uint8


class Here(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


class Elsewhere(Here):
    def get_device(self):
        return 5


class CacheHere(Cache):
    sketch = torch.zeros(1).as_subclass(Here)


C = CacheHere()


def slots(dtype=torch.float32):
    return torch.zeros(B, HKV, N, dtype=dtype)


I32 = torch.int32
CALLS = {
    "attend_decode": (lambda **a: F.fasa_attend_decode(C, a.pop("seq_len"), a.pop("q"), N, **a),
                      dict(seq_len=i32(B), q=q(B, HQ), q_pos=i32(B), mass=slots(), out=q(B, HQ),
                           workspace=torch.zeros(4096, dtype=U8))),
    "attend_prompt": (lambda **a: F.fasa_attend_prompt(C, a.pop("seq_len"), a.pop("q"), N, **a),
                      dict(seq_len=i32(B), q=q(B, 3, HQ), q_pos=i32(B), q_len=i32(B), out=q(B, 3, HQ),
                           workspace=torch.zeros(4096, dtype=U8))),
    "evict": (lambda **a: F.fasa_evict(C, a.pop("seq_len"), a.pop("cur_pos"), a.pop("mass"), a.pop("slot_pos"), N, 8,
                                       **a),
              dict(seq_len=i32(B), cur_pos=i32(B), mass=slots(), slot_pos=slots(I32), mass_out=slots(),
                   slot_pos_out=slots(I32), len_out=i32(B), workspace=torch.zeros(4096, dtype=U8))),
    "append_kv_at": (lambda **a: F.fasa_append_kv_at(C, a.pop("k_new"), a.pop("v_new"), a.pop("slot0"), a.pop("pos0"),
                                                     **a),
                     dict(k_new=q(B, HKV, 2), v_new=q(B, HKV, 2), slot0=i32(B), pos0=i32(B), slot_pos=slots(I32),
                          mass=slots())),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_elsewhere_are_refused(monkeypatch, name):
    call, args = CALLS[name]
    launched = []
    monkeypatch.setattr(F, "_lib", FakeLib())
    monkeypatch.setattr(F, "_launch", lambda name, *a: launched.append(name))
    args = {k: t.as_subclass(Here) for k, t in args.items()}
    call(**args)
    assert launched == ["fasa_" + name]
    for k, t in args.items():
        with pytest.raises(ValueError, match=k):
            call(**dict(args, **{k: t.as_subclass(Elsewhere)}))
    assert len(launched) == 1
