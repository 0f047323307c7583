"""Arrays of an eviction that share memory are refused before a launch (no GPU
needed)."""
import ctypes

import pytest

from rope_frequency_chunk_b200 import fasa as F
from tests.test_abi import L, _fake_cache  # noqa: F401  (L: fixture)

# batch 3, 2 KV heads, 1024 slots: 12 bytes per sequence array, 24 KB per slot array
SEQ, CUR, LEN = 0x90000, 0x91000, 0x92000
MASS, POS, MASS_OUT, POS_OUT = 0x100000, 0x200000, 0x300000, 0x400000
PER_SLOT = 3 * 2 * 1024 * 4


def evict(L, mass_out=MASS_OUT, pos_out=POS_OUT, len_out=LEN):
    c = ctypes.byref(_fake_cache(batch=3))
    d = ctypes.byref(F.fasa_evict_desc(SEQ, CUR, 1000, 100, 4, 10))
    # without a workspace: what passes the checks of the arrays is refused for that
    return L.fasa_evict(c, None, d, MASS, POS, mass_out, pos_out, len_out, None, 0, None)


@pytest.mark.parametrize("base", [SEQ, CUR])
def test_new_lengths_lie_apart_from_what_is_read(L, base):
    for off in (-8, -4, 0, 4, 8):
        assert evict(L, len_out=base + off) == 1, off
    assert evict(L, len_out=base - 12) == 4 and evict(L, len_out=base + 12) == 4


def test_outputs_are_the_inputs_or_apart(L):
    assert evict(L) == 4 and evict(L, mass_out=MASS, pos_out=POS) == 4
    for off in (4, -4, 4096, PER_SLOT - 4, 4 - PER_SLOT):
        assert evict(L, mass_out=MASS + off) == 1 and evict(L, pos_out=POS + off) == 1
    for off in (PER_SLOT, -PER_SLOT):
        assert evict(L, mass_out=MASS + off) == 4 and evict(L, pos_out=POS + off) == 4
