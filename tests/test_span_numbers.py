"""Figures that the span attention's comments and header state, checked on the
CPU: the rotation angle's error and when a decode takes one launch."""
import ctypes
import random
from decimal import Decimal, getcontext

import numpy as np

from tests.test_abi import L, _fake_cache  # noqa: F401  (L: fixture)
from tests.test_span_abi import span

getcontext().prec = 70
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def test_rotation_angle_error():
    """The kernels' arithmetic (float64 turns, whole ones dropped, a float32
    argument) against 70 digits: at most 1e-7 + pos * 4e-16 rad. The two
    positions are the worst of a search near 2^31."""
    rng = random.Random(0)
    cases = [(5e5, 1, 2147325392), (10.0, 2, 2 ** 31 - 1)]
    for _ in range(1500):
        pos = int(2 ** rng.uniform(0, 31)) if rng.random() < 0.5 else rng.randrange(2 ** 31 - 2 ** 20, 2 ** 31)
        cases.append((rng.choice([10.0, 1e4, 5e5, 1e6]), rng.randrange(64), pos))
    worst = 0.0
    for base, i, pos in cases:
        turns = base ** (-2.0 * i / 128.0) * 0.15915494309189535
        t = float(pos) * turns
        got = np.float32(t - np.rint(t))
        exact = Decimal(pos) * Decimal(base) ** (Decimal(-2 * i) / 128) / (2 * PI)
        err = abs(Decimal(float(got)) - (exact - exact.to_integral_value()))
        err = float(min(err, 1 - err) * 2 * PI)
        assert err <= 1e-7 + pos * 4e-16, (base, i, pos, err)
        worst = max(worst, err)
    assert 2e-7 < worst <= 9.3e-7  # the figure is neither exceeded nor far from what happens


def test_when_a_decode_is_one_launch(L):
    """No partial sums are kept (256 bytes of workspace) exactly where no row
    can touch more than four units of 64 slots."""
    c = ctypes.byref(_fake_cache(max_len=8192))
    ws = L.fasa_attend_decode_workspace_bytes
    for n in (1, 255, 256, 257, 8192):
        for w in (0, 1, 63, 64, 65, 128, 129, 192, 193, 256):
            for k in (0, 1, 64, 65, 128, 129):
                units = -(-w // 64) + -(-k // 64)
                one = n <= 256 or (w > 0 and units <= 3)
                assert (ws(c, span(max_seq_len=n, window=w, n_sink=k), 0) == 256) == one, (n, w, k)
