"""GPU: rotation angles of frequencies of either sign and any size at far positions, against 80
digits."""
import math
from decimal import Decimal, getcontext
from fractions import Fraction

import pytest

from tests import _cache as C
from tests._gpu import need_gpu, torch

pytestmark = pytest.mark.gpu

getcontext().prec = 100
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798214808651")
TWO_PI = Fraction(2 * PI)


@pytest.fixture(scope="module")
def X():
    need_gpu()
    from sparse_depth_token_gb300 import xmod
    xmod.load()
    return xmod


def _angle(freq, pos):
    """pos * freq modulo a turn, from -pi to pi."""
    t = Fraction(freq) * pos
    return float(t - TWO_PI * round(t / TWO_PI))


FREQS = {
    "base": [1e4 ** (-c / 64) for c in range(64)],
    "minus": [-(1e4 ** (-c / 64)) for c in range(64)],
    "slow": [(-1) ** c * 8e-5 * 0.7 ** c for c in range(64)],
    "wide": [(-1) ** c * 10.0 ** (8 - c / 3.0) for c in range(64)],
    "edges": [0.0, -0.0, 5e-324, -5e-324, 1e-300, -1e-20, 2.0 ** -64, -2.0 ** -64, 2.0 ** -10, -2.0 ** -10,
              math.pi, -math.pi, 2 * math.pi, -2 * math.pi, 1e300, -1e300] + [(-1) ** c * 0.1 / (c + 1) for c in range(48)],
}


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("which", sorted(FREQS))
def test_angles(X, which, inter):
    hd, freqs = 128, FREQS[which]
    positions = [0, 1, 2, 4095, 131071, 2 ** 24 + 1, 10 ** 9 + 7, 2 ** 31 - 1]
    M = len(positions)
    dm = C.dims(X, 1, 1, hd, "fp32")
    rope = X.rope(hd, interleaved=inter)
    for c, f in enumerate(freqs):
        rope.freq[c] = f
    x = torch.zeros(M, 2 * hd, device="cuda")
    first = slice(0, hd, 2) if inter else slice(0, hd // 2)
    second = slice(1, hd, 2) if inter else slice(hd // 2, hd)
    x[:, :hd][:, first] = 1.0
    out = torch.empty_like(x)
    X.qk_rope(dm, x, None, rope, out, pos=torch.tensor(positions, dtype=torch.int32, device="cuda"))
    out = out[:, :hd].double().cpu()
    for m, pos in enumerate(positions):
        for c, f in enumerate(freqs):
            t = _angle(f, pos)
            # the stated error of the angle, cosine's and sine's, and the rounding to fp32
            bound = min(2.0, pos * (abs(f) * 2.0 ** -53 + 2.0 ** -62) + 2e-9) + 1e-7 + 2.0 ** -24
            err = max(abs(float(out[m, first][c]) - math.cos(t)), abs(float(out[m, second][c]) - math.sin(t)))
            assert err <= bound, (pos, f, err, bound)
