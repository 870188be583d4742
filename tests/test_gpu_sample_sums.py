"""GPU: how exactly sampling weighs and sums: many small weights beside a large one, weights next
to min-p, sums of the largest rows. A weight is good to 2^-32 of itself and 2^-62 of the largest, sums
are exact, so that a row's sum S is good to S 2^-32 + V 2^-62 <= S 2^-31."""
import math

import pytest

from tests._gpu import need_gpu, torch
from tests.test_gpu_sample import DT, _check, _run, f32, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def X():
    need_gpu()
    from sparse_depth_token_gb300 import xmod
    xmod.load()
    return xmod


def _neighbours(x):
    """The fp32 numbers next to x, more than 2^-31 away from it."""
    t = torch.tensor(x, dtype=torch.float64).float()
    lo, hi = t, t
    while float(lo) > x - 2.0 ** -31:
        lo = torch.nextafter(lo, torch.tensor(0.0))
    while float(hi) < x + 2.0 ** -31:
        hi = torch.nextafter(hi, torch.tensor(2.0))
    return float(lo), float(hi)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [50257, 131072, 1 << 22])
@pytest.mark.parametrize("depth", [15.0, 20.0, 24.75, 27.25])
def test_many_small_weights(X, dtype, V, depth):
    """One large weight and V - 1 equal ones far below it: log probabilities, and numbers on both
    sides of the large one's end."""
    logits = torch.full((1, V), 16.0 - depth, device="cuda", dtype=DT[dtype])
    logits[0, 0] = 16.0
    w = math.exp(-depth)
    S = 1.0 + (V - 1) * w

    def chosen(u, **kw):
        token, logp, status = _run(X, logits, f32([u]), **kw)
        assert status == X.OK
        return int(token), float(logp)

    # fp32's rounding of ln(1 + f), of f and of the result beside the sum's own error
    def near(lp, want):
        assert abs(lp - want) <= 2.0 ** -31 + 2.0 ** -22 * abs(want), (lp, want)

    below, above = _neighbours(1.0 / S)
    top, lp = chosen(below)
    assert top == 0
    near(lp, -math.log1p((V - 1) * w))
    if above < 1.0:
        at, lp = chosen(above)
        # the running sum passes above * S, which is good to 2^-31, in the tail
        want = 1 + (above * S - 1.0) / w
        assert at >= 1 and abs(at - want) <= 1 + 2.0 ** -30 * S / w
        near(lp, -depth - math.log(S))
    # of the tail, top_p's share: the shortest run that reaches it is longer by less than one weight
    p = float(f32([1.0 - 0.375 * (S - 1.0) / S]))
    if (S - 1.0) / S > 2.0 ** -22:
        for kw in (dict(top_p=f32([p])), dict(top_p=f32([p]), top_k=ints([V - 1]))):
            whole = S - w if "top_k" in kw else S
            top, lp = chosen(0.0, **kw)
            assert top == 0
            want = -math.log(p * whole)
            assert abs(lp - want) <= 2.0 ** -30 + w + 2.0 ** -22 * abs(want), (lp, want)
    # half of the tail by number
    top, lp = chosen(0.0, top_k=ints([V // 2]))
    assert top == 0
    near(lp, -math.log1p((V // 2 - 1) * w))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("filters", [dict(), dict(top_p=0.9999999), dict(top_k=40000)])
def test_min_p_next_to_a_weight(X, dtype, filters):
    """min_p a 2^21st above and below a token's weight; it lies before the largest, so that u = 0
    chooses it if it stays."""
    depths = [0.5, 3.0, 6.0, 9.25, 12.5, 15.0, 17.5, 19.0, 20.5]
    V, n = 50257, len(depths)
    logits = torch.full((n, V), -math.inf, device="cuda", dtype=DT[dtype])
    for i, d in enumerate(depths):
        logits[i, 5], logits[i, 7] = 16.0 - d, 16.0
    # top_p that drops nothing of two tokens has to exceed the larger's share: only shallow rows then
    rows = [i for i, d in enumerate(depths) if "top_p" not in filters or d < 14]
    kw = {k: (f32([v] * n) if k == "top_p" else ints([v] * n)) for k, v in filters.items()}
    for side, want in ((1 - 2.0 ** -21, 5), (1 + 2.0 ** -21, 7)):
        min_p = f32([math.exp(-d) * side for d in depths])
        token, logp, status = _run(X, logits, f32([0.0] * n), min_p=min_p, **kw)
        assert status == X.OK
        assert [int(token[i]) for i in rows] == [want] * len(rows)


@pytest.mark.parametrize("at", [1.25, 200.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_largest_sums(X, dtype, at):
    """2^22 equal logits (of bf16, 200 lies outside the table of values): sums of 2^84 units."""
    V = X.MAX_VOCAB
    logits = torch.full((1, V), at, device="cuda", dtype=DT[dtype])
    for u in (0.0, 0.30000001, 0.5, 0.99999994):
        for kw, kept in ((dict(), V), (dict(top_k=ints([3000001])), 3000001), (dict(top_p=f32([0.75])), V * 3 // 4),
                         (dict(top_p=f32([0.5]), top_k=ints([1 << 21])), 1 << 20), (dict(min_p=f32([1.0])), V)):
            token, logp, status = _run(X, logits, f32([u]), **kw)
            assert status == X.OK
            assert int(token) == int(float(f32([u])) * kept)
            assert abs(float(logp) + math.log(kept)) <= 2.0 ** -22 * math.log(kept)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_largest_rows_of_close_logits(X, dtype):
    """Millions of weights within a few bins, whose own sums pass 2^64 units."""
    V = X.MAX_VOCAB
    g = torch.Generator(device="cuda").manual_seed(12)
    logits = (torch.randn(2, V, generator=g, device="cuda") * 0.01 + 300.0).to(DT[dtype])
    u = f32([0.37, 0.81])
    # 2^22 borders lie 2^-22 apart: one row in 128 has its u within 2^-30 of one
    for kw in (dict(), dict(top_p=f32([0.4, 0.9])), dict(top_k=ints([3000000, 2000000]), top_p=f32([0.7, 0.3]))):
        _check(X, logits, u, skip_close=True, **kw)


@pytest.mark.parametrize("t,err", [(1e-30, 2.0 ** -32), (1.0, 2.0 ** -32), (1e30, 2.0 ** -32), (9e32, 2.0 ** -32), (1e37, 2.0 ** -22),
                                   (3e38, 2.0 ** -22)])
def test_stated_error_at_any_temperature(X, t, err):
    """Numbers right beside the borders between a row's tokens, twice the stated error away."""
    t = float(f32([t]))
    depth = [0.0, 0.37, 0.9, 1.1] + ([] if t > 1e38 else [2.2, 3.3, 4.7, 6.1, 8.3])
    x = f32([max(-3.3e38, -d * t) for d in depth])
    p = torch.softmax(x.double() / t, 0)
    ends = p.cumsum(0)[:-1]
    for side in (-1, 1):
        # fp32 has 2^-24 near 1, so that most numbers lie further out
        u = (ends + side * 2 * err).float()
        nxt = torch.nextafter(u, f32([2.0 * side]))
        u = torch.where((u.double() - ends) * side < 2 * err, nxt, u)
        n = u.numel()
        token, logp, status = _run(X, x.expand(n, -1).contiguous(), u, temperature=f32([t] * n))
        assert status == X.OK
        want = torch.arange(n, device="cuda") + (1 if side > 0 else 0)
        assert torch.equal(token.long(), want)
        lp = p.log()[want]
        assert bool(((logp.double() - lp).abs() <= 2.0 ** -22 * lp.abs() + 2.0 ** -23 + 2 * err).all())
