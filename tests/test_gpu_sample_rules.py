"""GPU: sampling at the edges of its numbers."""
import math

import pytest

from tests._gpu import need_gpu, torch
from tests.test_gpu_sample import DT, _run, f32, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def X():
    need_gpu()
    from sparse_depth_token_gb300 import xmod
    xmod.load()
    return xmod


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [40, 5000])
def test_negative_zeros(X, dtype, V):
    """-0 is 0: as the number, as the temperature and in every filter."""
    g = torch.Generator().manual_seed(V)
    logits = (torch.randn(9, V, generator=g) * 2).cuda().to(DT[dtype])
    logits[:, 0] = -math.inf
    none = torch.zeros(9, device="cuda")
    for kw in (dict(), dict(top_k=ints([5] * 9)), dict(top_p=f32([0.8] * 9)), dict(min_p=f32([0.1] * 9)),
               dict(top_k=ints([30] * 9), top_p=f32([0.8] * 9), min_p=f32([0.01] * 9))):
        a, b = _run(X, logits, none, **kw), _run(X, logits, -none, **kw)
        assert a[2] == b[2] == X.OK
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert bool((a[0] >= 1).all()) and bool(torch.isfinite(a[1]).all())
    for name in ("temperature", "top_p", "min_p"):
        a, b = _run(X, logits, none + 0.4, **{name: none}), _run(X, logits, none + 0.4, **{name: -none})
        assert a[2] == b[2] == X.OK
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("t", [1e-45, 1e-38, 1.0e-36, 2.0e-36])
def test_log_probability_at_tiny_temperatures(X, t):
    """Logits 1e-36 apart: a temperature below 2^-120 log2(e) counts as that, for the choice and for
    its log probability."""
    least = float(f32([1.44269502])) * 2.0 ** -120
    logits = torch.full((64, 300), -1.0, device="cuda")
    logits[:, 3], logits[:, 7], logits[:, 200] = -1e-36, 0.0, -4e-37
    u = (torch.arange(64, device="cuda") + 0.5) / 64
    # 64-bit: the three weights of tokens 3, 7 and 200
    x = logits[0, [3, 7, 200]].double()
    p = torch.softmax(x / max(float(f32([t])), least), 0)
    ends = p.cumsum(0)
    assert float((u.double()[:, None] - ends[None, :2]).abs().min()) > 1e-4
    want = (u.double()[:, None] > ends[None, :2]).sum(1)
    token, logp, status = _run(X, logits, u, temperature=f32([t] * 64))
    assert status == X.OK
    assert token.tolist() == [[3, 7, 200][int(i)] for i in want]
    lp = p.log()[want]
    # the sum's error and fp32's of the difference over the temperature
    assert bool(((logp.double() - lp).abs() <= 2.0 ** -22 * lp.abs() + 3e-7).all())
