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
