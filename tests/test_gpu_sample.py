"""GPU: tokens sampled with temperature, top-k, top-p and min-p from given numbers against the
definition in 64 bits: vocabularies, ties, masks, borders, slices, refused rows."""
import math

import pytest

from tests import _more as R
from tests._gpu import need_gpu, torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
STATED = 2.0 ** -30     # a border closer than this (of 2^-33 a weight and their sums) may fall either way


@pytest.fixture(scope="module")
def X():
    need_gpu()
    from sparse_depth_token_gb300 import xmod
    xmod.load()
    return xmod


def f32(v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _run(X, logits, u, **kw):
    n = logits.shape[0]
    token = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    logp = torch.full((n,), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    X.sample_tokens(logits, u, token, logp=logp, status=status, **kw)
    return token, logp, int(status)


def _check(X, logits, u, rows=None, skip_close=False, **kw):
    token, logp, status = _run(X, logits, u, **kw)
    assert status == X.OK
    close = 0
    for i in range(len(u)) if rows is None else rows:
        want, lp, margin = R.sample_ref(logits[i], u[i], **{k: v[i] for k, v in kw.items() if v is not None})
        if margin <= STATED:
            close += 1
            continue
        assert int(token[i]) == want, (i, int(token[i]), want, margin)
        # the sum's relative error, and fp32's rounding of the result
        assert abs(float(logp[i]) - lp) <= 2.0 ** -23 * abs(lp) + 3e-7, (i, float(logp[i]), lp)
    assert skip_close or close == 0
    return token


def _settings(n, seed):
    g = torch.Generator().manual_seed(seed)
    pick = lambda v: torch.tensor(v)[torch.randint(0, len(v), (n,), generator=g)]  # noqa: E731
    return dict(temperature=pick([0.0, 0.3, 0.7, 1.0, 1.0, 2.5]).cuda(), top_k=pick([0, 1, 2, 7, 60, 1500, -1]).to(torch.int32).cuda(),
                top_p=pick([0.05, 0.5, 0.9, 0.999, 1.0, 1.0, 0.0]).cuda(), min_p=pick([0.0, 0.0, 0.01, 0.3, 1.0]).cuda())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,n,std", [(1, 5, 1.0), (2, 30, 1.0), (5, 40, 2.0), (33, 60, 0.5), (1000, 60, 2.5), (4097, 40, 6.0),
                                     (50257, 48, 2.5), (50257, 32, 0.1), (131071, 16, 2.5)])
def test_matches_the_definition(X, dtype, V, n, std):
    g = torch.Generator().manual_seed(V + n)
    logits = (torch.randn(n, V, generator=g) * std).cuda().to(DT[dtype])
    u = torch.rand(n, generator=g).cuda()
    _check(X, logits, u)
    _check(X, logits, u, **_settings(n, V))
    for k, v in _settings(n, V + 1).items():
        _check(X, logits, u, **{k: v})


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_more_rows_than_ctas(X, dtype):
    g = torch.Generator().manual_seed(1)
    logits = (torch.randn(1500, 700, generator=g) * 2).cuda().to(DT[dtype])
    u = torch.rand(1500, generator=g).cuda()
    # bf16 logits are often equal: of two equal weights one is exactly p = 0.5 of their sum, which
    # no sum in floating point need decide as the real numbers do; such a row says nothing
    _check(X, logits, u, rows=range(0, 1500, 13), skip_close=True, **_settings(1500, 3))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_numbers_spread_over_the_distribution(X, dtype):
    """An even comb of numbers on one row meets every token as often as its weight says."""
    g = torch.Generator().manual_seed(4)
    row = (torch.randn(12, generator=g) * 1.5).cuda().to(DT[dtype])
    n = 4096
    u = (torch.arange(n, device="cuda") + 0.5) / n
    token, _, _ = _run(X, row.expand(n, 12).contiguous(), u)
    count = torch.bincount(token.long(), minlength=12)
    want = torch.softmax(row.double(), 0) * n
    assert float((count - want).abs().max()) <= 1.0
    assert bool((token[1:] >= token[:-1]).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [100, 3000, 50257])
def test_ties(X, dtype, V):
    """Equal logits, and few values over many tokens: the lower tokens stay."""
    n = 24
    g = torch.Generator().manual_seed(V)
    u = torch.rand(n, generator=g).cuda()
    kw = dict(top_k=ints([1 + (i * V) // (n + 3) for i in range(n)]))
    _check(X, torch.full((n, V), 1.25, device="cuda", dtype=DT[dtype]), u, **kw)
    few = torch.randint(0, 3, (n, V), generator=g).cuda().to(DT[dtype])
    _check(X, few, u, **kw)
    # top_p ends inside a run of equal weights: p from numbers that no border meets
    kw = dict(top_p=(torch.rand(n, generator=g) * 0.9 + 0.05).cuda())
    _check(X, few, u, skip_close=True, **kw)
    kw["top_k"] = ints([V // 2] * n)
    _check(X, few, u, skip_close=True, **kw)
    zeros = few * 0.0
    zeros[:, ::2] *= -1.0           # -0 equals +0
    _check(X, zeros, u, top_k=ints([V // 3 + 1] * n))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("low", ["inf", "min"])
def test_masks(X, dtype, low):
    """Masked tokens are never chosen; with fewer tokens left than top_k all of them stay."""
    V, n = 5000, 32
    g = torch.Generator().manual_seed(9)
    logits = (torch.randn(n, V, generator=g) * 2).cuda().to(DT[dtype])
    fill = -math.inf if low == "inf" else torch.finfo(DT[dtype]).min
    for i in range(n):
        left = 1 + 3 * i
        off = torch.randperm(V, generator=g)[left:].cuda()
        logits[i, off] = fill
    u = torch.rand(n, generator=g).cuda()
    for kw in (dict(), dict(top_k=ints([40] * n)), dict(top_k=ints([V - 1] * n), top_p=f32([0.95] * n)),
               dict(top_p=f32([0.9] * n)), dict(temperature=f32([3.0] * n), min_p=f32([0.1] * n))):
        token = _check(X, logits, u, **kw)
        assert bool((logits.gather(1, token.long()[:, None]) > fill).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_borders(X, dtype):
    """u of 0 and just below 1, the smallest and largest settings, logits of any size."""
    g = torch.Generator().manual_seed(6)
    logits = (torch.randn(6, 300, generator=g) * 2).cuda().to(DT[dtype])
    logits[:, 0] = -math.inf
    u = f32([0.0, 1 - 2.0 ** -24, 2.0 ** -149, 0.5, 2.0 ** -60, 0.25])
    for kw in (dict(), dict(top_k=ints([300, 299, 2 ** 31 - 1, -2 ** 31, 3, 1])), dict(min_p=f32([1.0, 5.0, 1e-30, -1.0, 0.5, 1.0])),
               dict(top_p=f32([1e-30, 1 - 2.0 ** -24, 2.0, -1.0, 0.7, math.inf]))):
        token, logp, status = _run(X, logits, u, **kw)
        assert status == X.OK
        for i in (0, 3, 5):
            want, lp, margin = R.sample_ref(logits[i], u[i], **{k: v[i] for k, v in kw.items()})
            assert int(token[i]) == want and abs(float(logp[i]) - lp) <= 1e-6
        # just above 0: the first kept token; just below 1: the last, or the one before it
        assert bool((token >= 1).all()) and bool((token < 300).all())
    big = torch.zeros(4, 64, device="cuda")
    big[0, 5], big[0, 9] = 3e38, 3e38
    big[1] = torch.linspace(-1e30, 1e30, 64)
    big[2] = -3e38
    big[3, 7] = 1e-30
    for t in (1e-30, 1e-38, 1e-45, 1.0, 1e30):
        token, logp, status = _run(X, big, f32([0.3, 0.3, 0.3, 0.999]), temperature=f32([t] * 4))
        assert status == X.OK
        assert int(token[0]) == 5 or t == 1e30
        if t < 1e30:
            assert int(token[1]) == 63
        assert int(token[2]) == 19 and abs(float(logp[2]) + math.log(64)) < 1e-6


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_infinite_temperature(X, dtype):
    """Every logit above -infinity weighs the same, whatever the filters rank them by."""
    V, live = 1000, 700
    g = torch.Generator().manual_seed(31)
    logits = (torch.randn(8, V, generator=g) * 3).cuda().to(DT[dtype])
    logits[:, live:] = -math.inf
    # the token is u times 700 rounded down: 0.5 and the like are exact, the others no closer than
    # 0.3 to a border
    u, at = f32([0.0, 0.25, 0.5, 0.75, 0.1234, 0.9, 0.999, 0.6]), [0, 175, 350, 525, 86, 629, 699, 420]
    u[5] = 0.8995
    u[7] = 0.6005
    t = f32([math.inf] * 8)
    token, logp, status = _run(X, logits, u, temperature=t)
    assert status == X.OK and token.tolist() == at
    assert bool(((logp + math.log(live)).abs() < 1e-6).all())
    token, logp, status = _run(X, logits, u, temperature=t, top_k=ints([70] * 8))
    order = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :70].sort(dim=1).values
    assert status == X.OK and token.tolist() == [int(order[i, int(float(u[i]) * 70)]) for i in range(8)]
    assert bool(((logp + math.log(70)).abs() < 1e-6).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_largest_vocabulary(X, dtype):
    V = X.MAX_VOCAB
    g = torch.Generator(device="cuda").manual_seed(8)
    logits = (torch.randn(3, V + 3, generator=g, device="cuda") * 2.5).to(DT[dtype])[:, 1: V + 1]
    u = f32([0.3, 0.71, 0.999])
    for kw in (dict(), dict(top_p=f32([0.9, 0.5, 0.99])), dict(top_k=ints([50, 100000, 3])),
               dict(temperature=f32([1.7, 0.0, 0.6]), min_p=f32([1e-6, 0.1, 1e-3]))):
        # 2^22 borders lie 2^-22 apart, so that one row in 128 has its u within 2^-30 of one
        _check(X, logits, u, skip_close=True, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_temperature_zero_is_the_first_largest(X, dtype):
    logits = torch.zeros(3, 50, device="cuda", dtype=DT[dtype])
    logits[0, 7] = logits[0, 30] = 2.0
    logits[1, 49] = 1.0
    logits[2] = -0.0
    logits[2, 4] = 0.0
    for kw in (dict(temperature=f32([0.0] * 3)), dict(top_k=ints([1] * 3)), dict(top_p=f32([0.0] * 3)), dict(temperature=f32([-1.0] * 3))):
        token, logp, status = _run(X, logits, f32([0.9] * 3), **kw)
        assert token.tolist() == [7, 49, 0] and logp.tolist() == [0.0] * 3 and status == X.OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,first", [(0, 0), (1, 1), (3, 2), (5, 3), (8, 7)])
def test_slices(X, dtype, pad, first):
    """Rows that begin at any element; what lies beside them does not matter."""
    V, n = 1003, 20
    g = torch.Generator().manual_seed(pad)
    whole = torch.full((n, V + pad + first), math.nan, device="cuda", dtype=DT[dtype])
    logits = whole[:, first:first + V]
    logits.copy_((torch.randn(n, V, generator=g) * 2).cuda())
    u = torch.rand(n, generator=g).cuda()
    _check(X, logits, u, **_settings(n, pad))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_without_a_distribution(X, dtype):
    n, V = 8, 2000
    g = torch.Generator().manual_seed(2)
    good = torch.randn(n, V, generator=g).cuda().to(DT[dtype])
    u = torch.rand(n, generator=g).cuda()
    want, wl, _ = _run(X, good, u)

    def both(logits, uu, bad, **kw):
        token, logp, status = _run(X, logits, uu, **kw)
        assert status == X.ERR_DEVICE_CHECK
        assert int(token[bad]) == -1 and math.isnan(float(logp[bad]))
        keep = [i for i in range(n) if i != bad]
        assert torch.equal(token[keep], want[keep]) and torch.equal(logp[keep], wl[keep])

    for i, v in ((0, math.nan), (3, math.inf), (7, None)):
        x = good.clone()
        if v is None:
            x[i] = -math.inf
        else:
            x[i, V - 1] = v
        both(x, u, i)
    for v in (math.nan, 1.0, -1e-9, math.inf):
        bad = u.clone()
        bad[4] = v
        both(good, bad, 4)
    one = f32([1.0] * n)
    one[2] = math.nan
    for name in ("temperature", "top_p"):
        both(good, u, 2, **{name: one})
    both(good, u, 2, min_p=one - 1.0)


def test_streams_and_graphs(X):
    g = torch.Generator().manual_seed(3)
    logits = (torch.randn(40, 9000, generator=g) * 2).cuda()
    u = torch.rand(40, generator=g).cuda()
    kw = _settings(40, 8)
    token, logp = torch.zeros(40, dtype=torch.int32, device="cuda"), torch.zeros(40, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        X.sample_tokens(logits, u, token, logp=logp, **kw)
    for i in range(3):
        u.copy_(torch.rand(40, generator=g).cuda())
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph.replay()
        torch.cuda.synchronize()
        want, wl, _ = _run(X, logits, u, **kw)
        assert torch.equal(token, want) and torch.equal(logp, wl)


def test_binding_refusals(X):
    logits, u, token = torch.zeros(4, 10, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    for over in (dict(logits=logits.half()), dict(logits=logits.t().contiguous().t()), dict(logits=logits.cpu()), dict(u=u[:3]),
                 dict(u=u.double()), dict(token=token.long()), dict(temperature=u[:2]), dict(top_k=u), dict(top_p=token),
                 dict(min_p=u.cpu()), dict(logp=token)):
        with pytest.raises(X.XmodError) as e:
            X.sample_tokens(**{**dict(logits=logits, u=u, token=token), **over})
        assert e.value.status == X.ERR_INVALID_ARG, over.keys()
    X.sample_tokens(logits[:0], u[:0], token[:0])
