"""GPU: token log probabilities with entropy and alternatives, and their gradient, against
64-bit forms; ties, masked tokens, rows without a distribution, odd strides, graphs."""
import math

import numpy as np
import pytest

from tests._gpu import need_gpu, torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def X():
    need_gpu()
    from sparse_depth_token_gb300 import xmod
    xmod.load()
    return xmod


def _logits(N, V, dtype, pad=0, seed=0, std=3.0, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    x = std * torch.randn(N, V + pad, generator=g)
    if masked:
        x[torch.rand(N, V + pad, generator=g) < masked] = -math.inf
    t = torch.randint(0, V, (N,), generator=g)
    x[torch.arange(N), t] = 2.5
    return x.cuda().to(DT[dtype])[:, :V], t.to(torch.int32).cuda()


def _forward(X, x, target, k, entropy=True, status=None):
    N = x.shape[0]
    f = dict(dtype=torch.float32, device="cuda")
    out = dict(logp=torch.full((N,), 7.0, **f), lse=torch.full((N,), 7.0, **f),
               entropy=torch.full((N,), 7.0, **f) if entropy else None,
               top_idx=torch.full((N, k), -5, dtype=torch.int32, device="cuda") if k else None,
               top_logp=torch.full((N, k), 7.0, **f) if k else None)
    X.token_logprobs(x, target, status=status, **out)
    return out


def _check(x, target, out, k):
    """fp32 sums of V positive terms by blocks, lanes and threads: at most 64 + V / 256
    roundings in a row, each 2^-24 relative; exp's argument is off by 2^-24 of its size
    (up to |x - max|) and exp itself by 2 steps."""
    N, V = x.shape
    d = x.double()
    lse = torch.logsumexp(d, 1)
    lp = d - lse[:, None]
    steps = 64 + V / 256 + 2
    finite = torch.where(d > -math.inf, d, d.amax(1, keepdim=True))
    span = (d.amax(1) - finite.amin(1))
    rel = (steps + span * 1.5) * 2.0 ** -24
    size = d.amax(1).abs() + lse.abs() + span
    tol = rel + 4 * 2.0 ** -24 * size
    assert bool(((out["lse"].double() - lse).abs() <= tol).all())
    t = target.long()
    want = torch.where(t >= 0, lp.gather(1, t.clamp(min=0)[:, None])[:, 0], torch.zeros_like(lse))
    fin = torch.isfinite(want)
    assert torch.equal(out["logp"].double()[~fin], want[~fin])
    assert bool(((out["logp"].double() - want).abs() <= tol + 2.0 ** -23 * want.abs())[fin].all())
    if out["entropy"] is not None:
        p = lp.exp()
        ent = torch.special.entr(p).sum(1)
        # ln l and the mean of x - max, whose terms p (max - x) add up without cancelling
        mean = (p * torch.where(p > 0, d.amax(1, keepdim=True) - d, torch.zeros_like(d))).sum(1)
        bound = 2 * rel * (1 + mean) + 4 * 2.0 ** -24 * (1 + lse.abs() + d.amax(1).abs() + mean)
        assert bool(((out["entropy"].double() - ent).abs() <= bound).all())
    if k:
        idx = torch.sort(d, dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(out["top_idx"].long(), idx)
        want = lp.gather(1, idx)
        fin = torch.isfinite(want)
        assert torch.equal(out["top_logp"].double()[~fin], want[~fin])
        err = (out["top_logp"].double() - want).abs() - (tol[:, None] + 2.0 ** -23 * want.abs())
        assert bool((err[fin] <= 0).all())


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("N,V,k,pad,masked", [
    (1, 1, 1, 0, 0.0), (3, 7, 7, 0, 0.0), (5, 64, 64, 1, 0.3), (2, 255, 5, 3, 0.0), (9, 1000, 20, 0, 0.9),
    (4, 8193, 8, 0, 0.0), (1, 50257, 20, 0, 0.2), (40, 50257, 5, 0, 0.0), (700, 1023, 3, 9, 0.0),
    (2, 151937, 64, 0, 0.0), (300, 50257, 0, 7, 0.0), (33, 131072, 1, 0, 0.0)])
def test_logprobs_match_the_plain_form(X, dtype, N, V, k, pad, masked):
    x, t = _logits(N, V, dtype, pad, N + V, masked=masked)
    if N > 2:
        t[1] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _forward(X, x, t, k, status=status)
    assert int(status) == 0
    _check(x, t, out, k)
    again = _forward(X, x, t, k)
    assert all(torch.equal(out[n], again[n]) for n in out if out[n] is not None)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("V", [40, 5000, 70001])
@pytest.mark.parametrize("shape", ["equal", "ascending", "descending", "coarse", "zeros", "tail", "stairs"])
def test_alternatives_with_ties(X, dtype, V, shape):
    """Rows of equal logits, sorted ones (every logit a new best), few distinct values, -0
    beside +0, best values in the last places, plateaus: ties go to the lower token."""
    i = torch.arange(V, dtype=torch.float32)
    x = {"equal": torch.full((V,), 1.5), "ascending": i / 128, "descending": -i / 128,
         "coarse": ((i * 7919) % 13).floor(), "zeros": torch.where(i % 3 == 0, -0.0, 0.0),
         "tail": torch.where(i >= V - 30, 4.0, -1.0), "stairs": (i / 1000).floor()}[shape]
    x = torch.stack([x, x.flip(0), x.roll(V // 3)]).cuda().to(DT[dtype])
    t = torch.tensor([0, V - 1, V // 2], dtype=torch.int32, device="cuda")
    out = _forward(X, x, t, 32)
    _check(x, t, out, 32)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("V", [50, 50257])
def test_rows_without_a_distribution(X, dtype, V):
    """All tokens ruled out, a NaN, +infinity: NaN and a report, the other rows hold; a
    single token left has log probability 0 and entropy 0."""
    x, t = _logits(6, V, dtype, 0, 5)
    x[1] = -math.inf
    x[2, V // 2] = math.nan
    x[3, V - 1] = math.inf
    x[4] = -math.inf
    x[4, 3] = -40.0
    t[4] = 3
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _forward(X, x, t, 5, status=status)
    assert int(status) == X.ERR_DEVICE_CHECK
    for n in ("logp", "lse", "entropy", "top_logp"):
        assert bool(out[n][1:4].isnan().all()), n
    assert out["top_idx"][1].tolist() == [0, 1, 2, 3, 4]
    assert int(out["top_idx"][2, 0]) == V // 2 and int(out["top_idx"][3, 0]) == V - 1
    assert float(out["logp"][4]) == 0 and float(out["entropy"][4]) == 0 and float(out["lse"][4]) == -40
    rows = [0, 4, 5]
    _check(x[rows], t[rows], {n: v[rows] for n, v in out.items()}, 5)


def test_bad_targets_are_reported(X):
    x, t = _logits(4, 100, "bf16")
    t[2] = 100
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _forward(X, x, t, 0, status=status)
    assert int(status) == X.ERR_DEVICE_CHECK and math.isnan(float(out["logp"][2]))
    rows = [0, 1, 3]
    _check(x[rows], t[rows], {n: v[rows] for n, v in out.items() if v is not None} | {"entropy": out["entropy"][rows]}, 0)
    status.zero_()
    d = torch.empty_like(x)
    g = torch.ones(4, device="cuda")
    X.token_logprobs_bwd(x, t, out["lse"], g, d, status=status)
    assert int(status) == X.ERR_DEVICE_CHECK and bool((d[2] == 0).all()) and bool((d[1] != 0).any())


def test_single_outputs_and_empty_batches(X):
    """Each output alone gives the same bits as all together."""
    x, t = _logits(20, 3001, "bf16", 5)
    out = _forward(X, x, t, 4)
    f = dict(dtype=torch.float32, device="cuda")
    for names in (("logp",), ("lse",), ("entropy",), ("top_idx", "top_logp")):
        part = {n: torch.empty_like(out[n]) for n in names}
        X.token_logprobs(x, t if "logp" in names else None, **part)
        for n in names:
            assert torch.equal(part[n], out[n]), n
    none = torch.empty(0, 3001, dtype=torch.bfloat16, device="cuda")
    X.token_logprobs(none, None, lse=torch.empty(0, **f))
    X.token_logprobs_bwd(none, None, torch.empty(0, **f), None, none)


# ------------------------------------------------------------------ gradient

def _grad_ref(x, t, g, gh):
    d = x.double()
    lp = d - torch.logsumexp(d, 1, keepdim=True)
    p = lp.exp()
    out = -g.double()[:, None] * (t >= 0)[:, None] * p
    hot = torch.zeros_like(p)
    rows = (t >= 0).nonzero()[:, 0]
    hot[rows, t[rows].long()] = g.double()[rows]
    ent = torch.special.entr(p)
    h = ent.sum(1, keepdim=True)
    return out + hot + gh.double()[:, None] * (ent - p * h), p, lp, h


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("N,V,pad,dpad,masked", [
    (1, 1, 0, 0, 0.0), (3, 7, 0, 0, 0.0), (5, 64, 1, 1, 0.3), (2, 255, 3, 0, 0.0), (4, 8193, 0, 3, 0.0),
    (40, 50257, 0, 0, 0.2), (9, 50257, 0, 8, 0.0), (700, 1023, 9, 9, 0.0)])
@pytest.mark.parametrize("with_entropy", [True, False])
def test_gradient_matches_the_formula(X, dtype, N, V, pad, dpad, masked, with_entropy):
    x, t = _logits(N, V, dtype, pad, N + V, masked=masked)
    gen = torch.Generator().manual_seed(V)
    g = torch.randn(N, generator=gen).cuda()
    gh = (0.3 * torch.randn(N, generator=gen)).cuda() if with_entropy else torch.zeros(N, device="cuda")
    if N > 2:
        t[1] = -1
        g[2], gh[2] = 0.0, 0.0
    out = _forward(X, x, t, 0)
    d = torch.full((N, V + dpad), -3.0, dtype=DT[dtype], device="cuda")
    X.token_logprobs_bwd(x, t, out["lse"], g, d[:, :V], entropy=out["entropy"] if with_entropy else None,
                         g_entropy=gh if with_entropy else None)
    assert bool((d[:, V:] == -3).all())
    ref, p, lp, h = _grad_ref(x, t, g, gh)
    # p = exp(x - lse): the argument is off by the forward's error in lse and its own
    # rounding; y + H by H's error
    lse_err = (64 + V / 256 + 40) * 2.0 ** -24 + 6 * 2.0 ** -24 * (x.double().amax(1).abs() + 10)
    fin = torch.where(lp > -math.inf, lp, torch.zeros_like(lp))
    pe = lse_err[:, None] + 4 * 2.0 ** -24 * (1 + fin.abs())
    size = g.double().abs()[:, None] * p + gh.double().abs()[:, None] * p * (fin.abs() + h + 1)
    bound = pe * 2 * size + 4 * 2.0 ** -24 * ref.abs()
    hot = torch.zeros_like(p, dtype=torch.bool)
    rows = (t >= 0).nonzero()[:, 0]
    hot[rows, t[rows].long()] = True
    bound = bound + hot * 4 * 2.0 ** -24 * g.double().abs()[:, None]
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    tiny = 2.0 ** -126      # below it a result may be rounded to a subnormal or to zero
    err = (d[:, :V].double() - ref).abs() - bound - half * (ref.abs() + bound) - tiny
    assert float(err.max()) <= 0, float(err.max())
    if N > 2:
        assert bool((d[2, :V] == 0).all())


def test_gradient_matches_differences(X):
    """Central differences of sum(g logp + gH H), taken from the forward in fp32."""
    N, V, eps = 6, 503, 2.0 ** -6
    x, t = _logits(N, V, "fp32", 0, 11, std=1.0)
    gen = torch.Generator().manual_seed(12)
    g, gh = torch.randn(N, generator=gen).cuda(), torch.randn(N, generator=gen).cuda()
    out = _forward(X, x, t, 0)
    d = torch.empty_like(x)
    X.token_logprobs_bwd(x, t, out["lse"], g, d, entropy=out["entropy"], g_entropy=gh)

    def value(y):
        o = _forward(X, y, t, 0)
        return float((g.double() * o["logp"].double() + gh.double() * o["entropy"].double()).sum())

    for s in range(4):
        v = torch.randn(N, V, generator=torch.Generator().manual_seed(s)).cuda()
        num = (value(x + eps * v) - value(x - eps * v)) / (2 * eps)
        # third-order term eps^2 / 6 |J'''| with |J'''| <= N (|v|_inf^3) few, and the
        # values' fp32 errors over 2 eps
        tol = N * (eps ** 2 * 4 ** 3 + 2 * 100 * 2.0 ** -24 / eps) * 2
        assert abs(num - float((d.double() * v.double()).sum())) <= tol


@pytest.mark.parametrize("dtype", sorted(DT))
def test_gradient_in_place(X, dtype):
    x, t = _logits(33, 5003, dtype, 3, 13)
    g = torch.randn(33, generator=torch.Generator().manual_seed(1)).cuda()
    out = _forward(X, x, t, 0)
    d = torch.empty(33, 5003, dtype=x.dtype, device="cuda")
    X.token_logprobs_bwd(x, t, out["lse"], g, d, entropy=out["entropy"], g_entropy=0.1 * g)
    X.token_logprobs_bwd(x, t, out["lse"], g, x, entropy=out["entropy"], g_entropy=0.1 * g)
    assert torch.equal(x.contiguous(), d)


def test_row_without_a_distribution_has_zero_gradient_when_unused(X):
    x, t = _logits(3, 600, "bf16")
    x[1] = -math.inf
    t[1] = -1
    out = _forward(X, x, t, 0)
    d = torch.empty(3, 600, dtype=x.dtype, device="cuda")
    X.token_logprobs_bwd(x, t, out["lse"], torch.ones(3, device="cuda"), d)
    assert bool((d[1] == 0).all()) and bool(d.isfinite().all())


def test_rows_past_32_bit_offsets(X):
    """Rows whose element offsets pass 2^31 and 2^32."""
    V, ld = 1000, 2 ** 25 + 1
    buf = torch.empty(130 * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((130, V), (ld, 1))
    small, t = _logits(130, V, "bf16")
    x.copy_(small)
    out = _forward(X, x, t, 5)
    _check(small, t, out, 5)
    g = torch.ones(130, device="cuda")
    d, e = torch.empty_like(small), None
    X.token_logprobs_bwd(small, t, out["lse"], g, d)
    X.token_logprobs_bwd(x, t, out["lse"], g, x)
    assert torch.equal(x.contiguous(), d)


def test_captured_scoring_replays(X):
    """Forward and gradient recorded into a graph on a side stream and replayed on other
    logits give the eager calls' bits."""
    for N, V in ((2, 50257), (64, 8191)):
        a, t = _logits(N, V, "bf16", 0, 1)
        b, tb = _logits(N, V, "bf16", 0, 2)
        g = torch.ones(N, device="cuda")
        out = _forward(X, a, t, 5)
        d = torch.empty(N, V, dtype=a.dtype, device="cuda")
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            X.token_logprobs(a, t, **out)
            X.token_logprobs_bwd(a, t, out["lse"], g, d, entropy=out["entropy"], g_entropy=g)
        a.copy_(b)
        t.copy_(tb)
        graph.replay()
        torch.cuda.synchronize()
        ref = _forward(X, b, tb, 5)
        d2 = torch.empty_like(d)
        X.token_logprobs_bwd(b, tb, ref["lse"], g, d2, entropy=ref["entropy"], g_entropy=g)
        assert all(torch.equal(out[n], ref[n]) for n in out) and torch.equal(d, d2)


def test_loss_gradient_chains_into_a_layer(X):
    """The end of a training step: logits of a dense layer's output, their log
    probabilities, the gradient back through the projection into xmod_layer_bwd, against
    central differences of the loss (fp32)."""
    from sparse_depth_token_gb300 import inputs as I
    from tests._gpu import dev_layer, to_dev, workspace, xmod_dims
    w = I.WORKLOADS["tiny_fp32"].replace(B=1, T=16)
    lw = I.layer_weights(w, 0)
    dev = dev_layer(lw, "fp32")
    W = X.layer_weights(dev, 1.0, 1e4)
    dm = xmod_dims(w)
    V = 301
    head = (0.05 * torch.randn(V, w.d, generator=torch.Generator().manual_seed(1))).cuda()
    t = torch.randint(0, V, (w.T,), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    x = to_dev(I.residual_stream(w), "fp32").view(w.T, w.d)

    def forward(x):
        y = x.clone()
        X.layer_fwd(dm, X.LAYER_DENSE, 1, 0, W, y, None, None, None, workspace(dm, 1))
        return y, _forward(X, y @ head.T, t, 0)

    y, out = forward(x)
    dl = torch.empty(w.T, V, device="cuda")
    X.token_logprobs_bwd(y @ head.T, t, out["lse"], torch.ones(w.T, device="cuda"), dl)
    dy = dl @ head
    dx = torch.empty_like(x)
    shapes = {n: dev[n].shape for n in X.LayerWeights.NAMES}
    grads = {n: torch.empty(s, device="cuda") for n, s in shapes.items()}
    grads["varsigma"] = torch.empty(4, device="cuda")
    ws = torch.zeros(X.bwd_workspace_bytes(dm, 1), dtype=torch.uint8, device="cuda")
    X.layer_bwd(dm, X.LAYER_DENSE, 1, 0, W, x, None, dy, 0.0, dx, X.layer_grads(grads), ws)
    eps = 2.0 ** -7
    for s in range(3):
        v = torch.randn(w.T, w.d, generator=torch.Generator().manual_seed(10 + s)).cuda()
        num = (float(forward(x + eps * v)[1]["logp"].double().sum())
               - float(forward(x - eps * v)[1]["logp"].double().sum())) / (2 * eps)
        ana = float((dx.double() * v.double()).sum())
        # fp32 losses of 16 tokens near 6: 16 * 6 * 2^-20 over 2 eps = 6e-3; third order
        # below eps^2 |v|^3 ~ 6e-5 * 16; both on a derivative of order |dx| |v| ~ 1
        assert abs(num - ana) <= 6e-3 + 1e-3 + 1e-2 * abs(ana)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("first_row,first_token", [(1, 0), (3, 5), (2, 1)])
def test_slices_that_begin_anywhere(X, dtype, first_row, first_token):
    """Rows and tokens cut out of a larger array of odd rows: bases and rows at any element,
    forward, gradient and gradient in place."""
    full, _ = _logits(9, 5003, dtype, 0, 31)
    x = full[first_row:, first_token:]
    N, V = x.shape
    t = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(7)).to(torch.int32).cuda()
    small = x.contiguous()
    out = _forward(X, x, t, 9)
    _check(small, t, out, 9)
    g = torch.randn(N, generator=torch.Generator().manual_seed(8)).cuda()
    d = torch.empty_like(small)
    X.token_logprobs_bwd(small, t, out["lse"], g, d, entropy=out["entropy"], g_entropy=g)
    wide = torch.full((9, 5010), -3.0, dtype=x.dtype, device="cuda")
    part = wide[first_row:, 7:7 + V]
    X.token_logprobs_bwd(x, t, out["lse"], g, part, entropy=out["entropy"], g_entropy=g)
    assert torch.equal(part.contiguous(), d)
    part.fill_(-3.0)
    assert bool((wide == -3).all()), "a value outside the slice changed"
    before = full.clone()
    X.token_logprobs_bwd(x, t, out["lse"], g, x, entropy=out["entropy"], g_entropy=g)
    assert torch.equal(x.contiguous(), d)
    x.copy_(before[first_row:, first_token:])
    assert torch.equal(full, before), "a value outside the slice changed"


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("N,V", [(2, 50257), (700, 5000), (3, 131)])
@pytest.mark.parametrize("mask", ["inf", "lowest"])
def test_few_allowed_tokens(X, dtype, N, V, mask):
    """A grammar that leaves fewer tokens than alternatives are asked for: the rest are ruled
    out tokens in order, at -infinity or at the type's lowest value."""
    low = -math.inf if mask == "inf" else torch.finfo(DT[dtype]).min
    gen = torch.Generator().manual_seed(V)
    x = torch.full((N, V), low, dtype=DT[dtype], device="cuda")
    t = torch.randint(0, V, (N,), generator=gen).cuda()
    for i in range(3):
        at = torch.randint(0, V, (N,), generator=gen).cuda()
        x[torch.arange(N, device="cuda"), at] = 1.0 + i
    x[torch.arange(N, device="cuda"), t] = 0.5
    out = _forward(X, x, t.to(torch.int32), 20)
    d = x.double()
    idx = torch.sort(d, dim=1, descending=True, stable=True).indices[:, :20]
    assert torch.equal(out["top_idx"].long(), idx)
    lp = torch.log_softmax(d, 1)
    assert bool(((out["logp"].double() - lp.gather(1, t[:, None])[:, 0]).abs() <= 2.0 ** -18).all())
    assert bool(((out["entropy"].double() - torch.special.entr(lp.exp()).sum(1)).abs() <= 2.0 ** -18).all())
    want = lp.gather(1, idx)
    live = want > -1e30
    assert bool(((out["top_logp"].double() - want).abs()[live] <= 2.0 ** -18).all())
    assert bool((out["top_logp"][~live] < -1e30).all())


def test_all_tokens_at_the_lowest_value(X):
    """Finite logits, however low, are a distribution: the uniform one."""
    for dtype, t in DT.items():
        x = torch.full((2, 3000), torch.finfo(t).min, dtype=t, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = _forward(X, x, torch.zeros(2, dtype=torch.int32, device="cuda"), 4, status=status)
        assert int(status) == 0
        assert out["top_idx"].tolist() == [[0, 1, 2, 3]] * 2
        assert bool(((out["entropy"] - math.log(3000)).abs() < 1e-5).all())
        assert bool(((out["logp"] + math.log(3000)).abs() < 1e-5).all())


def test_binding_refusals(X):
    """Types, shapes and layouts that the call cannot take are refused by the binding."""
    x, t = _logits(4, 50, "bf16")
    f = torch.empty(4, device="cuda")
    idx, lp = torch.empty(4, 3, dtype=torch.int32, device="cuda"), torch.empty(4, 3, device="cuda")
    bad = [lambda: X.token_logprobs(x.double(), None, lse=f), lambda: X.token_logprobs(x.half(), None, lse=f),
           lambda: X.token_logprobs(x.t(), None, lse=f), lambda: X.token_logprobs(x[0], None, lse=f),
           lambda: X.token_logprobs(x[:1].expand(4, 50), None, lse=f),
           lambda: X.token_logprobs(x, t.long(), logp=f), lambda: X.token_logprobs(x, t, logp=f[:3]),
           lambda: X.token_logprobs(x, t.cpu(), logp=f), lambda: X.token_logprobs(x, t, logp=f.double()),
           lambda: X.token_logprobs(x, t), lambda: X.token_logprobs(x, None, logp=f),
           lambda: X.token_logprobs(x, None, top_idx=idx), lambda: X.token_logprobs(x, None, top_idx=idx, top_logp=lp[:, :2]),
           lambda: X.token_logprobs(x, None, lse=f, status=f),
           lambda: X.token_logprobs_bwd(x, t, f, f, x.float()), lambda: X.token_logprobs_bwd(x, None, f, f, x),
           lambda: X.token_logprobs_bwd(x, t, f, f, x, g_entropy=f),
           lambda: X.token_logprobs_bwd(x, t, f[:2], f, x)]
    for i, call in enumerate(bad):
        with pytest.raises(X.XmodError) as e:
            call()
        assert e.value.status == X.ERR_INVALID_ARG, i


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("V", [1009, 1021, 1022, 1024, 2033, 2041, 2042, 2048, 4096])
def test_row_lengths_around_the_kernels_borders(X, dtype, V):
    """Rows that a warp, a CTA's first chunk or more just hold, at any alignment."""
    x, t = _logits(11, V, dtype, 1, V)
    for k in (1, 31, 33):
        out = _forward(X, x, t, k)
        _check(x, t, out, k)
    g = torch.randn(11, generator=torch.Generator().manual_seed(9)).cuda()
    d = torch.empty(11, V, dtype=x.dtype, device="cuda")
    X.token_logprobs_bwd(x, t, out["lse"], g, d, entropy=out["entropy"], g_entropy=g)
    ref = _grad_ref(x, t, g, g)[0]
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    # the bound of the formula's test with |g| (1 + |ln p| + H) below 64
    assert bool(((d.double() - ref).abs() <= half * ref.abs() + 64 * 2.0 ** -17 * ref.abs() + 2.0 ** -17).all())


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("shape", ["equal", "ascending", "random"])
def test_longest_rows(X, dtype, shape):
    """Rows at the vocabulary's limit with the most alternatives, in orders that make the
    alternatives' search as long as it gets."""
    V = X.MAX_VOCAB
    i = torch.arange(V, dtype=torch.float32)
    x = {"equal": torch.full((V,), -2.0), "ascending": i * 2.0 ** -18,
         "random": torch.randn(V, generator=torch.Generator().manual_seed(4))}[shape]
    x = torch.stack([x, x.flip(0)]).cuda().to(DT[dtype])
    t = torch.tensor([5, V - 1], dtype=torch.int32, device="cuda")
    for k in (64, 3):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = _forward(X, x, t, k, status=status)
        assert status.item() == 0
        _check(x, t, out, k)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("V,k", [(600, 20), (2040, 32), (30000, 64), (50257, 40)])
def test_more_equal_logits_than_are_kept(X, dtype, V, k):
    """A few tokens above a plateau of equal ones, in many rows at once; and rows of which
    each logit is a new best."""
    gen = torch.Generator().manual_seed(V + k)
    N = 301
    x = torch.full((N, V), torch.finfo(DT[dtype]).min, dtype=DT[dtype])
    t = torch.randint(0, V, (N,), generator=gen)
    x[torch.arange(N), t] = 0.5
    x[1::7] = (torch.arange(V) / 64).to(DT[dtype])
    x[2::7, : V // 2] = -3.0
    x = x.cuda()
    out = _forward(X, x, t.to(torch.int32).cuda(), k)
    idx = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(out["top_idx"].long(), idx)


def test_rows_past_the_vocabulary_limit_are_refused(X):
    """Also one whose length is past 32 bits, which the call's number would cut short."""
    buf = torch.empty(2 ** 32 + 100, dtype=torch.bfloat16, device="cuda")
    f = torch.empty(1, device="cuda")
    for V in (X.MAX_VOCAB + 1, 2 ** 32 + 100):
        x = buf[:V].view(1, V)
        for call in (lambda: X.token_logprobs(x, None, lse=f), lambda: X.token_logprobs_bwd(x, None, f, None, x)):
            with pytest.raises(X.XmodError) as e:
                call()
            assert e.value.status == X.ERR_UNSUPPORTED
