"""GPU: norms of queries and keys with rotary positions, and their gradient, against plain
64-bit forms and differences."""
import math

import pytest

from tests import _more as R
from tests import _cache as C
from tests._gpu import need_gpu, torch

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def X():
    need_gpu()
    from sparse_depth_token_gb300 import xmod
    xmod.load()
    return xmod


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _case(X, dtype, hq, hkv, hd, M, rot, inter, scaling=0, norm="qk", pad=0, seed=0, positions=None, factor=4.0):
    gen = torch.Generator().manual_seed(seed)
    width = (hq + 2 * hkv) * hd
    s = dict(X=X, dtype=dtype, hq=hq, hkv=hkv, hd=hd, M=M, dm=C.dims(X, hq, hkv, hd, dtype, EPS))
    s["qkv"] = torch.randn(M, width + pad, generator=gen).cuda().to(C.DT[dtype])[:, :width]
    s["dout"] = torch.randn(M, (hq + hkv) * hd + pad, generator=gen).cuda().to(C.DT[dtype])[:, :(hq + hkv) * hd]
    s["gains"] = {n: (1 + 0.2 * torch.randn(hd, generator=gen)).cuda().to(C.DT[dtype]) for n in
                  (["q_norm"] if "q" in norm else []) + (["k_norm"] if "k" in norm else [])}
    s["w"] = X.layer_weights(s["gains"])
    s["rope"] = X.rope(hd, 1e4, rot_dim=rot, interleaved=inter, scaling=scaling, factor=factor, trained=1000)
    pos = torch.randint(0, 5000, (M,), generator=gen) if positions is None else torch.tensor(positions)
    s["pos"] = pos.to(torch.int32).cuda()
    return s


def _parts(s, t):
    """q and k heads of [M, (hq + hkv) hd] with their gain."""
    hq, hkv, hd = s["hq"], s["hkv"], s["hd"]
    x = t[:, :(hq + hkv) * hd].reshape(s["M"], hq + hkv, hd)
    return (x[:, :hq], s["gains"].get("q_norm")), (x[:, hq:], s["gains"].get("k_norm"))


def _check_forward(s, out, live=None):
    hd = s["hd"]
    # of the norm: the sum of squares (hd terms, halved by the root), its root and two products;
    # of the rotation: cosine and sine 1e-7 + 2e-9, three roundings; then the output's
    rel = (hd / 2 + 12) * 2.0 ** -24 + 1.02e-7
    for (x, gain), (y, _) in zip(_parts(s, s["qkv"]), _parts(s, out)):
        ref, size = R.rope_ref(x, gain, EPS, s["rope"], s["pos"])
        err = (y.double() - ref).abs() - size * rel - C.HALF[s["dtype"]] * (ref.abs() + size * rel)
        if live is not None:
            err = err[live]
        assert float(err.max()) <= 0, float(err.max())


def _check_backward(s, din, dq, dk, live=None):
    hd = s["hd"]
    rel = (hd + 24) * 2.0 ** -24 + 1.1e-7
    for (x, gain), (d, _), (y, _), dg in zip(_parts(s, s["qkv"]), _parts(s, s["dout"]), _parts(s, din), (dq, dk)):
        pos = s["pos"]
        if live is not None:
            x, d, y, pos = x[live], d[live], y[live], pos[live]
        ref, rg, size, terms = R.rope_grad_ref(x, gain, EPS, s["rope"], pos, d)
        err = (y.double() - ref).abs() - size * rel - C.HALF[s["dtype"]] * (ref.abs() + size * rel)
        assert float(err.max()) <= 0, float(err.max())
        if gain is not None and dg is not None:
            # fp32 sums over at most every token and head of the rounded terms
            eg = (dg.double() - rg).abs() - terms * (rel + x.shape[0] * x.shape[1] * 2.0 ** -24) - 2.0 ** -24 * rg.abs()
            assert float(eg.max()) <= 0, float(eg.max())


CASES = [
    # hq, hkv, hd, M, rot, interleaved, scaling, norm, pad
    (12, 4, 128, 37, 128, False, 0, "qk", 0), (12, 4, 128, 1, 64, True, 1, "qk", 8), (32, 8, 64, 300, 32, False, 2, "", 0),
    (4, 2, 32, 5, 8, False, 3, "qk", 16), (4, 2, 32, 9, 8, True, 3, "k", 0), (7, 1, 128, 64, 24, False, 0, "q", 0),
    (5, 5, 64, 33, 40, True, 2, "qk", 0), (16, 1, 128, 2000, 128, True, 3, "qk", 0), (3, 3, 32, 77, 32, False, 1, "qk", 8),
    (1, 1, 64, 3, 56, False, 0, "", 0), (32, 8, 128, 1111, 96, False, 3, "qk", 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES)
def test_forward(X, dtype, case):
    hq, hkv, hd, M, rot, inter, scaling, norm, pad = case
    s = _case(X, dtype, hq, hkv, hd, M, rot, inter, scaling, norm, pad)
    out = torch.full((M, (hq + hkv) * hd + pad), -3.0, dtype=C.DT[dtype], device="cuda")
    X.qk_rope(s["dm"], s["qkv"], s["w"], s["rope"], out, pos=s["pos"])
    _check_forward(s, out)
    assert bool((out[:, (hq + hkv) * hd:] == -3).all())
    # in place: the same bits, values untouched
    rows = s["qkv"].clone()
    X.qk_rope(s["dm"], rows, s["w"], s["rope"], rows, pos=s["pos"])
    n = (hq + hkv) * hd
    assert torch.equal(rows[:, :n], out[:, :n]) and torch.equal(rows[:, n:], s["qkv"][:, n:])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES)
def test_backward(X, dtype, case):
    hq, hkv, hd, M, rot, inter, scaling, norm, pad = case
    s = _case(X, dtype, hq, hkv, hd, M, rot, inter, scaling, norm, pad, seed=1)
    din = torch.full((M, (hq + hkv) * hd + pad), -3.0, dtype=C.DT[dtype], device="cuda")
    dq, dk = (torch.full((hd,), math.nan, device="cuda") if g in norm else None for g in "qk")
    ws = torch.full((X.qk_rope_bwd_workspace_bytes(s["dm"], M),), 0xff, dtype=torch.uint8, device="cuda")
    X.qk_rope_bwd(s["dm"], s["qkv"] if norm else None, s["w"], s["rope"], s["dout"], din, pos=s["pos"], dq_norm=dq,
                  dk_norm=dk, ws=ws if norm else None)
    _check_backward(s, din, dq, dk)
    n = (hq + hkv) * hd
    assert bool((din[:, n:] == -3).all())
    again = s["dout"].clone()       # in place, and with fewer gradients: the same bits
    X.qk_rope_bwd(s["dm"], s["qkv"] if norm else None, s["w"], s["rope"], again, again, pos=s["pos"])
    assert torch.equal(again[:, :n], din[:, :n])
    if norm == "qk":
        one = torch.empty_like(dk)
        X.qk_rope_bwd(s["dm"], s["qkv"], s["w"], s["rope"], s["dout"], again, pos=s["pos"], dk_norm=one, ws=ws)
        assert torch.equal(one, dk)


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_differences(X, inter):
    """din and the gains' gradients along random directions against central differences of the
    64-bit forward."""
    s = _case(X, "fp32", 4, 2, 64, 29, 48, inter, X.ROPE_PARTS, seed=3)
    din = torch.empty(29, 6 * 64, device="cuda")
    dq, dk = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    ws = torch.empty(X.qk_rope_bwd_workspace_bytes(s["dm"], 29), dtype=torch.uint8, device="cuda")
    X.qk_rope_bwd(s["dm"], s["qkv"], s["w"], s["rope"], s["dout"], din, pos=s["pos"], dq_norm=dq, dk_norm=dk, ws=ws)
    gen = torch.Generator().manual_seed(5)
    vx = torch.randn(29, 6, 64, generator=gen, dtype=torch.float64).cuda()
    vg = torch.randn(2, 64, generator=gen, dtype=torch.float64).cuda()

    def value(t):
        total = 0.0
        for i, ((x, gain), (d, _)) in enumerate(zip(_parts(s, s["qkv"]), _parts(s, s["dout"]))):
            v = vx[:, :4] if i == 0 else vx[:, 4:]
            y, _ = R.rope_ref(x.double() + t * v, gain.double() + t * vg[i], EPS, s["rope"], s["pos"])
            total += float((y * d.double()).sum())
        return total

    h = 1e-5
    want = (value(h) - value(-h)) / (2 * h)
    got = float((din.double().view(29, 6, 64) * vx).sum() + (dq.double() * vg[0]).sum() + (dk.double() * vg[1]).sum())
    # a sum of 11136 products of gradients of unit size off by 2e-5 each at most, with random
    # signs well below; differences off by h^2 times a third derivative of the same size
    assert abs(got - want) <= 2e-5 * math.sqrt(11136) * 4


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_padding_rows_and_own_positions(X, dtype):
    pos = [5, -1, 7, -2 ** 31, 0, 2 ** 17]
    s = _case(X, dtype, 4, 2, 64, 6, 64, False, positions=pos)
    live = torch.tensor([0, 2, 4, 5]).cuda()
    out = torch.full((6, 6 * 64), -3.0, dtype=C.DT[dtype], device="cuda")
    X.qk_rope(s["dm"], s["qkv"], s["w"], s["rope"], out, pos=s["pos"])
    _check_forward(s, out, live)
    assert bool((out[[1, 3]] == -3).all())
    s["qkv"][1] = math.nan          # of a padding row nothing is read
    s["dout"][3] = math.inf
    din = torch.full((6, 6 * 64), -3.0, dtype=C.DT[dtype], device="cuda")
    dq, dk = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    ws = torch.empty(X.qk_rope_bwd_workspace_bytes(s["dm"], 6), dtype=torch.uint8, device="cuda")
    X.qk_rope_bwd(s["dm"], s["qkv"], s["w"], s["rope"], s["dout"], din, pos=s["pos"], dq_norm=dq, dk_norm=dk, ws=ws)
    _check_backward(s, din, dq, dk, live)
    assert bool((din[[1, 3]] == -3).all())
    # no positions: row m is at m modulo T
    dm = X.dims(3, 4, 64, 4, 2, 64, 64, X.BF16 if dtype == "bf16" else X.FP32, EPS)
    s = _case(X, dtype, 4, 2, 64, 12, 64, True, positions=[m % 4 for m in range(12)])
    a, b = torch.empty_like(out[:0]).resize_(12, 6 * 64), torch.empty_like(out[:0]).resize_(12, 6 * 64)
    X.qk_rope(dm, s["qkv"], s["w"], s["rope"], a)
    X.qk_rope(dm, s["qkv"], s["w"], s["rope"], b, pos=s["pos"])
    assert torch.equal(a, b)


def test_rest_of_the_head_is_left_alone(X):
    """Infinities and NaN beyond the turning dimensions stay where they are."""
    s = _case(X, "bf16", 2, 1, 64, 1, 32, False, norm="", positions=[9])
    s["qkv"][0, 40] = math.inf
    s["qkv"][0, 41] = math.nan
    out = torch.empty(1, 3 * 64, dtype=torch.bfloat16, device="cuda")
    X.qk_rope(s["dm"], s["qkv"], s["w"], s["rope"], out, pos=s["pos"])
    assert torch.equal(out[0, 32:64].isnan(), s["qkv"][0, 32:64].isnan())
    assert torch.equal(out[0, 32:64].nan_to_num(1.0), s["qkv"][0, 32:64].nan_to_num(1.0))
    assert bool(out[0, :32].isfinite().all())


def test_as_the_append_turns(X):
    """Halves of the whole head without scaling are what the cache append writes."""
    hq, hkv, hd, M = 4, 2, 128, 50
    s = _case(X, "bf16", hq, hkv, hd, M, hd, False)
    c = C.Cache(X, [5000], hkv, hd, 16, "bf16")
    q = torch.empty(M, hq * hd, dtype=torch.bfloat16, device="cuda")
    slot = torch.arange(M, dtype=torch.int32, device="cuda")
    X.cache_append(s["dm"], c.handle, s["qkv"], X.layer_weights(s["gains"], rope_theta=1e4), torch.zeros_like(slot), slot,
                   s["pos"], q)
    out = torch.empty(M, (hq + hkv) * hd, dtype=torch.bfloat16, device="cuda")
    X.qk_rope(s["dm"], s["qkv"], s["w"], s["rope"], out, pos=s["pos"])
    # the same arithmetic but for the frequencies' last bits: at most a step of bf16 apart
    d = (out[:, :hq * hd].float() - q.float()).abs()
    assert bool((d <= 2.0 ** -7 * q.float().abs() + 1e-6).all()) and float((d > 0).float().mean()) < 0.01


def test_sums_over_many_tokens(X):
    """A large call's gains' gradients, twice the same bits, on a captured graph too."""
    s = _case(X, "bf16", 12, 4, 128, 20011, 128, False, seed=7)
    din = torch.empty(20011, 16 * 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(X.qk_rope_bwd_workspace_bytes(s["dm"], 20011), dtype=torch.uint8, device="cuda")
    dq, dk = torch.zeros(128, device="cuda"), torch.zeros(128, device="cuda")
    call = lambda: X.qk_rope_bwd(s["dm"], s["qkv"], s["w"], s["rope"], s["dout"], din, pos=s["pos"], dq_norm=dq,  # noqa: E731
                                 dk_norm=dk, ws=ws)
    call()
    a, b, c = dq.clone(), dk.clone(), din.clone()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    for t in (dq, dk, din):
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dq, a) and torch.equal(dk, b) and torch.equal(din, c)
    _check_backward(s, din, dq, dk)


def test_nothing(X):
    s = _case(X, "bf16", 4, 2, 64, 1, 64, False)
    none = torch.empty(0, 8 * 64, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(0, 6 * 64, dtype=torch.bfloat16, device="cuda")
    X.qk_rope(s["dm"], none, s["w"], s["rope"], out)
    dq, dk = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    ws = torch.full((X.qk_rope_bwd_workspace_bytes(s["dm"], 0),), 0xff, dtype=torch.uint8, device="cuda")
    X.qk_rope_bwd(s["dm"], none, s["w"], s["rope"], out, out, dq_norm=dq, dk_norm=dk, ws=ws)
    assert bool((dq == 0).all()) and bool((dk == 0).all())


def test_binding_refusals(X):
    s = _case(X, "bf16", 4, 2, 64, 5, 64, False)
    out = torch.empty(5, 6 * 64, dtype=torch.bfloat16, device="cuda")
    dq = torch.empty(64, device="cuda")
    ws = torch.empty(X.qk_rope_bwd_workspace_bytes(s["dm"], 5), dtype=torch.uint8, device="cuda")
    fwd = lambda **k: X.qk_rope(**{**dict(dm=s["dm"], qkv=s["qkv"], w=s["w"], rope=s["rope"], out=out, pos=s["pos"]), **k})  # noqa: E731
    bwd = lambda **k: X.qk_rope_bwd(**{**dict(dm=s["dm"], qkv=s["qkv"], w=s["w"], rope=s["rope"], dout=s["dout"],  # noqa: E731
                                              din=out, pos=s["pos"], dq_norm=dq, ws=ws), **k})
    wide = X.rope(128)
    for call, over in ((fwd, dict(qkv=s["qkv"].float())), (fwd, dict(out=out[:4])), (fwd, dict(out=out[:, :-8])),
                       (fwd, dict(pos=s["pos"].long())), (fwd, dict(pos=s["pos"][:4])), (fwd, dict(rope=wide)),
                       (fwd, dict(out=out.cpu())), (fwd, dict(w=X.layer_weights({"q_norm": s["gains"]["q_norm"].float()}))),
                       (fwd, dict(out=s["qkv"].view(-1)[:5 * 6 * 64].view(5, 6 * 64))),
                       (bwd, dict(qkv=None)), (bwd, dict(w=None)), (bwd, dict(dq_norm=dq[:32])),
                       (bwd, dict(dout=s["dout"].float())), (bwd, dict(din=s["qkv"]))):
        with pytest.raises(X.XmodError) as e:
            call(**over)
        assert e.value.status == X.ERR_INVALID_ARG, over.keys()
    for over in (dict(ws=None), dict(ws=ws[:64])):
        with pytest.raises(X.XmodError) as e:
            bwd(**over)
        assert e.value.status == X.ERR_WORKSPACE
