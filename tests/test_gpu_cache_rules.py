"""GPU: rules of the key/value cache at the edges of what a caller may pass: gains, code
bytes, scales of any sign and size, large queries, rows alone and in batches, pages past
32-bit offsets, pages outside the cache, far positions."""
import decimal
import math

import numpy as np
import pytest

from tests import _cache as C
from tests._gpu import need_gpu, torch

pytestmark = pytest.mark.gpu

KINDS = {"bf16": ("bf16", False), "fp32": ("fp32", False), "e4m3": ("bf16", True)}
P_ROUND = {"bf16": 2.0 ** -16, "fp32": 2.0 ** -24, "e4m3": 2.0 ** -11}   # the header's


@pytest.fixture(scope="module")
def X():
    need_gpu()
    from sparse_depth_token_gb300 import xmod
    xmod.load()
    return xmod


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def attend(X, c, q, seq, lens, hq, hd, dtype):
    dm = C.dims(X, hq, c.hkv, hd, dtype)
    M = len(lens)
    o = torch.full((M, hq * hd), -3.0, dtype=C.DT[dtype], device="cuda")
    lse = torch.full((M, hq), -3.0, device="cuda")
    ws = torch.zeros(X.cache_attention_workspace_bytes(dm, M), dtype=torch.uint8, device="cuda")
    X.cache_attention(dm, c.handle, q, ints(seq), ints(lens), o, ws, lse=lse)
    return o, lse, X.sync_status(ws)


# ------------------------------------------------------------------ gains

@pytest.mark.parametrize("which", ["q_norm", "k_norm"])
@pytest.mark.parametrize("layout", ["strided", "expanded"])
def test_gains_that_are_not_contiguous_are_refused(X, which, layout):
    """A kernel reads head_dim elements on end: a column of a matrix or one expanded element
    would be other values than the caller's."""
    hq, hkv, hd, M = 4, 2, 64, 3
    c = C.Cache(X, [16] * M, hkv, hd, 16, "bf16", fill=0.5)
    before = [t.clone() for t in c.tensors()]
    both = torch.stack([torch.ones(hd), torch.full((hd,), 5.0)], 1).cuda().bfloat16()
    gain = both[:, 0] if layout == "strided" else both[:1, 0].expand(hd)
    qkv = torch.ones(M, (hq + 2 * hkv) * hd, dtype=torch.bfloat16, device="cuda")
    q = torch.full((M, hq * hd), -3.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(X.XmodError) as e:
        X.cache_append(C.dims(X, hq, hkv, hd, "bf16"), c.handle, qkv, X.layer_weights({which: gain}), None,
                       ints([0] * M), None, q)
    assert e.value.status == X.ERR_INVALID_ARG
    assert bool((q == -3).all()) and all(torch.equal(a, b) for a, b in zip(before, c.tensors()))


# ------------------------------------------------------------------ code bytes

@pytest.mark.parametrize("hd", [32, 64, 128])
def test_e4m3_codes_are_the_quotients(X, hd):
    """Code bytes and scales of k and v (copied: no norm, no rotation) equal amax / 448 and
    the fp32 quotient x / scale rounded to e4m3, both computed on the host. bf16 values over
    a scale often lie exactly between two codes, where any other rounding of the quotient
    shows; heads from the smallest scales to the largest."""
    hkv, M = 4, 600
    g = torch.Generator().manual_seed(hd)
    x = torch.randn(M, 2 * hkv, hd, generator=g)
    x[:, :, 0] *= 1 + 2 * torch.rand(M, 2 * hkv, generator=g)
    # scales down to the smallest normal number and below it, and up to the largest
    size = torch.tensor([0.0] * 8 + [-121, -119.5, -118, -110, -90, -60, 60, 110, 123.0])
    x *= torch.exp2(size[torch.arange(M) % len(size)])[:, None, None]
    x[0, :, :] = 1.3671875      # 200 times the scale of 3.0625: between 192 and 208
    x[0, :, 1] = 3.0625
    x[1] = -0.0
    x = x.bfloat16()
    c = C.Cache(X, [M], hkv, hd, 16, "bf16", True, fill=1.0)
    qkv = torch.cat([torch.zeros(M, hkv, hd, dtype=torch.bfloat16), x], 1).reshape(M, -1).cuda()
    X.cache_append(C.dims(X, hkv, hkv, hd, "bf16"), c.handle, qkv, None, ints([0] * M), ints(list(range(M))))
    x = x.float()
    scale = x.abs().amax(-1) / torch.tensor(448.0)
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    by = torch.where(scale == 0, torch.full_like(scale, math.inf), scale)
    want = (x / by[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    assert want[0, 0, 2] == torch.tensor(192.0).to(torch.float8_e4m3fn).view(torch.uint8)
    assert 0 < int((scale == 0).sum()) < scale.numel() // 2
    pages = torch.tensor([c.place(0, i)[0] for i in range(M)]).cuda()
    offs = torch.arange(M).cuda() % c.page
    for n, name in enumerate(("k", "v")):
        code = getattr(c, name).view(torch.uint8)[pages, :, offs].cpu()
        sc = getattr(c, name + "_scale")[pages, :, offs].cpu()
        assert torch.equal(sc, scale[:, n * hkv:(n + 1) * hkv])
        off = code != want[:, n * hkv:(n + 1) * hkv]
        assert not bool(off.any()), (name, int(off.sum()), off.nonzero()[:4].tolist())


# ------------------------------------------------------------------ scales of e4m3 values

def _check_e4m3_rows(c, q, lens, o, lse, hq, hd):
    """Rows m over sequence m against 64 bits. Beside the errors of attention_ref, a weight
    p |scale| below 2^-28 of the row's largest (or of 2^-112) is held to half of f16's last
    step there: 2^-39 of a power of two at most twice the largest, times the codes."""
    for m, n in enumerate(lens):
        ref, rl, bound, dz = C.attention_ref(c, q[m].reshape(hq, hd), m, n, P_ROUND["e4m3"])
        spread = bound / (2 * dz + 2.0 ** -18 + P_ROUND["e4m3"])[:, None]
        rep = hq // c.hkv
        k = c.rows("k", m, n).repeat_interleave(rep, 0)
        qm = q[m].reshape(hq, hd).double()
        z = torch.einsum("hd,hnd->hn", qm, k) / math.sqrt(hd)
        w = torch.exp(z - z.amax(1, keepdim=True))
        # the error of the scores that count (attention_ref's is that of all)
        dz = torch.where(w > 2.0 ** -60, torch.einsum("hd,hnd->hn", qm.abs(), k.abs()), torch.zeros_like(w))
        dz = dz.amax(1) * math.sqrt(hd) * 2.0 ** -24
        pages = torch.from_numpy(c.table_np[m, :-(-n // c.page)].astype(np.int64)).cuda()
        sc = c.v_scale[pages].double().permute(1, 0, 2).reshape(c.hkv, -1)[:, :n].repeat_interleave(rep, 0)
        codes = c.v.view(torch.uint8)[pages].view(torch.float8_e4m3fn).double().abs()
        codes = codes.permute(1, 0, 2, 3).reshape(c.hkv, -1, hd)[:, :n].sum(1).repeat_interleave(rep, 0)
        largest = (w * sc.abs()).amax(1).clamp(min=2.0 ** -113)
        bound = spread * (2 * dz + 2.0 ** -18 + P_ROUND["e4m3"])[:, None] + (
            2.0 ** -38 * largest / w.sum(1))[:, None] * codes
        err = (o[m].view(hq, hd).double() - ref).abs() - bound - C.HALF["bf16"] * (ref.abs() + bound)
        assert float(err.max()) <= 0, (m, n, float(err.max()), float(ref.abs().max()))
        le = (lse[m].double() - rl).abs() - 2 * dz - 2.0 ** -18 - 2.0 ** -22 * rl.abs()
        assert float(le.max()) <= 0, (m, n, float(le.max()))


@pytest.mark.parametrize("hq,hkv,hd", [(12, 4, 128), (16, 1, 64), (2, 2, 32)])
@pytest.mark.parametrize("sign", ["all", "some"])
def test_negative_scales(X, hq, hkv, hd, sign):
    """A code stands for code * scale, whatever the scale's sign."""
    lens = [1, 64, 300, 1000]
    c = C.Cache(X, lens, hkv, hd, 16, "bf16", True)
    g = torch.Generator().manual_seed(5)
    for m, n in enumerate(lens):
        c.fill(m, n, m)
        for name in ("k_scale", "v_scale"):
            s = getattr(c, name)
            s *= -1.0 if sign == "all" else torch.where(torch.rand(s.shape, generator=g) < 0.5, -1.0, 1.0).cuda()
    q = torch.randn(len(lens), hq * hd, generator=g).cuda().bfloat16()
    o, lse, status = attend(X, c, q, range(len(lens)), lens, hq, hd, "bf16")
    assert status == X.OK
    _check_e4m3_rows(c, q, lens, o, lse, hq, hd)


@pytest.mark.parametrize("hq,hkv,hd", [(12, 4, 128), (16, 1, 64), (2, 2, 32)])
@pytest.mark.parametrize("pattern", ["rising", "falling", "outlier first", "outlier inside", "outlier last", "tiny",
                                     "huge", "mixed"])
def test_scales_of_all_sizes(X, hq, hkv, hd, pattern):
    """Value scales that span many powers of two along a sequence, and one key of nearly no
    probability (about 2^-200) with a scale 2^60 times the others': its scale must not cost
    the other keys' weights their bits."""
    lens = [70, 400, 2600]
    c = C.Cache(X, lens, hkv, hd, 32, "bf16", True)
    g = torch.Generator().manual_seed(6)
    q = torch.randn(len(lens), hq * hd, generator=g).abs().cuda().bfloat16()
    for m, n in enumerate(lens):
        c.fill(m, n, m)
        jitter = 0.5 + torch.rand(hkv, n, generator=g, dtype=torch.float64)
        steps = {"rising": lambda i: 60 * i / n - 30, "falling": lambda i: 30 - 60 * i / n,
                 "tiny": lambda i: 0 * i - 119, "huge": lambda i: 0 * i + 112,
                 "mixed": lambda i: 20 * torch.sin(i / 7)}.get(pattern, lambda i: 0 * i - 7)
        pages = torch.from_numpy(c.table_np[m, :-(-n // c.page)].astype(np.int64)).cuda()
        sc = torch.full((hkv, len(pages) * c.page), math.nan, dtype=torch.float64)
        sc[:, :n] = torch.exp2(steps(torch.arange(n, dtype=torch.float64))) * jitter
        c.v_scale[pages] = sc.view(hkv, -1, c.page).permute(1, 0, 2).float().cuda()
        if pattern.startswith("outlier"):
            at = {"first": 0, "inside": n // 2 + 3, "last": n - 1}[pattern.split()[1]]
            p, off = c.place(m, at)
            c.k[p, :, off] = torch.full((hkv, hd), -448.0, device="cuda").to(torch.float8_e4m3fn)
            # scores of about -150: the mean |q| is 0.8
            c.k_scale[p, :, off] = 150 / 448 / (0.8 * math.sqrt(hd))
            c.v_scale[p, :, off] = 2.0 ** 53
    o, lse, status = attend(X, c, q, range(len(lens)), lens, hq, hd, "bf16")
    assert status == X.OK
    assert bool(o.isfinite().all())
    _check_e4m3_rows(c, q, lens, o, lse, hq, hd)


@pytest.mark.parametrize("hq,hkv,hd", [(12, 4, 128), (16, 1, 64), (2, 2, 32)])
@pytest.mark.parametrize("kind", sorted(KINDS))
def test_queries_of_all_sizes(X, kind, hq, hkv, hd):
    """Queries from 2^-126 to 2^122, one element each: scores are one product, so that the
    largest of far apart ones takes all the weight, and tiny ones weight all keys alike."""
    dtype, e4m3 = KINDS[kind]
    n = 100
    lens = [n] * 6
    c = C.Cache(X, lens, hkv, hd, 16, dtype, e4m3)
    q = torch.zeros(len(lens), hq, hd)
    for m, size in enumerate((2.0 ** -126, 2.0 ** -104, 1.0, 2.0 ** 98, 2.0 ** 101, 2.0 ** 122)):
        c.fill(m, n, m)
        q[m, :, 5] = size
    for t in c.tensors():       # the keys' element 5: codes far apart, one scale
        if t is c.k:
            for m in range(len(lens)):
                for i in range(n):
                    p, off = c.place(m, i)
                    v = (8 + (i * 7 % n) // 8) * (1.0 if e4m3 else 0.125) if i % 8 == 0 else 1.0
                    c.k[p, :, off, 5] = torch.full((hkv,), v, device="cuda").to(c.k.dtype)
        elif t is c.k_scale:
            t.fill_(0.125)
    qd = q.view(len(lens), -1).cuda().to(C.DT[dtype])
    o, lse, status = attend(X, c, qd, range(len(lens)), lens, hq, hd, dtype)
    assert status == X.OK
    for m in range(len(lens)):
        ref, rl, bound, dz = C.attention_ref(c, qd[m].reshape(hq, hd), m, n, P_ROUND[kind])
        big = float(q[m].max()) > 2
        # one product: a score's relative error is that of its factors (rsqrt's 2 ulp, log2 e's
        # and ln 2's roundings and the products', 2^-21 in all); where the scores are far apart
        # none of it reaches the weights
        z = float(rl.abs().max())
        bound = bound / (2 * dz + 2.0 ** -18 + P_ROUND[kind])[:, None] * (
            2.0 ** -18 + P_ROUND[kind] + (0.0 if big else 2.0 ** -20))
        err = (o[m].view(hq, hd).double() - ref).abs() - bound - C.HALF[dtype] * (ref.abs() + bound)
        assert float(err.max()) <= 0, (m, float(err.max()))
        assert float((lse[m].double() - rl).abs().max()) <= 2.0 ** -17 + 2.0 ** -20 * z, m


def test_codes_of_another_8_bit_type_are_refused(X):
    """Codes are e4m3 or plain bytes of them; other 8-bit floating types would be misread."""
    shape = (4, 2, 16, 64)
    scale = torch.ones(shape[:3], device="cuda")
    table = ints([[0, 1], [2, 3]])
    for t in (torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz):
        x = torch.zeros(shape, dtype=torch.uint8, device="cuda").view(t)
        with pytest.raises(X.XmodError) as e:
            X.kv_cache(x, x.clone(), table, scale, scale.clone())
        assert e.value.status == X.ERR_INVALID_ARG
    for t in (torch.float8_e4m3fn, torch.uint8, torch.int8):
        x = torch.zeros(shape, dtype=torch.uint8, device="cuda").view(t)
        X.kv_cache(x, x.clone(), table, scale, scale.clone())


# ------------------------------------------------------------------ places

@pytest.mark.parametrize("kind", sorted(KINDS))
def test_append_past_32_bit_offsets(X, kind):
    """The slot that the append writes held NaN; k and v (copied), or their codes and scales,
    stand there afterwards and nothing beside them has changed."""
    dtype, e4m3 = KINDS[kind]
    hkv, hd, page, hq = 8, 128, 64, 16
    c = C.Cache(X, [200], hkv, hd, page, dtype, e4m3, first_page=(2 ** 32 + 2 ** 20) // (hkv * hd * page))
    assert c.k.numel() > 2 ** 32
    c.fill(0, 199, 7)
    pages = torch.from_numpy(c.table_np[0].astype(np.int64)).cuda()
    raw = lambda t: t.view(torch.uint8) if t.element_size() == 1 else t  # noqa: E731
    bits = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    before = [raw(t)[pages].clone() for t in c.tensors()]
    p, off = c.place(0, 199)
    assert not bool(c.k[p, :, off].double().isfinite().any())
    qkv = torch.randn(1, (hq + 2 * hkv) * hd, generator=torch.Generator().manual_seed(6)).cuda().to(C.DT[dtype])
    X.cache_append(C.dims(X, hq, hkv, hd, dtype), c.handle, qkv, None, None, ints([199]))
    for i, name in enumerate(("k", "v")):
        x = qkv[0, (hq + i * hkv) * hd:(hq + (i + 1) * hkv) * hd].view(hkv, hd)
        got = getattr(c, name)[p, :, off]
        if e4m3:
            x = x.float().cpu()
            scale = x.abs().amax(-1) / torch.tensor(448.0)
            assert torch.equal(getattr(c, name + "_scale")[p, :, off].cpu(), scale)
            x = (x / scale[:, None]).to(torch.float8_e4m3fn)
        assert torch.equal(bits(got.cpu()), bits(x.cpu()))
    at = c.table_np[0].tolist().index(p)
    for t, b in zip(c.tensors(), before):
        now = raw(t)[pages].clone()
        now[at, :, off] = b[at, :, off]
        assert torch.equal(bits(now), bits(b))


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("page", [16, 64])
def test_pages_outside_the_cache_are_read_as_page_0(X, kind, page):
    """The same bits as with the entry 0 in the table, and a report; rows that do not need
    the entry are not touched by it."""
    dtype, e4m3 = KINDS[kind]
    hq, hkv, hd, n = 8, 2, 64, 3 * page - 5
    c = C.Cache(X, [3 * page, 3 * page], hkv, hd, page, dtype, e4m3)
    for s in range(2):
        c.fill(s, 3 * page, s)
    first = int(c.table_np[0, 0])       # its place becomes page 0's: every page read holds numbers
    for t in c.tensors():
        t = t.view(torch.uint8) if t.element_size() == 1 else t
        t[0] = t[first]
    q = torch.randn(2, hq * hd, generator=torch.Generator().manual_seed(5)).cuda().to(C.DT[dtype])
    c.table[0, 1] = 0
    want = attend(X, c, q, [0, 1], [n, n], hq, hd, dtype)
    assert want[2] == X.OK and bool(want[0].isfinite().all())
    for bad in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        c.table[0, 1] = bad
        got = attend(X, c, q, [0, 1], [n, n], hq, hd, dtype)
        assert got[2] == X.ERR_DEVICE_CHECK
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert attend(X, c, q, [0, 1], [page, n], hq, hd, dtype)[2] == X.OK


# ------------------------------------------------------------------ alone and in a batch

@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("hq,hkv,hd", [(12, 4, 128), (16, 1, 64)])
def test_rows_alone_and_in_batches(X, kind, hq, hkv, hd):
    """The other rows of a call move the borders of the split, and with them the maximum that
    a weight is rounded against: the same row alone and in batches differs by the weights'
    stated rounding on both sides (and fp32's) at most."""
    dtype, e4m3 = KINDS[kind]
    lens = [700, 64, 3000, 129, 1, 1500]
    M = len(lens)
    c = C.Cache(X, lens, hkv, hd, 16, dtype, e4m3)
    for m, n in enumerate(lens):
        c.fill(m, n, m, 2.0)
    q = torch.randn(M, hq * hd, generator=torch.Generator().manual_seed(9)).cuda().to(C.DT[dtype])
    runs = []
    for rows in [[m] for m in range(M)] + [[0, 1], [2, 3], [4, 5], [1, 2, 3], list(range(M)), [2] * 9 + [0, 5] * 4]:
        o, lse, status = attend(X, c, q[rows], rows, [lens[m] for m in rows], hq, hd, dtype)
        assert status == X.OK
        runs.append((rows, o.double(), lse.double()))
    for m, n in enumerate(lens):
        ref, rl, bound, dz = C.attention_ref(c, q[m].reshape(hq, hd), m, n, P_ROUND[kind])
        spread = bound / (2 * dz + 2.0 ** -18 + P_ROUND[kind])[:, None]
        seen = [(o[i].view(hq, hd), lse[i]) for rows, o, lse in runs for i, r in enumerate(rows) if r == m]
        assert len(seen) >= 3
        for o, lse in seen[1:]:
            # fp32's part: exp and the sums, 2^-18 on either side; the scores are the same bits
            tol = spread * 2 * (P_ROUND[kind] + 2.0 ** -18) + C.HALF[dtype] * (o.abs() + seen[0][0].abs())
            assert bool(((o - seen[0][0]).abs() <= tol).all()), m
            assert float((lse - seen[0][1]).abs().max()) <= 2.0 ** -17 + 2.0 ** -22 * float(rl.abs().max()), m


# ------------------------------------------------------------------ rotation

def _turns(theta, hd, pos):
    """pos theta^(-2c/hd) / 2 pi modulo 1 for c < hd / 2, from 60-digit arithmetic."""
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        pi = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494")
        out = []
        for c in range(hd // 2):
            f = (decimal.Decimal(-2 * c) / hd * decimal.Decimal(theta).ln()).exp() / (2 * pi)
            out.append([float(pos_ * f % 1) for pos_ in map(decimal.Decimal, pos)])
    return torch.tensor(out, dtype=torch.float64).T


@pytest.mark.parametrize("theta", [1.0, 10.0, 1e4, 1e6])
@pytest.mark.parametrize("hd", [32, 128])
def test_rotation_against_long_arithmetic(X, theta, hd):
    """Angles are within 2^-52 turns times the position of the definition's, beside fp32."""
    pos = [0, 1, 3, 4097, 131071, 2 ** 24 - 1, 99999989, 2 ** 31 - 1]
    M, hq = len(pos), 2
    c = C.Cache(X, [16] * M, 1, hd, 16, "fp32", fill=0.5)
    x = torch.randn(M, (hq + 2) * hd, generator=torch.Generator().manual_seed(4))
    q = torch.empty(M, hq * hd, device="cuda")
    X.cache_append(C.dims(X, hq, 1, hd, "fp32"), c.handle, x.cuda(), X.layer_weights({}, rope_theta=theta), None,
                   ints([3] * M), ints(pos), q)
    turns = _turns(theta, hd, pos) * (2 * math.pi)
    cs, sn = turns.cos()[:, None], turns.sin()[:, None]
    h = x.double().view(M, hq + 2, hd)[:, :hq]
    a, b = h[..., :hd // 2], h[..., hd // 2:]
    want = torch.cat([a * cs - b * sn, b * cs + a * sn], -1)
    size = (a.abs() + b.abs()).repeat(1, 1, 2)
    off = 2 * math.pi * 2.0 ** -52 * torch.tensor(pos, dtype=torch.float64)[:, None, None]
    # fp32: the angle, its sine and cosine, two products and their sum (8 steps of the pair)
    tol = size * (8 * 2.0 ** -24 + off) + C.HALF["fp32"] * want.abs()
    err = (q.view(M, hq, hd).double().cpu() - want).abs() - tol
    assert float(err.max()) <= 0, (err.amax((1, 2)).tolist())


# ------------------------------------------------------------------ bits of the weights

@pytest.mark.parametrize("hq,hkv,hd", [(4, 4, 128), (8, 1, 64), (6, 2, 32)])
def test_e4m3_weights_keep_22_bits(X, hq, hkv, hd):
    """Two keys whose weighted values cancel: codes 8 and -9 (and multiples), with the second
    value's scale set so that p1 s1 8 = p2 s2 9 to fp32. What is left of o is the weights'
    rounding, 2^-22 each with at most 8 query heads per KV head, and fp32's."""
    M, rep = 150, hq // hkv
    g = torch.Generator().manual_seed(hd)
    c = C.Cache(X, [2] * M, hkv, hd, 16, "bf16", True)
    k = torch.zeros(M, hkv, 2, hd)
    k[..., 3] = torch.randint(8, 16, (M, hkv, 2), generator=g).float()
    v = torch.exp2(torch.randint(-3, 4, (M, hkv, 1, hd), generator=g).float()) * torch.tensor([8.0, -9.0])[:, None]
    v = v * torch.where(torch.rand(M, hkv, 1, hd, generator=g) < 0.5, -1.0, 1.0)
    ks = 0.05 + 0.1 * torch.rand(M, hkv, 2, generator=g)
    q = torch.zeros(M, hkv, 1, hd)
    q[..., 3] = (0.5 + torch.rand(M, hkv, 1, generator=g)).bfloat16().float() * math.sqrt(hd) / 8
    q = q.expand(M, hkv, rep, hd).reshape(M, hq * hd).cuda().bfloat16()
    z = q.view(M, hkv, rep, hd)[:, :, 0, 3].double().cpu()[..., None] * k[..., 3].double() * ks.double() / math.sqrt(hd)
    p = torch.softmax(z, -1)
    vs = torch.rand(M, hkv, 2, generator=g, dtype=torch.float64) + 0.5
    vs[..., 1] = vs[..., 0] * p[..., 0] * 8 / (p[..., 1] * 9)
    for m in range(M):
        page, off = c.place(m, 0)
        for name, x, s in (("k", k, ks), ("v", v, vs)):
            getattr(c, name)[page, :, off:off + 2] = x[m].cuda().to(torch.float8_e4m3fn)
            getattr(c, name + "_scale")[page, :, off:off + 2] = s[m].float().cuda()
    o, lse, status = attend(X, c, q, range(M), [2] * M, hq, hd, "bf16")
    assert status == X.OK
    for m in range(M):
        ref, rl, bound, dz = C.attention_ref(c, q[m].reshape(hq, hd), m, 2, 2.0 ** -22)
        err = (o[m].view(hq, hd).double() - ref).abs() - bound - C.HALF["bf16"] * (ref.abs() + bound)
        assert float(err.max()) <= 0, (m, float(err.max()), float(bound.max()))
