"""GPU: appending to the paged key/value cache and the attention of single tokens over it,
against plain 64-bit forms: types, head layouts, lengths, pages, padded rows, shared
sequences, refused rows, streams, graphs and a cache past 32-bit offsets; and the two
together token by token against a whole layer."""
import math

import numpy as np
import pytest

from sparse_depth_token_gb300 import inputs as I
from tests import _cache as C
from tests import _util as U
from tests._gpu import dev_layer, from_dev, need_gpu, to_dev, torch, workspace, xmod_dims

pytestmark = pytest.mark.gpu

THETA = 1e4
KINDS = {"bf16": ("bf16", False), "fp32": ("fp32", False), "e4m3": ("bf16", True)}


@pytest.fixture(scope="module")
def X():
    need_gpu()
    from sparse_depth_token_gb300 import xmod
    xmod.load()
    return xmod


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append

def _append_case(X, kind, hq, hkv, hd, page, M, norm, theta, pad=0, seed=0):
    dtype, e4m3 = KINDS[kind]
    r = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    n_seqs, room = 5, 3 * page
    flat = r.permutation(n_seqs * room)[:M]
    assert len(flat) == M
    seq, slot = flat // room, flat % room
    c = C.Cache(X, [room] * n_seqs, hkv, hd, page, dtype, e4m3, fill=0.5)
    width = (hq + 2 * hkv) * hd
    qkv = torch.randn(M, width + pad, generator=g).cuda().to(C.DT[dtype])[:, :width]
    pos = ints((slot * 7 + seq).tolist())
    gains = {}
    if norm:
        for i, n in enumerate(("q_norm", "k_norm")):
            gains[n] = (1 + 0.2 * torch.randn(hd, generator=g)).cuda().to(C.DT[dtype])
    w = X.layer_weights(gains, rope_theta=theta)
    return dtype, c, qkv, seq, slot, pos, gains, w


def _check_append(c, dtype, qkv, seq, slot, pos, gains, theta, q_out, hq, hkv, hd, live, before):
    """Live rows hold the transformed values, every other slot and row what it held."""
    M = qkv.shape[0]
    x = qkv.reshape(M, hq + 2 * hkv, hd) if qkv.is_contiguous() else qkv.contiguous().view(
        M, hq + 2 * hkv, hd)
    q, qs = C.transform_ref(x[:, :hq], gains.get("q_norm"), 1e-6, theta, pos)
    k, ks = C.transform_ref(x[:, hq:hq + hkv], gains.get("k_norm"), 1e-6, theta, pos)
    v, vs = x[:, hq + hkv:].double(), x[:, hq + hkv:].double().abs()
    lv = torch.tensor(live).cuda()
    # fp32: the norm's sum and root (16 steps), the angle, its sine and the two products
    # (8 steps of the pair's size); then the rounding to the stored type
    fp32 = 32 * 2.0 ** -24
    if q_out is not None:
        got = q_out.reshape(M, hq, hd).double()
        err = (got - q).abs() - fp32 * qs - C.HALF[dtype] * (q.abs() + fp32 * qs)
        assert float(err[lv].max()) <= 0, float(err[lv].max())
        assert bool((q_out.reshape(M, hq, hd)[~lv] == -3.0).all())
    pages = torch.tensor([c.place(int(s), int(i))[0] if ok else 0 for s, i, ok in
                          zip(seq, slot, live)]).cuda()
    offs = torch.tensor([int(i) % c.page if ok else 0 for i, ok in zip(slot, live)]).cuda()
    for name, ref, size in (("k", k, ks), ("v", v, vs)):
        t = getattr(c, name)
        rows = (t.view(torch.uint8) if c.e4m3 else t)[pages, :, offs]
        if c.e4m3:
            sc = getattr(c, name + "_scale")[pages, :, offs].double()
            want = ref.abs().amax(-1) / C.E4M3_MAX
            assert float(((sc - want).abs() - 2 * fp32 * size.amax(-1) / C.E4M3_MAX)[lv].max()) <= 0
            got = rows.view(t.dtype).double() * sc[..., None]
            # half a step of a normal code, or of the subnormal codes' spacing 2^-9
            half = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * want[..., None])
            err = (got - ref).abs() - half * (1 + 2.0 ** -16) - 2 * fp32 * size
        else:
            err = (rows.double() - ref).abs() - C.HALF[dtype] * (ref.abs() + fp32 * size) - (
                fp32 * size if name == "k" else 0)
        assert float(err[lv].max()) <= 0, (name, float(err[lv].max()))
    for t, b in zip(c.tensors(), before):
        t, b = (u.view(torch.uint8) if u.element_size() == 1 else u for u in (t, b))
        t = t.clone()
        t[pages[lv], :, offs[lv]] = b[pages[lv], :, offs[lv]]
        assert torch.equal(t, b), "a slot outside the call's changed"


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("hq,hkv,hd,page,M,norm,theta,pad", [
    (4, 2, 32, 16, 1, True, THETA, 0),
    (12, 4, 128, 16, 37, True, THETA, 0),
    (16, 1, 64, 48, 100, False, THETA, 8),
    (32, 8, 128, 64, 203, True, 0.0, 24),
    (3, 3, 128, 32, 9, False, 0.0, 0),
    (5, 5, 64, 16, 240, True, 1e6, 0),
])
def test_append_matches_the_plain_form(X, kind, hq, hkv, hd, page, M, norm, theta, pad):
    dtype, c, qkv, seq, slot, pos, gains, w = _append_case(X, kind, hq, hkv, hd, page, M, norm,
                                                           theta, pad)
    before = [t.clone() for t in c.tensors()]
    live = [(m % 5) != 3 for m in range(M)]
    seq_in = ints([int(s) if ok else -1 - m for m, (s, ok) in enumerate(zip(seq, live))])
    q_out = torch.full((M, hq * hd), -3.0, dtype=C.DT[dtype], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    X.cache_append(C.dims(X, hq, hkv, hd, dtype), c.handle, qkv, w, seq_in, ints(slot.tolist()),
                   pos, q_out, status=status)
    assert int(status) == 0
    _check_append(c, dtype, qkv, seq, slot, pos, gains, theta, q_out, hq, hkv, hd, live, before)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_append_in_place_defaults_and_no_q(X, kind):
    """seq and pos NULL: row m is sequence m at its slot; q in place; q not wanted."""
    dtype, e4m3 = KINDS[kind]
    hq, hkv, hd, page, M = 12, 4, 128, 16, 5
    slot = [0, 17, 31, 47, 16]
    qkv = torch.randn(M, (hq + 2 * hkv) * hd, generator=torch.Generator().manual_seed(3)).cuda().to(
        C.DT[dtype])
    w = X.layer_weights({}, rope_theta=THETA)
    dm = C.dims(X, hq, hkv, hd, dtype)
    outs = []
    for mode in ("apart", "place", "none"):
        c = C.Cache(X, [48] * M, hkv, hd, page, dtype, e4m3, fill=0.5)
        before = [t.clone() for t in c.tensors()]
        rows = qkv.clone()
        q_out = (torch.empty(M, hq * hd, dtype=rows.dtype, device="cuda") if mode == "apart" else
                 rows[:, :hq * hd] if mode == "place" else None)
        X.cache_append(dm, c.handle, rows, w, None, ints(slot), None, q_out)
        _check_append(c, dtype, qkv, range(M), np.array(slot), ints(slot), {}, THETA,
                      None if q_out is None else q_out.contiguous(), hq, hkv, hd, [True] * M, before)
        assert torch.equal(rows[:, hq * hd:], qkv[:, hq * hd:])
        outs.append([t.view(torch.uint8) for t in c.tensors()]
                    + ([q_out.contiguous()] if q_out is not None else []))
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[1]))
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[2]))


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_append_far_positions(X, kind):
    """Angles at positions up to 2^31 - 1, where an fp32 product of position and frequency
    has no correct digit left. theta 2^20 makes the frequencies exact powers of 2^(-40/hd)."""
    dtype, e4m3 = KINDS[kind]
    hq, hkv, hd, page = 2, 1, 128, 16
    pos = [0, 1, 4097, 16777217, 999999937, 2 ** 31 - 1]
    M = len(pos)
    c = C.Cache(X, [page] * M, hkv, hd, page, dtype, e4m3, fill=0.5)
    qkv = torch.randn(M, 4 * hd, generator=torch.Generator().manual_seed(4)).cuda().to(C.DT[dtype])
    q_out = torch.empty(M, hq * hd, dtype=qkv.dtype, device="cuda")
    X.cache_append(C.dims(X, hq, hkv, hd, dtype), c.handle, qkv, X.layer_weights({}, rope_theta=2.0 ** 20),
                   None, ints([3] * M), ints(pos), q_out)
    q, size = C.transform_ref(qkv.view(M, 4, hd)[:, :hq], None, 0, 2.0 ** 20, ints(pos))
    # beyond the rounding steps: a frequency in double is off by 2^-51 relative in the
    # kernel's table and in the reference each, times 2^31 radians
    tol = (32 * 2.0 ** -24 + 2.0 ** -19) * size + C.HALF[dtype] * q.abs() * (1 + 2.0 ** -8)
    assert bool(((q_out.view(M, hq, hd).double() - q).abs() <= tol).all())


def test_append_e4m3_edges(X):
    """Heads of zeros, of one value, tiny ones, and with infinities or NaN."""
    hq, hkv, hd = 1, 6, 128
    x = torch.zeros(1, hq + 2 * hkv, hd)
    x[0, 2, 5] = 3.0                # one value: its code is 448
    x[0, 3] = 1e-37                 # below the smallest scale
    x[0, 4] = torch.linspace(-1, 1, hd)
    x[0, 5, 7] = math.inf
    x[0, 6, 9] = math.nan
    x[0, 7:] = x[0, 1:7]
    c = C.Cache(X, [16], hkv, hd, 16, "bf16", True, fill=1.0)
    X.cache_append(C.dims(X, 6, 6, hd, "bf16"), c.handle,
                   torch.cat([x[:, :1].repeat(1, 6, 1), x[:, 1:]], 1).view(1, -1).cuda().bfloat16(), None, None, ints([0]))
    p, o = c.place(0, 0)
    for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        code, scale = t[p, :, o].float().cpu(), s[p, :, o].cpu()
        assert scale[0] == 0 and bool((code[0] == 0).all())
        assert code[1, 5] == 448 and scale[1] == np.float32(3.0) / np.float32(448) and code[1].sum() == 448
        assert scale[2] == 0 and bool((code[2] == 0).all())
        assert float(code[3].abs().max()) == 448
        assert math.isnan(scale[4]) and bool(code[4].isnan().all())
        assert math.isnan(scale[5]) and bool(code[5].isnan().all())


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_append_skips_and_reports_bad_rows(X, kind):
    dtype, e4m3 = KINDS[kind]
    hq, hkv, hd, page = 4, 2, 64, 16
    rooms = [32, 16]            # sequence 1's second page is -1 in the table
    dm = C.dims(X, hq, hkv, hd, dtype)
    for seq, slot in ((2, 0), (0, 32), (0, -1), (1, 16)):
        c = C.Cache(X, rooms, hkv, hd, page, dtype, e4m3, fill=0.5)
        before = [t.clone() for t in c.tensors()]
        qkv = torch.ones(2, (hq + 2 * hkv) * hd, device="cuda", dtype=C.DT[dtype])
        q_out = torch.full((2, hq * hd), -3.0, device="cuda", dtype=C.DT[dtype])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        X.cache_append(dm, c.handle, qkv, None, ints([0, seq]), ints([5, slot]), None, q_out, status=status)
        assert int(status) == X.ERR_DEVICE_CHECK
        _check_append(c, dtype, qkv, [0, seq], np.array([5, 0]), ints([5, 0]), {}, 0.0, q_out, hq, hkv, hd,
                      [True, False], before)


def test_append_nothing(X):
    c = C.Cache(X, [16], 2, 64, 16, "bf16")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    X.cache_append(C.dims(X, 4, 2, 64, "bf16"), c.handle,
                   torch.empty(0, 8 * 64, dtype=torch.bfloat16, device="cuda"), None, none, none)


# ------------------------------------------------------------------ attention

def _p_round(kind):
    """The stated rounding of the probabilities."""
    return {"bf16": 2.0 ** -16, "fp32": 2.0 ** -24, "e4m3": 2.0 ** -11}[kind]


def _check_attention(c, kind, q, seq, lens, o, lse, hq, hd):
    dtype = KINDS[kind][0]
    for m, (s, n) in enumerate(zip(seq, lens)):
        got, gl = o[m].view(hq, hd).double(), lse[m].double()
        if s < 0:
            assert bool((o[m] == -3).all()) and bool((lse[m] == -3).all()), m
            continue
        if n == 0:
            assert bool((o[m] == 0).all()) and bool((lse[m] == -math.inf).all()), m
            continue
        ref, rl, bound, dz = C.attention_ref(c, q[m].reshape(hq, hd), s, n, _p_round(kind))
        err = (got - ref).abs() - bound - C.HALF[dtype] * (ref.abs() + bound)
        assert float(err.max()) <= 0, (m, n, float(err.max()))
        # lse: the scores' error, and the sum's and the logarithm's (relative 2^-18, 2^-22)
        le = (gl - rl).abs() - 2 * dz - 2.0 ** -18 - 2.0 ** -22 * rl.abs()
        assert float(le.max()) <= 0, (m, n, float(le.max()))


LENS = [1, 0, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 200, 333, 1000, 2, 3]


def _attention(X, kind, hq, hkv, hd, page, lens, seq=None, pad=0, seed=1, scale=1.0):
    dtype, e4m3 = KINDS[kind]
    n_seqs = len(lens) if seq is None else max(seq) + 1
    rooms = [0] * n_seqs
    for s, n in zip(range(n_seqs) if seq is None else seq, lens):
        if s >= 0:
            rooms[s] = max(rooms[s], n)
    c = C.Cache(X, rooms, hkv, hd, page, dtype, e4m3, seed=seed)
    for s, n in enumerate(rooms):
        if n:
            c.fill(s, n, seed + s, scale)
    M = len(lens)
    q = (torch.randn(M, hq * hd + pad, generator=torch.Generator().manual_seed(seed + 99)) * scale).cuda().to(
        C.DT[dtype])[:, :hq * hd]
    dm = C.dims(X, hq, hkv, hd, dtype)
    o = torch.full((M, hq * hd), -3.0, dtype=C.DT[dtype], device="cuda")
    lse = torch.full((M, hq), -3.0, device="cuda")
    ws = torch.full((X.cache_attention_workspace_bytes(dm, M),), 0x7f, dtype=torch.uint8, device="cuda")
    X.reset_status(ws)
    call = lambda: X.cache_attention(dm, c.handle, q, None if seq is None else ints(seq), ints(lens), o, ws,  # noqa: E731
                                     lse=lse)
    return c, q, o, lse, ws, call


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("hq,hkv,hd,page", [
    (12, 4, 128, 16), (32, 8, 128, 64), (16, 1, 128, 32), (24, 1, 64, 16), (4, 2, 32, 16),
    (8, 8, 64, 128), (9, 1, 32, 48), (36, 2, 128, 16)])
def test_attention_matches_the_plain_form(X, kind, hq, hkv, hd, page):
    """Lengths around every tile and page border, none and one; unused slots hold NaN."""
    c, q, o, lse, ws, call = _attention(X, kind, hq, hkv, hd, page, LENS, pad=8)
    call()
    assert X.sync_status(ws) == X.OK
    _check_attention(c, kind, q, range(len(LENS)), LENS, o, lse, hq, hd)
    first = o.clone(), lse.clone()
    call()
    assert torch.equal(first[0], o) and torch.equal(first[1], lse)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_attention_rows_share_skip_and_repeat_sequences(X, kind):
    """Several new tokens of one sequence, each with its own length, and padding rows."""
    seq = [2, 0, -1, 2, 2, 1, -7, 0]
    lens = [300, 40, 5, 299, 298, 77, 0, 40]
    c, q, o, lse, ws, call = _attention(X, kind, 12, 4, 128, 32, lens, seq)
    call()
    assert X.sync_status(ws) == X.OK
    _check_attention(c, kind, q, seq, lens, o, lse, 12, 128)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("M,n", [(1, 20000), (2, 4999), (700, 90), (300, 1)])
def test_attention_long_and_wide(X, kind, M, n):
    lens = [max(1, n - (m * 37) % (n // 2 + 1)) for m in range(M)]
    c, q, o, lse, ws, call = _attention(X, kind, 16, 4, 128, 64, lens)
    call()
    assert X.sync_status(ws) == X.OK
    sample = sorted(set([0, M - 1] + list(range(0, M, 23))))
    _check_attention(c, kind, q[sample], sample, [lens[m] for m in sample], o[sample], lse[sample], 16, 128)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_attention_large_scores(X, kind):
    """Scores in the hundreds: one key takes nearly all the weight."""
    c, q, o, lse, ws, call = _attention(X, kind, 12, 4, 128, 16, [500, 65, 64, 1], scale=8.0)
    call()
    _check_attention(c, kind, q, range(4), [500, 65, 64, 1], o, lse, 12, 128)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_attention_reports_bad_rows(X, kind):
    """A sequence past the table skips its row; a length past the table or below 0 is
    clamped; a page outside the cache is read as page 0. All are reported, the other rows
    hold."""
    hq, hkv, hd, page = 8, 2, 64, 16
    for seq, n in ((3, 5), (0, 10 ** 6), (0, -4), (1, 20)):
        lens = [40, 30, 16, n]
        dtype, e4m3 = KINDS[kind]
        c = C.Cache(X, [48, 16, 16], hkv, hd, page, dtype, e4m3, fill=0.25)
        c.table_np[1, 1:] = -1
        c.table_np[0, 2] = c.table_np[0, 2]
        for s, k in enumerate((48, 16, 16)):
            c.fill(s, k, s)
        dm = C.dims(X, hq, hkv, hd, dtype)
        q = torch.randn(4, hq * hd, generator=torch.Generator().manual_seed(5)).cuda().to(C.DT[dtype])
        o = torch.full((4, hq * hd), -3.0, dtype=C.DT[dtype], device="cuda")
        lse = torch.full((4, hq), -3.0, device="cuda")
        ws = torch.zeros(X.cache_attention_workspace_bytes(dm, 4), dtype=torch.uint8, device="cuda")
        seqs = [0, 0, 2, seq]
        X.cache_attention(dm, c.handle, q, ints(seqs), ints(lens), o, ws, lse=lse)
        assert X.sync_status(ws) == X.ERR_DEVICE_CHECK
        good = seqs[:3] + ([-1] if seq == 3 else [])
        _check_attention(c, kind, q, good, lens, o, lse, hq, hd)
        if seq == 0:
            _check_attention(c, kind, q[3:], [0], [48 if n > 0 else 0], o[3:], lse[3:], hq, hd)


def test_attention_nothing(X):
    c = C.Cache(X, [16], 2, 64, 16, "bf16")
    dm = C.dims(X, 4, 2, 64, "bf16")
    none = torch.empty(0, 4 * 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(X.cache_attention_workspace_bytes(dm, 0), dtype=torch.uint8, device="cuda")
    X.cache_attention(dm, c.handle, none, None, torch.empty(0, dtype=torch.int32, device="cuda"), none, ws)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_cache_past_32_bit_offsets(X, kind):
    """Pages whose element and byte offsets pass 2^31 and 2^32."""
    dtype, e4m3 = KINDS[kind]
    hkv, hd, page, hq = 8, 128, 64, 16
    first = (2 ** 32 + 2 ** 20) // (hkv * hd * page)
    c = C.Cache(X, [200], hkv, hd, page, dtype, e4m3, first_page=first)
    assert c.k.numel() > 2 ** 32
    c.fill(0, 200, 7)
    dm = C.dims(X, hq, hkv, hd, dtype)
    qkv = torch.randn(1, (hq + 2 * hkv) * hd, generator=torch.Generator().manual_seed(6)).cuda().to(C.DT[dtype])
    q = torch.empty(1, hq * hd, dtype=C.DT[dtype], device="cuda")
    X.cache_append(dm, c.handle, qkv, None, None, ints([199]), None, q)
    p, off = c.place(0, 199)
    if not e4m3:
        assert torch.equal(c.v[p, :, off].reshape(-1), qkv[0, -hkv * hd:])
    o = torch.empty_like(q)
    lse = torch.empty(1, hq, device="cuda")
    ws = torch.zeros(X.cache_attention_workspace_bytes(dm, 1), dtype=torch.uint8, device="cuda")
    X.cache_attention(dm, c.handle, q, None, ints([200]), o, ws, lse=lse)
    assert X.sync_status(ws) == X.OK
    _check_attention(c, kind, q, [0], [200], o, lse, hq, hd)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("kind", sorted(KINDS))
def test_captured_steps_replay(X, kind):
    """Append and attention recorded once and replayed for later tokens: slots, lengths and
    inputs change in their buffers, with a second captured pair (own workspace) beside it
    and a side stream."""
    dtype, e4m3 = KINDS[kind]
    hq, hkv, hd, page, M, T = 12, 4, 128, 16, 3, 70
    dm = C.dims(X, hq, hkv, hd, dtype)
    w = X.layer_weights({}, rope_theta=THETA)
    gen = torch.Generator().manual_seed(8)
    data = torch.randn(2, T, M, (hq + 2 * hkv) * hd, generator=gen).cuda().to(C.DT[dtype])
    sets = []
    stream = torch.cuda.Stream()
    for i in range(2):
        c = C.Cache(X, [T] * M, hkv, hd, page, dtype, e4m3, seed=i)
        s = dict(c=c, qkv=data[i, 0].clone(), slot=ints([0] * M), n=ints([1] * M),
                 q=torch.zeros(M, hq * hd, dtype=C.DT[dtype], device="cuda"))
        s["o"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(M, hq, device="cuda")
        s["ws"] = torch.zeros(X.cache_attention_workspace_bytes(dm, M), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"], stream=stream):
            X.cache_append(dm, c.handle, s["qkv"], w, None, s["slot"], None, s["q"])
            X.cache_attention(dm, c.handle, s["q"], None, s["n"], s["o"], s["ws"], lse=s["lse"])
        sets.append(s)
    for t in range(T):
        for i, s in enumerate(sets):
            s["qkv"].copy_(data[i, t])
            s["slot"].fill_(t)
            s["n"].fill_(t + 1)
            s["graph"].replay()
    torch.cuda.synchronize()
    for i, s in enumerate(sets):
        _check_attention(s["c"], kind, s["q"], range(M), [T] * M, s["o"], s["lse"], hq, hd)
        o, lse = s["o"].clone(), s["lse"].clone()
        with torch.cuda.stream(stream):     # the eager call on another stream gives the same bits
            X.cache_attention(dm, s["c"].handle, s["q"], None, s["n"], s["o"], s["ws"], lse=s["lse"])
        stream.synchronize()
        assert torch.equal(o, s["o"]) and torch.equal(lse, s["lse"])
        # and the whole history agrees with one prompt append of the same tokens
        c2 = C.Cache(X, [T] * M, hkv, hd, page, dtype, e4m3, seed=i)
        rows = data[i].reshape(T * M, -1)
        X.cache_append(dm, c2.handle, rows, w, ints([m for _ in range(T) for m in range(M)]),
                       ints([t for t in range(T) for _ in range(M)]))
        for a, b in zip(s["c"].tensors(), c2.tensors()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_token_by_token_equals_the_threshold_layer(X):
    """A sparse layer under the causal threshold rule, generated token by token: each token
    that the rule routes is appended at its own position and attends to the routed tokens
    before it; the others skip the layer. The rows equal xmod_layer_fwd_threshold's on the
    whole sequence."""
    w = I.WORKLOADS["a4k8_bf16"].replace(B=3, T=100, d=256, hq=4, hkv=2, F=384, seed=21, weight_std=0.049)
    lw = I.layer_weights(w, 0)
    g = np.random.default_rng(0)
    lw["gq"] = I.f32_to_bf16_bits((1 + 0.1 * g.standard_normal(w.hd)).astype(np.float32))
    lw["gk"] = I.f32_to_bf16_bits((1 + 0.1 * g.standard_normal(w.hd)).astype(np.float32))
    dev = dev_layer(lw, "bf16")
    W = X.layer_weights(dev, lw["varsigma"], THETA)
    x = to_dev(I.residual_stream(w), "bf16").view(w.B, w.T, w.d)
    s = x.double() @ dev["w_router"].double()
    bias = torch.tensor([0.0, 1.0, -1.5], device="cuda")[:, None].expand(w.B, w.T).contiguous()
    near = (s + bias).abs() < 1e-3
    bias = torch.where(near, bias + 4e-3, bias).float().contiguous()
    s = s + bias.double()
    full = x.clone()
    ws = workspace(xmod_dims(w), w.K)
    X.layer_fwd_threshold(xmod_dims(w), 0, W, full, bias, ws)
    assert X.sync_status(ws) == X.OK
    full = full.view(w.B, w.T, w.d)

    dm = xmod_dims(w)
    c = C.Cache(X, [w.T] * w.B, w.hkv, w.hd, 16, "bf16")
    wqkv = torch.cat([dev["wq"], dev["wk"], dev["wv"]])
    ws2 = torch.zeros(X.cache_attention_workspace_bytes(dm, w.B), dtype=torch.uint8, device="cuda")
    X.reset_status(ws2)
    count = torch.zeros(w.B, dtype=torch.int32, device="cuda")
    seqs = torch.arange(w.B, dtype=torch.int32, device="cuda")
    q = torch.zeros(w.B, w.hq * w.hd, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros_like(q)
    out = []

    def norm(h, gain):
        h = h.float()
        return (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + w.eps) * gain.float()).bfloat16()

    for t in range(w.T):
        xt = x[:, t].contiguous()
        routed = s[:, t] >= 0
        seq = torch.where(routed, seqs, -1).to(torch.int32)
        qkv = norm(xt, dev["rms1"]) @ wqkv.T
        X.cache_append(dm, c.handle, qkv, W, seq, count, torch.full_like(count, t), q)
        count = count + routed.to(torch.int32)
        X.cache_attention(dm, c.handle, q, seq, count, o, ws2)
        a = o.float() @ dev["wo"].float().T
        v2 = norm(xt.float() + a, dev["rms2"]).float()
        hid = torch.nn.functional.silu(v2 @ dev["w_gate"].float().T) * (v2 @ dev["w_up"].float().T)
        f = hid @ dev["w_down"].float().T
        gate = lw["varsigma"] * torch.sigmoid(s[:, t]).float()[:, None]
        out.append(torch.where(routed[:, None], (xt.float() + gate * (a + f)).bfloat16(), xt))
    assert X.sync_status(ws2) == X.OK
    assert 0 < int(count.min()) and int(count.max()) < w.T
    got = from_dev(torch.stack(out, 1).contiguous(), "bf16")
    ref = from_dev(full, "bf16")
    # both sides round their stream once: half a spacing each, as for a stored output
    U.assert_close(got.reshape(ref.shape), ref, "bf16", "y", stored_ref=2 * ref)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_attention_of_many_short_rows(X, kind):
    """More rows than a CTA plans at once, short and empty ones, some skipped."""
    M = 4100
    lens = [(m * 7) % 23 for m in range(M)]
    seq = [m if m % 11 else -1 for m in range(M)]
    c, q, o, lse, ws, call = _attention(X, kind, 4, 2, 64, 16, lens, seq)
    call()
    assert X.sync_status(ws) == X.OK
    sample = list(range(0, 40)) + list(range(40, M, 97)) + [M - 1]
    _check_attention(c, kind, q[sample], [seq[m] for m in sample], [lens[m] for m in sample], o[sample], lse[sample],
                     4, 64)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_two_streams_at_once(X, kind):
    """Attention of two caches on two streams at the same time, each with its workspace,
    while a third appends: the same bits as one after the other."""
    a = _attention(X, kind, 12, 4, 128, 16, [3000, 5, 900, 64], seed=3)
    b = _attention(X, kind, 16, 1, 64, 32, [77, 2500, 1, 0, 640], seed=4)
    for s in (a, b):
        s[5]()
    torch.cuda.synchronize()
    want = [(s[2].clone(), s[3].clone()) for s in (a, b)]
    dtype, c, qkv, seq, slot, pos, gains, w = _append_case(X, kind, 12, 4, 128, 16, 200, True, THETA)
    q_out = torch.empty(200, 12 * 128, dtype=C.DT[dtype], device="cuda")
    dm = C.dims(X, 12, 4, 128, dtype)
    seq_t, slot_t = ints(seq.tolist()), ints(slot.tolist())
    X.cache_append(dm, c.handle, qkv, w, seq_t, slot_t, pos, q_out)
    held = [t.clone() for t in c.tensors()] + [q_out.clone()]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s[5]()
        with torch.cuda.stream(streams[2]):
            X.cache_append(dm, c.handle, qkv, w, seq_t, slot_t, pos, q_out)
    torch.cuda.synchronize()
    for s, (o, lse) in zip((a, b), want):
        assert torch.equal(s[2], o) and torch.equal(s[3], lse)
    for t, h in zip(c.tensors() + [q_out], held):
        assert torch.equal(t.view(torch.uint8), h.view(torch.uint8))


def test_binding_refusals(X):
    """Types, shapes, layouts and caches that do not belong together are refused."""
    hq, hkv, hd, M = 4, 2, 64, 3
    dm = C.dims(X, hq, hkv, hd, "bf16")
    c = C.Cache(X, [16] * M, hkv, hd, 16, "bf16")
    qkv = torch.zeros(M, (hq + 2 * hkv) * hd, dtype=torch.bfloat16, device="cuda")
    q, o = torch.zeros(M, hq * hd, dtype=torch.bfloat16, device="cuda"), torch.zeros(M, hq * hd, dtype=torch.bfloat16, device="cuda")
    i, ws = ints([1] * M), torch.zeros(X.cache_attention_workspace_bytes(dm, M), dtype=torch.uint8, device="cuda")
    w32 = X.layer_weights({"q_norm": torch.ones(hd, device="cuda")})
    odd = torch.zeros(M, (hq + 2 * hkv) * hd + 4, dtype=torch.bfloat16, device="cuda")
    other = C.dims(X, hq, hkv, 32, "bf16")
    bad = [lambda: X.cache_append(dm, c.handle, qkv.float(), None, None, i),
           lambda: X.cache_append(dm, c.handle, qkv[:, :-8], None, None, i),
           lambda: X.cache_append(dm, c.handle, odd[:, 4:], None, None, i),
           lambda: X.cache_append(dm, c.handle, odd[:, :-4], None, None, i),
           lambda: X.cache_append(dm, c.handle, qkv, None, None, i.long()),
           lambda: X.cache_append(dm, c.handle, qkv, None, None, i[:2]),
           lambda: X.cache_append(dm, c.handle, qkv, None, None, None),
           lambda: X.cache_append(dm, c.handle, qkv, None, i.cpu(), i),
           lambda: X.cache_append(dm, c.handle, qkv, w32, None, i),
           lambda: X.cache_append(dm, c.handle, qkv, None, None, i, None, q[:2]),
           lambda: X.cache_append(other, c.handle, qkv, None, None, i),
           lambda: X.cache_append(C.dims(X, hq, hkv, hd, "fp32"), c.handle, qkv.float(), None, None, i),
           lambda: X.cache_attention(dm, c.handle, q, None, i, o.float(), ws),
           lambda: X.cache_attention(dm, c.handle, q, None, i.float(), o, ws),
           lambda: X.cache_attention(dm, c.handle, q, None, None, o, ws),
           lambda: X.cache_attention(dm, c.handle, q.t(), None, i, o, ws),
           lambda: X.cache_attention(dm, c.handle, q, None, i, o, ws.cpu()),
           lambda: X.cache_attention(dm, c.handle, q, None, i, o, ws, lse=torch.zeros(M, device="cuda")),
           lambda: X.kv_cache(c.k, c.v.float(), c.table), lambda: X.kv_cache(c.k, c.v, c.table.long()),
           lambda: X.kv_cache(c.k.transpose(1, 2), c.v.transpose(1, 2), c.table),
           lambda: X.kv_cache(c.k, c.v, c.table, torch.zeros(1, device="cuda")),
           lambda: X.kv_cache(c.k, c.v, c.table, None, torch.zeros(1, device="cuda"))]
    for n, call in enumerate(bad):
        with pytest.raises(X.XmodError) as e:
            call()
        assert e.value.status == X.ERR_INVALID_ARG, n
    with pytest.raises(X.XmodError) as e:
        X.cache_attention(dm, c.handle, q, None, i, o, ws[:256])
    assert e.value.status == X.ERR_WORKSPACE


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_append_one_token_in_place(X, kind):
    """A single row has no row stride of its own: its q may lie in place all the same."""
    hq, hkv, hd, page = 4, 2, 64, 16
    dtype, c, qkv, seq, slot, pos, gains, w = _append_case(X, kind, hq, hkv, hd, page, 1, True, THETA)
    before = [t.clone() for t in c.tensors()]
    x = qkv.clone()
    X.cache_append(C.dims(X, hq, hkv, hd, dtype), c.handle, x, w, ints(seq.tolist()), ints(slot.tolist()),
                   pos, q_out=x[:, :hq * hd])
    _check_append(c, dtype, qkv, seq, slot, pos, gains, THETA, x[:, :hq * hd].contiguous(), hq, hkv, hd,
                  [True], before)
    assert torch.equal(x[:, hq * hd:], qkv[:, hq * hd:])


def test_row_strides_past_32_bits_are_refused(X):
    """The calls that take row strides as 32-bit numbers do not cut a longer one short."""
    hq, hkv, hd = 4, 2, 64
    c = C.Cache(X, [16, 16], hkv, hd, 16, "bf16", fill=0.5)
    dm, width = C.dims(X, hq, hkv, hd, "bf16"), (hq + 2 * hkv) * hd
    buf = torch.empty(2 ** 32 + 2 * width, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((2, width), (2 ** 32 + width, 1))
    near = buf[:2 * width].view(2, width)
    slot = ints([0, 1])
    ws = torch.zeros(X.cache_attention_workspace_bytes(dm, 2), dtype=torch.uint8, device="cuda")
    o = torch.empty(2, hq * hd, dtype=torch.bfloat16, device="cuda")
    held = [t.clone() for t in c.tensors()]
    for call in (lambda: X.cache_append(dm, c.handle, far, None, None, slot),
                 lambda: X.cache_append(dm, c.handle, near, None, None, slot, q_out=far[:, :hq * hd]),
                 lambda: X.cache_attention(dm, c.handle, far[:, :hq * hd], None, slot, o, ws)):
        with pytest.raises(X.XmodError) as e:
            call()
        assert e.value.status == X.ERR_UNSUPPORTED
    assert all(torch.equal(a, b) for a, b in zip(held, c.tensors()))


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_rewritten_slots_are_read_anew(X, kind):
    """Slots that a call reads, the next overwrites and the one after reads again, queued
    without a pause: the same bits as with one after each call."""
    dtype, e4m3 = KINDS[kind]
    hq, hkv, hd, page, M, n = 8, 4, 64, 16, 6, 200
    dm = C.dims(X, hq, hkv, hd, dtype)
    gen = torch.Generator().manual_seed(11)
    qkv = torch.randn(24, M, (hq + 2 * hkv) * hd, generator=gen).cuda().to(C.DT[dtype])
    slots = [ints([(37 * i + 5 * m) % n for m in range(M)]) for i in range(3)]
    lens = ints([n - m for m in range(M)])
    ws = torch.zeros(X.cache_attention_workspace_bytes(dm, M), dtype=torch.uint8, device="cuda")
    runs = []
    for pause in (True, False):
        c = C.Cache(X, [208] * M, hkv, hd, page, dtype, e4m3)
        for s in range(M):
            c.fill(s, n, s)
        o = torch.empty(24, M, hq * hd, dtype=C.DT[dtype], device="cuda")
        torch.cuda.synchronize()
        for i in range(24):
            X.cache_append(dm, c.handle, qkv[i], None, None, slots[i % 3])
            if pause:
                torch.cuda.synchronize()
            X.cache_attention(dm, c.handle, qkv[i, :, :hq * hd], None, lens, o[i], ws)
            if pause:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        runs.append(o)
    assert torch.equal(*(r.view(torch.uint8) for r in runs))
    assert bool(runs[0].float().isfinite().all())
