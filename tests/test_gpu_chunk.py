"""GPU: attention of a chunk of new tokens over the paged cache against a plain 64-bit form:
types, head layouts, chunks from nothing to thousands of tokens, what a row does not see,
refused chunks, streams, graphs, offsets past 32 bits; and the run of operators around it."""
import math

import pytest

from tests import _cache as C
from tests import _more as R
from tests._gpu import need_gpu, torch

pytestmark = pytest.mark.gpu

KINDS = {"bf16": ("bf16", False), "fp32": ("fp32", False), "e4m3": ("bf16", True)}
# the stated rounding of the weights: half a bf16 step
P_ROUND = {"bf16": 2.0 ** -8, "fp32": 0.0, "e4m3": 2.0 ** -8}
HEADS = [(4, 2, 64), (12, 4, 128), (6, 6, 32), (16, 1, 128), (10, 2, 64), (7, 1, 32)]


@pytest.fixture(scope="module")
def X():
    need_gpu()
    from sparse_depth_token_gb300 import xmod
    xmod.load()
    return xmod


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _setup(X, kind, hq, hkv, hd, page, shape, seq=None, pad=0, seed=1, scale=1.0, lead=0, tail=0):
    """shape: (tokens, slots) of each chunk; lead, tail: rows of q before the first and behind
    the last chunk."""
    dtype, e4m3 = KINDS[kind]
    ids = list(range(len(shape))) if seq is None else seq
    rooms = [0] * (max(max(ids), 0) + 1)
    for s, (_, n) in zip(ids, shape):
        if s >= 0:
            rooms[s] = max(rooms[s], n)
    c = C.Cache(X, rooms, hkv, hd, page, dtype, e4m3, seed=seed)
    for s, n in enumerate(rooms):
        if n:
            c.fill(s, n, seed + s, scale)
    first = [lead]
    for n, _ in shape:
        first.append(first[-1] + n)
    M = first[-1] + tail
    q = (torch.randn(M, hq * hd + pad, generator=torch.Generator().manual_seed(seed + 99)) * scale).cuda().to(
        C.DT[dtype])[:, :hq * hd]
    dm = C.dims(X, hq, hkv, hd, dtype)
    s = dict(X=X, kind=kind, c=c, q=q, dm=dm, shape=shape, ids=ids, first=first, hq=hq, hd=hd,
             o=torch.full((M, hq * hd), -3.0, dtype=C.DT[dtype], device="cuda"),
             lse=torch.full((M, hq), -3.0, device="cuda"), start=ints(first), len=ints([n for _, n in shape]),
             seq=None if seq is None else ints(seq))
    s["ws"] = torch.full((X.cache_attention_chunk_workspace_bytes(dm, len(shape), M),), 0x7f, dtype=torch.uint8,
                         device="cuda")
    X.reset_status(s["ws"])
    return s


def _call(s, **over):
    a = {**s, **over}
    a["X"].cache_attention_chunk(a["dm"], a["c"].handle, a["q"], a["start"], a["seq"], a["len"], a["o"], a["ws"],
                                 lse=a["lse"])


def _check_rows(s, i, rows=None):
    """Chunk i (or some of its rows) against the plain form."""
    kind, c, hq, hd = s["kind"], s["c"], s["hq"], s["hd"]
    n, slots = s["shape"][i]
    at = slice(s["first"][i], s["first"][i] + n)
    got, gl = s["o"][at].view(n, hq, hd).double(), s["lse"][at].double()
    if s["ids"][i] < 0:
        assert bool((got == -3).all()) and bool((gl == -3).all()), i
        return
    q = s["q"][at].reshape(n, hq, hd)
    for r in torch.arange(n).split(64) if rows is None else [torch.tensor([r]) for r in rows]:
        a, b = int(r[0]), int(r[-1]) + 1
        see = max(0, slots - (n - b))
        part = q[a:b] if see else q[a:b] * 0
        ref, rl, bound, lb = R.chunk_ref(c, part, s["ids"][i], see, P_ROUND[kind])
        half = C.HALF[KINDS[kind][0]]
        err = (got[a:b] - ref).abs() - bound - half * (ref.abs() + bound)
        assert float(err.max()) <= 0, (i, a, b, float(err.max()))
        empty = rl == -math.inf
        assert bool((gl[a:b][empty] == -math.inf).all())
        le = torch.where(empty, 0.0, (gl[a:b] - rl).abs() - 2 * lb)
        assert float(le.max()) <= 0, (i, a, b, float(le.max()))


def _check(s):
    assert s["X"].sync_status(s["ws"]) == s["X"].OK
    for i, (n, _) in enumerate(s["shape"]):
        if n:
            _check_rows(s, i)
    for edge in (s["o"][:s["first"][0]], s["o"][s["first"][-1]:], s["lse"][:s["first"][0]], s["lse"][s["first"][-1]:]):
        assert bool((edge == -3).all())


SHAPES = [
    [(1, 1)], [(1, 64), (1, 65), (1, 1)], [(5, 5), (0, 40), (17, 130), (2, 63), (33, 64), (64, 200)],
    [(129, 129), (3, 700)], [(40, 25), (3, 1), (2, 0), (9, 9)],     # rows before the first slot
]


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("hq,hkv,hd", HEADS)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_matches_the_plain_form(X, kind, hq, hkv, hd, shape):
    page = [16, 32, 64, 128, 48][shape]
    s = _setup(X, kind, hq, hkv, hd, page, SHAPES[shape], pad=8 * (shape % 2), lead=shape, tail=2 * shape)
    _call(s)
    _check(s)


def test_one_key_over_e4m3_is_its_value(X):
    """The largest weight times its value's scale is a power of two, which bf16 holds: what is left
    of a single key are the output's rounding and the exponent's (log2, ex2 and a product, each
    within 2^-21)."""
    for hq, hkv, hd in HEADS:
        s = _setup(X, "e4m3", hq, hkv, hd, 16, [(1, 1)] * 40, seed=hd + hq)
        _call(s)
        for i in range(40):
            at = s["first"][i]
            ref, _, bound, _ = R.chunk_ref(s["c"], s["q"][at: at + 1].reshape(1, hq, hd), i, 1, 3 * 2.0 ** -21)
            err = (s["o"][at].view(1, hq, hd).double() - ref).abs() - bound - C.HALF["bf16"] * (ref.abs() + bound)
            assert float(err.max()) <= 0, (hq, hd, i, float(err.max()))


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_wide_groups(X, kind):
    """More query heads on a KV head than a tile has rows."""
    s = _setup(X, kind, 160, 1, 32, 16, [(3, 40), (2, 2), (1, 100)])
    _call(s)
    _check(s)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("shape,hq,hkv,hd,page", [
    ([(700, 1500)], 12, 4, 128, 64), ([(3, 30011)], 16, 4, 128, 32), ([(1, 9000), (2, 20000)], 8, 2, 64, 16),
    ([(2000, 2000), (77, 4000), (500, 520)], 4, 2, 64, 128), ([(300, 5000)], 4, 4, 32, 16)])
def test_long(X, kind, shape, hq, hkv, hd, page):
    """Chunks that many CTAs share: sampled rows, the first and last ones among them."""
    s = _setup(X, kind, hq, hkv, hd, page, shape)
    _call(s)
    assert X.sync_status(s["ws"]) == X.OK
    for i, (n, _) in enumerate(shape):
        _check_rows(s, i, sorted({0, n // 3, n // 2, max(0, n - 65), max(0, n - 2), n - 1}))


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_large_scores(X, kind):
    """Scores of both signs up to some hundreds: weights from 1 to far below the last bit."""
    s = _setup(X, kind, 8, 2, 64, 16, [(70, 200), (5, 1000)], scale=5.0)
    _call(s)
    _check(s)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_rising_scores(X, kind):
    """Keys ever closer to the queries: the running maximum moves with every tile."""
    s = _setup(X, kind, 4, 2, 64, 16, [(40, 640)])
    c = s["c"]
    q = torch.randn(64, generator=torch.Generator().manual_seed(3)).cuda()
    s["q"].copy_(q.repeat(4)[None].expand(40, -1).to(s["q"].dtype))
    for i in range(640):
        p, o = c.place(0, i)
        k = (q * (i / 160.0)).expand(2, 64)
        if c.e4m3:
            c.k.view(torch.uint8)[p, :, o] = (k * 50).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            c.k_scale[p, :, o] = 0.02
        else:
            c.k[p, :, o] = k.to(c.k.dtype)
    _call(s)
    _check(s)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("n,slots", [(70, 70), (70, 200), (9, 64), (3, 500)])
def test_what_a_row_does_not_see(X, kind, n, slots):
    """Infinities and NaN in later tokens of the chunk change no earlier row, bit for bit; the
    rows that see them become NaN where their value or score is."""
    s = _setup(X, kind, 4, 2, 64, 16, [(n, slots)])
    _call(s)
    o, lse = s["o"].clone(), s["lse"].clone()
    c, bad = s["c"], n // 2
    p, at = c.place(0, slots - n + bad)
    if c.e4m3:
        c.v_scale[p, 0, at] = math.nan
        c.v.view(torch.uint8)[p, 1, at, 5] = 0x7F      # the code of NaN
        c.k_scale[p, 1, at] = math.nan
    else:
        c.v[p, 0, at] = math.nan
        c.v[p, 1, at, 5] = math.inf
        c.k[p, 1, at] = math.nan
    _call(s)
    assert torch.equal(s["o"][:bad], o[:bad]) and torch.equal(s["lse"][:bad], lse[:bad])
    got = s["o"].view(n, 4, 64)
    assert bool(got[bad:, :2].isnan().all()) and bool(got[bad:, 2:, 5].isnan().all())
    assert torch.equal(s["lse"][:, :2], lse[:, :2])     # the scores of head 0 are what they were
    assert bool(s["lse"][bad:, 2:].isnan().all())
    # an infinity alone, seen by the last row only
    s = _setup(X, kind, 4, 2, 64, 16, [(n, slots)])
    if kind != "e4m3":
        p, at = s["c"].place(0, slots - 1)
        s["c"].v[p, 0, at, 3] = math.inf
        _call(s)
        assert torch.equal(s["o"][:-1], o[:-1]) and torch.equal(s["lse"], lse)
        last = s["o"][-1].view(4, 64)
        assert bool((last[:2, 3] == math.inf).all())
        last[:2, 3] = o[-1].view(4, 64)[:2, 3]
        assert torch.equal(last.view(-1), o[-1])


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_chunks_share_skip_and_repeat_sequences(X, kind):
    s = _setup(X, kind, 4, 2, 64, 16, [(5, 90), (3, 12), (7, 200), (4, 90), (6, 33)], seq=[2, -1, 0, 2, 0], lead=1, tail=3)
    _call(s)
    _check(s)


def test_many_chunks(X):
    """More chunks than a CTA has threads, short, empty and skipped ones."""
    shape = [((i * 7) % 5, 5 + (i * 13) % 90) for i in range(1500)]
    seq = [i if i % 11 else -1 for i in range(1500)]
    s = _setup(X, "bf16", 4, 2, 64, 16, shape, seq=seq)
    _call(s)
    assert X.sync_status(s["ws"]) == X.OK
    for i in list(range(30)) + list(range(30, 1500, 37)) + [1499]:
        if shape[i][0]:
            _check_rows(s, i)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_single_tokens_agree_with_the_row_form(X, kind):
    """Chunks of one token against xmod_cache_attention: both within their stated errors."""
    lens = [1, 63, 64, 65, 300, 0]
    s = _setup(X, kind, 12, 4, 128, 16, [(1, n) for n in lens])
    _call(s)
    _check(s)
    ws = torch.zeros(X.cache_attention_workspace_bytes(s["dm"], 6), dtype=torch.uint8, device="cuda")
    o, lse = torch.zeros_like(s["o"]), torch.zeros_like(s["lse"])
    X.cache_attention(s["dm"], s["c"].handle, s["q"], None, s["len"], o, ws, lse=lse)
    # unit values: weights' roundings 2^-8 (fp32 none) on a mean of values below 6, o's own on both sides
    bound = {"bf16": 6 * 3 * 2.0 ** -8, "e4m3": 6 * 3 * 2.0 ** -8, "fp32": 1e-5}[kind]
    assert float((s["o"].float() - o.float()).abs().max()) <= bound
    assert bool((s["lse"][5] == -math.inf).all()) and float((s["lse"][:5] - lse[:5]).abs().max()) <= 1e-4


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_refused_chunks(X, kind):
    """Bad sequences and starts skip their chunk, lengths are clamped, bad pages read page 0;
    all are reported."""
    shape = [(4, 30), (3, 20), (5, 32)]
    for bad in ("seq", "descends", "past", "before", "len", "page"):
        s = _setup(X, kind, 4, 2, 64, 16, shape, seq=[0, 1, 2], tail=2)
        M = s["q"].shape[0]
        skipped = [1]
        if bad == "seq":
            s["seq"][1] = 3
        elif bad == "descends":
            s["start"][2:] = 2          # chunk 1 ends before it starts, chunk 2 has no rows
            skipped = [1, 2]
        elif bad == "past":
            s["start"][3] = M + 1
            skipped = [2]
        elif bad == "before":
            s["start"][0] = -1
            skipped = [0]
        elif bad == "len":
            s["len"][2] = 1000          # clamped to max_pages * page_size = 32
            skipped = []
        else:
            s["c"].table[1, 1] = -1
            s["c"].table_np[1, 1] = 0
            for t in s["c"].tensors():      # page 0 all finite
                t[0] = (torch.randn(t[0].shape) * 0.5).cuda().to(t.dtype)
            skipped = []
        s["o"].fill_(-3)
        s["lse"].fill_(-3)
        _call(s)
        assert X.sync_status(s["ws"]) == X.ERR_DEVICE_CHECK, bad
        for i in range(3):
            at = slice(s["first"][i], s["first"][i + 1])
            if i in skipped:
                assert bool((s["o"][at] == -3).all()) and bool((s["lse"][at] == -3).all()), bad
            else:
                _check_rows(s, i)
        assert bool((s["o"][-2:] == -3).all())


def test_nothing(X):
    s = _setup(X, "bf16", 4, 2, 64, 16, [(2, 5)])
    for start, n in (([0], []), ([0, 0], [5])):
        q = s["q"][:0]
        o = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
        _call(s, q=q, o=o, lse=None, start=ints(start), len=ints(n), seq=None)
    before = s["o"].clone()
    _call(s, start=ints([1, 1]))            # a chunk without rows
    _call(s, start=ints([0]), len=ints([]))
    assert torch.equal(s["o"], before) and X.sync_status(s["ws"]) == X.OK


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_the_same_bits_again(X, kind):
    s = _setup(X, kind, 12, 4, 128, 32, [(33, 900), (1, 4000), (250, 250)])
    _call(s)
    o, lse = s["o"].clone(), s["lse"].clone()
    for fill in (0, 0xff):
        s["ws"].fill_(fill)         # what an earlier use left does not matter
        X.reset_status(s["ws"])
        s["o"].fill_(-3)
        _call(s)
        assert torch.equal(s["o"], o) and torch.equal(s["lse"], lse)
    _call(s, lse=None)
    assert torch.equal(s["o"], o)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_past_32_bit_offsets(X, kind):
    """Pages whose elements lie past 2^32 bytes."""
    hkv, hd, page = 8, 128, 128
    per = hkv * page * hd * (1 if kind == "e4m3" else 2)
    far = 2 ** 32 // per + 3
    c = C.Cache(X, [300], hkv, hd, page, "bf16", kind == "e4m3", first_page=far, seed=2)
    c.fill(0, 300, 5)
    s = _setup(X, kind, 8, 8, 128, 16, [(50, 300)])
    s["c"] = c
    _call(s)
    _check(s)
    del c, s
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_captured_and_on_streams(X, kind):
    """Two recorded calls with their own workspaces, replayed with other lengths, at once with
    eager calls on a third stream: the same bits as alone."""
    sets = [_setup(X, kind, 12, 4, 128, 16, shape, seed=i) for i, shape in
            enumerate([[(4, 500), (9, 60)], [(130, 400)], [(2, 3000), (2, 2000)]])]
    streams = [torch.cuda.Stream() for _ in sets]
    graphs = []
    for s, st in zip(sets[:2], streams):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            _call(s)
        graphs.append(g)
    for s in sets[:2]:
        s["shape"] = [(n, slots - 7) for n, slots in s["shape"]]
        s["len"].copy_(ints([n for _, n in s["shape"]]))
    torch.cuda.synchronize()
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(streams[2]):
            _call(sets[2])
    torch.cuda.synchronize()
    for s in sets:
        _check(s)
        o = s["o"].clone()
        _call(s)
        assert torch.equal(s["o"], o)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_small_heads_at_once(X, kind):
    """Calls on two streams whose CTAs fit an SM together but for the tensor memory, which one
    waits for until the other is done: the same bits as alone."""
    sets = [_setup(X, kind, 12, 4, 32, 16, shape, seed=i) for i, shape in
            enumerate([[(300, 2000), (9, 60)], [(200, 3000)]])]
    alone = []
    for s in sets:
        _call(s)
        alone.append(s["o"].clone())
        s["o"].fill_(-3.0)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                _call(s)
    torch.cuda.synchronize()
    for s, o in zip(sets, alone):
        _check(s)
        assert torch.equal(s["o"], o)


def test_binding_refusals(X):
    s = _setup(X, "bf16", 4, 2, 64, 16, [(3, 5), (2, 9)])
    bad = [dict(q=s["q"].float()), dict(q=s["q"][:, :-8]), dict(q=s["q"].cpu()), dict(start=s["start"][:-1]),
           dict(start=s["start"].long()), dict(len=s["len"].float()), dict(o=s["o"][:-1]), dict(o=s["o"].float()),
           dict(lse=s["lse"][:, :2]), dict(seq=ints([0])), dict(o=s["q"]), dict(q=s["q"][:, ::2].repeat(1, 2)[:, ::2])]
    for over in bad:
        with pytest.raises(X.XmodError) as e:
            _call(s, **over)
        assert e.value.status == X.ERR_INVALID_ARG, over.keys()
    with pytest.raises(X.XmodError) as e:
        _call(s, ws=s["ws"][:1000])
    assert e.value.status == X.ERR_WORKSPACE
    other = C.dims(X, 8, 2, 64, "bf16")
    with pytest.raises(X.XmodError):
        _call(s, dm=other)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_prompt_by_pieces_and_a_chosen_token(X, kind):
    """The operators as a server runs them: projections turned, appended, attended to piece by
    piece and at once, then a token chosen: both ways see the same cache, and every piece is
    what the plain form gives for it."""
    dtype, e4m3 = KINDS[kind]
    hq, hkv, hd, T = 4, 2, 64, 150
    dm = C.dims(X, hq, hkv, hd, dtype)
    gen = torch.Generator().manual_seed(11)
    qkv = torch.randn(T, (hq + 2 * hkv) * hd, generator=gen).cuda().to(C.DT[dtype])
    gains = {n: (1 + 0.1 * torch.randn(hd, generator=gen)).cuda().to(C.DT[dtype]) for n in ("q_norm", "k_norm")}
    w = X.layer_weights(gains)
    rope = X.rope(hd, 1e4, rot_dim=32, interleaved=True, scaling=X.ROPE_PARTS, factor=8.0, trained=64)
    caches = [C.Cache(X, [T], hkv, hd, 16, dtype, e4m3, seed=4) for _ in range(2)]
    outs = []
    for c, cuts in zip(caches, ([0, T], [0, 1, 40, 104, 149, T])):
        o = torch.zeros(T, hq * hd, dtype=C.DT[dtype], device="cuda")
        for a, b in zip(cuts, cuts[1:]):
            rows = qkv[a:b].clone()
            pos = torch.arange(a, b, dtype=torch.int32, device="cuda")
            X.qk_rope(dm, rows, w, rope, rows, pos=pos)                   # in place
            q = torch.empty(b - a, hq * hd, dtype=C.DT[dtype], device="cuda")
            X.cache_append(dm, c.handle, rows, None, torch.zeros_like(pos), pos, None, q)
            ws = torch.zeros(X.cache_attention_chunk_workspace_bytes(dm, 1, b - a), dtype=torch.uint8, device="cuda")
            part = o[a:b]
            X.cache_attention_chunk(dm, c.handle, q, ints([0, b - a]), None, ints([b]), part, ws)
            assert X.sync_status(ws) == X.OK
            ref, _, bound, _ = R.chunk_ref(c, q.view(b - a, hq, hd), 0, b, P_ROUND[kind])
            err = (part.view(b - a, hq, hd).double() - ref).abs() - bound - C.HALF[dtype] * (ref.abs() + bound)
            assert float(err.max()) <= 0
        outs.append(o)
    live = [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in caches[0].tensors()]
    same = [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in caches[1].tensors()]
    for a, b in zip(live, same):
        assert torch.equal(a.nan_to_num(7.0) if a.is_floating_point() else a, b.nan_to_num(7.0) if b.is_floating_point() else b)
    head = torch.randn(hq * hd, 500, generator=gen).cuda()
    logits = outs[0].float() @ head
    u = torch.rand(T, generator=gen).cuda()
    token, logp = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda")
    X.sample_tokens(logits, u, token, top_p=torch.full((T,), 0.9, device="cuda"), logp=logp)
    for t in range(0, T, 7):
        want, lp, margin = R.sample_ref(logits[t], u[t], top_p=torch.tensor(0.9))
        assert margin > 2.0 ** -33 and int(token[t]) == want and abs(float(logp[t]) - lp) <= 1e-5
