"""Operators of serving and training a chunk of tokens at a time, as measured cases.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as the
calls a user makes of the library:

  chunk      attention of a chunk of new tokens of every sequence over the paged cache that
             holds them and what came before: softmax(q K^T / sqrt(hd)) V, query head h on KV
             head h / (hq / hkv), the chunk's token i on the sequence's slots up to its own
  rope       norms of queries and keys for each head and rotary positions in one pass: halves
             or neighbours paired, the whole head or its first dimensions, frequencies scaled
             for long contexts (linear, by the base, by parts of the spectrum)
  rope_bwd   its gradients at the projections and at the gains
  sample     a token for each row of logits from a given uniform number, with temperature,
             top-k, top-p and min-p

`own` chooses which of the two forms run() takes.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# ---------------------------------------------------------------- cases


def listed():
    return [
        # 8 sequences with 4 proposed tokens each to be verified at once, at the A4K8 stack's
        # heads and length: a call whose latency counts
        dict(name="chunk 8x4 over 4096", op="chunk", dtype="bf16", fmt="native", chunks=8, new=4, hq=12, hkv=4,
             hd=128, page=16, max_len=4096, kind="even"),
        # whole prompts of different lengths, packed: the first pass over them
        dict(name="chunk 6 prompts up to 8192", op="chunk", dtype="bf16", fmt="native", chunks=6, new=8192, hq=32,
             hkv=8, hd=128, page=64, max_len=8192, kind="whole"),
        # the next 500 tokens of one long text, prefilled in pieces
        dict(name="chunk 500 at 131072", op="chunk", dtype="bf16", fmt="native", chunks=1, new=500, hq=16, hkv=4,
             hd=128, page=64, max_len=131072, kind="even"),
        # a mixed serving step at the A3K16 stack's length over an 8-bit cache: some sequences
        # bring a piece of a prompt, some a few tokens, one none
        dict(name="chunk 16 ragged at 16384 e4m3", op="chunk", dtype="bf16", fmt="e4m3", chunks=16, new=511, hq=16,
             hkv=4, hd=128, page=32, max_len=16384, kind="ragged"),
        # the fp32 path at a small model's heads
        dict(name="chunk 6x100 at 1000 fp32", op="chunk", dtype="fp32", fmt="native", chunks=6, new=100, hq=8, hkv=4,
             hd=64, page=16, max_len=1000, kind="ragged"),
        # one new token of 8 sequences: the decode step of a dense layer of the A4K8 stack
        dict(name="rope 8 tokens", op="rope", dtype="bf16", M=8, hq=12, hkv=4, hd=128, rot=128, inter=False,
             scaling="none", factor=1.0, norm=True, room=4096),
        # the prompts of 8 sequences of 4096 tokens at once, in a context 16 times the trained one
        dict(name="rope 32768 tokens by parts", op="rope", dtype="bf16", M=32768, hq=12, hkv=4, hd=128, rot=128,
             inter=False, scaling="parts", factor=16.0, norm=True, room=65536),
        # the training step of 4 sequences of 4096 tokens
        dict(name="rope gradient 16384", op="rope_bwd", dtype="bf16", M=16384, hq=12, hkv=4, hd=128, rot=128,
             inter=False, scaling="none", factor=1.0, norm=True, room=4096),
        # a small fp32 model that turns neighbours in half of each head
        dict(name="rope gradient 307 fp32", op="rope_bwd", dtype="fp32", M=307, hq=8, hkv=4, hd=64, rot=32, inter=True,
             scaling="linear", factor=4.0, norm=True, room=1024),
        # a serving step's rows with every filter on
        dict(name="sample 8 rows", op="sample", dtype="bf16", N=8, V=50257, pad=0, std=2.5, masked=0.0,
             temperature=0.8, k=50, p=0.95, min_p=0.02),
        # a large serving batch of fp32 logits, every row with its own settings, a grammar's
        # mask over a third of the tokens
        dict(name="sample 256 rows fp32", op="sample", dtype="fp32", N=256, V=50257, pad=7, std=2.5, masked=0.3,
             temperature=0.0, k=0, p=0.0, min_p=0.0),
        # rollouts: 4096 rows from the middle of the distribution
        dict(name="sample 4096 rows top-p", op="sample", dtype="bf16", N=4096, V=50257, pad=0, std=2.5, masked=0.0,
             temperature=1.0, k=-1, p=0.9, min_p=-1.0),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "rope", "rope_bwd", "sample", "sample"])
    if op == "sample":
        V = _log(rng, 100, 100000)
        return dict(op=op, dtype=rng.choice(["bf16", "fp32"]), N=_log(rng, 1, min(4096, 10 ** 8 // V)), V=V,
                    pad=rng.choice([0, 0, 3, 8]), std=rng.choice([0.5, 2.5, 2.5, 6.0]), masked=rng.choice([0.0, 0.2, 0.9]),
                    temperature=rng.choice([0.0, 0.3, 0.8, 1.0, 1.7]), k=rng.choice([-1, 0, 1, 20, 300]),
                    p=rng.choice([-1.0, 0.0, 0.5, 0.95]), min_p=rng.choice([-1.0, 0.0, 0.05]))
    hq, hkv = rng.choice([(12, 4), (32, 8), (4, 2), (8, 4), (16, 1)])
    hd = rng.choice([128, 128, 128, 64, 32])
    if op != "chunk":
        rot = rng.choice([hd, hd, hd // 2, hd // 4])
        scaling = rng.choice(["none", "linear", "base", "parts"])
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), M=_log(rng, 1, 16384 if hq <= 16 else 6000),
                    hq=hq, hkv=hkv, hd=hd, rot=rot, inter=rng.random() < 0.5, scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 40.0]), norm=rng.random() < 0.6,
                    room=_log(rng, 64, 131072))
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    fmt = rng.choice(["native", "native", "e4m3"]) if dtype == "bf16" else "native"
    chunks, kind = _log(rng, 1, 24), rng.choice(["even", "ragged", "ragged", "whole"])
    # at most a quarter of a gigabyte of keys and values, and an eighth of the largest case's products
    size = 1 if fmt == "e4m3" else DTYPES[dtype].itemsize
    max_len = _log(rng, 1, min(131072, 2 ** 28 // (2 * chunks * hkv * hd * size)))
    most = 2 ** 38 // (4 * hq * hd * (1 if dtype == "bf16" else 8))
    new = max_len if kind == "whole" else _log(rng, 1, max_len)
    while chunks * new * max_len > most:
        new = max(1, new // 2)
        if kind == "whole":
            max_len = new
        elif new == 1 and chunks * max_len > most:
            max_len //= 2
    return dict(op=op, dtype=dtype, fmt=fmt, chunks=chunks, new=new, hq=hq, hkv=hkv, hd=hd,
                page=rng.choice([16, 32, 64, 128]), max_len=max_len, kind=kind)


def _chunks(case):
    """(new tokens, slots) of a case's chunks, before the seed's shuffle. "even": all alike;
    "ragged": both spread over their ranges, with a chunk of no tokens among six or more;
    "whole": the cache holds nothing but the chunk."""
    n, new, top = case["chunks"], case["new"], case["max_len"]
    if case["kind"] == "even":
        return [(new, top)] * n
    out = []
    for i in range(n):
        a, b = ((i + 1) * 0.6180339887) % 1.0, ((i + 1) * 0.7548776662) % 1.0
        c = new if i == 0 else 1 + int((new - 1) * (a if case["kind"] == "whole" else a * a))
        out.append((c, c if case["kind"] == "whole" else top if i == 0 else c + int((top - c) * b)))
    if n >= 6 and case["kind"] == "ragged":
        out[1] = (0, out[1][1])
    return out


def _esize(case):
    return 1 if case.get("fmt") == "e4m3" else DTYPES[case["dtype"]].itemsize


def work(case):
    op = case["op"]
    es = DTYPES[case["dtype"]].itemsize
    if op == "chunk":
        shape = _chunks(case)
        rows, slots = sum(c for c, _ in shape), sum(n for c, n in shape if c)
        seen = sum(c * n - c * (c - 1) // 2 for c, n in shape)
        width = 2 * case["hkv"] * (case["hd"] * _esize(case) + (4 if case["fmt"] == "e4m3" else 0))
        return {"bytes": slots * width + rows * case["hq"] * (2 * case["hd"] * es + 4),
                "flops": 4 * seen * case["hq"] * case["hd"]}
    if op in ("rope", "rope_bwd"):
        n = case["M"] * (case["hq"] + case["hkv"]) * case["hd"]
        if op == "rope":
            return {"bytes": 2 * n * es + 4 * case["M"], "flops": 7 * n}
        # without norms the projections are not needed
        return {"bytes": (3 if case["norm"] else 2) * n * es + 4 * case["M"] + 8 * case["hd"], "flops": 16 * n}
    n = case["N"] * case["V"]
    return {"bytes": n * es + case["N"] * 28, "flops": n * 4}


# ---------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _new_cache(case, g, need):
    """A cache whose pages lie in shuffled order; need[s] of sequence s's table entries are
    pages, the rest -1. Every slot holds values, as after earlier use."""
    page, hkv, hd = case["page"], case["hkv"], case["hd"]
    n_pages = max(1, sum(need)) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    counts = torch.tensor(need, device="cuda")
    col = torch.arange(max(1, max(need)), device="cuda")[None, :]
    at = ((torch.cumsum(counts, 0) - counts)[:, None] + col).clamp(max=n_pages - 1)
    c = {"table": torch.where(col < counts[:, None], order[at], torch.full_like(order[at], -1)).contiguous()}
    for name in ("k", "v"):
        shape = (n_pages, hkv, page, hd)
        if case["fmt"] == "e4m3":
            x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
            c[name] = (x * 120.0).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            c[name + "_scale"] = torch.empty(shape[:3], device="cuda").uniform_(0.004, 0.012, generator=g)
        else:
            c[name] = torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda").normal_(generator=g)
            c[name + "_scale"] = None
    return c


def _settings(case, name, choices, r, dtype):
    """A row's setting: the case's own, 0: drawn for every row from `choices`, -1: off."""
    v = case[name]
    if v == -1:
        return None
    return torch.tensor([r.choice(choices) for _ in range(case["N"])] if v == 0 else [v] * case["N"], dtype=dtype,
                        device="cuda")


def _handles(case, s):
    """What a program that uses the library keeps beside its tensors."""
    from sparse_depth_token_gb300 import xmod as X
    s["X"] = X
    if case["op"] == "sample":
        return
    s["dims"] = X.dims(1, 1, 8 * case["hq"], case["hq"], case["hkv"], case["hd"], 8,
                       X.BF16 if case["dtype"] == "bf16" else X.FP32, s.get("eps", 1e-6))
    if case["op"] == "chunk":
        c = s["cache"]
        s["handle"] = X.kv_cache(c["k"], c["v"], c["table"], c["k_scale"], c["v_scale"])
        need = X.cache_attention_chunk_workspace_bytes(s["dims"], case["chunks"], len(s["q"]))
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
        return
    s["weights"] = X.layer_weights({"q_norm": s["q_norm"], "k_norm": s["k_norm"]})
    s["rope"] = X.rope(case["hd"], s["theta"], rot_dim=case["rot"], interleaved=case["inter"],
                       scaling={"none": X.ROPE_PLAIN, "linear": X.ROPE_LINEAR, "base": X.ROPE_BASE,
                                "parts": X.ROPE_PARTS}[case["scaling"]],
                       factor=case["factor"], trained=s["trained"])
    if case["op"] == "rope_bwd" and case["norm"]:
        s["ws"] = torch.zeros(X.qk_rope_bwd_workspace_bytes(s["dims"], case["M"]), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    r = random.Random(seed)
    s = {"case": case}
    dt, op = DTYPES[case["dtype"]], case["op"]
    if op == "chunk":
        hq, hd, page = case["hq"], case["hd"], case["page"]
        shape = _chunks(case)
        r.shuffle(shape)
        s["cache"] = _new_cache(case, g, [-(-n // page) for _, n in shape])
        s["shape"] = shape
        first = [0]
        for c, _ in shape:
            first.append(first[-1] + c)
        s["first"] = first
        s["start"], s["len"] = _ints(first), _ints([n for _, n in shape])
        s["q"] = torch.empty(first[-1], hq * hd, dtype=dt, device="cuda").normal_(generator=g)
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(first[-1], hq, device="cuda")
    elif op in ("rope", "rope_bwd"):
        M, hq, hkv, hd = (case[k] for k in ("M", "hq", "hkv", "hd"))
        s["theta"], s["trained"], s["eps"] = 10000.0, 4096, 1e-6
        room = case["room"]
        if M <= room // 8:      # one token of each sequence, anywhere
            pos = [r.randrange(room) for _ in range(M)]
        else:                   # whole sequences, one after the other
            length = max(1, min(room, M // 4))
            pos = [(room - length) + m % length for m in range(M)]
        s["pos"] = _ints(pos)
        s["qkv"] = torch.empty(M, (hq + 2 * hkv) * hd, dtype=dt, device="cuda").normal_(generator=g)
        for name in ("q_norm", "k_norm"):
            s[name] = (1 + 0.1 * torch.randn(hd, generator=g, device="cuda")).to(dt) if case["norm"] else None
        s["out"] = torch.zeros(M, (hq + hkv) * hd, dtype=dt, device="cuda")
        if op == "rope_bwd":
            s["dout"] = torch.empty(M, (hq + hkv) * hd, dtype=dt, device="cuda").normal_(generator=g)
            s["dq_norm"], s["dk_norm"] = (torch.zeros(hd, device="cuda") for _ in range(2))
    else:
        N, V = case["N"], case["V"]
        x = torch.empty(N, V + case["pad"], device="cuda").normal_(0.0, case["std"], generator=g)
        # half of the rows know their token well
        sure = torch.rand(N, generator=g, device="cuda") < 0.5
        best = torch.randint(0, V, (N,), generator=g, device="cuda")
        x[torch.arange(N, device="cuda"), best] += torch.where(sure, 5.0 * case["std"], 0.0)
        if case["masked"]:      # tokens that a grammar has ruled out
            off = torch.rand(V + case["pad"], generator=g, device="cuda") < case["masked"]
            x.masked_fill_(off, -math.inf)
            x[torch.arange(N, device="cuda"), best] = 3.0
        s["logits"] = x.to(dt)[:, :V]
        s["u"] = torch.rand(N, generator=g, device="cuda")
        s["temperature"] = _settings(case, "temperature", [0.0, 0.5, 0.8, 1.0, 1.3], r, torch.float32)
        s["k"] = _settings(case, "k", [0, 1, 20, 50, 1000], r, torch.int32)
        s["p"] = _settings(case, "p", [0.3, 0.9, 0.99, 1.0], r, torch.float32)
        s["min_p"] = _settings(case, "min_p", [0.0, 0.0, 0.02, 0.1], r, torch.float32)
        s["token"] = torch.zeros(N, dtype=torch.int32, device="cuda")
        s["logp"] = torch.zeros(N, device="cuda")
    if own:
        _handles(case, s)
    return s


# ---------------------------------------------------------------- plain forms


def _frequencies(s):
    """(radians per position of every pair, factor of cosine and sine) in 64 bits."""
    case = s["case"]
    rot, theta, factor = case["rot"], s["theta"], case["factor"]
    c = torch.arange(0, rot, 2, device="cuda", dtype=torch.float64)
    if case["scaling"] == "base":
        theta = theta * factor ** (rot / max(1, rot - 2))
    f = theta ** (-c / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] != "parts":
        return f, 1.0
    # pairs that turn 32 times and more in the trained context keep their frequency, those that
    # turn once or less are slowed down by the factor, between them it goes linearly by pair
    pair = lambda turns: rot * math.log(s["trained"] / (2 * math.pi * turns)) / (2 * math.log(theta))
    low, high = max(0, math.floor(pair(32.0))), min(rot - 1, math.ceil(pair(1.0)))
    slowed = ((c / 2 - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
    return f * (1 - slowed) + f / factor * slowed, 0.1 * math.log(factor) + 1.0


def _turn(s):
    """cos and sin [M, 1, rot / 2] in 32 bits, from angles in 64."""
    f, size = _frequencies(s)
    angle = s["pos"].double()[:, None] * f
    return (angle.cos() * size).float()[:, None, :], (angle.sin() * size).float()[:, None, :]


def _halves(case, h):
    rot = case["rot"]
    if case["inter"]:
        return h[..., 0:rot:2], h[..., 1:rot:2]
    return h[..., : rot // 2], h[..., rot // 2: rot]


def _joined(case, a, b, rest):
    pair = torch.stack([a, b], -1).flatten(-2) if case["inter"] else torch.cat([a, b], -1)
    return torch.cat([pair, rest], -1)


def _plain_rope(s):
    case = s["case"]
    M, hq, hkv, hd = case["M"], case["hq"], case["hkv"], case["hd"]
    x = s["qkv"][:, : (hq + hkv) * hd].float().view(M, hq + hkv, hd)
    if case["norm"]:
        gain = torch.cat([s["q_norm"].float().expand(hq, hd), s["k_norm"].float().expand(hkv, hd)])
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * gain
    cs, sn = _turn(s)
    a, b = _halves(case, x)
    s["out"].copy_(_joined(case, a * cs - b * sn, b * cs + a * sn, x[..., case["rot"]:]).reshape(M, -1))
    return [s["out"]]


def _plain_rope_bwd(s):
    case = s["case"]
    M, hq, hkv, hd = case["M"], case["hq"], case["hkv"], case["hd"]
    d = s["dout"].float().view(M, hq + hkv, hd)
    cs, sn = _turn(s)
    a, b = _halves(case, d)
    d = _joined(case, a * cs + b * sn, b * cs - a * sn, d[..., case["rot"]:])
    if not case["norm"]:
        s["out"].copy_(d.reshape(M, -1))
        return [s["out"]]
    x = s["qkv"][:, : (hq + hkv) * hd].float().view(M, hq + hkv, hd)
    gain = torch.cat([s["q_norm"].float().expand(hq, hd), s["k_norm"].float().expand(hkv, hd)])
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    n = x * r
    dg = d * n
    s["dq_norm"].copy_(dg[:, :hq].sum((0, 1), dtype=torch.float64))
    s["dk_norm"].copy_(dg[:, hq:].sum((0, 1), dtype=torch.float64))
    d = d * gain
    s["out"].copy_(((d - n * (d * n).mean(-1, keepdim=True)) * r).reshape(M, -1))
    return [s["out"], s["dq_norm"], s["dk_norm"]]


def _plain_chunk(s):
    """The chunks side by side, filled up to the longest; where that is much, one by one."""
    case, c = s["case"], s["cache"]
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    rep, shape, first = hq // hkv, s["shape"], s["first"]
    size = len(shape) * hq * max(n for n, _ in shape) * max(n for _, n in shape)
    groups = [range(len(shape))] if size <= 2 ** 28 else [[i] for i in range(len(shape))]
    for group in groups:
        B, n, slots = len(group), max(shape[i][0] for i in group), max(shape[i][1] for i in group)
        if n == 0:
            continue
        ids = torch.arange(group[0], group[0] + B, device="cuda")
        table = c["table"][ids, : -(-slots // case["page"])].clamp(min=0).long()

        def rows(name):     # [B, hkv, slots, hd] in 32 bits
            t = c[name][table] if case["fmt"] != "e4m3" else c[name].view(torch.uint8)[table].view(torch.float8_e4m3fn)
            t = t.float()
            if case["fmt"] == "e4m3":
                t = t * c[name + "_scale"][table][..., None]
            return t.permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, hd)[:, :, :slots]

        i = torch.arange(n, device="cuda")[None, :]
        count = s["start"][ids + 1] - s["start"][ids]
        live = i < count[:, None]                                                   # [B, n]
        seen = s["len"][ids][:, None] - count[:, None] + 1 + i
        at = (s["start"][ids][:, None] + i).clamp(max=first[-1] - 1).long()
        q = s["q"][at].float().view(B, n, hkv, rep, hd).permute(0, 2, 3, 1, 4).reshape(B, hkv, rep * n, hd)
        score = (q @ rows("k").transpose(-1, -2)).mul_(1.0 / math.sqrt(hd)).view(B, hkv, rep, n, slots)
        off = torch.arange(slots, device="cuda")[None, None, :] >= seen[..., None]  # [B, n, slots]
        score.masked_fill_(off[:, None, None], -math.inf)
        top = score.amax(-1, keepdim=True)
        base = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
        e = score.sub_(base).exp_()
        total = e.sum(-1, keepdim=True)
        o = (e.view(B, hkv, rep * n, slots) @ rows("v")).view(B, hkv, rep, n, hd) / torch.where(
            total > 0, total, torch.ones_like(total))
        lse = (base + total.log())[..., 0]
        s["o"][at[live]] = o.permute(0, 3, 1, 2, 4).reshape(B, n, hq * hd)[live].to(s["o"].dtype)
        s["lse"][at[live]] = lse.permute(0, 3, 1, 2).reshape(B, n, hq)[live]
        del score, e, off
    return [s["o"], s["lse"]]


def _plain_sample(s):
    """Weights and their sums in 64 bits: a token is chosen by comparing with them."""
    x, order = torch.sort(s["logits"].float() + 0.0, dim=1, descending=True, stable=True)
    V = x.shape[1]
    one = torch.ones(len(x), 1, dtype=torch.float64, device="cuda")
    temp = one if s["temperature"] is None else s["temperature"].double()[:, None]
    greedy = temp <= 0
    w = ((x.double() - x[:, :1].double()) / torch.where(greedy, one, temp)).exp()
    rank = torch.arange(V, device="cuda")[None, :]
    keep = torch.where(greedy, rank < 1, rank >= 0)
    if s["k"] is not None:
        k = s["k"].long()[:, None]
        keep &= (rank < k) | (k <= 0)
    if s["p"] is not None:
        mass = torch.where(keep, w, torch.zeros_like(w))
        before = mass.cumsum(1) - mass
        p = s["p"].double()[:, None]
        keep &= (before < p * mass.sum(1, keepdim=True)) | (p >= 1) | (rank < 1)
        del mass, before
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None].clamp(max=1.0)
    w = torch.where(keep, w, torch.zeros_like(w))
    del keep
    byid = torch.zeros_like(w).scatter_(1, order, w)
    del w, order
    cum = byid.cumsum(1)
    total = cum[:, -1:]
    token = (cum <= s["u"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=V - 1)
    s["token"].copy_(token[:, 0])
    s["logp"].copy_((byid.gather(1, token) / total).log()[:, 0])
    return [s["token"], s["logp"]]


# ---------------------------------------------------------------- the library's calls


def _own_chunk(s):
    s["X"].cache_attention_chunk(s["dims"], s["handle"], s["q"], s["start"], None, s["len"], s["o"], s["ws"],
                                 lse=s["lse"])
    return [s["o"], s["lse"]]


def _own_rope(s):
    s["X"].qk_rope(s["dims"], s["qkv"], s["weights"], s["rope"], s["out"], pos=s["pos"])
    return [s["out"]]


def _own_rope_bwd(s):
    norm = s["case"]["norm"]
    s["X"].qk_rope_bwd(s["dims"], s["qkv"] if norm else None, s["weights"], s["rope"], s["dout"], s["out"],
                       pos=s["pos"], dq_norm=s["dq_norm"] if norm else None, dk_norm=s["dk_norm"] if norm else None,
                       ws=s["ws"] if norm else None)
    return [s["out"], s["dq_norm"], s["dk_norm"]] if norm else [s["out"]]


def _own_sample(s):
    s["X"].sample_tokens(s["logits"], s["u"], s["token"], temperature=s["temperature"], top_k=s["k"], top_p=s["p"],
                         min_p=s["min_p"], logp=s["logp"])
    return [s["token"], s["logp"]]


def run(state):
    op = state["case"]["op"]
    if own:
        call = {"chunk": _own_chunk, "rope": _own_rope, "rope_bwd": _own_rope_bwd, "sample": _own_sample}[op]
    else:
        call = {"chunk": _plain_chunk, "rope": _plain_rope, "rope_bwd": _plain_rope_bwd, "sample": _plain_sample}[op]
    return call(state)


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_chunk(s):
    """One sequence and KV head after the other, over exactly its own slots."""
    case, c = s["case"], s["cache"]
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    rep = hq // hkv
    o = torch.zeros(len(s["q"]), hq, hd, dtype=torch.float64, device="cuda")
    lse = torch.zeros(len(s["q"]), hq, dtype=torch.float64, device="cuda")
    for i, (n, slots) in enumerate(s["shape"]):
        if not n:
            continue
        used = c["table"][i, : -(-slots // case["page"])].long()
        mask = torch.ones(n, slots, dtype=torch.bool, device="cuda").triu(slots - n + 1)
        at = slice(s["first"][i], s["first"][i] + n)
        for g in range(hkv):
            kv = []
            for name in ("k", "v"):
                if case["fmt"] == "e4m3":
                    t = c[name].view(torch.uint8)[used, g].view(torch.float8_e4m3fn).double()
                    t = t * c[name + "_scale"][used, g].double().unsqueeze(-1)
                else:
                    t = c[name][used, g].double()
                kv.append(t.reshape(-1, hd)[:slots])
            q = s["q"][at].double().view(n, hq, hd)[:, g * rep:(g + 1) * rep]
            z = torch.einsum("nhd,md->hnm", q, kv[0]) / hd ** 0.5
            z.masked_fill_(mask, -math.inf)
            total = torch.logsumexp(z, -1)
            lse[at, g * rep:(g + 1) * rep] = total.T
            z -= total[..., None]
            o[at, g * rep:(g + 1) * rep] = torch.einsum("hnm,md->nhd", z.exp_(), kv[1])
            del z
    return [o.view(len(s["q"]), -1), lse]


def _spin(s):
    """The pairs' turns as complex numbers [M, 1, rot / 2], each scaling worked out pair by pair."""
    case = s["case"]
    rot, factor, base = case["rot"], case["factor"], s["theta"]
    freq, size = [], 1.0
    for c in range(rot // 2):
        f = math.pow(base, -2.0 * c / rot)
        if case["scaling"] == "linear":
            f /= factor
        elif case["scaling"] == "base":
            f = math.pow(base * math.pow(factor, rot / max(1.0, rot - 2.0)), -2.0 * c / rot)
        elif case["scaling"] == "parts":
            edge = [rot / 2.0 * math.log(s["trained"] / (2.0 * math.pi * t)) / math.log(base) for t in (32.0, 1.0)]
            lo, hi = max(0, math.floor(edge[0])), min(rot - 1, math.ceil(edge[1]))
            t = min(1.0, max(0.0, (c - lo) / max(hi - lo, 0.001)))
            f = (1.0 - t) * f + t * f / factor
            size = 1.0 + math.log(factor) / 10.0
        freq.append(f)
    angle = s["pos"].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    return torch.polar(torch.full_like(angle, size), angle)[:, None, :]


def _complex(case, h):
    rot = case["rot"]
    if case["inter"]:
        return torch.view_as_complex(h[..., :rot].reshape(*h.shape[:-1], rot // 2, 2).contiguous())
    return torch.complex(h[..., : rot // 2].contiguous(), h[..., rot // 2: rot].contiguous())


def _real(case, z, rest):
    if case["inter"]:
        return torch.cat([torch.view_as_real(z).reshape(*z.shape[:-1], -1), rest], -1)
    return torch.cat([z.real, z.imag, rest], -1)


def _exact_rope(s):
    case = s["case"]
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    out = []
    for at, heads, gain in ((0, hq, s["q_norm"]), (hq, hkv, s["k_norm"])):
        h = s["qkv"][:, at * hd:(at + heads) * hd].double().reshape(-1, heads, hd)
        if gain is not None:
            h = h / torch.sqrt(h.square().sum(-1, keepdim=True) / hd + s["eps"]) * gain.double()
        out.append(_real(case, _complex(case, h) * _spin(s), h[..., case["rot"]:]).reshape(case["M"], -1))
    return [torch.cat(out, 1)]


def _exact_rope_bwd(s):
    """By the norm's Jacobian, blocks of rows at a time."""
    case = s["case"]
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    spin = _spin(s).conj()
    out, sums = [], []
    for at, heads, gain in ((0, hq, s["q_norm"]), (hq, hkv, s["k_norm"])):
        d = s["dout"][:, at * hd:(at + heads) * hd].double().reshape(-1, heads, hd)
        d = _real(case, _complex(case, d) * spin, d[..., case["rot"]:])
        if gain is not None:
            x = s["qkv"][:, at * hd:(at + heads) * hd].double().reshape(-1, heads, hd)
            ms = x.square().sum(-1, keepdim=True) / hd + s["eps"]
            sums.append(torch.einsum("mhd,mhd->d", d, x / ms.sqrt()))
            d = d * gain.double()
            d = d / ms.sqrt() - x * (d * x).sum(-1, keepdim=True) / (hd * ms.sqrt() ** 3)
        out.append(d.reshape(case["M"], -1))
    return [torch.cat(out, 1)] + sums


def _exact_sample(s):
    """A few rows at a time, each filter by the position at which it cuts the sorted row."""
    N, V = s["logits"].shape
    tokens, logps = [], []
    for rows in torch.arange(N, device="cuda").split(128):
        x = s["logits"][rows].double()
        n = len(rows)
        full = torch.full((n, 1), V, dtype=torch.long, device="cuda")
        top, order = torch.sort(x + 0.0, dim=1, descending=True, stable=True)
        temp = torch.ones(n, 1, dtype=torch.float64, device="cuda")
        if s["temperature"] is not None:
            temp = s["temperature"][rows].double()[:, None]
        cold = temp <= 0
        temp = torch.where(cold, torch.ones_like(temp), temp)
        w = torch.exp(top / temp - top[:, :1] / temp)
        sums = torch.cumsum(w, 1)
        cut = torch.where(cold, torch.ones_like(full), full)
        if s["k"] is not None:
            k = s["k"][rows].long()[:, None]
            cut = torch.where(k > 0, torch.minimum(cut, k), cut)
        if s["p"] is not None:
            p = s["p"][rows].double()[:, None]
            within = torch.searchsorted(sums, p * sums.gather(1, cut - 1)) + 1
            cut = torch.where(p < 1, torch.minimum(cut, within), cut)
        if s["min_p"] is not None:
            least = s["min_p"][rows].double()[:, None].clamp(max=1.0)
            cut = torch.minimum(cut, (w >= least).sum(1, keepdim=True))
        prob = torch.zeros_like(w)
        prob.scatter_(1, order, w * (torch.arange(V, device="cuda") < cut) / sums.gather(1, cut - 1))
        steps = torch.cumsum(prob, 1)
        u = s["u"][rows].double()[:, None] * steps[:, -1:]
        token = torch.searchsorted(steps, u, right=True).clamp(max=V - 1)
        tokens.append(token[:, 0].to(torch.int32))
        logps.append(prob.gather(1, token).log()[:, 0])
    return [torch.cat(tokens), torch.cat(logps)]


def exact(case, seed):
    s = prepare(case, seed)
    return {"chunk": _exact_chunk, "rope": _exact_rope, "rope_bwd": _exact_rope_bwd, "sample": _exact_sample}[
        case["op"]](s)
