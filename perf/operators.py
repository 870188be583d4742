"""Operators around one generation step of the sparse-depth stack, as measured cases.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as the
calls a user makes of the library:

  append     the projections q | k | v of new tokens: QK-norm, rotary embedding at each
             token's own position, keys and values into a paged cache (in the layer's type,
             or in e4m3 with one fp32 scale per token and head), the rotated q to the caller
  attention  one query token per row over that cache: softmax(q K^T / sqrt(hd)) V, query head
             h on KV head h / (hq / hkv), over the first len[m] entries of row m's sequence
  logprobs   log probabilities of given tokens from logits, with the entropy and the top
             alternatives (ties to the lower token)
  logprobs_bwd  the gradient of the log probabilities and the entropy at the logits

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
        # one new token of 8 sequences: the decode step of a dense layer of the A4K8 stack
        dict(name="append 8 tokens", op="append", dtype="bf16", fmt="native", M=8, hq=12, hkv=4, hd=128,
             page=16, max_pages=64, skip=0.0, norm=True, decode=True),
        # the prompts of 8 sequences of 4096 tokens at once
        dict(name="append 32768 prompt tokens", op="append", dtype="bf16", fmt="native", M=32768, hq=12, hkv=4,
             hd=128, page=64, max_pages=64, skip=0.0, norm=True, decode=False),
        # a ragged batch of prompts into an 8-bit cache; every eighth row or so is padding
        dict(name="append 5003 tokens e4m3", op="append", dtype="bf16", fmt="e4m3", M=5003, hq=32, hkv=8, hd=128,
             page=32, max_pages=64, skip=0.12, norm=False, decode=False),
        # one new token of 8 sequences over a sparse layer's cache: 4096 / 8 routed tokens
        dict(name="attend 8x512", op="attention", dtype="bf16", fmt="native", M=8, hq=12, hkv=4, hd=128, page=16,
             max_len=512, ragged=True),
        # a serving batch of 64 sequences of up to 8192 tokens
        dict(name="attend 64x8192 ragged", op="attention", dtype="bf16", fmt="native", M=64, hq=32, hkv=8, hd=128,
             page=64, max_len=8192, ragged=True),
        # a single long sequence: the split over the cache's length carries it
        dict(name="attend 1x131079", op="attention", dtype="bf16", fmt="native", M=1, hq=16, hkv=4, hd=128, page=64,
             max_len=131079, ragged=False),
        # a batch at the A3K16 stack's length over an 8-bit cache
        dict(name="attend 32x16384 e4m3", op="attention", dtype="bf16", fmt="e4m3", M=32, hq=16, hkv=4, hd=128,
             page=32, max_len=16384, ragged=True),
        # the fp32 path at a small model's heads
        dict(name="attend 24x1000 fp32", op="attention", dtype="fp32", fmt="native", M=24, hq=8, hkv=4, hd=64, page=16,
             max_len=1000, ragged=True),
        # the sampled tokens of one step with the alternatives a server reports
        dict(name="logprobs 8 rows top 20", op="logprobs", dtype="bf16", N=8, V=50257, pad=0, top=20, masked=0.3,
             entropy=True),
        # scoring a batch of 4096 prompt positions, with a few alternatives each
        dict(name="logprobs 4096 rows top 5", op="logprobs", dtype="bf16", N=4096, V=50257, pad=0, top=5, masked=0.0,
             entropy=True),
        # training on 4096 positions, entropy term included
        dict(name="logprobs gradient 4096", op="logprobs_bwd", dtype="bf16", N=4096, V=50257, pad=0, masked=0.0,
             entropy=True),
        # a small fp32 batch with an odd vocabulary and padded rows
        dict(name="logprobs gradient 61 fp32", op="logprobs_bwd", dtype="fp32", N=61, V=8191, pad=9, masked=0.1,
             entropy=False),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "logprobs", "logprobs_bwd"])
    if op in ("append", "attention"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        fmt = rng.choice(["native", "native", "e4m3"]) if dtype == "bf16" else "native"
        hq, hkv = rng.choice([(12, 4), (16, 4), (32, 8), (4, 2), (8, 8), (16, 1)])
        hd = rng.choice([128, 128, 128, 64, 32])
        page = rng.choice([16, 32, 64, 128])
    if op == "append":
        decode = rng.random() < 0.4
        M = _log(rng, 1, 600) if decode else _log(rng, 16, 20000 if hq <= 16 else 10000)
        room = min(4096, max(page, 65536 // M)) if decode else 2048
        return dict(op=op, dtype=dtype, fmt=fmt, M=M, hq=hq, hkv=hkv, hd=hd, page=page, max_pages=max(1, room // page),
                    skip=rng.choice([0.0, 0.0, 0.2, 0.9]), norm=rng.random() < 0.5, decode=decode)
    if op == "attention":
        M = _log(rng, 1, 96)
        # at most a gigabyte of keys and values
        size = 1 if fmt == "e4m3" else DTYPES[dtype].itemsize
        most = min(131072, 10 ** 9 // (2 * M * hkv * (hd * size + (4 if fmt == "e4m3" else 0))))
        return dict(op=op, dtype=dtype, fmt=fmt, M=M, hq=hq, hkv=hkv, hd=hd, page=page,
                    max_len=_log(rng, 1, most), ragged=rng.random() < 0.7)
    V = _log(rng, 100, 100000)
    N = _log(rng, 1, min(4096, 10 ** 8 // V))
    case = dict(op=op, dtype=rng.choice(["bf16", "fp32"]), N=N, V=V, pad=rng.choice([0, 0, 3, 8]),
                masked=rng.choice([0.0, 0.2]), entropy=rng.random() < 0.6)
    if op == "logprobs":
        case["top"] = rng.choice([0, 1, 5, 20])
    return case


def _lens(case):
    """The cache lengths of a case's rows (before the seed's shuffle): spread over
    [1, max_len] when ragged, with an empty cache among four rows or more."""
    M, top = case["M"], case["max_len"]
    if not case["ragged"]:
        return [top] * M
    out = [1 + int((top - 1) * (((i + 1) * 0.6180339887) % 1.0)) for i in range(M)]
    out[0] = top
    if M >= 4:
        out[1] = 0
    return out


def _skipped(case):
    return int(case["M"] * case["skip"])


def _esize(case):
    return 1 if case.get("fmt") == "e4m3" else DTYPES[case["dtype"]].itemsize


def work(case):
    op = case["op"]
    es = DTYPES[case["dtype"]].itemsize
    if op == "append":
        rows = case["M"] - _skipped(case)
        q, kv = case["hq"] * case["hd"], 2 * case["hkv"] * case["hd"]
        scales = 8 * case["hkv"] if case["fmt"] == "e4m3" else 0
        return {"bytes": rows * (es * (q + kv) + es * q + _esize(case) * kv + scales) + 12 * case["M"],
                "flops": rows * 7 * (q + kv)}
    if op == "attention":
        keys = sum(_lens(case))
        width = case["hkv"] * case["hd"]
        scales = 8 * case["hkv"] if case["fmt"] == "e4m3" else 0
        return {"bytes": keys * (2 * width * _esize(case) + scales) + case["M"] * case["hq"] * (2 * case["hd"] * es + 4),
                "flops": 4 * keys * case["hq"] * case["hd"]}
    n = case["N"] * case["V"]
    if op == "logprobs":
        return {"bytes": n * es + case["N"] * (16 + 8 * case["top"]), "flops": n * 6}
    return {"bytes": 2 * n * es + 16 * case["N"], "flops": n * 8}


# ---------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _new_cache(case, g, n_seqs, need, max_pages):
    """A cache whose pages lie in shuffled order; `need`[s] of sequence s's table entries
    are pages, the rest -1. Every slot holds values, as after earlier use."""
    page, hkv, hd = case["page"], case["hkv"], case["hd"]
    total = max(1, sum(need))
    n_pages = total + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    counts = torch.tensor(need, device="cuda")
    col = torch.arange(max_pages, device="cuda")[None, :]
    first = torch.cumsum(counts, 0) - counts
    at = (first[:, None] + col).clamp(max=n_pages - 1)
    table = torch.where(col < counts[:, None], order[at], torch.full_like(order[at], -1)).contiguous()
    c = {"table": table, "page": page}
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


def _handles(case, s):
    """What a program that uses the library keeps beside its tensors."""
    from sparse_depth_token_gb300 import xmod as X
    s["X"] = X
    if case["op"] not in ("append", "attention"):
        return
    s["dims"] = X.dims(1, 1, 8 * case["hq"], case["hq"], case["hkv"], case["hd"], 8,
                       X.BF16 if case["dtype"] == "bf16" else X.FP32, s.get("eps", 1e-6))
    c = s["cache"]
    s["handle"] = X.kv_cache(c["k"], c["v"], c["table"], c["k_scale"], c["v_scale"])
    if case["op"] == "append":
        s["weights"] = X.layer_weights({"q_norm": s["q_norm"], "k_norm": s["k_norm"]}, rope_theta=s["theta"])
    else:
        s["ws"] = torch.zeros(X.cache_attention_workspace_bytes(s["dims"], case["M"]), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    r = random.Random(seed)
    s = {"case": case}
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    if op == "append":
        M, hq, hkv, hd, page = (case[k] for k in ("M", "hq", "hkv", "hd", "page"))
        room = page * case["max_pages"]
        if case["decode"]:      # one new token of each sequence
            seq = list(range(M))
            slot = [r.randrange(room) for _ in seq]
        else:                   # whole prompts, one sequence after the other
            seq = [m // room for m in range(M)]
            slot = [m % room for m in range(M)]
        n_seqs = max(seq) + 1
        s["cache"] = _new_cache(case, g, n_seqs, [case["max_pages"]] * n_seqs, case["max_pages"])
        # a sparse layer's cache holds the routed tokens only: their positions run ahead of the slots
        stride = 3
        s["pos"] = _ints([stride * v + q % stride for v, q in zip(slot, seq)])
        for m in r.sample(range(M), _skipped(case)):
            seq[m] = -1
        s["seq"], s["slot"] = _ints(seq), _ints(slot)
        s["qkv"] = torch.empty(M, (hq + 2 * hkv) * hd, dtype=dt, device="cuda").normal_(generator=g)
        s["q_out"] = torch.zeros(M, hq * hd, dtype=dt, device="cuda")
        s["theta"], s["eps"] = 10000.0, 1e-6
        for name in ("q_norm", "k_norm"):
            s[name] = (1 + 0.1 * torch.randn(hd, generator=g, device="cuda")).to(dt) if case["norm"] else None
    elif op == "attention":
        lens = _lens(case)
        r.shuffle(lens)
        page = case["page"]
        need = [-(-n // page) for n in lens]
        s["cache"] = _new_cache(case, g, case["M"], need, max(1, max(need)))
        s["len"] = _ints(lens)
        s["q"] = torch.empty(case["M"], case["hq"] * case["hd"], dtype=dt, device="cuda").normal_(generator=g)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["M"], case["hq"], device="cuda")
    else:
        N, V = case["N"], case["V"]
        x = torch.empty(N, V + case["pad"], device="cuda").normal_(0.0, 2.5, generator=g)
        target = torch.randint(0, V, (N,), generator=g, device="cuda")
        # half of the rows know their token well
        sure = torch.rand(N, generator=g, device="cuda") < 0.5
        x[torch.arange(N, device="cuda"), target] += torch.where(sure, 14.0, 0.0)
        if case["masked"]:      # tokens a grammar or a sampler has ruled out
            off = torch.rand(V + case["pad"], generator=g, device="cuda") < case["masked"]
            x.masked_fill_(off, -math.inf)
            x[torch.arange(N, device="cuda"), target] = 3.0
        s["logits"] = x.to(dt)[:, :V]
        s["target"] = target.to(torch.int32)
        f = dict(device="cuda", dtype=torch.float32)
        if op == "logprobs":
            s["logp"], s["lse"] = torch.empty(N, **f), torch.empty(N, **f)
            s["entropy"] = torch.empty(N, **f) if case["entropy"] else None
            s["top_idx"] = torch.empty(N, case["top"], dtype=torch.int32, device="cuda") if case["top"] else None
            s["top_logp"] = torch.empty(N, case["top"], **f) if case["top"] else None
        else:
            if N > 3:           # padding positions have no token
                s["target"][:: max(3, N // 7)] = -1
            xf = s["logits"].float()
            s["lse"] = torch.logsumexp(xf, 1)
            y = xf - s["lse"][:, None]
            s["entropy"] = -torch.where(y.exp() > 0, y.exp() * y, torch.zeros_like(y)).sum(1)
            del xf, y
            s["g_logp"] = torch.randn(N, generator=g, **f)
            s["g_entropy"] = 0.1 * torch.randn(N, generator=g, **f) if case["entropy"] else None
            s["dlogits"] = torch.empty(N, V, dtype=dt, device="cuda")
    if own:
        _handles(case, s)
    return s


# ---------------------------------------------------------------- plain forms


def _plain_append(s):
    case, c = s["case"], s["cache"]
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    rows = (s["seq"] >= 0).nonzero()[:, 0]
    x = s["qkv"][rows].float().view(len(rows), hq + 2 * hkv, hd)
    pos = s["pos"][rows].double()
    turn = pos[:, None] * s["theta"] ** (-torch.arange(0, hd, 2, device="cuda", dtype=torch.float64) / hd)
    cs, sn = turn.cos().float()[:, None, :], turn.sin().float()[:, None, :]

    def transform(h, gain):
        if gain is not None:
            h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * gain.float()
        a, b = h[..., : hd // 2], h[..., hd // 2:]
        return torch.cat([a * cs - b * sn, b * cs + a * sn], -1)

    q = transform(x[:, :hq], s["q_norm"])
    k = transform(x[:, hq:hq + hkv], s["k_norm"])
    v = x[:, hq + hkv:]
    s["q_out"][rows] = q.reshape(len(rows), hq * hd).to(s["q_out"].dtype)
    slot = s["slot"][rows].long()
    page = c["table"][s["seq"][rows].long(), slot // c["page"]].long()
    off = slot % c["page"]
    out = [s["q_out"]]
    for name, t in (("k", k), ("v", v)):
        if case["fmt"] == "e4m3":
            scale = t.abs().amax(-1) / E4M3_MAX
            code = torch.where(scale[..., None] > 0, t / scale[..., None], torch.zeros_like(t)).to(torch.float8_e4m3fn)
            c[name].view(torch.uint8)[page, :, off] = code.view(torch.uint8)
            c[name + "_scale"][page, :, off] = scale
            out += [c[name], c[name + "_scale"]]
        else:
            c[name][page, :, off] = t.to(c[name].dtype)
            out += [c[name]]
    return out


def _plain_attention(s):
    case, c = s["case"], s["cache"]
    M, hq, hkv, hd = case["M"], case["hq"], case["hkv"], case["hd"]
    table = c["table"].clamp(min=0).long()

    def rows(name):     # [M, hkv, max_pages * page, hd] in 32 bits
        t = c[name][table] if case["fmt"] != "e4m3" else c[name].view(torch.uint8)[table].view(torch.float8_e4m3fn)
        t = t.float()
        if case["fmt"] == "e4m3":
            t = t * c[name + "_scale"][table][..., None]
        return t.permute(0, 2, 1, 3, 4).reshape(M, hkv, -1, hd)

    k = rows("k")
    q = s["q"].float().view(M, hkv, hq // hkv, hd)
    score = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(hd))
    del k
    seen = torch.arange(score.shape[-1], device="cuda")[None, :] < s["len"][:, None]
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    base = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = torch.exp(score - base)
    total = e.sum(-1, keepdim=True)
    o = (e @ rows("v")) / torch.where(total > 0, total, torch.ones_like(total))
    s["o"].copy_(o.reshape(M, hq * hd))
    s["lse"].copy_((base + total.log()).view(M, hq))
    return [s["o"], s["lse"]]


def _plain_logprobs(s):
    case = s["case"]
    N, V = case["N"], case["V"]
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    y = x - top
    e = y.exp()
    total = e.sum(1)
    log_total = total.log()
    lse = top[:, 0] + log_total
    out = [x.gather(1, s["target"].long()[:, None])[:, 0] - lse, lse]
    if case["entropy"]:
        out.append(log_total - torch.where(e > 0, e * y, torch.zeros_like(e)).sum(1) / total)
    if case["top"]:
        del y, e
        bits = (x + 0.0).view(torch.int32)      # -0 counts as 0
        order = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long()
        del bits
        key = (order << 32) | (0xFFFFFFFF - torch.arange(V, device="cuda"))[None, :]
        del order
        best = 0xFFFFFFFF - (torch.topk(key, case["top"], 1).values & 0xFFFFFFFF)
        out += [best.to(torch.int32), x.gather(1, best) - lse[:, None]]
    return out


def _plain_logprobs_bwd(s):
    x = s["logits"].float()
    y = x - s["lse"][:, None]
    p = y.exp()
    t = s["target"].long()
    g = torch.where(t >= 0, s["g_logp"], torch.zeros_like(s["g_logp"]))
    d = -g[:, None] * p
    if s["g_entropy"] is not None:
        inner = torch.where(p > 0, y + s["entropy"][:, None], torch.zeros_like(y))
        d = d - s["g_entropy"][:, None] * p * inner
    d = d.scatter_add(1, t.clamp(min=0)[:, None], g[:, None])
    s["dlogits"].copy_(d)
    return [s["dlogits"]]


# ---------------------------------------------------------------- the library's calls


def _own_append(s):
    c = s["cache"]
    s["X"].cache_append(s["dims"], s["handle"], s["qkv"], s["weights"], s["seq"], s["slot"], s["pos"], s["q_out"])
    return [s["q_out"]] + [c[n] for n in ("k", "k_scale", "v", "v_scale") if c[n] is not None]


def _own_attention(s):
    s["X"].cache_attention(s["dims"], s["handle"], s["q"], None, s["len"], s["o"], s["ws"], lse=s["lse"])
    return [s["o"], s["lse"]]


def _own_logprobs(s):
    s["X"].token_logprobs(s["logits"], s["target"], s["logp"], entropy=s["entropy"], lse=s["lse"],
                          top_idx=s["top_idx"], top_logp=s["top_logp"])
    return [t for t in (s["logp"], s["lse"], s["entropy"], s["top_idx"], s["top_logp"]) if t is not None]


def _own_logprobs_bwd(s):
    s["X"].token_logprobs_bwd(s["logits"], s["target"], s["lse"], s["g_logp"], s["dlogits"],
                              entropy=s["entropy"], g_entropy=s["g_entropy"])
    return [s["dlogits"]]


def run(state):
    op = state["case"]["op"]
    if own:
        call = {"append": _own_append, "attention": _own_attention, "logprobs": _own_logprobs,
                "logprobs_bwd": _own_logprobs_bwd}[op]
    else:
        call = {"append": _plain_append, "attention": _plain_attention, "logprobs": _plain_logprobs,
                "logprobs_bwd": _plain_logprobs_bwd}[op]
    return call(state)


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_append(s):
    """Token by token of the definition, vectorised over tokens: complex rotation."""
    case, c = s["case"], s["cache"]
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    keep = s["seq"] >= 0
    x = s["qkv"].double().reshape(case["M"], -1, hd)
    angle = s["pos"].double()[:, None] / torch.pow(
        torch.tensor(s["theta"], dtype=torch.float64, device="cuda"),
        torch.arange(hd // 2, device="cuda", dtype=torch.float64) * 2 / hd)
    spin = torch.polar(torch.ones_like(angle), angle)[:, None, :]

    def turned(h, gain):
        if gain is not None:
            h = h / torch.sqrt(h.square().sum(-1, keepdim=True) / hd + s["eps"]) * gain.double()
        z = torch.complex(h[..., : hd // 2].contiguous(), h[..., hd // 2:].contiguous()) * spin
        return torch.cat([z.real, z.imag], -1)

    parts = {"k": turned(x[:, hq:hq + hkv], s["k_norm"]), "v": x[:, hq + hkv:]}
    q = torch.where(keep[:, None], turned(x[:, :hq], s["q_norm"]).reshape(case["M"], -1), s["q_out"].double())
    out = [q]
    # flat place of every kept token's rows: ((page * hkv + head) * page_size + offset)
    at = torch.div(s["slot"], c["page"], rounding_mode="floor")
    pages = c["table"].long().gather(0, s["seq"].clamp(min=0).long()[:, None].expand(-1, c["table"].shape[1]))
    page = pages.gather(1, at.long()[:, None])
    heads = torch.arange(hkv, device="cuda")[None, :]
    place = ((page * hkv + heads) * c["page"] + (s["slot"] % c["page"]).long()[:, None])[keep].reshape(-1)
    for name in ("k", "v"):
        t = parts[name][keep].reshape(-1, hd)
        held = c[name].double().reshape(-1, hd)
        if case["fmt"] == "e4m3":
            scale = t.abs().max(-1).values / E4M3_MAX
            held[place] = t / scale[:, None]
            scales = c[name + "_scale"].double().reshape(-1)
            scales[place] = scale
            out += [held.view(c[name].shape), scales.view(c[name + "_scale"].shape)]
        else:
            held[place] = t
            out += [held.view(c[name].shape)]
    return out


def _exact_attention(s):
    """One sequence after the other, over exactly its own entries."""
    case, c = s["case"], s["cache"]
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    o = torch.zeros(case["M"], hq, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((case["M"], hq), -math.inf, dtype=torch.float64, device="cuda")
    for m, n in enumerate(s["len"].tolist()):
        if not n:
            continue
        used = c["table"][m, : -(-n // c["page"])].long()
        kv = []
        for name in ("k", "v"):
            t = c[name].view(torch.uint8)[used].view(c[name].dtype) if case["fmt"] == "e4m3" else c[name][used]
            t = t.double()
            if c[name + "_scale"] is not None:
                t = t * c[name + "_scale"][used].double().unsqueeze(-1)
            kv.append(t.transpose(0, 1).reshape(hkv, -1, hd)[:, :n])
        q = s["q"][m].double().view(hkv, hq // hkv, hd)
        z = torch.einsum("ghd,gnd->ghn", q, kv[0]) / hd ** 0.5
        w = torch.softmax(z, -1)
        o[m] = torch.einsum("ghn,gnd->ghd", w, kv[1]).reshape(hq, hd)
        lse[m] = torch.logsumexp(z, -1).reshape(-1)
    return [o.view(case["M"], -1), lse]


def _exact_logprobs(s):
    case = s["case"]
    N = case["N"]
    outs = []
    for rows in torch.arange(N, device="cuda").split(256):
        x = s["logits"][rows].double()
        lp = torch.log_softmax(x, 1)
        part = [lp[torch.arange(len(rows), device="cuda"), s["target"][rows].long()], torch.logsumexp(x, 1)]
        if case["entropy"]:
            part.append(torch.special.entr(lp.exp()).sum(1))
        if case["top"]:
            idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, : case["top"]]
            part += [idx.to(torch.int32), lp.gather(1, idx)]
        outs.append(part)
    return [torch.cat(p) for p in zip(*outs)]


def _exact_logprobs_bwd(s):
    """d/dx of g log p_t + g_H H, row blocks at a time, from the softmax's Jacobian."""
    case = s["case"]
    outs = []
    for rows in torch.arange(case["N"], device="cuda").split(256):
        p = torch.softmax(s["logits"][rows].double(), 1)
        t = s["target"][rows].long()
        hot = torch.zeros_like(p)
        live = (t >= 0).nonzero()[:, 0]
        hot[live, t[live]] = 1.0
        g = s["g_logp"][rows].double() * (t >= 0)
        d = g[:, None] * (hot - p)
        if s["g_entropy"] is not None:
            ent = torch.special.entr(p)
            d += s["g_entropy"][rows].double()[:, None] * (ent - p * ent.sum(1, keepdim=True))
        outs.append(d)
    return [torch.cat(outs)]


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "logprobs": _exact_logprobs,
            "logprobs_bwd": _exact_logprobs_bwd}[case["op"]](s)
