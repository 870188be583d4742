"""Plain 64-bit forms of the operators around a chunk of tokens: its attention over the paged
cache, norms with rotary positions, and sampling."""
from __future__ import annotations

import math

from tests import _cache as C
from tests._gpu import torch


# ------------------------------------------------------------------ attention of a chunk

def chunk_ref(cache, q, s, slots, p_round):
    """(o [n, hq, hd], lse [n, hq], bound of o, bound of lse) of a chunk's queries q [n, hq, hd],
    the last of which sees `slots` slots of sequence s. The bounds are the kernel's arithmetic:
    a score's fp32 dot product of hd terms is off by at most hd 2^-24 sum|q k| / sqrt(hd), a
    probability relatively by twice the largest such error (numerator and denominator), by
    2^-18 (exp, sums) and by p_round, the rounding of the weights; the output is a mean of
    values so weighted."""
    n, hq, hd = q.shape
    seen = slots - n + 1 + torch.arange(n, device="cuda")
    o = torch.zeros(n, hq, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    if slots == 0:
        return o, lse, torch.zeros_like(o), torch.zeros_like(lse)
    rep = hq // cache.hkv
    k = cache.rows("k", s, slots).repeat_interleave(rep, 0)
    v = cache.rows("v", s, slots).repeat_interleave(rep, 0)
    live = (torch.arange(slots, device="cuda")[None, :] < seen[:, None])[:, None, :]     # [n, 1, slots]
    q = q.double()
    z = torch.where(live, torch.einsum("nhd,hmd->nhm", q, k), -math.inf) / math.sqrt(hd)
    size = torch.where(live, torch.einsum("nhd,hmd->nhm", q.abs(), k.abs()), 0.0)
    dz = size.amax(2) * math.sqrt(hd) * 2.0 ** -24
    w = torch.where(live, torch.softmax(z, 2), 0.0)
    some = seen > 0
    # a value that a row does not see may be NaN: row by row only what it sees
    clean = torch.nan_to_num(v, 0.0, 0.0, 0.0)
    o[some] = torch.einsum("nhm,hmd->nhd", w, clean)[some]
    lse[some] = torch.logsumexp(z, 2)[some]
    spread = torch.einsum("nhm,hmd->nhd", w, clean.abs())
    bound = torch.where(some[:, None, None], spread * (2 * dz + 2.0 ** -18 + p_round)[..., None], 0.0)
    return o, lse, bound, torch.where(some[:, None], dz + 2.0 ** -18 + 2.0 ** -23 * lse.abs(), 0.0)


# ------------------------------------------------------------------ norms and rotary positions

def _pairs(x, rot, inter):
    if inter:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _join(a, b, rest, inter):
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1), rest], -1)


def rotate(x, r, pos, back=False):
    """x [M, H, hd] in 64 bits, turned (or turned back) at pos by the structure r; and the scale
    of each element's rounding errors, amplitude (|a| + |b|) over its pair."""
    rot, inter = r.rot_dim, bool(r.interleaved)
    f = torch.tensor(list(r.freq)[:rot // 2], dtype=torch.float64, device="cuda")
    t = (pos.double()[:, None] * f)[:, None, :]
    c, s = t.cos() * r.amplitude, t.sin() * r.amplitude * (-1 if back else 1)
    a, b = _pairs(x, rot, inter)
    size = abs(r.amplitude) * (a.abs() + b.abs())
    rest = x[..., rot:]
    return _join(a * c - b * s, b * c + a * s, rest, inter), _join(size, size, rest.abs(), inter)


def rope_ref(x, gain, eps, r, pos):
    """(out, scale of the rounding errors) of heads x [M, H, hd] in 64 bits."""
    x = x.double()
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.double()
    return rotate(x, r, pos)


def rope_grad_ref(x, gain, eps, r, pos, d):
    """(dx, dgain, scale of dx's rounding errors, sum of |terms| of dgain) in 64 bits."""
    d, size = rotate(d.double(), r, pos, back=True)
    if gain is None:
        return d, None, size, None
    x, g = x.double(), gain.double()
    hd = x.shape[-1]
    inv = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * inv
    dn = d * g
    dx = (dn - n * (dn * n).mean(-1, keepdim=True)) * inv
    err = (size * g.abs() + n.abs() * (size * g.abs() * n.abs()).mean(-1, keepdim=True)) * inv
    assert dx.shape[-1] == hd
    return dx, (d * n).sum((0, 1)), err, (size * n.abs()).sum((0, 1))


# ------------------------------------------------------------------ sampling

def sample_ref(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """(token, logp, margin) of one row in 64 bits; margin: the distance of u, top_p and min_p to
    the nearest border that would change the choice, relative to the sums compared."""
    x = logits.double()
    V = x.numel()
    top, order = torch.sort(x + 0.0, descending=True, stable=True)
    T = 1.0 if temperature is None else float(temperature)
    if T <= 0:
        return int(order[0]), 0.0, 1.0
    w = torch.where(torch.isinf(top) & (top < 0), torch.zeros_like(top), torch.exp((top - top[0]) / T))
    cum = w.cumsum(0)
    cut, margin = V, 1.0
    if top_k is not None and 0 < int(top_k) < V:
        cut = int(top_k)
    if top_p is not None and float(top_p) < 1:
        need = max(float(top_p), 0.0) * cum[cut - 1]
        within = int((cum[:cut] < need).sum()) + 1
        if float(top_p) > 0:
            margin = min(margin, float((cum[:cut] - need).abs().min() / cum[cut - 1]))
        cut = min(cut, within)
    if min_p is not None and float(min_p) > 0:
        least = min(float(min_p), 1.0)
        ratio = w / least
        off = (ratio - 1).abs()
        margin = min(margin, float(off[off > 0].min()) if bool((off > 0).any()) else 1.0)
        cut = min(cut, int((w >= least).sum()))
    kept = torch.zeros_like(w)
    kept[order[:cut]] = w[:cut]
    run = kept.cumsum(0)
    total = run[-1]
    token = int((run <= float(u) * total).sum())
    alive = kept > 0
    if float(u) > 0:
        margin = min(margin, float((run[alive] / total - float(u)).abs().min()))
    return token, math.log(float(kept[token] / total)), margin


dims = C.dims
