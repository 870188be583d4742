"""Plain 64-bit forms of the key/value cache operators, and caches to run them on."""
from __future__ import annotations

import math

import numpy as np

from tests._gpu import torch

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}     # half a step, relative
E4M3_MAX = 448.0


def dims(X, hq, hkv, hd, dtype, eps=1e-6):
    return X.dims(1, 1, 64, hq, hkv, hd, 64, X.BF16 if dtype == "bf16" else X.FP32, eps)


class Cache:
    """A paged cache on the GPU: `rooms` slots for each sequence, pages in shuffled order,
    every slot holding `fill` (NaN by default), table entries past a sequence's pages -1."""

    def __init__(self, X, rooms, hkv, hd, page, dtype, e4m3=False, fill=math.nan, seed=0, spare=2,
                 first_page=0):
        r = np.random.default_rng(seed)
        need = [-(-n // page) for n in rooms]
        self.n_pages = first_page + sum(need) + spare
        order = first_page + r.permutation(sum(need) + spare)
        self.table_np = np.full((len(rooms), max(1, max(need))), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table_np[s, :n] = order[at:at + n]
            at += n
        self.page, self.hkv, self.hd, self.e4m3, self.dtype = page, hkv, hd, e4m3, dtype
        shape = (self.n_pages, hkv, page, hd)
        t = torch.float8_e4m3fn if e4m3 else DT[dtype]
        new = torch.empty if first_page else (lambda *a, **k: torch.full(a[0], fill, **k))
        self.k, self.v = (new(shape, dtype=t, device="cuda") for _ in range(2))
        self.k_scale = self.v_scale = None
        if e4m3:
            self.k_scale, self.v_scale = (torch.full(shape[:3], fill, device="cuda") for _ in range(2))
        self.table = torch.from_numpy(self.table_np).cuda()
        self.handle = X.kv_cache(self.k, self.v, self.table, self.k_scale, self.v_scale)

    def place(self, s, i):
        return int(self.table_np[s, i // self.page]), i % self.page

    def fill(self, s, n, seed, scale=1.0):
        """Random keys and values in the first n slots of sequence s."""
        g = torch.Generator().manual_seed(seed)
        pages = torch.from_numpy(self.table_np[s, :-(-n // self.page)].astype(np.int64)).cuda()
        for name in ("k", "v"):
            x = torch.randn(len(pages), self.hkv, self.page, self.hd, generator=g).cuda() * scale
            live = (torch.arange(len(pages) * self.page).view(len(pages), self.page) < n).cuda()
            x = torch.where(live[:, None, :, None], x, torch.full_like(x, math.nan))
            if self.e4m3:
                getattr(self, name).view(torch.uint8)[pages] = (x * 100).clamp(-448, 448).to(
                    torch.float8_e4m3fn).view(torch.uint8)
                sc = (0.005 + 0.01 * torch.rand(len(pages), self.hkv, self.page, generator=g)).cuda()
                getattr(self, name + "_scale")[pages] = torch.where(
                    live[:, None, :], sc, torch.full_like(sc, math.nan))
            else:
                getattr(self, name)[pages] = x.to(DT[self.dtype])

    def rows(self, name, s, n):
        """[hkv, n, hd] in 64 bits."""
        pages = torch.from_numpy(self.table_np[s, :-(-n // self.page)].astype(np.int64)).cuda()
        t = getattr(self, name)
        t = (t.view(torch.uint8)[pages].view(t.dtype) if self.e4m3 else t[pages]).double()
        if self.e4m3:
            t = t * getattr(self, name + "_scale")[pages].double()[..., None]
        return t.permute(1, 0, 2, 3).reshape(self.hkv, -1, self.hd)[:, :n]

    def tensors(self):
        return [t for t in (self.k, self.v, self.k_scale, self.v_scale) if t is not None]


def attention_ref(cache, q, s, n, p_round):
    """(o [hq, hd], lse [hq], bound [hq, hd]) of one query q [hq, hd] over n >= 1 slots in
    64 bits; bound: the kernel's arithmetic error. A score's fp32 dot product of hd terms
    is off by at most hd 2^-24 sum|q k| / sqrt(hd), a probability relatively by twice the
    largest such error (numerator and denominator), by 2^-18 (exp, sums) and by p_round,
    the rounding of the probabilities; the output is a mean of values so weighted."""
    hq, hd = q.shape
    rep = hq // cache.hkv
    k = cache.rows("k", s, n).repeat_interleave(rep, 0)
    v = cache.rows("v", s, n).repeat_interleave(rep, 0)
    q = q.double()
    z = torch.einsum("hd,hnd->hn", q, k) / math.sqrt(hd)
    dz = torch.einsum("hd,hnd->hn", q.abs(), k.abs()).amax(1) * math.sqrt(hd) * 2.0 ** -24
    w = torch.softmax(z, 1)
    o = torch.einsum("hn,hnd->hd", w, v)
    spread = torch.einsum("hn,hnd->hd", w, v.abs())
    return o, torch.logsumexp(z, 1), spread * (2 * dz + 2.0 ** -18 + p_round)[:, None], dz


def transform_ref(x, gain, eps, theta, pos):
    """QK-norm and rotation of heads x [M, H, hd] at pos [M], in 64 bits; and the scale of
    each element's rounding errors, |a| + |b| over its pair after the norm."""
    x = x.double()
    hd = x.shape[-1]
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.double()
    a, b = x[..., :hd // 2], x[..., hd // 2:]
    size = (a.abs() + b.abs()).repeat(1, 1, 2)
    if theta:
        ang = pos.double()[:, None] * theta ** (
            -2.0 * torch.arange(hd // 2, dtype=torch.float64, device=x.device) / hd)
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        a, b = a * c - b * s, b * c + a * s
    return torch.cat([a, b], -1), size
