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
