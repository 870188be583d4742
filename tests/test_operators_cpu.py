"""Host-side checks of the generation operators that need no GPU: bad arguments return
before anything reaches the device, and the binding refuses tensors it cannot pass."""
import ctypes
import math

import pytest

from sparse_depth_token_gb300 import xmod as X

torch = pytest.importorskip("torch")

FAKE = 0x10000      # 16-byte aligned, never dereferenced


def _dims(**kw):
    base = dict(B=1, T=1, d=64, n_heads=4, n_kv_heads=2, head_dim=64, d_ff=64, dtype=X.BF16)
    base.update(kw)
    return X.dims(**base)


def _cache(**kw):
    base = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, table=FAKE, n_pages=8, page_size=16, n_seqs=2,
                max_pages=4, format=X.CACHE_NATIVE)
    base.update(kw)
    return X.KVCache(*[base[n] for n, _ in X.KVCache._fields_])


def _append(dm=None, cache=None, M=3, qkv=FAKE, ld=512, w=None, seq=FAKE, slot=FAKE, pos=FAKE, q=FAKE + (1 << 20),
            ldq=256, status=None):
    return X.load().xmod_cache_append(ctypes.byref(dm or _dims()), ctypes.byref(cache or _cache()), M, qkv, ld,
                                      ctypes.byref(w) if w else None, seq, slot, pos, q, ldq, status, None)


def _attend(dm=None, cache=None, M=3, q=FAKE, ldq=256, seq=None, n=FAKE, o=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40):
    return X.load().xmod_cache_attention(ctypes.byref(dm or _dims()), ctypes.byref(cache or _cache()), M, q, ldq, seq, n,
                                         o, lse, ws, ws_bytes, None)


BAD_CACHES = [dict(k=None), dict(v=FAKE + 8), dict(table=None), dict(table=FAKE + 2), dict(n_pages=0),
              dict(page_size=24), dict(page_size=0), dict(n_seqs=0), dict(max_pages=-1), dict(format=2),
              dict(k_scale=FAKE), dict(format=1), dict(format=1, k_scale=FAKE), dict(max_pages=1 << 28)]


@pytest.mark.parametrize("bad", BAD_CACHES)
@pytest.mark.parametrize("call", [_append, _attend])
def test_bad_caches(call, bad):
    assert call(cache=_cache(**bad)) == X.ERR_INVALID_ARG


@pytest.mark.parametrize("call", [_append, _attend])
def test_bad_dims(call):
    assert call(dm=_dims(n_kv_heads=3)) == X.ERR_INVALID_ARG
    assert call(dm=_dims(dtype=7)) == X.ERR_INVALID_ARG
    assert call(dm=_dims(head_dim=96)) == X.ERR_UNSUPPORTED
    assert call(dm=_dims(head_dim=256)) == X.ERR_UNSUPPORTED
    e4m3 = _cache(format=X.CACHE_E4M3, k_scale=FAKE, v_scale=FAKE)
    assert call(dm=_dims(dtype=X.FP32), cache=e4m3) == X.ERR_UNSUPPORTED
    assert call(cache=_cache(n_pages=1 << 27)) == X.ERR_UNSUPPORTED       # rows past 2^31
    assert call(M=-1) == X.ERR_INVALID_ARG
    assert call(M=0) == X.OK


def test_append_arguments():
    for bad in (dict(qkv=None), dict(qkv=FAKE + 8), dict(ld=504), dict(ld=516), dict(slot=None), dict(slot=FAKE + 2),
                dict(seq=FAKE + 1), dict(pos=FAKE + 3), dict(q=FAKE + 4), dict(ldq=248), dict(ldq=260),
                dict(status=FAKE + 2), dict(q=FAKE, ldq=256)):
        assert _append(**bad) == X.ERR_INVALID_ARG, bad
    assert _append(w=X.LayerWeights(*([None] * 10), 1.0, FAKE + 4)) == X.ERR_INVALID_ARG
    assert _append(w=X.LayerWeights(*([None] * 10), 1.0, None, None, -1.0)) == X.ERR_INVALID_ARG
    assert _append(w=X.LayerWeights(*([None] * 10), 1.0, None, None, math.inf)) == X.ERR_INVALID_ARG


def test_attention_arguments():
    for bad in (dict(q=None), dict(q=FAKE + 8), dict(ldq=248), dict(ldq=260), dict(n=None), dict(n=FAKE + 2),
                dict(seq=FAKE + 2), dict(o=None), dict(o=FAKE + 8), dict(lse=FAKE + 2)):
        assert _attend(**bad) == X.ERR_INVALID_ARG, bad
    assert _attend(ws=None) == X.ERR_WORKSPACE
    assert _attend(ws=FAKE + 8) == X.ERR_WORKSPACE
    need = X.cache_attention_workspace_bytes(_dims(), 3)
    assert need > 0 and _attend(ws_bytes=need - 1) == X.ERR_WORKSPACE
    assert X.cache_attention_workspace_bytes(_dims(n_kv_heads=3), 3) == 0
    assert X.cache_attention_workspace_bytes(_dims(), -1) == 0


def _logprobs(dt=X.BF16, N=3, V=100, x=FAKE, ld=100, t=FAKE, lp=FAKE, h=FAKE, lse=FAKE, k=5, ti=FAKE, tl=FAKE, st=None):
    return X.load().xmod_token_logprobs(dt, N, V, x, ld, t, lp, h, lse, k, ti, tl, st, None)


def _logprobs_bwd(dt=X.BF16, N=3, V=100, x=FAKE, ld=100, t=FAKE, lse=FAKE, h=FAKE, g=FAKE, gh=FAKE, d=FAKE + 4096,
                  ldd=100, st=None):
    return X.load().xmod_token_logprobs_bwd(dt, N, V, x, ld, t, lse, h, g, gh, d, ldd, st, None)


def test_logprob_arguments():
    for bad in (dict(dt=5), dict(N=-1), dict(V=0), dict(ld=99), dict(x=None), dict(x=FAKE + 1), dict(k=-1),
                dict(k=101), dict(k=0), dict(ti=None), dict(tl=None), dict(t=None), dict(lp=None), dict(lp=FAKE + 2),
                dict(h=FAKE + 1), dict(st=FAKE + 2)):
        assert _logprobs(**bad) == X.ERR_INVALID_ARG, bad
    assert _logprobs(k=X.MAX_TOP_K + 1) == X.ERR_UNSUPPORTED
    assert _logprobs(N=0) == X.OK


def test_logprob_gradient_arguments():
    for bad in (dict(dt=5), dict(N=-1), dict(V=0), dict(ld=99), dict(ldd=99), dict(x=None), dict(x=FAKE + 1),
                dict(d=None), dict(d=FAKE + 3), dict(dt=X.FP32, x=FAKE + 2), dict(lse=None), dict(t=None), dict(h=None), dict(g=FAKE + 2),
                dict(d=FAKE, ldd=128), dict(st=FAKE + 1)):
        assert _logprobs_bwd(**bad) == X.ERR_INVALID_ARG, bad
    assert _logprobs_bwd(N=0) == X.OK


def test_top_k_limit_matches_the_header():
    import os
    import re
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "xmod.h")
    assert int(re.search(r"#define\s+XMOD_MAX_TOP_K\s+(\d+)", open(header).read()).group(1)) == X.MAX_TOP_K


def test_vocabulary_limit():
    """Rows past the limit are refused before anything is launched."""
    import os
    import re
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "xmod.h")
    assert re.search(r"#define\s+XMOD_MAX_VOCAB\s+\(1 << 22\)", open(header).read())
    V = X.MAX_VOCAB + 1
    assert V == 2 ** 22 + 1
    assert _logprobs(V=V, ld=V) == X.ERR_UNSUPPORTED
    assert _logprobs_bwd(V=V, ld=V, ldd=V) == X.ERR_UNSUPPORTED


def test_binding_refuses_host_tensors():
    """Host memory is refused before any pointer is taken."""
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    for call in (lambda: X.kv_cache(k, k, torch.zeros(1, 4, dtype=torch.int32)),
                 lambda: X.token_logprobs(torch.zeros(2, 8), None, lse=torch.zeros(2)),
                 lambda: X.token_logprobs_bwd(torch.zeros(2, 8), None, torch.zeros(2), None, torch.zeros(2, 8))):
        with pytest.raises(X.XmodError) as e:
            call()
        assert e.value.status == X.ERR_INVALID_ARG
