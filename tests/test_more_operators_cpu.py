"""Host-side checks of the operators around a chunk of tokens that need no GPU: bad arguments
return before anything reaches the device; rotary frequencies."""
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


def _chunk(dm=None, cache=None, n=2, M=3, q=FAKE, ldq=256, start=FAKE, seq=None, lens=FAKE, o=FAKE + (1 << 20), lse=None,
           ws=FAKE, ws_bytes=1 << 40):
    return X.load().xmod_cache_attention_chunk(ctypes.byref(dm or _dims()), ctypes.byref(cache or _cache()), n, M, q, ldq,
                                               start, seq, lens, o, lse, ws, ws_bytes, None)


def test_chunk_arguments():
    for bad in (dict(k=None), dict(v=FAKE + 8), dict(table=None), dict(page_size=24), dict(n_seqs=0), dict(format=2),
                dict(k_scale=FAKE), dict(format=1), dict(max_pages=1 << 28)):
        assert _chunk(cache=_cache(**bad)) == X.ERR_INVALID_ARG, bad
    for bad in (dict(n=-1), dict(M=-1), dict(q=None), dict(q=FAKE + 8), dict(ldq=248), dict(ldq=260), dict(start=None),
                dict(start=FAKE + 2), dict(seq=FAKE + 1), dict(lens=None), dict(lens=FAKE + 2), dict(o=None),
                dict(o=FAKE + (1 << 20) + 8), dict(o=FAKE), dict(lse=FAKE + 2)):
        assert _chunk(**bad) == X.ERR_INVALID_ARG, bad
    assert _chunk(dm=_dims(head_dim=96)) == X.ERR_UNSUPPORTED
    assert _chunk(dm=_dims(n_kv_heads=3)) == X.ERR_INVALID_ARG
    e4m3 = _cache(format=X.CACHE_E4M3, k_scale=FAKE, v_scale=FAKE)
    assert _chunk(dm=_dims(dtype=X.FP32), cache=e4m3) == X.ERR_UNSUPPORTED
    assert _chunk(cache=_cache(n_pages=1 << 27)) == X.ERR_UNSUPPORTED
    assert _chunk(ws=None) == X.ERR_WORKSPACE and _chunk(ws=FAKE + 8) == X.ERR_WORKSPACE
    need = X.cache_attention_chunk_workspace_bytes(_dims(), 2, 3)
    assert need > 0 and _chunk(ws_bytes=need - 1) == X.ERR_WORKSPACE
    assert _chunk(n=0) == X.OK and _chunk(M=0) == X.OK
    assert _chunk(M=(1 << 30) + 1) == X.ERR_UNSUPPORTED      # a segment's last token fits 32 bits
    for args in ((_dims(n_kv_heads=3), 2, 3), (_dims(), -1, 3), (_dims(), 2, -1), (_dims(head_dim=96), 2, 3)):
        assert X.cache_attention_chunk_workspace_bytes(*args) == 0


def _rope(**kw):
    r = X.rope(64)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _fwd(dm=None, M=3, x=FAKE, ldx=512, w=None, rope=None, pos=FAKE, out=FAKE + (1 << 20), ldo=384):
    return X.load().xmod_qk_rope(ctypes.byref(dm or _dims()), M, x, ldx, ctypes.byref(w) if w else None,
                                 ctypes.byref(rope or _rope()), pos, out, ldo, None)


def _bwd(dm=None, M=3, x=FAKE, ldx=512, w=None, rope=None, pos=FAKE, d=FAKE + (1 << 20), ldd=384, out=FAKE + (2 << 20),
         ldo=384, dq=None, dk=None, ws=FAKE, ws_bytes=1 << 40):
    return X.load().xmod_qk_rope_bwd(ctypes.byref(dm or _dims()), M, x, ldx, ctypes.byref(w) if w else None,
                                     ctypes.byref(rope or _rope()), pos, d, ldd, out, ldo, dq, dk, ws, ws_bytes, None)


def test_rope_arguments():
    gains = X.LayerWeights(*([None] * 10), 1.0, FAKE, FAKE)
    for bad in (dict(M=-1), dict(x=None), dict(x=FAKE + 8), dict(ldx=376), dict(ldx=388), dict(pos=FAKE + 2),
                dict(out=None), dict(out=FAKE + 4), dict(ldo=376), dict(ldo=388), dict(out=FAKE, ldo=384),
                dict(w=X.LayerWeights(*([None] * 10), 1.0, FAKE + 4)), dict(rope=_rope(rot_dim=12)),
                dict(rope=_rope(rot_dim=0)), dict(rope=_rope(rot_dim=72)), dict(rope=_rope(amplitude=math.inf)),
                dict(dm=_dims(n_kv_heads=3))):
        assert _fwd(**bad) == X.ERR_INVALID_ARG, bad
    r = _rope()
    r.freq[31] = math.nan
    assert _fwd(rope=r) == X.ERR_INVALID_ARG
    assert _fwd(dm=_dims(head_dim=96)) == X.ERR_UNSUPPORTED
    assert _fwd(M=0) == X.OK
    for bad in (dict(M=-1), dict(d=None), dict(d=FAKE + 8), dict(ldd=376), dict(out=None), dict(ldo=388),
                dict(dq=FAKE), dict(dk=FAKE), dict(w=gains, x=None), dict(w=gains, dq=FAKE + 2),
                dict(w=gains, out=FAKE), dict(out=FAKE + (1 << 20), ldo=392), dict(rope=_rope(rot_dim=20))):
        assert _bwd(**bad) == X.ERR_INVALID_ARG, bad
    assert _bwd(w=gains, dq=FAKE, ws=None) == X.ERR_WORKSPACE
    need = X.qk_rope_bwd_workspace_bytes(_dims(), 3)
    assert need > 0 and _bwd(w=gains, dq=FAKE, ws_bytes=need - 1) == X.ERR_WORKSPACE
    assert X.qk_rope_bwd_workspace_bytes(_dims(), -1) == 0
    assert _bwd(M=0) == X.OK


def test_rope_frequencies():
    for bad in (dict(rot_dim=12), dict(rot_dim=0), dict(rot_dim=136), dict(theta=1.0), dict(theta=math.inf),
                dict(theta=math.nan), dict(scaling=4), dict(scaling=X.ROPE_LINEAR, factor=0.5),
                dict(scaling=X.ROPE_BASE, factor=math.nan), dict(scaling=X.ROPE_PARTS, factor=2.0, trained=0)):
        with pytest.raises(X.XmodError) as e:
            X.rope(128, **bad)
        assert e.value.status == X.ERR_INVALID_ARG, bad
    with pytest.raises(X.XmodError):
        X.rope(64, rot_dim=128)
    r = X.rope(128, 1e4)
    assert r.rot_dim == 128 and r.amplitude == 1.0 and not r.interleaved
    assert all(abs(r.freq[c] / 1e4 ** (-c / 64) - 1) < 1e-14 for c in range(64))
    r = X.rope(64, 5e5, rot_dim=16, interleaved=True, scaling=X.ROPE_LINEAR, factor=4.0)
    assert r.interleaved and all(abs(r.freq[c] * 4 / 5e5 ** (-c / 8) - 1) < 1e-14 for c in range(8))
    assert all(r.freq[c] == 0 for c in range(8, 64))
    # by the base: the fastest pair as it was, the slowest slowed down by the factor
    r = X.rope(64, 1e4, scaling=X.ROPE_BASE, factor=8.0)
    assert r.freq[0] == 1.0 and abs(r.freq[31] * 8 / 1e4 ** (-31 / 32) - 1) < 1e-13
    # by parts: fast pairs as they were, slow ones slowed down, the others between
    r = X.rope(128, 1e4, scaling=X.ROPE_PARTS, factor=16.0, trained=4096)
    plain = [1e4 ** (-c / 64) for c in range(64)]
    lo = math.floor(128 * math.log(4096 / (2 * math.pi * 32)) / (2 * math.log(1e4)))
    hi = math.ceil(128 * math.log(4096 / (2 * math.pi)) / (2 * math.log(1e4)))
    assert 0 < lo < hi < 63
    for c in range(64):
        ratio = r.freq[c] / plain[c]
        if c <= lo:
            assert abs(ratio - 1) < 1e-14
        elif c >= hi:
            assert abs(ratio * 16 - 1) < 1e-13
        else:
            assert abs(ratio - (1 - (c - lo) / (hi - lo) * 15 / 16)) < 1e-13
    assert abs(r.amplitude - (0.1 * math.log(16) + 1)) < 1e-6


def _sample(dt=X.BF16, N=3, V=100, x=FAKE, ld=100, t=FAKE, k=FAKE, p=FAKE, m=FAKE, u=FAKE, tok=FAKE, lp=FAKE, st=None):
    return X.load().xmod_sample_tokens(dt, N, V, x, ld, t, k, p, m, u, tok, lp, st, None)


def test_sample_arguments():
    for bad in (dict(dt=5), dict(N=-1), dict(V=0), dict(ld=99), dict(x=None), dict(x=FAKE + 1), dict(dt=X.FP32, x=FAKE + 2),
                dict(t=FAKE + 2), dict(k=FAKE + 1), dict(p=FAKE + 2), dict(m=FAKE + 3), dict(u=None), dict(u=FAKE + 2),
                dict(tok=None), dict(tok=FAKE + 2), dict(lp=FAKE + 1), dict(st=FAKE + 2)):
        assert _sample(**bad) == X.ERR_INVALID_ARG, bad
    assert _sample(V=X.MAX_VOCAB + 1, ld=X.MAX_VOCAB + 1) == X.ERR_UNSUPPORTED
    assert _sample(N=0) == X.OK


def test_binding_refuses_host_tensors():
    rows, dm = torch.zeros(2, 512, dtype=torch.bfloat16), _dims()
    for call in (lambda: X.sample_tokens(torch.zeros(2, 8), torch.zeros(2), torch.zeros(2, dtype=torch.int32)),
                 lambda: X.qk_rope(dm, rows, None, X.rope(64), rows),
                 lambda: X.qk_rope_bwd(dm, None, None, X.rope(64), rows, rows),
                 lambda: X.cache_attention_chunk(dm, None, rows, None, None, torch.zeros(1, dtype=torch.int32), rows, None)):
        with pytest.raises(X.XmodError) as e:
            call()
        assert e.value.status == X.ERR_INVALID_ARG
