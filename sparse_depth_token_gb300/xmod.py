"""Thin Python binding of the C ABI in include/xmod.h (argument marshalling only).

Every function forwards device pointers (torch tensors' data_ptr()) and the
current CUDA stream to libxmod.so; all computation happens in the library's
CUDA kernels. There is no fallback: if the library is missing or fails to load,
load() raises.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

OK = 0
ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_DEVICE_CHECK, ERR_WORKSPACE = (
    -1, -2, -3, -4, -5, -6)
BF16, FP32 = 0, 1
GATE_XMOD, GATE_MOD = 0, 1
LAYER_DENSE, LAYER_SPARSE, LAYER_ATTN, LAYER_ROUTED_FFN, LAYER_SPARSE_FULLKV = 0, 1, 2, 3, 4

EXPORTS = ("xmod_version", "xmod_status_string", "xmod_workspace_bytes", "xmod_reset_status",
           "xmod_sync_status", "xmod_router_topk", "xmod_topk", "xmod_gather", "xmod_block_fwd",
           "xmod_gated_scatter", "xmod_layer_fwd", "xmod_stack_fwd", "xmod_launch_count",
           "xmod_profile_enable", "xmod_profile_read", "xmod_router_topk_noalloc",
           "xmod_stack_fwd_ex", "xmod_layer_fwd_threshold", "xmod_stack_fwd_sched",
           "xmod_bwd_workspace_bytes", "xmod_layer_bwd", "xmod_stack_bwd_workspace_bytes",
           "xmod_stack_bwd", "xmod_selftest_wait_timeout", "xmod_cache_append",
           "xmod_cache_attention_workspace_bytes", "xmod_cache_attention", "xmod_token_logprobs",
           "xmod_token_logprobs_bwd", "xmod_cache_attention_chunk_workspace_bytes",
           "xmod_cache_attention_chunk", "xmod_rope_init", "xmod_qk_rope",
           "xmod_qk_rope_bwd_workspace_bytes", "xmod_qk_rope_bwd", "xmod_sample_tokens")

CACHE_NATIVE, CACHE_E4M3 = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_PARTS = 0, 1, 2, 3
MAX_TOP_K = 64   # alternatives token_logprobs reports at most
MAX_VOCAB = 1 << 22   # logits of a row of token_logprobs and its gradient at most

# Largest B*T the allocation-free router entry point accepts (its fixed scratch).
NOALLOC_MAX_TOKENS = 2 * 1024 * 1024


class XmodError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} ({status})")


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("d", ctypes.c_int),
                ("n_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("d_ff", ctypes.c_int), ("dtype", ctypes.c_int),
                ("rms_eps", ctypes.c_float)]


class LayerWeights(ctypes.Structure):
    NAMES = ("w_router", "rms1", "wq", "wk", "wv", "wo", "rms2", "w_gate", "w_up", "w_down")
    _fields_ = [(n, ctypes.c_void_p) for n in NAMES] + [
        ("varsigma", ctypes.c_float), ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
        ("rope_theta", ctypes.c_float)]


class LayerGrads(ctypes.Structure):
    NAMES = ("w_router", "rms1", "wq", "wk", "wv", "wo", "rms2", "w_gate", "w_up", "w_down",
             "varsigma", "route_loss", "q_norm", "k_norm")
    _fields_ = [(n, ctypes.c_void_p) for n in NAMES]


ROUTE_TOPK, ROUTE_THRESHOLD = 0, 1


class StackOpts(ctypes.Structure):
    _fields_ = [("bias_step", ctypes.c_float), ("layer_stats", ctypes.c_void_p),
                ("update_hist", ctypes.c_void_p), ("routing", ctypes.c_int)]


class KVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("n_seqs", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("format", ctypes.c_int)]


class Rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("amplitude", ctypes.c_float), ("freq", ctypes.c_double * 64)]


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int),
                ("total_ms", ctypes.c_double)]


_VP = ctypes.c_void_p
_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libxmod.so (building it first if allowed). Raises if unavailable."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if not os.path.exists(path) or not _build.up_to_date():
        if not build_if_missing:
            raise RuntimeError(f"CUDA library not built: {path}")
        _build.build()
    L = ctypes.CDLL(path)
    L.xmod_version.restype = ctypes.c_char_p
    L.xmod_status_string.restype = ctypes.c_char_p
    L.xmod_status_string.argtypes = [ctypes.c_int]
    L.xmod_workspace_bytes.restype = ctypes.c_size_t
    L.xmod_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int]
    L.xmod_reset_status.argtypes = [_VP, ctypes.c_size_t, _VP]
    L.xmod_sync_status.argtypes = [_VP, _VP]
    L.xmod_router_topk.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, _VP, _VP, _VP, _VP, _VP,
                                   _VP, _VP, _VP, ctypes.c_size_t, _VP]
    L.xmod_topk.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, _VP, _VP, _VP, _VP,
                            ctypes.c_size_t, _VP]
    L.xmod_gather.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, _VP, _VP, _VP, _VP, _VP]
    L.xmod_block_fwd.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, _VP, _VP,
                                 ctypes.POINTER(LayerWeights), _VP, _VP, _VP, ctypes.c_size_t, _VP]
    L.xmod_gated_scatter.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, _VP, _VP, _VP, _VP, _VP,
                                     ctypes.c_float, ctypes.c_int, _VP, _VP]
    L.xmod_layer_fwd.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                 ctypes.POINTER(LayerWeights), _VP, _VP, _VP, _VP, _VP,
                                 ctypes.c_size_t, _VP]
    L.xmod_stack_fwd.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, ctypes.c_double, ctypes.c_int,
                                 ctypes.c_int, ctypes.c_int, ctypes.POINTER(LayerWeights),
                                 ctypes.c_int, _VP, _VP, _VP, ctypes.c_size_t, _VP]
    L.xmod_stack_fwd_ex.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, ctypes.c_double,
                                    ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                    ctypes.POINTER(LayerWeights), ctypes.c_int, _VP, _VP,
                                    ctypes.POINTER(StackOpts), _VP, ctypes.c_size_t, _VP]
    L.xmod_stack_fwd_sched.argtypes = [ctypes.POINTER(Dims), ctypes.c_int,
                                       ctypes.POINTER(ctypes.c_int32), ctypes.c_int, ctypes.c_int,
                                       ctypes.POINTER(LayerWeights), _VP, _VP,
                                       ctypes.POINTER(StackOpts), _VP, ctypes.c_size_t, _VP]
    L.xmod_layer_fwd_threshold.argtypes = [ctypes.POINTER(Dims), ctypes.c_int,
                                           ctypes.POINTER(LayerWeights), _VP, _VP, _VP, _VP,
                                           ctypes.c_size_t, _VP]
    L.xmod_launch_count.restype = ctypes.c_uint64
    L.xmod_profile_enable.argtypes = [ctypes.c_int]
    L.xmod_profile_read.argtypes = [ctypes.POINTER(KernelTime), ctypes.c_int,
                                    ctypes.POINTER(ctypes.c_int)]
    L.xmod_router_topk_noalloc.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, _VP, _VP, _VP, _VP,
                                           _VP, _VP, _VP]
    L.xmod_selftest_wait_timeout.argtypes = [_VP, ctypes.c_size_t, _VP]
    L.xmod_bwd_workspace_bytes.restype = ctypes.c_size_t
    L.xmod_bwd_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int]
    L.xmod_layer_bwd.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                 ctypes.POINTER(LayerWeights), _VP, _VP, _VP, ctypes.c_float,
                                 _VP, ctypes.POINTER(LayerGrads), _VP, ctypes.c_size_t, _VP]
    L.xmod_stack_bwd_workspace_bytes.restype = ctypes.c_size_t
    L.xmod_stack_bwd_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int]
    L.xmod_stack_bwd.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, ctypes.c_double,
                                 ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                 ctypes.POINTER(LayerWeights), ctypes.c_int, _VP, _VP, _VP,
                                 ctypes.c_float, _VP, ctypes.POINTER(LayerGrads), _VP, _VP,
                                 ctypes.c_size_t, _VP]
    L.xmod_cache_append.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(KVCache), ctypes.c_int,
                                    _VP, ctypes.c_int, ctypes.POINTER(LayerWeights), _VP, _VP,
                                    _VP, _VP, ctypes.c_int, _VP, _VP]
    L.xmod_cache_attention_workspace_bytes.restype = ctypes.c_size_t
    L.xmod_cache_attention_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int]
    L.xmod_cache_attention.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(KVCache),
                                       ctypes.c_int, _VP, ctypes.c_int, _VP, _VP, _VP, _VP, _VP,
                                       ctypes.c_size_t, _VP]
    L.xmod_token_logprobs.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int, _VP,
                                      ctypes.c_int64, _VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP,
                                      _VP, _VP]
    L.xmod_token_logprobs_bwd.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int, _VP,
                                          ctypes.c_int64, _VP, _VP, _VP, _VP, _VP, _VP,
                                          ctypes.c_int64, _VP, _VP]
    L.xmod_cache_attention_chunk_workspace_bytes.restype = ctypes.c_size_t
    L.xmod_cache_attention_chunk_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int,
                                                             ctypes.c_int]
    L.xmod_cache_attention_chunk.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(KVCache),
                                             ctypes.c_int, ctypes.c_int, _VP, ctypes.c_int, _VP,
                                             _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]
    L.xmod_rope_init.argtypes = [ctypes.POINTER(Rope), ctypes.c_int, ctypes.c_int,
                                 ctypes.c_double, ctypes.c_int, ctypes.c_double, ctypes.c_int]
    L.xmod_qk_rope.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, _VP, ctypes.c_int,
                               ctypes.POINTER(LayerWeights), ctypes.POINTER(Rope), _VP, _VP,
                               ctypes.c_int, _VP]
    L.xmod_qk_rope_bwd_workspace_bytes.restype = ctypes.c_size_t
    L.xmod_qk_rope_bwd_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int]
    L.xmod_qk_rope_bwd.argtypes = [ctypes.POINTER(Dims), ctypes.c_int, _VP, ctypes.c_int,
                                   ctypes.POINTER(LayerWeights), ctypes.POINTER(Rope), _VP, _VP,
                                   ctypes.c_int, _VP, ctypes.c_int, _VP, _VP, _VP,
                                   ctypes.c_size_t, _VP]
    L.xmod_sample_tokens.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int, _VP,
                                     ctypes.c_int64, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]
    _lib = L
    return L


def _p(t):
    """Device pointer of a tensor (None passes NULL). Raw ints pass through."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _raw_stream(stream, dev):
    """A stream's handle; None: the current one's (a Stream object costs as much to build as
    a kernel to launch)."""
    if stream is None:
        return _torch_module._C._cuda_getCurrentRawStream(dev)
    return _stream(stream)


def _stream(stream):
    if stream is None:
        return _torch().cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, st):
    if st != OK:
        raise XmodError(fn, st)


def version() -> str:
    return load().xmod_version().decode()


def status_string(st: int) -> str:
    return load().xmod_status_string(int(st)).decode()


def dims(B, T, d, n_heads, n_kv_heads, head_dim, d_ff, dtype=BF16, rms_eps=1e-6) -> Dims:
    return Dims(B, T, d, n_heads, n_kv_heads, head_dim, d_ff, dtype, rms_eps)


def layer_weights(tensors: dict, varsigma: float = 1.0, rope_theta: float = 0.0) -> LayerWeights:
    """tensors: name -> device tensor for the names of LayerWeights.NAMES, plus the
    optional QK-norm gains "q_norm" / "k_norm" [head_dim]; rope_theta > 0 turns on the
    rotary embedding. The struct keeps a reference to the tensors so their memory
    outlives every call using it."""
    lw = LayerWeights(*[_p(tensors.get(n)) for n in LayerWeights.NAMES], float(varsigma),
                      _p(tensors.get("q_norm")), _p(tensors.get("k_norm")), float(rope_theta))
    lw._keep = dict(tensors)
    lw._gains = [(t.dtype, t.numel(), t.is_contiguous(), t.get_device())
                 for t in (tensors.get("q_norm"), tensors.get("k_norm")) if hasattr(t, "dtype")]
    return lw


def workspace_bytes(dm: Dims, K: int) -> int:
    return int(load().xmod_workspace_bytes(ctypes.byref(dm), int(K)))


def reset_status(ws, stream=None):
    _check("xmod_reset_status", load().xmod_reset_status(_p(ws), ws.numel() * ws.element_size(),
                                                         _stream(stream)))


def sync_status(ws, stream=None) -> int:
    return int(load().xmod_sync_status(_p(ws), _stream(stream)))


def _wsb(ws):
    return ws.numel() * ws.element_size() if ws is not None else 0


def router_topk(dm, K, x, w_r, bias, logits, r, idx, r_sel, ws, stream=None):
    _check("xmod_router_topk", load().xmod_router_topk(
        ctypes.byref(dm), int(K), _p(x), _p(w_r), _p(bias), _p(logits), _p(r), _p(idx), _p(r_sel),
        _p(ws), _wsb(ws), _stream(stream)))


def topk(dm, K, logits, idx, r_sel, ws, stream=None):
    _check("xmod_topk", load().xmod_topk(ctypes.byref(dm), int(K), _p(logits), _p(idx), _p(r_sel),
                                         _p(ws), _wsb(ws), _stream(stream)))


def gather(dm, K, x, idx, xs, stream=None, status=None):
    """status: None, or a device int32 tensor that receives XMOD_ERR_DEVICE_CHECK when a
    position is out of range or not ascending (that row is skipped)."""
    _check("xmod_gather", load().xmod_gather(ctypes.byref(dm), int(K), _p(x), _p(idx), _p(xs),
                                             _p(status), _stream(stream)))


def block_fwd(dm, n_per_seq, xs, idx, w: LayerWeights, a_out, f_out, ws, stream=None):
    _check("xmod_block_fwd", load().xmod_block_fwd(
        ctypes.byref(dm), int(n_per_seq), _p(xs), _p(idx), ctypes.byref(w), _p(a_out), _p(f_out),
        _p(ws), _wsb(ws), _stream(stream)))


def gated_scatter(dm, K, x, idx, r_sel, a, f, varsigma, gate, stream=None, status=None):
    """status: as for gather (a bad position's row is not written)."""
    _check("xmod_gated_scatter", load().xmod_gated_scatter(
        ctypes.byref(dm), int(K), _p(x), _p(idx), _p(r_sel), _p(a), _p(f), float(varsigma),
        int(gate), _p(status), _stream(stream)))


def layer_fwd(dm, kind, K, gate, w: LayerWeights, x, bias, idx_out, r_sel_out, ws, stream=None):
    _check("xmod_layer_fwd", load().xmod_layer_fwd(
        ctypes.byref(dm), int(kind), int(K), int(gate), ctypes.byref(w), _p(x), _p(bias),
        _p(idx_out), _p(r_sel_out), _p(ws), _wsb(ws), _stream(stream)))


def stack_fwd(dm, K, A, N0, N1, gate, layers, x, bias, ws, stream=None):
    # the array copies the structs; the caller's LayerWeights keep the tensors alive
    arr = (LayerWeights * len(layers))(*layers)
    _check("xmod_stack_fwd", load().xmod_stack_fwd(
        ctypes.byref(dm), int(K), float(A), int(N0), int(N1), int(gate), arr, len(layers), _p(x),
        _p(bias), _p(ws), _wsb(ws), _stream(stream)))


def stack_fwd_ex(dm, K, A, N0, N1, gate, layers, x, bias, ws, bias_step=0.0, layer_stats=None,
                 update_hist=None, routing=ROUTE_TOPK, stream=None):
    """xmod_stack_fwd_ex: the stack with the token-choice bias dynamics (bias_step), the
    selection rule (ROUTE_TOPK or ROUTE_THRESHOLD) and, when given, the routing
    statistics: layer_stats int32 [n_sparse, B, 4] and update_hist int32
    [N1, B, AK + 1] (device tensors)."""
    arr = (LayerWeights * len(layers))(*layers)
    opts = StackOpts(float(bias_step), _p(layer_stats), _p(update_hist), int(routing))
    _check("xmod_stack_fwd_ex", load().xmod_stack_fwd_ex(
        ctypes.byref(dm), int(K), float(A), int(N0), int(N1), int(gate), arr, len(layers), _p(x),
        _p(bias), ctypes.byref(opts), _p(ws), _wsb(ws), _stream(stream)))


def stack_fwd_sched(dm, K, kinds, gate, layers, x, bias, ws, bias_step=0.0, layer_stats=None,
                    update_hist=None, routing=ROUTE_TOPK, stream=None):
    """xmod_stack_fwd_sched: the stack in an explicit layer order (kinds: DENSE / SPARSE
    per layer), e.g. the segment stacks of X-MoD notes Eq. 35 / 36."""
    arr = (LayerWeights * len(layers))(*layers)
    ks = (ctypes.c_int32 * len(kinds))(*[int(k) for k in kinds])
    opts = StackOpts(float(bias_step), _p(layer_stats), _p(update_hist), int(routing))
    _check("xmod_stack_fwd_sched", load().xmod_stack_fwd_sched(
        ctypes.byref(dm), int(K), ks, len(kinds), int(gate), arr, _p(x), _p(bias),
        ctypes.byref(opts), _p(ws), _wsb(ws), _stream(stream)))


def layer_fwd_threshold(dm, gate, w, x, bias, ws, count_out=None, stream=None):
    """xmod_layer_fwd_threshold: one sparse layer under the causal threshold rule;
    count_out (device int32 [B]) receives each sequence's routed token count."""
    _check("xmod_layer_fwd_threshold", load().xmod_layer_fwd_threshold(
        ctypes.byref(dm), int(gate), ctypes.byref(w), _p(x), _p(bias), _p(count_out), _p(ws),
        _wsb(ws), _stream(stream)))


def launch_count() -> int:
    return int(load().xmod_launch_count())


def profile_enable(on: bool) -> None:
    load().xmod_profile_enable(1 if on else 0)


def profile_read(max_kinds: int = 64) -> dict:
    """{kernel kind: (launches, total_ms)} recorded since the last read."""
    arr = (KernelTime * max_kinds)()
    n = ctypes.c_int(0)
    _check("xmod_profile_read", load().xmod_profile_read(arr, max_kinds, ctypes.byref(n)))
    return {arr[i].name.decode(): (arr[i].launches, arr[i].total_ms) for i in range(n.value)}


def router_topk_noalloc(dm, K, x, w_r, bias, idx, r_sel, status=None, stream=None):
    """xmod_router_topk without a workspace, for callers that cannot allocate device
    memory: the library's own fixed scratch holds the logits (B*T <= NOALLOC_MAX_TOKENS).
    `status` (optional device int32 tensor) receives the call's device status."""
    if dm.B * dm.T > NOALLOC_MAX_TOKENS:
        raise XmodError("xmod_router_topk_noalloc", ERR_UNSUPPORTED)
    _check("xmod_router_topk_noalloc", load().xmod_router_topk_noalloc(
        ctypes.byref(dm), int(K), _p(x), _p(w_r), _p(bias), _p(idx), _p(r_sel), _p(status),
        _stream(stream)))


def bwd_workspace_bytes(dm: Dims, K: int) -> int:
    return int(load().xmod_bwd_workspace_bytes(ctypes.byref(dm), int(K)))


def layer_grads(tensors: dict) -> LayerGrads:
    """LayerGrads from fp32 device tensors keyed by LayerGrads.NAMES (missing: NULL)."""
    return LayerGrads(*[_p(tensors.get(n)) for n in LayerGrads.NAMES])


def layer_bwd(dm, kind, K, gate, w: LayerWeights, x, bias, dy, route_coef, dx, grads: LayerGrads,
              ws, stream=None):
    """xmod_layer_bwd: dx and the weight gradients of sum(dy * y) + route_coef * L_route."""
    _check("xmod_layer_bwd", load().xmod_layer_bwd(
        ctypes.byref(dm), int(kind), int(K), int(gate), ctypes.byref(w), _p(x), _p(bias), _p(dy),
        float(route_coef), _p(dx), ctypes.byref(grads), _p(ws), _wsb(ws), _stream(stream)))


def stack_bwd_workspace_bytes(dm: Dims, K: int) -> int:
    return int(load().xmod_stack_bwd_workspace_bytes(ctypes.byref(dm), int(K)))


def stack_bwd(dm, K, A, N0, N1, gate, layers, x, bias, dy, route_coef, dx, grads, checkpoints,
              ws, stream=None):
    """xmod_stack_bwd: the Eq. 3 stack's backward; grads is a list of LayerGrads (one per
    layer), checkpoints a device buffer [n_layers, B, T, d]."""
    arr = (LayerWeights * len(layers))(*layers)
    garr = (LayerGrads * len(grads))(*grads)
    _check("xmod_stack_bwd", load().xmod_stack_bwd(
        ctypes.byref(dm), int(K), float(A), int(N0), int(N1), int(gate), arr, len(layers), _p(x),
        _p(bias), _p(dy), float(route_coef), _p(dx), garr, _p(checkpoints), _p(ws), _wsb(ws),
        _stream(stream)))


def kv_cache(k, v, table, k_scale=None, v_scale=None) -> KVCache:
    """KVCache from device tensors: k, v [n_pages, n_kv_heads, page_size, head_dim]
    contiguous (with k_scale / v_scale [n_pages, n_kv_heads, page_size] fp32: e4m3 codes,
    as float8_e4m3fn or plain bytes), table [n_seqs, max_pages] int32 contiguous. The struct
    keeps the tensors, so their memory outlives every call using it."""
    T = _torch()
    e4m3 = k_scale is not None
    ts = (k, v, table) + ((k_scale, v_scale) if e4m3 else ())
    if (any(t is None or not t.is_cuda or t.device != k.device or not t.is_contiguous()
            for t in ts) or k.dim() != 4
            or table.dim() != 2 or k.shape != v.shape or k.dtype is not v.dtype
            or table.dtype is not T.int32 or (v_scale is not None) != e4m3
            or (e4m3 and (k.dtype not in (T.float8_e4m3fn, T.uint8, T.int8) or any(
                t.shape != k.shape[:3] or t.dtype is not T.float32 for t in ts[3:])))):
        raise XmodError("kv_cache", ERR_INVALID_ARG)
    c = KVCache(_p(k), _p(v), _p(k_scale), _p(v_scale), _p(table), k.shape[0], k.shape[2],
                table.shape[0], table.shape[1], CACHE_E4M3 if e4m3 else CACHE_NATIVE)
    c._keep = ts
    c.n_kv_heads, c.head_dim, c.dtype, c.device = k.shape[1], k.shape[3], k.dtype, k.get_device()
    return c


def _device(fn, t):
    """Device index of a tensor; it has to be the current device."""
    dev = t.get_device()
    if dev < 0 or dev != (_torch_module or _torch())._C._cuda_getDevice():
        raise XmodError(fn, ERR_INVALID_ARG)
    return dev


def _vec(fn, t, dtype, n, dev):
    """Pointer of an optional contiguous tensor of n elements of that dtype on device dev."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != dev:
        raise XmodError(fn, ERR_INVALID_ARG)
    return t.data_ptr()


def _mat(fn, t, dtype, rows, width, dev, most=2 ** 31 - 1):
    """(pointer, row stride) of a [rows, width] tensor with contiguous rows on device dev;
    strides up to `most`."""
    if (t.dtype is not dtype or t.get_device() != dev or t.shape != (rows, width)
            or (width > 1 and t.stride(1) != 1)):
        raise XmodError(fn, ERR_INVALID_ARG)
    ld = t.stride(0) if rows > 1 else width
    if ld > most:
        raise XmodError(fn, ERR_UNSUPPORTED)
    return t.data_ptr(), ld


def _cols(fn, t, dtype, rows, width, dev):
    """(pointer, row stride) of the first `width` columns of a matrix with `rows` rows."""
    if (t.dtype is not dtype or t.get_device() != dev or t.dim() != 2 or t.shape[0] != rows
            or t.shape[1] < width or t.stride(1) != 1):
        raise XmodError(fn, ERR_INVALID_ARG)
    ld = t.stride(0) if rows > 1 else width
    if ld > 2 ** 31 - 1:
        raise XmodError(fn, ERR_UNSUPPORTED)
    return t.data_ptr(), ld


def _check_gains(fn, w, dtype, n, dev):
    """The QK-norm gains that a LayerWeights was made of are read as n elements of that dtype
    on end, on device dev."""
    for g in getattr(w, "_gains", ()):
        if g != (dtype, n, True, dev):
            raise XmodError(fn, ERR_INVALID_ARG)


def _elem(fn, dm, cache, dev):
    """torch dtype of the dims' elements; the cache has to be of these dims and there."""
    el = _torch_module.bfloat16 if dm.dtype == BF16 else _torch_module.float32
    if (cache.n_kv_heads != dm.n_kv_heads or cache.head_dim != dm.head_dim or cache.device != dev
            or (cache.format == CACHE_NATIVE and cache.dtype is not el)):
        raise XmodError(fn, ERR_INVALID_ARG)
    return el


def cache_append(dm, cache: KVCache, qkv, w, seq, slot, pos=None, q_out=None, status=None,
                 stream=None):
    """xmod_cache_append: the rows of qkv [M, (n_heads + 2 n_kv_heads) head_dim] into the
    cache, their transformed q into q_out (None: not wanted). w: a LayerWeights (its QK-norm
    gains and rope_theta count) or None. status: as for gather."""
    fn = "xmod_cache_append"
    M, dev = qkv.shape[0], _device(fn, qkv)
    el, i32 = _elem(fn, dm, cache, dev), _torch_module.int32
    qw = dm.n_heads * dm.head_dim
    qkv_p, ld = _mat(fn, qkv, el, M, qw + 2 * dm.n_kv_heads * dm.head_dim, dev)
    q_p, ldq = _mat(fn, q_out, el, M, qw, dev) if q_out is not None else (None, 0)
    _check_gains(fn, w, el, dm.head_dim, dev)
    st = load().xmod_cache_append(
        dm, cache, M, qkv_p, ld, w, _vec(fn, seq, i32, M, dev), _vec(fn, slot, i32, M, dev),
        _vec(fn, pos, i32, M, dev), q_p, ldq, _vec(fn, status, i32, 1, dev),
        _raw_stream(stream, dev))
    if st:
        raise XmodError(fn, st)


def cache_attention_workspace_bytes(dm: Dims, M: int) -> int:
    return int(load().xmod_cache_attention_workspace_bytes(ctypes.byref(dm), int(M)))


def cache_attention(dm, cache: KVCache, q, seq, lens, o, ws, lse=None, stream=None):
    """xmod_cache_attention: o [M, n_heads head_dim] (and lse [M, n_heads] fp32) of the
    queries q over the first lens[m] slots of sequence seq[m] (None: m)."""
    fn = "xmod_cache_attention"
    M, dev = q.shape[0], _device(fn, q)
    el, i32 = _elem(fn, dm, cache, dev), _torch_module.int32
    qw = dm.n_heads * dm.head_dim
    q_p, ldq = _mat(fn, q, el, M, qw, dev)
    st = load().xmod_cache_attention(
        dm, cache, M, q_p, ldq, _vec(fn, seq, i32, M, dev), _vec(fn, lens, i32, M, dev),
        _vec(fn, o, el, M * qw, dev), _vec(fn, lse, _torch_module.float32, M * dm.n_heads, dev),
        _vec(fn, ws, ws.dtype, ws.numel(), dev), ws.numel() * ws.element_size(),
        _raw_stream(stream, dev))
    if st:
        raise XmodError(fn, st)


def cache_attention_chunk_workspace_bytes(dm: Dims, n_chunks: int, M: int) -> int:
    return int(load().xmod_cache_attention_chunk_workspace_bytes(ctypes.byref(dm), int(n_chunks),
                                                                 int(M)))


def cache_attention_chunk(dm, cache: KVCache, q, start, seq, lens, o, ws, lse=None, stream=None):
    """xmod_cache_attention_chunk: o [M, n_heads head_dim] (and lse [M, n_heads] fp32) of the
    queries q, whose rows start[c] .. start[c + 1] - 1 are the last tokens of the first lens[c]
    slots of sequence seq[c] (None: c)."""
    fn = "xmod_cache_attention_chunk"
    M, n, dev = q.shape[0], lens.numel(), _device(fn, q)
    el, i32 = _elem(fn, dm, cache, dev), _torch_module.int32
    qw = dm.n_heads * dm.head_dim
    q_p, ldq = _mat(fn, q, el, M, qw, dev)
    st = load().xmod_cache_attention_chunk(
        dm, cache, n, M, q_p, ldq, _vec(fn, start, i32, n + 1, dev), _vec(fn, seq, i32, n, dev),
        _vec(fn, lens, i32, n, dev), _vec(fn, o, el, M * qw, dev),
        _vec(fn, lse, _torch_module.float32, M * dm.n_heads, dev),
        _vec(fn, ws, ws.dtype, ws.numel(), dev), ws.numel() * ws.element_size(),
        _raw_stream(stream, dev))
    if st:
        raise XmodError(fn, st)


def rope(head_dim, theta=10000.0, rot_dim=None, interleaved=False, scaling=ROPE_PLAIN, factor=1.0,
         trained=0) -> Rope:
    """xmod_rope_init: rotary positions that turn the first rot_dim (None: all) of head_dim
    dimensions. The structure's freq and amplitude may be changed afterwards."""
    r = Rope()
    rot = head_dim if rot_dim is None else rot_dim
    if not 0 < rot <= head_dim:
        raise XmodError("xmod_rope_init", ERR_INVALID_ARG)
    _check("xmod_rope_init", load().xmod_rope_init(
        ctypes.byref(r), int(rot), 1 if interleaved else 0, float(theta), int(scaling),
        float(factor), int(trained)))
    return r


def qk_rope(dm, qkv, w, rope: Rope, out, pos=None, stream=None):
    """xmod_qk_rope: the q and k heads of qkv [M, >= (n_heads + n_kv_heads) head_dim], normed (w: a
    LayerWeights, whose QK-norm gains count, or None) and turned at pos [M] (None: m mod T),
    into out [M, (n_heads + n_kv_heads) head_dim] (qkv itself, or its first columns: in place)."""
    fn = "xmod_qk_rope"
    M, dev = qkv.shape[0], _device(fn, qkv)
    el = _torch_module.bfloat16 if dm.dtype == BF16 else _torch_module.float32
    width = (dm.n_heads + dm.n_kv_heads) * dm.head_dim
    x, ldx = _cols(fn, qkv, el, M, width, dev)
    y, ldy = _cols(fn, out, el, M, width, dev)
    _check_gains(fn, w, el, dm.head_dim, dev)
    st = load().xmod_qk_rope(dm, M, x, ldx, w, rope, _vec(fn, pos, _torch_module.int32, M, dev), y,
                             ldy, _raw_stream(stream, dev))
    if st:
        raise XmodError(fn, st)


def qk_rope_bwd_workspace_bytes(dm: Dims, M: int) -> int:
    return int(load().xmod_qk_rope_bwd_workspace_bytes(ctypes.byref(dm), int(M)))


def qk_rope_bwd(dm, qkv, w, rope: Rope, dout, din, pos=None, dq_norm=None, dk_norm=None, ws=None,
                stream=None):
    """xmod_qk_rope_bwd: din of the gradient dout (both [M, (n_heads + n_kv_heads) head_dim]; may
    be one tensor) and, with gains, dq_norm and dk_norm [head_dim] fp32; qkv and ws may be None
    without gains."""
    fn = "xmod_qk_rope_bwd"
    M, dev = dout.shape[0], _device(fn, dout)
    el = _torch_module.bfloat16 if dm.dtype == BF16 else _torch_module.float32
    width, f32 = (dm.n_heads + dm.n_kv_heads) * dm.head_dim, _torch_module.float32
    x, ldx = _cols(fn, qkv, el, M, width, dev) if qkv is not None else (None, 0)
    d, ldd = _cols(fn, dout, el, M, width, dev)
    y, ldy = _cols(fn, din, el, M, width, dev)
    _check_gains(fn, w, el, dm.head_dim, dev)
    st = load().xmod_qk_rope_bwd(
        dm, M, x, ldx, w, rope, _vec(fn, pos, _torch_module.int32, M, dev), d, ldd, y, ldy,
        _vec(fn, dq_norm, f32, dm.head_dim, dev), _vec(fn, dk_norm, f32, dm.head_dim, dev),
        _vec(fn, ws, ws.dtype, ws.numel(), dev) if ws is not None else None, _wsb(ws),
        _raw_stream(stream, dev))
    if st:
        raise XmodError(fn, st)


def _logits(fn, t):
    """(dtype code, rows, width, pointer, row stride, device) of logits."""
    T = _torch()
    dt = BF16 if t.dtype is T.bfloat16 else FP32 if t.dtype is T.float32 else None
    if dt is None or t.dim() != 2:
        raise XmodError(fn, ERR_INVALID_ARG)
    N, V = t.shape
    if V > MAX_VOCAB:
        raise XmodError(fn, ERR_UNSUPPORTED)
    dev = _device(fn, t)
    return (dt, N, V) + _mat(fn, t, t.dtype, N, V, dev, 2 ** 62) + (dev,)


def token_logprobs(logits, target=None, logp=None, entropy=None, lse=None, top_idx=None,
                   top_logp=None, status=None, stream=None):
    """xmod_token_logprobs: logits [N, V] bf16 or fp32 (rows may be strided); the outputs
    that are given are written (logp, entropy, lse [N] fp32, top_idx int32 and top_logp
    fp32 [N, k])."""
    fn = "xmod_token_logprobs"
    dt, N, V, x, ld, dev = _logits(fn, logits)
    i32, f32 = _torch_module.int32, _torch_module.float32
    k = top_idx.shape[1] if top_idx is not None else 0
    st = load().xmod_token_logprobs(
        dt, N, V, x, ld, _vec(fn, target, i32, N, dev), _vec(fn, logp, f32, N, dev),
        _vec(fn, entropy, f32, N, dev), _vec(fn, lse, f32, N, dev), k,
        _vec(fn, top_idx, i32, N * k, dev), _vec(fn, top_logp, f32, N * k, dev),
        _vec(fn, status, i32, 1, dev), _raw_stream(stream, dev))
    if st:
        raise XmodError(fn, st)


def token_logprobs_bwd(logits, target, lse, g_logp, dlogits, entropy=None, g_entropy=None,
                       status=None, stream=None):
    """xmod_token_logprobs_bwd: dlogits [N, V] of the gradients g_logp and g_entropy [N]
    (either may be None); dlogits may be logits itself."""
    fn = "xmod_token_logprobs_bwd"
    dt, N, V, x, ld, dev = _logits(fn, logits)
    i32, f32 = _torch_module.int32, _torch_module.float32
    d, ldd = _mat(fn, dlogits, logits.dtype, N, V, dev, 2 ** 62)
    st = load().xmod_token_logprobs_bwd(
        dt, N, V, x, ld, _vec(fn, target, i32, N, dev), _vec(fn, lse, f32, N, dev),
        _vec(fn, entropy, f32, N, dev), _vec(fn, g_logp, f32, N, dev),
        _vec(fn, g_entropy, f32, N, dev), d, ldd, _vec(fn, status, i32, 1, dev),
        _raw_stream(stream, dev))
    if st:
        raise XmodError(fn, st)


def sample_tokens(logits, u, token, temperature=None, top_k=None, top_p=None, min_p=None,
                  logp=None, status=None, stream=None):
    """xmod_sample_tokens: a token of each row of logits [N, V] (bf16 or fp32; rows may be
    strided) for u [N] fp32 in [0, 1); temperature, top_p, min_p [N] fp32 and top_k [N] int32
    may each be None (1; off). token [N] int32 and logp [N] fp32 (None: not wanted) are
    written."""
    fn = "xmod_sample_tokens"
    dt, N, V, x, ld, dev = _logits(fn, logits)
    i32, f32 = _torch_module.int32, _torch_module.float32
    st = load().xmod_sample_tokens(
        dt, N, V, x, ld, _vec(fn, temperature, f32, N, dev), _vec(fn, top_k, i32, N, dev),
        _vec(fn, top_p, f32, N, dev), _vec(fn, min_p, f32, N, dev), _vec(fn, u, f32, N, dev),
        _vec(fn, token, i32, N, dev), _vec(fn, logp, f32, N, dev), _vec(fn, status, i32, 1, dev),
        _raw_stream(stream, dev))
    if st:
        raise XmodError(fn, st)


def selftest_wait_timeout(ws, stream=None):
    """xmod_selftest_wait_timeout: one CTA runs the kernels' bounded wait on a barrier
    that nothing completes until it gives up (about 2 s); the status word of ws then holds
    ERR_TIMEOUT."""
    _check("xmod_selftest_wait_timeout",
           load().xmod_selftest_wait_timeout(_p(ws), _wsb(ws), _stream(stream)))
