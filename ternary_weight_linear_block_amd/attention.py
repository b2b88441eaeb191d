"""The attention half of the block around the ternary linear layer: Python binding of
its entry points in include/twl.h (argument checks and marshalling only).

The rules of block.py hold here too: contiguous CUDA (HIP) tensors on the current
device (but for the rows of qk_norm_rope's qkv), outputs and workspaces that a call
allocates belong to the stream the call runs on, tensors that require grad are refused
unless gradients are off.
"""
from __future__ import annotations

import functools

from . import _lib
from .block import _check, _check_rows, _empty, _env, _handle, _matrix, _workspace

def _need(name):
    """A workspace query, cached by device and sizes."""
    @functools.lru_cache(4096)
    def need(device, *sizes):
        return getattr(_env().lib, name)(*sizes)
    return need


_int8_need = _need("twl_int8_workspace_bytes")
_attention_need = _need("twl_attention_workspace_bytes")


def int8_workspace_bytes(M, N, K):
    """Bytes of workspace int8_linear needs for these sizes on the current device."""
    return int(_lib.load().twl_int8_workspace_bytes(M, N, K))


def int8_linear(x_i8, a_scale, w_i8, w_scale, bias=None, out_dtype=None, out=None, workspace=None, stream=None):
    """The product of int8 activations [M, K] with a weight [N, K] held in 8 bits, times
    a_scale [M] and w_scale [N] (fp32), plus bias [N] (fp32) (twl_int8_linear).  The
    activations are those of rotate_quant_act or norm_rotate_quant_act; rotate_quant_act
    of the weight's rows, with the same sign table, makes (w_i8, w_scale).

    Returns out [M, N], float32 unless out_dtype (or the given out) is bfloat16, or int32
    for the exact sums alone (a_scale and w_scale may then be None).  The workspace
    (uint8, int8_workspace_bytes) is allocated for each call that needs one unless
    given; in a graph capture it then belongs to that graph."""
    env = _env()
    device = env.device()
    M, K = _matrix(x_i8, "x_i8")
    N = _matrix(w_i8, "w_i8")[0]
    if out_dtype is None:
        out_dtype = env.torch.float32 if out is None else out.dtype
    kind = _lib.OUT_ACC_I32 if out_dtype == env.int32[0] else env.kinds.get(out_dtype)
    if kind is None:
        raise TypeError(f"out_dtype is {out_dtype}, expected float32, bfloat16 or int32")
    handle = _handle(stream, env, device)
    p_x = _check(x_i8, "x_i8", (M, K), env.int8, device)
    p_w = _check(w_i8, "w_i8", (N, K), env.int8, device)
    p_a = p_s = p_bias = None
    if kind != _lib.OUT_ACC_I32 or a_scale is not None:
        p_a = _check(a_scale, "a_scale", (M,), env.fp32, device)
    if kind != _lib.OUT_ACC_I32 or w_scale is not None:
        p_s = _check(w_scale, "w_scale", (N,), env.fp32, device)
    if bias is not None:
        p_bias = _check(bias, "bias", (N,), env.fp32, device)
    if out is None:
        out = _empty(env, x_i8, (M, N), out_dtype, stream)
        p_out = out.data_ptr()
    else:
        p_out = _check(out, "out", (M, N), (out_dtype,), device)
    ws, ws_len, _held = _workspace(env, x_i8, _int8_need(device, M, N, K), workspace, stream, device)
    st = env.lib.twl_int8_linear(p_x, p_a, p_w, p_s, p_bias, M, N, K, p_out, kind, ws, ws_len, handle)
    if st:
        _lib.check(st, "twl_int8_linear")
    return out


def _cache(t, name, device, env):
    """Sizes and pointer of a cache argument [n_pages, n_kv, page, D]."""
    if len(getattr(t, "shape", ())) != 4:
        raise ValueError(f"{name} must be a tensor [n_pages, n_kv, page, D]")
    return t.shape, _check(t, name, t.shape, env.bf16, device)


def qk_norm_rope(qkv, positions, cos_sin, n_q, n_kv, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                 slots=None, k_cache=None, v_cache=None, q=None, stream=None):
    """RMSNorm of every query and key head, position rotation, keys and values into the
    pages of a cache (twl_qk_norm_rope).

    qkv [M, (n_q + 2 n_kv) D] fp32 or bf16, a projection's output (its rows may lie a
    multiple of 8 elements apart: a slice of a wider tensor); positions [M] int32 and
    cos_sin [n_pos, rot] fp32 (cosines, then sines; both None: no rotation); weights [D]
    bf16 (None: no norm); k_cache and v_cache [n_pages, n_kv, page, D] bf16 with slots [M]
    int32.  Without caches, keys and values come back as tensors [M, n_kv, D].  A token
    whose position is outside the table is padding, nothing is written for it; one whose
    slot is outside the cache gets its queries only.  Returns (q [M, n_q, D], k_cache,
    v_cache) or (q, k, v)."""
    env = _env()
    device = env.device()
    M, width = _matrix(qkv, "qkv")
    heads = n_q + 2 * n_kv
    if n_q < 1 or n_kv < 1 or width % heads:
        raise ValueError(f"qkv has {width} columns, expected (n_q + 2 n_kv) D with n_q = {n_q}, n_kv = {n_kv}")
    D = width // heads
    kind = env.kinds.get(qkv.dtype)
    if kind is None:
        raise TypeError(f"qkv has dtype {qkv.dtype}, expected float32 or bfloat16")
    handle = _handle(stream, env, device)
    p_qkv, stride = _check_rows(qkv, "qkv", (M, width), (qkv.dtype,), device)
    p_qw = p_kw = p_cs = p_pos = p_slots = None
    n_pos = rot = 0
    if q_weight is not None:
        p_qw = _check(q_weight, "q_weight", (D,), env.bf16, device)
    if k_weight is not None:
        p_kw = _check(k_weight, "k_weight", (D,), env.bf16, device)
    if cos_sin is not None:
        n_pos, rot = _matrix(cos_sin, "cos_sin")
        p_cs = _check(cos_sin, "cos_sin", (n_pos, rot), env.fp32, device)
        p_pos = _check(positions, "positions", (M,), env.int32, device)
    elif positions is not None:
        raise ValueError("positions are given, but no cos_sin")
    if (k_cache is None) != (v_cache is None):
        raise ValueError("k_cache and v_cache must be given together")
    if k_cache is None:
        if slots is not None:
            raise ValueError("slots are given, but no caches")
        n_pages, page = M, 1
        k_cache = _empty(env, qkv, (M, n_kv, D), env.bf16[0], stream)
        v_cache = _empty(env, qkv, (M, n_kv, D), env.bf16[0], stream)
        p_k, p_v = k_cache.data_ptr(), v_cache.data_ptr()
    else:
        shape, p_k = _cache(k_cache, "k_cache", device, env)
        n_pages, page = shape[0], shape[2]
        if shape[1] != n_kv or shape[3] != D:
            raise ValueError(f"k_cache has shape {tuple(shape)}, expected [n_pages, {n_kv}, page, {D}]")
        p_v = _check(v_cache, "v_cache", shape, env.bf16, device)
        p_slots = _check(slots, "slots", (M,), env.int32, device)
    if q is None:
        q = _empty(env, qkv, (M, n_q, D), env.bf16[0], stream)
        p_q = q.data_ptr()
    else:
        p_q = _check(q, "q", (M, n_q, D), env.bf16, device)
    st = env.lib.twl_qk_norm_rope(p_qkv, kind, stride, p_qw, p_kw, eps, p_cs, n_pos, rot, 1 if interleaved else 0, p_pos,
                                  p_slots, M, n_q, n_kv, D, p_q, p_k, p_v, n_pages, page, handle)
    if st:
        _lib.check(st, "twl_qk_norm_rope")
    return q, k_cache, v_cache


def attention_workspace_bytes(T, B, n_q, n_kv, D, page, table_pages, window=0, sinks=0):
    """Bytes of workspace window_attention needs for these sizes on the current device."""
    return int(_lib.load().twl_attention_workspace_bytes(T, B, n_q, n_kv, D, page, table_pages, window, sinks))


def window_attention(q, k_cache, v_cache, page_table, q_start, kv_len, scale=None, window=0, sinks=0, out=None,
                     workspace=None, stream=None):
    """Causal attention of new tokens over the pages of a cache, with a sliding window (0:
    none) and the first `sinks` tokens always visible (twl_window_attention).

    q [T, n_q, D] bf16, the new tokens of all sequences one after the other; k_cache and
    v_cache [n_pages, n_kv, page, D] bf16; page_table [B, pages] int32 (a page outside the
    cache is not seen); q_start [B + 1] int32, the first row of each sequence and the end
    of the last; kv_len [B] int32, each sequence's tokens in the cache, the new ones
    included; scale 1 / sqrt(D) unless given.  Returns out like q (rows behind the last
    sequence are left as they were).  Lengths stay on the device: a captured call serves
    others.  The workspace (uint8, attention_workspace_bytes) is allocated for each call
    that needs one unless given; in a graph capture it then belongs to that graph."""
    env = _env()
    device = env.device()
    if len(getattr(q, "shape", ())) != 3:
        raise ValueError("q must be a tensor [T, n_q, D]")
    T, n_q, D = q.shape
    handle = _handle(stream, env, device)
    p_q = _check(q, "q", (T, n_q, D), env.bf16, device)
    shape, p_k = _cache(k_cache, "k_cache", device, env)
    n_pages, n_kv, page, _ = shape
    if shape[3] != D:
        raise ValueError(f"k_cache has shape {tuple(shape)}, expected [n_pages, n_kv, page, {D}]")
    p_v = _check(v_cache, "v_cache", shape, env.bf16, device)
    B, table_pages = _matrix(page_table, "page_table")
    p_table = _check(page_table, "page_table", (B, table_pages), env.int32, device)
    p_start = _check(q_start, "q_start", (B + 1,), env.int32, device)
    p_len = _check(kv_len, "kv_len", (B,), env.int32, device)
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = _empty(env, q, None, q.dtype, stream)
        p_out = out.data_ptr()
    else:
        p_out = _check(out, "out", (T, n_q, D), env.bf16, device)
    need = _attention_need(device, T, B, n_q, n_kv, D, page, table_pages, window, sinks)
    ws, ws_len, _held = _workspace(env, q, need, workspace, stream, device)
    st = env.lib.twl_window_attention(p_q, p_k, p_v, p_table, p_start, p_len, scale, window, sinks, T, B, n_q, n_kv, D,
                                      n_pages, page, table_pages, p_out, ws, ws_len, handle)
    if st:
        _lib.check(st, "twl_window_attention")
    return out
