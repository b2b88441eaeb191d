"""The operators of the block around the ternary linear layer: Python binding of
their entry points in include/twl.h (argument checks and marshalling only).

Tensors must be contiguous CUDA (HIP) tensors on the current device (but for
the rows of norm_rotate_quant_act's gate); bf16 arguments may also be given as
their int16 bit patterns.  Outputs and workspaces that a call allocates belong to
the stream the call runs on.  No operator has a backward pass: a tensor that
requires grad is refused unless gradients are off (torch.no_grad()).
"""
from __future__ import annotations

import functools

from . import _lib


class _Env:
    """What every call looks up: torch, the loaded library and the dtypes."""

    def __init__(self):
        import torch
        self.torch, self.lib = torch, _lib.load()
        self.bf16 = (torch.bfloat16, torch.int16)
        self.fp16 = (torch.float16, torch.int16)
        self.fp32, self.int32, self.int8, self.uint8 = (torch.float32,), (torch.int32,), (torch.int8,), (torch.uint8,)
        self.kinds = {torch.float32: _lib.OUT_F32, torch.bfloat16: _lib.OUT_BF16}
        self.device, self.empty_like = torch.cuda.current_device, torch.empty_like
        # workspace sizes by (device, sizes): the planners behind them cost 1 us a call
        self.lora_need = functools.lru_cache(4096)(lambda device, *sizes: self.lib.twl_lora_workspace_bytes(*sizes))
        self.gated_need = functools.lru_cache(4096)(lambda device, *sizes: self.lib.twl_gated_workspace_bytes(*sizes))
        # the stream handle alone: making a torch.cuda.Stream for it costs 2.4 us a call
        self.stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)


_ENV = None


def _env():
    global _ENV
    if _ENV is None:
        _ENV = _Env()
    return _ENV


def _check(t, name, shape, dtypes, device):
    """The device pointer of a tensor argument of this shape on this device."""
    try:
        if t.get_device() == device and t.dtype in dtypes and t.shape == shape and t.is_contiguous() and not t.requires_grad:
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if _env().torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad, which this operator does not compute: detach it or call under torch.no_grad()")
    return t.data_ptr()


def _check_rows(t, name, shape, dtypes, device):
    """As _check for a matrix whose rows may lie apart or, with stride 0, be one row
    for all: pointer and distance of the rows in elements."""
    if t.is_contiguous() or t.shape != shape or t.stride(1) != 1:
        return _check(t, name, shape, dtypes, device), shape[1]
    return _check(t[0], name, shape[1:], dtypes, device), t.stride(0)


def _matrix(t, name):
    """The sizes of a two-dimensional tensor argument."""
    try:
        m, n = t.shape
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    except ValueError:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected two dimensions") from None
    return m, n


def _handle(stream, env, device):
    """The handle of the stream a call runs on."""
    if stream is None:
        return env.stream(device)
    if stream.device.index != device:
        raise ValueError(f"stream is on {stream.device}, the current device is cuda:{device}")
    return stream.cuda_stream


def _empty(env, like, shape, dtype, stream):
    """A new tensor beside `like`, of its own shape unless given, that belongs to
    the stream of the call."""
    if stream is not None:
        with env.torch.cuda.stream(stream):
            return _empty(env, like, shape, dtype, None)
    return env.empty_like(like, dtype=dtype) if shape is None else like.new_empty(shape, dtype=dtype)


def _workspace(env, like, need, workspace, stream, device):
    """Pointer and size of the workspace of a call, and the tensor that holds it."""
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = _empty(env, like, (need,), env.torch.uint8, stream)
        return workspace.data_ptr(), need, workspace
    size = workspace.numel() if hasattr(workspace, "numel") else 0
    return _check(workspace, "workspace", (size,), env.uint8, device), size, workspace


def norm_rotate_quant_act(x, weight, sign, eps=1e-6, residual=None, post_weight=None, gate=None,
                          branch_scale=1.0, return_normed=False, x_i8=None, a_scale=None, h=None,
                          normed=None, stream=None):
    """The step between two blocks (twl_norm_rotate_quant_act): RMSNorm of the
    block's output x with post_weight, times gate ([K] or [M, K]) and
    branch_scale, plus residual -> h; RMSNorm of h with weight -> normed;
    rotate_quant_act(normed, sign).

    x and residual [M, K] bf16, weights [K] bf16, sign [K] int8 (None: no
    rotation).  The rows of a gate [M, K] may lie a multiple of 8 elements apart
    (a slice of a wider tensor) or be one row expanded.  Returns (x_i8, a_scale,
    h, normed): h is None when nothing changes x (no residual, post_weight, gate
    or branch_scale), normed unless return_normed, x_i8 and a_scale without sign.
    Buffers given for the outputs are written and returned; h may be x or residual
    itself.  return_normed, or normed=, is required without sign."""
    env = _env()
    device = env.device()
    M, K = _matrix(x, "x")
    wide, row, bf16 = (M, K), (K,), env.bf16
    handle = _handle(stream, env, device)
    p_x, p_weight = _check(x, "x", wide, bf16, device), _check(weight, "weight", row, bf16, device)
    p_residual = p_post = p_gate = p_sign = p_x_i8 = p_a_scale = p_h = p_normed = None
    gate_stride = 0
    if residual is not None:
        p_residual = _check(residual, "residual", wide, bf16, device)
    if post_weight is not None:
        p_post = _check(post_weight, "post_weight", row, bf16, device)
    if gate is not None:
        if len(getattr(gate, "shape", ())) == 2:
            p_gate, gate_stride = _check_rows(gate, "gate", wide, bf16, device)
        else:
            p_gate = _check(gate, "gate", row, bf16, device)
    if sign is not None:
        p_sign = _check(sign, "sign", row, env.int8, device)
        if x_i8 is None:
            x_i8 = _empty(env, x, None, env.int8[0], stream)
            p_x_i8 = x_i8.data_ptr()
        else:
            p_x_i8 = _check(x_i8, "x_i8", wide, env.int8, device)
        if a_scale is None:
            a_scale = _empty(env, x, (M,), env.fp32[0], stream)
            p_a_scale = a_scale.data_ptr()
        else:
            p_a_scale = _check(a_scale, "a_scale", (M,), env.fp32, device)
    elif x_i8 is not None or a_scale is not None:
        raise ValueError("x_i8 and a_scale need sign")
    if residual is not None or post_weight is not None or gate is not None or branch_scale != 1.0:
        if h is None:
            h = _empty(env, x, None, x.dtype, stream)
            p_h = h.data_ptr()
        else:
            p_h = _check(h, "h", wide, bf16, device)
    elif h is not None:
        raise ValueError("h is given, but no residual, post_weight, gate or branch_scale: it would be x")
    if normed is not None:
        p_normed = _check(normed, "normed", wide, bf16, device)
    elif return_normed:
        normed = _empty(env, x, None, x.dtype, stream)
        p_normed = normed.data_ptr()
    st = env.lib.twl_norm_rotate_quant_act(
        p_x, p_residual, p_post, p_gate, gate_stride, branch_scale, p_weight, eps, p_sign, M, K, p_h, p_normed,
        p_x_i8, p_a_scale, handle)
    if st:
        _lib.check(st, "twl_norm_rotate_quant_act")
    return x_i8, a_scale, h, normed


def lora_workspace_bytes(M, K, R, n_adapters):
    """Bytes of workspace lora_add needs for these sizes on the current device."""
    return int(_lib.load().twl_lora_workspace_bytes(M, K, R, n_adapters))


def lora_add(y, x, ids, lora_a, lora_b, scale, out=None, workspace=None, stream=None):
    """y + scale[id] * (x A[id]^T) B[id]^T for each token's adapter id
    (twl_lora_add): low-rank adapters of many requests beside a shared projection.

    y [M, N] fp32 or bf16, x [M, K] bf16 (the projection's input before the
    rotation), ids [M] int32 (outside 0 .. n-1: no adapter), lora_a [n, R, K] and
    lora_b [n, N, R] bf16, scale [n] fp32.  Returns out (a new tensor unless given;
    y itself for the update in place).  The workspace (uint8,
    lora_workspace_bytes) is allocated for each call unless given; in a graph
    capture it then belongs to that graph."""
    env = _env()
    device = env.device()
    M, N = _matrix(y, "y")
    K = _matrix(x, "x")[1]
    try:
        n, R, _ = lora_a.shape
    except (AttributeError, ValueError):
        raise ValueError("lora_a must be a tensor [n, R, K]") from None
    kind = env.kinds.get(y.dtype)
    if kind is None:
        raise TypeError(f"y has dtype {y.dtype}, expected float32 or bfloat16")
    handle = _handle(stream, env, device)
    like_y = (y.dtype,)
    p_y = _check(y, "y", (M, N), like_y, device)
    p_x = _check(x, "x", (M, K), env.bf16, device)
    p_ids = _check(ids, "ids", (M,), env.int32, device)
    p_a = _check(lora_a, "lora_a", (n, R, K), env.bf16, device)
    p_b = _check(lora_b, "lora_b", (n, N, R), env.bf16, device)
    p_scale = _check(scale, "scale", (n,), env.fp32, device)
    if out is None:
        out = _empty(env, y, None, y.dtype, stream)
        p_out = out.data_ptr()
    else:
        p_out = _check(out, "out", (M, N), like_y, device)
    ws, ws_len, _held = _workspace(env, y, env.lora_need(device, M, K, R, n), workspace, stream, device)
    st = env.lib.twl_lora_add(p_y, p_x, p_ids, p_a, p_b, p_scale, M, N, K, R, n, kind, p_out, ws, ws_len, handle)
    if st:
        _lib.check(st, "twl_lora_add")
    return out


def pack_ternary_gated(code_gate, s_gate, code_up, s_up, bad_codes=None, stream=None):
    """Gate and up codes [N, K] int8 and scales [N, K/128] fp16 -> (packed, q
    [2 N, K/128], smax [2 N]) of ternary_gated_linear (twl_pack_ternary_gated)."""
    env = _env()
    device = env.device()
    N, K = _matrix(code_gate, "code_gate")
    G = K // _lib.GROUP
    handle = _handle(stream, env, device)
    ptrs = [_check(code_gate, "code_gate", (N, K), env.int8, device), _check(s_gate, "s_gate", (N, G), env.fp16, device),
            _check(code_up, "code_up", (N, K), env.int8, device), _check(s_up, "s_up", (N, G), env.fp16, device)]
    bad = None
    if bad_codes is not None:
        bad = _check(bad_codes, "bad_codes", bad_codes.shape, env.int32, device)
        if bad_codes.numel() < 1:
            raise ValueError("bad_codes is empty")
    packed = _empty(env, code_gate, (int(env.lib.twl_packed_bytes(2 * N, K)),), env.torch.uint8, stream)
    q = _empty(env, code_gate, (2 * N, G), env.torch.int8, stream)
    smax = _empty(env, code_gate, (2 * N,), env.torch.float32, stream)
    st = env.lib.twl_pack_ternary_gated(*ptrs, N, K, packed.data_ptr(), q.data_ptr(), smax.data_ptr(), bad, handle)
    if st:
        _lib.check(st, "twl_pack_ternary_gated")
    return packed, q, smax


def gated_workspace_bytes(M, N, K):
    """Bytes of workspace ternary_gated_linear may need for these sizes on the current device."""
    return int(_lib.load().twl_gated_workspace_bytes(M, N, K))


def ternary_gated_linear(x_i8, a_scale, packed, q, smax, out_dtype=None, path=_lib.PATH_AUTO, out=None,
                         workspace=None, stream=None):
    """SiLU(gate) * up of the two ternary projections that pack_ternary_gated packed,
    for the int8 activations of rotate_quant_act or norm_rotate_quant_act
    (twl_ternary_gated_linear).

    Returns out [M, N], bf16 unless out_dtype (or the given out) is float32.  The
    workspace (uint8, gated_workspace_bytes) is allocated for each call that needs
    one unless given; in a graph capture it then belongs to that graph."""
    env = _env()
    device = env.device()
    M, K = _matrix(x_i8, "x_i8")
    N2 = _matrix(q, "q")[0]
    if N2 % 2:
        raise ValueError(f"q has {N2} rows, expected 2 N of pack_ternary_gated")
    N = N2 // 2
    if out_dtype is None:
        out_dtype = env.torch.bfloat16 if out is None else out.dtype
    kind = env.kinds.get(out_dtype)
    if kind is None:
        raise TypeError(f"out_dtype is {out_dtype}, expected float32 or bfloat16")
    handle = _handle(stream, env, device)
    lib = env.lib
    p_x = _check(x_i8, "x_i8", (M, K), env.int8, device)
    p_a = _check(a_scale, "a_scale", (M,), env.fp32, device)
    p_w = _check(packed, "packed", (lib.twl_packed_bytes(N2, K),), env.uint8, device)
    p_q = _check(q, "q", (N2, K // _lib.GROUP), env.int8, device)
    p_s = _check(smax, "smax", (N2,), env.fp32, device)
    if out is None:
        out = _empty(env, x_i8, (M, N), out_dtype, stream)
        p_out = out.data_ptr()
    else:
        p_out = _check(out, "out", (M, N), (out_dtype,), device)
    ws, ws_len, _held = _workspace(env, x_i8, env.gated_need(device, M, N, K), workspace, stream, device)
    st = lib.twl_ternary_gated_linear(p_x, p_a, p_w, p_q, p_s, M, N, K, p_out, kind, path, ws, ws_len, handle)
    if st:
        _lib.check(st, "twl_ternary_gated_linear")
    return out
