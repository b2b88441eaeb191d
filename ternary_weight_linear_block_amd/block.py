"""The operators of the block around the ternary linear layer: Python binding of
their entry points in include/twl.h (argument checks and marshalling only).

Tensors must be contiguous CUDA (HIP) tensors on the current device; bf16
arguments may also be given as their int16 bit patterns.  Outputs and workspaces
that a call allocates belong to the stream the call runs on.
"""
from __future__ import annotations

import contextlib

from . import _lib


def _torch():
    import torch
    return torch


def _check(t, name, shape, dtypes):
    """The device pointer of a tensor argument of this shape."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _matrix(t, name):
    """The sizes of a two-dimensional tensor argument."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected two dimensions")
    return t.shape


def _on(stream):
    """Context in which allocations belong to the stream of the call, and its handle."""
    torch = _torch()
    if stream is None:
        return contextlib.nullcontext(), torch.cuda.current_stream().cuda_stream
    if stream.device.index != torch.cuda.current_device():
        raise ValueError(f"stream is on {stream.device}, the current device is cuda:{torch.cuda.current_device()}")
    return torch.cuda.stream(stream), stream.cuda_stream


def norm_rotate_quant_act(x, weight, sign, eps=1e-6, residual=None, post_weight=None, gate=None,
                          branch_scale=1.0, return_normed=False, x_i8=None, a_scale=None, h=None,
                          normed=None, stream=None):
    """The step between two blocks (twl_norm_rotate_quant_act): RMSNorm of the
    block's output x with post_weight, times gate ([K] or [M, K]) and
    branch_scale, plus residual -> h; RMSNorm of h with weight -> normed;
    rotate_quant_act(normed, sign).

    x and residual [M, K] bf16, weights [K] bf16, sign [K] int8 (None: no
    rotation).  Returns (x_i8, a_scale, h, normed): h is None when nothing
    changes x (no residual, post_weight, gate or branch_scale), normed unless
    return_normed, x_i8 and a_scale without sign.  Buffers given for the outputs
    are written and returned; h may be x or residual itself.  return_normed, or
    normed=, is required without sign."""
    torch = _torch()
    lib = _lib.load()
    M, K = _matrix(x, "x")
    bf16 = (torch.bfloat16, torch.int16)
    branch = residual is not None or post_weight is not None or gate is not None or branch_scale != 1.0
    ctx, handle = _on(stream)
    gate_stride = 0
    p = {"x": _check(x, "x", (M, K), bf16), "weight": _check(weight, "weight", (K,), bf16)}
    for name, t, shape, dtypes in (("residual", residual, (M, K), bf16), ("post_weight", post_weight, (K,), bf16),
                                   ("sign", sign, (K,), (torch.int8,))):
        p[name] = None if t is None else _check(t, name, shape, dtypes)
    p["gate"] = None
    if gate is not None:
        wide = isinstance(gate, torch.Tensor) and gate.dim() == 2
        p["gate"] = _check(gate, "gate", (M, K) if wide else (K,), bf16)
        gate_stride = K if wide else 0
    if sign is None and (x_i8 is not None or a_scale is not None):
        raise ValueError("x_i8 and a_scale need sign")
    if h is not None and not branch:
        raise ValueError("h is given, but no residual, post_weight, gate or branch_scale: it would be x")
    with ctx:
        if sign is not None and x_i8 is None:
            x_i8 = torch.empty((M, K), dtype=torch.int8, device=x.device)
        if sign is not None and a_scale is None:
            a_scale = torch.empty((M,), dtype=torch.float32, device=x.device)
        if branch and h is None:
            h = torch.empty((M, K), dtype=x.dtype, device=x.device)
        if return_normed and normed is None:
            normed = torch.empty((M, K), dtype=x.dtype, device=x.device)
    for name, t, shape, dtypes in (("h", h, (M, K), bf16), ("normed", normed, (M, K), bf16),
                                   ("x_i8", x_i8, (M, K), (torch.int8,)), ("a_scale", a_scale, (M,), (torch.float32,))):
        p[name] = None if t is None else _check(t, name, shape, dtypes)
    st = lib.twl_norm_rotate_quant_act(
        p["x"], p["residual"], p["post_weight"], p["gate"], gate_stride, branch_scale, p["weight"], eps,
        p["sign"], M, K, p["h"], p["normed"], p["x_i8"], p["a_scale"], handle)
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
    torch = _torch()
    lib = _lib.load()
    M, N = _matrix(y, "y")
    K = _matrix(x, "x")[1]
    if not isinstance(lora_a, torch.Tensor) or lora_a.dim() != 3:
        raise ValueError("lora_a must be a tensor [n, R, K]")
    n, R = lora_a.shape[:2]
    bf16 = (torch.bfloat16, torch.int16)
    kinds = {torch.float32: _lib.OUT_F32, torch.bfloat16: _lib.OUT_BF16}
    if y.dtype not in kinds:
        raise TypeError(f"y has dtype {y.dtype}, expected float32 or bfloat16")
    ctx, handle = _on(stream)
    p_y = _check(y, "y", (M, N), (y.dtype,))
    p_x = _check(x, "x", (M, K), bf16)
    p_ids = _check(ids, "ids", (M,), (torch.int32,))
    p_a = _check(lora_a, "lora_a", (n, R, K), bf16)
    p_b = _check(lora_b, "lora_b", (n, N, R), bf16)
    p_scale = _check(scale, "scale", (n,), (torch.float32,))
    need = lora_workspace_bytes(M, K, R, n)
    with ctx:
        if out is None:
            out = torch.empty((M, N), dtype=y.dtype, device=y.device)
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=y.device)
    p_out = _check(out, "out", (M, N), (y.dtype,))
    ws, ws_len = None, 0
    if workspace is not None:
        ws, ws_len = _check(workspace, "workspace", (workspace.numel(),), (torch.uint8,)), workspace.numel()
    st = lib.twl_lora_add(p_y, p_x, p_ids, p_a, p_b, p_scale, M, N, K, R, n, kinds[y.dtype], p_out, ws, ws_len, handle)
    _lib.check(st, "twl_lora_add")
    return out


def pack_ternary_gated(code_gate, s_gate, code_up, s_up, bad_codes=None, stream=None):
    """Gate and up codes [N, K] int8 and scales [N, K/128] fp16 -> (packed, q
    [2 N, K/128], smax [2 N]) of ternary_gated_linear (twl_pack_ternary_gated)."""
    torch = _torch()
    lib = _lib.load()
    N, K = _matrix(code_gate, "code_gate")
    fp16 = (torch.float16, torch.int16)
    ctx, handle = _on(stream)
    G = K // _lib.GROUP
    ptrs = [_check(code_gate, "code_gate", (N, K), (torch.int8,)), _check(s_gate, "s_gate", (N, G), fp16),
            _check(code_up, "code_up", (N, K), (torch.int8,)), _check(s_up, "s_up", (N, G), fp16)]
    bad = None if bad_codes is None else _check(bad_codes, "bad_codes", bad_codes.shape, (torch.int32,))
    if bad_codes is not None and bad_codes.numel() < 1:
        raise ValueError("bad_codes is empty")
    with ctx:
        packed = torch.empty((int(lib.twl_packed_bytes(2 * N, K)),), dtype=torch.uint8, device=code_gate.device)
        q = torch.empty((2 * N, G), dtype=torch.int8, device=code_gate.device)
        smax = torch.empty((2 * N,), dtype=torch.float32, device=code_gate.device)
    st = lib.twl_pack_ternary_gated(*ptrs, N, K, packed.data_ptr(), q.data_ptr(), smax.data_ptr(), bad, handle)
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
    torch = _torch()
    lib = _lib.load()
    M, K = _matrix(x_i8, "x_i8")
    N2, G = _matrix(q, "q")
    if N2 % 2:
        raise ValueError(f"q has {N2} rows, expected 2 N of pack_ternary_gated")
    N = N2 // 2
    kinds = {torch.float32: _lib.OUT_F32, torch.bfloat16: _lib.OUT_BF16}
    dtype = out_dtype if out_dtype is not None else out.dtype if out is not None else torch.bfloat16
    if dtype not in kinds:
        raise TypeError(f"out_dtype is {dtype}, expected float32 or bfloat16")
    ctx, handle = _on(stream)
    p_x = _check(x_i8, "x_i8", (M, K), (torch.int8,))
    p_a = _check(a_scale, "a_scale", (M,), (torch.float32,))
    p_w = _check(packed, "packed", (int(lib.twl_packed_bytes(N2, K)),), (torch.uint8,))
    p_q = _check(q, "q", (N2, K // _lib.GROUP), (torch.int8,))
    p_s = _check(smax, "smax", (N2,), (torch.float32,))
    need = gated_workspace_bytes(M, N, K)
    with ctx:
        if out is None:
            out = torch.empty((M, N), dtype=dtype, device=x_i8.device)
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x_i8.device)
    p_out = _check(out, "out", (M, N), (dtype,))
    ws, ws_len = None, 0
    if workspace is not None:
        ws, ws_len = _check(workspace, "workspace", (workspace.numel(),), (torch.uint8,)), workspace.numel()
    st = lib.twl_ternary_gated_linear(p_x, p_a, p_w, p_q, p_s, M, N, K, p_out, kinds[dtype], path, ws, ws_len, handle)
    _lib.check(st, "twl_ternary_gated_linear")
    return out
