"""CPU oracle of the block operators around the ternary linear layer: the
definitions of include/twl.h in float64 NumPy, written without the kernels'
splits and layouts."""
import numpy as np

from .twl_oracle import bf16_to_f32, linear_acc, round_bf16, rotate_quant_act


def bf16_bits(v: np.ndarray) -> np.ndarray:
    """float64 -> bf16 bit patterns (through float32, nearest even)."""
    return round_bf16(np.asarray(v).astype(np.float32))


def _rms(t, w_bits, eps):
    return t / np.sqrt(np.mean(t * t, axis=1, keepdims=True) + eps) * bf16_to_f32(w_bits).astype(np.float64)


def norm_rotate_quant_act(x_bits, weight_bits, sign, eps, residual_bits=None, post_bits=None, gate_bits=None,
                          branch_scale=1.0):
    """-> (x_i8, a_scale, h bits, normed bits)."""
    b = bf16_to_f32(x_bits).astype(np.float64)
    if post_bits is not None:
        b = _rms(b, post_bits, eps)
    if gate_bits is not None:
        b = b * bf16_to_f32(gate_bits).astype(np.float64)
    b = b * branch_scale
    if residual_bits is not None:
        b = bf16_to_f32(residual_bits).astype(np.float64) + b
    h = bf16_bits(b)
    normed = bf16_bits(_rms(bf16_to_f32(h).astype(np.float64), weight_bits, eps))
    x_i8, a_scale = rotate_quant_act(normed, sign) if sign is not None else (None, None)
    return x_i8, a_scale, h, normed


def lora_add(y, x, ids, a, b, scale):
    """y + scale[id] (x A[id]^T) B[id]^T in float64 -> (out, bound parts): out
    [M, N], and for an error bound the magnitudes |B| (|x| |A|) and |B| |v|, both
    times |scale|, zero for tokens without an adapter."""
    y, x, a, b = (np.asarray(t, np.float64) for t in (y, x, a, b))
    out, mag_x, mag_v = y.copy(), np.zeros_like(y), np.zeros_like(y)
    for t, i in enumerate(ids):
        if 0 <= i < len(a):
            v = a[i] @ x[t]
            s = float(scale[i])
            out[t] += s * (b[i] @ v)
            mag_x[t] = abs(s) * (np.abs(b[i]) @ (np.abs(a[i]) @ np.abs(x[t])))
            mag_v[t] = abs(s) * (np.abs(b[i]) @ np.abs(v))
    return out, mag_x, mag_v


def gated_linear(x_i8, a_scale, code_gate, q_gate, smax_gate, code_up, q_up, smax_up):
    """SiLU(gate) * up of the two projections in float64 -> (out, |gate|, |up|)."""
    def project(code, q, smax):
        acc = linear_acc(x_i8, code, q).astype(np.float64)
        return acc * np.asarray(a_scale, np.float64)[:, None] * np.asarray(smax, np.float64)[None, :] / 127.0

    g, u = project(code_gate, q_gate, smax_gate), project(code_up, q_up, smax_up)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u, np.abs(g), np.abs(u)
