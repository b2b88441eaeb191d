"""CPU oracle of the attention half of a block: the definitions of include/twl.h in
float64 NumPy, written without the kernels' tiles, splits and layouts."""
import numpy as np


def int8_linear(x_i8, a_scale, w_i8, w_scale, bias=None):
    """-> (acc int64, y float64, |acc a w| float64)."""
    acc = (x_i8.astype(np.float64) @ w_i8.astype(np.float64).T).astype(np.int64)  # below 2^53: exact
    y = acc * (a_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)[None, :])
    mag = np.abs(y)
    return acc, (y if bias is None else y + bias.astype(np.float64)), mag


def heads_norm_rope(x, weight, eps, cos, sin, interleaved):
    """x [M, n, D], cos and sin [M, rot/2] -> (y, |a c| + |b s|), both [M, n, D]."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=2, keepdims=True) + eps) * weight.astype(np.float64)
    y, mag = x.copy(), np.abs(x)
    half = cos.shape[1]
    for i in range(half):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos[:, i, None].astype(np.float64), sin[:, i, None].astype(np.float64)
        a, b = x[:, :, lo], x[:, :, hi]
        y[:, :, lo], y[:, :, hi] = a * c - b * s, b * c + a * s
        mag[:, :, lo], mag[:, :, hi] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, mag


def sees(p, j, window, sinks):
    """Whether the query at position p sees key j."""
    return 0 <= j <= p and (window == 0 or p - j < window or j < sinks)


def mask(n, kv, window, sinks):
    """bool [n, kv] of a sequence's new tokens and keys."""
    p = (kv - n + np.arange(n))[:, None]
    j = np.arange(kv)[None, :]
    seen = j <= p
    if window > 0:
        seen &= (p - j < window) | (j < sinks)
    return seen


def attend(q, k, v, seen, scale):
    """One head: q [n, D], k and v [kv, D], seen bool [n, kv] -> (out, sum_j w |v| / sum_j w,
    largest sum_d |q k| scale of a row)."""
    s = q @ k.T * scale
    s = np.where(seen, s, -np.inf)
    top = np.max(s, axis=1, keepdims=True, initial=-np.inf)
    w = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    total = w.sum(axis=1, keepdims=True)
    w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    size = np.max(np.where(seen, np.abs(q) @ np.abs(k).T * abs(scale), 0.0), axis=1, keepdims=True, initial=0.0)
    return w @ v, w @ np.abs(v), size


def gather(cache, pages, kv):
    """A sequence's keys of every key head from a cache [n_pages, n_kv, page, D]: ([n_kv, kv, D],
    bool [kv]: the key's page is one)."""
    n_pages, n_kv, page, D = cache.shape
    j = np.arange(kv)
    entry = np.full(kv, -1)
    inside = j // page < len(pages)
    entry[inside] = np.asarray(pages)[j[inside] // page]
    good = (entry >= 0) & (entry < n_pages)
    out = np.zeros((n_kv, kv, D))
    if good.any():
        out[:, good] = cache[entry[good], :, j[good] % page].transpose(1, 0, 2)
    return out, good


def window_attention(q, k_cache, v_cache, page_table, q_start, kv_len, scale, window, sinks):
    """-> (out, weighted |v|, score sizes), all [T, n_q, ...]; NaN in rows without a sequence."""
    T, n_q, D = q.shape
    n_kv = k_cache.shape[1]
    out = np.full((T, n_q, D), np.nan)
    mag, size = np.zeros((T, n_q, D)), np.zeros((T, n_q, 1))
    for b in range(len(kv_len)):
        r0 = min(max(int(q_start[b]), 0), T)
        n, kv = min(max(int(q_start[b + 1]), r0), T) - r0, max(int(kv_len[b]), 0)
        k, good = gather(k_cache, page_table[b], kv)
        v, _ = gather(v_cache, page_table[b], kv)
        seen = mask(n, kv, window, sinks) & good[None, :]
        for h in range(n_q):
            g = h // (n_q // n_kv)
            rows = slice(r0, r0 + n)
            out[rows, h], mag[rows, h], size[rows, h] = attend(
                q[rows, h].astype(np.float64), np.where(good[:, None], k[g], 0.0), np.where(seen.any(0)[:, None], v[g], 0.0), seen, scale)
    return out, mag, size
