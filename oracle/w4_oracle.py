"""Products with 4-bit weights, fp64 on the CPU, by the definition: w[f, c] = scale[f, c // G] (q[f, c] - zero[f, c // G])
with q of column 2 i in the low four bits of byte i of row f; y = x W^T + bias, dx = dy W."""
import numpy as np


def _np(t):
    return t.detach().cpu() if hasattr(t, "detach") else t


def _f64(t):
    return np.asarray(_np(t).float().numpy() if hasattr(t, "detach") else t, dtype=np.float64)


def w4_values(data, scale, zero=None):
    """W [F, D]."""
    data, scale = np.asarray(_np(data)), _f64(scale)
    F, half = data.shape
    q = np.empty((F, 2 * half))
    q[:, 0::2], q[:, 1::2] = data & 15, data >> 4
    G = 2 * half // scale.shape[1]
    z = np.full(scale.shape, 8.0) if zero is None else _f64(zero)
    return np.repeat(scale, G, 1) * (q - np.repeat(z, G, 1))


def w4_linear_fwd(x, data, scale, zero=None, bias=None):
    return _f64(x) @ w4_values(data, scale, zero).T + (0 if bias is None else _f64(bias))


def w4_linear_bwd(dy, data, scale, zero=None):
    return _f64(dy) @ w4_values(data, scale, zero)


def _bf16(v):
    """fp64 rounded to fp32, then to the nearest bf16 (ties to even), as the fp32 division and its rounding give them."""
    bits = np.asarray(v, dtype=np.float32).view(np.uint32).astype(np.uint64)
    bits = (bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000
    return bits.astype(np.uint32).view(np.float32).astype(np.float64)


def w4_quantize(w, group, symmetric=True):
    """(q [F, D], scale [F, D / group], zero [F, D / group]) as whole numbers and fp64."""
    w = _f64(w)
    g = w.reshape(w.shape[0], -1, group)
    lo, hi = np.minimum(g.min(-1), 0), np.maximum(g.max(-1), 0)
    scale = _bf16(np.maximum(-lo, hi) / 7 if symmetric else (hi / 2 - lo / 2).astype(np.float32) / np.float32(7.5))
    safe = np.where(scale > 0, scale, 1)
    zero = np.full(scale.shape, 8.0) if symmetric else np.where(scale > 0, np.clip(np.rint(-lo / safe), 0, 15), 0)
    q = np.clip(np.rint(g / safe[..., None]) + zero[..., None], 0, 15)
    q = np.where(scale[..., None] > 0, q, zero[..., None])
    return q.reshape(w.shape), scale, zero
