"""Rotary positions with several axes and the per-head norm of queries and keys, fp64 on the CPU.

The definition, written out per feature: axis a turns rot[a] features, its pair i by the angle
p * theta_a^(-2 i / rot[a]) at position p; pairs are numbered through the axes in order, pair j
being features (2 j, 2 j + 1) ("interleaved") or (j, j + R / 2) ("halves"); features from R on
pass.  The norm is x / sqrt(mean(x^2) + eps) * w over a head's features.
"""
import numpy as np


def _f64(t):
    return np.asarray(t.detach().float().cpu().numpy() if hasattr(t, "detach") else t, dtype=np.float64)


def rope_angles(pos, axes, theta=10000.0):
    """Angle of every pair of every token: [..., N, R / 2] for pos [..., N, 3]."""
    pos = np.asarray(pos, dtype=np.float64)
    th = [theta] * 3 if np.isscalar(theta) else list(theta)
    cols = [pos[..., a:a + 1] * float(th[a]) ** (-2.0 * np.arange(r // 2) / r) for a, r in enumerate(axes) if r]
    return np.concatenate(cols, -1) if cols else np.zeros(pos.shape[:-1] + (0,))


def pair_features(R, pairing):
    """(first feature, second feature) of each pair."""
    j = np.arange(R // 2)
    return (2 * j, 2 * j + 1) if pairing == "interleaved" else (j, j + R // 2)


def rope(x, angles, pairing="interleaved", backward=False):
    """x [B, H, N, d] turned by angles [N, R / 2] or [B, N, R / 2] (backward: by their negatives)."""
    y = _f64(x).copy()
    ang = -angles if backward else angles
    if ang.ndim == 3:
        ang = ang[:, None]
    c, s = np.cos(ang), np.sin(ang)
    f, g = pair_features(2 * angles.shape[-1], pairing)
    a, b = y[..., f].copy(), y[..., g].copy()
    y[..., f] = a * c - b * s
    y[..., g] = a * s + b * c
    return y


def qk_norm(x, w, eps):
    x = _f64(x)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return n if w is None else n * _f64(w)


def qk_norm_rope_fwd(x, w, angles, pairing="interleaved", eps=1e-6):
    return rope(qk_norm(x, w, eps), angles, pairing)


def qk_norm_rope_bwd(dy, x, w, angles, pairing="interleaved", eps=1e-6):
    """(dx, dw) for one of queries and keys."""
    x = _f64(x)
    g = rope(dy, angles, pairing, backward=True)
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xhat = x * rstd
    gw = g if w is None else g * _f64(w)
    dx = rstd * (gw - xhat * (gw * xhat).mean(-1, keepdims=True))
    return dx, (g * xhat).sum((0, 1, 2))
