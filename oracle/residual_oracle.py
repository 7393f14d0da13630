"""The gated residual with the norms around a block's branches, fp64 on the CPU, by the definition:

t = z or its RMS norm times w_post;  r = x + alpha gate[b] t;  y = norm(r) w_pre (1 + scale[b]) + shift[b]
(norm: "layer", without an affine of its own, or "rms"), and the gradients for dr (of r) and dy (of y).
Shapes: x, z, r, y, dr, dy [B, N, D]; gate, scale, shift [B, D]; w_post, w_pre [D]; None: 1, 0, 0, 1, 1.
"""
import numpy as np


def _f64(t, absent=None):
    if t is None:
        return absent
    return np.asarray(t.detach().float().cpu().numpy() if hasattr(t, "detach") else t, dtype=np.float64)


def _norm(v, kind, eps):
    """(xhat, rstd [..., 1])."""
    if kind == "layer":
        v = v - v.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return v * rstd, rstd


def _norm_bwd(g, xhat, rstd, kind):
    """The gradient at the norm's input for the gradient g at xhat."""
    g = g - xhat * (g * xhat).mean(-1, keepdims=True) - (g.mean(-1, keepdims=True) if kind == "layer" else 0)
    return rstd * g


def residual_norm_fwd(x, z, gate=None, w_post=None, scale=None, shift=None, w_pre=None, post="none", pre="layer", alpha=1.0,
                      eps=1e-6):
    """(r, y); y is None with pre "none"."""
    x, z = _f64(x), _f64(z)
    ones, zeros = np.ones((x.shape[0], x.shape[2])), np.zeros((x.shape[0], x.shape[2]))
    gate, scale, shift = _f64(gate, ones)[:, None], _f64(scale, zeros)[:, None], _f64(shift, zeros)[:, None]
    t = _norm(z, "rms", eps)[0] * _f64(w_post, 1.0) if post == "rms" else z
    r = x + alpha * gate * t
    if pre == "none":
        return r, None
    return r, _norm(r, pre, eps)[0] * _f64(w_pre, 1.0) * (1 + scale) + shift


def residual_norm_bwd(dr, dy, r, z, gate=None, w_post=None, scale=None, w_pre=None, post="none", pre="layer", alpha=1.0,
                      eps=1e-6):
    """(dx, dz, d_gate [B, D], dw_post [D], d_scale, d_shift [B, D], dw_pre [D]); the last three None with pre "none"."""
    z = _f64(z)
    B, _, D = z.shape
    gate, scale = _f64(gate, np.ones((B, D)))[:, None], _f64(scale, np.zeros((B, D)))[:, None]
    w_post, w_pre = _f64(w_post, np.ones(D)), _f64(w_pre, np.ones(D))
    g, d_scale, d_shift, dw_pre = _f64(dr, np.zeros_like(z)), None, None, None
    if pre != "none":
        dy = _f64(dy)
        xhat, rstd = _norm(_f64(r), pre, eps)
        d_scale, d_shift = (dy * xhat * w_pre).sum(1), dy.sum(1)
        dw_pre = (dy * xhat * (1 + scale)).sum((0, 1))
        g = g + _norm_bwd(dy * w_pre * (1 + scale), xhat, rstd, pre)
    u = alpha * gate * g
    if post == "rms":
        zhat, rz = _norm(z, "rms", eps)
        return (g, _norm_bwd(u * w_post, zhat, rz, "rms"), alpha * (g * zhat * w_post).sum(1), (u * zhat).sum((0, 1)), d_scale,
                d_shift, dw_pre)
    return g, u, alpha * (g * z).sum(1), None, d_scale, d_shift, dw_pre
