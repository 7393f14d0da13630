"""The gated feed-forward, fp64 on the CPU: h = act(x Wg^T) * (x Wu^T) and its gradients, by the definition.

act "silu": g / (1 + exp(-g)); "gelu_tanh": g / 2 (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))).
"""
import numpy as np


def _f64(t):
    return np.asarray(t.detach().float().cpu().numpy() if hasattr(t, "detach") else t, dtype=np.float64)


def activation(g, act):
    """(act(g), act'(g))."""
    g = np.asarray(g, dtype=np.float64)
    if act == "silu":
        s = 0.5 * (1 + np.tanh(0.5 * g))   # the logistic function without overflow
        return g * s, s + g * s * (1 - s)
    assert act == "gelu_tanh"
    c = np.sqrt(2 / np.pi)
    t = np.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def ffn_gated_fwd(x, w_gate, w_up, act="silu"):
    x = _f64(x)
    return activation(x @ _f64(w_gate).T, act)[0] * (x @ _f64(w_up).T)


def ffn_gated_bwd(dh, x, w_gate, w_up, act="silu"):
    """(dx, dw_gate, dw_up) for 2-D x [M, D], dh [M, F]."""
    x, dh, wg, wu = _f64(x), _f64(dh), _f64(w_gate), _f64(w_up)
    a, slope = activation(x @ wg.T, act)
    dg, du = dh * (x @ wu.T) * slope, dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x
