"""The gated residual's oracle against torch fp64 norms with autograd, central differences and the AdaLN oracle (CPU only)."""
import numpy as np
import pytest
import torch

import oracle

B, N, D = 2, 3, 7


def inputs(seed=0):
    rng = np.random.default_rng(seed)
    r = rng.standard_normal
    return dict(x=3 * r((B, N, D)), z=r((B, N, D)), gate=r((B, D)), w_post=1 + r(D), scale=r((B, D)), shift=r((B, D)), w_pre=1 + r(D))


def torch_forward(t, post, pre, alpha, eps):
    F = torch.nn.functional
    b = F.rms_norm(t["z"], (D,), t["w_post"], eps) if post == "rms" else t["z"]
    r = t["x"] + alpha * t["gate"][:, None] * b
    if pre == "none":
        return r, None
    n = F.layer_norm(r, (D,), t["w_pre"], eps=eps) if pre == "layer" else F.rms_norm(r, (D,), t["w_pre"], eps)
    return r, n * (1 + t["scale"][:, None]) + t["shift"][:, None]


@pytest.mark.parametrize("post", ["none", "rms"])
@pytest.mark.parametrize("pre", ["none", "layer", "rms"])
def test_forward_and_gradients(post, pre):
    alpha, eps = 0.7, 1e-3
    a = inputs()
    t = {n: torch.from_numpy(v).requires_grad_() for n, v in a.items()}
    r, y = torch_forward(t, post, pre, alpha, eps)
    got_r, got_y = oracle.residual_norm_fwd(**a, post=post, pre=pre, alpha=alpha, eps=eps)
    assert np.abs(got_r - r.detach().numpy()).max() < 1e-12
    rng = np.random.default_rng(1)
    dr, dy = rng.standard_normal((B, N, D)), rng.standard_normal((B, N, D))
    loss = (r * torch.from_numpy(dr)).sum()
    if y is not None:
        assert np.abs(got_y - y.detach().numpy()).max() < 1e-12
        loss = loss + (y * torch.from_numpy(dy)).sum()
    else:
        assert got_y is None
    loss.backward()
    names = ("x", "z", "gate", "w_post", "scale", "shift", "w_pre")
    grads = oracle.residual_norm_bwd(dr, dy if pre != "none" else None, got_r, a["z"], a["gate"], a["w_post"], a["scale"], a["w_pre"],
                                     post=post, pre=pre, alpha=alpha, eps=eps)

    def value(**changed):
        r, y = oracle.residual_norm_fwd(**{**a, **changed}, post=post, pre=pre, alpha=alpha, eps=eps)
        return float((r * dr).sum() + (0 if y is None else (y * dy).sum()))

    for n, g in zip(names, grads):
        if t[n].grad is None:
            assert g is None, n
            continue
        assert np.abs(g - t[n].grad.numpy()).max() < 1e-10, n
        e, step = rng.standard_normal(a[n].shape), 1e-6
        slope = (value(**{n: a[n] + step * e}) - value(**{n: a[n] - step * e})) / (2 * step)
        assert slope == pytest.approx(float((g * e).sum()), rel=1e-5, abs=1e-6), n


def test_without_a_branch_it_is_adaln():
    a = inputs(2)
    y = oracle.residual_norm_fwd(a["x"], 0 * a["z"], a["gate"], scale=a["scale"], shift=a["shift"])[1]
    assert np.abs(y - oracle.adaln_fwd(a["x"], a["scale"], a["shift"])).max() < 1e-13
    dy = a["z"]
    got = oracle.residual_norm_bwd(None, dy, a["x"], 0 * a["z"], a["gate"], scale=a["scale"])
    for g, want in zip((got[0], got[4], got[5]), oracle.adaln_bwd(a["x"], a["scale"], dy)):
        assert np.abs(g - want).max() < 1e-12
