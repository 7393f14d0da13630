"""The gated feed-forward oracle against torch fp64 (its activations, autograd) and central differences (CPU only)."""
import numpy as np
import pytest
import torch

import oracle

F = torch.nn.functional
TORCH_ACT = {"silu": F.silu, "gelu_tanh": lambda g: F.gelu(g, approximate="tanh")}


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_forward_and_gradients(act):
    rng = np.random.default_rng(1)
    M, D, Fh = 7, 5, 9
    x, wg, wu, dh = (rng.standard_normal(s) for s in ((M, D), (Fh, D), (Fh, D), (M, Fh)))
    t = [torch.from_numpy(v).requires_grad_() for v in (x, wg, wu)]
    h = TORCH_ACT[act](t[0] @ t[1].T) * (t[0] @ t[2].T)
    h.backward(torch.from_numpy(dh))
    assert np.abs(oracle.ffn_gated_fwd(x, wg, wu, act) - h.detach().numpy()).max() < 1e-13
    got = oracle.ffn_gated_bwd(dh, x, wg, wu, act)
    for g, v in zip(got, t):
        assert np.abs(g - v.grad.numpy()).max() < 1e-12
    loss = lambda *a: float((oracle.ffn_gated_fwd(*a, act) * dh).sum())
    for i in range(3):
        e, step = rng.standard_normal(t[i].shape), 1e-6
        lo, hi = [x, wg, wu], [x, wg, wu]
        lo[i], hi[i] = lo[i] - step * e, hi[i] + step * e
        assert (loss(*hi) - loss(*lo)) / (2 * step) == pytest.approx(float((got[i] * e).sum()), rel=1e-6, abs=1e-7)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_activation_far_out(act):
    a, slope = oracle.activation(np.array([-1e3, -40.0, 0.0, 40.0, 1e3]), act)
    assert np.allclose(a, [0, 0, 0, 40, 1e3], atol=1e-12) and np.allclose(slope, [0, 0, 0.5, 1, 1], atol=1e-12)
