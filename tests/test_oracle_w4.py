"""The 4-bit weights' oracle: bytes worked by hand, torch fp64 autograd, and rounding against a search (CPU only)."""
import numpy as np
import pytest
import torch

import oracle


def test_bytes_by_hand():
    data = np.zeros((2, 16), dtype=np.uint8)
    data[0, 0], data[1, 15] = 0xF3, 0x90          # row 0: q = 3, 15; row 1: the last two are 0, 9
    scale = np.array([[0.5], [2.0]])
    w = oracle.w4_values(data, scale)
    assert w[0, 0] == 0.5 * (3 - 8) and w[0, 1] == 0.5 * (15 - 8) and w[1, 30] == -16 and w[1, 31] == 2
    w = oracle.w4_values(data, scale, np.array([[1], [9]], dtype=np.uint8))
    assert w[0, 0] == 1 and w[0, 1] == 7 and w[1, 31] == 0


def test_products_and_gradient():
    rng = np.random.default_rng(0)
    F, D, G = 9, 128, 32
    data = rng.integers(0, 256, (F, D // 2), dtype=np.uint8)
    scale, zero, bias = rng.random((F, D // G)), rng.integers(0, 16, (F, D // G), dtype=np.uint8), rng.standard_normal(F)
    x, dy = rng.standard_normal((3, D)), rng.standard_normal((3, F))
    t = torch.from_numpy(x).requires_grad_()
    q = torch.from_numpy(np.stack((data & 15, data >> 4), -1).reshape(F, D // G, G).astype(np.float64))
    w = ((q - torch.from_numpy(zero).double()[..., None]) * torch.from_numpy(scale)[..., None]).view(F, D)
    y = torch.nn.functional.linear(t, w, torch.from_numpy(bias))
    y.backward(torch.from_numpy(dy))
    assert np.abs(oracle.w4_linear_fwd(x, data, scale, zero, bias) - y.detach().numpy()).max() < 1e-12
    assert np.abs(oracle.w4_linear_bwd(dy, data, scale, zero) - t.grad.numpy()).max() < 1e-12


@pytest.mark.parametrize("symmetric", [True, False])
def test_rounding_takes_the_nearest_value(symmetric):
    rng = np.random.default_rng(3)
    w = torch.from_numpy(rng.standard_normal((5, 96))).to(torch.bfloat16)
    w[0, 32:64] = 0
    w[1, :32] = w[1, :32].abs()
    q, scale, zero = oracle.w4_quantize(w, 32, symmetric)
    assert q.min() >= 0 and q.max() <= 15 and (q == np.rint(q)).all()
    x = w.double().numpy().reshape(5, 3, 32)
    values = scale[..., None, None] * (np.arange(16) - zero[..., None, None])     # all that a group can hold
    best = np.abs(x[..., None] - values).min(-1)
    got = np.abs(scale[..., None] * (q.reshape(5, 3, 32) - zero[..., None]) - x)
    assert (got <= best + 1e-12).all()
    assert scale[0, 1] == 0 and (q.reshape(5, 3, 32)[0, 1] == zero[0, 1]).all()
    top = np.abs(x).max(-1) / 7 if symmetric else (np.maximum(x.max(-1), 0) - np.minimum(x.min(-1), 0)) / 15
    assert (np.abs(scale - top) <= 2.0 ** -8 * top).all()
