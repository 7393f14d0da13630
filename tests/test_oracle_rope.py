"""The rotary and qk-norm oracle against something other than itself: complex multiplication and
autograd in torch fp64, central differences, closed forms (CPU only)."""
import numpy as np
import pytest
import torch

import oracle
from dynamic_sparse_attention_estimate_gb300.inputs import block_major_permutation, token_positions

CASES = [((6, 4, 6), 16, "interleaved"), ((6, 4, 6), 16, "halves"), ((0, 0, 8), 12, "interleaved"),
         ((2, 0, 6), 8, "halves"), ((0, 0, 0), 4, "interleaved")]


def _torch_rope(x, ang, pairing):
    """Pair by pair as complex numbers, in torch."""
    R = 2 * ang.shape[-1]
    f, g = oracle.pair_features(R, pairing)
    z = torch.complex(x[..., f], x[..., g]) * torch.polar(torch.ones_like(ang), ang)
    out = x.clone()
    out[..., f] = z.real
    out[..., g] = z.imag
    return out


@pytest.mark.parametrize("axes,d,pairing", CASES)
def test_rope_is_a_complex_rotation(axes, d, pairing):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 3, 5, d))
    ang = oracle.rope_angles(rng.integers(0, 50, (5, 3)), axes)
    want = _torch_rope(torch.from_numpy(x), torch.from_numpy(ang), pairing).numpy()
    got = oracle.rope(x, ang, pairing)
    assert np.abs(got - want).max() < 1e-13
    # turned back, and its length kept
    assert np.abs(oracle.rope(got, ang, pairing, backward=True) - x).max() < 1e-13
    assert np.abs((got ** 2).sum(-1) - (x ** 2).sum(-1)).max() < 1e-12


def test_position_zero_is_the_identity_and_products_see_differences_only():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 1, 16))
    axes = (4, 6, 6)
    assert np.array_equal(oracle.rope(q, oracle.rope_angles(np.zeros((1, 3)), axes)), q)
    dot = lambda p, r: float((oracle.rope(q, oracle.rope_angles(np.array([p]), axes)) *
                              oracle.rope(k, oracle.rope_angles(np.array([r]), axes))).sum())
    assert dot((3, 7, 2), (1, 9, 5)) == pytest.approx(dot((13, 10, 22), (11, 12, 25)), abs=1e-12)


@pytest.mark.parametrize("axes,d,pairing", CASES)
def test_gradients_against_autograd_and_differences(axes, d, pairing):
    rng = np.random.default_rng(3)
    x, dy, w = rng.standard_normal((2, 2, 4, d)), rng.standard_normal((2, 2, 4, d)), rng.standard_normal(d)
    ang = oracle.rope_angles(rng.integers(0, 9, (2, 4, 3)), axes)
    eps = 1e-3
    dx, dw = oracle.qk_norm_rope_bwd(dy, x, w, ang, pairing, eps)
    tx, tw = torch.from_numpy(x).requires_grad_(), torch.from_numpy(w).requires_grad_()
    n = torch.nn.functional.rms_norm(tx, (d,), tw, eps)
    _torch_rope(n, torch.from_numpy(ang)[:, None], pairing).backward(torch.from_numpy(dy))
    assert np.abs(dx - tx.grad.numpy()).max() < 1e-12 and np.abs(dw - tw.grad.numpy()).max() < 1e-12
    loss = lambda a, b: float((oracle.qk_norm_rope_fwd(a, b, ang, pairing, eps) * dy).sum())
    ex, ew, h = rng.standard_normal(x.shape), rng.standard_normal(d), 1e-5
    assert (loss(x + h * ex, w) - loss(x - h * ex, w)) / (2 * h) == pytest.approx(float((dx * ex).sum()), rel=1e-6, abs=1e-7)
    assert (loss(x, w + h * ew) - loss(x, w - h * ew)) / (2 * h) == pytest.approx(float((dw * ew).sum()), rel=1e-6, abs=1e-7)


@pytest.mark.parametrize("latent,shape", [((4, 16, 16), None), ((8, 8, 12), (4, 4, 4)), ((7, 8, 16), (4, 4, 4))])
def test_token_positions_are_the_raster_coordinates_of_the_block_major_order(latent, shape):
    pos = token_positions(latent, shape)
    T, Y, X = latent
    assert pos.dtype == torch.int32 and pos.shape == (T * Y * X, 3) and pos.is_contiguous()
    p = pos.numpy().astype(np.int64)
    assert np.array_equal((p[:, 0] * Y + p[:, 1]) * X + p[:, 2], block_major_permutation(latent, shape))
    assert (p >= 0).all() and (p < np.array(latent)).all()
