"""What the GPU tests of the qk norm's backward can see: mistakes planted in the oracle's gradients have to fail their
checks, right ones as a kernel returns them have to pass (CPU only)."""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_helpers import np64
from tests.test_gpu_rope import check_weight_sum, direction_check, norm_case, positions

AXES, EPS = (24, 20, 20), 1e-5


def rounded(a):
    return np64(torch.from_numpy(a).to(torch.bfloat16))


def dx_with(c, ang, projection):
    """dq with its projection term taken so many times."""
    x, w = np64(c["q"]), np64(c["wq"])
    g = oracle.rope(c["dq"], ang, "interleaved", backward=True) * w
    rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    xhat = x * rstd
    return rstd * (g - projection * xhat * (g * xhat).mean(-1, keepdims=True))


def test_differences_see_a_wrong_projection():
    latent = (2, 3, 4)
    c = norm_case(2, 3, latent, 64, 5)
    ang = oracle.rope_angles(positions(latent), AXES)
    dq, dwq = oracle.qk_norm_rope_bwd(c["dq"], c["q"], c["wq"], ang, "interleaved", EPS)
    assert np.abs(dx_with(c, ang, 1.0) - dq).max() < 1e-12
    passes = lambda got, name: [direction_check(got, name, c, ang, EPS, rng) for _ in range(4)]
    rng = np.random.default_rng(6)
    assert all(passes(rounded(dq), "dq")) and all(passes(dwq.astype(np.float32).astype(np.float64), "dwq"))
    for projection in (0.0, 0.5, 0.8, 1.2):
        assert not all(passes(rounded(dx_with(c, ang, projection)), "dq")), projection
    for part in (0.99, 1.01):
        assert not all(passes(dwq * part, "dwq")), part


@pytest.mark.parametrize("d,latent", [(64, (17, 19, 31)), (128, (17, 19, 31))])
def test_weight_sums_see_a_lost_or_doubled_unit(d, latent):
    """One tile of tokens out of some hundreds, left out of a weight's gradient or taken twice."""
    B, H, N, tokens, L = 2, 3, int(np.prod(latent)), 1024 // d, 120
    c = norm_case(B, H, latent, d, 22)
    axes = AXES if d == 64 else (44, 42, 42)
    ang = oracle.rope_angles(positions(latent), axes)
    args = (c["dq"], c["q"], c["wq"], ang, "interleaved", EPS)
    dw = oracle.qk_norm_rope_bwd(*args)[1]
    check_weight_sum("right", torch.from_numpy(dw), *args, L)
    for b, first in ((0, 0), (1, N // 2 // tokens * tokens), (1, N - N % tokens)):
        s = slice(first, first + tokens)
        part = oracle.qk_norm_rope_bwd(c["dq"][b:b + 1, :, s], c["q"][b:b + 1, :, s], c["wq"], ang[s], "interleaved", EPS)[1]
        for wrong in (dw - part, dw + part):
            with pytest.raises(AssertionError, match="bound exceeded"):
                check_weight_sum("wrong", torch.from_numpy(wrong), *args, L)
