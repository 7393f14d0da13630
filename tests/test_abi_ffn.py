"""Host validation of the gated feed-forward calls: refused before anything is launched (CPU only)."""
import pytest
import torch

import dynamic_sparse_attention_estimate_gb300 as pkg
from dynamic_sparse_attention_estimate_gb300.binding import FfnDims

INVALID, WORKSPACE = 1, 3


@pytest.fixture(scope="module")
def lib():
    from dynamic_sparse_attention_estimate_gb300.build import build
    build()
    return pkg.load_library()


@pytest.fixture(autouse=True)
def no_gpu():
    """Made-up device addresses are only passed where no launch could follow."""
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses are only passed where no GPU is visible")


A = [0x1000000 * i for i in range(1, 10)]


def fwd(lib, d, x=A[0], wg=A[1], wu=A[2], h=A[3], ws=None, nbytes=0):
    return lib.dsv_ffn_gated_fwd(d, x, wg, wu, h, ws, nbytes, None)


def bwd(lib, d, dh=A[0], x=A[1], wg=A[2], wu=A[3], dx=A[4], dwg=A[5], dwu=A[6], ws=A[7], nbytes=1 << 30):
    return lib.dsv_ffn_gated_bwd(d, dh, x, wg, wu, dx, dwg, dwu, ws, nbytes, None)


@pytest.mark.parametrize("M,D,F,act,what", [
    (0, 64, 64, 0, b"M must"), (-1, 64, 64, 0, b"M must"), (2 ** 31, 64, 64, 0, b"M must"), (4, 0, 64, 0, b"multiples of 8"),
    (4, 60, 64, 0, b"multiples of 8"), (4, 64, 4, 0, b"multiples of 8"), (4, 64, 2 ** 20 + 8, 0, b"multiples of 8"),
    (4, 64, 64, 2, b"act"), (4, 64, 64, -1, b"act")])
def test_bad_dims(lib, M, D, F, act, what):
    d = FfnDims(M, D, F, act)
    assert fwd(lib, d) == INVALID and what in lib.dsv_last_error_message()
    assert bwd(lib, d) == INVALID and what in lib.dsv_last_error_message()
    assert lib.dsv_ffn_gated_bwd_workspace(d) == lib.dsv_ffn_gated_fwd_workspace(d) == 0
    assert lib.dsv_ffn_gated_fwd(None, *A[:4], None, 0, None) == INVALID


def test_pointers_overlaps_and_workspace(lib):
    d = FfnDims(16, 64, 128, 0)
    for n in ("x", "wg", "wu", "h"):
        assert fwd(lib, d, **{n: None}) == INVALID and b"NULL" in lib.dsv_last_error_message()
        assert fwd(lib, d, **{n: A[4] + 8}) == INVALID and b"aligned" in lib.dsv_last_error_message()
    for n in ("dh", "x", "wg", "wu", "dx", "dwg", "dwu"):
        assert bwd(lib, d, **{n: None}) == INVALID and b"NULL" in lib.dsv_last_error_message()
    assert fwd(lib, d, h=A[0]) == INVALID and b"h overlaps x" in lib.dsv_last_error_message()
    assert fwd(lib, d, h=A[1] + 64 * 128 * 2 - 16) == INVALID and b"h overlaps w_gate" in lib.dsv_last_error_message()
    assert bwd(lib, d, dwu=A[5]) == INVALID and b"dw_up overlaps dw_gate" in lib.dsv_last_error_message()
    assert bwd(lib, d, dx=A[0]) == INVALID and b"dx overlaps dh" in lib.dsv_last_error_message()
    assert bwd(lib, d, ws=A[1]) == INVALID and b"ws overlaps x" in lib.dsv_last_error_message()
    need = lib.dsv_ffn_gated_bwd_workspace(d)
    assert need >= 2 * 16 * 128 * 2
    assert bwd(lib, d, ws=None) == WORKSPACE
    assert bwd(lib, d, ws=A[7] + 16) == WORKSPACE
    assert bwd(lib, d, nbytes=need - 1) == WORKSPACE


def test_forward_workspace(lib):
    """Only products that are split over D need one: few tiles, a long D, more than a few tokens."""
    for M, D, F in ((16, 64, 128), (65536, 2048, 5632), (1, 4096, 512), (4, 4096, 512), (16384, 768, 2048)):
        assert lib.dsv_ffn_gated_fwd_workspace(FfnDims(M, D, F, 0)) == 0
    d = FfnDims(128, 4096, 512, 0)
    need = lib.dsv_ffn_gated_fwd_workspace(d)
    assert 0 < need <= 76 * 256 * 256 * 4
    assert fwd(lib, d) == WORKSPACE and b"NULL" in lib.dsv_last_error_message()
    assert fwd(lib, d, ws=A[4] + 16, nbytes=need) == WORKSPACE
    assert fwd(lib, d, ws=A[4], nbytes=need - 1) == WORKSPACE
    assert fwd(lib, d, ws=A[1], nbytes=need) == INVALID and b"ws overlaps w_gate" in lib.dsv_last_error_message()


def test_python_refuses_cpu_tensors(lib):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.dsv_ffn_gated_fwd(x, x, x)
