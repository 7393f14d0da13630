"""Host validation of the calls with 4-bit weights: refused before anything is launched (CPU only)."""
import pytest
import torch

import dynamic_sparse_attention_estimate_gb300 as pkg
from dynamic_sparse_attention_estimate_gb300.binding import W4Dims

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


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


A = [0x1000000 * i for i in range(1, 12)]
FWD = dict(x=A[0], data=A[1], scale=A[2], zero=A[3], bias=A[4], y=A[5])
BWD = dict(dy=A[0], data=A[1], scale=A[2], zero=A[3], dx=A[4])
QUANT = dict(w=A[0], data=A[1], scale=A[2], zero=A[3])


def fwd(lib, d, **changed):
    return lib.dsv_w4_linear_fwd(d, *{**FWD, **changed}.values(), None)


def bwd(lib, d, ws=A[6], nbytes=1 << 30, **changed):
    return lib.dsv_w4_linear_bwd(d, *{**BWD, **changed}.values(), ws, nbytes, None)


def quant(lib, d, **changed):
    return lib.dsv_w4_quantize(d, *{**QUANT, **changed}.values(), None)


def refused(lib, status, what, code=INVALID):
    assert status == code and what in lib.dsv_last_error_message(), lib.dsv_last_error_message()


@pytest.mark.parametrize("M,D,F,G,what,code", [
    (0, 128, 16, 64, b"M must", INVALID), (65, 128, 16, 64, b"M must", INVALID), (1, 128, 16, 16, b"group", UNSUPPORTED),
    (1, 128, 16, 0, b"group", UNSUPPORTED), (1, 128, 16, 256, b"group", UNSUPPORTED), (1, 0, 16, 64, b"D must", INVALID),
    (1, 96, 16, 64, b"D must", INVALID), (1, 2 ** 20 + 128, 16, 64, b"D must", INVALID), (1, 128, 0, 64, b"F >= 1", INVALID),
    (1, 2 ** 20, 2 ** 20 + 1, 64, b"F >= 1", INVALID)])
def test_bad_dims(lib, M, D, F, G, what, code):
    d = W4Dims(M, D, F, G, 0)
    refused(lib, fwd(lib, d), what, code)
    refused(lib, bwd(lib, d), what, code)
    if b"M must" not in what:
        refused(lib, quant(lib, d), what, code)
    assert lib.dsv_w4_linear_bwd_workspace(d) == 0
    assert lib.dsv_w4_linear_fwd(None, *FWD.values(), None) == INVALID


def test_pointers_overlaps_and_workspace(lib):
    d = W4Dims(2, 128, 48, 32, 0)
    for call, names, may_miss in ((fwd, FWD, ("zero", "bias")), (bwd, BWD, ("zero",)), (quant, QUANT, ("zero",))):
        for n in names:
            if n not in may_miss:
                refused(lib, call(lib, d, **{n: None}), n.encode() + b" is NULL")
            refused(lib, call(lib, d, **{n: A[8] + 8}), n.encode() + b" is not 16-byte aligned")
    refused(lib, fwd(lib, d, y=A[0]), b"y overlaps x")
    refused(lib, fwd(lib, d, y=A[1] + 48 * 64 - 16), b"y overlaps data")
    refused(lib, fwd(lib, d, y=A[4]), b"y overlaps bias")
    refused(lib, bwd(lib, d, dx=A[3]), b"dx overlaps zero")
    refused(lib, bwd(lib, d, dx=A[0]), b"dx overlaps dy")
    refused(lib, bwd(lib, W4Dims(2, 128, 48, 32, 1), dx=A[0] + 2 * 48 * 4 - 16), b"dx overlaps dy")
    refused(lib, quant(lib, d, data=A[0]), b"data overlaps w")
    refused(lib, quant(lib, d, scale=A[1]), b"scale overlaps data")
    refused(lib, quant(lib, d, zero=A[2]), b"zero overlaps scale")
    need = lib.dsv_w4_linear_bwd_workspace(d)
    assert need >= 2 * 128 * 4
    refused(lib, bwd(lib, d, ws=None), b"NULL", WORKSPACE)
    refused(lib, bwd(lib, d, ws=A[6] + 16), b"aligned", WORKSPACE)
    refused(lib, bwd(lib, d, nbytes=need - 1), b"below", WORKSPACE)
    refused(lib, bwd(lib, d, ws=A[1]), b"ws overlaps data")


def test_python_refuses(lib):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w = pkg.W4Weight(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        pkg.dsv_w4_linear_fwd(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.dsv_w4_linear_bwd(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.dsv_w4_quantize(x)
