"""Host validation of the gated residual's calls: refused before anything is launched (CPU only)."""
import pytest
import torch

import dynamic_sparse_attention_estimate_gb300 as pkg
from dynamic_sparse_attention_estimate_gb300.binding import ResidualDims

INVALID, WORKSPACE = 1, 3
NONE, RMS, LAYER = 0, 1, 2


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


A = [0x1000000 * i for i in range(1, 20)]
FWD = dict(x=A[0], z=A[1], gate=A[2], w_post=A[3], scale=A[4], shift=A[5], w_pre=A[6], r=A[7], y=A[8])
BWD = dict(dr=A[0], dy=A[1], r=A[2], z=A[3], gate=A[4], w_post=A[5], scale=A[6], w_pre=A[7], dx=A[8], dz=A[9], d_gate=A[10],
           dw_post=A[11], d_scale=A[12], d_shift=A[13], dw_pre=A[14])


def dims(B=2, N=16, D=64, post=RMS, pre=LAYER, f32=0, alpha=1.0, eps=1e-6, strides=None, d_stride=None):
    return ResidualDims(B, N, D, post, pre, f32, alpha, eps, *(strides or (D, D, D)), D if d_stride is None else d_stride)


def fwd(lib, d, **changed):
    return lib.dsv_residual_norm_fwd(d, *{**FWD, **changed}.values(), None)


def bwd(lib, d, ws=A[15], nbytes=1 << 30, **changed):
    return lib.dsv_residual_norm_bwd(d, *{**BWD, **changed}.values(), ws, nbytes, None)


def refused(lib, status, what, code=INVALID):
    assert status == code and what in lib.dsv_last_error_message(), lib.dsv_last_error_message()


@pytest.mark.parametrize("changed,what", [
    (dict(B=0), b"B must"), (dict(B=65536), b"B must"), (dict(N=0), b"B must"), (dict(N=2 ** 30), b"below 2^31"),
    (dict(D=4), b"multiple of 8"), (dict(D=60), b"multiple of 8"), (dict(D=8200), b"multiple of 8"), (dict(post=LAYER), b"post must"),
    (dict(post=-1), b"post must"), (dict(pre=3), b"pre must"), (dict(eps=-1.0), b"eps"), (dict(eps=float("nan")), b"eps"),
    (dict(eps=float("inf")), b"eps"), (dict(alpha=float("inf")), b"alpha"), (dict(alpha=float("nan")), b"alpha")])
def test_bad_dims(lib, changed, what):
    d = dims(**changed)
    refused(lib, fwd(lib, d), what)
    refused(lib, bwd(lib, d), what)
    assert lib.dsv_residual_norm_bwd_workspace(d) == 0
    assert lib.dsv_residual_norm_fwd(None, *FWD.values(), None) == INVALID


def test_null_and_misaligned(lib):
    d = dims()
    for n in ("x", "z", "r", "y"):
        refused(lib, fwd(lib, d, **{n: None}), n.encode() + b" is NULL")
    for n in FWD:
        refused(lib, fwd(lib, d, **{n: A[16] + 8}), n.encode() + b" is not 16-byte aligned")
    for n in ("dy", "r", "z", "dx", "dz"):
        refused(lib, bwd(lib, d, **{n: None}), n.encode() + b" is NULL")
    for n in BWD:
        refused(lib, bwd(lib, d, **{n: A[16] + 8}), n.encode() + b" is not 16-byte aligned")


def test_what_no_norm_reads_is_refused(lib):
    gone = dict(scale=None, shift=None, w_pre=None, y=None)
    for n in gone:
        refused(lib, fwd(lib, dims(pre=NONE), **{**gone, n: FWD[n]}), b"without a pre norm")
    gone = dict(dy=None, r=None, scale=None, w_pre=None, d_scale=None, d_shift=None, dw_pre=None)
    for n in gone:
        refused(lib, bwd(lib, dims(pre=NONE), **{**gone, n: BWD[n]}), b"without a pre norm")
    refused(lib, fwd(lib, dims(post=NONE)), b"w_post without a post norm")
    refused(lib, bwd(lib, dims(post=NONE)), b"w_post without a post norm")
    refused(lib, bwd(lib, dims(post=NONE), w_post=None), b"dw_post without a post norm")


def test_strides(lib):
    for s in (-8, 4, 2 ** 41):
        refused(lib, fwd(lib, dims(strides=(s, 64, 64))), b"gate: the stride")
        refused(lib, fwd(lib, dims(strides=(64, s, 64))), b"scale: the stride")
        refused(lib, fwd(lib, dims(strides=(64, 64, s))), b"shift: the stride")
        refused(lib, bwd(lib, dims(strides=(s, 64, 64))), b"gate: the stride")
    for s in (0, 63, 66, 2 ** 41):
        refused(lib, bwd(lib, dims(d_stride=s)), b"d_stride")


def test_overlaps(lib):
    e = 2 * 16 * 64
    refused(lib, fwd(lib, dims(), r=A[0] + 16), b"r overlaps x")
    refused(lib, fwd(lib, dims(f32=1), r=A[1] - 16), b"r overlaps z")
    refused(lib, fwd(lib, dims(), y=A[0]), b"y overlaps x")
    refused(lib, fwd(lib, dims(), r=A[0], y=A[0]), b"y overlaps r")
    refused(lib, fwd(lib, dims(), y=A[1]), b"y overlaps z")
    refused(lib, fwd(lib, dims(), y=A[6]), b"y overlaps w_pre")
    refused(lib, fwd(lib, dims(strides=(64, 4096, 64)), y=A[4] + 2 * 4096), b"y overlaps scale")
    refused(lib, bwd(lib, dims(), dx=A[0] + 16), b"dx overlaps dr")
    refused(lib, bwd(lib, dims(), dx=A[2]), b"dx overlaps r")
    refused(lib, bwd(lib, dims(), dz=A[3]), b"dz overlaps z")
    refused(lib, bwd(lib, dims(), dx=A[0], dz=A[0] + 2 * e - 16), b"dz overlaps dx")
    refused(lib, bwd(lib, dims(), dw_post=A[9]), b"dw_post overlaps dz")
    refused(lib, bwd(lib, dims(), d_gate=A[3]), b"d_gate overlaps z")
    refused(lib, bwd(lib, dims(), d_scale=A[15]), b"d_scale overlaps ws")
    refused(lib, bwd(lib, dims(), d_scale=A[10]), b"d_scale overlaps d_gate")
    # one gradient [B][6][D]: parts interleave, halves of parts do not
    wide = dims(d_stride=6 * 64)
    refused(lib, bwd(lib, wide, d_scale=A[10] + 4 * 32), b"d_scale overlaps d_gate")
    refused(lib, bwd(lib, wide, d_scale=A[10] + 4 * (6 * 64 - 32)), b"d_scale overlaps d_gate")
    refused(lib, bwd(lib, wide, d_scale=A[10] + 4 * 64, d_shift=A[10] + 4 * 64), b"d_shift overlaps d_scale")
    refused(lib, bwd(lib, wide, d_scale=A[10] + 4 * 64, d_shift=A[10] + 4 * 5 * 64, nbytes=0), b"below", WORKSPACE)


def test_workspace(lib):
    d = dims()
    need = lib.dsv_residual_norm_bwd_workspace(d)
    assert need >= 2 * 3 * 64 * 4
    refused(lib, bwd(lib, d, ws=None), b"NULL", WORKSPACE)
    refused(lib, bwd(lib, d, ws=A[15] + 16), b"aligned", WORKSPACE)
    refused(lib, bwd(lib, d, nbytes=need - 1), b"below", WORKSPACE)
    refused(lib, bwd(lib, d, ws=A[3], nbytes=need), b"ws overlaps z")


def test_python_refuses(lib):
    x = torch.zeros(1, 4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.dsv_residual_norm_fwd(x, x)
    with pytest.raises(TypeError, match="dr|r must"):
        pkg.dsv_residual_norm_bwd(None, x, None, x)
    with pytest.raises(ValueError, match="post must"):
        pkg.binding._residual_dims(1, 4, 8, False, "layer", "layer", 1.0, 0.0, 8, 8, 8, 8)
