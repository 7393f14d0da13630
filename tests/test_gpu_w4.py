"""GPU parity of the products with 4-bit weights against the fp64 oracle.

Tolerances, from the arithmetic.  A product of K terms accumulates in fp32 on the tensor cores, 16 terms to an instruction:
with S = sum |terms| it is off by at most (K / 8 + 8) 2^-23 S.
  y:  its 128-column sums are scaled and added (K / 128 products and sums) and joined over 4 warps and up to 4 groups:
      e = (D / 8 + D / 64 + 24) 2^-23 S, and 2^-8 |y| for its rounding (2^-23 (S + |bias|) for the bias).
  dx: dy * scale is rounded once in fp32 and held in two bf16 numbers (2^-16 of it for dy in fp32, exact for bf16); a warp adds
      two products for each row, then 4 warps and at most F / 64 + 1 runs of rows: (F / 4 + F / 64 + 24) 2^-23 S.
These hold for every element; the norm of the error is held to 2^-8 / sqrt 3 of the output's, which roundings of random sign leave.
"""
import numpy as np
import pytest
import torch

import oracle
from dynamic_sparse_attention_estimate_gb300 import (DSVError, W4Weight, dsv_w4_linear_bwd, dsv_w4_linear_bwd_workspace,
                                                     dsv_w4_linear_fwd, dsv_w4_quantize)
from dynamic_sparse_attention_estimate_gb300.binding import dsv_last_device_status
from tests.gpu_helpers import need_gpu, np64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def case(M, D, F, G, zeros, seed=0):
    gen = torch.Generator().manual_seed(seed + 7 * M + D + 3 * F + G)
    c = dict(data=torch.randint(0, 256, (F, D // 2), generator=gen, dtype=torch.uint8),
             scale=(0.01 + 0.1 * torch.rand(F, D // G, generator=gen)).to(BF16),
             zero=torch.randint(0, 16, (F, D // G), generator=gen, dtype=torch.uint8) if zeros else None,
             x=torch.randn(M, D, generator=gen).to(BF16), dy=torch.randn(M, F, generator=gen),
             bias=torch.randn(F, generator=gen).to(BF16))
    return c


def weight(c):
    return W4Weight(c["data"].cuda(), c["scale"].cuda(), None if c["zero"] is None else c["zero"].cuda())


def check(name, got, ref, bound):
    err = np.abs(np64(got) - ref)
    excess = float((err - bound).max())
    assert excess <= 0, f"{name}: bound exceeded by {excess:.3e}"
    n = float(np.linalg.norm(ref))
    if n > 0 and ref.size >= 4096:
        assert float(np.linalg.norm(err)) / n <= 2.0 ** -8 / 3 ** 0.5, name


def check_fwd(c, y, bias=True):
    w, x = oracle.w4_values(c["data"], c["scale"], c["zero"]), np64(c["x"])
    b = np64(c["bias"]) if bias else 0.0
    ref = x @ w.T + b
    assert np.array_equal(ref, oracle.w4_linear_fwd(c["x"], c["data"], c["scale"], c["zero"], c["bias"] if bias else None))
    S, D = np.abs(x) @ np.abs(w).T, x.shape[1]
    check("y", y, ref, 2.0 ** -8 * np.abs(ref) + (D / 8 + D / 64 + 24) * 2.0 ** -23 * S + 2.0 ** -23 * (S + np.abs(b)))


def check_bwd(c, dx, dy):
    w, d = oracle.w4_values(c["data"], c["scale"], c["zero"]), np64(dy)
    ref = oracle.w4_linear_bwd(dy, c["data"], c["scale"], c["zero"])
    S, F = np.abs(d) @ np.abs(w), d.shape[1]
    bound = 2.0 ** -8 * np.abs(ref) + (F / 4 + F / 64 + 24) * 2.0 ** -23 * S
    check("dx", dx, ref, bound + (2.0 ** -16 * S if dy.dtype is F32 else 0))


# vectors one to 64 on both sides of each tile; one group of columns and part of a chunk, several chunks to a warp; one row,
# part of a tile of rows, more runs of rows than one, runs of several chunks
SHAPES = [(1, 32, 1, 32), (1, 64, 5, 64), (2, 128, 16, 128), (3, 96, 33, 32), (1, 768, 4608, 64), (4, 192, 700, 64), (5, 1184, 513, 32),
          (6, 320, 65, 64), (8, 640, 129, 128), (9, 256, 100, 128), (16, 128, 257, 64), (17, 2048, 64, 64), (31, 160, 40, 32),
          (32, 512, 90, 128), (33, 64, 50, 64), (64, 384, 77, 128), (64, 96, 31, 32), (2, 8192, 24, 64), (7, 1152, 12345, 64),
          (1, 128, 50000, 64), (4, 8192, 16, 32),
          (3, 8192, 4000, 64), (9, 8192, 2600, 32), (2, 4096, 5633, 128)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,D,F,G", SHAPES)
def test_both_directions_match_the_oracle(M, D, F, G, zeros):
    need_gpu()
    c = case(M, D, F, G, zeros)
    w = weight(c)
    check_fwd(c, dsv_w4_linear_fwd(c["x"].cuda(), w, c["bias"].cuda()))
    check_fwd(c, dsv_w4_linear_fwd(c["x"].cuda(), w), bias=False)
    for dy in (c["dy"], c["dy"].to(BF16)):
        check_bwd(c, dsv_w4_linear_bwd(dy.cuda(), w), dy)
    assert dsv_last_device_status() == 0


@pytest.mark.parametrize("M", list(range(1, 34)) + [63, 64])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_every_number_of_vectors(M, G):
    need_gpu()
    c = case(M, 256, 70, G, True, seed=1)
    w = weight(c)
    check_fwd(c, dsv_w4_linear_fwd(c["x"].cuda(), w, c["bias"].cuda()))
    check_bwd(c, dsv_w4_linear_bwd(c["dy"].cuda(), w), c["dy"])


def test_whole_numbers_are_exact():
    """Small whole numbers and scales that are powers of two: every sum is exact, and the outputs that fit bf16 are too."""
    need_gpu()
    M, D, F, G = 5, 320, 150, 64
    c = case(M, D, F, G, True)
    gen = torch.Generator().manual_seed(4)
    c["scale"] = (2.0 ** torch.randint(-1, 2, (F, D // G), generator=gen)).to(BF16)
    c["x"] = torch.zeros(M, D, dtype=BF16)
    c["x"][:, ::40] = torch.randint(-1, 2, (M, 8), generator=gen).to(BF16)
    dy = torch.zeros(M, F)
    dy[:, ::30] = torch.randint(-1, 2, (M, 5), generator=gen).float()
    w = weight(c)
    y, dx = dsv_w4_linear_fwd(c["x"].cuda(), w), dsv_w4_linear_bwd(dy.cuda(), w)
    assert np.array_equal(np64(y), oracle.w4_linear_fwd(c["x"], c["data"], c["scale"], c["zero"]))
    assert np.array_equal(np64(dx), oracle.w4_linear_bwd(dy, c["data"], c["scale"], c["zero"]))


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("F,D,G", [(1, 32, 32), (7, 96, 32), (33, 320, 64), (257, 1152, 128), (1000, 64, 64)])
def test_quantize_is_the_oracles(F, D, G, symmetric):
    need_gpu()
    gen = torch.Generator().manual_seed(F + D)
    w = (torch.randn(F, D, generator=gen) * torch.exp(2 * torch.randn(F, 1, generator=gen))).to(BF16)
    w[0, :G] = 0
    w[-1, -G:] = w[-1, -G:].abs()
    q, scale, zero = oracle.w4_quantize(w, G, symmetric)
    got = dsv_w4_quantize(w.cuda(), G, symmetric)
    data = got.data.cpu().numpy()
    assert np.array_equal(np.stack((data & 15, data >> 4), -1).reshape(F, D), q)
    assert np.array_equal(np64(got.scale), scale)
    assert got.zero is None if symmetric else np.array_equal(got.zero.cpu().numpy(), zero)


@pytest.mark.parametrize("symmetric", [True, False])
def test_quantize_of_the_largest_weights(symmetric):
    """A group may hold both ends of the type: its scale is finite, and every weight within half a step (and what the scale's and the
    zero point's roundings move the ends: 15 steps of 2^-8 and half a step)."""
    need_gpu()
    top = torch.finfo(BF16).max
    w = torch.linspace(-1, 1, 2 * 128, dtype=torch.float64).reshape(2, 128).mul(top).to(BF16)
    w[0, 0], w[0, 1], w[1, 5] = top, -top, -top
    got = dsv_w4_quantize(w.cuda(), 64, symmetric)
    assert bool(torch.isfinite(got.scale).all())
    values = oracle.w4_values(got.data, got.scale, got.zero)
    step = np.repeat(np64(got.scale), 64, 1)
    assert float((np.abs(values - np64(w)) / step).max()) <= 1.0 + 15 * 2.0 ** -8


def guarded(shape, dtype, fill, pad=4096):
    numel = int(np.prod(shape))
    buf = torch.full((numel + 2 * pad,), fill, dtype=dtype, device="cuda")
    return buf[pad:pad + numel].view(shape), buf, pad


@pytest.mark.parametrize("M,D,F,G", [(1, 32, 1, 32), (5, 1184, 513, 32), (9, 256, 100, 128), (33, 64, 50, 64)])
def test_nothing_around_the_outputs_is_written(M, D, F, G):
    need_gpu()
    c = case(M, D, F, G, True)
    w = weight(c)
    y, dx = guarded((M, F), BF16, -77), guarded((M, D), BF16, -77)
    ws = guarded((dsv_w4_linear_bwd_workspace(M, D, F, G) // 4,), F32, -77)
    ws[0].fill_(float("nan"))
    dsv_w4_linear_fwd(c["x"].cuda(), w, c["bias"].cuda(), out=y[0])
    dsv_w4_linear_bwd(c["dy"].cuda(), w, out=dx[0], workspace=ws[0])
    torch.cuda.synchronize()
    for view, buf, pad in (y, dx, ws):
        assert (buf[:pad] == -77).all() and (buf[pad + view.numel():] == -77).all()
    check_fwd(c, y[0])
    check_bwd(c, dx[0], c["dy"])


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M", [2, 9, 33])
def test_a_bad_vector_stays_in_its_row(M, G):
    need_gpu()
    c = case(M, 384, 90, G, True)
    w, x, dy = weight(c), c["x"].cuda(), c["dy"].cuda()
    y, dx = dsv_w4_linear_fwd(x, w), dsv_w4_linear_bwd(dy, w)
    x[1, 5], dy[1, 5] = float("nan"), float("nan")
    y2, dx2 = dsv_w4_linear_fwd(x, w), dsv_w4_linear_bwd(dy, w)
    keep = torch.arange(M, device="cuda") != 1
    assert torch.equal(y2[keep], y[keep]) and torch.equal(dx2[keep], dx[keep])
    assert torch.isnan(y2[1]).all() and torch.isnan(dx2[1]).all()
    x[1, 5], dy[1, 5] = float("inf"), float("-inf")
    values = torch.from_numpy(oracle.w4_values(c["data"], c["scale"], c["zero"])).cuda()
    y3, dx3 = dsv_w4_linear_fwd(x, w), dsv_w4_linear_bwd(dy, w)
    for got, v in ((y3, values[:, 5]), (dx3, -values[5])):
        want = v * float("inf")          # a weight of 0 gives NaN, as the definition does
        assert torch.equal(torch.isnan(got[1]), torch.isnan(want)) and torch.equal(got[1][~torch.isnan(want)].double(), want[~torch.isnan(want)])


def test_a_bad_scale_stays_in_its_weights():
    """A group whose scale is not finite reaches its own row of y and its own columns of dx."""
    need_gpu()
    c = case(3, 256, 40, 64, False)
    w = weight(c)
    y, dx = dsv_w4_linear_fwd(c["x"].cuda(), w), dsv_w4_linear_bwd(c["dy"].cuda(), w)
    w.scale[17, 2] = float("nan")
    y2, dx2 = dsv_w4_linear_fwd(c["x"].cuda(), w), dsv_w4_linear_bwd(c["dy"].cuda(), w)
    rows, cols = torch.arange(40, device="cuda") != 17, torch.arange(256, device="cuda") // 64 != 2
    assert torch.equal(y2[:, rows], y[:, rows]) and torch.isnan(y2[:, 17]).all()
    assert torch.equal(dx2[:, cols], dx[:, cols]) and torch.isnan(dx2[:, ~cols]).all()


@pytest.mark.parametrize("G", [32, 64, 128])
def test_tensors_that_start_inside_an_allocation(G):
    """16-byte boundaries that are none of 32."""
    need_gpu()
    c = case(5, 384, 300, G, True)
    w, x, dy = weight(c), c["x"].cuda(), c["dy"].cuda()
    y, dx = dsv_w4_linear_fwd(x, w), dsv_w4_linear_bwd(dy, w)

    def moved(t):
        skip = 16 // t.element_size()
        out = torch.empty(t.numel() + skip, dtype=t.dtype, device="cuda")[skip:].view(t.shape).copy_(t)
        assert out.data_ptr() % 32 == 16
        return out

    w = W4Weight(*map(moved, w))
    assert torch.equal(dsv_w4_linear_fwd(moved(x), w, out=moved(y)), y) and torch.equal(dsv_w4_linear_bwd(moved(dy), w, out=moved(dx)), dx)


def test_the_smallest_numbers_keep_their_bits():
    """Vectors of 2^-100 to 2^-60: the weights' unpacking scales them no further down."""
    need_gpu()
    c = case(4, 256, 70, 64, True)
    c["x"] = (c["x"].float() * torch.tensor([2.0 ** -60, 2.0 ** -80, 2.0 ** -90, 2.0 ** -100])[:, None]).to(BF16)
    c["dy"] = c["dy"] * torch.tensor([2.0 ** -60, 2.0 ** -80, 2.0 ** -90, 2.0 ** -100])[:, None]
    w = weight(c)
    check_fwd(c, dsv_w4_linear_fwd(c["x"].cuda(), w), bias=False)
    check_bwd(c, dsv_w4_linear_bwd(c["dy"].cuda(), w), c["dy"])


def test_shapes_of_vectors():
    need_gpu()
    c = case(6, 128, 48, 64, False)
    w = weight(c)
    y = dsv_w4_linear_fwd(c["x"].cuda(), w)
    assert torch.equal(dsv_w4_linear_fwd(c["x"].cuda().view(2, 3, 128), w), y.view(2, 3, 48))
    assert torch.equal(dsv_w4_linear_fwd(c["x"][0].cuda(), w), dsv_w4_linear_fwd(c["x"][:1].cuda(), w)[0])
    assert dsv_w4_linear_bwd(c["dy"].cuda().view(3, 2, 48), w).shape == (3, 2, 128)


def test_repeats_streams_and_a_replayed_graph():
    need_gpu()
    c = case(4, 1152, 5000, 64, True)
    w, x, dy = weight(c), c["x"].cuda(), c["dy"].cuda()
    y, dx = dsv_w4_linear_fwd(x, w), dsv_w4_linear_bwd(dy, w)
    found = []
    torch.cuda.synchronize()
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            for _ in range(4):
                found.append((dsv_w4_linear_fwd(x, w), dsv_w4_linear_bwd(dy, w)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, y) and torch.equal(b, dx) for a, b in found)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        cy, cdx = dsv_w4_linear_fwd(x, w), dsv_w4_linear_bwd(dy, w)
    other = case(4, 1152, 5000, 64, True, seed=3)
    for a, n in ((x, "x"), (dy, "dy"), (w.data, "data"), (w.scale, "scale"), (w.zero, "zero")):
        a.copy_(other[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cy, dsv_w4_linear_fwd(x, w)) and torch.equal(cdx, dsv_w4_linear_bwd(dy, w))
    check_fwd(other, cy, bias=False)
    check_bwd(other, cdx, other["dy"])


def test_offsets_past_32_bits():
    """More than 2^32 bytes of weights: the last rows come out as they do alone, and their gradient is of those rows alone."""
    need_gpu()
    D, F, G, tail = 8192, 1100000, 64, 96
    gen = torch.Generator(device="cuda").manual_seed(0)
    data = torch.randint(0, 256, (F, D // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scale = torch.full((F, D // G), 0.01, dtype=BF16, device="cuda")
    x = torch.randn(2, D, generator=gen, device="cuda").to(BF16)
    last = W4Weight(data[-tail:].clone(), scale[-tail:].clone())
    w = W4Weight(data, scale)
    assert torch.equal(dsv_w4_linear_fwd(x, w)[:, -tail:], dsv_w4_linear_fwd(x, last))
    dy = torch.zeros(2, F, device="cuda")
    dy[:, -tail:] = torch.randint(-2, 3, (2, tail), generator=gen, device="cuda").float()
    want = oracle.w4_linear_bwd(dy[:, -tail:], last.data, last.scale)
    S = np.abs(np64(dy[:, -tail:])) @ np.abs(oracle.w4_values(last.data, last.scale))
    got = np64(dsv_w4_linear_bwd(dy, w))
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (tail / 4 + 24) * 2.0 ** -23 * S).all()


def test_refusals():
    need_gpu()
    c = case(2, 128, 40, 64, True)
    w, x, dy = weight(c), c["x"].cuda(), c["dy"].cuda()
    for bad in (x.float(), x.half(), x[:, :64], x.t(), x.cpu()):
        with pytest.raises(ValueError):
            dsv_w4_linear_fwd(bad, w)
    for bad in (dy.half(), dy[:, :8].contiguous(), dy.cpu(), dy.t()):
        with pytest.raises(ValueError):
            dsv_w4_linear_bwd(bad, w)
    for bad in (w._replace(data=w.data.short()), w._replace(scale=w.scale.float()), w._replace(zero=w.zero[:, :1]),
                w._replace(data=w.data.cpu()), w._replace(scale=w.scale[:20]), w._replace(data=w.data[:, ::2])):
        with pytest.raises(ValueError):
            dsv_w4_linear_fwd(x, bad)
    with pytest.raises(DSVError, match="group"):
        dsv_w4_linear_fwd(x, W4Weight(w.data, torch.zeros(40, 8, dtype=BF16, device="cuda")))
    with pytest.raises(DSVError, match="M must"):
        dsv_w4_linear_fwd(torch.zeros(65, 128, dtype=BF16, device="cuda"), w)
    with pytest.raises(DSVError, match="M must"):
        dsv_w4_linear_fwd(torch.zeros(0, 128, dtype=BF16, device="cuda"), w)
    with pytest.raises(ValueError, match="bias"):
        dsv_w4_linear_fwd(x, w, torch.zeros(40, device="cuda"))
    with pytest.raises(ValueError, match="group"):
        dsv_w4_quantize(torch.zeros(4, 96, dtype=BF16, device="cuda"), 64)
    with pytest.raises(DSVError, match="WORKSPACE"):
        dsv_w4_linear_bwd(dy, w, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    assert dsv_last_device_status() == 0


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,F,G", [(1, 40, 32), (4, 300, 64), (4, 40, 32), (7, 300, 128), (8, 2000, 32), (8, 9000, 64), (13, 300, 64)])
def test_a_gradient_in_32_bits_keeps_them(M, F, G, zeros):
    """Pairs of rows with the same weights, a and d - a of 20 bits: what is left of them is d, which only their last bits hold.  All
    numbers are whole multiples of a power of two, four pairs of 2^20 to a vector: every sum is below 2^23 of them and exact in fp32,
    and so is the output, at most 4 x 3 of them."""
    need_gpu()
    D = 256
    gen = torch.Generator().manual_seed(M + F + G)
    c = case(M, D, F, G, zeros)
    c["scale"] = torch.full((F, D // G), 0.25, dtype=BF16)
    zero = c["zero"] if zeros else torch.full((F, D // G), 8, dtype=torch.uint8)
    dy = torch.zeros(M, F)
    for m in range(M):
        for f in (2 * torch.randperm(F // 2, generator=gen)[:4]).tolist():
            a = float(torch.randint(2 ** 19, 2 ** 20, (1,), generator=gen))
            dy[m, f], dy[m, f + 1] = a, float(torch.randint(-3, 4, (1,), generator=gen)) - a
    q = torch.randint(-1, 2, (F // 2, D), generator=gen).repeat_interleave(2, 0)   # the weight's difference from its zero point
    zero[0::2] = zero[0::2].clamp(1, 14)
    zero[1::2] = zero[0::2]
    q = q + zero.repeat_interleave(G, 1)[:q.shape[0]]
    c["data"] = torch.zeros(F, D // 2, dtype=torch.uint8)
    c["data"][:q.shape[0]] = (q[:, 0::2] | q[:, 1::2] << 4).to(torch.uint8)
    dx = dsv_w4_linear_bwd(dy.cuda(), weight(c))
    assert np.array_equal(np64(dx), oracle.w4_linear_bwd(dy, c["data"], c["scale"], c["zero"]))


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,G", [(2, 32), (2, 64), (4, 128), (9, 32), (9, 64)])
def test_products_between_the_types_largest_numbers(M, G, dtype, sign):
    """A gradient whose product with the scale, 1.9996 x 2^127, is finite in fp32 and rounds to infinity in bf16: times a weight of 0 it
    is 0, times any other an output that rounds to infinity of its sign, as 64 bits have it.  The other rows are zeros."""
    need_gpu()
    c = case(M, 256, 70, G, True)
    c["scale"] = torch.full((70, 256 // G), 181 * 2.0 ** 20, dtype=BF16)
    dy = torch.zeros(M, 70, dtype=dtype)
    dy[1, 37] = sign * 181 * 2.0 ** 93
    exact = oracle.w4_linear_bwd(dy, c["data"], c["scale"], c["zero"])
    assert 3.4e38 < np.abs(exact[exact != 0]).min() < 3.4028e38 and (exact[1] == 0).any()
    dx = dsv_w4_linear_bwd(dy.cuda(), weight(c)).cpu()
    assert torch.equal(dx, torch.from_numpy(exact).to(BF16))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M", [8, 12, 33])
@pytest.mark.parametrize("D,G", [(128, 32), (160, 32), (384, 64), (320, 64), (256, 128), (640, 128)])
def test_forward_of_many_rows(M, D, G, zeros):
    """From 9728 rows on a CTA takes 32 of them: each group and tile of vectors, columns that fill their chunks (or end in one), and a
    last CTA of three rows."""
    need_gpu()
    c = case(M, D, 9731, G, zeros)
    check_fwd(c, dsv_w4_linear_fwd(c["x"].cuda(), weight(c), c["bias"].cuda()))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M", [3, 8, 11])
@pytest.mark.parametrize("D,F,G", [(8192, 9100, 32), (8192, 9001, 64), (8192, 9300, 128), (8160, 4500, 32)])
def test_backward_of_long_runs_of_rows(M, D, F, G, zeros):
    """64 blocks of 128 columns leave four to seven runs of rows, of five to ten chunks of 256 rows (the last shape: three, five): each of a
    CTA's three stages is read and filled again, with every row's gradient in the sums."""
    need_gpu()
    c = case(M, D, F, G, zeros)
    w = weight(c)
    for dy in (c["dy"], c["dy"].to(BF16)):
        check_bwd(c, dsv_w4_linear_bwd(dy.cuda(), w), dy)
