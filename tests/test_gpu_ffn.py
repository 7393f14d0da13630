"""GPU parity of the gated feed-forward kernels against the fp64 oracle.

Tolerances, from the arithmetic.  A product of K terms accumulates in fp32 on the tensor cores, 16 terms to
an instruction: with S = sum |x| |w| it is off by at most (K / 8 + 8) 2^-23 S =: e(K, S).  The
activation's own evaluation adds 2^-18 of its value (two approximate instructions and a few products).
  h:  2^-8 |h| (one rounding) + 1.2 |u| e(g) + |a| e(u) + 2^-18 |a u|            (|act'| < 1.2)
  dg: E = 2^-8 |dg| + |dh| (1.2 e(u) + 0.9 |u| e(g)) + 2^-16 |dh u|               (|act''| < 0.9)
  du: E = 2^-8 |du| + 1.2 |dh| e(g) + 2^-18 |du|         (dg, du of a few tokens: without the 2^-8)
  dx: 2^-8 |dx| + E_dg |Wg| + E_du |Wu| + e(2F, |dg| |Wg| + |du| |Wu|);   dW likewise over the tokens.
These hold for every element; the norm of the error is held to what roundings of random sign leave: each
rounding is uniform within half a step, at most 2^-8 / sqrt 3 of the value, and two of them are in a
gradient: 2^-8 sqrt(2 / 3) = 3.2e-3 of its norm.
"""
import numpy as np
import pytest
import torch

import oracle
from dynamic_sparse_attention_estimate_gb300 import (DSVError, dsv_ffn_gated_bwd, dsv_ffn_gated_bwd_workspace,
                                                     dsv_ffn_gated_fwd, dsv_ffn_gated_fwd_workspace)
from dynamic_sparse_attention_estimate_gb300.binding import dsv_last_device_status
from tests.gpu_helpers import need_gpu, np64

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
NORM = 2.0 ** -8 * (2.0 / 3.0) ** 0.5


def case(M, D, F, seed=0):
    gen = torch.Generator().manual_seed(seed + 31 * M + D + F)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=gen) * scale).to(BF16)
    return dict(x=r(M, D), wg=r(F, D, scale=1.5 / D ** 0.5), wu=r(F, D, scale=1 / D ** 0.5), dh=r(M, F))


def acc(K, S):
    return (K / 8 + 8) * 2.0 ** -23 * S


def check(name, got, ref, bound):
    err = np.abs(np64(got) - ref)
    excess = float((err - bound).max())
    assert excess <= 0, f"{name}: bound exceeded by {excess:.3e}"
    n = float(np.linalg.norm(ref))
    if n > 0 and ref.size >= 4096:   # enough values for roundings to average
        rel = float(np.linalg.norm(err)) / n
        assert rel <= NORM, f"{name}: rel-L2 {rel:.3e}"


def terms(c, act):
    x, wg, wu = np64(c["x"]), np64(c["wg"]), np64(c["wu"])
    D = x.shape[1]
    g, u = x @ wg.T, x @ wu.T
    a, slope = oracle.activation(g, act)
    eg, eu = acc(D, np.abs(x) @ np.abs(wg).T), acc(D, np.abs(x) @ np.abs(wu).T)
    return x, wg, wu, g, u, a, slope, eg, eu


def check_fwd(c, h, act):
    _, _, _, _, u, a, _, eg, eu = terms(c, act)
    ref = oracle.ffn_gated_fwd(c["x"], c["wg"], c["wu"], act)
    check("h", h, ref, 2.0 ** -8 * np.abs(ref) + 1.2 * np.abs(u) * eg + np.abs(a) * eu + 2.0 ** -18 * np.abs(a * u))


def check_bwd(c, dx, dwg, dwu, act):
    x, wg, wu, _, u, a, slope, eg, eu = terms(c, act)
    dh = np64(c["dh"])
    M, F = dh.shape
    dg, du = np.abs(dh * u * slope), np.abs(dh * a)
    few = M <= 2 or (M <= 4 and x.shape[1] * F <= 1 << 22)
    step = 0.0 if few else 2.0 ** -8             # for a few tokens dg and du stay fp32
    Eg = step * dg + np.abs(dh) * (1.2 * eu + 0.9 * np.abs(u) * eg) + 2.0 ** -16 * np.abs(dh * u)
    Eu = step * du + 1.2 * np.abs(dh) * eg + 2.0 ** -18 * du
    rx, rg, ru = oracle.ffn_gated_bwd(c["dh"], c["x"], c["wg"], c["wu"], act)
    ax, ag, au = np.abs(x), np.abs(wg), np.abs(wu)
    check("dx", dx, rx, 2.0 ** -8 * np.abs(rx) + Eg @ ag + Eu @ au + acc(2 * F, dg @ ag + du @ au))
    check("dw_gate", dwg, rg, 2.0 ** -8 * np.abs(rg) + Eg.T @ ax + acc(M, dg.T @ ax))
    check("dw_up", dwu, ru, 2.0 ** -8 * np.abs(ru) + Eu.T @ ax + acc(M, du.T @ ax))


# one token and a few (2, 3, 4, 5, 8), one feature group, sides around 64, 128 and 256 and their multiples, several
# tiles to a pair of CTAs, products split over a long D, F or M (with a last part that is shorter)
SHAPES = [(2, 8, 24), (2, 4096, 1000), (3, 1000, 104), (4, 264, 1000), (5, 1000, 104), (8, 264, 1000), (1, 4096, 24), (40, 4096, 264), (260, 3080, 136), (9000, 72, 88), (16, 136, 6200), (1, 8, 8), (1, 64, 128), (2, 72, 136), (127, 64, 64), (128, 128, 128), (129, 136, 264), (300, 200, 120),
          (64, 8, 2056), (257, 520, 16), (777, 776, 520), (1000, 1032, 248), (4000, 136, 2600), (9, 2048, 1000),
          (3, 40, 4104)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,D,F", SHAPES)
def test_forward_matches_oracle(M, D, F, act):
    need_gpu()
    c = case(M, D, F)
    h = dsv_ffn_gated_fwd(c["x"].cuda(), c["wg"].cuda(), c["wu"].cuda(), act=act)
    assert dsv_last_device_status() == 0
    check_fwd(c, h, act)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,D,F", SHAPES)
def test_backward_matches_oracle(M, D, F, act):
    need_gpu()
    c = case(M, D, F)
    g = {n: t.cuda() for n, t in c.items()}
    dx, dwg, dwu = dsv_ffn_gated_bwd(g["dh"], g["x"], g["wg"], g["wu"], act=act)
    assert dsv_last_device_status() == 0
    check_bwd(c, dx, dwg, dwu, act)


def guarded(t, pad=4096):
    """A copy of t inside a larger buffer of a fixed pattern: (view, buffer, the pattern)."""
    buf = torch.full((t.numel() + 2 * pad,), -77.0, dtype=t.dtype, device="cuda")
    view = buf[pad:pad + t.numel()].view(t.shape)
    return view, buf, pad


# dx and the weights' gradients in one launch or two, either cut along K, either first, with and without units that
# a pair takes ahead of the others
CUTS = [(10127, 8, 1320), (4, 2600, 6232), (10155, 8, 5112), (10796, 8, 8), (2216, 8, 264), (8846, 8, 320), (513, 8, 1056),
        (806, 8, 4696), (5, 8, 6704), (2205, 8, 456), (1187, 8, 2880), (4948, 8, 1048), (792, 3088, 8)]


@pytest.mark.parametrize("M,D,F", CUTS)
def test_backward_however_it_is_cut(M, D, F):
    need_gpu()
    c = case(M, D, F, seed=5)
    g = {n: t.cuda() for n, t in c.items()}
    ws = torch.full((dsv_ffn_gated_bwd_workspace(M, D, F),), 0xff, dtype=torch.uint8, device="cuda")   # NaN sums
    first = dsv_ffn_gated_bwd(g["dh"], g["x"], g["wg"], g["wu"], workspace=ws)
    assert dsv_last_device_status() == 0
    check_bwd(c, *first, "silu")
    again = dsv_ffn_gated_bwd(g["dh"], g["x"], g["wg"], g["wu"], workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("M,D,F", [(1, 8, 8), (129, 136, 264), (300, 200, 120), (40, 4096, 264), (16, 136, 6200)])
def test_nothing_around_the_outputs_is_written(M, D, F):
    need_gpu()
    c = case(M, D, F)
    g = {n: t.cuda() for n, t in c.items()}
    outs = [guarded(t) for t in (torch.empty(M, F, dtype=BF16), c["x"], c["wg"], c["wu"])]
    fws, fbuf, fpad = guarded(torch.empty(dsv_ffn_gated_fwd_workspace(M, D, F) // 2, dtype=BF16))
    dsv_ffn_gated_fwd(g["x"], g["wg"], g["wu"], out=outs[0][0], workspace=fws)
    ws, wbuf, wpad = guarded(torch.empty(dsv_ffn_gated_bwd_workspace(M, D, F) // 2, dtype=BF16))
    dsv_ffn_gated_bwd(g["dh"], g["x"], g["wg"], g["wu"], out=tuple(o[0] for o in outs[1:]), workspace=ws)
    torch.cuda.synchronize()
    for view, buf, pad in outs + [(ws, wbuf, wpad), (fws, fbuf, fpad)]:
        assert (buf[:pad] == -77).all() and (buf[pad + view.numel():] == -77).all()
    check_fwd(c, outs[0][0], "silu")
    check_bwd(c, outs[1][0], outs[2][0], outs[3][0], "silu")


def test_a_bad_token_stays_in_its_row():
    """Infinities and NaN in one token reach its own row of h and dx (and every weight gradient), no other row."""
    need_gpu()
    M, D, F = 200, 136, 264
    c = case(M, D, F)
    g = {n: t.cuda() for n, t in c.items()}
    clean = dsv_ffn_gated_fwd(g["x"], g["wg"], g["wu"])
    dclean = dsv_ffn_gated_bwd(g["dh"], g["x"], g["wg"], g["wu"])[0]
    g["x"][130, 7] = float("nan")
    g["x"][131, 8] = float("inf")
    h = dsv_ffn_gated_fwd(g["x"], g["wg"], g["wu"])
    dx = dsv_ffn_gated_bwd(g["dh"], g["x"], g["wg"], g["wu"])[0]
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[130] = keep[131] = False
    assert torch.equal(h[keep], clean[keep]) and torch.equal(dx[keep], dclean[keep])
    assert torch.isnan(h[130]).all() and not torch.isfinite(h[131]).any()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_large_activations_do_not_overflow(act):
    """Gates up to several hundred: the logistic function saturates to 0 and 1, and its slope to 0."""
    need_gpu()
    c = case(130, 64, 136, seed=3)
    c["wg"] = (c["wg"].float() * 64).to(BF16)
    g = {n: t.cuda() for n, t in c.items()}
    check_fwd(c, dsv_ffn_gated_fwd(g["x"], g["wg"], g["wu"], act=act), act)
    out = dsv_ffn_gated_bwd(g["dh"], g["x"], g["wg"], g["wu"], act=act)
    assert all(torch.isfinite(t).all() for t in out)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M", [1, 3, 5, 300])
def test_the_slope_where_g_squared_overflows(M, act):
    """|g| = 2^67: act(g) is g or 0 and its slope 1 or 0, all in powers of two, so every result is exact."""
    D, F = 16, 32
    x, wg, wu = torch.zeros(M, D, dtype=BF16), torch.zeros(F, D, dtype=BF16), torch.zeros(F, D, dtype=BF16)
    x[:, 0], wg[:, 0], wu[:, 0] = 2.0 ** 34, 2.0 ** 33, 2.0 ** -34
    wg[F // 2:, 0] *= -1
    dh = torch.ones(M, F, dtype=BF16)
    dx, dwg, dwu = dsv_ffn_gated_bwd(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), act)
    h = dsv_ffn_gated_fwd(x.cuda(), wg.cuda(), wu.cuda(), act)
    rx, rg, ru, rh = (torch.zeros(*s, dtype=torch.float64) for s in ((M, D), (F, D), (F, D), (M, F)))
    rx[:, 0] = F // 2 * (2.0 ** 33 + 2.0 ** 67 * 2.0 ** -34)
    rg[:F // 2, 0] = M * 2.0 ** 34
    ru[:F // 2, 0] = M * 2.0 ** 67 * 2.0 ** 34
    rh[:, :F // 2] = 2.0 ** 67
    for got, ref in ((dx, rx), (dwg, rg), (dwu, ru), (h, rh)):
        assert torch.equal(got.double().cpu(), ref.to(BF16).double())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,D", [(1, 16), (3, 16), (5, 16), (40, 4096), (300, 16)])
def test_a_zero_slope_where_dh_times_u_overflows(M, D, act):
    """g = -2^67: act(g) and its slope are 0, dh u = 2^160 is past fp32; every result is 0 all the same (the second
    half of the features has u = 0 and nothing large: act'(0) = 1/2)."""
    need_gpu()
    F = 32
    x, wg, wu = torch.zeros(M, D, dtype=BF16), torch.zeros(F, D, dtype=BF16), torch.zeros(F, D, dtype=BF16)
    x[:, 0] = 2.0 ** 34
    wg[:F // 2, 0], wu[:F // 2, 0] = -2.0 ** 33, 2.0 ** 26
    dh = torch.ones(M, F, dtype=BF16)
    dh[:, :F // 2] = 2.0 ** 100
    assert dsv_ffn_gated_fwd_workspace(M, D, F) == 0 or M == 40
    for t in dsv_ffn_gated_bwd(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), act):
        assert not t.any() and not torch.isnan(t).any()
    assert not dsv_ffn_gated_fwd(x.cuda(), wg.cuda(), wu.cuda(), act).any()


# dx and the weights' gradients in one launch whose first product goes round the 76 pairs once or twice and on: either
# first, its last round whole or with pairs that take a unit of the other ahead, more than one group of 19 m tiles
ROUNDS = [(1140, 3176, 520), (1171, 3368, 552), (1029, 4024, 520), (2230, 3864, 1040), (4858, 776, 2352), (5055, 1816, 2520),
          (8192, 1024, 2816)]


@pytest.mark.parametrize("M,D,F", ROUNDS)
def test_backward_of_several_rounds_in_one_launch(M, D, F):
    need_gpu()
    c = case(M, D, F, seed=6)
    g = {n: t.cuda() for n, t in c.items()}
    ws = torch.full((dsv_ffn_gated_bwd_workspace(M, D, F),), 0xff, dtype=torch.uint8, device="cuda")   # dg, du of NaN
    outs = [guarded(t) for t in (c["x"], c["wg"], c["wu"])]
    for o, _, _ in outs:
        o.fill_(float("nan"))
    dsv_ffn_gated_bwd(g["dh"], g["x"], g["wg"], g["wu"], out=tuple(o[0] for o in outs), workspace=ws)
    assert dsv_last_device_status() == 0
    for view, buf, pad in outs:
        assert (buf[:pad] == -77).all() and (buf[pad + view.numel():] == -77).all()
    first = [o[0] for o in outs]
    check_bwd(c, *first, "silu")
    again = dsv_ffn_gated_bwd(g["dh"], g["x"], g["wg"], g["wu"])
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_leading_dims_repeatability_streams_and_graphs():
    need_gpu()
    B, N, D, F = 3, 70, 264, 520
    c = case(B * N, D, F)
    g = {n: t.cuda() for n, t in c.items()}
    g["x"], g["dh"] = g["x"].view(B, N, D), g["dh"].view(B, N, F)
    step = lambda: (dsv_ffn_gated_fwd(g["x"], g["wg"], g["wu"]), *dsv_ffn_gated_bwd(g["dh"], g["x"], g["wg"], g["wu"]))
    want = step()
    assert want[0].shape == (B, N, F) and want[1].shape == (B, N, D)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    other = step()
    torch.cuda.synchronize()
    for a, b, w in zip(got, other, want):
        assert torch.equal(a, w) and torch.equal(b, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = step()
    for seed in (0, 5):
        for n, t in case(B * N, D, F, seed).items():
            g[n].view(-1).copy_(t.view(-1))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for a, w in zip(captured, want):
            assert torch.equal(a, w)
    assert dsv_last_device_status() == 0


def test_host_threads_side_by_side():
    """Calls of three host threads on streams of their own, in turn on sizes that take different kernels."""
    import threading
    need_gpu()
    cases = [{n: t.cuda() for n, t in case(*s).items()} for s in ((300, 512, 1232), (777, 776, 520), (5, 1000, 104), (2, 72, 136))]
    step = lambda g: (dsv_ffn_gated_fwd(g["x"], g["wg"], g["wu"]), *dsv_ffn_gated_bwd(g["dh"], g["x"], g["wg"], g["wu"]))
    want = [step(g) for g in cases]
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for i in range(40):
                got = step(cases[i % 4])
                stream.synchronize()
                wrong.extend(i for a, w in zip(got, want[i % 4]) if not torch.equal(a, w))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and dsv_last_device_status() == 0


def test_offsets_past_32_bits():
    """h, dh, dg and du of more than 2^31 elements: the last rows as a call of their own (dh is zero before them, so
    the weights' gradients are theirs too)."""
    need_gpu()
    last, D, F = 300, 8, 1032
    M = 2 ** 21 + 5
    assert (M - last) * F > 2 ** 31
    c = case(last, D, F, seed=9)
    x, dh = torch.ones(M, D, dtype=BF16, device="cuda"), torch.zeros(M, F, dtype=BF16, device="cuda")
    x[-last:], dh[-last:] = c["x"].cuda(), c["dh"].cuda()
    wg, wu = c["wg"].cuda(), c["wu"].cuda()
    h = dsv_ffn_gated_fwd(x, wg, wu)
    check_fwd(c, h[-last:], "silu")
    assert torch.equal(h[0], h[M - last - 1])   # rows of ones, first and last of them
    del h
    dx, dwg, dwu = dsv_ffn_gated_bwd(dh, x, wg, wu)
    assert dsv_last_device_status() == 0
    check_bwd(c, dx[-last:], dwg, dwu, "silu")
    assert not dx[:M - last].any()


def test_gradients_against_differences():
    """Central differences of the fp64 loss sum(dh * forward) along random directions: what separates them is the
    roundings of the gradient's entries (norm NORM), of random sign against a random direction."""
    need_gpu()
    M, D, F = 96, 72, 136
    c = case(M, D, F, seed=9)
    g = {n: t.cuda() for n, t in c.items()}
    grads = [np64(t) for t in dsv_ffn_gated_bwd(g["dh"], g["x"], g["wg"], g["wu"])]
    x, wg, wu, dh = (np64(c[n]) for n in ("x", "wg", "wu", "dh"))
    loss = lambda *a: float((oracle.ffn_gated_fwd(*a) * dh).sum())
    rng = np.random.default_rng(2)
    for i in range(3):
        e = rng.standard_normal(grads[i].shape)
        lo, hi = [x, wg, wu], [x, wg, wu]
        lo[i], hi[i] = lo[i] - 1e-5 * e, hi[i] + 1e-5 * e
        want = (loss(*hi) - loss(*lo)) / 2e-5
        # a random direction sees an error of norm NORM |grad|: 6 standard deviations
        assert abs(float((grads[i] * e).sum()) - want) <= 6 * NORM * float(np.linalg.norm(grads[i])) + 1e-6 * abs(want)


def test_python_refusals():
    need_gpu()
    c = {n: t.cuda() for n, t in case(16, 64, 128).items()}
    x, wg, wu, dh = c["x"], c["wg"], c["wu"], c["dh"]
    with pytest.raises(ValueError, match="act"):
        dsv_ffn_gated_fwd(x, wg, wu, act="relu")
    with pytest.raises(ValueError, match="x:"):
        dsv_ffn_gated_fwd(x.float(), wg, wu)
    with pytest.raises(ValueError, match="x:"):
        dsv_ffn_gated_fwd(x.t(), wg, wu)
    with pytest.raises(ValueError, match="w_gate"):
        dsv_ffn_gated_fwd(x, wg[:, :32], wu)
    with pytest.raises(ValueError, match="w_up"):
        dsv_ffn_gated_fwd(x, wg, wu[:64])
    with pytest.raises(ValueError, match="out"):
        dsv_ffn_gated_fwd(x, wg, wu, out=torch.empty(16, 64, dtype=BF16, device="cuda"))
    with pytest.raises(DSVError, match="M must"):
        dsv_ffn_gated_fwd(x[:0], wg, wu)
    with pytest.raises(DSVError, match="multiples of 8"):
        dsv_ffn_gated_fwd(torch.zeros(4, 12, dtype=BF16, device="cuda"), torch.zeros(8, 12, dtype=BF16, device="cuda"),
                          torch.zeros(8, 12, dtype=BF16, device="cuda"))
    with pytest.raises(DSVError, match="aligned"):
        dsv_ffn_gated_fwd(torch.zeros(16 * 64 + 4, dtype=BF16, device="cuda")[4:].view(16, 64), wg, wu)
    with pytest.raises(DSVError, match="overlaps"):
        dsv_ffn_gated_bwd(dh, x, wg, wu, out=(x, torch.empty_like(wg), torch.empty_like(wu)))
    with pytest.raises(DSVError, match="workspace"):
        dsv_ffn_gated_bwd(dh, x, wg, wu, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="dh"):
        dsv_ffn_gated_bwd(dh[:, :64], x, wg, wu)
    for bad in ((None, x, wg, wu), (dh, x, wg, None)):
        with pytest.raises(DSVError, match="NULL"):
            dsv_ffn_gated_bwd(*bad)
    for bad in ((None, wg, wu), (x, None, wu)):
        with pytest.raises(TypeError):
            dsv_ffn_gated_fwd(*bad)
