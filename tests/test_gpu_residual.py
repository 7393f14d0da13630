"""GPU parity of the gated residual and its norms against the fp64 oracle.

Tolerances, from the arithmetic, for every element.  u = 2^-24 is fp32's rounding, `step` the output's (2^-8 for bf16,
2^-24 for fp32).  A sum over D adds at most 16 terms in a lane (each with a product before it), then 5 shuffles, then at most
16 warps: it is off by at most G = 40 u times its terms' magnitudes.
  rz, rstd: a mean square is off by G (its terms are positive), its root by half of that, and 2 u.
  r:  dr = |alpha gate t| (G / 2 + 8 u) + u |r|, and step |r|.
  xhat = c rstd, c = r - mean:  dc = dr + 2 u |r| + G mean|r| + mean dr;  rstd is off by rho = mean(|c| dc) / (var + eps) + G.
  y:  |f| rstd (dc + |c| rho) + 8 u (|xhat f| + |shift| + |y|) + step |y|.
Backward, with r given: dc = 2 u |r| + G mean|r|;  dx = rstd dc + |xhat| (rho + 2 u)  (of xhat);  h = dy f is off by 3 u;
  mean h: (G + 4 u) mean|h|;  m = mean(h xhat): mean(|h| dx) + (G + rho + 8 u) mean|h xhat|;
  g: dg = rstd (3 u |h| + dmean + dx |m| + |xhat| dm + (|h| + |mean h| + |xhat m|) (rho + 8 u)) + 2 u (|dr| + |g|).
  u = c g: du = |c| dg + 8 u |u|;  mean(u zhat): mean(|zhat| du) + 2 G mean|u zhat|;
  dz: rz (du + |zhat| dmean + 2 G (|u| + |zhat mean|)) + step |dz|.
Sums over tokens: the terms' own errors, and (rows + 40) u times their magnitudes, rows = B N.
The norm of a bf16 output's error is held to what roundings of random sign leave: 2^-8 / sqrt 3 of the output's norm.
"""
import numpy as np
import pytest
import torch

import oracle
from dynamic_sparse_attention_estimate_gb300 import (DSVError, dsv_adaln_fwd, dsv_residual_norm_bwd,
                                                     dsv_residual_norm_bwd_workspace, dsv_residual_norm_fwd)
from dynamic_sparse_attention_estimate_gb300.binding import dsv_last_device_status
from tests.gpu_helpers import need_gpu, np64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
G = 40 * U
EPS = 1e-6


def case(B, N, D, f32=False, seed=0):
    gen = torch.Generator().manual_seed(seed + 31 * N + D + B)
    r = lambda *s, scale=1.0, dtype=BF16: (torch.randn(*s, generator=gen) * scale).to(dtype)
    stream = F32 if f32 else BF16
    c = dict(x=r(B, N, D, scale=2, dtype=stream), z=r(B, N, D), gate=r(B, D), w_post=(1 + r(D, scale=0.2, dtype=F32)).to(BF16),
             scale=r(B, D, scale=0.5), shift=r(B, D), w_pre=(1 + r(D, scale=0.2, dtype=F32)).to(BF16), dr=r(B, N, D, dtype=stream),
             dy=r(B, N, D))
    c["r"] = r(B, N, D, scale=2, dtype=stream)
    return c


def cut(c, post, pre):
    """(vectors by name, the norms) that a call with these norms takes."""
    v = dict(gate=c["gate"], w_post=c["w_post"] if post == "rms" else None)
    for n in ("scale", "shift", "w_pre"):
        v[n] = c[n] if pre != "none" else None
    return v, dict(post=post, pre=pre, alpha=0.75, eps=EPS)


def check(name, got, ref, bound):
    err = np.abs(np64(got) - ref)
    excess = float((err - bound).max())
    assert excess <= 0, f"{name}: bound exceeded by {excess:.3e}"
    n = float(np.linalg.norm(ref))
    if got.dtype is BF16 and n > 0 and ref.size >= 4096:   # enough values for roundings to average
        rel = float(np.linalg.norm(err)) / n
        assert rel <= 2.0 ** -8 / 3 ** 0.5, f"{name}: rel-L2 {rel:.3e}"


def mean(v):
    return v.mean(-1, keepdims=True)


def step_of(t):
    return 2.0 ** -8 if t.dtype is BF16 else U


def norm_terms(r, dr, pre):
    """(xhat, rstd, the errors of c, of rstd (relative))."""
    c = r - mean(r) if pre == "layer" else r
    dc = dr + 2 * U * np.abs(r) + (G * mean(np.abs(r)) + mean(dr) if pre == "layer" else 0)
    var = mean(c * c) + EPS
    return c / np.sqrt(var), 1 / np.sqrt(var), dc, mean(np.abs(c) * dc) / var + G


def check_fwd(c, got, post, pre):
    v, how = cut(c, post, pre)
    r, y = oracle.residual_norm_fwd(c["x"], c["z"], **v, **how)
    t = np.abs(r - np64(c["x"]))
    dr = t * (G / 2 + 8 * U) + U * np.abs(r)
    check("r", got[0], r, dr + step_of(got[0]) * np.abs(r))
    if pre == "none":
        assert got[1] is None
        return
    xhat, rstd, dc, rho = norm_terms(r, dr, pre)
    f = np.abs((1 + np64(c["scale"])) * np64(c["w_pre"]))[:, None]
    bound = f * (rstd * dc + np.abs(xhat) * rho) + 8 * U * (f * np.abs(xhat) + np.abs(np64(c["shift"]))[:, None] + np.abs(y))
    check("y", got[1], y, bound + 2.0 ** -8 * np.abs(y))


def check_bwd(c, got, post, pre, dr=True):
    v, how = cut(c, post, pre)
    v.pop("shift")
    given = c["dr"] if dr else None
    ref = oracle.residual_norm_bwd(given, c["dy"] if pre != "none" else None, c["r"] if pre != "none" else None, c["z"], **v, **how)
    g, z, gate = ref[0], np64(c["z"]), 0.75 * np64(c["gate"])[:, None]
    rows = (z.shape[0] * z.shape[1] + 40) * U
    dg = 2 * U * ((np.abs(np64(given)) if dr else 0) + np.abs(g))
    if pre != "none":
        dy, f = np64(c["dy"]), ((1 + np64(c["scale"])) * np64(c["w_pre"]))[:, None]
        xhat, rstd, dc, rho = norm_terms(np64(c["r"]), 0 * z, pre)
        dxh, h = rstd * dc + np.abs(xhat) * (rho + 2 * U), dy * f
        mh, m = mean(h) if pre == "layer" else 0 * rstd, mean(h * xhat)
        dmh = (G + 4 * U) * mean(np.abs(h)) if pre == "layer" else 0
        dm = mean(np.abs(h) * dxh) + (G + rho + 8 * U) * mean(np.abs(h * xhat))
        dg = dg + rstd * (3 * U * np.abs(h) + dmh + dxh * np.abs(m) + np.abs(xhat) * dm
                          + (np.abs(h) + np.abs(mh) + np.abs(xhat * m)) * (rho + 8 * U))
        w = np.abs(np64(c["w_pre"]))
        T, dT = np.abs(dy * xhat), np.abs(dy) * dxh
        check("d_scale", got[4], ref[4], w * (dT.sum(1) + (rows + 8 * U) * T.sum(1)))
        check("d_shift", got[5], ref[5], rows * np.abs(dy).sum(1))
        check("dw_pre", got[6], ref[6], (np.abs(1 + np64(c["scale"]))[:, None] * (dT + (rows + 8 * U) * T)).sum((0, 1)))
    else:
        assert got[4] is None and got[5] is None and got[6] is None
    check("dx", got[0], g, dg + step_of(got[0]) * np.abs(g))
    if post == "rms":
        w = np64(c["w_post"])
        rz = 1 / np.sqrt(mean(z * z) + EPS)
        zhat, cw = z * rz, gate * w
        u = cw * g
        du = np.abs(cw) * dg + 8 * U * np.abs(u)
        dmean = mean(np.abs(zhat) * du) + 2 * G * mean(np.abs(u * zhat))
        bound = rz * (du + np.abs(zhat) * dmean + 2 * G * (np.abs(u) + np.abs(zhat * mean(u * zhat))))
        check("dz", got[1], ref[1], bound + 2.0 ** -8 * np.abs(ref[1]))
        S, dS = np.abs(g * zhat), np.abs(zhat) * dg
        check("dw_post", got[3], ref[3], (np.abs(gate) * (dS + (rows + G) * S)).sum((0, 1)))
    else:
        assert got[3] is None
        check("dz", got[1], ref[1], np.abs(gate) * dg + (8 * U + 2.0 ** -8) * np.abs(ref[1]))
        S, dS, w = np.abs(g * z), np.abs(z) * dg, 1.0
    check("d_gate", got[2], ref[2], 0.75 * np.abs(w) * (dS + (rows + G) * S).sum(1))


def fwd(c, post, pre, **extra):
    v, how = cut(c, post, pre)
    return dsv_residual_norm_fwd(c["x"], c["z"], **v, **how, **extra)


def bwd(c, post, pre, dr=True, **extra):
    v, how = cut(c, post, pre)
    v.pop("shift")
    some = pre != "none"
    return dsv_residual_norm_bwd(c["dr"] if dr else None, c["dy"] if some else None, c["r"] if some else None, c["z"], **v, **how,
                                 **extra)


def on_gpu(c):
    return {n: t.cuda() for n, t in c.items()}


NORMS = [(post, pre) for post in ("none", "rms") for pre in ("none", "layer", "rms")]
# one token and a few, one vector of features, rows of one to sixteen warps and either side of each, samples more than
# CTAs, several rows in turn to a group of a CTA
SHAPES = [(1, 1, 8), (2, 3, 24), (1, 5, 256), (3, 37, 264), (2, 77, 1024), (1, 130, 1160), (2, 9, 2048), (1, 19, 4096), (1, 7, 4104),
          (2, 5, 8192), (1, 3000, 64), (200, 2, 128), (3, 301, 768), (1, 4, 1536), (2, 40, 5128),
          (1, 3500, 1032), (2, 900, 4104)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("B,N,D", SHAPES)
def test_both_directions_match_the_oracle(B, N, D, f32):
    need_gpu()
    c = case(B, N, D, f32)
    g = on_gpu(c)
    for post, pre in NORMS:
        check_fwd(c, fwd(g, post, pre), post, pre)
        check_bwd(c, bwd(g, post, pre), post, pre)
    check_bwd(c, bwd(g, "rms", "layer", dr=False), "rms", "layer", dr=False)
    assert dsv_last_device_status() == 0


# samples that share a CTA of the vectors' sums with one to eight warps each, and that take the SMs several times over
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("B,N,D", [(80, 400, 264), (17, 130, 520), (6, 700, 128), (5, 2000, 40), (153, 3, 776), (2, 1300, 96)])
def test_many_samples(B, N, D, f32):
    need_gpu()
    c = case(B, N, D, f32)
    g = on_gpu(c)
    for post, pre in (("rms", "layer"), ("none", "none")):
        check_fwd(c, fwd(g, post, pre), post, pre)
        check_bwd(c, bwd(g, post, pre), post, pre)
    # without the weights there is no last kernel
    c["w_pre"] = torch.ones_like(c["w_pre"])
    g["w_pre"] = c["w_pre"].cuda()
    with_w = bwd(g, "none", "rms")
    without = dsv_residual_norm_bwd(g["dr"], g["dy"], g["r"], g["z"], gate=g["gate"], scale=g["scale"], **cut(g, "none", "rms")[1])
    assert without[6] is None and torch.equal(with_w[0], without[0]) and torch.equal(with_w[1], without[1])
    check_bwd(c, with_w, "none", "rms")
    check_bwd(c, (*without[:6], with_w[6]), "none", "rms")


@pytest.mark.parametrize("f32", [False, True])
def test_vectors_that_are_not_there(f32):
    need_gpu()
    c = case(2, 33, 200, f32)
    g = on_gpu(c)
    for n in ("gate", "w_post", "w_pre"):
        c[n] = torch.ones_like(c[n])
    for n in ("scale", "shift"):
        c[n] = torch.zeros_like(c[n])
    for post in ("none", "rms"):
        for pre in ("layer", "rms"):
            how = dict(post=post, pre=pre, alpha=0.75, eps=EPS)
            check_fwd(c, dsv_residual_norm_fwd(g["x"], g["z"], **how), post, pre)
            got = dsv_residual_norm_bwd(g["dr"], g["dy"], g["r"], g["z"], **how)
            assert got[2] is None and got[3] is None and got[4] is None and got[6] is None
            full = bwd(on_gpu(c), post, pre)
            for i in (0, 1, 5):
                assert torch.equal(got[i], full[i])
            check_bwd(c, full, post, pre)


def test_parts_of_one_projection_and_of_one_gradient():
    """gate, shift, scale are parts of [B, 6, D]; their gradients go into parts of another, and nothing else of it changes."""
    need_gpu()
    B, N, D = 3, 50, 264
    c = case(B, N, D)
    g = on_gpu(c)
    mod = torch.full((B, 6, D), float("nan"), dtype=BF16, device="cuda")
    for i, n in ((2, "gate"), (3, "shift"), (4, "scale")):
        mod[:, i] = g[n]
        g[n] = mod[:, i]
    check_fwd(c, fwd(g, "rms", "layer"), "rms", "layer")
    d_mod = torch.full((B, 6, D), -7.0, device="cuda")
    parts = (d_mod[:, 2], d_mod[:, 4], d_mod[:, 3])
    got = bwd(g, "rms", "layer", d_mod=parts)
    check_bwd(c, got, "rms", "layer")
    assert got[2].data_ptr() == parts[0].data_ptr()
    assert (d_mod[:, [0, 1, 5]] == -7).all()
    # the sums that are not asked for
    again = bwd(g, "rms", "layer", d_mod=(None, d_mod[:, 0], None))
    assert again[2] is None and again[5] is None and torch.equal(again[4], got[4]) and torch.equal(again[0], got[0])


def test_one_row_for_all_samples():
    """Broadcast gate, scale and shift (stride 0) give what the rows written out give; each sample has its own gradient."""
    need_gpu()
    c = case(4, 21, 136)
    for n in ("gate", "scale", "shift"):
        c[n] = c[n][:1].expand(4, 136).contiguous()
    g = on_gpu(c)
    flat = fwd(g, "rms", "rms"), bwd(g, "rms", "rms")
    check_bwd(c, flat[1], "rms", "rms")
    for n in ("gate", "scale", "shift"):
        g[n] = g[n][:1].expand(4, 136)
    for a, b in zip(flat, (fwd(g, "rms", "rms"), bwd(g, "rms", "rms"))):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("D", [136, 2048, 5128])
def test_in_place(D, f32):
    need_gpu()
    g = on_gpu(case(2, 45, D, f32))
    r, y = fwd(g, "rms", "layer")
    x = g["x"].clone()
    y2 = torch.empty_like(y)
    got = fwd({**g, "x": x}, "rms", "layer", out=(x, y2))
    assert got[0] is x and torch.equal(x, r) and torch.equal(y2, y)
    want = bwd(g, "rms", "layer")
    dr, dz = g["dr"].clone(), torch.empty_like(g["z"])
    got = bwd({**g, "dr": dr}, "rms", "layer", out=(dr, dz))
    assert got[0] is dr and all(torch.equal(a, b) for a, b in zip(got, want))


def test_alpha_and_eps_that_are_tensors_are_read_in_every_call():
    need_gpu()
    g = on_gpu(case(1, 9, 64))
    alpha, eps = torch.tensor(0.5), torch.tensor(1e-3)
    for a, e in ((0.5, 1e-3), (2.0, 1e-3), (2.0, 10.0)):
        alpha.fill_(a)
        eps.fill_(e)
        got = dsv_residual_norm_fwd(g["x"], g["z"], g["gate"], alpha=alpha, eps=eps)
        want = dsv_residual_norm_fwd(g["x"], g["z"], g["gate"], alpha=a, eps=float(torch.tensor(e)))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def guarded(shape, dtype, pad=4096):
    numel = int(np.prod(shape))
    buf = torch.full((numel + 2 * pad,), -77.0, device="cuda").to(dtype)
    return buf[pad:pad + numel].view(shape), buf, pad


@pytest.mark.parametrize("B,N,D", [(1, 1, 8), (3, 37, 264), (2, 5, 8192), (200, 2, 128)])
def test_nothing_around_the_outputs_is_written(B, N, D):
    need_gpu()
    c = case(B, N, D)
    g = on_gpu(c)
    full, vec = (B, N, D), (B, D)
    nbytes = dsv_residual_norm_bwd_workspace(B, N, D)
    outs = [guarded(full, BF16) for _ in range(4)] + [guarded(vec, F32) for _ in range(3)]
    ws = guarded((nbytes // 4,), F32)
    ws[0].fill_(float("nan"))
    fwd(g, "rms", "layer", out=(outs[0][0], outs[1][0]))
    got = bwd(g, "rms", "layer", out=(outs[2][0], outs[3][0]), d_mod=tuple(o[0] for o in outs[4:]), workspace=ws[0])
    torch.cuda.synchronize()
    for view, buf, pad in outs + [ws]:
        assert (buf[:pad] == -77).all() and (buf[pad + view.numel():] == -77).all()
    check_fwd(c, (outs[0][0], outs[1][0]), "rms", "layer")
    check_bwd(c, got, "rms", "layer")


@pytest.mark.parametrize("pre", ["layer", "rms"])
def test_a_bad_token_stays_in_its_row(pre):
    need_gpu()
    g = on_gpu(case(2, 40, 264))
    clean, dclean = fwd(g, "rms", pre), bwd(g, "rms", pre)
    keep = torch.ones(2, 40, dtype=torch.bool, device="cuda")
    for n, (i, v) in {"z": (3, float("inf")), "x": (4, float("nan")), "r": (5, float("inf")), "dr": (6, float("nan"))}.items():
        g[n][1, i, 7] = v
        keep[1, i] = False
    got, dgot = fwd(g, "rms", pre), bwd(g, "rms", pre)
    for i in range(2):
        assert torch.equal(got[i][keep], clean[i][keep]) and torch.equal(dgot[i][keep], dclean[i][keep])
    for i in (2, 4, 5):                       # the other sample's sums
        assert torch.equal(dgot[i][0], dclean[i][0])
    assert torch.isnan(got[1][1, 4]).all() and torch.isnan(got[1][1, 3]).any()


def test_rows_that_are_constant_or_zero():
    need_gpu()
    c = case(1, 6, 520, f32=True)
    c["z"][0, 2] = 0
    c["x"][0, 2] = 3.5
    g = on_gpu(c)
    r, y = fwd(g, "rms", "layer")
    assert (r[0, 2] == 3.5).all() and torch.equal(y[0, 2], g["shift"][0])
    # with eps = 0 a row of zeros is NaN behind its norm, in that row alone
    v, how = cut(g, "rms", "layer")
    r0, y0 = dsv_residual_norm_fwd(g["x"], g["z"], **v, **{**how, "eps": 0.0})
    bad = torch.isnan(r0).any(-1)[0]
    assert bad.tolist() == [i == 2 for i in range(6)] and torch.isnan(y0).any(-1)[0].tolist() == bad.tolist()


def test_a_stream_far_from_zero():
    """A mean 10^4 times the spread: the deviations are taken from the mean before they are squared."""
    need_gpu()
    c = case(1, 30, 1160, f32=True)
    for n in ("x", "r"):
        c[n] = c[n] + 2e4
    g = on_gpu(c)
    check_fwd(c, fwd(g, "none", "layer"), "none", "layer")
    check_bwd(c, bwd(g, "none", "layer"), "none", "layer")


@pytest.mark.parametrize("post,pre", [("none", "layer"), ("rms", "layer"), ("rms", "rms")])
def test_gradients_match_differences(post, pre):
    """The forward's own central differences along one direction of every input.  y's roundings (uniform, of standard
    deviation 2^-8 |y| / sqrt 12 at most) leave sqrt(sum (dy 2^-8 y)^2 / 12) in each of the two losses; six of those over the step,
    and how far the oracle's difference of this step is from its slope, bound the distance."""
    need_gpu()
    B, N, D = 2, 60, 520
    c = case(B, N, D, f32=True)
    v, how = cut(c, post, pre)
    step, gen = 0.125, torch.Generator().manual_seed(9)
    r, _ = dsv_residual_norm_fwd(c["x"].cuda(), c["z"].cuda(), **{n: t if t is None else t.cuda() for n, t in v.items()}, **how)
    back = {n: t for n, t in v.items() if n != "shift"}
    grads = dsv_residual_norm_bwd(c["dr"].cuda(), c["dy"].cuda(), r, c["z"].cuda(),
                                  **{n: t if t is None else t.cuda() for n, t in back.items()}, **how)
    dr, dy = np64(c["dr"]), np64(c["dy"])
    names = ("x", "z", "gate", "w_post", "scale", "shift", "w_pre")
    for i, n in enumerate(names):
        if grads[i] is None:
            continue
        base = c[n]
        e = (torch.randn(base.shape, generator=gen) * 0.25).to(base.dtype)
        lo, hi = ((base.float() + s * step * e.float()).to(base.dtype) for s in (-1, 1))
        moved = (np64(hi) - np64(lo)) / (2 * step)               # the direction that the rounded inputs moved in
        loss, exact, noise = [], [], 0.0
        for t in (lo, hi):
            a = {"x": c["x"], "z": c["z"], **v, n: t}
            r, y = dsv_residual_norm_fwd(**{k: s if s is None else s.cuda() for k, s in a.items()}, **how)
            loss.append(float((np64(r) * dr).sum() + (np64(y) * dy).sum()))
            r, y = oracle.residual_norm_fwd(**a, **how)
            exact.append(float((r * dr).sum() + (y * dy).sum()))
            noise += float(((dy * y * 2.0 ** -8) ** 2).sum() / 12)
        slope = float((np64(grads[i]) * moved).sum())
        true = oracle.residual_norm_bwd(c["dr"], c["dy"], oracle.residual_norm_fwd(c["x"], c["z"], **v, **how)[0], c["z"], **back, **how)
        wanted = float((true[i] * moved).sum())
        bend = abs((exact[1] - exact[0]) / (2 * step) - wanted)
        # the gradient's own roundings: z's is bf16
        own = 6 * float(np.sqrt(((true[i] * moved * 2.0 ** -8) ** 2).sum() / 12)) + 1e-4 * float(np.abs(true[i] * moved).sum() / np.sqrt(moved.size))
        tol = 6 * noise ** 0.5 / (2 * step) + bend + own
        assert abs((loss[1] - loss[0]) / (2 * step) - slope) <= tol, n


def test_without_a_branch_it_is_adaln():
    need_gpu()
    g = on_gpu(case(2, 65, 768))
    y = dsv_residual_norm_fwd(g["x"], torch.zeros_like(g["z"]), g["gate"], None, g["scale"], g["shift"])[1]
    z = dsv_adaln_fwd(g["x"], g["scale"], g["shift"])
    ref = oracle.adaln_fwd(g["x"], g["scale"], g["shift"])
    assert (np.abs(np64(y) - np64(z)) <= 2 * 2.0 ** -8 * np.abs(ref) + 1e-4).all()


@pytest.mark.parametrize("f32", [False, True])
def test_tensors_that_start_inside_an_allocation(f32):
    """16-byte boundaries that are none of 32."""
    need_gpu()
    g = on_gpu(case(2, 30, 392, f32))
    want, dwant = fwd(g, "rms", "layer"), bwd(g, "rms", "layer")

    def moved(t):
        skip = 16 // t.element_size()
        out = torch.empty(t.numel() + skip, dtype=t.dtype, device="cuda")[skip:].view(t.shape)
        assert out.data_ptr() % 32 == 16
        return out

    for n in g:
        g[n] = moved(g[n]).copy_(g[n])
    got = fwd(g, "rms", "layer", out=tuple(moved(t) for t in want))
    dgot = bwd(g, "rms", "layer", out=tuple(moved(t) for t in dwant[:2]), d_mod=tuple(moved(dwant[i]) for i in (2, 4, 5)))
    assert all(torch.equal(a, b) for a, b in zip(got + dgot, want + dwant))


def test_repeats_streams_and_a_replayed_graph():
    need_gpu()
    B, N, D = 2, 600, 776
    g = on_gpu(case(B, N, D))
    first, dfirst = fwd(g, "rms", "layer"), bwd(g, "rms", "layer")
    same = lambda a, b: all(torch.equal(s, t) for s, t in zip(a, b))
    for _ in range(3):
        assert same(fwd(g, "rms", "layer"), first) and same(bwd(g, "rms", "layer"), dfirst)
    streams = [torch.cuda.Stream() for _ in range(2)]
    found = []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(4):
                found.append((fwd(g, "rms", "layer"), bwd(g, "rms", "layer")))
    torch.cuda.synchronize()
    assert all(same(a, first) and same(b, dfirst) for a, b in found)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        a, b = fwd(g, "rms", "layer"), bwd(g, "rms", "layer")
    other = on_gpu(case(B, N, D, seed=5))
    for n in g:
        g[n].copy_(other[n])
    graph.replay()
    torch.cuda.synchronize()
    assert same(a, fwd(other, "rms", "layer")) and same(b, bwd(other, "rms", "layer"))


def test_offsets_past_32_bits():
    """More than 2^31 elements in each tensor: the last rows come out as they do alone."""
    need_gpu()
    N, D, tail = 270000, 8192, 64
    gen = torch.Generator(device="cuda").manual_seed(0)
    full = lambda: torch.empty(1, N, D, dtype=BF16, device="cuda").normal_(generator=gen)
    g = dict(x=full(), z=full(), **{n: torch.randn(1, D, generator=gen, device="cuda").to(BF16) for n in ("gate", "scale", "shift")},
             w_post=torch.ones(D, dtype=BF16, device="cuda"), w_pre=torch.ones(D, dtype=BF16, device="cuda"))
    r, y = fwd(g, "rms", "layer")
    last = {**g, "x": g["x"][:, -tail:].contiguous(), "z": g["z"][:, -tail:].contiguous()}
    rt, yt = fwd(last, "rms", "layer")
    assert torch.equal(r[:, -tail:], rt) and torch.equal(y[:, -tail:], yt)
    g.update(r=r, dr=g.pop("x"), dy=y)
    got = bwd(g, "rms", "layer")
    last.update(r=rt, dr=last["x"], dy=yt)
    want = bwd(last, "rms", "layer")
    assert torch.equal(got[0][:, -tail:], want[0]) and torch.equal(got[1][:, -tail:], want[1])


def test_refusals():
    need_gpu()
    g = on_gpu(case(2, 10, 64))
    for n in ("gate", "scale", "shift", "w_post", "w_pre"):
        for bad in (g[n].float(), g[n][..., :32], g[n].cpu(), g[n].repeat_interleave(2, -1)[..., ::2]):
            with pytest.raises(ValueError, match=n):
                fwd({**g, n: bad}, "rms", "layer")
    for n in ("z", "dr", "dy", "r"):
        with pytest.raises(ValueError):
            bwd({**g, n: g[n][:, :5]}, "rms", "layer")
        with pytest.raises(ValueError):
            bwd({**g, n: g[n].half()}, "rms", "layer")
    with pytest.raises(ValueError, match="contiguous"):
        fwd({**g, "x": g["x"].transpose(0, 1)}, "rms", "layer")
    with pytest.raises(DSVError, match="overlaps"):
        fwd(g, "rms", "layer", out=(torch.empty_like(g["x"]), g["z"]))
    with pytest.raises(DSVError, match="w_post without"):
        dsv_residual_norm_fwd(g["x"], g["z"], g["gate"], g["w_post"])
    with pytest.raises(DSVError, match="y is NULL"):
        fwd(g, "rms", "layer", out=(torch.empty_like(g["x"]), None))
    with pytest.raises(DSVError, match="z is NULL"):
        dsv_residual_norm_fwd(g["x"], None)
    with pytest.raises(DSVError, match="dy is NULL"):
        dsv_residual_norm_bwd(g["dr"], None, g["r"], g["z"])
    with pytest.raises(DSVError, match="D must"):
        dsv_residual_norm_fwd(g["x"][..., :60].contiguous(), g["z"][..., :60].contiguous())
    with pytest.raises(DSVError, match="stride"):
        fwd({**g, "gate": torch.zeros(2, 68, dtype=BF16, device="cuda")[:, :64]}, "rms", "layer")
    with pytest.raises(ValueError, match="one stride"):
        vecs = torch.zeros(2, 6, 64, device="cuda")
        bwd(g, "rms", "layer", d_mod=(vecs[:, 0], vecs[:, 1], torch.zeros(2, 64, device="cuda")))
    with pytest.raises(ValueError, match="post must"):
        dsv_residual_norm_fwd(g["x"], g["z"], post="layer")
    assert dsv_last_device_status() == 0


def far_terms(r):
    """(xhat, rstd, the errors of c = r - mean r, of rstd (relative)) of a layer norm of fp32 rows r, however far from 0 they lie.  The
    rounded mean is off by at most far = G mean|r|; the deviations d from it, |d| <= |c| + far, are off by u |d|, their own mean, which
    is taken off them, by G mean|d|:  dc = G (mean|c| + far) + 3 u (|c| + far).  mean d^2 is off by (G + 2 u) (var + far^2) and the
    square of d's mean by 2 far G (mean|c| + far) + 2 u far^2, so that rho = (twice G (var + far^2) + 2 far G (mean|c| + far)) /
    (var + eps) + G covers rstd, which has half of it."""
    c = r - mean(r)
    far, var = G * mean(np.abs(r)), mean(c * c)
    dc = G * (mean(np.abs(c)) + far) + 3 * U * (np.abs(c) + far)
    rho = (2 * G * (var + far * far) + 2 * far * G * (mean(np.abs(c)) + far)) / (var + EPS) + G
    return c / np.sqrt(var + EPS), 1 / np.sqrt(var + EPS), dc, rho


# sums of D equal numbers that are not exact; with a spread of a few last bits; a bf16 stream whose new rows lie between its numbers
@pytest.mark.parametrize("far,spread", [(0.1, 0.0), (10.1, 0.0), (1000.1, 0.0), (10.1, 1e-5), (1000.1, 1e-3), (-30000.7, 1e-2)])
@pytest.mark.parametrize("D", [8, 520, 768, 1160, 1536, 5128, 7000])
def test_rows_far_from_zero_with_little_spread(D, far, spread):
    need_gpu()
    B, N = 2, 9
    c = case(B, N, D, f32=True)
    c["x"] = (far + spread * c["x"].double()).float()
    c["r"], c["z"] = c["x"], torch.zeros_like(c["z"])
    xhat, rstd, dc, rho = far_terms(np64(c["x"]))
    w, f = np.abs(np64(c["w_pre"])), ((1 + np64(c["scale"])) * np64(c["w_pre"]))[:, None]
    dxh = rstd * dc + np.abs(xhat) * (rho + 2 * U)
    for shift in (c["shift"], torch.zeros_like(c["shift"])):       # without it the smallest xhat shows
        c["shift"] = shift
        v, how = cut(c, "none", "layer")
        y = oracle.residual_norm_fwd(c["x"], c["z"], **v, **how)[1]
        got = fwd(on_gpu(c), "none", "layer")
        assert torch.equal(got[0].cpu(), c["x"])
        check("y", got[1], y, np.abs(f) * dxh + 8 * U * (np.abs(f * xhat) + np.abs(np64(shift))[:, None] + np.abs(y)) + 2.0 ** -8 * np.abs(y))
    v.pop("shift")
    ref, got = oracle.residual_norm_bwd(c["dr"], c["dy"], c["r"], c["z"], **v, **how), bwd(on_gpu(c), "none", "layer")
    dy = np64(c["dy"])
    h = dy * f
    mh, m = mean(h), mean(h * xhat)
    # sum h (r - mean) is sum h d less the mean of d times sum h: each is off by as much as dc
    dmh, dm = (G + 4 * U) * mean(np.abs(h)), 2 * mean(np.abs(h) * dxh) + (G + rho + 8 * U) * mean(np.abs(h * xhat))
    dg = rstd * (3 * U * np.abs(h) + dmh + dxh * np.abs(m) + np.abs(xhat) * dm + (np.abs(h) + np.abs(mh) + np.abs(xhat * m)) * (rho + 8 * U))
    check("dx", got[0], ref[0], dg + 3 * U * (np.abs(np64(c["dr"])) + np.abs(ref[0])))
    T, dT, rows = np.abs(dy * xhat), np.abs(dy) * dxh, (N + 40) * U
    check("d_scale", got[4], ref[4], w * (dT.sum(1) + (rows + 8 * U) * T.sum(1)))
    check("dw_pre", got[6], ref[6], (np.abs(1 + np64(c["scale"]))[:, None] * (dT + (B * rows + 8 * U) * T)).sum((0, 1)))


@pytest.mark.parametrize("D", [520, 768, 5128])
def test_constant_rows_between_the_streams_numbers(D):
    """A bf16 stream of 1000 and a branch of 0.1: the new rows, whose norm is taken before their rounding, are constant in fp32."""
    need_gpu()
    c = case(1, 5, D)
    c["x"], c["z"], c["gate"] = torch.full_like(c["x"], 1000.0), torch.full_like(c["z"], 0.1), torch.ones_like(c["gate"])
    c["shift"] = torch.zeros_like(c["shift"])
    y = np64(fwd(on_gpu(c), "none", "layer")[1])
    f = np.abs((1 + np64(c["scale"])) * np64(c["w_pre"]))[:, None]
    # r is 1000 and alpha gate z, rounded once: the same number in every feature
    xhat, rstd, dc, rho = far_terms(np.full((1, 1, 1), 1000.0 + 0.75 * float(c["z"][0, 0, 0])))
    assert (np.abs(y) <= f * rstd * dc * (1 + 2.0 ** -8) * (1 + 8 * U)).all()


@pytest.mark.parametrize("far", [1000.0, 0.1, -30000.0])
@pytest.mark.parametrize("D", [8, 520, 1160, 8192])
def test_the_gradient_of_constant_rows_of_a_bf16_stream(D, far):
    """Up to 8192 equal numbers of eight bits add up exactly in 24: xhat is 0, and with it d_scale and dw_pre, and the gradient
    is dr + rstd (h - mean h), with rstd = eps^-1/2."""
    need_gpu()
    c = case(2, 7, D)
    c["r"] = torch.full_like(c["r"], far)
    got = bwd(on_gpu(c), "none", "layer")
    assert not got[4].any() and not got[6].any()
    h, dr = np64(c["dy"]) * ((1 + np64(c["scale"])) * np64(c["w_pre"]))[:, None], np64(c["dr"])
    rstd, want = EPS ** -0.5, np64(c["dr"]) + (h - mean(h)) * EPS ** -0.5
    bound = rstd * (3 * U * np.abs(h) + (G + 4 * U) * mean(np.abs(h)) + 16 * U * (np.abs(h) + np.abs(mean(h)))) + 2 * U * (np.abs(dr) + np.abs(want))
    check("dx", got[0], want, bound + 2.0 ** -8 * np.abs(want))


@pytest.mark.parametrize("N,D,norms", [(470, 6152, NORMS), (780, 8192, [("rms", "layer"), ("none", "rms")])])
def test_long_rows_of_an_fp32_stream_in_turn(N, D, norms):
    """Rows of 13 to 16 warps: a CTA has one at a time and three to six in turn, so that both stages are filled again and the vectors'
    sums are of several rows."""
    need_gpu()
    c = case(1, N, D, f32=True)
    g = on_gpu(c)
    for post, pre in norms:
        check_fwd(c, fwd(g, post, pre), post, pre)
        check_bwd(c, bwd(g, post, pre), post, pre)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("B,N,D", [(80, 400, 264), (6, 700, 128), (5, 2000, 40), (1, 3500, 1032), (3, 900, 2048)])
def test_vectors_gradients_by_their_own_rows(B, N, D, f32):
    """d_gate, d_scale and d_shift are sums over the N rows of a sample: (N + 40) roundings, whatever B is.  And by their norm: N random
    additions leave u sqrt(N / 6) times the root of the terms' squares, the terms' own errors, up to G = 40 u of each and another in
    every row, G times it."""
    need_gpu()
    c = case(B, N, D, f32)
    v, how = cut(c, "rms", "layer")
    v.pop("shift")
    got = bwd(on_gpu(c), "rms", "layer")
    ref = oracle.residual_norm_bwd(c["dr"], c["dy"], c["r"], c["z"], **v, **how)
    dy, z, w = np64(c["dy"]), np64(c["z"]), np.abs(np64(c["w_pre"]))
    xhat, rstd, dc, rho = norm_terms(np64(c["r"]), 0 * z, "layer")
    T, dT = dy * xhat, np.abs(dy) * (rstd * dc + np.abs(xhat) * (rho + 2 * U))
    S = ref[0] * z / np.sqrt(mean(z * z) + EPS)
    u, rows = 0.75 * np.abs(np64(c["w_post"])), (N + 40) * U
    check("d_scale", got[4], ref[4], w * (dT.sum(1) + (rows + 8 * U) * np.abs(T).sum(1)))
    check("d_shift", got[5], ref[5], rows * np.abs(dy).sum(1))
    for name, i, terms in (("d_gate", 2, u * S), ("d_scale", 4, w * T), ("d_shift", 5, dy)):
        err, size = np64(got[i]) - ref[i], np.sqrt((terms * terms).sum(1))
        rel = float(np.linalg.norm(err) / np.linalg.norm(size))
        assert rel <= (N / 6) ** 0.5 * U + G, f"{name}: {rel:.3e}"


@pytest.mark.parametrize("post,pre", [("none", "layer"), ("rms", "layer"), ("none", "rms")])
@pytest.mark.parametrize("D", [264, 2048])
def test_the_gradient_of_the_forwards_own_bf16_stream(D, post, pre):
    """y is the norm of r before its rounding, and the backward takes r as it was stored: against the gradient at the r before its
    rounding it is off by what 2^-8 |r| does to the row's norm (to first order; the second, of the size of rho, four times in front)."""
    need_gpu()
    c = case(2, 70, D)
    g = on_gpu(c)
    v, how = cut(c, post, pre)
    r = oracle.residual_norm_fwd(c["x"], c["z"], **v, **how)[0]
    v.pop("shift")
    g["r"] = fwd(g, post, pre)[0]
    got, ref = bwd(g, post, pre), oracle.residual_norm_bwd(c["dr"], c["dy"], r, c["z"], **v, **how)
    dy, f, w = np64(c["dy"]), ((1 + np64(c["scale"])) * np64(c["w_pre"]))[:, None], np.abs(np64(c["w_pre"]))
    # the stored r: half a step, of a number that fp32 has rounded before
    xhat, rstd, dc, rho = norm_terms(r, 2.0 ** -8 * np.abs(r) + G * np.abs(r - np64(c["x"])) + 8 * U * np.abs(r), pre)
    dxh, h, room = rstd * dc + np.abs(xhat) * (rho + 2 * U), dy * f, 1 + 4 * float(rho.max())
    mh, m = mean(h) if pre == "layer" else 0 * rstd, mean(h * xhat)
    dmh = (G + 4 * U) * mean(np.abs(h)) if pre == "layer" else 0
    dm = mean(np.abs(h) * dxh) + (G + rho + 8 * U) * mean(np.abs(h * xhat))
    dg = rstd * (3 * U * np.abs(h) + dmh + dxh * np.abs(m) + np.abs(xhat) * dm + (np.abs(h) + np.abs(mh) + np.abs(xhat * m)) * (rho + 8 * U))
    check("dx", got[0], ref[0], room * dg + 2 * U * np.abs(np64(c["dr"])) + (2.0 ** -8 + 2 * U) * (np.abs(ref[0]) + room * dg))
    T, dT, rows = np.abs(dy * xhat), np.abs(dy) * dxh, (70 + 40) * U
    check("d_scale", got[4], ref[4], w * (room * dT.sum(1) + (rows + 8 * U) * (T + dT).sum(1)))
