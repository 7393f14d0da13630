"""GPU parity of the rotary and qk-norm kernels against the fp64 oracle.

Tolerances, from the arithmetic.  A bf16 output is one rounding of an fp32 result: at most 2^-8 of the
value (half a step).  The fp32 result itself is a handful of products and sums, each off by 2^-24 of its
operands, on table entries rounded to fp32: together below 2^-20 of the magnitudes of the terms that make
up the value.  So per element |got - ref| <= 2^-8 |ref| + 2^-19 mag (2^-19: the same bound again for the
rounding's own argument).  A weight's gradient is an fp32 sum: a chain of at most 128 additions (a
token's heads, a CTA's tokens, the CTAs) on terms within 2^-20, so |got - ref| <= 2^-16 sum |term|.
"""
import numpy as np
import pytest
import torch

import oracle
from dynamic_sparse_attention_estimate_gb300 import (DSVError, RopeTable, dsv_qk_norm_rope_bwd,
                                                     dsv_qk_norm_rope_bwd_workspace, dsv_qk_norm_rope_fwd,
                                                     dsv_rope3d_bwd, dsv_rope3d_fwd, dsv_rope3d_table)
from dynamic_sparse_attention_estimate_gb300.binding import dsv_last_device_status
from dynamic_sparse_attention_estimate_gb300.inputs import token_positions
from tests.gpu_helpers import need_gpu, np64

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(BF16)


def close(name, got, ref, mag):
    excess = np.abs(np64(got) - ref) - (2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * mag)
    assert float(excess.max()) <= 0, f"{name}: bound exceeded by {excess.max():.3e}"


def rope_mag(x, ang, pairing):
    """|x0| + |x1| for each rotated feature, |x| for the others."""
    m = np.abs(np64(x) if isinstance(x, torch.Tensor) else x).copy()
    f, g = oracle.pair_features(2 * ang.shape[-1], pairing)
    both = m[..., f] + m[..., g]
    m[..., f] = both
    m[..., g] = both
    return m


def laid_out(t, layout):
    """t [B, H, N, d] in this memory layout, as a [B, H, N, d] view on the GPU."""
    B, H, N, d = t.shape
    if layout == "heads":                                          # contiguous [B][H][N][d]
        return t.cuda()
    if layout == "tokens":                                         # [B][N][H][d]
        return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    if layout == "packed":                                         # the middle of [B][N][3][H][d]
        p = torch.full((B, N, 3, H, d), float("nan"), dtype=t.dtype)
        p[:, :, 1] = t.transpose(1, 2)
        return p.cuda()[:, :, 1].transpose(1, 2)
    assert layout == "padded"                                      # rows of d + 24, tokens past the last one
    p = torch.full((H, B, N + 3, d + 24), float("nan"), dtype=t.dtype)
    p[:, :, :N, 8:8 + d] = t.transpose(0, 1)
    return p.cuda()[:, :, :N, 8:8 + d].transpose(0, 1)


LAYOUTS = ("heads", "tokens", "packed", "padded")

# (B, H, (T, Y, X), d, axes, pairing, layout): one token, odd counts around a CTA's 8 or 16 tokens, one
# head and more heads than a group loads ahead, unused axes, features that pass, a pair count
# that ends inside a vector
SHAPES = [
    (1, 1, (1, 1, 1), 64, (24, 20, 20), "interleaved", "heads"),
    (1, 1, (1, 1, 1), 128, (44, 42, 42), "halves", "packed"),
    (2, 5, (3, 5, 7), 64, (24, 20, 20), "interleaved", "packed"),
    (2, 5, (3, 5, 7), 64, (24, 20, 20), "halves", "packed"),
    (3, 2, (2, 3, 3), 128, (44, 42, 42), "interleaved", "tokens"),
    (1, 25, (1, 9, 15), 128, (44, 42, 42), "halves", "tokens"),
    (2, 3, (1, 1, 17), 64, (0, 0, 64), "interleaved", "padded"),
    (1, 4, (33, 1, 1), 64, (16, 0, 0), "halves", "heads"),
    (1, 7, (2, 4, 4), 128, (6, 4, 2), "interleaved", "padded"),
    (2, 2, (4, 4, 4), 128, (10, 14, 8), "halves", "padded"),
    (1, 3, (1, 16, 8), 64, (0, 32, 32), "interleaved", "heads"),
    (1, 2, (4, 16, 16), 64, (24, 20, 20), "interleaved", "heads"),
]


def positions(latent):
    return token_positions(latent, None)


@pytest.mark.parametrize("B,H,latent,d,axes,pairing,layout", SHAPES)
@pytest.mark.parametrize("backward", [False, True], ids=["fwd", "bwd"])
def test_rope3d_matches_oracle(B, H, latent, d, axes, pairing, layout, backward):
    need_gpu()
    gen = torch.Generator().manual_seed(H * 100 + d)
    N = int(np.prod(latent))
    x = normal(gen, B, H, N, d)
    rope = dsv_rope3d_table(axes, latent, pairing=pairing)
    pos = positions(latent)
    f = dsv_rope3d_bwd if backward else dsv_rope3d_fwd
    y = f(laid_out(x, layout), pos.cuda(), rope)
    assert y.is_contiguous() and dsv_last_device_status() == 0
    ang = oracle.rope_angles(pos, axes)
    close("y", y, oracle.rope(x, ang, pairing, backward), rope_mag(x, ang, pairing))
    # features past the rotated ones are copies
    R = sum(axes)
    assert torch.equal(y[..., R:].cpu(), x[..., R:])


@pytest.mark.parametrize("layout", LAYOUTS)
def test_rope3d_output_layouts_and_what_lies_around_them(layout):
    need_gpu()
    gen = torch.Generator().manual_seed(7)
    B, H, latent, d, axes = 2, 3, (3, 5, 3), 64, (24, 20, 20)
    x = normal(gen, B, H, 45, d).cuda()
    rope, pos = dsv_rope3d_table(axes, latent), positions(latent).cuda()
    want = dsv_rope3d_fwd(x, pos, rope)
    out = laid_out(torch.zeros(B, H, 45, d, dtype=BF16), layout)
    base = out._base if out._base is not None else out
    before = base.clone()
    got = dsv_rope3d_fwd(x, pos, rope, out=out)
    assert got is out and torch.equal(out, want)
    out.zero_()                     # everything but the view's own elements is as it was
    assert torch.equal(base.view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_rope3d_in_place(layout, pairing):
    need_gpu()
    gen = torch.Generator().manual_seed(8)
    latent, axes = (3, 5, 3), (24, 20, 20)
    x = laid_out(normal(gen, 2, 3, 45, 64), layout)
    rope, pos = dsv_rope3d_table(axes, latent, pairing=pairing), positions(latent).cuda()
    want = dsv_rope3d_fwd(x, pos, rope)
    assert dsv_rope3d_fwd(x, pos, rope, out=x) is x
    assert torch.equal(x, want)


def test_rope3d_broadcast_input_and_batched_positions():
    need_gpu()
    gen = torch.Generator().manual_seed(9)
    B, H, latent, d, axes = 3, 4, (2, 3, 5), 128, (44, 42, 42)
    one = normal(gen, 1, 1, 30, d)
    pos = torch.stack([torch.randint(0, 5, (30, 3), generator=gen) for _ in range(B)]).to(torch.int32)
    rope = dsv_rope3d_table(axes, (5, 5, 5))
    y = dsv_rope3d_fwd(one.cuda().expand(B, H, 30, d), pos.cuda(), rope)
    ang = oracle.rope_angles(pos, axes)
    x = one.expand(B, H, 30, d)
    close("y", y, oracle.rope(x, ang), rope_mag(x, ang[:, None], "interleaved"))


def test_table_keeps_far_phases():
    """Entries are single roundings of fp64 values, at positions whose fp32 angles would be lost."""
    need_gpu()
    axes, lengths, theta = (8, 0, 6), (3, 5, 200001), (1e4, 1.0, 500.0)
    rope = dsv_rope3d_table(axes, lengths, theta)
    got = np64(rope.data)
    want = []
    for a in range(3):
        ang = oracle.rope_angles(np.arange(lengths[a])[:, None] * np.eye(3)[a], [axes[i] if i == a else 0 for i in range(3)], theta)
        want.append(np.stack([np.cos(ang), np.sin(ang)], -1).reshape(-1))
    want = np.concatenate(want)
    # half an fp32 step of the value, and the fp64 angle's own error (2^-52 of up to 200,000)
    assert got.shape == want.shape
    assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -32).all()


def test_a_caller_made_table():
    """Scaled positions: the table is the caller's to fill."""
    need_gpu()
    gen = torch.Generator().manual_seed(10)
    latent, axes = (2, 2, 4), (24, 20, 20)
    x, pos = normal(gen, 1, 2, 16, 64), positions(latent)
    ang = oracle.rope_angles(pos.numpy() * 0.5, axes)
    parts = []
    for a in range(3):
        t = oracle.rope_angles(0.5 * np.arange(latent[a])[:, None] * np.eye(3)[a], [axes[i] if i == a else 0 for i in range(3)])
        parts.append(np.stack([np.cos(t), np.sin(t)], -1).reshape(-1))
    rope = RopeTable(torch.from_numpy(np.concatenate(parts)).float().cuda(), axes, latent)
    close("y", dsv_rope3d_fwd(x.cuda(), pos.cuda(), rope), oracle.rope(x, ang), rope_mag(x, ang, "interleaved"))


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
def test_positions_outside_the_table_turn_nothing_and_are_reported(pairing):
    need_gpu()
    gen = torch.Generator().manual_seed(11)
    latent, axes = (2, 3, 5), (24, 20, 20)
    x, pos = normal(gen, 1, 2, 30, 64), positions(latent)
    bad = pos.clone()
    bad[3, 0], bad[7, 1], bad[11, 2], bad[29] = -1, 3, 2 ** 31 - 1, -2 ** 31
    rope = dsv_rope3d_table(axes, latent, pairing=pairing)
    assert dsv_last_device_status() == 0
    y = dsv_rope3d_fwd(x.cuda(), bad.cuda(), rope)
    assert dsv_last_device_status() == 5
    assert dsv_last_device_status() == 0
    seen = torch.where((bad < 0) | (bad >= torch.tensor(latent)), torch.zeros_like(bad), bad)   # angle 0
    ang = oracle.rope_angles(seen, axes)
    close("y", y, oracle.rope(x, ang, pairing), rope_mag(x, ang, pairing))
    # an axis that turns nothing is not looked at
    rope = dsv_rope3d_table((0, 20, 20), latent)
    pos[:, 0] = 1000
    dsv_rope3d_fwd(x.cuda(), pos.cuda(), rope)
    assert dsv_last_device_status() == 0


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
def test_infinities_and_nans_stay_in_their_pair(pairing):
    need_gpu()
    gen = torch.Generator().manual_seed(12)
    axes, latent, d = (6, 6, 4), (4, 4, 2), 64
    x, pos = normal(gen, 1, 3, 32, d), positions(latent)
    clean = x.clone()
    x[0, 1, 9, 2] = float("inf")
    x[0, 2, 20, 40] = float("-inf")   # past the rotated features
    x[0, 0, 31, 63] = float("nan")
    rope = dsv_rope3d_table(axes, latent, pairing=pairing)
    y = dsv_rope3d_fwd(x.cuda(), pos.cuda(), rope).cpu()
    want = dsv_rope3d_fwd(clean.cuda(), pos.cuda(), rope).cpu()
    f, g = oracle.pair_features(16, pairing)
    pair = int(np.where((f == 2) | (g == 2))[0][0])
    touched = torch.zeros_like(y, dtype=torch.bool)
    touched[0, 1, 9, [int(f[pair]), int(g[pair])]] = True
    touched[0, 2, 20, 40] = True
    touched[0, 0, 31, 63] = True
    assert torch.equal(y[~touched], want[~touched])
    assert y[0, 2, 20, 40] == float("-inf") and torch.isnan(y[0, 0, 31, 63])
    assert not torch.isfinite(y[0, 1, 9, int(f[pair])])


# ---------------------------------------------------------------- norm + rotation

def norm_case(B, H, latent, d, seed):
    gen = torch.Generator().manual_seed(seed)
    N = int(np.prod(latent))
    spread = 0.2 + 3 * torch.rand(B, 1, N, 1, generator=gen)
    q, k = ((torch.randn(B, H, N, d, generator=gen) * spread).to(BF16) for _ in range(2))
    v, dq, dk, dv = (normal(gen, B, H, N, d) for _ in range(4))
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=gen)).to(BF16) for _ in range(2))
    return dict(q=q, k=k, v=v, dq=dq, dk=dk, dv=dv, wq=wq, wk=wk)


def check_fwd(name, y, x, w, ang, pairing, eps):
    ref = oracle.qk_norm_rope_fwd(x, w, ang, pairing, eps)
    mag = rope_mag(oracle.qk_norm(x, w, eps), ang, pairing)
    close(name, y, ref, mag)


def check_bwd(name, dx, dw, dy, x, w, ang, pairing, eps):
    rx, rw = oracle.qk_norm_rope_bwd(dy, x, w, ang, pairing, eps)
    x64, one = np64(x), np.ones(x.shape[-1]) if w is None else np.abs(np64(w))
    rstd = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + eps)
    xhat = np.abs(x64) * rstd
    g = rope_mag(dy, ang, pairing)                     # magnitudes of the turned gradient's terms
    mag = rstd * (g * one + xhat * (g * one * xhat).mean(-1, keepdims=True))
    close(name, dx, rx, mag)
    if dw is None:
        return
    excess = np.abs(np64(dw) - rw) - 2.0 ** -16 * (g * xhat).sum((0, 1, 2))
    assert float(excess.max()) <= 0, f"d{name}: bound exceeded by {excess.max():.3e}"


@pytest.mark.parametrize("B,H,latent,d,axes,pairing,layout", SHAPES)
def test_qk_norm_rope_matches_oracle(B, H, latent, d, axes, pairing, layout):
    need_gpu()
    c = norm_case(B, H, latent, d, H * 7 + d)
    rope, pos = dsv_rope3d_table(axes, latent, pairing=pairing), positions(latent)
    ang, eps = oracle.rope_angles(pos, axes), 1e-5
    q, k, v = (laid_out(c[n], layout) for n in "qkv")
    wq, wk = c["wq"].cuda(), c["wk"].cuda()
    qo, ko, vo = dsv_qk_norm_rope_fwd(q, k, v, wq, wk, pos.cuda(), rope, eps)
    assert qo.is_contiguous() and ko.is_contiguous() and torch.equal(vo.cpu(), c["v"])
    check_fwd("q", qo, c["q"], c["wq"], ang, pairing, eps)
    check_fwd("k", ko, c["k"], c["wk"], ang, pairing, eps)
    out = tuple(laid_out(torch.zeros(B, H, ang.shape[0], d, dtype=BF16), layout) for _ in range(3))
    bases = [t._base if t._base is not None else t for t in out]
    before = [b.clone() for b in bases]
    dq, dk, dv, dwq, dwk = dsv_qk_norm_rope_bwd(*(c[n].cuda() for n in ("dq", "dk", "dv")), q, k, wq, wk, pos.cuda(),
                                                rope, eps, out=out)
    assert torch.equal(dv.cpu(), c["dv"])
    check_bwd("q", dq, dwq, c["dq"], c["q"], c["wq"], ang, pairing, eps)
    check_bwd("k", dk, dwk, c["dk"], c["k"], c["wk"], ang, pairing, eps)
    assert dsv_last_device_status() == 0
    for t, base, was in zip(out, bases, before):       # nothing around the views was written
        t.zero_()
        assert torch.equal(base.view(torch.int16), was.view(torch.int16))


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
def test_qk_norm_rope_positions_of_each_sample_and_keys_shared_by_the_heads(pairing):
    """pos [B, N, 3]; keys and values of one head read by all (stride 0): their gradients come out for each head."""
    need_gpu()
    gen = torch.Generator().manual_seed(13)
    B, H, N, d, axes, eps = 3, 5, 37, 64, (24, 20, 20), 1e-5
    c = norm_case(B, H, (1, 1, N), d, 14)
    pos = torch.stack([torch.randint(0, 9, (N, 3), generator=gen) for _ in range(B)]).to(torch.int32)
    rope = dsv_rope3d_table(axes, (9, 9, 9), pairing=pairing)
    ang = oracle.rope_angles(pos, axes)
    one = ang[:, None]   # for the magnitudes
    for n in "kv":
        c[n] = c[n][:, :1].expand(B, H, N, d)
    k1, v1 = (c[n][:, :1].contiguous().cuda().expand(B, H, N, d) for n in "kv")
    assert k1.stride(1) == 0
    q, wq, wk = laid_out(c["q"], "packed"), c["wq"].cuda(), c["wk"].cuda()
    qo, ko, vo = dsv_qk_norm_rope_fwd(q, k1, v1, wq, wk, pos.cuda(), rope, eps)
    assert torch.equal(vo.cpu(), c["v"])
    dq, dk, dv, dwq, dwk = dsv_qk_norm_rope_bwd(*(c[n].cuda() for n in ("dq", "dk", "dv")), q, k1, wq, wk, pos.cuda(), rope, eps)
    assert torch.equal(dv.cpu(), c["dv"]) and dsv_last_device_status() == 0
    for n, y, dx, dw in (("q", qo, dq, dwq), ("k", ko, dk, dwk)):
        x, w, dy = c[n], c["w" + n], c["d" + n]
        close(n, y, oracle.qk_norm_rope_fwd(x, w, ang, pairing, eps), rope_mag(oracle.qk_norm(x, w, eps), one, pairing))
        for b in range(B):   # (a sample at a time: the checks take one list of angles)
            s = slice(b, b + 1)
            check_bwd("d" + n, dx[s], None, dy[s], x[s], w, ang[b], pairing, eps)
        rw = sum(oracle.qk_norm_rope_bwd(dy[b:b + 1], x[b:b + 1], w, ang[b], pairing, eps)[1] for b in range(B))
        bound = 2.0 ** -16 * (rope_mag(dy, one, pairing) * np.abs(oracle.qk_norm(x, None, eps))).sum((0, 1, 2))
        assert (np.abs(np64(dw) - rw) <= bound).all()


def test_qk_norm_alone_without_weights_and_without_values():
    need_gpu()
    c = norm_case(2, 3, (1, 5, 5), 64, 3)
    q, k = c["q"].cuda(), c["k"].cuda()
    ang = np.zeros((25, 0))
    qo, ko, vo = dsv_qk_norm_rope_fwd(q, k, None, None, c["wk"].cuda(), None, None)
    assert vo is None
    check_fwd("q", qo, c["q"], None, ang, "interleaved", 1e-6)
    check_fwd("k", ko, c["k"], c["wk"], ang, "interleaved", 1e-6)
    dq, dk, dv, dwq, dwk = dsv_qk_norm_rope_bwd(c["dq"].cuda(), c["dk"].cuda(), None, q, k, None, c["wk"].cuda(), None, None)
    assert dv is None and dwq is None
    check_bwd("q", dq, None, c["dq"], c["q"], None, ang, "interleaved", 1e-6)
    check_bwd("k", dk, dwk, c["dk"], c["k"], c["wk"], ang, "interleaved", 1e-6)
    dq2, dk2, dv, dwq, dwk = dsv_qk_norm_rope_bwd(c["dq"].cuda(), c["dk"].cuda(), None, q, k, None, None, None, None)
    assert dwq is None and dwk is None and torch.equal(dq2, dq)
    check_bwd("k", dk2, None, c["dk"], c["k"], None, ang, "interleaved", 1e-6)


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
def test_zero_rows_tiny_rows_and_zero_eps(pairing):
    """A padded (all-zero) token gives zeros and finite gradients; with eps = 0 it gives NaN, in that row alone."""
    need_gpu()
    c = norm_case(1, 3, (1, 3, 7), 128, 4)
    for n in "qk":
        c[n][0, :, 5] = 0
        c[n][0, 1, 11] *= 2.0 ** -60
    axes, latent = (44, 42, 42), (1, 3, 7)
    rope, pos = dsv_rope3d_table(axes, latent, pairing=pairing), positions(latent).cuda()
    ang = oracle.rope_angles(pos.cpu(), axes)
    g = {n: t.cuda() for n, t in c.items()}
    qo, ko, _ = dsv_qk_norm_rope_fwd(g["q"], g["k"], g["v"], g["wq"], g["wk"], pos, rope)
    assert not qo[0, :, 5].any() and not ko[0, :, 5].any()
    check_fwd("q", qo, c["q"], c["wq"], ang, pairing, 1e-6)
    dq, dk, _, dwq, dwk = dsv_qk_norm_rope_bwd(g["dq"], g["dk"], g["dv"], g["q"], g["k"], g["wq"], g["wk"], pos, rope)
    check_bwd("q", dq, dwq, c["dq"], c["q"], c["wq"], ang, pairing, 1e-6)
    check_bwd("k", dk, dwk, c["dk"], c["k"], c["wk"], ang, pairing, 1e-6)
    qo, ko, _ = dsv_qk_norm_rope_fwd(g["q"], g["k"], g["v"], g["wq"], g["wk"], pos, rope, eps=0.0)
    bad = torch.isnan(qo).any(-1)
    assert bad[0, :, 5].all() and int(bad.sum()) == 3
    # finite rows alone, odd counts (groups without a token): eps = 0 leaves no NaN anywhere
    for n in "qk":
        g[n][0, :, 5] = g[n][0, :, 6]
    dq, dk, _, dwq, dwk = dsv_qk_norm_rope_bwd(g["dq"], g["dk"], g["dv"], g["q"], g["k"], g["wq"], g["wk"], pos, rope, eps=0.0)
    check_bwd("q", dq, dwq, c["dq"], g["q"].cpu(), c["wq"], ang, pairing, 0.0)
    check_bwd("k", dk, dwk, c["dk"], g["k"].cpu(), c["wk"], ang, pairing, 0.0)


def test_gradients_against_differences():
    """Central differences of the fp64 loss sum(dy * forward) along random directions against the kernel's
    gradients: the gradient's bf16 rounding (2^-8 of each entry, random signs) is what separates them."""
    need_gpu()
    c = norm_case(2, 3, (2, 3, 4), 64, 5)
    axes, latent, eps = (24, 20, 20), (2, 3, 4), 1e-5
    rope, pos = dsv_rope3d_table(axes, latent), positions(latent)
    ang = oracle.rope_angles(pos, axes)
    g = {n: t.cuda() for n, t in c.items()}
    dq, _, _, dwq, _ = dsv_qk_norm_rope_bwd(g["dq"], g["dk"], g["dv"], g["q"], g["k"], g["wq"], g["wk"], pos.cuda(), rope, eps)
    rng = np.random.default_rng(6)
    x, w, dy = np64(c["q"]), np64(c["wq"]), np64(c["dq"])
    loss = lambda a, b: float((oracle.qk_norm_rope_fwd(a, b, ang, "interleaved", eps) * dy).sum())
    h = 1e-5
    for _ in range(4):
        e, ew = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        want = (loss(x + h * e, w) - loss(x - h * e, w)) / (2 * h)
        assert abs(float((np64(dq) * e).sum()) - want) <= 2.0 ** -8 * float(np.abs(np64(dq) * e).sum()) + 1e-6 * abs(want)
        want = (loss(x, w + h * ew) - loss(x, w - h * ew)) / (2 * h)
        assert abs(float((np64(dwq) * ew).sum()) - want) <= 2.0 ** -14 * float(np.abs(np64(dwq) * ew).sum()) + 1e-6 * abs(want)


def check_weight_sum(name, dw, dy, x, w, ang, pairing, eps, L):
    excess = np.abs(np64(dw) - oracle.qk_norm_rope_bwd(dy, x, w, ang, pairing, eps)[1])
    xhat = np.abs(oracle.qk_norm(x, None, eps))
    excess -= (L * 2.0 ** -24 + 2.0 ** -20) * (rope_mag(dy, ang, pairing) * xhat).sum((0, 1, 2))
    assert float(excess.max()) <= 0, f"{name}: bound exceeded by {excess.max():.3e}"


# Clips whose backward's 608 persistent CTAs take several units (a tile of tokens, all heads or a chunk of them) each, with
# a last turn that not all of them have: both head dims and pairings, one chunk of heads and several.
MANY = [(2, 3, (59, 113, 3), 64), (2, 3, (59, 113, 3), 128), (1, 9, (5, 23, 43), 64), (2, 4, (1, 47, 53), 128)]


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("B,H,latent,d", MANY)
def test_backward_of_several_units_to_a_cta(B, H, latent, d, pairing):
    """dq, dk, dwq and dwk in full.  A weight's gradient is a chain of L fp32 additions on terms within 2^-20: the heads
    and turns of a thread, a CTA's groups of lanes, the CTAs a warp sums, the 32 warps; off by at most
    (L 2^-24 + 2^-20) sum |term|."""
    need_gpu()
    c = norm_case(B, H, latent, d, 21 + H)
    axes, eps = (24, 20, 20) if d == 64 else (44, 42, 42), 1e-5
    rope, pos = dsv_rope3d_table(axes, latent, pairing=pairing), positions(latent)
    ang, N = oracle.rope_angles(pos, axes), int(np.prod(latent))
    tokens = 1024 // d                                           # of a tile
    ctas = dsv_qk_norm_rope_bwd_workspace(B, H, N, d) // (8 * d)   # a row of two sums of d for each
    units = B * -(-N // tokens) * H
    assert units > ctas                                          # (at most: with a chunk for each head)
    L = H + -(-units // ctas) + tokens + -(-ctas // 32) + 32
    q, k = (laid_out(c[n], "packed") for n in "qk")
    dq, dk, dv, dwq, dwk = dsv_qk_norm_rope_bwd(*(c[n].cuda() for n in ("dq", "dk", "dv")), q, k, c["wq"].cuda(),
                                                c["wk"].cuda(), pos.cuda(), rope, eps)
    assert dsv_last_device_status() == 0 and torch.equal(dv.cpu(), c["dv"])
    for x, dx, dw in (("q", dq, dwq), ("k", dk, dwk)):
        check_bwd(x, dx, None, c["d" + x], c[x], c["w" + x], ang, pairing, eps)
        check_weight_sum("d" + x, dw, c["d" + x], c[x], c["w" + x], ang, pairing, eps, L)


def direction_check(got, grad_name, c, ang, eps, rng):
    """Central differences of the fp64 loss sum(dy * forward) along a random direction against `got`.  dq: its entries'
    roundings are uniform within half a step, at most 2^-8 / sqrt 3 of a value each and of random sign: six standard
    deviations of their sum.  dwq: the fp32 sums' worst case, L = 120 additions on terms within 2^-20."""
    x, w, dy, h = np64(c["q"]), np64(c["wq"]), np64(c["dq"]), 1e-5
    loss = lambda a, b: float((oracle.qk_norm_rope_fwd(a, b, ang, "interleaved", eps) * dy).sum())
    e = rng.standard_normal(got.shape)
    if grad_name == "dq":
        want = (loss(x + h * e, w) - loss(x - h * e, w)) / (2 * h)
        bound = 6 * 2.0 ** -8 / 3 ** 0.5 * float(np.linalg.norm(got))
    else:
        want = (loss(x, w + h * e) - loss(x, w - h * e)) / (2 * h)
        S = (rope_mag(c["dq"], ang, "interleaved") * np.abs(oracle.qk_norm(c["q"], None, eps))).sum((0, 1, 2))
        bound = (120 * 2.0 ** -24 + 2.0 ** -20) * float((S * np.abs(e)).sum())
    return abs(float((got * e).sum()) - want) <= bound + 1e-6 * abs(want)


def test_gradients_against_differences_within_their_roundings():
    need_gpu()
    c = norm_case(2, 3, (2, 3, 4), 64, 5)
    axes, latent, eps = (24, 20, 20), (2, 3, 4), 1e-5
    rope, pos = dsv_rope3d_table(axes, latent), positions(latent)
    ang = oracle.rope_angles(pos, axes)
    g = {n: t.cuda() for n, t in c.items()}
    dq, _, _, dwq, _ = dsv_qk_norm_rope_bwd(g["dq"], g["dk"], g["dv"], g["q"], g["k"], g["wq"], g["wk"], pos.cuda(), rope, eps)
    rng = np.random.default_rng(6)
    for _ in range(4):
        assert direction_check(np64(dq), "dq", c, ang, eps, rng) and direction_check(np64(dwq), "dwq", c, ang, eps, rng)


def test_bitwise_repeatable_and_workspace_contents_do_not_matter():
    need_gpu()
    B, H, latent, d = 1, 9, (4, 32, 33), 128
    c = norm_case(B, H, latent, d, 6)
    axes = (44, 42, 42)
    rope, pos = dsv_rope3d_table(axes, latent), positions(latent).cuda()
    g = {n: t.cuda() for n, t in c.items()}
    ws = torch.full((dsv_qk_norm_rope_bwd_workspace(B, H, pos.shape[0], d),), 255, dtype=torch.uint8, device="cuda")
    run = lambda **kw: dsv_qk_norm_rope_bwd(g["dq"], g["dk"], g["dv"], g["q"], g["k"], g["wq"], g["wk"], pos, rope, **kw)
    a, b = run(), run(workspace=ws)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    with pytest.raises(DSVError, match="workspace"):
        run(workspace=ws[:-256])


def test_graph_capture_and_other_streams():
    need_gpu()
    latent, axes = (4, 16, 16), (24, 20, 20)
    rope, pos = dsv_rope3d_table(axes, latent), positions(latent).cuda()
    cases = [norm_case(1, 2, latent, 64, s) for s in (1, 2)]
    g = {n: t.cuda() for n, t in cases[0].items()}

    def step():
        qo, ko, vo = dsv_qk_norm_rope_fwd(g["q"], g["k"], g["v"], g["wq"], g["wk"], pos, rope)
        return (qo, ko, vo, dsv_rope3d_fwd(vo, pos, rope),
                *dsv_qk_norm_rope_bwd(g["dq"], g["dk"], g["dv"], g["q"], g["k"], g["wq"], g["wk"], pos, rope))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graphs, outs = [], []
    for _ in range(2):                       # two captured steps, each with its own workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs.append(step())
        graphs.append(graph)
    for c in cases:
        for n, t in g.items():
            t.copy_(c[n])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):        # the two replays side by side
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for o in outs:
            for u, v in zip(o, want):
                assert torch.equal(u, v)
    assert dsv_last_device_status() == 0


@pytest.mark.slow
def test_positions_from_any_row_of_a_list():
    need_gpu()
    latent = (2, 5, 7)
    pos, rope = token_positions(latent, None).cuda(), dsv_rope3d_table((24, 20, 20), latent)
    x = torch.randn(2, 3, 70, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    want = dsv_rope3d_fwd(x, pos, rope)
    for first in (1, 2, 3):   # 12 bytes a row: a list's slice is copied where it does not start on 16
        with pytest.raises(DSVError, match="pos is not 16-byte aligned"):
            dsv_rope3d_fwd(x[:, :, first:], pos[first:], rope)
        assert torch.equal(dsv_rope3d_fwd(x[:, :, first:], pos[first:].clone(), rope), want[:, :, first:])
    assert torch.equal(dsv_rope3d_fwd(x[:, :, 4:], pos[4:], rope), want[:, :, 4:])
    with pytest.raises(TypeError, match="pos"):
        dsv_rope3d_fwd(x, [0], rope)


def test_offsets_past_32_bits():
    """The long clip, 16 heads: 3.2 G elements in the packed tensor; its last tokens against the oracle."""
    need_gpu()
    B, H, latent, d, axes = 1, 16, (127, 64, 64), 128, (44, 42, 42)
    pos = token_positions(latent, (4, 4, 4))
    N = pos.shape[0]
    gen = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.empty((B, N, 3, H, d), dtype=BF16, device="cuda").normal_(generator=gen)
    assert qkv.numel() > 2 ** 31
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    w = torch.ones(d, dtype=BF16, device="cuda")
    rope = dsv_rope3d_table(axes, latent)
    qo, ko, vo = dsv_qk_norm_rope_fwd(q, k, v, w, w, pos.cuda(), rope)
    rows = torch.tensor([0, 1, N // 2, N - 9, N - 2, N - 1])
    ang = oracle.rope_angles(pos[rows], axes)
    assert torch.equal(vo, v)
    del vo
    for x, y in ((q, qo), (k, ko)):
        check_fwd("long", y[:, :, rows], x[:, :, rows].cpu(), w.cpu(), ang, "interleaved", 1e-6)
    dq, dk, dv, _, _ = dsv_qk_norm_rope_bwd(qo, ko, qo, q, k, w, w, pos.cuda(), rope)
    assert torch.equal(dv, qo)
    check_bwd("long", dk[:, :, rows], None, ko[:, :, rows].cpu(), k[:, :, rows].cpu(), w.cpu(), ang, "interleaved", 1e-6)
    y = dsv_rope3d_bwd(q, pos.cuda(), rope, out=dq)
    close("rope", y[:, :, rows], oracle.rope(q[:, :, rows].cpu(), ang, backward=True),
          rope_mag(q[:, :, rows].cpu(), ang, "interleaved"))


def test_python_refusals():
    need_gpu()
    x = torch.zeros(1, 2, 8, 64, dtype=BF16, device="cuda")
    pos = torch.zeros(8, 3, dtype=torch.int32, device="cuda")
    rope = dsv_rope3d_table((24, 20, 20), (4, 4, 4))
    with pytest.raises(ValueError, match="bfloat16"):
        dsv_rope3d_fwd(x.float(), pos, rope)
    with pytest.raises(ValueError, match="contiguous features"):
        dsv_rope3d_fwd(torch.zeros(1, 2, 64, 8, dtype=BF16, device="cuda").transpose(2, 3), pos, rope)
    with pytest.raises(ValueError, match="pos"):
        dsv_rope3d_fwd(x, pos[:7], rope)
    with pytest.raises(ValueError, match="pos"):
        dsv_rope3d_fwd(x, pos.long(), rope)
    with pytest.raises(ValueError, match="pos"):
        dsv_rope3d_fwd(x, None, rope)
    with pytest.raises(ValueError, match="rope.data"):
        dsv_rope3d_fwd(x, pos, rope._replace(data=rope.data[:-1]))
    with pytest.raises(ValueError, match="out"):
        dsv_rope3d_fwd(x, pos, rope, out=x[:, :1])
    with pytest.raises(DSVError, match="overlap"):
        dsv_rope3d_fwd(x, pos, rope, out=torch.zeros(1, 2, 1, 64, dtype=BF16, device="cuda").expand(1, 2, 8, 64))
    with pytest.raises(DSVError, match="strides"):
        dsv_rope3d_fwd(torch.zeros(1, 2, 8, 66, dtype=BF16, device="cuda")[..., :64], pos, rope)
    with pytest.raises(DSVError, match="aligned"):
        dsv_rope3d_fwd(torch.zeros(1, 2, 8, 72, dtype=BF16, device="cuda")[..., 1:65], pos, rope)
    with pytest.raises(ValueError, match="wq"):
        dsv_qk_norm_rope_fwd(x, x, x, torch.ones(64, device="cuda"), None, pos, rope)
    with pytest.raises(ValueError, match="k:"):
        dsv_qk_norm_rope_fwd(x, x[:, :1], x, None, None, pos, rope)
    with pytest.raises(DSVError, match="B, H, N"):
        dsv_qk_norm_rope_fwd(x[:, :, :0], x[:, :, :0], None, None, None, pos[:0], rope)
    with pytest.raises(ValueError, match="RopeTable"):
        dsv_qk_norm_rope_fwd(x, x, None, None, None, pos, None)
    with pytest.raises(DSVError, match="NULL"):
        dsv_qk_norm_rope_bwd(None, x, None, x, x, None, None, pos, rope)
    with pytest.raises(DSVError, match="both"):
        dsv_qk_norm_rope_bwd(x, x, x, x, x, None, None, pos, rope, out=(torch.empty_like(x), torch.empty_like(x), None))
    with pytest.raises(ValueError, match="dk_out"):
        dsv_qk_norm_rope_bwd(x, x.transpose(1, 2), None, x, x, None, None, pos, rope)
