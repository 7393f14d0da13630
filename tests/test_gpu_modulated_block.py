"""A run of the operators together, as a DiT block with its modulation uses them, forward and backward, against torch fp64
autograd:

  condition -> 4-bit projection -> six vectors;  AdaLN -> branch -> gated residual with norms on both sides of it -> gated
  feed-forward -> gated residual with a last norm;  the vectors' gradients, parts of one tensor, back through the projection.

The branch and the down projection are torch products in bf16.  Tolerance: a tensor here has passed at most 20 roundings to
bf16 (each operator's result, forward and backward), each at most 2^-8 of its norm; were all of them to
add up they would come to 20 * 2^-8 = 0.078 of the gradient's norm.
"""
import numpy as np
import pytest
import torch

import oracle
from dynamic_sparse_attention_estimate_gb300 import (W4Weight, dsv_adaln_bwd, dsv_adaln_fwd, dsv_ffn_gated_bwd, dsv_ffn_gated_fwd,
                                                     dsv_residual_norm_bwd, dsv_residual_norm_fwd, dsv_w4_linear_bwd,
                                                     dsv_w4_linear_fwd, dsv_w4_quantize)
from dynamic_sparse_attention_estimate_gb300.binding import dsv_last_device_status
from tests.gpu_helpers import need_gpu, np64

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
TOL = 20 * 2.0 ** -8
B, N, W, FF, COND = 3, 150, 136, 200, 192
SHIFT1, SCALE1, GATE1, SHIFT2, SCALE2, GATE2 = range(6)


def weights(seed=0, f32=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=gen) * scale).to(BF16)
    near_one = lambda: (1 + 0.2 * torch.randn(W, generator=gen)).to(BF16)
    stream = torch.float32 if f32 else BF16
    return dict(x=r(B, N, W).to(stream), dr=r(B, N, W).to(stream), dy=r(B, N, W), cond=r(B, COND), wa=r(W, W, scale=W ** -0.5),
                wd=r(W, FF, scale=FF ** -0.5), wg=r(FF, W, scale=W ** -0.5), wu=r(FF, W, scale=W ** -0.5), post1=near_one(),
                post2=near_one(), last=near_one(), bias=r(6 * W, scale=0.2))


def block_step(p, wm):
    """(stream, normed stream, gradients by name) through the library."""
    mod = dsv_w4_linear_fwd(p["cond"], wm, p["bias"]).view(B, 6, W)
    # adaln takes bf16 rows: with an fp32 stream its input is rounded first
    x1 = p["x"].to(BF16)
    shift1, scale1 = mod[:, SHIFT1].contiguous(), mod[:, SCALE1].contiguous()
    y1 = dsv_adaln_fwd(x1, scale1, shift1)
    a = y1 @ p["wa"].t()
    r1, y2 = dsv_residual_norm_fwd(p["x"], a, mod[:, GATE1], p["post1"], mod[:, SCALE2], mod[:, SHIFT2], post="rms")
    h = dsv_ffn_gated_fwd(y2, p["wg"], p["wu"])
    m = h @ p["wd"].t()
    r2, y3 = dsv_residual_norm_fwd(r1, m, mod[:, GATE2], p["post2"], w_pre=p["last"], post="rms", pre="rms")

    g = {}
    flat = lambda t: t.reshape(B * N, -1)
    d_mod = torch.empty((B, 6, W), device=mod.device)
    dr1, dm, _, g["post2"], _, _, g["last"] = dsv_residual_norm_bwd(p["dr"], p["dy"], r2, m, mod[:, GATE2], p["post2"], None, p["last"],
                                                                    post="rms", pre="rms", d_mod=(d_mod[:, GATE2], None, None))
    g["wd"] = flat(dm).t() @ flat(h)
    dy2, g["wg"], g["wu"] = dsv_ffn_gated_bwd(dm @ p["wd"], y2, p["wg"], p["wu"])
    dx, da, _, g["post1"], *_ = dsv_residual_norm_bwd(dr1, dy2, r1, a, mod[:, GATE1], p["post1"], mod[:, SCALE2], post="rms",
                                                      d_mod=(d_mod[:, GATE1], d_mod[:, SCALE2], d_mod[:, SHIFT2]))
    g["wa"] = flat(da).t() @ flat(y1)
    dx1, ds1, db1 = dsv_adaln_bwd(x1, scale1, da @ p["wa"])
    d_mod[:, SCALE1], d_mod[:, SHIFT1] = ds1, db1
    g["x"] = dx + dx1
    g["cond"] = dsv_w4_linear_bwd(d_mod.view(B, 6 * W), wm)
    return r2, y3, g


def reference(p, wm):
    """The same block in torch fp64 with autograd."""
    t = {n: torch.from_numpy(np64(v)) for n, v in p.items()}
    names = [n for n in t if n not in ("dr", "dy", "bias")]
    for n in names:
        t[n].requires_grad_()
    F = torch.nn.functional
    values = torch.from_numpy(oracle.w4_values(*wm))
    mod = (t["cond"] @ values.T + t["bias"]).view(B, 6, 1, W)
    norm = lambda v: F.layer_norm(v, (W,), eps=1e-6)
    rms = lambda v, w: F.rms_norm(v, (W,), w, 1e-6)
    a = (norm(t["x"]) * (1 + mod[:, SCALE1]) + mod[:, SHIFT1]) @ t["wa"].T
    r1 = t["x"] + mod[:, GATE1] * rms(a, t["post1"])
    y2 = norm(r1) * (1 + mod[:, SCALE2]) + mod[:, SHIFT2]
    m = (F.silu(y2 @ t["wg"].T) * (y2 @ t["wu"].T)) @ t["wd"].T
    r2 = r1 + mod[:, GATE2] * rms(m, t["post2"])
    y3 = rms(r2, t["last"])
    ((r2 * t["dr"]).sum() + (y3 * t["dy"]).sum()).backward()
    return r2.detach().numpy(), y3.detach().numpy(), {n: t[n].grad.numpy() for n in names}


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("symmetric", [True, False])
def test_block_matches_autograd_eager_and_captured(f32, symmetric):
    need_gpu()
    cpu = weights(f32=f32)
    gen = torch.Generator().manual_seed(7)
    wm = dsv_w4_quantize((torch.randn(6 * W, COND, generator=gen) * 0.4 * COND ** -0.5).to(BF16).cuda(), 64, symmetric)
    p = {n: v.cuda() for n, v in cpu.items()}
    r2, y3, grads = block_step(p, wm)
    torch.cuda.synchronize()
    assert dsv_last_device_status() == 0
    want_r2, want_y3, want = reference(cpu, wm)

    def close(name, got, ref):
        rel = float(np.linalg.norm(np64(got) - ref) / np.linalg.norm(ref))
        assert rel <= TOL, f"{name}: rel-L2 {rel:.3e}"

    close("stream", r2, want_r2)
    close("normed", y3, want_y3)
    assert set(grads) == set(want)
    for n in grads:
        close("d" + n, grads[n], want[n])

    # the same step captured, while the eager results live, then replayed on other inputs
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        c2, c3, cgrads = block_step(p, wm)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c2, r2) and torch.equal(c3, y3) and all(torch.equal(cgrads[n], grads[n]) for n in grads)
    for n, v in weights(1, f32).items():
        p[n].copy_(v)
    graph.replay()
    e2, e3, egrads = block_step(p, wm)
    torch.cuda.synchronize()
    assert torch.equal(c2, e2) and torch.equal(c3, e3) and all(torch.equal(cgrads[n], egrads[n]) for n in egrads)
    assert dsv_last_device_status() == 0


def test_weights_of_4_bits_stand_for_the_rounded_projection():
    """The 4-bit projection of weights that are whole steps of their scales is the plain product of those weights."""
    need_gpu()
    gen = torch.Generator().manual_seed(2)
    q = torch.randint(-7, 8, (6 * W, COND), generator=gen)
    q[:, ::64] = 7                                    # each group's largest: its scale is 1 / 8
    w, x = (q / 8).to(BF16), torch.randint(-3, 4, (B, COND), generator=gen).to(BF16)
    wm = dsv_w4_quantize(w.cuda(), 64)
    assert isinstance(wm, W4Weight) and (wm.scale == 0.125).all()
    want = (x.double() @ w.double().T).to(BF16)
    assert torch.equal(dsv_w4_linear_fwd(x.cuda(), wm).cpu(), want)
