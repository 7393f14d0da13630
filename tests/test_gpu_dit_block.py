"""A run of the operators together, as a DiT block uses them, forward and backward, against torch fp64 autograd:

  AdaLN -> packed Q/K/V projection -> qk norm + rotation -> estimate, sparse attention -> output projection,
  residual -> AdaLN -> gated feed-forward -> down projection, residual.

The plain projections are torch products in bf16.  Tolerance: a tensor here has passed at most 20 roundings to
bf16 (each operator's result, forward and backward), each at most 2^-8 of its norm; were all of them to
add up they would come to 20 * 2^-8 = 0.078 of the gradient's norm.
"""
import numpy as np
import pytest
import torch

import oracle
from dynamic_sparse_attention_estimate_gb300 import (dsv_adaln_bwd, dsv_adaln_fwd, dsv_estimate_topk, dsv_ffn_gated_bwd,
                                                     dsv_ffn_gated_fwd, dsv_qk_norm_rope_bwd, dsv_qk_norm_rope_fwd,
                                                     dsv_rope3d_table, dsv_sparse_attn_bwd, dsv_sparse_attn_fwd)
from dynamic_sparse_attention_estimate_gb300.binding import dsv_last_device_status
from dynamic_sparse_attention_estimate_gb300.inputs import token_positions
from tests.gpu_helpers import need_gpu, np64

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
TOL = 20 * 2.0 ** -8
B, H, d, LATENT, BLOCK, K, FF = 2, 2, 64, (4, 8, 8), (4, 4, 4), 96, 200
AXES = (24, 20, 20)
N, W = int(np.prod(LATENT)), H * d


def weights(seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=gen) * scale).to(BF16)
    p = dict(x=r(B, N, W), dout=r(B, N, W), wqkv=r(3 * W, W, scale=W ** -0.5), wo=r(W, W, scale=W ** -0.5),
             wq=(1 + 0.2 * torch.randn(d, generator=gen)).to(BF16), wk=(1 + 0.2 * torch.randn(d, generator=gen)).to(BF16),
             wg=r(FF, W, scale=W ** -0.5), wu=r(FF, W, scale=W ** -0.5), wd=r(W, FF, scale=FF ** -0.5))
    for n in ("s1", "b1", "s2", "b2"):
        p[n] = r(B, W, scale=0.3)
    lr = lambda: torch.randint(-4, 5, (B, H, N, 16), generator=gen).to(BF16)
    return p, lr(), lr()


def block_step(p, idx, pos, rope):
    """(out, gradients by name) through the library."""
    y1 = dsv_adaln_fwd(p["x"], p["s1"], p["b1"])
    qkv = (y1 @ p["wqkv"].t()).view(B, N, 3, H, d)
    qkv_views = [qkv[:, :, i].transpose(1, 2) for i in range(3)]
    q, k, v = dsv_qk_norm_rope_fwd(*qkv_views, p["wq"], p["wk"], pos, rope)
    o, lse = dsv_sparse_attn_fwd(q, k, v, idx)
    a = o.transpose(1, 2).reshape(B, N, W)
    x2 = p["x"] + a @ p["wo"].t()
    y2 = dsv_adaln_fwd(x2, p["s2"], p["b2"])
    h = dsv_ffn_gated_fwd(y2, p["wg"], p["wu"])
    out = x2 + h @ p["wd"].t()

    g = {}
    flat = lambda t: t.reshape(B * N, -1)
    g["wd"] = flat(p["dout"]).t() @ flat(h)
    dy2, g["wg"], g["wu"] = dsv_ffn_gated_bwd(p["dout"] @ p["wd"], y2, p["wg"], p["wu"])
    dx2, g["s2"], g["b2"] = dsv_adaln_bwd(x2, p["s2"], dy2)
    dx2 = dx2 + p["dout"]
    g["wo"] = flat(dx2).t() @ flat(a)
    do = (dx2 @ p["wo"]).view(B, N, H, d).transpose(1, 2).contiguous()
    dq, dk, dv = dsv_sparse_attn_bwd(do, q, k, v, o, lse, idx)
    dqkv = torch.empty_like(qkv)
    out_views = tuple(dqkv[:, :, i].transpose(1, 2) for i in range(3))
    g["wq"], g["wk"] = dsv_qk_norm_rope_bwd(dq, dk, dv, *qkv_views[:2], p["wq"], p["wk"], pos, rope, out=out_views)[3:]
    g["wqkv"] = flat(dqkv).t() @ flat(y1)
    dx, g["s1"], g["b1"] = dsv_adaln_bwd(p["x"], p["s1"], dqkv.view(B, N, 3 * W) @ p["wqkv"])
    g["x"] = dx + dx2
    return out, g


def reference(p, idx, pos):
    """The same block in torch fp64 with autograd, dense attention under the selection's mask."""
    t = {n: torch.from_numpy(np64(v)) for n, v in p.items()}
    names = [n for n in t if n != "dout"]
    for n in names:
        t[n].requires_grad_()
    ang = torch.from_numpy(oracle.rope_angles(pos.cpu(), AXES))
    turn = torch.polar(torch.ones_like(ang), ang)

    def adaln(x, s, b):
        return torch.nn.functional.layer_norm(x, (W,), eps=1e-6) * (1 + s[:, None]) + b[:, None]

    def rot(x):
        return torch.view_as_real(torch.view_as_complex(x.reshape(B, H, N, d // 2, 2).contiguous()) * turn).flatten(-2)

    norm = lambda x, w: torch.nn.functional.rms_norm(x, (d,), w, 1e-6)
    qkv = (adaln(t["x"], t["s1"], t["b1"]) @ t["wqkv"].T).view(B, N, 3, H, d).permute(2, 0, 3, 1, 4)
    q, k, v = rot(norm(qkv[0], t["wq"])), rot(norm(qkv[1], t["wk"])), qkv[2]
    mask = torch.zeros(B, H, N // 64, N, dtype=torch.bool).scatter_(-1, idx.cpu().long(), True)
    s = (q @ k.mT / d ** 0.5).masked_fill(~mask.repeat_interleave(64, 2), float("-inf"))
    a = (s.softmax(-1) @ v).transpose(1, 2).reshape(B, N, W)
    x2 = t["x"] + a @ t["wo"].T
    y2 = adaln(x2, t["s2"], t["b2"])
    out = x2 + (torch.nn.functional.silu(y2 @ t["wg"].T) * (y2 @ t["wu"].T)) @ t["wd"].T
    out.backward(t["dout"])
    return out.detach().numpy(), {n: t[n].grad.numpy() for n in names}


def test_block_matches_autograd_eager_and_captured():
    need_gpu()
    cpu, q_lr, k_lr = weights()
    p = {n: v.cuda() for n, v in cpu.items()}
    pos = token_positions(LATENT, BLOCK).cuda()
    rope = dsv_rope3d_table(AXES, LATENT)
    idx = dsv_estimate_topk(q_lr.cuda(), k_lr.cuda(), K)
    out, grads = block_step(p, idx, pos, rope)
    torch.cuda.synchronize()
    assert dsv_last_device_status() == 0
    ref, rgrads = reference(cpu, idx, pos)

    def close(name, got, want):
        rel = float(np.linalg.norm(np64(got) - want) / np.linalg.norm(want))
        assert rel <= TOL, f"{name}: rel-L2 {rel:.3e}"

    close("out", out, ref)
    assert set(grads) == set(rgrads)
    for n in grads:
        close("d" + n, grads[n], rgrads[n])

    # the same step captured, while the eager results live, then replayed on other inputs
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        cout, cgrads = block_step(p, idx, pos, rope)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cout, out) and all(torch.equal(cgrads[n], grads[n]) for n in grads)
    for n, v in weights(1)[0].items():
        p[n].copy_(v)
    graph.replay()
    eager, egrads = block_step(p, idx, pos, rope)
    torch.cuda.synchronize()
    assert torch.equal(cout, eager) and all(torch.equal(cgrads[n], egrads[n]) for n in egrads)
    assert dsv_last_device_status() == 0
