"""The measured cases of the operators around the sparse attention of a video DiT block.

rope3d        rotary positions with several axes (time, height, width), both directions;
qk_norm_rope  the per-head RMS norm of queries and keys with that rotation, out of a packed token-major
              projection into the attention's [B, H, N, d] layout (V is carried along), both directions;
ffn_gated     act(x Wg^T) * (x Wu^T), both directions.

Sizes are the repository's clips (latents 4x16x16, 16x32x32, 16x64x64, 127x64x64, head dims 64 and 128) and generic ones.
"""
import math

import numpy as np
import torch

own = False

BF16 = torch.bfloat16


def listed():
    return [
        # one head pair of the tiny clip: a call whose launch is most of its time
        dict(name="rope_tiny", op="rope3d", back=False, B=1, H=2, T=4, Y=16, X=16, d=64, half=False, packed=False),
        # queries of the mid clip, already head-major
        dict(name="rope_mid", op="rope3d", back=False, B=1, H=16, T=16, Y=64, X=64, d=128, half=False, packed=False),
        # a batch of images (one frame, odd sides), token-major gradients, pairs in halves
        dict(name="rope_images_bwd", op="rope3d", back=True, B=3, H=9, T=1, Y=45, X=81, d=128, half=True, packed=True),
        # the short clip's projection on its way into the attention
        dict(name="qknorm_short", op="qk_norm_rope", back=False, B=1, H=12, T=16, Y=32, X=32, d=64, half=False),
        # the long clip: tensors whose offsets pass 2^31 elements
        dict(name="qknorm_long", op="qk_norm_rope", back=False, B=1, H=16, T=127, Y=64, X=64, d=128, half=False),
        # the mid clip's gradients on their way back to the projection
        dict(name="qknorm_mid_bwd", op="qk_norm_rope", back=True, B=1, H=16, T=16, Y=64, X=64, d=128, half=False),
        # two short ragged clips, pairs in halves: a small backward call
        dict(name="qknorm_ragged_bwd", op="qk_norm_rope", back=True, B=2, H=5, T=3, Y=13, X=17, d=64, half=True),
        # a single token: the weights' bytes are the work
        dict(name="ffn_token", op="ffn_gated", back=False, M=1, D=1024, F=2816, act="silu"),
        # the short clip at its attention width of 12 * 64
        dict(name="ffn_short", op="ffn_gated", back=False, M=16384, D=768, F=2048, act="gelu_tanh"),
        # the mid clip at a width of 16 * 128
        dict(name="ffn_mid", op="ffn_gated", back=False, M=65536, D=2048, F=5632, act="silu"),
        # a training step's backward, 16,384 tokens at that width
        dict(name="ffn_bwd", op="ffn_gated", back=True, M=16384, D=2048, F=5632, act="silu"),
        # odd token count, sides off every tile
        dict(name="ffn_ragged_bwd", op="ffn_gated", back=True, M=777, D=776, F=2056, act="gelu_tanh"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope3d", "qk_norm_rope", "ffn_gated"))
    back = rng.random() < 0.5
    if op == "ffn_gated":
        while True:
            c = dict(op=op, back=back, M=_log(rng, 1, 65536), D=8 * _log(rng, 8, 512), F=8 * _log(rng, 8, 1024),
                     act=rng.choice(("silu", "gelu_tanh")))
            if c["M"] * c["D"] * c["F"] * (3 if back else 1) <= 65536 * 2048 * 5632:
                return c
    while True:
        c = dict(op=op, back=back, B=rng.randint(1, 3), H=rng.randint(1, 24), T=_log(rng, 1, 128), Y=_log(rng, 4, 96),
                 X=_log(rng, 4, 96), d=rng.choice((64, 128)), half=rng.random() < 0.5)
        if op == "rope3d":
            c["packed"] = rng.random() < 0.5
        if c["B"] * c["H"] * c["T"] * c["Y"] * c["X"] * c["d"] <= 16 * 127 * 64 * 64 * 128 // 2:
            return c


# ---------------------------------------------------------------- inputs

def _axes(d):
    """Rotated features of (time, height, width): the two sides a third each, time the rest."""
    side = 2 * (d // 6)
    return (d - 2 * side, side, side)


def _table(axes, lengths, theta=10000.0):
    """(cos, sin) pairs, axis after axis, row after row of positions."""
    parts = []
    for r, n in zip(axes, lengths):
        i = torch.arange(r // 2, dtype=torch.float64)
        ang = torch.arange(n, dtype=torch.float64)[:, None] * theta ** (-2.0 * i / max(r, 1))
        parts.append(torch.stack((ang.cos(), ang.sin()), -1).reshape(-1))
    return torch.cat(parts).float()


def _positions(T, Y, X):
    """(t, h, w) of each token; 4x4x4 cubes of neighbours where the sides allow it, raster order elsewhere."""
    g = torch.stack(torch.meshgrid(torch.arange(T), torch.arange(Y), torch.arange(X), indexing="ij"), -1)
    if Y % 4 == 0 and X % 4 == 0 and T >= 4:
        t4 = T // 4 * 4
        a = g[:t4].reshape(t4 // 4, 4, Y // 4, 4, X // 4, 4, 3).permute(0, 2, 4, 1, 3, 5, 6).reshape(-1, 3)
        g = torch.cat((a, g[t4:].reshape(-1, 3)))
    return g.reshape(-1, 3).to(torch.int32).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape, scale=1.0):
        out = torch.empty(shape, dtype=BF16, device=dev)
        out.normal_(generator=gen)
        return out.mul_(scale) if scale != 1.0 else out

    s = dict(case)
    if case["op"] == "ffn_gated":
        M, D, F = case["M"], case["D"], case["F"]
        s["x"] = normal(M, D)
        s["wg"] = normal(F, D, scale=1 / math.sqrt(D))
        s["wu"] = normal(F, D, scale=1 / math.sqrt(D))
        if case["back"]:
            s["dh"] = normal(M, F)
        return s
    B, H, d = case["B"], case["H"], case["d"]
    T, Y, X = case["T"], case["Y"], case["X"]
    N = T * Y * X
    s["axes"], s["lengths"] = _axes(d), (T, Y, X)
    s["table"] = _table(s["axes"], s["lengths"]).to(dev)
    s["pos"] = _positions(T, Y, X).to(dev)
    if case["op"] == "rope3d":
        s["x"] = normal(B, N, H, d).transpose(1, 2) if case["packed"] else normal(B, H, N, d)
        return s
    qkv = normal(B, N, 3, H, d)
    # queries and keys leave a projection with a spread of their own for each token
    qkv.mul_(0.25 + 2 * torch.rand(B, N, 1, 1, 1, generator=gen, device=dev).to(BF16))
    s["q"], s["k"], s["v"] = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    s["wq"] = (1 + 0.2 * torch.randn(d, generator=gen, device=dev)).to(BF16)
    s["wk"] = (1 + 0.2 * torch.randn(d, generator=gen, device=dev)).to(BF16)
    if case["back"]:
        s["dq"], s["dk"], s["dv"] = (normal(B, H, N, d) for _ in range(3))
        del s["v"]
    return s


# ---------------------------------------------------------------- plain forms

EPS = 1e-6


def _cos_sin(s):
    """cos and sin [N, R/2] fp32 of every token's pairs, gathered from the table."""
    cols, at = [], 0
    for a in range(3):
        pairs = s["axes"][a] // 2
        n = s["lengths"][a] * pairs * 2
        cols.append(s["table"][at:at + n].view(s["lengths"][a], pairs, 2)[s["pos"][:, a].long()])
        at += n
    t = torch.cat(cols, 1)
    return t[..., 0], t[..., 1]


def _rotate(x, cos, sin, half):
    """x [..., N, d] rotated pair by pair; features past the rotated ones pass."""
    R = 2 * cos.shape[-1]
    r = x[..., :R]
    a, b = (r[..., :R // 2], r[..., R // 2:]) if half else (r[..., 0::2], r[..., 1::2])
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.cat((u, v), -1) if half else torch.stack((u, v), -1).flatten(-2)
    return y if R == x.shape[-1] else torch.cat((y, x[..., R:]), -1)


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _norm_back(g, x, w):
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xhat = x * rstd
    gw = g * w
    dx = rstd * (gw - xhat * (gw * xhat).mean(-1, keepdim=True))
    return dx, (g * xhat).sum((0, 1, 2))


def _act(g, act):
    """Activation and its derivative."""
    if act == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return g * sg, sg * (1 + g * (1 - sg))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "ffn_gated":
        x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
        g, u = x @ wg.t(), x @ wu.t()
        a, da = _act(g, s["act"])
        if not s["back"]:
            return (a * u).to(BF16)
        dh = s["dh"].float()
        dg, du = dh * u * da, dh * a
        return (dg @ wg + du @ wu).to(BF16), (dg.t() @ x).to(BF16), (du.t() @ x).to(BF16)
    cos, sin = _cos_sin(s)
    if s["op"] == "rope3d":
        return _rotate(s["x"].float(), cos, -sin if s["back"] else sin, s["half"]).to(BF16)
    wq, wk = s["wq"].float(), s["wk"].float()
    if not s["back"]:
        q = _rotate(_norm(s["q"].float(), wq), cos, sin, s["half"]).to(BF16)
        k = _rotate(_norm(s["k"].float(), wk), cos, sin, s["half"]).to(BF16)
        return q, k, s["v"].contiguous()
    dq, dwq = _norm_back(_rotate(s["dq"].float(), cos, -sin, s["half"]), s["q"].float(), wq)
    dk, dwk = _norm_back(_rotate(s["dk"].float(), cos, -sin, s["half"]), s["k"].float(), wk)
    # the projection's packed layout [B, N, 3, H, d]
    dqkv = torch.stack([g.to(BF16).transpose(1, 2) for g in (dq, dk, s["dv"])], 2)
    return dqkv, dwq, dwk


def _run_own(s):
    import dynamic_sparse_attention_estimate_gb300 as dsv
    if s["op"] == "ffn_gated":
        if s["back"]:
            return dsv.dsv_ffn_gated_bwd(s["dh"], s["x"], s["wg"], s["wu"], act=s["act"])
        return dsv.dsv_ffn_gated_fwd(s["x"], s["wg"], s["wu"], act=s["act"])
    rope = dsv.RopeTable(s["table"], s["axes"], s["lengths"], "halves" if s["half"] else "interleaved")
    if s["op"] == "rope3d":
        return (dsv.dsv_rope3d_bwd if s["back"] else dsv.dsv_rope3d_fwd)(s["x"], s["pos"], rope)
    if not s["back"]:
        return dsv.dsv_qk_norm_rope_fwd(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["pos"], rope, eps=EPS)
    B, H, N, d = s["q"].shape
    dqkv = torch.empty((B, N, 3, H, d), dtype=BF16, device=s["q"].device)
    out = tuple(dqkv[:, :, i].transpose(1, 2) for i in range(3))
    dwq, dwk = dsv.dsv_qk_norm_rope_bwd(s["dq"], s["dk"], s["dv"], s["q"], s["k"], s["wq"], s["wk"], s["pos"], rope,
                                        eps=EPS, out=out)[3:]
    return dqkv, dwq, dwk


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "ffn_gated":
        M, D, F = case["M"], case["D"], case["F"]
        if case["back"]:  # g and u again, dx, and both weights' gradients
            return {"bytes": 2 * (2 * M * D + 4 * D * F + M * F), "flops": 12 * M * D * F}
        return {"bytes": 2 * (M * D + 2 * D * F + M * F), "flops": 4 * M * D * F}
    B, H, N, d = case["B"], case["H"], case["T"] * case["Y"] * case["X"], case["d"]
    e = B * H * N * d
    small = 12 * N + 4 * sum(r * n for r, n in zip(_axes(d), (case["T"], case["Y"], case["X"])))
    if case["op"] == "rope3d":
        return {"bytes": 4 * e + small, "flops": 3 * e}
    if case["back"]:
        return {"bytes": 16 * e + small + 12 * d, "flops": 30 * e}
    return {"bytes": 12 * e + small + 4 * d, "flops": 16 * e}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ffn_gated":
        x, wg, wu = s["x"].double(), s["wg"].double(), s["wu"].double()
        outs = [[], None, None]
        step = 8192
        for m in range(0, case["M"], step):
            xm = x[m:m + step]
            g, u = torch.matmul(xm, wg.mT), torch.matmul(xm, wu.mT)
            if case["act"] == "silu":
                sig = torch.sigmoid(g)
                slope = sig + g * sig * (1 - sig)
                a = g * sig
            else:
                inner = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
                a = g * torch.sigmoid(2 * inner)
                slope = torch.sigmoid(2 * inner) + 2 * a * torch.sigmoid(-2 * inner) * math.sqrt(2 / math.pi) * (1 + 0.134145 * g ** 2)
            if not case["back"]:
                outs[0].append(a * u)
                continue
            dh = s["dh"][m:m + step].double()
            dg, du = dh * u * slope, dh * a
            outs[0].append(torch.matmul(dg, wg) + torch.matmul(du, wu))
            for i, t in ((1, dg), (2, du)):
                p = torch.matmul(t.mT, xm)
                outs[i] = p if outs[i] is None else outs[i] + p
        first = torch.cat(outs[0])
        return (first, outs[1], outs[2]) if case["back"] else first
    # complex rotation: one factor e^(i angle) for each token and pair
    turn, at = [], 0
    for a in range(3):
        n, pairs = s["lengths"][a], s["axes"][a] // 2
        rows = s["table"][at:at + 2 * n * pairs].double().view(n, pairs, 2)
        turn.append(torch.view_as_complex(rows)[s["pos"][:, a].long()])
        at += 2 * n * pairs
    turn = torch.cat(turn, -1)

    def rotated(x, factor):
        R = 2 * factor.shape[-1]
        z = x[..., :R].unflatten(-1, (2, R // 2)).mT if case["half"] else x[..., :R].unflatten(-1, (R // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * factor)
        y = (z.mT if case["half"] else z).flatten(-2)
        return torch.cat((y, x[..., R:]), -1)

    if case["op"] == "rope3d":
        return rotated(s["x"].double(), turn.conj() if case["back"] else turn)
    B, H, N, d = s["q"].shape
    if not case["back"]:
        outs = []
        for name, w in (("q", "wq"), ("k", "wk")):
            y = torch.empty((B, H, N, d), dtype=torch.float64, device=turn.device)
            for h in range(H):  # a head at a time: the long clip in 64 bits
                x = s[name][:, h].double()
                x = x / (x.square().sum(-1, keepdim=True) / d + EPS).sqrt()
                y[:, h] = rotated(x * s[w].double(), turn)
            outs.append(y)
        return outs[0], outs[1], s["v"].contiguous()
    dqkv = torch.empty((B, N, 3, H, d), dtype=torch.float64, device=turn.device)
    dqkv[:, :, 2] = s["dv"].transpose(1, 2)
    sums = []
    for i, (name, w) in enumerate((("q", "wq"), ("k", "wk"))):
        total = torch.zeros(d, dtype=torch.float64, device=turn.device)
        for h in range(H):
            x, g = s[name][:, h].double(), rotated(s["d" + name][:, h].double(), turn.conj())
            size = (x.square().sum(-1, keepdim=True) / d + EPS).sqrt()
            total += (g * x / size).sum((0, 1))
            g = g * s[w].double()
            dqkv[:, :, i, h] = g / size - x * ((g * x).sum(-1, keepdim=True) / (d * size ** 3))
        sums.append(total)
    return dqkv, sums[0], sums[1]
