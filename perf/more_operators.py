"""The measured cases of a DiT block's modulation: the branches' way back into the residual stream, and the projection
that makes the modulation vectors.

residual_norm  r = x + alpha * gate * post(z) and y = pre(r) * (1 + scale) + shift in one pass, both directions (post: the
               branch's RMS norm or none; pre: the next branch's layer or RMS norm, or none);
w4_linear      y = x W^T + bias for a few vectors x and weights of 4 bits with a scale to each group of columns, and
               dx = dy W (the weights are frozen).

Sizes are the repository's clips (16x32x32, 16x64x64 and 127x64x64 tokens, widths 12 * 64 and 16 * 128) and generic ones;
modulation projections make six vectors of a block's width.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6


def listed():
    rn, w4 = "residual_norm", "w4_linear"
    return [
        # the condition's own tokens beside a clip: a call whose launch is most of its time
        dict(name="rn_condition", op=rn, back=False, B=2, N=77, D=1024, f32=False, post="none", pre="layer", alpha=1.0),
        # between attention and feed-forward on the short clip
        dict(name="rn_short", op=rn, back=False, B=1, N=16384, D=768, f32=False, post="none", pre="layer", alpha=1.0),
        # three images of odd sides, a residual stream in 32 bits, norms on both sides of the branch
        dict(name="rn_images", op=rn, back=False, B=3, N=3645, D=1160, f32=True, post="rms", pre="layer", alpha=1.0),
        # the long clip with norms on both sides
        dict(name="rn_long", op=rn, back=False, B=1, N=520192, D=2048, f32=False, post="rms", pre="rms", alpha=0.5),
        # the short clip's gradients
        dict(name="rn_short_bwd", op=rn, back=True, B=1, N=16384, D=768, f32=False, post="none", pre="layer", alpha=1.0),
        # the mid clip's gradients, norms on both sides
        dict(name="rn_mid_bwd", op=rn, back=True, B=1, N=65536, D=2048, f32=False, post="rms", pre="layer", alpha=1.0),
        # two ragged clips, a stream in 32 bits: a small backward call
        dict(name="rn_ragged_bwd", op=rn, back=True, B=2, N=663, D=1160, f32=True, post="rms", pre="rms", alpha=0.5),
        # one block's six vectors for one sample: the smallest projection
        dict(name="w4_block", op=w4, back=False, M=1, D=768, F=4608, G=64, zeros=False, bias=True, f32=False),
        # a block's projection for a batch of eight
        dict(name="w4_batch", op=w4, back=False, M=8, D=2048, F=12288, G=128, zeros=True, bias=True, f32=False),
        # all of 24 blocks in one call, guidance's two conditions
        dict(name="w4_stack", op=w4, back=False, M=2, D=2048, F=294912, G=64, zeros=False, bias=False, f32=False),
        # the condition's gradient through eight blocks' projections, four samples; their sums over tokens are in 32 bits
        dict(name="w4_stack_bwd", op=w4, back=True, M=4, D=2048, F=98304, G=64, zeros=False, bias=False, f32=True),
        # odd sides, short groups with zero points
        dict(name="w4_ragged_bwd", op=w4, back=True, M=5, D=1184, F=7103, G=32, zeros=True, bias=False, f32=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    back = rng.random() < 0.5
    if rng.random() < 0.5:
        while True:
            c = dict(op="residual_norm", back=back, B=rng.randint(1, 4), N=_log(rng, 1, 262144), D=8 * _log(rng, 8, 1024),
                     f32=rng.random() < 0.4, post=rng.choice(("none", "rms")), pre=rng.choice(("none", "layer", "rms", "layer")),
                     alpha=rng.choice((1.0, 0.5)))
            if c["B"] * c["N"] * c["D"] <= 520192 * 2048 // (4 if back else 2):
                return c
    while True:
        G = rng.choice((32, 64, 128))
        c = dict(op="w4_linear", back=back, M=_log(rng, 1, 32), D=G * _log(rng, 1, 8192 // G), F=_log(rng, 16, 300000), G=G,
                 zeros=rng.random() < 0.5, bias=not back and rng.random() < 0.5, f32=back and rng.random() < 0.5)
        if c["F"] * c["D"] <= 294912 * 2048 and c["M"] * c["F"] * c["D"] <= 2 * 294912 * 2048:
            return c


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape, scale=1.0, dtype=BF16):
        out = torch.empty(shape, dtype=dtype, device=dev)
        out.normal_(generator=gen)
        return out.mul_(scale) if scale != 1.0 else out

    s = dict(case)
    if case["op"] == "w4_linear":
        M, D, F, G = case["M"], case["D"], case["F"], case["G"]
        # 4-bit values as rounding leaves them of normal weights, two to a byte: the even column in the low bits
        s["data"] = torch.empty((F, D // 2), dtype=torch.uint8, device=dev)
        step = max(1, (1 << 27) // D)
        for f in range(0, F, step):
            q = normal(min(step, F - f), D, scale=2.6).add_(8.5).clamp_(0, 15.5).to(torch.uint8)
            s["data"][f:f + step] = q[:, 0::2] | (q[:, 1::2] << 4)
        s["scale"] = (torch.rand(F, D // G, generator=gen, device=dev).add_(0.5).mul_(0.4 / math.sqrt(D))).to(BF16)
        s["zero"] = torch.randint(5, 11, (F, D // G), generator=gen, device=dev).to(torch.uint8) if case["zeros"] else None
        if case["back"]:
            s["dy"] = normal(M, F, dtype=F32 if case["f32"] else BF16)
        else:
            s["x"] = normal(M, D)
            s["bias"] = normal(F, scale=0.1) if case["bias"] else None
        return s
    B, N, D = case["B"], case["N"], case["D"]
    stream = F32 if case["f32"] else BF16
    # a stream whose tokens have a spread of their own, and features that stand out
    spread = 0.5 + 3 * torch.rand(B, N, 1, generator=gen, device=dev)
    s["r" if case["back"] else "x"] = x = normal(B, N, D, dtype=stream).mul_(spread.to(stream))
    x[..., ::97] += 4.0
    s["z"] = normal(B, N, D).mul_(0.7 * spread.flip(1).to(BF16))
    # gate, shift and scale are parts of one projection of the condition
    s["mod"] = normal(B, 6, D, scale=0.4)
    s["gate"], s["shift"], s["scale"] = s["mod"][:, 2], s["mod"][:, 3], s["mod"][:, 4]
    s["w_post"] = (1 + 0.2 * normal(D, dtype=F32)).to(BF16) if case["post"] == "rms" else None
    s["w_pre"] = (1 + 0.2 * normal(D, dtype=F32)).to(BF16) if case["pre"] == "rms" else None
    if case["back"]:
        s["dr"] = normal(B, N, D, dtype=stream)
        s["dy"] = normal(B, N, D) if case["pre"] != "none" else None
    return s


# ---------------------------------------------------------------- plain forms

def _rstd(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _rows(v):
    """[B, D] -> fp32 [B, 1, D]."""
    return v.float()[:, None]


def _residual_norm(s):
    z = s["z"].float()
    if s["post"] == "rms":
        z = z * _rstd(z) * s["w_post"].float()
    r = s["x"].float() + s["alpha"] * _rows(s["gate"]) * z
    if s["pre"] == "none":
        return r.to(s["x"].dtype), None
    n = r
    if s["pre"] == "layer":
        n = n - n.mean(-1, keepdim=True)
    n = n * _rstd(n)
    if s["w_pre"] is not None:
        n = n * s["w_pre"].float()
    return r.to(s["x"].dtype), (n * (1 + _rows(s["scale"])) + _rows(s["shift"])).to(BF16)


def _residual_norm_back(s):
    g = s["dr"].float()
    d_scale = d_shift = dw_pre = dw_post = None
    if s["pre"] != "none":
        n, dy = s["r"].float(), s["dy"].float()
        if s["pre"] == "layer":
            n = n - n.mean(-1, keepdim=True)
        rstd = _rstd(n)
        n = n * rstd
        t = (dy * n).sum(1)
        factor = 1 + s["scale"].float()
        d_shift, d_scale = dy.sum(1), t
        if s["w_pre"] is not None:
            w = s["w_pre"].float()
            d_scale, dw_pre, factor = t * w, (t * factor).sum(0), factor * w
        h = dy * factor[:, None]
        h = h - n * (h * n).mean(-1, keepdim=True) - (h.mean(-1, keepdim=True) if s["pre"] == "layer" else 0)
        g = g + rstd * h
    z, gate = s["z"].float(), s["alpha"] * s["gate"].float()
    u = g * gate[:, None]
    if s["post"] == "rms":
        rstd, w = _rstd(z), s["w_post"].float()
        z = z * rstd
        t = (g * z).sum(1)
        d_gate, dw_post = s["alpha"] * t * w, (t * gate).sum(0)
        u = u * w
        u = rstd * (u - z * (u * z).mean(-1, keepdim=True))
    else:
        d_gate = s["alpha"] * (g * z).sum(1)
    return g.to(s["dr"].dtype), u.to(BF16), d_gate, dw_post, d_scale, d_shift, dw_pre


def _weights(s):
    F, D = s["F"], s["D"]
    q = torch.stack((s["data"] & 15, s["data"] >> 4), -1).view(F, D // s["G"], s["G"]).float()
    return ((q - (8 if s["zero"] is None else s["zero"].float()[..., None])) * s["scale"].float()[..., None]).view(F, D)


def _given(*outs):
    """The outputs that the call has."""
    return tuple(t for t in outs if t is not None)


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "w4_linear":
        if s["back"]:
            return (s["dy"].float() @ _weights(s)).to(BF16)
        y = s["x"].float() @ _weights(s).t()
        return (y if s["bias"] is None else y + s["bias"].float()).to(BF16)
    return _given(*(_residual_norm_back(s) if s["back"] else _residual_norm(s)))


def _run_own(s):
    import dynamic_sparse_attention_estimate_gb300 as dsv
    if s["op"] == "w4_linear":
        w = dsv.W4Weight(s["data"], s["scale"], s["zero"])
        return dsv.dsv_w4_linear_bwd(s["dy"], w) if s["back"] else dsv.dsv_w4_linear_fwd(s["x"], w, s["bias"])
    pre = s["pre"] != "none"
    mods = (s["gate"], s["w_post"], s["scale"] if pre else None)
    how = dict(post=s["post"], pre=s["pre"], alpha=s["alpha"], eps=EPS)
    if s["back"]:
        return _given(*dsv.dsv_residual_norm_bwd(s["dr"], s["dy"], s["r"] if pre else None, s["z"], *mods, s["w_pre"], **how))
    return _given(*dsv.dsv_residual_norm_fwd(s["x"], s["z"], *mods, s["shift"] if pre else None, s["w_pre"], **how))


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "w4_linear":
        M, D, F, G = case["M"], case["D"], case["F"], case["G"]
        held = F * D // 2 + F * (D // G) * (3 if case["zeros"] else 2) + (2 * F if case["bias"] else 0)
        return {"bytes": held + 2 * M * D + (4 if case["f32"] else 2) * M * F, "flops": 2 * M * D * F}
    B, D = case["B"], case["D"]
    e, w = B * case["N"] * D, 4 if case["f32"] else 2
    pre, rms = case["pre"] != "none", (case["post"] == "rms") + (case["pre"] == "rms")
    if case["back"]:  # dr, z, dx, dz, and with a norm behind it r and dy; then the vectors and their gradients
        small = B * D * ((6 + 8) if pre else 6) + 6 * D * rms
        return {"bytes": e * ((3 * w + 6) if pre else (2 * w + 4)) + small, "flops": e * (40 if pre else 20)}
    return {"bytes": e * (2 * w + (4 if pre else 2)) + B * D * (6 if pre else 2) + 2 * D * rms, "flops": e * (16 if pre else 8)}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_w4(s):
    F, D, G = s["F"], s["D"], s["G"]
    out = []
    step = max(1, (1 << 27) // D)
    for f in range(0, F, step):
        b = s["data"][f:f + step].to(torch.int16)
        w = torch.empty((b.shape[0], D), dtype=F64, device=b.device)
        w[:, 0::2] = (b % 16).to(F64)
        w[:, 1::2] = torch.div(b, 16, rounding_mode="floor").to(F64)
        w -= 8 if s["zero"] is None else s["zero"][f:f + step].to(F64).repeat_interleave(G, 1)
        w *= s["scale"][f:f + step].to(F64).repeat_interleave(G, 1)
        if s["back"]:
            part = torch.einsum("mf,fd->md", s["dy"][:, f:f + step].to(F64), w)
            out = [part if not out else out[0] + part]
        else:
            y = torch.einsum("md,fd->mf", s["x"].to(F64), w)
            out.append(y if s["bias"] is None else y + s["bias"][f:f + step].to(F64))
    return out[0] if s["back"] else torch.cat(out, 1)


def _mean_square(v):
    return torch.linalg.vector_norm(v, dim=-1, keepdim=True).square() / v.shape[-1]


def _exact_rows(s, b, rows):
    """Forward of some rows of a sample: (r, y)."""
    z = s["z"][b, rows].to(F64)
    if s["post"] == "rms":
        z = z / (_mean_square(z) + EPS).sqrt() * s["w_post"].to(F64)
    r = s["x"][b, rows].to(F64) + z * (s["gate"][b].to(F64) * s["alpha"])
    if s["pre"] == "none":
        return r, None
    c = r - r.sum(-1, keepdim=True) / r.shape[-1] if s["pre"] == "layer" else r
    c = c / (_mean_square(c) + EPS).sqrt()
    w = 1 if s["w_pre"] is None else s["w_pre"].to(F64)
    return r, c * (w * (1 + s["scale"][b].to(F64))) + s["shift"][b].to(F64)


def _through_norm(v, g, centred):
    """(xhat, the gradient at v for the gradient g at xhat) of a norm without weights."""
    D = v.shape[-1]
    if centred:
        v = v - v.sum(-1, keepdim=True) / D
    size = (_mean_square(v) + EPS).sqrt()
    hat = v / size
    dv = (g - hat * ((g * hat).sum(-1, keepdim=True) / D)) / size
    return hat, dv - dv.sum(-1, keepdim=True) / D if centred else dv


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "w4_linear":
        return _exact_w4(s)
    B, N, D = case["B"], case["N"], case["D"]
    dev, pre, rms = s["z"].device, case["pre"] != "none", case["post"] == "rms"
    full = lambda: torch.empty((B, N, D), dtype=F64, device=dev)
    first, second = full(), full() if pre or case["back"] else None
    sums = torch.zeros((3, B, D), dtype=F64, device=dev)     # of g zhat, dy xhat and dy over the tokens
    step = max(1, (1 << 26) // D)
    one = torch.ones(D, dtype=F64, device=dev)
    wz = s["w_post"].to(F64) if rms else one
    wr = one if s["w_pre"] is None else s["w_pre"].to(F64)
    for b in range(B):
        gate = s["alpha"] * s["gate"][b].to(F64)
        for n in range(0, N, step):
            rows = slice(n, min(N, n + step))
            if not case["back"]:
                r, y = _exact_rows(s, b, rows)
                first[b, rows] = r
                if pre:
                    second[b, rows] = y
                continue
            g = s["dr"][b, rows].to(F64)
            if pre:
                dy = s["dy"][b, rows].to(F64)
                hat, back = _through_norm(s["r"][b, rows].to(F64), dy * (wr * (1 + s["scale"][b].to(F64))), case["pre"] == "layer")
                g = g + back
                sums[1, b] += (dy * hat).sum(0)
                sums[2, b] += dy.sum(0)
            first[b, rows] = g
            z = s["z"][b, rows].to(F64)
            if rms:
                hat, second[b, rows] = _through_norm(z, g * (gate * wz), False)
                sums[0, b] += (g * hat).sum(0)
            else:
                second[b, rows] = g * gate
                sums[0, b] += (g * z).sum(0)
    if not case["back"]:
        return _given(first, second)
    return _given(first, second, case["alpha"] * sums[0] * wz, (case["alpha"] * s["gate"].to(F64) * sums[0]).sum(0) if rms else None,
                  sums[1] * wr if pre else None, sums[2] if pre else None,
                  ((1 + s["scale"].to(F64)) * sums[1]).sum(0) if s["w_pre"] is not None else None)
