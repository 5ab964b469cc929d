"""Measured cases of the training operators around the retention core.

The operators: the residual sum with its scale and the norm before the next
block (``msr_resid_norm_fwd`` / ``_bwd``), the per-head norm after the
retention with its affine and swish gate (``msr_gated_norm_fwd`` / ``_bwd``),
activations kept in 8 bits (``msr_ckpt_pack`` / ``_unpack``) and the weight
gradient of a projection whose input was kept so (``msr_ckpt_wgrad``).

``run`` computes a case in elementary torch operations, or, with ``own`` set,
by the library's entry points; both from what ``prepare`` gives.

8-bit form: 32 neighbouring values share a power of two 2^e, the smallest
with max|x| <= 448 * 2^e (e4m3) or 127 * 2^e (int8); q = x * 2^-e rounded to
nearest even, stored with e + 127 in one byte.
"""
import math

import torch

own = False

GROUP = 32
TOP = {"e4m3": 448.0, "i8": 127.0}
QTYPE = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # a few sequences' newest tokens between two small blocks: latency only
        dict(name="resid_fwd_f32_5x256", op="resid_fwd", dtype="f32", rows=5, d=256, norm="layer", affine=True,
             scaled=False, keep="none"),
        # training forward between two blocks of the 4 x 8192-token model, the sum kept in 8 bits
        dict(name="resid_fwd_bf16_32768x4096_e4m3", op="resid_fwd", dtype="bf16", rows=32768, d=4096, norm="layer",
             affine=True, scaled=True, keep="e4m3"),
        # its backward at 8 x 2048 tokens from the 16-bit sum, the branch's learned scale included
        dict(name="resid_bwd_bf16_16384x2048_rms", op="resid_bwd", dtype="bf16", rows=16384, d=2048, norm="rms",
             affine=True, scaled=True, keep="none"),
        # long sequences (2 x 16384, one token short) from the 8-bit sum
        dict(name="resid_bwd_bf16_32767x2560_i8", op="resid_bwd", dtype="bf16", rows=32767, d=2560, norm="layer",
             affine=True, scaled=False, keep="i8"),
        # the small float32 layer: 256 tokens, 4 heads of 64
        dict(name="gated_fwd_f32_256x4x64", op="gated_fwd", dtype="f32", rows=256, heads=4, d=64, norm="layer",
             affine=False, keep="none"),
        # the 8 x 2048-token layer's forward
        dict(name="gated_fwd_bf16_16384x8x256", op="gated_fwd", dtype="bf16", rows=16384, heads=8, d=256,
             norm="layer", affine=True, keep="none"),
        # its backward from the 16-bit tensors
        dict(name="gated_bwd_bf16_16384x8x256", op="gated_bwd", dtype="bf16", rows=16384, heads=8, d=256,
             norm="layer", affine=True, keep="none", again=False),
        # the 4 x 8192-token layer's backward from 8 bits, the gated rows formed again for W_O's gradient
        dict(name="gated_bwd_bf16_32768x16x512_e4m3", op="gated_bwd", dtype="bf16", rows=32768, heads=16, d=512,
             norm="layer", affine=True, keep="e4m3", again=True),
        # a small float32 activation kept and read back, ragged
        dict(name="ckpt_f32_77x320_i8", op="ckpt", dtype="f32", rows=77, d=320, keep="i8"),
        # one of Q, K, V of the long-sequence model kept and read back
        dict(name="ckpt_bf16_32768x2560_e4m3", op="ckpt", dtype="bf16", rows=32768, d=2560, keep="e4m3"),
        # weight gradient of [Q | K | V | G] of the 8 x 2048-token layer
        dict(name="wgrad_bf16_16384_2048x8192_e4m3", op="wgrad", dtype="bf16", rows=16384, d=2048, out=8192,
             keep="e4m3", normed=False),
        # a small float32 projection behind a norm, ragged token count
        dict(name="wgrad_f32_999_256x1024_i8", op="wgrad", dtype="f32", rows=999, d=256, out=1024, keep="i8",
             normed=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["resid_fwd", "resid_bwd", "gated_fwd", "gated_bwd", "ckpt", "wgrad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    keep = rng.choice(["none", "e4m3", "i8"]) if op not in ("ckpt", "wgrad") else rng.choice(["e4m3", "i8"])
    case = dict(op=op, dtype=dtype, keep=keep)
    if op in ("gated_fwd", "gated_bwd"):
        d = rng.choice([64, 128, 256, 512])
        heads = rng.randint(1, 16)
        case.update(rows=_log_int(rng, 1, max(1, 2 ** 26 // (heads * d))), heads=heads, d=d)
    elif op == "wgrad":
        case.update(rows=_log_int(rng, 1, 16384), d=64 * _log_int(rng, 1, 40), out=64 * _log_int(rng, 1, 64))
    else:
        d = 64 * _log_int(rng, 1, 128)
        case.update(rows=_log_int(rng, 1, 2 ** 26 // d), d=d)
    if op in ("resid_fwd", "resid_bwd", "gated_fwd", "gated_bwd"):
        case.update(norm=rng.choice(["layer", "rms"]), affine=rng.random() < 0.7)
    if op in ("resid_fwd", "resid_bwd"):
        case["scaled"] = rng.random() < 0.5
    if op == "gated_bwd":
        case["again"] = rng.random() < 0.5
    if op == "wgrad":
        case["normed"] = dtype == "f32" and rng.random() < 0.5
    return case


# ----------------------------------------------------------------- inputs --
def _scale_bits(amax, fmt):
    """e + 127 of each group from its largest magnitude (float32 arithmetic
    on powers of two only: exact)."""
    m, e = torch.frexp(amax)                       # amax = m * 2^e, 0.5 <= m < 1
    top_m, top_e = math.frexp(TOP[fmt])
    e = e - top_e + (m > top_m).to(e.dtype)
    return torch.where(amax > 0, e.clamp(min=-127) + 127, torch.zeros_like(e)).to(torch.uint8)


def _pow2(bits):
    """2^(byte - 127) in float32, from its bits (a power function may be off by one)."""
    b = bits.to(torch.int32)
    return torch.where(b > 0, b << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _pack(x, fmt):
    g = x.float().reshape(*x.shape[:-1], -1, GROUP)
    bits = _scale_bits(g.abs().amax(-1), fmt)
    v = g * (1.0 / _pow2(bits))[..., None]
    q = v.round().to(torch.int8) if fmt == "i8" else v.to(torch.float8_e4m3fn)
    return q.reshape(x.shape), bits


def _unpack(q, bits):
    g = q.float().reshape(*q.shape[:-1], -1, GROUP)
    return (g * _pow2(bits)[..., None]).reshape(q.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = DTYPE[case["dtype"]]
    op, keep = case["op"], case["keep"]
    T, d = case["rows"], case["d"]

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=gen)
        return x.to(dtype)

    s = dict(case=case)
    if op in ("resid_fwd", "resid_bwd"):
        if case["affine"]:
            s["weight"] = normal(d, std=0.2, mean=1.0)
            s["bias"] = normal(d, std=0.1) if case["norm"] == "layer" else None
        # a residual stream: channels of unequal size, rows off centre
        spread = torch.exp(normal(d, std=0.5))
        if op == "resid_fwd":
            s["X"] = (normal(T, d) * spread + 0.3 * normal(T, 1)).to(t)
            s["B"] = normal(T, d, std=0.5, dtype=t)
        else:
            H = (normal(T, d) * spread + 0.3 * normal(T, 1)).to(t)
            s["mean"], s["rstd"] = _stats64(H, case["norm"])
            s["dY"] = normal(T, d, std=0.1, dtype=t)
            s["dH"] = normal(T, d, std=0.1, dtype=t)
            s["H"], s["H_qs"] = (H, None) if keep == "none" else _pack(H, keep)
            if case["scaled"]:
                B = normal(T, d, std=0.5, dtype=t)
                s["B"], s["B_qs"] = (B, None) if keep == "none" else _pack(B, keep)
        if case["scaled"]:
            s["scale"] = normal(d, std=0.05, mean=0.7)
    elif op in ("gated_fwd", "gated_bwd"):
        h = case["heads"]
        if case["affine"]:
            s["weight"] = normal(h, d, std=0.2, mean=1.0)
            s["bias"] = normal(h, d, std=0.1) if case["norm"] == "layer" else None
        # retention outputs: the heads' decays give them unequal sizes
        size = torch.logspace(-1, 1, h, device="cuda").reshape(h, 1)
        O = (normal(T, h, d) * size).to(t)
        G = normal(T, h, d, std=1.5, dtype=t)
        if op == "gated_bwd":
            s["mean"], s["rstd"] = _stats64(O, case["norm"])
            s["dZ"] = normal(T, h, d, std=0.1, dtype=t)
        s["O"], s["O_qs"], s["G"], s["G_qs"] = O, None, G, None
        if op == "gated_bwd" and keep != "none":
            (s["O"], s["O_qs"]), (s["G"], s["G_qs"]) = _pack(O, keep), _pack(G, keep)
    elif op == "ckpt":
        s["X"] = (normal(T, d) * torch.exp(normal(d, std=0.5))).to(t)
    else:
        X = normal(T, d, dtype=t)
        s["q"], s["qs"] = _pack(X, keep)
        s["dY"] = normal(T, case["out"], std=0.1, dtype=t)
        if case["normed"]:
            s["mean"], s["rstd"] = _stats64(X, "layer")
            s["weight"] = normal(d, std=0.2, mean=1.0)
            s["bias"] = normal(d, std=0.1)
    return s


def _stats64(x, norm):
    """The forward's float32 statistics of each row (chunks of rows in 64 bits)."""
    rows = x.reshape(-1, x.shape[-1])
    mean = torch.empty(rows.shape[0], dtype=torch.float32, device=x.device)
    rstd = torch.empty_like(mean)
    step = max(1, 2 ** 25 // rows.shape[1])
    for i in range(0, rows.shape[0], step):
        r = rows[i:i + step].double()
        mu = r.mean(-1, keepdim=True) if norm == "layer" else torch.zeros_like(r[:, :1])
        mean[i:i + step] = mu[:, 0].float()
        rstd[i:i + step] = (1.0 / torch.sqrt(((r - mu) ** 2).mean(-1) + EPS)).float()
    lead = x.shape[:-1]
    return (mean.reshape(lead) if norm == "layer" else None), rstd.reshape(lead)


# ------------------------------------------------------------ plain forms --
def _plain_norm(h, norm):
    mu = h.mean(-1, keepdim=True) if norm == "layer" else None
    c = h if mu is None else h - mu
    r = 1.0 / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS)
    return c * r, mu, r


def _present(*xs):
    return [x for x in xs if x is not None]


def _plain(s):
    case = s["case"]
    t = DTYPE[case["dtype"]]
    op, keep = case["op"], case["keep"]
    w, c = s.get("weight"), s.get("bias")
    if op == "resid_fwd":
        b = s["B"].float()
        if case["scaled"]:
            b = b * s["scale"]
        H = (s["X"].float() + b).to(t)
        xh, mu, r = _plain_norm(H.float(), case["norm"])
        y = xh if w is None else xh * w
        y = y if c is None else y + c
        kept = None if keep == "none" else _unpack(*_pack(H, keep)).to(t)
        return _present(y.to(t), H, None if mu is None else mu[:, 0], r[:, 0], kept)
    if op == "resid_bwd":
        h = s["H"].float() if keep == "none" else _unpack(s["H"], s["H_qs"])
        r = s["rstd"][:, None]
        xh = h * r if s["mean"] is None else (h - s["mean"][:, None]) * r
        dy = s["dY"].float()
        g = dy if w is None else dy * w
        u = g - xh * (g * xh).mean(-1, keepdim=True)
        if case["norm"] == "layer":
            u = u - g.mean(-1, keepdim=True)
        dh = s["dH"].float() + r * u
        out = [dh.to(t)]
        if case["scaled"]:
            b = s["B"].float() if keep == "none" else _unpack(s["B"], s["B_qs"])
            out += [(dh * s["scale"]).to(t), (dh * b).sum(0, dtype=torch.float64).float()]
        if w is not None:
            out.append((dy * xh).sum(0, dtype=torch.float64).float())
        if c is not None:
            out.append(dy.sum(0, dtype=torch.float64).float())
        return out
    if op == "gated_fwd":
        xh, mu, r = _plain_norm(s["O"].float(), case["norm"])
        n = xh if w is None else xh * w
        n = n if c is None else n + c
        g = s["G"].float()
        z = (n * (g / (1.0 + torch.exp(-g)))).to(t)
        kept = [] if keep == "none" else [_unpack(*_pack(s[k], keep)).to(t) for k in ("O", "G")]
        return _present(z, None if mu is None else mu[..., 0], r[..., 0], *kept)
    if op == "gated_bwd":
        o, g = (s[k].float() if keep == "none" else _unpack(s[k], s[k + "_qs"]) for k in ("O", "G"))
        r = s["rstd"][..., None]
        xh = o * r if s["mean"] is None else (o - s["mean"][..., None]) * r
        n = xh if w is None else xh * w
        n = n if c is None else n + c
        sg = 1.0 / (1.0 + torch.exp(-g))
        dz = s["dZ"].float()
        dn = dz * (g * sg)
        dG = dz * n * (sg * (1.0 + g * (1.0 - sg)))
        u = dn if w is None else dn * w
        v = u - xh * (u * xh).mean(-1, keepdim=True)
        if case["norm"] == "layer":
            v = v - u.mean(-1, keepdim=True)
        out = [(r * v).to(t), dG.to(t)]
        if w is not None:
            out.append((dn * xh).sum(0, dtype=torch.float64).float())
        if c is not None:
            out.append(dn.sum(0, dtype=torch.float64).float())
        if case["again"]:
            out.append((n * (g * sg)).to(t))
        return out
    if op == "ckpt":
        return [_unpack(*_pack(s["X"], keep)).to(t)]
    x = _unpack(s["q"], s["qs"])
    if case["normed"]:
        x = (x - s["mean"][:, None]) * s["rstd"][:, None] * w + c
    return [x.t() @ s["dY"].float()]


# -------------------------------------------------- the library's kernels --
def _library(s):
    import linear_recurrence_sequence_amd as msr
    case = s["case"]
    t = DTYPE[case["dtype"]]
    op, keep = case["op"], case["keep"]
    w, c = s.get("weight"), s.get("bias")
    norm = msr.MSR_NORM_LAYER if case.get("norm", "layer") == "layer" else msr.MSR_NORM_RMS
    fmt = {"none": msr.MSR_Q_NONE, "e4m3": msr.MSR_Q_E4M3, "i8": msr.MSR_Q_I8}[keep]

    def f32(*shape):
        return torch.empty(shape, dtype=torch.float32, device="cuda")

    def kept(shape):
        return msr.msr_ckpt_empty(shape, fmt, "cuda") if fmt else (None, None)

    def back(q, qs):
        return None if q is None else msr.msr_ckpt_unpack(q, qs, t)

    if op == "resid_fwd":
        T, d = s["X"].shape
        mean = f32(T) if case["norm"] == "layer" else None
        rstd = f32(T)
        hq, hqs = kept((T, d))
        Y, H = msr.msr_resid_norm_fwd(s["X"], s["B"], scale=s.get("scale"), weight=w, bias=c, norm=norm, eps=EPS,
                                      mean=mean, rstd=rstd, H_q=hq, H_qs=hqs)
        return _present(Y, H, mean, rstd, back(hq, hqs))
    if op == "resid_bwd":
        d = case["d"]
        scaled = case["scaled"]
        dB = torch.empty_like(s["dY"]) if scaled else None
        ds, dw, dc = f32(d) if scaled else None, None if w is None else f32(d), None if c is None else f32(d)
        dX = msr.msr_resid_norm_bwd(s["dY"], s["H"], s["mean"], s["rstd"], H_qs=s["H_qs"], dH=s["dH"], B=s.get("B"),
                                    B_qs=s.get("B_qs"), scale=s.get("scale"), weight=w, norm=norm, dB=dB, dscale=ds,
                                    dweight=dw, dbias=dc)
        return _present(dX, dB, ds, dw, dc)
    if op == "gated_fwd":
        shape = s["O"].shape
        mean = f32(*shape[:-1]) if case["norm"] == "layer" else None
        rstd = f32(*shape[:-1])
        (oq, oqs), (gq, gqs) = kept(shape), kept(shape)
        Z = msr.msr_gated_norm_fwd(s["O"], s["G"], weight=w, bias=c, norm=norm, eps=EPS, mean=mean, rstd=rstd,
                                   O_q=oq, O_qs=oqs, G_q=gq, G_qs=gqs)
        return _present(Z, mean, rstd, back(oq, oqs), back(gq, gqs))
    if op == "gated_bwd":
        h, d = case["heads"], case["d"]
        dw, dc = None if w is None else f32(h, d), None if c is None else f32(h, d)
        Z = torch.empty_like(s["dZ"]) if case["again"] else None
        dO, dG = msr.msr_gated_norm_bwd(s["dZ"], s["O"], s["G"], s["mean"], s["rstd"], O_qs=s["O_qs"],
                                        G_qs=s["G_qs"], weight=w, bias=c, norm=norm, dweight=dw, dbias=dc, Z=Z)
        return _present(dO, dG, dw, dc, Z)
    if op == "ckpt":
        return [msr.msr_ckpt_unpack(*msr.msr_ckpt_pack(s["X"], fmt), t)]
    return [msr.msr_ckpt_wgrad(s["q"], s["qs"], s["dY"], mean=s.get("mean"), rstd=s.get("rstd"), weight=w, bias=c)]


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------- work --
def work(case):
    es = SIZE[case["dtype"]]
    op, keep = case["op"], case["keep"]
    T = case["rows"]
    cols = case["d"] * case.get("heads", 1)
    n = T * cols
    q = n + n // GROUP
    kept = 0 if keep == "none" else q
    held = es * n if keep == "none" else q
    stats = 4 * T * case.get("heads", 1) * (2 if case.get("norm", "layer") == "layer" else 1)
    cvec = 4 * cols * (0 if not case.get("affine") else 2 if case["norm"] == "layer" else 1)
    if op == "resid_fwd":
        # kept values are written in 8 bits and read back into the element type
        return dict(bytes=4 * es * n + stats + cvec + 4 * cols * case["scaled"] + (2 * q + es * n if kept else 0),
                    flops=10 * n)
    if op == "resid_bwd":
        b = (held + es * n + 8 * cols) if case["scaled"] else 0
        return dict(bytes=3 * es * n + held + stats + 2 * cvec + b, flops=15 * n)
    if op == "gated_fwd":
        return dict(bytes=3 * es * n + stats + cvec + 2 * (2 * q + es * n if kept else 0), flops=15 * n)
    if op == "gated_bwd":
        return dict(bytes=3 * es * n + 2 * held + stats + 2 * cvec + (es * n if case["again"] else 0), flops=30 * n)
    if op == "ckpt":
        return dict(bytes=2 * es * n + 2 * q, flops=4 * n)
    extra = 8 * T + 8 * cols if case["normed"] else 0
    return dict(bytes=q + es * T * case["out"] + 4 * cols * case["out"] + extra, flops=2 * n * case["out"])


# ------------------------------------------------------------------ exact --
def _two64(e):
    """2^e in 64 bits, from its bits."""
    return ((e + 1023) << 52).view(torch.float64)


def _held64(x, bits):
    """Stored values in 64 bits: themselves, or q * 2^(byte - 127)."""
    if bits is None:
        return x.double()
    return x.double() * _two64(bits.long() - 127).repeat_interleave(GROUP, dim=-1)


def _rounded64(x, keep):
    """What the 8-bit form keeps of x, from its definition: the smallest
    power of two that holds the group, then the nearest code."""
    v = x.double().reshape(-1, GROUP)
    top = v.abs().max(dim=1, keepdim=True).values
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / TOP[keep])).long()
    e = torch.where(top > TOP[keep] * _two64(e), e + 1, e)
    e = torch.where(top <= TOP[keep] * _two64(e - 1), e - 1, e).clamp(min=-127)
    v = v / _two64(e)
    if keep == "i8":
        return (torch.round(v) * _two64(e)).reshape(x.shape)
    # 3 bits behind the leading one, subnormals below 2^-6
    step = _two64(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent.long() - 4)
    return (torch.round(v / step) * step * _two64(e)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op, keep = case["op"], case["keep"]
    t = DTYPE[case["dtype"]]
    layer = case.get("norm") == "layer"
    one = torch.ones((), dtype=torch.float64, device="cuda")
    w = s["weight"].double() if s.get("weight") is not None else one
    c = s["bias"].double() if s.get("bias") is not None else 0 * one
    if op == "ckpt":
        return [_rounded64(s["X"], keep)]
    if op == "wgrad":
        x = _held64(s["q"], s["qs"])
        if case["normed"]:
            x = (x - s["mean"].double()[:, None]) * s["rstd"].double()[:, None] * w + c
        return [torch.matmul(x.transpose(0, 1).contiguous(), s["dY"].double())]

    def normalised(x):
        m = x.mean(dim=-1) if layer else torch.zeros_like(x[..., 0])
        q = 1.0 / torch.sqrt((x * x).mean(dim=-1) - m * m + EPS)
        return (x - m[..., None]) * q[..., None], m, q

    if op == "resid_fwd":
        f = s["scale"].double() if case["scaled"] else one
        H = s["X"].double() + f * s["B"].double()
        xh, m, q = normalised(H.to(t).double())   # the norm reads the sum as it is held
        out = [xh * w + c, H] + ([m] if layer else []) + [q]
        return out + ([None] if keep != "none" else [])   # kept: a rounding of a rounding, no 64-bit value
    if op == "gated_fwd":
        xh, m, q = normalised(s["O"].double())
        g = s["G"].double()
        out = [g * torch.sigmoid(g) * (xh * w + c)] + ([m] if layer else []) + [q]
        if keep != "none":
            out += [_rounded64(s["O"], keep), _rounded64(s["G"], keep)]
        return out
    r = s["rstd"].double()[..., None]
    m = s["mean"].double()[..., None] if s["mean"] is not None else 0 * one
    if op == "resid_bwd":
        xh = (_held64(s["H"], s["H_qs"]) - m) * r
        dy = s["dY"].double()
        g = dy * w
        d = case["d"]
        lead = g.sum(-1, keepdim=True) / d if layer else 0 * one
        dh = s["dH"].double() + r * (g - lead - xh * ((g * xh).sum(-1, keepdim=True) / d))
        out = [dh]
        if case["scaled"]:
            out += [dh * s["scale"].double(), (dh * _held64(s["B"], s["B_qs"])).sum(0)]
        if case["affine"]:
            out.append((dy * xh).sum(0))
        return out + ([dy.sum(0)] if s.get("bias") is not None else [])
    xh = (_held64(s["O"], s["O_qs"]) - m) * r
    g = _held64(s["G"], s["G_qs"])
    n = xh * w + c
    sw = g * torch.sigmoid(g)
    dz = s["dZ"].double()
    dG = dz * n * (torch.sigmoid(g) + sw * torch.sigmoid(-g))
    dn = dz * sw
    u = dn * w
    d = case["d"]
    lead = u.sum(-1, keepdim=True) / d if layer else 0 * one
    dO = r * (u - lead - xh * ((u * xh).sum(-1, keepdim=True) / d))
    out = [dO, dG]
    if case["affine"]:
        out.append((dn * xh).sum(0))
    if s.get("bias") is not None:
        out.append(dn.sum(0))
    return out + ([sw * n] if case["again"] else [])
