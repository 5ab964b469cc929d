"""Norms with gate and residual between retention cores, and activations
kept in 8 bits, against the float64 oracle (``oracle.training``).

Bounds.  An element-type output is off by at most half a step of its type on
the value (u: bf16 2^-8, fp32 2^-24, relative) plus the float32 arithmetic
before it: 48 * 2^-24 times the value's *size* (the oracle's bound on its
terms).  48: a row's sum adds at most 8 * 2 values per lane, 6 exchanges and
8 waves (30 roundings; a mean enters twice at most, through mu and through
m1 or m2, whose terms the size holds separately), the root, division,
sigmoid (2 ulp exp2, 1 ulp reciprocal, their products) and the last products
add fewer than 18.  Column sums add the rows a thread walks one after the
other and then the walkers in 64 bits: 48 + that chain.  Kept values, codes
and the residual sum are compared bit by bit."""
import numpy as np
import pytest

import oracle
import workloads
from gpu_util import dev, host, say, torch_dtype
from oracle import training as ot

pytestmark = pytest.mark.gpu

U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
E32 = 2.0 ** -24
OPS = 48
FMTS = ["none", "e4m3", "i8"]


def _msr():
    import linear_recurrence_sequence_amd as msr
    return msr


def _fmt(fmt):
    msr = _msr()
    return {"none": msr.MSR_Q_NONE, "e4m3": msr.MSR_Q_E4M3, "i8": msr.MSR_Q_I8}[fmt]


def _norm(layer):
    msr = _msr()
    return msr.MSR_NORM_LAYER if layer else msr.MSR_NORM_RMS


def f32(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()


def empty32(*shape):
    import torch
    return torch.full(shape, float("nan"), dtype=torch.float32, device="cuda")


def within(name, got, want, size, dtype, ops=OPS):
    got, want = host(got), np.asarray(want, np.float64)
    assert got.shape == want.shape, name
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), name
    tol = U[dtype] * np.abs(want) + ops * E32 * size + 2.0 ** -133
    bad = np.abs(got - want) > tol
    worst = np.nanmax(np.abs(got - want) / tol) if got.size else 0.0
    print(f"{name}: {worst:.3f} of the bound", flush=True)
    assert not np.any(bad), (name, worst)


def same_bits(name, got, want):
    """got (tensor) equals want (float64 values exact in got's type), NaN where NaN."""
    got = host(got)
    assert np.array_equal(got, np.asarray(want, np.float64), equal_nan=True), \
        (name, int(np.sum(~((got == want) | (np.isnan(got) & np.isnan(want))))))


def keep(x, fmt):
    """A tensor kept in 8 bits by the library: (q, qs, the values it stands for by the oracle)."""
    msr = _msr()
    q, qs = msr.msr_ckpt_pack(x, _fmt(fmt))
    return q, qs, ot.q_unpack(*ot.q_pack(host(x), fmt))


def normal(rng, shape, dtype, std=1.0):
    return workloads.normal(rng, shape, std, dtype)


# ------------------------------------------------------------- 8-bit form --
@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (5, 7, 96), (2, 33, 4, 64), (257, 320), (1, 8192), (1030, 2560)])
def test_pack_and_unpack_bits(fmt, dtype, shape):
    import torch
    msr = _msr()
    rng = np.random.default_rng(sum(shape))
    x = normal(rng, shape, "f32") * np.exp2(rng.integers(-12, 12, shape[:-1] + (1,))).astype(np.float32)
    say("ckpt", fmt, dtype, shape)
    X = dev(x, dtype)
    q, qs = msr.msr_ckpt_pack(X, _fmt(fmt))
    wq, wqs = ot.q_pack(host(X), fmt)
    assert np.array_equal(qs.cpu().numpy(), wqs)
    same_bits("q", q, wq)
    want = ot.q_unpack(wq, wqs)
    same_bits("f32", msr.msr_ckpt_unpack(q, qs, torch.float32), want)
    same_bits("bf16", msr.msr_ckpt_unpack(q, qs), want)


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pack_special_values(fmt, dtype):
    """Zeros, signed zeros, ties, the borders of an exponent, the type's largest and smallest values, subnormals,
    infinities and NaN."""
    import torch
    msr = _msr()
    top = ot.Q_TOP[fmt]
    rng = np.random.default_rng(5)
    rows = np.zeros((24, 32), np.float32)
    rows[1] = -0.0
    rows[2] = top
    rows[3] = top * 2.0 ** -30
    rows[4, 3] = top * (1 + 2.0 ** -7)                     # just past a border, in bf16 too
    rows[5] = np.linspace(-top, top, 32)
    codes = ot.e4m3_values()[:126] if fmt == "e4m3" else np.arange(0.0, 127.0)
    mid = (codes[:-1] + codes[1:]) / 2
    for i in range(4):                                     # ties between neighbouring codes, exact in bf16
        rows[6 + i, :31] = mid[31 * i:31 * i + 31][:31]
        rows[6 + i, 31] = top
    rows[10] = 3.3e38
    rows[11, 0] = np.finfo(np.float32).max if dtype == "f32" else 3.3895314e38
    rows[12] = 2.0 ** -126
    rows[13] = 2.0 ** -133                                 # bf16's smallest subnormal
    rows[14, :8] = 1.4e-45 if dtype == "f32" else 2.0 ** -133
    rows[15] = rng.standard_normal(32) * 2.0 ** -125
    rows[16, 7] = np.inf
    rows[17, 31] = -np.inf
    rows[18, 0] = np.nan
    rows[19] = np.nan
    rows[20] = rng.standard_normal(32) * 2.0 ** -120
    rows[21, 5] = 1.0
    rows[22] = np.tile([1.0, -1.0], 16)
    rows[23] = rng.standard_normal(32)
    say("ckpt special values", fmt, dtype)
    X = torch.from_numpy(rows).cuda().to(torch_dtype(dtype))
    q, qs = msr.msr_ckpt_pack(X, _fmt(fmt))
    wq, wqs = ot.q_pack(host(X), fmt)
    assert np.array_equal(qs.cpu().numpy(), wqs)
    same_bits("q", q, wq)
    out = msr.msr_ckpt_unpack(q, qs, torch.float32)
    same_bits("values", out, ot.q_unpack(wq, wqs).astype(np.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_unpack_normalises(dtype):
    msr = _msr()
    rng = np.random.default_rng(8)
    T, d = 37, 192
    x = dev(normal(rng, (T, d), dtype, 2.0) + 1, dtype)
    w, c = 1 + 0.3 * rng.standard_normal(d), rng.standard_normal(d)
    for fmt in ("e4m3", "i8"):
        q, qs, xv = keep(x, fmt)
        mu, r = (v.astype(np.float32) for v in ot.norm_stats(xv, True, 1e-5))
        for use in ((1, 1, 1, 1), (0, 1, 0, 0), (0, 0, 1, 0), (1, 0, 0, 1), (0, 1, 1, 0)):
            say("unpack", dtype, fmt, use)
            m_, r_ = mu if use[0] else 0 * mu, r if use[1] else 1 + 0 * r
            w_, c_ = np.float32(w if use[2] else 1 + 0 * w), np.float32(c if use[3] else 0 * c)
            xh, size = ot.normalised(xv, m_, r_)
            got = msr.msr_ckpt_unpack(q, qs, torch_dtype(dtype), mean=f32(mu) if use[0] else None,
                                      rstd=f32(r) if use[1] else None, weight=f32(w_) if use[2] else None,
                                      bias=f32(c_) if use[3] else None)
            within("y", got, xh * w_ + c_, size * np.abs(w_) + np.abs(c_), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", [(1, 32), (8, 96), (9, 1024), (17, 1056), (16, 2080), (65, 320), (1, 8192), (7, 33344)])
def test_unpack_normalises_any_width(T, d, dtype):
    """Widths that whole rows share a workgroup in, that are cut in equal and unequal pieces, and row counts about
    those a workgroup takes; nothing is written beside the result."""
    import torch
    msr = _msr()
    rng = np.random.default_rng(T + d)
    q, qs, xv = keep(dev(normal(rng, (T, d), dtype, 2.0) + 1, dtype), "i8" if d % 64 else "e4m3")
    mu, r = (v.astype(np.float32) for v in ot.norm_stats(xv, True, 1e-5))
    w, c = (1 + 0.3 * rng.standard_normal(d)).astype(np.float32), rng.standard_normal(d).astype(np.float32)
    say("unpack", dtype, T, d)
    out, check = _guarded((T, d), torch_dtype(dtype))
    got = msr.msr_ckpt_unpack(q, qs, mean=f32(mu), rstd=f32(r), weight=f32(w), bias=f32(c), out=out)
    torch.cuda.synchronize()
    xh, size = ot.normalised(xv, mu, r)
    within("y", got, xh * w + c, size * np.abs(w) + np.abs(c), dtype)
    check()


# ------------------------------------------------------------- resid norm --
SHAPES = [(1, 64), (5, 64), (67, 128), (2, 192), (33, 256), (7, 320), (9, 512), (70, 576), (5, 1024), (3, 2560),
          (13, 4096), (6, 4160), (3, 8192), (3001, 256), (1500, 1088)]


def _resid_inputs(T, d, dtype, seed):
    rng = np.random.default_rng(seed)
    x = normal(rng, (T, d), dtype) * 2 + 0.5
    b = normal(rng, (T, d), dtype)
    vec = lambda m, s: (m + s * rng.standard_normal(d)).astype(np.float32)
    return dev(x, dtype), dev(b, dtype), vec(0.8, 0.1), vec(1, 0.3), vec(0, 0.3), rng


def _sum32(x, b, scale, alpha, dtype):
    """The residual sum, product and sum each rounded to float32, then to the type: exact values."""
    import torch
    h = np.float32(alpha) * host(x).astype(np.float32)
    if b is not None:
        h = h + (host(b).astype(np.float32) * scale if scale is not None else host(b).astype(np.float32))
    return torch.from_numpy(h).to(torch_dtype(dtype)).double().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_resid_norm_fwd(T, d, dtype):
    msr = _msr()
    x, b, scale, w, c, _ = _resid_inputs(T, d, dtype, T + d)
    for i, (layer, fmt, opts) in enumerate([(True, "none", "bswc"), (False, "e4m3", "bsw"), (True, "i8", "bc"),
                                            (False, "none", ""), (True, "e4m3", "wc"), (False, "i8", "bswc")]):
        alpha = 1.0 if i % 2 else 0.75
        say("resid fwd", dtype, T, d, layer, fmt, opts, alpha)
        B, S = (b if "b" in opts else None), (scale if "s" in opts else None)
        mean, rstd = empty32(T), empty32(T)
        kept = {}
        if fmt != "none":
            kept["H_q"], kept["H_qs"] = msr.msr_ckpt_empty((T, d), _fmt(fmt), "cuda")
            if B is not None:
                kept["B_q"], kept["B_qs"] = msr.msr_ckpt_empty((T, d), _fmt(fmt), "cuda")
        Y, H = msr.msr_resid_norm_fwd(x, B, scale=None if S is None else f32(S), weight=f32(w) if "w" in opts else None,
                                      bias=f32(c) if "c" in opts else None, alpha=alpha, norm=_norm(layer), eps=1e-5,
                                      mean=mean, rstd=rstd, **kept)
        h = _sum32(x, B, S, alpha, dtype)
        same_bits("H", H, h)
        assert (H is x) == (B is None and alpha == 1.0)
        y, size, mu, r = ot.resid_norm(h, layer, 1e-5, w if "w" in opts else 1.0, c if "c" in opts else 0.0)
        within("Y", Y, y, size, dtype)
        within("rstd", rstd, r, r, "f32")
        if layer:
            within("mean", mean, mu, np.abs(h).mean(-1), "f32")
        else:
            assert bool(mean.isnan().all())                       # not written
        if fmt != "none":
            for q, qs, v in ((kept["H_q"], kept["H_qs"], h),) + (
                    ((kept["B_q"], kept["B_qs"], host(b)),) if B is not None else ()):
                wq, wqs = ot.q_pack(v, fmt)
                assert np.array_equal(qs.cpu().numpy(), wqs)
                same_bits("kept", q, wq)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,d", SHAPES)
def test_resid_norm_bwd(T, d, fmt, dtype):
    msr = _msr()
    H, b, scale, w, _, rng = _resid_inputs(T, d, dtype, 2 * T + d)
    dy, dh = dev(normal(rng, (T, d), dtype, 0.2), dtype), dev(normal(rng, (T, d), dtype, 0.2), dtype)
    hq, hs, hv = (H, None, host(H)) if fmt == "none" else keep(H, fmt)
    bq, bs, bv = (b, None, host(b)) if fmt == "none" else keep(b, fmt)
    for layer, opts, alpha in ((True, "hswcB", 1.0), (False, "hsw", 0.6), (True, "", 1.0), (True, "wc", -1.5),
                               (False, "hsB", 1.0), (True, "hB", 2.0)):
        say("resid bwd", dtype, fmt, T, d, layer, opts, alpha)
        mu, r = (v.astype(np.float32) for v in ot.norm_stats(host(H), layer, 1e-5))
        ds, dw, dc = (empty32(d) if k in opts else None for k in "swc")
        dB = empty32(T, d).to(torch_dtype(dtype)) if "B" in opts else None
        s = scale if "s" in opts else 1.0 + 0 * scale
        dX = msr.msr_resid_norm_bwd(dy, hq, f32(mu) if layer else None, f32(r), H_qs=hs, dH=dh if "h" in opts else None,
                                    B=bq if "s" in opts else None, B_qs=bs if "s" in opts else None,
                                    scale=f32(scale) if "s" in opts else None, weight=f32(w) if "w" in opts else None,
                                    alpha=alpha, norm=_norm(layer), dB=dB, dscale=ds, dweight=dw, dbias=dc)
        ref = ot.resid_norm_grad(host(dy), hv, mu, r, layer, host(dh) if "h" in opts else 0.0,
                                 w if "w" in opts else 1.0, bv)
        g, size = ref["dh"]
        al = float(np.float32(alpha))
        within("dX", dX, al * g, abs(al) * size, dtype)
        if dB is not None:
            within("dB", dB, s * g, np.abs(s) * size, dtype)
        chain = OPS + T // 256 + 64                               # rows a thread walks, and its workgroup's rows
        for name, t in (("dscale", ds), ("dweight", dw), ("dbias", dc)):
            if t is not None:
                within(name, t, *ref[name], "f32", ops=chain)


# ------------------------------------------------------------- gated norm --
GATED = [(1, 1, 64), (1, 16, 512), (5, 3, 64), (37, 4, 64), (9, 5, 128), (130, 1, 128), (6, 10, 256), (33, 8, 256),
         (7, 3, 512), (11, 16, 512), (3000, 2, 64), (700, 7, 128), (260, 128, 64), (21, 5, 256), (17, 1, 512), (19, 2, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,d", GATED)
def test_gated_norm(T, H, d, dtype):
    import torch
    msr = _msr()
    rng = np.random.default_rng(T + 7 * H + d)
    size = np.exp2(np.linspace(-3, 3, H))[:, None]
    O = dev(normal(rng, (T, H, d), "f32") * size + 0.3, dtype)
    G = dev(normal(rng, (T, H, d), dtype, 2.0), dtype)
    dz = dev(normal(rng, (T, H, d), dtype, 0.2), dtype)
    w = (1 + 0.3 * rng.standard_normal((H, d))).astype(np.float32)
    c = (0.3 * rng.standard_normal((H, d))).astype(np.float32)
    for layer, fmt, opts in ((True, "none", "wcz"), (False, "e4m3", "w"), (True, "i8", "cz"), (False, "none", ""),
                             (True, "e4m3", "wcz")):
        say("gated", dtype, T, H, d, layer, fmt, opts)
        wn, cn = (w if "w" in opts else 1.0), (c if "c" in opts else 0.0)
        kw = dict(weight=f32(w) if "w" in opts else None, bias=f32(c) if "c" in opts else None, norm=_norm(layer))
        mean, rstd = empty32(T, H), empty32(T, H)
        kept = {}
        if fmt != "none":
            kept["O_q"], kept["O_qs"] = msr.msr_ckpt_empty((T, H, d), _fmt(fmt), "cuda")
            kept["G_q"], kept["G_qs"] = msr.msr_ckpt_empty((T, H, d), _fmt(fmt), "cuda")
        Z = msr.msr_gated_norm_fwd(O, G, eps=1e-5, mean=mean, rstd=rstd, **kept, **kw)
        z, zs, mu, r = ot.gated_norm(host(O), host(G), layer, 1e-5, wn, cn)
        within("Z", Z, z, zs, dtype)
        within("rstd", rstd, r, r, "f32")
        if layer:
            within("mean", mean, mu, np.abs(host(O)).mean(-1), "f32")
        o, g, ov, gv, oqs, gqs = O, G, host(O), host(G), None, None
        if fmt != "none":
            o, oqs, g, gqs = kept["O_q"], kept["O_qs"], kept["G_q"], kept["G_qs"]
            for x, q, qs in ((O, o, oqs), (G, g, gqs)):
                wq, wqs = ot.q_pack(host(x), fmt)
                assert np.array_equal(qs.cpu().numpy(), wqs)
                same_bits("kept", q, wq)
            ov, gv = (ot.q_unpack(*ot.q_pack(host(x), fmt)) for x in (O, G))
        dw, dc = (empty32(H, d) if k in opts else None for k in "wc")
        Z2 = torch.empty_like(dz) if "z" in opts else None
        dO, dG = msr.msr_gated_norm_bwd(dz, o, g, mean if layer else None, rstd, O_qs=oqs, G_qs=gqs, Z=Z2, dweight=dw,
                                        dbias=dc, **kw)
        m32 = host(mean) if layer else 0.0 * host(rstd)
        ref = ot.gated_norm_grad(host(dz), ov, gv, m32, host(rstd), layer, wn, cn)
        within("dO", dO, *ref["do"], dtype)
        within("dG", dG, *ref["dg"], dtype)
        chain = OPS + T // 64 + 32                                # tokens a thread walks, and its workgroup's tokens
        for name, t in (("dweight", dw), ("dbias", dc)):
            if t is not None:
                within(name, t, *ref[name], "f32", ops=chain)
        if Z2 is not None:
            within("Z again", Z2, *ref["z"], dtype)
            if fmt == "none":
                # the same expression from stored statistics: at most both roundings apart
                within("Z of both passes", Z2, host(Z), 4 * np.abs(host(Z)) * U[dtype] / E32 / OPS + zs, dtype)


# ----------------------------------------------------------------- wgrad --
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,i,o", [(1, 64, 64), (63, 64, 128), (64, 128, 64), (65, 192, 320), (200, 320, 192),
                                   (1000, 64, 64), (1023, 256, 512), (4097, 128, 192), (8256, 192, 64)])
def test_wgrad(T, i, o, dtype):
    """Exact products of the kept values and dY, added in float32: at most one rounding a token of the sum of
    their magnitudes (the matrix cores' order is unspecified), + OPS.  Normalised bf16: each x rounded, too."""
    msr = _msr()
    rng = np.random.default_rng(T + i + o)
    x = dev(normal(rng, (T, i), dtype), dtype)
    dy = dev(normal(rng, (T, o), dtype, 0.3), dtype)
    w, c = (1 + 0.3 * rng.standard_normal(i)).astype(np.float32), (0.3 * rng.standard_normal(i)).astype(np.float32)
    old = rng.standard_normal((i, o)).astype(np.float32)
    for fmt, acc, normed in (("e4m3", False, False), ("i8", True, False), ("i8", False, True)):
        say("wgrad", dtype, T, i, o, fmt, acc, normed)
        q, qs, xv = keep(x, fmt)
        kw, xs = {}, np.abs(xv)
        rounded = 0.0
        if normed:
            mu, r = (v.astype(np.float32) for v in ot.norm_stats(xv, True, 1e-5))
            kw = dict(mean=f32(mu), rstd=f32(r), weight=f32(w), bias=f32(c))
            xv, xs = ot.normalised(xv, mu, r)
            xv, xs = xv * w + c, xs * np.abs(w) + np.abs(c)
            rounded = U[dtype] * (np.abs(xv).T @ np.abs(host(dy)))
        dW = msr.msr_ckpt_wgrad(q, qs, dy, dW=f32(old) if acc else None, accumulate=acc, **kw)
        want = xv.T @ host(dy) + (old if acc else 0.0)
        size = xs.T @ np.abs(host(dy)) + np.abs(old) * acc
        within("dW", dW, want, size + rounded / (E32 * (OPS + T)), "f32", ops=OPS + T)


@pytest.mark.parametrize("T", [2048, 2049, 3000, 3105])
def test_wgrad_on_large_tiles(T):
    """bf16 on the 256 x 256 tiles: whole slabs, one token in the last slab, slices of unequal length, a last slab
    half full.  The same bound as above; the reference products in float64 (torch, on the GPU)."""
    import torch
    msr = _msr()
    rng = np.random.default_rng(T)
    i, o = 2048, 4096
    x, dy = dev(normal(rng, (T, i), "bf16"), "bf16"), dev(normal(rng, (T, o), "bf16", 0.3), "bf16")
    say("wgrad on large tiles", T)
    q, qs = msr.msr_ckpt_pack(x, msr.MSR_Q_I8)
    dW = msr.msr_ckpt_wgrad(q, qs, dy)
    xv = msr.msr_ckpt_unpack(q, qs, torch.float32).double().t().contiguous()
    dyd = dy.double()
    err, size = (dW.double() - xv @ dyd).abs(), xv.abs() @ dyd.abs()
    assert bool((err <= (OPS + T) * E32 * size).all()), float((err / size).max() / E32)
    # most entries are far below the bound: a wrong or missing slab is not
    assert float((err / size).mean()) < 4 * E32


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("normed", [False, True])
def test_wgrad_single_products(dtype, normed):
    """One token: dW is one product an entry.  float32 dY is taken in three bf16 cuts and a weighted X too, so a
    missing cut would show as 2^-16 of the product: at most 8 roundings (six products' sum, the weighted x, the
    result) of 2^-24 each are allowed, for bf16 also the rounding of the weighted x."""
    msr = _msr()
    rng = np.random.default_rng(17)
    i, o = 192, 320
    x, dy = dev(normal(rng, (1, i), "f32") + 3, dtype), dev(normal(rng, (1, o), "f32") + 3, dtype)
    w = (1 + 0.3 * rng.standard_normal(i)).astype(np.float32)
    for fmt in ("e4m3", "i8"):
        say("single products", dtype, normed, fmt)
        q, qs, xv = keep(x, fmt)
        dW = host(msr.msr_ckpt_wgrad(q, qs, dy, weight=f32(w) if normed else None))
        want = (xv * (w.astype(np.float64) if normed else 1.0)).T @ host(dy)
        rel = 8 * E32 + (U["bf16"] if normed and dtype == "bf16" else 0.0)
        assert np.all(np.abs(dW - want) <= rel * np.abs(want)), np.max(np.abs(dW - want) / np.abs(want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_wgrad_keeps_bad_values_in_their_row_and_column(dtype):
    """A group that reads back as NaN spoils the rows of dW of its 32 inputs, an infinity or a NaN in dY the columns of
    its output; the padding of ragged tokens and of other rows spoils nothing."""
    msr = _msr()
    T, i, o = 77, 128, 192
    rng = np.random.default_rng(19)
    x, dy = normal(rng, (T, i), dtype), normal(rng, (T, o), dtype)
    x[76, 40], dy[75, 3], dy[76, 100] = np.nan, np.inf, np.nan
    say("wgrad with bad values", dtype)
    q, qs, xv = keep(dev(x, dtype), "e4m3")
    dW = host(msr.msr_ckpt_wgrad(q, qs, dev(dy, dtype)))
    bad = np.zeros((i, o), bool)
    bad[32:64], bad[:, [3, 100]] = True, True
    assert np.array_equal(~np.isfinite(dW), bad)
    xg, dg = np.delete(xv, np.arange(32, 64), 1), np.delete(dy.astype(np.float64), [3, 100], 1)
    got = np.delete(np.delete(dW, np.arange(32, 64), 0), [3, 100], 1)
    assert np.all(np.abs(got - xg.T @ dg) <= (OPS + T) * E32 * (np.abs(xg).T @ np.abs(dg)))


# ----------------------------------------------------- limits and isolation --
@pytest.mark.parametrize("normed", [False, True])
def test_wgrad_of_tiny_gradients(normed):
    """float32 gradients down to its smallest: each is taken to 2^-133 (X is 1; normalised, to 2^-25 of it as well)."""
    import torch
    msr = _msr()
    T = 64
    e, m = np.meshgrid(np.arange(-149, -85), 1 + 2.0 ** -np.arange(1.0, 24.0))
    v = np.resize((m * 2.0 ** e).ravel(), (64 * 23,)).astype(np.float32)
    say("wgrad of tiny gradients", normed)
    q, qs = msr.msr_ckpt_pack(torch.ones(T, 64, device="cuda"))
    kw = dict(rstd=torch.ones(T, device="cuda")) if normed else {}
    dW = host(msr.msr_ckpt_wgrad(q, qs, torch.from_numpy(v).cuda().expand(T, -1).contiguous(), **kw))
    want = T * v.astype(np.float64)
    # T products of one sign: each sum rounds by half a unit of at most its end
    tol = T * 2.0 ** -133 + want * (T * E32 + (2.0 ** -25 if normed else 0))
    assert np.all(np.abs(dW - want) <= tol), np.max(np.abs(dW - want) / tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,i,o", [(65, 64, 128), (77, 64, 128), (100, 320, 192), (1000, 2048, 2048), (16383, 512, 8192)])
def test_wgrad_last_token_infinite(T, i, o, dtype):
    """An infinity in the last token's gradient gives infinities of its products' signs, however many tokens lie
    beside it in the last block of a reduction."""
    import torch
    msr = _msr()
    say("wgrad, last token infinite", dtype, T, i, o)
    gen = torch.Generator().manual_seed(T)
    x = torch.randn(T, i, generator=gen).cuda()
    x[-1] = torch.where(torch.arange(i, device="cuda") % 3 == 0, -2.0, 1.0)
    dY = torch.randn(T, o, generator=gen).cuda().to(torch_dtype(dtype))
    dY[-1, 5], dY[-1, 70] = float("inf"), float("-inf")
    q, qs = msr.msr_ckpt_pack(x)
    dW = msr.msr_ckpt_wgrad(q, qs, dY)
    sign = torch.sign(msr.msr_ckpt_unpack(q, qs, torch.float32)[-1])
    assert torch.equal(dW[:, 5], sign * float("inf")) and torch.equal(dW[:, 70], sign * float("-inf"))
    rest = torch.ones(o, dtype=torch.bool, device="cuda")
    rest[[5, 70]] = False
    assert bool(dW[:, rest].isfinite().all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_tokens(dtype):
    """No rows: nothing read, the sums over tokens are zero, an accumulated gradient stays."""
    import torch
    msr = _msr()
    t = torch_dtype(dtype)
    say("no tokens", dtype)
    X = torch.empty((0, 128), dtype=t, device="cuda")
    mean, rstd = empty32(0), empty32(0)
    Y, H = msr.msr_resid_norm_fwd(X, X, mean=mean, rstd=rstd)
    assert Y.shape == H.shape == (0, 128)
    ds, dw, dc = (empty32(128) for _ in range(3))
    msr.msr_resid_norm_bwd(X, X, mean, rstd, B=X, dscale=ds, dweight=dw, dbias=dc)
    O = torch.empty((2, 0, 3, 64), dtype=t, device="cuda")
    st = empty32(2, 0, 3)
    assert msr.msr_gated_norm_fwd(O, O).shape == O.shape
    gw, gc = empty32(3, 64), empty32(3, 64)
    msr.msr_gated_norm_bwd(O, O, O, st, st, dweight=gw, dbias=gc)
    q, qs = msr.msr_ckpt_pack(X)
    assert q.shape == (0, 128) and msr.msr_ckpt_unpack(q, qs).shape == (0, 128)
    dW = msr.msr_ckpt_wgrad(q, qs, X)
    old = torch.ones((128, 128), dtype=torch.float32, device="cuda")
    msr.msr_ckpt_wgrad(q, qs, X, dW=old, accumulate=True)
    torch.cuda.synchronize()
    for z in (ds, dw, dc, gw, gc, dW):
        assert bool((z == 0).all())
    assert bool((old == 1).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [256, 2560])
def test_bad_rows_stay_alone(d, fmt):
    """Rows with a NaN or an infinity spoil themselves and the sums over tokens, no other row; constant and zero
    rows give what the formula gives (variance 0, r = 1 / sqrt(eps))."""
    import torch
    msr = _msr()
    T = 41
    rng = np.random.default_rng(d)
    h = normal(rng, (T, d), "f32")
    h[3, 5], h[11, 0], h[17] = np.nan, np.inf, -np.inf
    h[20], h[21] = 0.0, 2.5
    dy, dh = (dev(normal(rng, (T, d), "f32"), "f32") for _ in range(2))
    say("bad rows", d, fmt)
    H = f32(h)
    kept = dict(zip(("H_q", "H_qs"), msr.msr_ckpt_empty((T, d), _fmt(fmt), "cuda"))) if fmt != "none" else {}
    mean, rstd = empty32(T), empty32(T)
    Y, _ = msr.msr_resid_norm_fwd(H, mean=mean, rstd=rstd, **kept)
    good = np.setdiff1d(np.arange(T), [3, 11, 17])
    y, size, mu, r = ot.resid_norm(h[good], True, 1e-5)
    within("Y", Y[good], y, size, "f32")
    assert bool(Y[[3, 11, 17]].isnan().all(dim=1).all())
    hv = h if fmt == "none" else ot.q_unpack(*ot.q_pack(h, fmt))
    dX = msr.msr_resid_norm_bwd(dy, kept.get("H_q", H), mean, rstd, H_qs=kept.get("H_qs"), dH=dh)
    ref = ot.resid_norm_grad(host(dy)[good], hv[good], host(mean)[good], host(rstd)[good], True, host(dh)[good])
    within("dX", dX[good], *ref["dh"], "f32")
    assert bool(dX[3].isnan().any())
    # gated: head-wise
    O, G = H[:, :256].reshape(T, 4, 64).contiguous(), dev(normal(rng, (T, 4, 64), "f32"), "f32")
    Z = msr.msr_gated_norm_fwd(O, G)
    ok = np.isfinite(h[:, :256].reshape(T, 4, 64)).all(-1)
    z, zs, _, _ = ot.gated_norm(host(O)[ok], host(G)[ok], True, 1e-5)
    within("Z", Z[torch.from_numpy(ok)], z, zs, "f32")
    # gates far out: swish and its slope go to g, 0 and 1, 0
    G = f32(np.tile(np.array([-1e4, -200.0, -88.0, 0.0, 88.0, 200.0, 1e4, 1e30], np.float32), (T, 4, 8)))
    O = dev(normal(rng, (T, 4, 64), "f32"), "f32")
    st, rs = empty32(T, 4), empty32(T, 4)
    Z = msr.msr_gated_norm_fwd(O, G, mean=st, rstd=rs)
    dO, dG = msr.msr_gated_norm_bwd(f32(np.full((T, 4, 64), 1e-3)), O, G, st, rs)
    assert bool(Z.isfinite().all()) and bool(dG.isfinite().all())


def _guarded(shape, dtype):
    """A tensor inside a larger buffer of a known pattern, and a check that nothing around it changed."""
    import torch
    n = int(np.prod(shape))
    pad = 256
    buf = torch.full((n + 2 * pad,), 77, dtype=torch.float32, device="cuda").to(dtype)
    before = buf.view(torch.uint8).clone()
    es = buf.element_size()

    def check():
        now = buf.view(torch.uint8)
        assert torch.equal(now[:pad * es], before[:pad * es]) and torch.equal(now[-pad * es:], before[-pad * es:])
    return buf[pad:pad + n].view(shape), check


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nothing_is_written_outside(dtype):
    """Outputs and workspaces inside larger buffers, at sizes that end inside a workgroup's rows and tiles."""
    import torch
    msr = _msr()
    t = torch_dtype(dtype)
    code = 1 if dtype == "bf16" else 0
    rng = np.random.default_rng(4)
    checks = []

    def out(shape, ty=t):
        v, c = _guarded(shape, ty)
        checks.append(c)
        return v
    for T, d in ((7, 64), (3, 320), (5, 576), (67, 192)):
        say("guards", dtype, T, d)
        X = dev(normal(rng, (T, d), dtype), dtype)
        mean, rstd = out((T,), torch.float32), out((T,), torch.float32)
        hq, hs, bq, bs = (out((T, d), torch.int8), out((T, d // 32), torch.uint8), out((T, d), torch.int8),
                          out((T, d // 32), torch.uint8))
        msr.msr_resid_norm_fwd(X, X, H=out((T, d)), Y=out((T, d)), mean=mean, rstd=rstd, H_q=hq, H_qs=hs, B_q=bq,
                               B_qs=bs)
        ws = out((msr.msr_resid_norm_bwd_workspace_bytes(T, d),), torch.uint8)
        msr.msr_resid_norm_bwd(X, hq, mean, rstd, H_qs=hs, B=bq, B_qs=bs, dX=out((T, d)), dB=out((T, d)),
                               dscale=out((d,), torch.float32), dweight=out((d,), torch.float32),
                               dbias=out((d,), torch.float32), workspace=ws)
        q, qs = msr.msr_ckpt_pack(X, msr.MSR_Q_I8, q=out((T, d), torch.int8), qs=out((T, d // 32), torch.uint8))
        msr.msr_ckpt_unpack(q, qs, out=out((T, d)))
        ws = out((msr.msr_ckpt_wgrad_workspace_bytes(code, T, d, d, accumulate=True),), torch.uint8)
        dW = out((d, d), torch.float32)
        dW.zero_()
        msr.msr_ckpt_wgrad(q, qs, X, dW=dW, accumulate=True, workspace=ws)
    for T, H, d in ((5, 3, 64), (3, 5, 512), (3, 7, 256), (65, 1, 64)):
        say("guards", dtype, T, H, d)
        O = dev(normal(rng, (T, H, d), dtype), dtype)
        mean, rstd = out((T, H), torch.float32), out((T, H), torch.float32)
        oq, os_, gq, gs = (out((T, H, d), torch.int8), out((T, H, d // 32), torch.uint8), out((T, H, d), torch.int8),
                           out((T, H, d // 32), torch.uint8))
        msr.msr_gated_norm_fwd(O, O, Z=out((T, H, d)), mean=mean, rstd=rstd, O_q=oq, O_qs=os_, G_q=gq, G_qs=gs)
        ws = out((msr.msr_gated_norm_bwd_workspace_bytes(T, H, d),), torch.uint8)
        msr.msr_gated_norm_bwd(O, oq, gq, mean, rstd, O_qs=os_, G_qs=gs, dO=out((T, H, d)), dG=out((T, H, d)),
                               Z=out((T, H, d)), dweight=out((H, d), torch.float32),
                               dbias=out((H, d), torch.float32), workspace=ws)
    torch.cuda.synchronize()
    for c in checks:
        c()


def test_large_offsets():
    """More than 2^31 values (and bytes): the last rows are where they belong."""
    import torch
    msr = _msr()
    T, d = 270000, 8192
    say("large offsets", T, d)
    X = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    tail = dev(normal(np.random.default_rng(3), (9, d), "bf16"), "bf16")
    X[-9:] = tail
    q, qs = msr.msr_ckpt_empty((T, d), msr.MSR_Q_I8, "cuda")
    mean, rstd = empty32(T), empty32(T)
    Y, H = msr.msr_resid_norm_fwd(X, mean=mean, rstd=rstd, H_q=q, H_qs=qs)
    Ys, _ = msr.msr_resid_norm_fwd(tail)
    assert torch.equal(Y[-9:], Ys) and not bool(Y[-20:-9].any())
    del Y
    assert torch.equal(msr.msr_ckpt_unpack(q, qs)[-9:], msr.msr_ckpt_unpack(*msr.msr_ckpt_pack(tail, msr.MSR_Q_I8)))
    q2, qs2 = msr.msr_ckpt_pack(X, msr.MSR_Q_I8)
    assert torch.equal(q2, q) and torch.equal(qs2, qs)
    del q2, qs2
    dX = msr.msr_resid_norm_bwd(X, q, mean, rstd, H_qs=qs)
    dXs = msr.msr_resid_norm_bwd(tail, *(lambda p: (p[0], mean[-9:].contiguous(), rstd[-9:].contiguous()))(
        msr.msr_ckpt_pack(tail, msr.MSR_Q_I8)), H_qs=qs[-9:].contiguous())
    assert torch.equal(dX[-9:], dXs)


# ---------------------------------------------------- streams, graphs, runs --
def _pass(msr, s, outs):
    """One training pass of both seams with everything kept in 8 bits; outs: its preallocated tensors."""
    o = outs
    msr.msr_resid_norm_fwd(s["x"], s["b"], scale=s["scale"], weight=s["w"], bias=s["c"], H=o["h"], Y=o["y"],
                           mean=o["m"], rstd=o["r"], H_q=o["hq"], H_qs=o["hs"], B_q=o["bq"], B_qs=o["bs"])
    msr.msr_gated_norm_fwd(o["y"].view(s["o4"]), s["g"], Z=o["z"], mean=o["m2"], rstd=o["r2"], O_q=o["oq"],
                           O_qs=o["os"], G_q=o["gq"], G_qs=o["gs"])
    msr.msr_gated_norm_bwd(s["dz"], o["oq"], o["gq"], o["m2"], o["r2"], O_qs=o["os"], G_qs=o["gs"], dO=o["do"],
                           dG=o["dg"], Z=o["z2"], dweight=o["gw"], dbias=o["gc"], workspace=o["ws2"])
    msr.msr_resid_norm_bwd(o["do"].view(s["x"].shape), o["hq"], o["m"], o["r"], H_qs=o["hs"], B=o["bq"], B_qs=o["bs"],
                           scale=s["scale"], weight=s["w"], dX=o["dx"], dB=o["db"], dscale=o["ds"], dweight=o["dw"],
                           dbias=o["dc"], workspace=o["ws1"])
    msr.msr_ckpt_wgrad(o["hq"], o["hs"], o["dx"], mean=o["m"], rstd=o["r"], weight=s["w"], bias=s["c"], dW=o["W"],
                       workspace=o["ws3"])


RESULTS = ("h", "y", "z", "z2", "do", "dg", "gw", "gc", "dx", "db", "ds", "dw", "dc", "W")


def _pass_state(T, H, d, seed):
    import torch
    msr = _msr()
    rng = np.random.default_rng(seed)
    D = H * d
    t = lambda *s, std=1.0: dev(normal(rng, s, "bf16", std), "bf16")
    s = dict(x=t(T, D), b=t(T, D), g=t(T, H, d), dz=t(T, H, d, std=0.3), scale=f32(0.7 + 0.1 * rng.standard_normal(D)),
             w=f32(1 + 0.1 * rng.standard_normal(D)), c=f32(0.1 * rng.standard_normal(D)), o4=(T, H, d))
    bf = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    o = dict(h=bf(T, D), y=bf(T, D), z=bf(T, H, d), z2=bf(T, H, d), do=bf(T, H, d), dg=bf(T, H, d), dx=bf(T, D),
             db=bf(T, D), m=empty32(T), r=empty32(T), m2=empty32(T, H), r2=empty32(T, H), gw=empty32(H, d),
             gc=empty32(H, d), ds=empty32(D), dw=empty32(D), dc=empty32(D), W=empty32(D, D))
    for n, shape in (("h", (T, D)), ("b", (T, D)), ("o", (T, H, d)), ("g", (T, H, d))):
        o[n + "q"], o[n + "s"] = msr.msr_ckpt_empty(shape, msr.MSR_Q_E4M3, "cuda")
    ws = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
    o["ws1"] = ws(msr.msr_resid_norm_bwd_workspace_bytes(T, D))
    o["ws2"] = ws(msr.msr_gated_norm_bwd_workspace_bytes(T, H, d))
    o["ws3"] = ws(msr.msr_ckpt_wgrad_workspace_bytes(1, T, D, D, normed=True))
    return s, o


def test_captured_pass_replays():
    """The pass captured once and replayed on other inputs, eager work between the replays: the same bits as the
    eager pass each time (also: two eager passes give the same bits)."""
    import torch
    msr = _msr()
    T, H, d = 333, 5, 64
    s, o = _pass_state(T, H, d, 11)
    _pass(msr, s, o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _pass(msr, s, o)
    for seed in (12, 13, 14):
        say("replay", seed)
        s2, o2 = _pass_state(T, H, d, seed)
        _pass(msr, s2, o2)
        torch.cuda.synchronize()
        want = {k: o2[k].clone() for k in RESULTS}
        _pass(msr, s2, o2)
        for k in ("x", "b", "g", "dz", "scale", "w", "c"):
            s[k].copy_(s2[k])
        graph.replay()
        torch.cuda.synchronize()
        for k in RESULTS:
            assert torch.equal(o[k], want[k]), k
            assert torch.equal(o2[k], want[k]), k


def test_other_stream():
    """On a stream that is not the current one (given as a stream and as a handle), with tensors the binding
    allocates: ordered with that stream's work, and its memory not reused before."""
    import torch
    msr = _msr()
    T, D = 4096, 1024
    rng = np.random.default_rng(2)
    x, b = (dev(normal(rng, (T, D), "bf16"), "bf16") for _ in range(2))
    mean, rstd = empty32(T), empty32(T)
    want, wh = msr.msr_resid_norm_fwd(x, b, mean=mean, rstd=rstd)
    dw, wdw = empty32(D), empty32(D)
    wdx = msr.msr_resid_norm_bwd(b, wh, mean, rstd, dweight=wdw)
    wW = msr.msr_ckpt_wgrad(*msr.msr_ckpt_pack(x), b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        say("stream", type(stream))
        big = torch.randn((4096, 4096), device="cuda")
        with torch.cuda.stream(side):
            for _ in range(4):                                  # the side stream is busy
                big = big @ big * 1e-4
        Y, Hh = msr.msr_resid_norm_fwd(x, b, stream=stream)
        dX = msr.msr_resid_norm_bwd(b, Hh, mean, rstd, dweight=dw, stream=stream)
        q, qs = msr.msr_ckpt_pack(x, stream=stream)
        W = msr.msr_ckpt_wgrad(q, qs, b, stream=stream)
        junk = [torch.full((T, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
        side.synchronize()
        assert torch.equal(Y, want) and torch.equal(Hh, wh) and torch.equal(dX, wdx) and torch.equal(dw, wdw)
        assert torch.equal(W, wW)
        del junk
    torch.cuda.synchronize()


def test_two_streams_at_once():
    """The same pass on two streams, each with its own tensors and workspaces, enqueued alternately."""
    import torch
    msr = _msr()
    T, H, d = 700, 3, 128
    want, sets = [], []
    for seed in (21, 22):
        s, o = _pass_state(T, H, d, seed)
        _pass(msr, s, o)
        torch.cuda.synchronize()
        want.append({k: o[k].clone() for k in RESULTS})
        sets.append(_pass_state(T, H, d, seed))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    say("two streams")
    for _ in range(4):
        for st, (s, o) in zip(streams, sets):
            with torch.cuda.stream(st):
                _pass(msr, s, o)
    torch.cuda.synchronize()
    for w, (_, o) in zip(want, sets):
        for k in RESULTS:
            assert torch.equal(o[k], w[k]), k


@pytest.mark.parametrize("dtype,fmt", [("f32", "none"), ("f32", "i8"), ("bf16", "none"), ("bf16", "e4m3")])
def test_training_step_of_a_block(dtype, fmt):
    """A block's forward and backward as they are used together: norm, projections, retention, gated norm, output
    projection, residual sum and the next norm; every gradient against the float64 formulas on the tensors that
    the step itself kept (its 8-bit ones read back), so that only the arithmetic in between is compared.  The
    retention core's own tolerance (1e-4 and 2e-2 of each gradient's largest value) holds for what passes it."""
    import math
    import torch
    msr = _msr()
    B, N, dm, H, d, chunk = 2, 96, 128, 2, 64, 32
    T = B * N
    tol = {"f32": 1e-4, "bf16": 2e-2}[dtype]
    rng = np.random.default_rng(31)
    t = torch_dtype(dtype)
    x = dev(normal(rng, (B, N, dm), dtype), dtype)
    W = {k: dev(normal(rng, (dm, H * d), dtype, dm ** -0.5), dtype) for k in "QKVG"}
    WO = dev(normal(rng, (H * d, dm), dtype, (H * d) ** -0.5), dtype)
    vec = lambda n, m: f32(m + 0.1 * rng.standard_normal(n))
    w1, c1, w2, c2, sc = vec(dm, 1), vec(dm, 0), vec(dm, 1), vec(dm, 0), vec(dm, 0.8)
    gw, gc = vec(H * d, 1).view(H, d), vec(H * d, 0).view(H, d)
    gam = workloads.gammas(H)
    s = 1 / math.sqrt(d)
    st = lambda *sh: empty32(*sh)
    kept = lambda *sh: msr.msr_ckpt_empty(sh, _fmt(fmt), "cuda") if fmt != "none" else (None, None)
    say("training step", dtype, fmt)
    # forward
    m1, r1, m2, r2, mg, rg = st(B, N), st(B, N), st(B, N), st(B, N), st(B, N, H), st(B, N, H)
    xq, xs = kept(B, N, dm)
    y, _ = msr.msr_resid_norm_fwd(x, weight=w1, bias=c1, mean=m1, rstd=r1, H_q=xq, H_qs=xs)
    proj = {k: (y.view(T, dm) @ W[k]).view(B, N, H, d) for k in "QKVG"}
    R = torch.empty(msr.msr_chunkwise_states_shape(B, N, H, d, d, chunk), dtype=t, device="cuda")
    o = msr.msr_chunkwise_fwd_save(proj["Q"], proj["K"], proj["V"], gam, chunk, R, qk_scale=s)
    (oq, os_), (gq, gs) = kept(B, N, H, d), kept(B, N, H, d)
    z = msr.msr_gated_norm_fwd(o, proj["G"], weight=gw, bias=gc, mean=mg, rstd=rg, O_q=oq, O_qs=os_, G_q=gq, G_qs=gs)
    br = (z.view(T, H * d) @ WO).view(B, N, dm)
    (hq, hs), (bq, bs) = kept(B, N, dm), kept(B, N, dm)
    y2, h = msr.msr_resid_norm_fwd(x, br, scale=sc, weight=w2, bias=c2, mean=m2, rstd=r2, H_q=hq, H_qs=hs, B_q=bq,
                                   B_qs=bs)
    # backward of <dy, y2> + <dh, h>
    dy, dh = (dev(normal(rng, (B, N, dm), dtype, 0.3), dtype) for _ in range(2))
    q8 = fmt != "none"
    dsc, dw2, dc2, dw1, dc1 = (empty32(dm) for _ in range(5))
    dgw, dgc = empty32(H, d), empty32(H, d)
    dbr = torch.empty_like(x)
    dx = msr.msr_resid_norm_bwd(dy, hq if q8 else h, m2, r2, H_qs=hs, dH=dh, B=bq if q8 else br, B_qs=bs, scale=sc,
                                weight=w2, dB=dbr, dscale=dsc, dweight=dw2, dbias=dc2)
    dz = (dbr.view(T, dm) @ WO.t().contiguous()).view(B, N, H, d)
    z2 = torch.empty_like(o)
    do, dg = msr.msr_gated_norm_bwd(dz, oq if q8 else o, gq if q8 else proj["G"], mg, rg, O_qs=os_, G_qs=gs,
                                    weight=gw, bias=gc, Z=z2, dweight=dgw, dbias=dgc)
    dWO = z2.view(T, H * d).float().t() @ dbr.view(T, dm).float()
    dq, dk, dv = msr.msr_chunkwise_bwd_saved(proj["Q"], proj["K"], proj["V"], do, gam, chunk, R, qk_scale=s)
    dproj = dict(Q=dq, K=dk, V=dv, G=dg)
    dy1 = sum((dproj[k].view(T, H * d).float() @ W[k].float().t()) for k in "QKVG").to(t).view(B, N, dm)
    dx1 = msr.msr_resid_norm_bwd(dy1, xq if q8 else x, m1, r1, H_qs=xs, dH=dx, weight=w1, dweight=dw1, dbias=dc1)
    if q8:
        dW = {k: msr.msr_ckpt_wgrad(xq.view(T, dm), xs.view(T, -1), dproj[k].view(T, H * d), mean=m1.view(T),
                                    rstd=r1.view(T), weight=w1, bias=c1) for k in "QKVG"}
    torch.cuda.synchronize()
    # the same in float64 on the kept tensors
    back = lambda v, q, qs: ot.q_unpack(host(q), qs.cpu().numpy()) if q8 else host(v)
    flat = lambda a: a.reshape(T, -1)
    hv, bv, xv = back(h, hq, hs), back(br, bq, bs), back(x, xq, xs)
    ov, gv = back(o, oq, os_), back(proj["G"], gq, gs)
    g2 = ot.resid_norm_grad(flat(host(dy)), flat(hv), host(m2).ravel(), host(r2).ravel(), True, flat(host(dh)),
                            host(w2), flat(bv))
    dhv = g2["dh"][0]
    dbr64 = dhv * host(sc)
    dz64 = (dbr64 @ host(WO).T).reshape(T, H, d)
    gg = ot.gated_norm_grad(dz64, ov.reshape(T, H, d), gv.reshape(T, H, d), host(mg).reshape(T, H),
                            host(rg).reshape(T, H), True, host(gw), host(gc))
    dq64, dk64, dv64 = oracle.retention_grad(*(host(proj[k]) for k in "QKV"), gg["do"][0].reshape(B, N, H, d), gam,
                                             s)[:3]
    dp64 = dict(Q=dq64, K=dk64, V=dv64, G=gg["dg"][0])
    dy64 = sum(np.asarray(dp64[k]).reshape(T, -1) @ host(W[k]).T for k in "QKVG")
    g1 = ot.resid_norm_grad(dy64, flat(xv), host(m1).ravel(), host(r1).ravel(), True, dhv, host(w1))
    xh, _ = ot.normalised(flat(xv), host(m1).ravel(), host(r1).ravel())
    y64 = xh * host(w1) + host(c1)
    pairs = [("dx", dx1, g1["dh"][0]), ("dw1", dw1, g1["dweight"][0]), ("dc1", dc1, g1["dbias"][0]),
             ("dscale", dsc, g2["dscale"][0]), ("dw2", dw2, g2["dweight"][0]), ("dc2", dc2, g2["dbias"][0]),
             ("dgw", dgw, gg["dweight"][0]), ("dgc", dgc, gg["dbias"][0]),
             ("dWO", dWO, gg["z"][0].reshape(T, -1).T @ dbr64)]
    if q8:
        pairs += [("dW" + k, dW[k], y64.T @ np.asarray(dp64[k]).reshape(T, -1)) for k in "QKVG"]
    for name, got, want in pairs:
        err = oracle.max_rel_err(host(got).reshape(want.shape), want)
        print(f"{name}: {err:.2e}", flush=True)
        assert err < tol, (name, err)


# ------------------------------------------- beside the library's own paths --
def test_agrees_with_the_blocks_layer_norm_and_gate():
    """msr_retnet_block_fwd's LayerNorm and the layer's GroupNorm with gate compute the same formulas: the layer
    from its pieces (these entry points and plain products) against msr_layer_fwd."""
    import math
    import torch
    msr = _msr()
    B, N, dm, H, d, chunk = 1, 70, 128, 2, 64, 32
    rng = np.random.default_rng(6)
    X = normal(rng, (B, N, dm), "f32")
    Ws = [normal(rng, (dm, H * d), "f32", dm ** -0.5) for _ in range(4)] + [normal(rng, (H * d, dm), "f32", dm ** -0.5)]
    Xd, (WQ, WK, WV, WG, WO) = dev(X, "f32"), [dev(w, "f32") for w in Ws]
    gam = workloads.gammas(H)
    say("layer from its pieces")
    want = msr.msr_layer_fwd(Xd, WQ, WK, WV, WG, WO, gam, H, d, d, chunk, rope_base=0.0, gn_eps=1e-5)
    q, k, v, g = ((Xd.view(-1, dm).double() @ w.double()).float().view(B, N, H, d) for w in (WQ, WK, WV, WG))
    o = msr.msr_chunkwise_fwd(q, k, v, gam, chunk, qk_scale=1 / math.sqrt(d))
    z = msr.msr_gated_norm_fwd(o, g, eps=1e-5)
    got = (z.view(-1, H * d).double() @ WO.double()).view(B, N, dm)
    torch.cuda.synchronize()
    ref = oracle.msr_layer(X, *Ws, gam, H, d, d, chunk, rope_base=0.0, eps=1e-5)
    assert oracle.max_rel_err(got.cpu().numpy(), ref) < 1e-4
    assert oracle.max_rel_err(host(want), ref) < 1e-4
