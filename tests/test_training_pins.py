"""Pins of the oracle's norms, gradients and 8-bit form (``oracle.training``)
against the layer's oracle, differences and brute force over the codes, and
the refusals of the entry points that compute them (no GPU is touched: every
call here fails validation or has nothing to do)."""
import ctypes
import os

import numpy as np
import pytest

import linear_recurrence_sequence_amd as msr
import oracle
from oracle import training as ot

FAKE = 0x1000  # never dereferenced: every call below fails validation first
built = pytest.mark.skipif(not os.path.exists(msr.library_path()), reason="libmsr.so not built")


# ----------------------------------------------------------------- oracle --
def test_forward_forms_agree_with_the_layers_oracle():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 5, 64)) * 3 + 1
    assert np.allclose(ot.resid_norm(x, True, 1e-5)[0], oracle.layer_norm(x, 1e-5), rtol=1e-13)
    o, g = rng.standard_normal((2, 5, 3, 64)), rng.standard_normal((2, 5, 3, 64))
    want = oracle.swish(g) * oracle.group_norm_heads(o, 1e-5).reshape(o.shape)
    assert np.allclose(ot.gated_norm(o, g, True, 1e-5)[0], want, rtol=1e-13)
    # rms: mean square one where the mean square is far above eps
    assert np.allclose((ot.resid_norm(x, False, 0.0)[0] ** 2).mean(-1), 1.0)


@pytest.mark.parametrize("layer", [True, False])
def test_gradients_against_differences(layer):
    """Central differences of <dy, y> + <dh_in, h> and <dz, z> in each argument.  Step 1e-5: the difference
    quotient is off by O(1e-10) from the third derivative and by 1e-16 / 1e-5 from rounding."""
    rng = np.random.default_rng(1)
    n, d, eps, s = 4, 6, 1e-3, 1e-5
    h, dy, dh_in, b = (rng.standard_normal((n, d)) for _ in range(4))
    w, c, sc = rng.standard_normal(d), rng.standard_normal(d), rng.standard_normal(d)
    x = h - sc * b
    loss = lambda x, w, c, sc: float((dy * ot.resid_norm(x + sc * b, layer, eps, w, c)[0]).sum()
                                     + (dh_in * (x + sc * b)).sum())
    mu, r = ot.norm_stats(h, layer, eps)
    got = ot.resid_norm_grad(dy, h, mu, r, layer, dh_in, w, b)

    def diff(f, v):
        out = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            e = np.zeros_like(v)
            e[i] = s
            out[i] = (f(v + e) - f(v - e)) / (2 * s)
        return out
    for name, want in (("dh", diff(lambda v: loss(v, w, c, sc), x)), ("dweight", diff(lambda v: loss(x, v, c, sc), w)),
                       ("dbias", diff(lambda v: loss(x, w, v, sc), c)),
                       ("dscale", diff(lambda v: loss(x, w, c, v), sc))):
        assert np.max(np.abs(got[name][0] - want)) < 1e-7, name
        assert np.all(got[name][1] >= np.abs(got[name][0]) * (1 - 1e-12)), name
    o, g, dz = rng.standard_normal((n, 2, d)), rng.standard_normal((n, 2, d)), rng.standard_normal((n, 2, d))
    w, c = rng.standard_normal((2, d)), rng.standard_normal((2, d))
    loss = lambda o, g, w, c: float((dz * ot.gated_norm(o, g, layer, eps, w, c)[0]).sum())
    mu, r = ot.norm_stats(o, layer, eps)
    got = ot.gated_norm_grad(dz, o, g, mu, r, layer, w, c)
    for name, want in (("do", diff(lambda v: loss(v, g, w, c), o)), ("dg", diff(lambda v: loss(o, v, w, c), g)),
                       ("dweight", diff(lambda v: loss(o, g, v, c), w)),
                       ("dbias", diff(lambda v: loss(o, g, w, v), c))):
        assert np.max(np.abs(got[name][0] - want)) < 1e-7, name
        assert np.all(got[name][1] >= np.abs(got[name][0]) * (1 - 1e-12)), name
    assert np.allclose(got["z"][0], ot.gated_norm(o, g, layer, eps, w, c)[0])


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_8_bit_form_against_all_codes(fmt):
    """Every code is a nearest one (of two, the even one) among all codes of the group's exponent, and one
    exponent less would not hold the group."""
    codes = np.array(sorted(set(ot.e4m3_values()[np.isfinite(ot.e4m3_values())]))) if fmt == "e4m3" \
        else np.arange(-127.0, 128.0)
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((40, 64)) * np.exp2(rng.integers(-20, 20, (40, 1)))).astype(np.float32)
    x[0] = 0
    x[1, :32] = ot.Q_TOP[fmt] * 2.0 ** -3                       # the border of an exponent
    x[2, :32] = np.nextafter(np.float32(ot.Q_TOP[fmt]), np.float32(1e9))   # just past it
    x[3, :4] = codes[[3, 10, 20, 30]] * 0.5 + codes[[4, 11, 21, 31]] * 0.5  # ties
    q, qs = ot.q_pack(x, fmt)
    e = qs.astype(int) - 127
    assert e[0, 0] == -127 and e[1, 0] == -3 and e[2, 0] == 1
    amax = np.abs(x.reshape(40, 2, 32)).max(-1)
    assert np.all(amax <= ot.Q_TOP[fmt] * 2.0 ** e)
    assert np.all((amax > ot.Q_TOP[fmt] * 2.0 ** (e - 1)) | (e == -127))
    v = x.astype(np.float64) / np.repeat(2.0 ** e, 32, axis=-1)
    err = np.abs(codes[None, None, :] - v[..., None])
    best = err.min(-1)
    assert np.array_equal(np.abs(q - v), best)
    tie = (err == best[..., None]).sum(-1) > 1
    if fmt == "i8":
        assert np.all(q[tie] % 2 == 0)
    else:                                                       # the even significand: an even position among the codes >= 0
        assert np.all(np.searchsorted(codes[codes >= 0], np.abs(q[tie])) % 2 == 0)
    assert np.array_equal(ot.q_unpack(q, qs), q * np.repeat(2.0 ** e, 32, axis=-1))
    y = x[:2].copy()
    y[0, 5], y[1, 40] = np.inf, np.nan
    q, qs = ot.q_pack(y, fmt)
    assert qs[0, 0] == 255 and qs[1, 1] == 255 and qs[0, 1] != 255 and qs[1, 0] != 255
    assert np.all(np.isnan(ot.q_unpack(q, qs)) == (np.repeat(qs, 32, axis=-1) == 255))


# --------------------------------------------------------------- refusals --
@built
def test_resid_norm_refusals():
    L = msr.lib()
    fwd = lambda dtype=1, norm=0, rows=4, d=128, alpha=1.0, eps=1e-5, X=FAKE, B=FAKE, scale=None, w=None, H=FAKE, \
        Y=FAKE, fmt=0, Hq=None, Hs=None, Bq=None, Bs=None: L.msr_resid_norm_fwd(
            dtype, norm, rows, d, alpha, eps, X, B, scale, w, None, H, Y, None, None, fmt, Hq, Hs, Bq, Bs, None)
    assert fwd(dtype=2) == 3 and fwd(dtype=-2 ** 31) == 3
    assert fwd(fmt=3) == 3 and fwd(fmt=-1) == 3
    assert fwd(norm=2) == 4 and fwd(norm=-1) == 4
    assert fwd(rows=-1) == 2 and fwd(d=0) == 2 and fwd(d=-64) == 2
    assert fwd(d=96) == 4 and fwd(d=8256) == 4
    assert fwd(alpha=float("nan")) == 2 and fwd(alpha=float("inf")) == 2
    assert fwd(eps=-1.0) == 2 and fwd(eps=float("nan")) == 2 and fwd(eps=float("inf")) == 2
    assert fwd(X=None) == 1 and fwd(Y=None) == 1
    assert fwd(fmt=1) == 1 and fwd(fmt=1, Hq=FAKE) == 1            # a format needs both
    assert fwd(Hq=FAKE, Hs=FAKE) == 3                             # and they a format
    assert fwd(fmt=1, Hq=FAKE, Hs=FAKE, Bq=FAKE) == 1
    assert fwd(fmt=2, B=None, Hq=FAKE, Hs=FAKE, Bq=FAKE, Bs=FAKE) == 1
    assert fwd(B=None, scale=FAKE) == 1
    assert fwd(X=FAKE + 8) == 4 and "aligned" in msr.msr_last_error()
    assert fwd(w=FAKE + 4) == 4
    assert fwd(rows=0, X=None, Y=None) == 0
    bwd = lambda dtype=1, norm=0, rows=4, d=128, alpha=1.0, dY=FAKE, fmt=0, H=FAKE, Hs=None, B=None, Bs=None, \
        mean=FAKE, rstd=FAKE, dX=FAKE, ds=None, dw=None, ws=None, wsb=0: L.msr_resid_norm_bwd(
            dtype, norm, rows, d, alpha, dY, None, fmt, H, Hs, B, Bs, mean, rstd, None, None, dX, None, ds, dw,
            None, ws, wsb, None)
    assert bwd(dtype=5) == 3 and bwd(fmt=7) == 3 and bwd(norm=9) == 4
    assert bwd(d=100) == 4 and bwd(rows=-4) == 2 and bwd(alpha=float("nan")) == 2
    assert bwd(dY=None) == 1 and bwd(H=None) == 1 and bwd(rstd=None) == 1 and bwd(dX=None) == 1
    assert bwd(mean=None) == 1
    assert bwd(fmt=1) == 1                                        # no scale bytes
    assert bwd(ds=FAKE) == 1 and "dscale needs B" in msr.msr_last_error()
    assert bwd(fmt=1, Hs=FAKE, B=FAKE, ds=FAKE) == 1              # B's scale bytes
    assert bwd(dw=FAKE) == 5 and bwd(dw=FAKE, ws=FAKE, wsb=16) == 5
    assert bwd(H=FAKE + 2) == 4
    assert bwd(rows=0, dY=None, H=None, rstd=None, dX=None) == 0
    assert msr.msr_resid_norm_bwd_workspace_bytes(0, 128) == 0 == msr.msr_resid_norm_bwd_workspace_bytes(-1, 128)
    assert msr.msr_resid_norm_bwd_workspace_bytes(4, 100) == 0 == msr.msr_resid_norm_bwd_workspace_bytes(4, 1 << 20)
    assert 0 < msr.msr_resid_norm_bwd_workspace_bytes(1, 64) < msr.msr_resid_norm_bwd_workspace_bytes(1 << 20, 8192)


@built
def test_gated_norm_refusals():
    L = msr.lib()
    fwd = lambda dtype=1, norm=0, rows=4, heads=2, dv=64, eps=1e-5, O=FAKE, Z=FAKE, fmt=0, q=(None,) * 4: \
        L.msr_gated_norm_fwd(dtype, norm, rows, heads, dv, eps, O, FAKE, None, None, Z, None, None, fmt, *q, None)
    assert fwd(dtype=2) == 3 and fwd(fmt=3) == 3 and fwd(norm=2) == 4
    assert fwd(rows=-1) == 2 and fwd(heads=0) == 2 and fwd(dv=-64) == 2
    assert fwd(heads=129) == 4 and fwd(dv=96) == 4 and fwd(dv=1024) == 4
    assert fwd(eps=-1e-9) == 2 and fwd(eps=float("nan")) == 2
    assert fwd(O=None) == 1 and fwd(Z=None) == 1
    assert fwd(fmt=1) == 1 and fwd(fmt=1, q=(FAKE, FAKE, FAKE, None)) == 1
    assert fwd(q=(FAKE, FAKE, None, None)) == 3
    assert fwd(O=FAKE + 4) == 4
    assert fwd(rows=0, O=None, Z=None) == 0
    bwd = lambda dtype=1, norm=0, rows=4, heads=2, dv=64, dZ=FAKE, fmt=0, Os=None, Gs=None, mean=FAKE, rstd=FAKE, \
        dO=FAKE, dw=None, ws=None, wsb=0: L.msr_gated_norm_bwd(
            dtype, norm, rows, heads, dv, dZ, fmt, FAKE, Os, FAKE, Gs, mean, rstd, None, None, dO, FAKE, None, dw,
            None, ws, wsb, None)
    assert bwd(dtype=-1) == 3 and bwd(fmt=-1) == 3 and bwd(norm=-1) == 4
    assert bwd(dv=48) == 4 and bwd(heads=-1) == 2
    assert bwd(dZ=None) == 1 and bwd(mean=None) == 1 and bwd(rstd=None) == 1 and bwd(dO=None) == 1
    assert bwd(fmt=2) == 1 and bwd(fmt=2, Os=FAKE) == 1
    assert bwd(dw=FAKE) == 5 and bwd(dw=FAKE, ws=FAKE, wsb=255) == 5
    assert bwd(dO=FAKE + 8) == 4
    assert bwd(rows=0, dZ=None, rstd=None, dO=None) == 0
    assert msr.msr_gated_norm_bwd_workspace_bytes(0, 2, 64) == 0 == msr.msr_gated_norm_bwd_workspace_bytes(4, 2, 65)


@built
def test_ckpt_refusals():
    L = msr.lib()
    pack = lambda dtype=1, fmt=1, rows=4, cols=64, X=FAKE, q=FAKE, qs=FAKE: L.msr_ckpt_pack(dtype, fmt, rows, cols, X,
                                                                                          q, qs, None)
    assert pack(dtype=2) == 3 and pack(fmt=0) == 3 and pack(fmt=3) == 3
    assert pack(rows=-1) == 2 and pack(cols=0) == 2 and pack(cols=48) == 4
    assert pack(X=None) == 1 and pack(q=None) == 1 and pack(qs=None) == 1
    assert pack(X=FAKE + 2) == 4 and pack(q=FAKE + 8) == 4
    assert pack(rows=0, X=None) == 0
    unpack = lambda dtype=0, fmt=2, rows=4, cols=64, q=FAKE, X=FAKE, w=None: L.msr_ckpt_unpack(
        dtype, fmt, rows, cols, q, FAKE, None, None, w, None, X, None)
    assert unpack(dtype=9) == 3 and unpack(fmt=0) == 3 and unpack(cols=33) == 4 and unpack(rows=-2) == 2
    assert unpack(q=None) == 1 and unpack(X=None) == 1 and unpack(w=FAKE + 4) == 4
    assert unpack(rows=0, q=None) == 0
    wg = lambda dtype=1, fmt=1, rows=100, i=64, o=128, q=FAKE, dY=FAKE, acc=0, dW=FAKE, ws=FAKE, wsb=1 << 40: \
        L.msr_ckpt_wgrad(dtype, fmt, rows, i, o, q, FAKE, None, None, None, None, dY, acc, dW, ws, wsb, None)
    assert wg(dtype=4) == 3 and wg(fmt=0) == 3
    assert wg(rows=-1) == 2 and wg(i=0) == 2 and wg(o=-64) == 2
    assert wg(i=96) == 4 and wg(o=100) == 4 and wg(i=1 << 21) == 4 and wg(rows=(1 << 20) + 1) == 4
    assert wg(q=None) == 1 and wg(dY=None) == 1 and wg(dW=None) == 1
    assert wg(ws=None) == 5 and wg(wsb=64) == 5
    assert wg(dW=FAKE + 4) == 4
    assert wg(rows=0, q=None, dY=None, acc=1, ws=None, wsb=0) == 0
    for rows in (1, 63, 64, 65, 4096, 99999):
        for i, o in ((64, 64), (2048, 8192), (192, 320)):
            for dtype, normed, terms in ((1, 0, 1), (1, 1, 1), (0, 0, 3), (0, 1, 6)):
                a, b = (msr.msr_ckpt_wgrad_workspace_bytes(dtype, rows, i, o, normed, acc) for acc in (False, True))
                assert i * (-(-rows // 64) * 64) * 2 * terms <= a <= b
    assert msr.msr_ckpt_wgrad_workspace_bytes(1, 64, 65, 64) == 0


@built
def test_binding_refusals():
    """Shapes, types and formats are checked before any pointer reaches the library."""
    import torch
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    z = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype)
    X = z(3, 5, 128)
    q, qs = msr.msr_ckpt_empty((3, 5, 128), msr.MSR_Q_I8, "cpu")
    assert q.dtype == torch.int8 and q.shape == (3, 5, 128) and qs.shape == (3, 5, 4) and qs.dtype == u8
    q8, _ = msr.msr_ckpt_empty((3, 5, 128), msr.MSR_Q_E4M3, "cpu")
    assert q8.dtype == torch.float8_e4m3fn
    st = z(3, 5, dtype=f32)
    O = z(3, 5, 2, 64)
    st2 = z(3, 5, 2, dtype=f32)
    cases = [
        (lambda: msr.msr_ckpt_empty((3, 40), msr.MSR_Q_I8, "cpu"), "multiple of 32"),
        (lambda: msr.msr_ckpt_empty((3, 64), 0, "cpu"), "unknown 8-bit format"),
        (lambda: msr.msr_resid_norm_fwd(X, X[:2]), "B must have shape"),
        (lambda: msr.msr_resid_norm_fwd(X, X, weight=z(128)), "weight must be torch.float32"),
        (lambda: msr.msr_resid_norm_fwd(X, X, rstd=z(15, dtype=f32)), "rstd must have shape"),
        (lambda: msr.msr_resid_norm_fwd(X, X, H_q=q), "needs its scale bytes"),
        (lambda: msr.msr_resid_norm_fwd(X, X, H_qs=qs), "without H_q"),
        (lambda: msr.msr_resid_norm_fwd(X, X, H_q=X, H_qs=qs), "float8_e4m3fn or torch.int8"),
        (lambda: msr.msr_resid_norm_fwd(X, X, H_q=q, H_qs=qs[..., :2]), "scale bytes must have shape"),
        (lambda: msr.msr_resid_norm_fwd(X, X, H_q=q, H_qs=qs, B_q=q8, B_qs=qs), "share one format"),
        (lambda: msr.msr_resid_norm_fwd(X, X, B_q=q, B_qs=qs), "B_q without H_q"),
        (lambda: msr.msr_resid_norm_bwd(X, X, None, st), "required"),
        (lambda: msr.msr_resid_norm_bwd(X, q, st, st), "H must be torch.bfloat16"),
        (lambda: msr.msr_resid_norm_bwd(X, q, st, st, H_qs=qs, B=X), "B must be held as H is"),
        (lambda: msr.msr_resid_norm_bwd(X, X, st, st, dscale=z(64, dtype=f32)), "dscale must have shape"),
        (lambda: msr.msr_gated_norm_fwd(O, O[:, :4]), "G must have shape"),
        (lambda: msr.msr_gated_norm_fwd(O, O, weight=z(128, dtype=f32)), "weight must have shape"),
        (lambda: msr.msr_gated_norm_bwd(O, O, O, st2, None), "required"),
        (lambda: msr.msr_gated_norm_bwd(O, O, O, st2, st2, Z=z(3, 5, 128)), "Z must have shape"),
        (lambda: msr.msr_ckpt_pack(z(3, 40)), "multiple of 32"),
        (lambda: msr.msr_ckpt_pack(X, 0), "unknown 8-bit format"),
        (lambda: msr.msr_ckpt_unpack(q, qs, out=z(3, 5, 64)), "out must have shape"),
        (lambda: msr.msr_ckpt_wgrad(q, qs, z(3, 4, 64)), "dY must have shape"),
        (lambda: msr.msr_ckpt_wgrad(q, qs, X, accumulate=True), "accumulate needs dW"),
        # all of it right: the next check is the device
        (lambda: msr.msr_resid_norm_fwd(X, X, H_q=q, H_qs=qs), "on the GPU"),
        (lambda: msr.msr_resid_norm_bwd(X, X, st, st), "on the GPU"),
        (lambda: msr.msr_gated_norm_fwd(O, O), "on the GPU"),
        (lambda: msr.msr_gated_norm_bwd(O, O, O, st2, st2), "on the GPU"),
        (lambda: msr.msr_ckpt_pack(X), "on the GPU"),
        (lambda: msr.msr_ckpt_unpack(q, qs), "on the GPU"),
        (lambda: msr.msr_ckpt_wgrad(q, qs, X), "on the GPU"),
    ]
    for call, msg in cases:
        with pytest.raises(ValueError, match=msg):
            call()
    with pytest.raises(TypeError, match="unsupported tensor dtype"):
        msr.msr_ckpt_pack(X.to(torch.float16))
    with pytest.raises(TypeError, match="unsupported tensor dtype"):
        msr.msr_ckpt_unpack(q, qs, torch.float16)
