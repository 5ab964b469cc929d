// libmsr C ABI, training between retention cores: argument validation,
// workspace layout and dispatch of the norms with gate and residual and of
// the activations kept in 8 bits (documented in include/msr.h).
#include <algorithm>
#include <cmath>

#include "../../include/msr.h"
#include "msr_launch.h"
#include "msr_q8.h"
#include "msr_status.h"

using namespace msr;

namespace {

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
Elt elt_of(msr_dtype d) { return d == MSR_BF16 ? kBF16 : kF32; }
size_t size_of(msr_dtype d) { return d == MSR_BF16 ? 2 : 4; }

msr_status check_types(msr_dtype dtype, msr_qfmt fmt, bool need_fmt) {
  if (dtype != MSR_F32 && dtype != MSR_BF16) return fail(MSR_ERR_DTYPE, "unknown dtype %d", (int)dtype);
  if (fmt != MSR_Q_E4M3 && fmt != MSR_Q_I8 && (need_fmt || fmt != MSR_Q_NONE))
    return fail(MSR_ERR_DTYPE, "%s 8-bit format %d", need_fmt && fmt == MSR_Q_NONE ? "an operation on 8-bit values "
                "needs a format, got" : "unknown", (int)fmt);
  return MSR_OK;
}

msr_status check_norm(msr_norm norm) {
  if (norm != MSR_NORM_LAYER && norm != MSR_NORM_RMS) return fail(MSR_ERR_UNSUPPORTED, "unknown norm %d", (int)norm);
  return MSR_OK;
}

msr_status check_eps(float eps) {
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(MSR_ERR_SHAPE, "eps must be finite and >= 0");
  return MSR_OK;
}

// The kernels move 16 bytes at a time.
template <class... P>
msr_status check_aligned(const P*... p) {
  for (const void* q : {(const void*)p...})
    if (reinterpret_cast<uintptr_t>(q) % 16) return fail(MSR_ERR_UNSUPPORTED, "tensors must be 16-byte aligned");
  return MSR_OK;
}

msr_status check_resid(msr_norm norm, int32_t rows, int32_t d, float alpha) {
  msr_status s;
  if ((s = check_norm(norm))) return s;
  if (rows < 0 || d <= 0) return fail(MSR_ERR_SHAPE, "invalid sizes rows=%d d=%d", rows, d);
  if (d % 64 || d > 8192)
    return fail(MSR_ERR_UNSUPPORTED, "d = %d is not a multiple of 64 up to 8192", d);
  if (!std::isfinite(alpha)) return fail(MSR_ERR_SHAPE, "alpha must be finite");
  return MSR_OK;
}

msr_status check_gated(msr_norm norm, int32_t rows, int32_t heads, int32_t d_v) {
  msr_status s;
  if ((s = check_norm(norm))) return s;
  if (rows < 0 || heads <= 0 || d_v <= 0)
    return fail(MSR_ERR_SHAPE, "invalid sizes rows=%d heads=%d d_v=%d", rows, heads, d_v);
  if (heads > kMaxHeads) return fail(MSR_ERR_UNSUPPORTED, "heads=%d exceeds %d", heads, kMaxHeads);
  if (d_v != 64 && d_v != 128 && d_v != 256 && d_v != 512)
    return fail(MSR_ERR_UNSUPPORTED, "d_v = %d has no kernel; supported: 64 128 256 512", d_v);
  return MSR_OK;
}

msr_status check_ws(const void* workspace, size_t got, size_t need) {
  if (need > 0 && (!workspace || got < need))
    return fail(MSR_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace ? got : 0);
  return MSR_OK;
}

}  // namespace

extern "C" {

msr_status msr_resid_norm_fwd(msr_dtype dtype, msr_norm norm, int32_t rows, int32_t d, float alpha, float eps,
                              const void* X, const void* B, const float* scale, const float* weight,
                              const float* bias, void* H, void* Y, float* mean, float* rstd, msr_qfmt fmt, void* H_q,
                              uint8_t* H_qs, void* B_q, uint8_t* B_qs, void* stream) {
  msr_status s;
  if ((s = check_types(dtype, fmt, false))) return s;
  if ((s = check_resid(norm, rows, d, alpha))) return s;
  if ((s = check_eps(eps))) return s;
  if (rows == 0) return ok();
  if (!X || !Y) return fail(MSR_ERR_NULL, "X and Y must be non-NULL");
  if (fmt != MSR_Q_NONE && (!H_q || !H_qs)) return fail(MSR_ERR_NULL, "H_q and H_qs must be non-NULL with a format");
  if ((B_q == nullptr) != (B_qs == nullptr)) return fail(MSR_ERR_NULL, "B_q and B_qs go together");
  if (fmt == MSR_Q_NONE && (H_q || B_q)) return fail(MSR_ERR_DTYPE, "H_q and B_q need a format");
  if (B_q && !B) return fail(MSR_ERR_NULL, "B_q needs B");
  if (scale && !B) return fail(MSR_ERR_NULL, "scale needs B");
  if ((s = check_aligned(X, B, scale, weight, bias, H, Y, H_q, B_q))) return s;
  ResidNormArgs a{};
  a.elt = elt_of(dtype); a.fmt = (int)fmt; a.layer = norm == MSR_NORM_LAYER;
  a.rows = rows; a.d = d; a.alpha = alpha; a.eps = eps;
  a.X = X; a.B = B; a.scale = scale; a.weight = weight; a.bias = bias;
  a.H = H; a.Y = Y; a.mean = a.layer ? mean : nullptr; a.rstd = rstd;
  a.H_q = (uint8_t*)H_q; a.H_qs = H_qs; a.B_q = (uint8_t*)B_q; a.B_qs = B_qs;
  return from_hip(launch_resid_norm_fwd(a, (hipStream_t)stream), "msr_resid_norm_fwd");
}

size_t msr_resid_norm_bwd_workspace_bytes(int32_t rows, int32_t d) {
  if (rows < 0 || d <= 0 || d % 64 || d > 8192) return 0;
  return up256((size_t)3 * resid_norm_bwd_parts(rows, d) * d * sizeof(float));
}

msr_status msr_resid_norm_bwd(msr_dtype dtype, msr_norm norm, int32_t rows, int32_t d, float alpha, const void* dY,
                              const void* dH_in, msr_qfmt fmt, const void* H, const uint8_t* H_qs, const void* B,
                              const uint8_t* B_qs, const float* mean, const float* rstd, const float* scale,
                              const float* weight, void* dX, void* dB, float* dscale, float* dweight, float* dbias,
                              void* workspace, size_t ws_bytes, void* stream) {
  msr_status s;
  if ((s = check_types(dtype, fmt, false))) return s;
  if ((s = check_resid(norm, rows, d, alpha))) return s;
  const bool sums = dscale || dweight || dbias;
  if (rows > 0) {
    if (!dY || !H || !rstd || !dX) return fail(MSR_ERR_NULL, "dY, H, rstd and dX must be non-NULL");
    if (norm == MSR_NORM_LAYER && !mean) return fail(MSR_ERR_NULL, "mean must be non-NULL for MSR_NORM_LAYER");
    if (dscale && !B) return fail(MSR_ERR_NULL, "dscale needs B");
    if (fmt != MSR_Q_NONE && (!H_qs || (dscale && !B_qs)))
      return fail(MSR_ERR_NULL, "H_qs (and B_qs with dscale) must be non-NULL with a format");
    if (sums && (s = check_ws(workspace, ws_bytes, msr_resid_norm_bwd_workspace_bytes(rows, d)))) return s;
  }
  if ((s = check_aligned(dY, dH_in, H, B, scale, weight, dX, dB, workspace)))
    return s;
  ResidNormBwdArgs a{};
  a.elt = elt_of(dtype); a.fmt = (int)fmt; a.layer = norm == MSR_NORM_LAYER;
  a.rows = rows; a.d = d; a.alpha = alpha;
  a.dY = dY; a.dH_in = dH_in; a.H = H; a.H_qs = H_qs; a.B = B; a.B_qs = B_qs;
  a.mean = mean; a.rstd = rstd; a.scale = scale; a.weight = weight;
  a.dX = dX; a.dB = dB; a.part = (float*)workspace;
  return from_hip(launch_resid_norm_bwd(a, dscale, dweight, dbias, (hipStream_t)stream), "msr_resid_norm_bwd");
}

msr_status msr_gated_norm_fwd(msr_dtype dtype, msr_norm norm, int32_t rows, int32_t heads, int32_t d_v, float eps,
                              const void* O, const void* G, const float* weight, const float* bias, void* Z,
                              float* mean, float* rstd, msr_qfmt fmt, void* O_q, uint8_t* O_qs, void* G_q,
                              uint8_t* G_qs, void* stream) {
  msr_status s;
  if ((s = check_types(dtype, fmt, false))) return s;
  if ((s = check_gated(norm, rows, heads, d_v))) return s;
  if ((s = check_eps(eps))) return s;
  if (rows == 0) return ok();
  if (!O || !G || !Z) return fail(MSR_ERR_NULL, "O, G and Z must be non-NULL");
  if (fmt != MSR_Q_NONE && (!O_q || !O_qs || !G_q || !G_qs))
    return fail(MSR_ERR_NULL, "O_q, O_qs, G_q and G_qs must be non-NULL with a format");
  if (fmt == MSR_Q_NONE && (O_q || G_q)) return fail(MSR_ERR_DTYPE, "O_q and G_q need a format");
  if ((s = check_aligned(O, G, weight, bias, Z, O_q, G_q))) return s;
  GatedNormArgs a{};
  a.elt = elt_of(dtype); a.fmt = (int)fmt; a.layer = norm == MSR_NORM_LAYER;
  a.rows = rows; a.heads = heads; a.d_v = d_v; a.eps = eps;
  a.O = O; a.G = G; a.weight = weight; a.bias = bias; a.Z = Z;
  a.mean = a.layer ? mean : nullptr; a.rstd = rstd;
  a.O_q = (uint8_t*)O_q; a.O_qs = O_qs; a.G_q = (uint8_t*)G_q; a.G_qs = G_qs;
  return from_hip(launch_gated_norm_fwd(a, (hipStream_t)stream), "msr_gated_norm_fwd");
}

size_t msr_gated_norm_bwd_workspace_bytes(int32_t rows, int32_t heads, int32_t d_v) {
  if (check_gated(MSR_NORM_LAYER, rows, heads, d_v)) return 0;
  return up256((size_t)2 * gated_norm_bwd_parts(rows, heads, d_v) * heads * d_v * sizeof(float));
}

msr_status msr_gated_norm_bwd(msr_dtype dtype, msr_norm norm, int32_t rows, int32_t heads, int32_t d_v,
                              const void* dZ, msr_qfmt fmt, const void* O, const uint8_t* O_qs, const void* G,
                              const uint8_t* G_qs, const float* mean, const float* rstd, const float* weight,
                              const float* bias, void* dO, void* dG, void* Z, float* dweight, float* dbias,
                              void* workspace, size_t ws_bytes, void* stream) {
  msr_status s;
  if ((s = check_types(dtype, fmt, false))) return s;
  if ((s = check_gated(norm, rows, heads, d_v))) return s;
  if (rows > 0) {
    if (!dZ || !O || !G || !rstd || !dO || !dG) return fail(MSR_ERR_NULL, "dZ, O, G, rstd, dO and dG must be non-NULL");
    if (norm == MSR_NORM_LAYER && !mean) return fail(MSR_ERR_NULL, "mean must be non-NULL for MSR_NORM_LAYER");
    if (fmt != MSR_Q_NONE && (!O_qs || !G_qs))
      return fail(MSR_ERR_NULL, "O_qs and G_qs must be non-NULL with a format");
    if ((dweight || dbias) &&
        (s = check_ws(workspace, ws_bytes, msr_gated_norm_bwd_workspace_bytes(rows, heads, d_v))))
      return s;
  }
  if ((s = check_aligned(dZ, O, G, weight, bias, dO, dG, Z, workspace))) return s;
  GatedNormBwdArgs a{};
  a.elt = elt_of(dtype); a.fmt = (int)fmt; a.layer = norm == MSR_NORM_LAYER;
  a.rows = rows; a.heads = heads; a.d_v = d_v;
  a.dZ = dZ; a.O = O; a.O_qs = O_qs; a.G = G; a.G_qs = G_qs;
  a.mean = mean; a.rstd = rstd; a.weight = weight; a.bias = bias;
  a.dO = dO; a.dG = dG; a.Z = Z; a.part = (float*)workspace;
  return from_hip(launch_gated_norm_bwd(a, dweight, dbias, (hipStream_t)stream), "msr_gated_norm_bwd");
}

}  // extern "C"

static msr_status check_ckpt(msr_dtype dtype, msr_qfmt fmt, int32_t rows, int32_t cols) {
  msr_status s;
  if ((s = check_types(dtype, fmt, true))) return s;
  if (rows < 0 || cols <= 0) return fail(MSR_ERR_SHAPE, "invalid sizes rows=%d cols=%d", rows, cols);
  if (cols % 32) return fail(MSR_ERR_UNSUPPORTED, "cols = %d is not a multiple of 32", cols);
  return MSR_OK;
}

extern "C" {

msr_status msr_ckpt_pack(msr_dtype dtype, msr_qfmt fmt, int32_t rows, int32_t cols, const void* X, void* q,
                         uint8_t* qs, void* stream) {
  msr_status s;
  if ((s = check_ckpt(dtype, fmt, rows, cols))) return s;
  if (rows == 0) return ok();
  if (!X || !q || !qs) return fail(MSR_ERR_NULL, "X, q and qs must be non-NULL");
  if ((s = check_aligned(X, q))) return s;
  return from_hip(launch_ckpt_pack(elt_of(dtype), (int)fmt, rows, cols, X, (uint8_t*)q, qs, (hipStream_t)stream),
                  "msr_ckpt_pack");
}

msr_status msr_ckpt_unpack(msr_dtype dtype, msr_qfmt fmt, int32_t rows, int32_t cols, const void* q,
                           const uint8_t* qs, const float* mean, const float* rstd, const float* weight,
                           const float* bias, void* X, void* stream) {
  msr_status s;
  if ((s = check_ckpt(dtype, fmt, rows, cols))) return s;
  if (rows == 0) return ok();
  if (!X || !q || !qs) return fail(MSR_ERR_NULL, "X, q and qs must be non-NULL");
  if ((s = check_aligned(q, weight, bias, X))) return s;
  const CkptArgs a{rows, cols, (const uint8_t*)q, qs, mean, rstd, weight, bias};
  return from_hip(launch_ckpt_unpack(elt_of(dtype), (int)fmt, a, X, (hipStream_t)stream), "msr_ckpt_unpack");
}

}  // extern "C"

// Weight gradient: the operands as bf16 pieces in the workspace (X^T always,
// dY where it is float32; a bf16 dY is read in place, but for a last slab
// that it does not fill: the product reads a copy with zeros behind it, whose
// rows meet zeros of X that would make an infinity a NaN), the product over
// the reduction indexes (tokens times terms), 64 of them a slab, in `splits`
// slices of whole slabs.  Each slice gives a float32 partial; a single one is
// dW itself.
namespace {
struct WgradPlan {
  int64_t slabs = 0;
  bool small = false;                // the product on 128 x 64 tiles
  int splits = 0;
  size_t xt = 0, dyt = 0, part = 0, total = 0;
};

WgradPlan wgrad_plan(msr_dtype dtype, int terms, int32_t rows, int32_t d_in, int32_t d_out, bool accumulate) {
  WgradPlan w;
  w.slabs = ((int64_t)rows + 63) / 64 * terms;
  // Fewest microseconds by a model of the product: rounds of workgroups over
  // the card (one a CU), each so many slabs deep (1.7 us a slab on 256 x 256
  // tiles, 0.5 on 128 x 64), and the partials' traffic.  Within 5 % of the
  // fastest of 1, 2, 3, 4, 8, 16 and 32 slices on 13 shapes from 64 x 64 to
  // 2048 x 8192 (2048 x 2048 over 16384 tokens: 165 us with 4, 335 with 1, 389
  // with 32); the small tiles took 28 us against 39 at 2048 x 2048 over 1000
  // tokens, 43 against 50 at 1024 x 1024 over 8192.
  const double part_us = (double)d_in * d_out * 8.0 / 4e6;      // written and read back at 4 TB/s
  double best = 0.0;
  for (const bool small : {false, true}) {
    const int tm = small ? 128 : 256, tn = small ? 64 : 256;
    const double slab = small ? 0.5 : 1.7;
    const int64_t tiles = (int64_t)((d_in + tm - 1) / tm) * ((d_out + tn - 1) / tn);
    for (int64_t s = 1; s <= std::min<int64_t>(w.slabs, 64); ++s) {
      double us = (double)((tiles * s + 255) / 256) * ((double)((w.slabs + s - 1) / s) * slab + 4.0);
      if (s > 1) us += (double)s * (part_us + 0.15) + 4.0;
      if (w.splits == 0 || us < best) {
        best = us;
        w.small = small;
        w.splits = (int)s;
      }
    }
  }
  size_t off = 0;
  const WgradPieces p = wgrad_pieces(terms);
  const size_t tokens = (size_t)(w.slabs / terms) * 64;
  w.xt = off; off += up256((size_t)d_in * tokens * p.x * 2);
  const size_t dy_rows = dtype == MSR_F32 ? tokens * p.dy : rows % 64 ? 64 : 0;
  w.dyt = off; off += up256(dy_rows * d_out * 2);
  w.part = off; off += w.splits > 1 || accumulate ? up256((size_t)w.splits * d_in * d_out * sizeof(float)) : 0;
  w.total = off;
  return w;
}

// bf16 terms of an operand pair (k_ckpt.hip)
int wgrad_terms(msr_dtype dtype, bool normed) { return dtype == MSR_BF16 ? 1 : normed ? 6 : 3; }

msr_status check_wgrad(msr_dtype dtype, msr_qfmt fmt, int32_t rows, int32_t d_in, int32_t d_out) {
  msr_status s;
  if ((s = check_types(dtype, fmt, true))) return s;
  if (rows < 0 || d_in <= 0 || d_out <= 0)
    return fail(MSR_ERR_SHAPE, "invalid sizes rows=%d d_in=%d d_out=%d", rows, d_in, d_out);
  if (d_in % 64 || d_out % 64 || d_in > (1 << 20) || d_out > (1 << 20))
    return fail(MSR_ERR_UNSUPPORTED, "d_in = %d and d_out = %d must be multiples of 64 up to 2^20", d_in, d_out);
  // a tile's 256 rows of X^T (three pieces a token) have 32-bit byte offsets
  if (rows > (1 << 20)) return fail(MSR_ERR_UNSUPPORTED, "rows = %d exceeds 2^20", rows);
  return MSR_OK;
}
}  // namespace

extern "C" {

size_t msr_ckpt_wgrad_workspace_bytes(msr_dtype dtype, int32_t rows, int32_t d_in, int32_t d_out, int32_t normed,
                                      int32_t accumulate) {
  if (check_wgrad(dtype, MSR_Q_I8, rows, d_in, d_out)) return 0;
  return wgrad_plan(dtype, wgrad_terms(dtype, normed != 0), rows, d_in, d_out, accumulate != 0).total;
}

msr_status msr_ckpt_wgrad(msr_dtype dtype, msr_qfmt fmt, int32_t rows, int32_t d_in, int32_t d_out, const void* q,
                          const uint8_t* qs, const float* mean, const float* rstd, const float* weight,
                          const float* bias, const void* dY, int32_t accumulate, float* dW, void* workspace,
                          size_t ws_bytes, void* stream) {
  msr_status s;
  if ((s = check_wgrad(dtype, fmt, rows, d_in, d_out))) return s;
  if (!dW) return fail(MSR_ERR_NULL, "dW must be non-NULL");
  if (rows > 0 && (!q || !qs || !dY)) return fail(MSR_ERR_NULL, "q, qs and dY must be non-NULL");
  const int terms = wgrad_terms(dtype, mean || rstd || weight || bias);
  const WgradPlan w = wgrad_plan(dtype, terms, rows, d_in, d_out, accumulate != 0);
  if ((s = check_ws(workspace, ws_bytes, w.total))) return s;
  if ((s = check_aligned(q, weight, bias, dY, dW, workspace))) return s;
  hipStream_t st = (hipStream_t)stream;
  const int64_t n = (int64_t)d_in * d_out;
  if (rows == 0)
    return accumulate ? ok() : from_hip(launch_sum_parts(nullptr, 0, dW, n, false, st), "msr_ckpt_wgrad");
  char* ws = (char*)workspace;
  const bool f32 = dtype == MSR_F32;
  float* part = w.splits > 1 || accumulate ? (float*)(ws + w.part) : dW;
  uint16_t* dyt = f32 || rows % 64 ? (uint16_t*)(ws + w.dyt) : nullptr;
  const int64_t slabs = w.slabs / terms;
  const WgradOperands ops{{rows, d_in, (const uint8_t*)q, qs, mean, rstd, weight, bias}, (uint16_t*)(ws + w.xt), slabs,
                          dY, rows, d_out, dyt};
  hipError_t err = launch_wgrad_operands(elt_of(dtype), (int)fmt, terms, ops, st);
  if (err != hipSuccess) return from_hip(err, "msr_ckpt_wgrad(operands)");
  err = launch_gemm_parts(ws + w.xt, slabs * wgrad_pieces(terms).x * 64, f32 ? dyt : dY, d_out, part, d_in, d_out,
                          (int)w.slabs, f32 ? nullptr : dyt, terms, w.splits, w.small, st);
  if (err != hipSuccess) return from_hip(err, "msr_ckpt_wgrad(product)");
  if (part != dW) err = launch_sum_parts(part, w.splits, dW, n, accumulate != 0, st);
  return from_hip(err, "msr_ckpt_wgrad(sum)");
}

}  // extern "C"
