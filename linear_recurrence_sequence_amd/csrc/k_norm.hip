// Norms between retention cores, forward and backward, for gfx950.
//
// [RN-zh] = page "Transformer取代者登場！微軟、清華剛推出RetNet：成本低、速度快、
// 性能強（2）": the layer's per-head GroupNorm and swish gate (section
// "門控多尺度 Retention", Eq. (8)) and the block's LayerNorm and residual
// connections (section "Retention 網路總體結構").
//
// resid_norm, per row of d:
//   h = rn(alpha x + s (.) b), mu = mean(h) (0 for RMS), r = 1 / sqrt(mean((h -
//   mu)^2) + eps), y = (h - mu) r (.) w + c
//   backward: xh = (h - mu) r, g = dy (.) w,
//   dh = dh_in + r (g - [LAYER] mean(g) - xh mean(g xh)), dx = alpha dh,
//   db = s (.) dh, ds = sum_t dh b, dw = sum_t dy xh, dc = sum_t dy
// gated_norm, per (token, head) row of d_v:
//   n = (o - mu) r (.) w + c, z = swish(g) (.) n
//   backward: sg = sigmoid(g), dn = dz g sg, dg = dz n sg (1 + g (1 - sg)),
//   u = dn (.) w, do = r (u - [LAYER] mean(u) - xh mean(u xh)),
//   dw = sum_t dn xh, dc = sum_t dn
//
// All of it streams: each tensor is read once and written once, bound by
// HBM.  A lane holds 8 neighbouring values (16-byte loads of bf16); a row's
// sums stay in registers and lane exchanges.  The sums over tokens (ds, dw,
// dc) are carried in registers while a thread walks down its columns; the
// walkers' float32 partials are then added in a fixed order in 64 bits by
// k_col_sums (no atomics: the same bits every time).
#include <algorithm>

#include "msr_launch.h"
#include "msr_q8.h"

namespace msr {

namespace {

constexpr int kMaxWaves = 16;

// Sum of x over the lanes that share a row: a group of LPR lanes of a wave,
// or (LPR == 0) the whole workgroup through red, whose two halves take
// turns: a wave writes a half again only after the barrier of the other
// half, which every wave reaches after reading the first.
template <int LPR, int NV>
__device__ __forceinline__ void row_sums(float (&x)[NV], float (*red)[kMaxWaves][2], int& turn) {
  static_assert(NV <= 2, "red holds two values per wave");
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = group_sum<LPR == 0 ? 64 : LPR>(x[i]);
  if constexpr (LPR == 0) {
    const int nw = blockDim.x >> 6, wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) red[turn][wave][i] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s = 0.f;
      for (int w = 0; w < nw; ++w) s += red[turn][w][i];
      x[i] = s;
    }
    turn ^= 1;
  }
}

__device__ __forceinline__ void load_vec8(float* v, const float* p, int64_t unit, bool ok, float def) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = def;
  if (p && ok) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p + 8 * unit), b = *reinterpret_cast<const f32x4*>(p + 8 * unit + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
  }
}
__device__ __forceinline__ void store_vec8(float* p, const float* v) {
  *reinterpret_cast<f32x4*>(p) = (f32x4){v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = (f32x4){v[4], v[5], v[6], v[7]};
}

// alpha x + s b, each product and the sum rounded to float32 (no fused
// multiply-add): the same value in every implementation of the formula, and
// so the same rounding to T and the same 8-bit codes.
__device__ __forceinline__ float scaled_sum(float alpha, float x, float s, float b) {
#pragma clang fp contract(off)
  const float p = alpha * x, q = s * b;
  return p + q;
}

// Rows of a row kernel: LPR lanes (a group of a wave) per row, or LPR == 0:
// the workgroup per row.  A thread holds units u0 + k step, k < VPT, of the
// row's d / 8.
template <int LPR>
struct RowMap {
  int rpb, rib, u0, step;      // rows per workgroup, row in the workgroup, first unit, unit step
  __device__ __forceinline__ RowMap() {
    if constexpr (LPR > 0) {
      rpb = blockDim.x / LPR;
      rib = threadIdx.x / LPR;
      u0 = threadIdx.x % LPR;
      step = LPR;
    } else {
      rpb = 1;
      rib = 0;
      u0 = threadIdx.x;
      step = blockDim.x;
    }
  }
};

template <class T, int LPR, int VPT, int F>
__global__ __launch_bounds__(LPR ? 256 : 512) void k_resid_norm_fwd(ResidNormArgs a) {
  __shared__ float red[2][kMaxWaves][2];
  const RowMap<LPR> m;
  const int units = a.d / 8;
  const float inv_d = 1.f / (float)a.d;
  float w[VPT][8], c[VPT][8], s[VPT][8];
  bool on[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int u = m.u0 + k * m.step;
    on[k] = u < units;
    load_vec8(w[k], a.weight, u, on[k], 1.f);
    load_vec8(c[k], a.bias, u, on[k], 0.f);
    load_vec8(s[k], a.scale, u, on[k], 1.f);
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * m.rpb + m.rib; row < a.rows; row += (int64_t)gridDim.x * m.rpb) {
    const int64_t base = row * units;
    float h[VPT][8];
    float sum[1] = {0.f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int64_t u = base + m.u0 + k * m.step;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = 0.f;
      if (on[k]) {
        Row8<T> rx, rb;
        float x[8], b[8];
        load_row8(rx, (const T*)a.X + 8 * u, true);
        if (a.B) load_row8(rb, (const T*)a.B + 8 * u, true);
        unpack_row8(x, rx);
        if (a.B) {
          unpack_row8(b, rb);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[k][e] = scaled_sum(a.alpha, x[e], s[k][e], b[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) h[k][e] = a.alpha * x[e];
        }
        Row8<T> rh;
        pack_row8(rh, h[k]);
        unpack_row8(h[k], rh);                 // the norm reads the sum as it is held
        if (a.H) store_row8((T*)a.H + 8 * u, rh);
        if constexpr (F != kQNone) {
          q_store8<F>(h[k], a.H_q, a.H_qs, u);
          if (a.B_q) q_store8<F>(b, a.B_q, a.B_qs, u);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] += h[k][e];
    }
    float mu = 0.f;
    if (a.layer) {
      row_sums<LPR>(sum, red, turn);
      mu = sum[0] * inv_d;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (on[k]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          h[k][e] -= mu;
          q[0] += h[k][e] * h[k][e];
        }
      }
    row_sums<LPR>(q, red, turn);
    const float r = 1.f / sqrtf(q[0] * inv_d + a.eps);
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (on[k]) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = h[k][e] * r * w[k][e] + c[k][e];
        Row8<T> ry;
        pack_row8(ry, y);
        store_row8((T*)a.Y + 8 * (base + m.u0 + k * m.step), ry);
      }
    if (m.u0 == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = r;
    }
  }
}

template <class T, int LPR, int VPT, int F, bool DS>
__global__ __launch_bounds__(LPR ? 256 : 512) void k_resid_norm_bwd(ResidNormBwdArgs a) {
  __shared__ float red[2][kMaxWaves][2];
  __shared__ float comb[LPR ? 256 * 8 : 8];
  const RowMap<LPR> m;
  const int units = a.d / 8;
  const float inv_d = 1.f / (float)a.d;
  float w[VPT][8], s[VPT][8], aw[VPT][8], ac[VPT][8], as[DS ? VPT : 1][8];
  bool on[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int u = m.u0 + k * m.step;
    on[k] = u < units;
    load_vec8(w[k], a.weight, u, on[k], 1.f);
    load_vec8(s[k], a.scale, u, on[k], 1.f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      aw[k][e] = ac[k][e] = 0.f;
      if constexpr (DS) as[k][e] = 0.f;
    }
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * m.rpb + m.rib; row < a.rows; row += (int64_t)gridDim.x * m.rpb) {
    const int64_t base = row * units;
    Row8<T> rdy[VPT], rdh[VPT];
    Held<T, F> rh[VPT], rb[DS ? VPT : 1];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (on[k]) {
        const int64_t u = base + m.u0 + k * m.step;
        load_row8(rdy[k], (const T*)a.dY + 8 * u, true);
        rh[k].load(a.H, a.H_qs, u);
        if (a.dH_in) load_row8(rdh[k], (const T*)a.dH_in + 8 * u, true);
        if constexpr (DS) rb[k].load(a.B, a.B_qs, u);
      }
    const float mu = a.layer ? a.mean[row] : 0.f, r = a.rstd[row];
    float xh[VPT][8], g[VPT][8];
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (on[k]) {
        rh[k].values(xh[k]);
        unpack_row8(g[k], rdy[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xh[k][e] = (xh[k][e] - mu) * r;
          aw[k][e] += g[k][e] * xh[k][e];
          ac[k][e] += g[k][e];
          g[k][e] *= w[k][e];
          sum[0] += g[k][e];
          sum[1] += g[k][e] * xh[k][e];
        }
      }
    row_sums<LPR>(sum, red, turn);
    const float m1 = a.layer ? sum[0] * inv_d : 0.f, m2 = sum[1] * inv_d;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (on[k]) {
        const int64_t u = base + m.u0 + k * m.step;
        float dh[8], o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) dh[e] = 0.f;
        if (a.dH_in) unpack_row8(dh, rdh[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dh[e] += r * (g[k][e] - m1 - xh[k][e] * m2);
        if constexpr (DS) {
          float b[8];
          rb[k].values(b);
#pragma unroll
          for (int e = 0; e < 8; ++e) as[k][e] += dh[e] * b[e];
        }
        Row8<T> ro;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = a.alpha * dh[e];
        pack_row8(ro, o);
        store_row8((T*)a.dX + 8 * u, ro);
        if (a.dB) {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = s[k][e] * dh[e];
          pack_row8(ro, o);
          store_row8((T*)a.dB + 8 * u, ro);
        }
      }
  }
  // this workgroup's partial sums over its rows, one row of d per requested vector
  auto put = [&](float (&v)[VPT][8], float* dst) {
    if constexpr (LPR == 0) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (on[k]) store_vec8(dst + (int64_t)blockIdx.x * a.d + 8 * (m.u0 + k * m.step), v[k]);
    } else {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        __syncthreads();
        store_vec8(comb + 8 * threadIdx.x, v[k]);
        __syncthreads();
        if (m.rib == 0 && on[k]) {
          float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          for (int i = 0; i < m.rpb; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] += comb[8 * (i * LPR + m.u0) + e];
          store_vec8(dst + (int64_t)blockIdx.x * a.d + 8 * (m.u0 + k * m.step), t);
        }
      }
    }
  };
  const int64_t plane = (int64_t)gridDim.x * a.d;
  float* dst = a.part;
  if (a.sum_w) { put(aw, dst); dst += plane; }
  if (a.sum_c) { put(ac, dst); dst += plane; }
  if constexpr (DS) put(as, dst);
}

// Column sums: out[v][j] = sum_p part[v][p][j] in 64 bits, in order of p
// within each of 16 waves, then of the waves.  64 columns per workgroup.
__global__ __launch_bounds__(1024) void k_col_sums(const float* __restrict__ part, int P, int n, ColSumOut out) {
  __shared__ double acc[kMaxWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = blockIdx.x * 64 + lane;
  const float* src = part + (int64_t)blockIdx.y * P * n + j;
  double s = 0.0;
  if (j < n) {
    int p = wave;
    for (; p + 7 * kMaxWaves < P; p += 8 * kMaxWaves) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = src[(int64_t)(p + i * kMaxWaves) * n];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += (double)v[i];
    }
    for (; p < P; p += kMaxWaves) s += (double)src[(int64_t)p * n];
  }
  acc[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && j < n) {
    double t = 0.0;
    for (int w = 0; w < kMaxWaves; ++w) t += acc[w][lane];
    float* o = blockIdx.y == 0 ? out.v[0] : blockIdx.y == 1 ? out.v[1] : out.v[2];
    o[j] = (float)t;
  }
}

// One thread: unit `col` of the heads * d_v / 8 units of a token, for tokens
// t0, t0 + R, ...; a head's units lie in one group of LPH = d_v / 8 lanes
// (units per token and threads per workgroup are multiples of LPH).  Up to
// 256 units a workgroup holds whole tokens (blockDim.x is a multiple of
// units) and every thread is on; beyond, a token spans workgroups and the
// threads past the R-th token are off.
struct GateMap {
  int units, col, t0;
  bool on;
  __device__ __forceinline__ GateMap(int heads, int lph, int R) {
    units = heads * lph;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    t0 = (int)(i / units);
    col = (int)(i - (int64_t)t0 * units);
    on = t0 < R;
  }
};

__device__ __forceinline__ float sigmoid_fast(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}

template <class T, int LPH, int F>
__global__ __launch_bounds__(256) void k_gated_norm_fwd(GatedNormArgs a) {
  const GateMap m(a.heads, LPH, a.R);
  if (!m.on) return;
  constexpr float inv_d = 1.f / (8.f * LPH);
  float w[8], c[8];
  load_vec8(w, a.weight, m.col, true, 1.f);
  load_vec8(c, a.bias, m.col, true, 0.f);
  const int head = m.col / LPH;
  for (int64_t t = m.t0; t < a.rows; t += a.R) {
    const int64_t u = t * m.units + m.col;
    Row8<T> ro, rg;
    load_row8(ro, (const T*)a.O + 8 * u, true);
    load_row8(rg, (const T*)a.G + 8 * u, true);
    float o[8], g[8];
    unpack_row8(o, ro);
    unpack_row8(g, rg);
    if constexpr (F != kQNone) {
      q_store8<F>(o, a.O_q, a.O_qs, u);
      q_store8<F>(g, a.G_q, a.G_qs, u);
    }
    float mu = 0.f;
    if (a.layer) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s += o[e];
      mu = group_sum<LPH>(s) * inv_d;
    }
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      o[e] -= mu;
      q += o[e] * o[e];
    }
    const float r = 1.f / sqrtf(group_sum<LPH>(q) * inv_d + a.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = g[e] * sigmoid_fast(g[e]) * (o[e] * r * w[e] + c[e]);
    pack_row8(ro, o);
    store_row8((T*)a.Z + 8 * u, ro);
    if (m.col % LPH == 0) {
      if (a.mean) a.mean[t * a.heads + head] = mu;
      if (a.rstd) a.rstd[t * a.heads + head] = r;
    }
  }
}

template <class T, int LPH, int F>
__global__ __launch_bounds__(256) void k_gated_norm_bwd(GatedNormBwdArgs a) {
  __shared__ float comb[256 * 8];
  const GateMap m(a.heads, LPH, a.R);
  if (!m.on) return;                           // only where a token spans workgroups: no barrier below then
  constexpr float inv_d = 1.f / (8.f * LPH);
  float w[8], c[8], aw[8], ac[8];
  load_vec8(w, a.weight, m.col, true, 1.f);
  load_vec8(c, a.bias, m.col, true, 0.f);
#pragma unroll
  for (int e = 0; e < 8; ++e) aw[e] = ac[e] = 0.f;
  const int head = m.col / LPH;
  for (int64_t t = m.t0; t < a.rows; t += a.R) {
    const int64_t u = t * m.units + m.col;
    Row8<T> rz;
    Held<T, F> ho, hg;
    load_row8(rz, (const T*)a.dZ + 8 * u, true);
    ho.load(a.O, a.O_qs, u);
    hg.load(a.G, a.G_qs, u);
    const float mu = a.layer ? a.mean[t * a.heads + head] : 0.f, r = a.rstd[t * a.heads + head];
    float xh[8], g[8], dz[8], z[8];
    ho.values(xh);
    hg.values(g);
    unpack_row8(dz, rz);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      xh[e] = (xh[e] - mu) * r;
      const float n = xh[e] * w[e] + c[e], sg = sigmoid_fast(g[e]), sw = g[e] * sg;
      z[e] = sw * n;
      const float dn = dz[e] * sw;
      g[e] = dz[e] * n * (sg * (1.f + g[e] * (1.f - sg)));
      aw[e] += dn * xh[e];
      ac[e] += dn;
      dz[e] = dn * w[e];
      s1 += dz[e];
      s2 += dz[e] * xh[e];
    }
    const float m1 = a.layer ? group_sum<LPH>(s1) * inv_d : 0.f, m2 = group_sum<LPH>(s2) * inv_d;
#pragma unroll
    for (int e = 0; e < 8; ++e) xh[e] = r * (dz[e] - m1 - xh[e] * m2);
    Row8<T> ro;
    pack_row8(ro, xh);
    store_row8((T*)a.dO + 8 * u, ro);
    pack_row8(ro, g);
    store_row8((T*)a.dG + 8 * u, ro);
    if (a.Z) {
      pack_row8(ro, z);
      store_row8((T*)a.Z + 8 * u, ro);
    }
  }
  // partial sums: one row of heads * d_v per requested vector and workgroup
  // (its tokens added up first), or per t0 where a token spans workgroups
  const int64_t n = 8 * (int64_t)m.units;
  const bool whole = m.units <= 256;
  const int64_t P = whole ? (int64_t)gridDim.x : (int64_t)a.R;
  float* dst = a.part + (whole ? (int64_t)blockIdx.x : (int64_t)m.t0) * n + 8 * m.col;
  auto put = [&](const float* v) {
    if (whole) {
      __syncthreads();
      store_vec8(comb + 8 * threadIdx.x, v);
      __syncthreads();
      if ((int)threadIdx.x < m.units) {
        float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int i = threadIdx.x; i < (int)blockDim.x; i += m.units)
#pragma unroll
          for (int e = 0; e < 8; ++e) t[e] += comb[8 * i + e];
        store_vec8(dst, t);
      }
    } else {
      store_vec8(dst, v);
    }
    dst += P * n;
  };
  if (a.sum_w) put(aw);
  if (a.sum_c) put(ac);
}

// ------------------------------------------------------------- launch shapes
// Row kernels: lanes per row and units per thread.  Up to 512 columns a row
// is a group of a wave; beyond, a workgroup.
struct RowShape {
  int lpr, vpt, threads, rpb;
};
RowShape row_shape(int d) {
  const int units = d / 8;
  RowShape s{0, 1, 256, 1};
  if (units <= 64) {
    s.lpr = 8;
    while (s.lpr < units) s.lpr *= 2;
    s.rpb = 256 / s.lpr;
    return s;
  }
  s.vpt = units <= 512 ? 1 : 2;
  s.threads = ((units + s.vpt - 1) / s.vpt + 63) / 64 * 64;
  return s;
}
// Workgroups of a row kernel: as many as the card keeps in flight at once
// (2048 threads per CU), and no more than there are rows.
int row_grid(const RowShape& s, int64_t rows, int per_cu_threads) {
  const int64_t want = (rows + s.rpb - 1) / s.rpb, cap = (int64_t)256 * std::max(1, per_cu_threads / s.threads);
  return (int)std::max<int64_t>(1, std::min(want, cap));
}
constexpr int kFwdThreads = 2048, kBwdThreads = 1024;

}  // namespace

int resid_norm_bwd_parts(int64_t rows, int d) { return rows ? row_grid(row_shape(d), rows, kBwdThreads) : 0; }

namespace {
// Launch of a gated_norm kernel: threads per workgroup, workgroups, tokens
// side by side (R) and partial rows (P).
struct GateShape {
  int threads, grid, R, P;
};
GateShape gate_shape(int64_t rows, int heads, int d_v, int per_cu_threads) {
  GateShape g{256, 0, 0, 0};
  const int units = heads * d_v / 8;
  const int64_t cap = (int64_t)256 * per_cu_threads;     // threads in flight
  if (units <= 256) {
    const int tok = 256 / units;                         // tokens per workgroup
    g.threads = tok * units;
    g.grid = (int)std::min<int64_t>((rows + tok - 1) / tok, cap / 256);
    g.R = g.grid * tok;
    g.P = g.grid;
  } else {
    g.R = (int)std::min<int64_t>(rows, std::max<int64_t>(1, cap / units));
    g.grid = (int)(((int64_t)g.R * units + 255) / 256);
    g.P = g.R;
  }
  return g;
}
}  // namespace

int gated_norm_bwd_parts(int64_t rows, int heads, int d_v) { return gate_shape(rows, heads, d_v, kBwdThreads).P; }

hipError_t launch_col_sums(const float* part, int P, int n, const ColSumOut& out, int vecs, hipStream_t st) {
  if (vecs == 0) return hipSuccess;
  TraceScope ts("k_col_sums", st);
  hipLaunchKernelGGL(k_col_sums, dim3((n + 63) / 64, vecs), dim3(1024), 0, st, part, P, n, out);
  return hipGetLastError();
}

#define MSR_ROW_CASES(F_, CALL)                                                          \
  switch (s.lpr) {                                                                       \
    case 8: CALL(8, 1, F_) break;                                                        \
    case 16: CALL(16, 1, F_) break;                                                      \
    case 32: CALL(32, 1, F_) break;                                                      \
    case 64: CALL(64, 1, F_) break;                                                      \
    default:                                                                             \
      if (s.vpt == 1) { CALL(0, 1, F_) } else { CALL(0, 2, F_) }                         \
  }
#define MSR_FMT_CASES(CASES, CALL)                                                       \
  switch (a.fmt) {                                                                       \
    case kQE4M3: CASES(kQE4M3, CALL) break;                                              \
    case kQI8: CASES(kQI8, CALL) break;                                                  \
    default: CASES(kQNone, CALL)                                                         \
  }

hipError_t launch_resid_norm_fwd(const ResidNormArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  TraceScope ts("k_resid_norm_fwd", st);
  const RowShape s = row_shape(a.d);
  const dim3 grid(row_grid(s, a.rows, kFwdThreads)), block(s.threads);
#define MSR_F32(L, V, F_) hipLaunchKernelGGL((k_resid_norm_fwd<float, L, V, F_>), grid, block, 0, st, a);
#define MSR_B16(L, V, F_) hipLaunchKernelGGL((k_resid_norm_fwd<bf16, L, V, F_>), grid, block, 0, st, a);
  if (a.elt == kBF16) { MSR_FMT_CASES(MSR_ROW_CASES, MSR_B16) } else { MSR_FMT_CASES(MSR_ROW_CASES, MSR_F32) }
#undef MSR_F32
#undef MSR_B16
  return hipGetLastError();
}

hipError_t launch_resid_norm_bwd(const ResidNormBwdArgs& a0, float* dscale, float* dweight, float* dbias,
                                 hipStream_t st) {
  ResidNormBwdArgs a = a0;
  const RowShape s = row_shape(a.d);
  const int P = resid_norm_bwd_parts(a.rows, a.d);
  a.sum_w = dweight != nullptr;
  a.sum_c = dbias != nullptr;
  if (a.rows) {
    TraceScope ts("k_resid_norm_bwd", st);
    const dim3 grid(P), block(s.threads);
#define MSR_F32(L, V, F_)                                                                       \
  if (dscale) hipLaunchKernelGGL((k_resid_norm_bwd<float, L, V, F_, true>), grid, block, 0, st, a); \
  else hipLaunchKernelGGL((k_resid_norm_bwd<float, L, V, F_, false>), grid, block, 0, st, a);
#define MSR_B16(L, V, F_)                                                                       \
  if (dscale) hipLaunchKernelGGL((k_resid_norm_bwd<bf16, L, V, F_, true>), grid, block, 0, st, a); \
  else hipLaunchKernelGGL((k_resid_norm_bwd<bf16, L, V, F_, false>), grid, block, 0, st, a);
    if (a.elt == kBF16) { MSR_FMT_CASES(MSR_ROW_CASES, MSR_B16) } else { MSR_FMT_CASES(MSR_ROW_CASES, MSR_F32) }
#undef MSR_F32
#undef MSR_B16
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  ColSumOut out{};
  int n = 0;
  if (dweight) out.v[n++] = dweight;
  if (dbias) out.v[n++] = dbias;
  if (dscale) out.v[n++] = dscale;
  return launch_col_sums(a.part, P, a.d, out, n, st);
}

#define MSR_GATE_CASES(F_, CALL)                                                         \
  switch (a.d_v) {                                                                       \
    case 64: CALL(8, F_) break;                                                          \
    case 128: CALL(16, F_) break;                                                        \
    case 256: CALL(32, F_) break;                                                        \
    default: CALL(64, F_)                                                                \
  }

hipError_t launch_gated_norm_fwd(const GatedNormArgs& a0, hipStream_t st) {
  GatedNormArgs a = a0;
  if (a.rows == 0) return hipSuccess;
  TraceScope ts("k_gated_norm_fwd", st);
  const GateShape gs = gate_shape(a.rows, a.heads, a.d_v, kFwdThreads);
  a.R = gs.R;
  const dim3 grid(gs.grid), block(gs.threads);
#define MSR_F32(L, F_) hipLaunchKernelGGL((k_gated_norm_fwd<float, L, F_>), grid, block, 0, st, a);
#define MSR_B16(L, F_) hipLaunchKernelGGL((k_gated_norm_fwd<bf16, L, F_>), grid, block, 0, st, a);
  if (a.elt == kBF16) { MSR_FMT_CASES(MSR_GATE_CASES, MSR_B16) } else { MSR_FMT_CASES(MSR_GATE_CASES, MSR_F32) }
#undef MSR_F32
#undef MSR_B16
  return hipGetLastError();
}

hipError_t launch_gated_norm_bwd(const GatedNormBwdArgs& a0, float* dweight, float* dbias, hipStream_t st) {
  GatedNormBwdArgs a = a0;
  const GateShape gs = gate_shape(a.rows, a.heads, a.d_v, kBwdThreads);
  a.R = gs.R;
  a.sum_w = dweight != nullptr;
  a.sum_c = dbias != nullptr;
  if (a.rows) {
    TraceScope ts("k_gated_norm_bwd", st);
    const dim3 grid(gs.grid), block(gs.threads);
#define MSR_F32(L, F_) hipLaunchKernelGGL((k_gated_norm_bwd<float, L, F_>), grid, block, 0, st, a);
#define MSR_B16(L, F_) hipLaunchKernelGGL((k_gated_norm_bwd<bf16, L, F_>), grid, block, 0, st, a);
    if (a.elt == kBF16) { MSR_FMT_CASES(MSR_GATE_CASES, MSR_B16) } else { MSR_FMT_CASES(MSR_GATE_CASES, MSR_F32) }
#undef MSR_F32
#undef MSR_B16
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  ColSumOut out{};
  int n = 0;
  if (dweight) out.v[n++] = dweight;
  if (dbias) out.v[n++] = dbias;
  return launch_col_sums(a.part, gs.P, a.heads * a.d_v, out, n, st);
}

}  // namespace msr
