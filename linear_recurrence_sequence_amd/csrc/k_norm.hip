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
// HBM.  A lane holds 8 values (16-byte loads); a row's sums stay in registers
// and lane exchanges.  The sums over tokens (ds, dw, dc) are carried in
// registers while a thread walks down its columns; the walkers' float32
// partials are then added in a fixed order in 64 bits by k_col_sums (no
// atomics: the same bits every time).
#include <algorithm>

#include "msr_launch.h"
#include "msr_q8.h"

namespace msr {

namespace {

constexpr int kMaxWaves = 16;

// Sum of x over the lanes that share a row: a group of LPR lanes of a wave,
// or (LPR == 0) the tpr threads (whole waves) of the workgroup's row `rib`,
// through red, whose two halves take turns: a wave writes a half again only
// after the barrier of the other half, which every wave reaches after
// reading the first.
template <int LPR, int NV>
__device__ __forceinline__ void row_sums(float (&x)[NV], float (*red)[kMaxWaves][2], int& turn, int rib, int tpr) {
  static_assert(NV <= 2 && kMaxWaves == 16, "red holds two values per wave, summed by 16 lanes");
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = group_sum<LPR == 0 ? 64 : LPR>(x[i]);
  if constexpr (LPR == 0) {
    const int nw = tpr >> 6, w0 = rib * nw, wave = threadIdx.x >> 6, l = threadIdx.x & 15;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) red[turn][wave][i] = x[i];
    __syncthreads();
    const int from = min(w0 + l, kMaxWaves - 1);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float v = red[turn][from][i];
      x[i] = group_sum<16>(l < nw ? v : 0.f);
    }
    turn ^= 1;
  }
}

// alpha x + s b, each product and the sum rounded to float32 (no fused
// multiply-add): the same value in every implementation of the formula, and
// so the same rounding to T and the same 8-bit codes.
__device__ __forceinline__ float scaled_sum(float alpha, float x, float s, float b) {
#pragma clang fp contract(off)
  const float p = alpha * x, q = s * b;
  return p + q;
}

// Walks first, first + stride, ... below end: load(row, at) issues the loads
// of a turn, step(row, at) computes it, AHEAD turns later.  The turns' rows
// sit in registers (the loop is unrolled over them, nothing is copied).
// Turns past the end load nothing (their windows are empty).
template <int AHEAD, class Row, class Load, class Step>
__device__ __forceinline__ void pipelined(int64_t first, int64_t end, int64_t stride, Load&& load, Step&& step) {
  Row q[AHEAD + 1];
  static_for<AHEAD>([&](auto i) __attribute__((always_inline)) { load(q[i], first + i * stride); });
  bool more = first < end;
  while (more) {
    static_for<AHEAD + 1>([&](auto i) __attribute__((always_inline)) {
      if (more) {
        load(q[(i + AHEAD) % (AHEAD + 1)], first + AHEAD * stride);
        step(q[i], first);
        first += stride;
        more = first < end;
      }
    });
  }
}

// Rows of a row kernel: LPR lanes (a group of a wave) per row, or LPR == 0:
// tpr threads (whole waves).  A thread holds units u0 + k step, k < VPT, of
// the row's d / 8; the workgroup rpb rows side by side, and unit k of a
// thread lies off(k) elements behind the start of the first of them
// (outside every window where the row has no such unit).
template <int LPR>
struct RowMap {
  int tpr, rpb, rib, u0, d;         // threads per row, rows, row in the workgroup, first unit, columns
  __device__ __forceinline__ RowMap(int tpr_, int d_) : d(d_) {
    tpr = LPR ? LPR : tpr_;
    rpb = blockDim.x / tpr;
    rib = threadIdx.x / tpr;
    if constexpr (LPR == 0) rib = __builtin_amdgcn_readfirstlane(rib);   // whole waves
    u0 = threadIdx.x - rib * tpr;
  }
  __device__ __forceinline__ int unit(int k) const { return u0 + k * tpr; }
  // in its row, and behind the start of the workgroup's first row
  template <class T>
  __device__ __forceinline__ Unit at(int k) const {
    return unit(k) < d / 8 ? unit_of<T>(0, unit(k), d / 8) : kNoUnit;
  }
  template <class T>
  __device__ __forceinline__ Unit off(int k) const {
    return unit(k) < d / 8 ? unit_of<T>((uint32_t)(rib * d), unit(k), d / 8) : kNoUnit;
  }
};

// 2 tensors read, 2 written (and 33/32 bytes a value with an 8-bit copy),
// about 10 operations a value: bound by HBM.  A row's mean, then its centred
// squares, in registers (the sums of squares of an off-centre row would
// cancel); weight, bias and scale stay in registers for the workgroup's
// rows, and the next row's loads are in flight.  32768 x 4096 bf16 with an
// e4m3 copy: 215 us, 5.6 TB/s.
template <class T, int LPR, int VPT, int F>
__global__ __launch_bounds__(LPR ? 256 : 512) void k_resid_norm_fwd(ResidNormArgs a) {
  __shared__ float red[2][kMaxWaves][2];
  const RowMap<LPR> m(blockDim.x, a.d);
  const float inv_d = 1.f / (float)a.d;
  float w[VPT][8], c[VPT][8], s[VPT][8];
  Unit off[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    off[k] = m.template off<T>(k);
    const Unit at = m.template at<T>(k);
    load_vec8(w[k], a.weight, at, 1.f);
    load_vec8(c[k], a.bias, at, 0.f);
    // without B its window reads 0, and -1 * 0 = -0 changes no alpha x
    load_vec8(s[k], a.scale, at, a.B ? 1.f : -1.f);
  }
  struct Row {
    Row8<T> x[VPT], b[VPT];
  };
  const int64_t first = (int64_t)blockIdx.x * a.chunk * m.rpb;
  const int64_t end = min(a.rows, first + (int64_t)a.chunk * m.rpb);
  // elements of the rows that this turn's windows hold
  auto span = [&](int64_t row0) { return (uint32_t)(max((int64_t)0, min((int64_t)m.rpb, end - row0)) * a.d); };
  auto load = [&](Row& q, int64_t row0) __attribute__((always_inline)) {
    const uint32_t bytes = span(row0) * (uint32_t)sizeof(T);
    const Win wx((const T*)a.X + row0 * a.d, bytes), wb(a.B ? (const T*)a.B + row0 * a.d : nullptr, bytes);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      win_load8(q.x[k], wx, off[k]);
      win_load8(q.b[k], wb, off[k]);
    }
  };
  int turn = 0;
  auto step = [&](const Row& cur, int64_t row0) __attribute__((always_inline)) {
    const int64_t at = row0 * a.d;
    const uint32_t n = span(row0), bytes = n * (uint32_t)sizeof(T);
    const Win wh(a.H ? (T*)a.H + at : nullptr, bytes), wy((T*)a.Y + at, bytes);
    float h[VPT][8];
    float sum[1] = {0.f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float x[8], b[8];
      unpack_row8(x, cur.x[k]);
      unpack_row8(b, cur.b[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = scaled_sum(a.alpha, x[e], s[k][e], b[e]);
      Row8<T> rh;
      pack_row8(rh, h[k]);
      unpack_row8(h[k], rh);                   // the norm reads the sum as it is held
      win_store8(wh, off[k], rh);
      if constexpr (F != kQNone) {
        q_store8(h[k], HeldWin<T, F>(a.H_q, a.H_qs, at, n), off[k]);
        if (a.B_q) q_store8(b, HeldWin<T, F>(a.B_q, a.B_qs, at, n), off[k]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] += h[k][e];
    }
    float mu = 0.f;
    if (a.layer) {
      row_sums<LPR>(sum, red, turn, 0, m.tpr);
      mu = sum[0] * inv_d;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const bool on = off[k].on();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[k][e] -= mu;
        q[0] += on ? h[k][e] * h[k][e] : 0.f;
      }
    }
    row_sums<LPR>(q, red, turn, 0, m.tpr);
    const float r = 1.f / sqrtf(q[0] * inv_d + a.eps);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = h[k][e] * r * w[k][e] + c[k][e];
      Row8<T> ry;
      pack_row8(ry, y);
      win_store8(wy, off[k], ry);
    }
    const uint32_t so = m.u0 == 0 ? 4u * (uint32_t)m.rib : kOutside, sn = 4u * (uint32_t)(n / (uint32_t)a.d);
    win_store_f32(Win(a.mean ? a.mean + row0 : nullptr, sn), so, mu);
    win_store_f32(Win(a.rstd ? a.rstd + row0 : nullptr, sn), so, r);
  };
  pipelined<1, Row>(first, end, m.rpb, load, step);
}

// What the backward reads of one row, as loaded: the loads of the next rows
// are in flight while this one's sums go round.
template <class T, int VPT, int F, bool DS>
struct BwdRow {
  Row8<T> dy[VPT], dh[VPT];
  Held<T, F> h[VPT], b[DS ? VPT : 1];
  float mu, r;
};

// Threads of the backward's workgroup at most: what the registers hold
// without spilling.
template <class T, int LPR, int VPT>
constexpr int bwd_threads() { return LPR ? 256 : sizeof(T) == 2 && VPT == 1 ? 1024 : 512; }

// 3 tensors read (4 with DS), 1 or 2 written, about 15 operations a value:
// bound by HBM.  Rows are walked by a fixed set of workgroups, several rows
// side by side, so that a workgroup's columns keep their sums over tokens in
// registers; both row sums go round in one exchange.  32767 x 2560 bf16 from
// int8: 100 us, 5.8 TB/s (126 us with one row a workgroup, plain loads and no
// row ahead); 16384 x 2048 with dscale: 70 us, 5.8 TB/s.
template <class T, int LPR, int VPT, int F, bool DS>
__global__ __launch_bounds__((bwd_threads<T, LPR, VPT>())) void k_resid_norm_bwd(ResidNormBwdArgs a) {
  constexpr int kThreads = bwd_threads<T, LPR, VPT>();
  constexpr int kUnits = LPR ? LPR : VPT == 1 ? 512 : 1024;     // of a row, at most
  __shared__ float red[2][kMaxWaves][2];
  // weight and scale (read each row: two 16-byte reads a unit cost less than
  // the registers), then the partial sums of the rows side by side
  __shared__ __attribute__((aligned(16))) float lds[kUnits * 16 > kThreads * 8 ? kUnits * 16 : kThreads * 8];
  const RowMap<LPR> m(a.tpr, a.d);
  const int units = a.d / 8;
  const float inv_d = 1.f / (float)a.d;
  f32x4* const vec = reinterpret_cast<f32x4*>(lds);             // [weight, scale][half][unit]
  for (int i = threadIdx.x; i < 4 * units; i += blockDim.x) {
    const int v = i / (2 * units), j = i % (2 * units);          // vector, 16-byte piece of it
    const int half = sizeof(T) == 2 ? j & 1 : j >= units, u = sizeof(T) == 2 ? j >> 1 : j - half * units;
    const float* p = v ? a.scale : a.weight;
    vec[v * 2 * kUnits + half * kUnits + u] =
        p ? *reinterpret_cast<const f32x4*>(p + 4 * j) : (f32x4){1.f, 1.f, 1.f, 1.f};
  }
  auto vec8 = [&](float* o, int v, int u) {
    const f32x4 x = vec[v * 2 * kUnits + u], y = vec[v * 2 * kUnits + kUnits + u];
#pragma unroll
    for (int e = 0; e < 4; ++e) { o[e] = x[e]; o[4 + e] = y[e]; }
  };
  __syncthreads();
  float aw[VPT][8], ac[VPT][8], as[DS ? VPT : 1][8];
  Unit off[VPT];
  int unit[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    off[k] = m.template off<T>(k);
    unit[k] = min(m.unit(k), units - 1);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      aw[k][e] = ac[k][e] = 0.f;
      if constexpr (DS) as[k][e] = 0.f;
    }
  }
  using Row = BwdRow<T, VPT, F, DS>;
  // elements of the rows that this turn's windows hold; rows past the end and
  // units past a row read as zeros, r among them, and change nothing
  auto span = [&](int64_t row0) { return (uint32_t)(max((int64_t)0, min((int64_t)m.rpb, a.rows - row0)) * a.d); };
  auto load = [&](Row& q, int64_t row0) __attribute__((always_inline)) {
    const int64_t at = row0 * a.d;
    const uint32_t n = span(row0), bytes = n * (uint32_t)sizeof(T), sn = 4u * (n / (uint32_t)a.d);
    const Win wy((const T*)a.dY + at, bytes), wd(a.dH_in ? (const T*)a.dH_in + at : nullptr, bytes);
    const HeldWin<T, F> wh(a.H, a.H_qs, at, n), wb(DS ? a.B : nullptr, DS ? a.B_qs : nullptr, at, n);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      win_load8(q.dy[k], wy, off[k]);
      q.h[k].load(wh, off[k]);
      win_load8(q.dh[k], wd, off[k]);
      if constexpr (DS) q.b[k].load(wb, off[k]);
    }
    q.mu = win_load_f32(Win(a.layer ? a.mean + row0 : nullptr, sn), 4u * (uint32_t)m.rib);
    q.r = win_load_f32(Win(a.rstd + row0, sn), 4u * (uint32_t)m.rib);
  };
  const float layer = a.layer ? inv_d : 0.f;
  int turn = 0;
  auto step = [&](const Row& cur, int64_t row0) __attribute__((always_inline)) {
    const int64_t at = row0 * a.d;
    const uint32_t bytes = span(row0) * (uint32_t)sizeof(T);
    const Win wx((T*)a.dX + at, bytes), wb(a.dB ? (T*)a.dB + at : nullptr, bytes);
    const float r = cur.r, mur = cur.mu * r;
    float xh[VPT][8], g[VPT][8];
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float w[8];
      vec8(w, 0, unit[k]);
      cur.h[k].raw(xh[k]);
      unpack_row8(g[k], cur.dy[k]);
      const float rs = cur.h[k].scale() * r;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[k][e] = xh[k][e] * rs - mur;
        aw[k][e] += g[k][e] * xh[k][e];
        ac[k][e] += g[k][e];
        g[k][e] *= w[e];
        sum[0] += g[k][e];
        sum[1] += g[k][e] * xh[k][e];
      }
    }
    row_sums<LPR>(sum, red, turn, m.rib, m.tpr);
    const float m1 = sum[0] * layer * r, m2 = sum[1] * inv_d * r;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float dh[8], o[8];
      unpack_row8(dh, cur.dh[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) dh[e] += r * g[k][e] - (xh[k][e] * m2 + m1);
      if constexpr (DS) {
        float b[8];
        cur.b[k].values(b);
#pragma unroll
        for (int e = 0; e < 8; ++e) as[k][e] += dh[e] * b[e];
      }
      Row8<T> ro;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = a.alpha * dh[e];
      pack_row8(ro, o);
      win_store8(wx, off[k], ro);
      if (a.dB) {
        float s[8];
        vec8(s, 1, unit[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = s[e] * dh[e];
        pack_row8(ro, o);
        win_store8(wb, off[k], ro);
      }
    }
  };
  // every thread of the workgroup takes every turn (row_sums has a barrier)
  const int64_t stride = (int64_t)gridDim.x * m.rpb;
  pipelined<1, Row>((int64_t)blockIdx.x * m.rpb, a.rows, stride, load, step);
  // this workgroup's partial sums over its rows (those side by side added
  // first), one row of d per requested vector
  auto put = [&](float (&v)[VPT][8], float* dst) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      __syncthreads();
      store_vec8(lds, {8 * threadIdx.x, 8 * threadIdx.x + 4}, v[k]);
      __syncthreads();
      if (m.rib == 0 && off[k].on()) {
        float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < m.rpb; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) t[e] += lds[8 * (i * m.tpr + m.u0) + e];
        store_vec8(dst + (int64_t)blockIdx.x * a.d, m.template at<T>(k), t);
      }
    }
  };
  const int64_t plane = (int64_t)gridDim.x * a.d;
  float* dst = a.part;
  if (a.sum_w) { put(aw, dst); dst += plane; }
  if (a.sum_c) { put(ac, dst); dst += plane; }
  if constexpr (DS) put(as, dst);
}

// Column sums, 2-4 us: out[v][j] = sum_p part[v][p][j] in 64 bits, in order of p
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
  // this thread's unit in a token
  template <class T>
  __device__ __forceinline__ Unit at(int lph) const {
    return unit_of<T>(8u * (uint32_t)(col - col % lph), col % lph, lph);
  }
  // its unit, and the bytes of its statistics, behind those of the first of
  // the tokens that the grid holds side by side (R units <= 2^20)
  template <class T>
  __device__ __forceinline__ Unit off(int lph) const {
    const uint32_t t = 8u * (uint32_t)(t0 * units);
    const Unit u = at<T>(lph);
    return on ? Unit{t + u.lo, t + u.hi} : kNoUnit;
  }
  __device__ __forceinline__ uint32_t stat_off(int heads, int lph) const {
    return on ? 4u * (uint32_t)(t0 * heads + col / lph) : kOutside;
  }
};

__device__ __forceinline__ float sigmoid_fast(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}

// Elements and statistics that the windows of a turn hold: of the tokens
// from `first` on, at most R side by side.
struct GateSpan {
  int64_t at, sat;
  uint32_t n, sn;
  __device__ __forceinline__ GateSpan(int64_t first, int64_t rows, int R, int units, int heads)
      : at(first * 8 * units), sat(first * heads) {
    const uint32_t t = (uint32_t)max((int64_t)0, min((int64_t)R, rows - first));
    n = t * 8u * (uint32_t)units;
    sn = t * 4u * (uint32_t)heads;
  }
};

// 2 tensors read, 1 written, about 15 operations a value: bound by HBM.
// 16384 x 8 x 256 bf16: 36 us, 5.6 TB/s.
template <class T, int LPH, int F>
__global__ __launch_bounds__(256) void k_gated_norm_fwd(GatedNormArgs a) {
  const GateMap m(a.heads, LPH, a.R);
  constexpr float inv_d = 1.f / (8.f * LPH);
  float w[8], c[8];
  const Unit off = m.template off<T>(LPH);
  load_vec8(w, a.weight, m.template at<T>(LPH), 1.f);
  load_vec8(c, a.bias, m.template at<T>(LPH), 0.f);
  const uint32_t soff = m.col % LPH == 0 ? m.stat_off(a.heads, LPH) : kOutside;
  struct Row {
    Row8<T> o, g;
  };
  auto load = [&](Row& q, int64_t first) __attribute__((always_inline)) {
    const GateSpan sp(first, a.rows, a.R, m.units, a.heads);
    const uint32_t bytes = sp.n * (uint32_t)sizeof(T);
    win_load8(q.o, Win((const T*)a.O + sp.at, bytes), off);
    win_load8(q.g, Win((const T*)a.G + sp.at, bytes), off);
  };
  auto step = [&](const Row& cur, int64_t first) __attribute__((always_inline)) {
    const GateSpan sp(first, a.rows, a.R, m.units, a.heads);
    float o[8], g[8];
    unpack_row8(o, cur.o);
    unpack_row8(g, cur.g);
    if constexpr (F != kQNone) {
      q_store8(o, HeldWin<T, F>(a.O_q, a.O_qs, sp.at, sp.n), off);
      q_store8(g, HeldWin<T, F>(a.G_q, a.G_qs, sp.at, sp.n), off);
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += o[e];
    const float mu = a.layer ? group_sum<LPH>(s) * inv_d : 0.f;
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      o[e] -= mu;
      q += o[e] * o[e];
    }
    const float r = 1.f / sqrtf(group_sum<LPH>(q) * inv_d + a.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = g[e] * sigmoid_fast(g[e]) * (o[e] * r * w[e] + c[e]);
    Row8<T> rz;
    pack_row8(rz, o);
    win_store8(Win((T*)a.Z + sp.at, sp.n * (uint32_t)sizeof(T)), off, rz);
    win_store_f32(Win(a.mean ? a.mean + sp.sat : nullptr, sp.sn), soff, mu);
    win_store_f32(Win(a.rstd ? a.rstd + sp.sat : nullptr, sp.sn), soff, r);
  };
  pipelined<1, Row>(0, a.rows, a.R, load, step);
}

// 3 tensors read, 2 or 3 written, about 30 operations a value, two of them
// (exp2, reciprocal) at a quarter of the rate: bound by HBM, with half of the
// VALU's time behind it.  32768 x 16 x 512 bf16 from e4m3, Z again: 494 us,
// 5.5 TB/s; 16384 x 8 x 256 from bf16: 63 us, 5.4 TB/s.
template <class T, int LPH, int F>
__global__ __launch_bounds__(256) void k_gated_norm_bwd(GatedNormBwdArgs a) {
  // this thread's weight and bias (read each token: four 16-byte reads cost
  // less than 16 registers), then the partial sums
  __shared__ f32x4 vec[4][256];
  const GateMap m(a.heads, LPH, a.R);
  constexpr float inv_d = 1.f / (8.f * LPH);
  float aw[8], ac[8];
  {
    float w[8], c[8];
    load_vec8(w, a.weight, m.template at<T>(LPH), 1.f);
    load_vec8(c, a.bias, m.template at<T>(LPH), 0.f);
    vec[0][threadIdx.x] = (f32x4){w[0], w[1], w[2], w[3]};
    vec[1][threadIdx.x] = (f32x4){w[4], w[5], w[6], w[7]};
    vec[2][threadIdx.x] = (f32x4){c[0], c[1], c[2], c[3]};
    vec[3][threadIdx.x] = (f32x4){c[4], c[5], c[6], c[7]};
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) aw[e] = ac[e] = 0.f;
  const Unit off = m.template off<T>(LPH);
  const uint32_t soff = m.stat_off(a.heads, LPH);
  struct Row {
    Row8<T> z;
    Held<T, F> o, g;
    float mu, r;
  };
  auto load = [&](Row& q, int64_t first) __attribute__((always_inline)) {
    const GateSpan sp(first, a.rows, a.R, m.units, a.heads);
    win_load8(q.z, Win((const T*)a.dZ + sp.at, sp.n * (uint32_t)sizeof(T)), off);
    q.o.load(HeldWin<T, F>(a.O, a.O_qs, sp.at, sp.n), off);
    q.g.load(HeldWin<T, F>(a.G, a.G_qs, sp.at, sp.n), off);
    q.mu = win_load_f32(Win(a.layer ? a.mean + sp.sat : nullptr, sp.sn), soff);
    q.r = win_load_f32(Win(a.rstd + sp.sat, sp.sn), soff);
  };
  const float layer = a.layer ? inv_d : 0.f;
  // tokens past the end read as zeros, dZ among them, and change nothing
  auto step = [&](const Row& cur, int64_t first) __attribute__((always_inline)) {
    const GateSpan sp(first, a.rows, a.R, m.units, a.heads);
    const uint32_t bytes = sp.n * (uint32_t)sizeof(T);
    const float r = cur.r, mur = cur.mu * r, rs = cur.o.scale() * r;
    float xh[8], g[8], dz[8], z[8];
    cur.o.raw(xh);
    cur.g.values(g);
    unpack_row8(dz, cur.z);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 w = vec[h][threadIdx.x], c = vec[2 + h][threadIdx.x];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 4 * h + j;
        xh[e] = xh[e] * rs - mur;
        const float n = xh[e] * w[j] + c[j], sg = sigmoid_fast(g[e]), sw = g[e] * sg;
        z[e] = sw * n;
        const float dn = dz[e] * sw;
        g[e] = dz[e] * n * (sg + sw * (1.f - sg));
        aw[e] += dn * xh[e];
        ac[e] += dn;
        dz[e] = dn * w[j];
        s1 += dz[e];
        s2 += dz[e] * xh[e];
      }
    }
    Row8<T> ro;
    pack_row8(ro, g);
    win_store8(Win((T*)a.dG + sp.at, bytes), off, ro);
    pack_row8(ro, z);
    win_store8(Win(a.Z ? (T*)a.Z + sp.at : nullptr, bytes), off, ro);
    const float m1 = group_sum<LPH>(s1) * layer * r, m2 = group_sum<LPH>(s2) * inv_d * r;
#pragma unroll
    for (int e = 0; e < 8; ++e) xh[e] = r * dz[e] - (xh[e] * m2 + m1);
    pack_row8(ro, xh);
    win_store8(Win((T*)a.dO + sp.at, bytes), off, ro);
  };
  pipelined<2, Row>(0, a.rows, a.R, load, step);
  float* const comb = reinterpret_cast<float*>(vec);
  // partial sums: one row of heads * d_v per requested vector and workgroup
  // (its tokens added up first), or per t0 where a token spans workgroups
  const int64_t n = 8 * (int64_t)m.units;
  const bool whole = m.units <= 256;
  const int64_t P = whole ? (int64_t)gridDim.x : (int64_t)a.R;
  float* dst = a.part + (whole ? (int64_t)blockIdx.x : (int64_t)m.t0) * n;
  const Unit at = m.template at<T>(LPH);
  auto put = [&](const float* v) {
    if (whole) {
      __syncthreads();
      store_vec8(comb, {8 * threadIdx.x, 8 * threadIdx.x + 4}, v);
      __syncthreads();
      if ((int)threadIdx.x < m.units) {
        float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int i = threadIdx.x; i < (int)blockDim.x; i += m.units)
#pragma unroll
          for (int e = 0; e < 8; ++e) t[e] += comb[8 * i + e];
        store_vec8(dst, at, t);
      }
    } else if (m.on) {
      store_vec8(dst, at, v);
    }
    dst += P * n;
  };
  if (a.sum_w) put(aw);
  if (a.sum_c) put(ac);
}

// ------------------------------------------------------------- launch shapes
// Row kernels: lanes per row (0: whole waves), threads per row and units per
// thread.  Up to 512 columns a row is a group of a wave; beyond, as many
// waves as hold it at one unit (two above 4096 columns) a thread.
struct RowShape {
  int lpr, tpr, vpt;
};
RowShape row_shape(int d) {
  const int units = d / 8;
  RowShape s{0, 0, 1};
  if (units <= 64) {
    s.lpr = 8;
    while (s.lpr < units) s.lpr *= 2;
    s.tpr = s.lpr;
    return s;
  }
  s.vpt = units <= 512 ? 1 : 2;
  s.tpr = ((units + s.vpt - 1) / s.vpt + 63) / 64 * 64;
  return s;
}
// Threads per CU of the walking kernels.  More loads and stores in flight
// than these lower the rate HBM reaches for several streams read and written
// at once: gated_norm backward at 32768 x 16 x 512 from e4m3 (3 read, 3
// written) took 500 us with 256 threads a CU, 537 with 512 and 590 with 1024;
// the residual norm's at 32767 x 2560 from int8, whose rows meet at a
// barrier, 101 us with 960 and 132 with 512; gated_norm forward 38 us at
// 16384 x 8 x 256 with 2048, 40 with 512 or 1024.
constexpr int kBwdThreads = 1024, kGateFwdThreads = 2048, kGateBwdThreads = 256;
// Turns a workgroup of resid_norm forward takes (rows in sequence, so that
// weight, bias and scale are read once for them) where that leaves kFwdGrid
// workgroups: 216 us at 32768 x 4096 with 4, 222 with 2, 266 with 1, 227 with 8.
constexpr int kFwdChunk = 4, kFwdGrid = 2048;

// The backward's workgroup: rows side by side, threads, and workgroups (as
// many as kBwdThreads per CU make, no more than there are rows).
struct BwdShape {
  int rpb, threads, grid;
};
BwdShape bwd_shape(Elt elt, const RowShape& s, int64_t rows) {
  BwdShape b;
  const int most = s.lpr ? 256 : elt == kBF16 && s.vpt == 1 ? 1024 : 512;
  b.rpb = std::max(1, most / s.tpr);
  b.threads = b.rpb * s.tpr;
  b.grid = (int)std::min<int64_t>((rows + b.rpb - 1) / b.rpb, (int64_t)256 * std::max(1, kBwdThreads / b.threads));
  return b;
}

}  // namespace

int resid_norm_bwd_parts(int64_t rows, int d) {
  return std::max(bwd_shape(kBF16, row_shape(d), rows).grid, bwd_shape(kF32, row_shape(d), rows).grid);
}

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

int gated_norm_bwd_parts(int64_t rows, int heads, int d_v) { return gate_shape(rows, heads, d_v, kGateBwdThreads).P; }

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

hipError_t launch_resid_norm_fwd(const ResidNormArgs& a0, hipStream_t st) {
  ResidNormArgs a = a0;
  if (a.rows == 0) return hipSuccess;
  TraceScope ts("k_resid_norm_fwd", st);
  const RowShape s = row_shape(a.d);
  const int rpb = s.lpr ? 256 / s.lpr : 1;
  a.chunk = (int)std::max<int64_t>(1, std::min<int64_t>(kFwdChunk, a.rows / (rpb * kFwdGrid)));
  const int64_t per = (int64_t)a.chunk * rpb;
  const dim3 grid((unsigned)((a.rows + per - 1) / per)), block(rpb * s.tpr);
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
  const BwdShape bs = bwd_shape(a.elt, s, a.rows);
  const int P = bs.grid;
  a.tpr = s.tpr;
  a.sum_w = dweight != nullptr;
  a.sum_c = dbias != nullptr;
  if (a.rows) {
    TraceScope ts("k_resid_norm_bwd", st);
    const dim3 grid(P), block(bs.threads);
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
  const GateShape gs = gate_shape(a.rows, a.heads, a.d_v, kGateFwdThreads);
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
  const GateShape gs = gate_shape(a.rows, a.heads, a.d_v, kGateBwdThreads);
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
