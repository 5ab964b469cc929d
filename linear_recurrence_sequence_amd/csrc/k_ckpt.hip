// Activations held in 8 bits between the forward and the backward pass, for
// gfx950: packing, reading back, and the operands of a weight gradient from
// them.  Format and arithmetic: msr_q8.h.
//
// All of it streams: es + 33/32 bytes a value (es the element type's), bound
// by HBM.
#include <algorithm>

#include "msr_launch.h"
#include "msr_q8.h"

namespace msr {

namespace {

// Packing: a workgroup takes kFlat units of 8 values in a row, 256 at a time.
// One short piece a workgroup, in order: 32768 x 2560 bf16 packs in 40 us
// (6.3 TB/s) and reads back in 42; a grid of 2048 workgroups with strides
// took 46 each.
constexpr int kFlat = 512;

template <class T, int F>
__global__ __launch_bounds__(256) void k_ckpt_pack(const T* __restrict__ X, uint8_t* __restrict__ q,
                                                   uint8_t* __restrict__ qs, int64_t units) {
  const int64_t at = (int64_t)blockIdx.x * kFlat * 8;
  const int n = (int)min((int64_t)kFlat, units - (int64_t)blockIdx.x * kFlat);
  const Win wx(X + at, 8u * (uint32_t)n * (uint32_t)sizeof(T));
  const HeldWin<T, F> wq(q, qs, at, 8u * (uint32_t)n);
  Row8<T> r[kFlat / 256];
#pragma unroll
  for (int i = 0; i < kFlat / 256; ++i) win_load8(r[i], wx, unit_of<T>(2048 * i, threadIdx.x, 256));
#pragma unroll
  for (int i = 0; i < kFlat / 256; ++i) {
    float v[8];
    unpack_row8(v, r[i]);
    q_store8(v, wq, unit_of<T>(2048 * i, threadIdx.x, 256));
  }
}

// ((x - mean) rstd) weight + bias of 8 neighbouring columns, each absent
// vector's window empty (loads of several rows are in flight together).
struct Norm8 {
  float w[8], c[8];
  // the columns at element offset `col` of windows of weight and bias
  __device__ __forceinline__ void load(const CkptArgs& a, const Win& ww, const Win& wc, uint32_t col) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 x = win_load_f32x4(ww, 4 * col + 16 * h), y = win_load_f32x4(wc, 4 * col + 16 * h);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[4 * h + e] = a.weight ? x[e] : 1.f;
        c[4 * h + e] = y[e];
      }
    }
  }
  __device__ __forceinline__ void apply(float* v, float mu, float r) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (v[e] - mu) * r * w[e] + c[e];
  }
};

// Reading back.  A thread's unit is 16 bytes of T: a wave stores whole lines
// in one run (float32 as 8 values a thread, two stores of every other 16
// bytes, and through the caches, took 64 us where this takes 57: 16384 x 4096).
template <class T>
constexpr int kUnit = 16 / (int)sizeof(T);

template <class T, int F>
struct Codes {
  uint2 q;
  uint32_t b;
  // the unit at element offset `off`
  __device__ __forceinline__ void load(const HeldWin<T, F>& w, uint32_t off) {
    if constexpr (sizeof(T) == 2) {
      const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(w.q.r, (int)off, 0, kStream);
      q = make_uint2(v[0], v[1]);
    } else {
      q = make_uint2(__builtin_amdgcn_raw_buffer_load_b32(w.q.r, (int)off, 0, kStream), 0u);
    }
    b = __builtin_amdgcn_raw_buffer_load_b8(w.qs.r, (int)(off >> 5), 0, 0);
  }
  __device__ __forceinline__ void values(float* v) const {
    float t[8];
    q_decode8<F>(t, q);
    const float s = q_pow2(b);
#pragma unroll
    for (int e = 0; e < kUnit<T>; ++e) v[e] = t[e] * s;
  }
};
template <class T>
__device__ __forceinline__ void store_unit(const Win& w, uint32_t off, const float* v) {
  if constexpr (sizeof(T) == 2) {
    Row8<bf16> o;
    pack_row8(o, v);
    win_store16(w, 2 * off, o.u);
  } else {
    win_store16(w, 4 * off, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                       __float_as_uint(v[3])));
  }
}

template <class T, int F>
__global__ __launch_bounds__(256) void k_ckpt_unpack(const uint8_t* __restrict__ q, const uint8_t* __restrict__ qs,
                                                     T* __restrict__ X, int64_t count) {
  constexpr int V = kUnit<T>, kTurns = kFlat / 256;
  const int64_t at = (int64_t)blockIdx.x * kFlat * V;
  const uint32_t n = (uint32_t)min((int64_t)kFlat * V, count - at);
  const HeldWin<T, F> wq(q, qs, at, n);
  const Win wx(X + at, n * (uint32_t)sizeof(T));
  Codes<T, F> h[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) h[i].load(wq, V * (threadIdx.x + 256 * i));
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    float v[V];
    h[i].values(v);
    store_unit<T>(wx, V * (threadIdx.x + 256 * i), v);
  }
}

// Read back and normalised.  Weight and bias are 8 bytes for each byte of
// codes, so a thread keeps its unit's for kNormRows turns.  A turn is a piece
// of neighbouring units: `width` of a row (its units cut evenly into `pieces`
// of at most 256), or, pieces 1, as many whole rows as 256 threads hold.
// 16384 x 4096 with mean, rstd, weight and bias: bf16 38 us (62 with the
// vectors read for each unit), float32 63 (105); 4 turns 40, 16 turns 41.
constexpr int kNormRows = 8;

template <class T, int F>
__global__ __launch_bounds__(256) void k_ckpt_unpack_norm(CkptArgs a, T* __restrict__ X, int pieces, int width) {
  constexpr int V = kUnit<T>;
  const int cu = a.cols / V, tid = threadIdx.x;
  const int piece = pieces == 1 ? 0 : (int)(blockIdx.x % (unsigned)pieces);
  const int rpt = pieces == 1 ? (int)blockDim.x / cu : 1;          // rows a turn
  const int64_t row0 = (int64_t)(blockIdx.x / (unsigned)pieces) * (rpt * kNormRows);
  const int rib = pieces == 1 ? tid / cu : 0;                      // this thread's of them
  const int c0 = piece * width;                                    // first unit of the piece
  const uint32_t col = (uint32_t)(tid - rib * cu);
  const int wide = V * min(width, cu - c0);
  const int64_t x0 = V * (int64_t)c0;
  const Win ww(a.weight ? a.weight + x0 : nullptr, 4u * (uint32_t)wide);
  const Win wc(a.bias ? a.bias + x0 : nullptr, 4u * (uint32_t)wide);
  f32x4 w[V / 4], c[V / 4];
#pragma unroll
  for (int k = 0; k < V / 4; ++k) {
    w[k] = a.weight ? win_load_f32x4(ww, 4u * (V * col) + 16 * k) : (f32x4){1.f, 1.f, 1.f, 1.f};
    c[k] = win_load_f32x4(wc, 4u * (V * col) + 16 * k);
  }
  Codes<T, F> h[kNormRows];
  float mu[kNormRows], r[kNormRows];
  // elements of turn i (rows past the end: none)
  auto span = [&](int i) {
    return (uint32_t)wide * (uint32_t)max((int64_t)0, min((int64_t)rpt, a.rows - row0 - i * rpt));
  };
  const uint32_t left = (uint32_t)min((int64_t)(rpt * kNormRows), a.rows - row0);
  const Win wm(a.mean ? a.mean + row0 : nullptr, 4u * left), wr(a.rstd ? a.rstd + row0 : nullptr, 4u * left);
#pragma unroll
  for (int i = 0; i < kNormRows; ++i) {
    h[i].load(HeldWin<T, F>(a.q, a.qs, (row0 + i * rpt) * a.cols + x0, span(i)), V * (uint32_t)tid);
    mu[i] = win_load_f32(wm, 4u * (uint32_t)(i * rpt + rib));
    r[i] = win_load_f32(wr, 4u * (uint32_t)(i * rpt + rib));
  }
#pragma unroll
  for (int i = 0; i < kNormRows; ++i) {
    float v[V];
    h[i].values(v);
    const float ri = a.rstd ? r[i] : 1.f;
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = (v[e] - mu[i]) * ri * w[e / 4][e % 4] + c[e / 4][e % 4];
    const Win wx(X + (row0 + i * rpt) * a.cols + x0, span(i) * (uint32_t)sizeof(T));
    store_unit<T>(wx, V * (uint32_t)tid, v);
  }
}

// Operands of the weight gradient X^T dY in bf16.  bf16 tensors: X read back
// (normalised: rounded) and dY as it is, one term.  float32 tensors run on
// the bf16 matrix cores as well, with float32's accuracy: a float32 is the
// sum of three bf16 (its 24 significant bits cut in three), and products of
// bf16 are exact in the float32 accumulators.  A value held in 8 bits is one
// bf16, so three products -- X with each third of dY -- are all of it; a
// normalised X is three bf16 as well, and of the nine products the six down
// to 2^-16 are taken (the others are below 2^-26 of the value).  The bf16
// units are 16 times as fast as the float32 ones: 16384 x 2560 x 4096 took
// 1005 us against 4250 us on the latter.
// Each piece is written once, 64 tokens of it a slab; the product picks the
// pieces that meet (written once a term instead, X normalised: 2054 us for
// 1908, and 1434 MB of workspace for 780).

// x cut into three bf16 (as floats) that add up to it: each takes the leading
// 8 bits of what is left (toward zero: nothing overflows).  Infinities and
// NaN stay in the first.
__device__ __forceinline__ void cut3(float x, float (&p)[3]) {
  const uint32_t u = __float_as_uint(x);
  const bool finite = (u & 0x7f800000u) != 0x7f800000u;
  p[0] = finite ? __uint_as_float(u & 0xffff0000u) : x;
  const float r = finite ? x - p[0] : 0.f;
  p[1] = __uint_as_float(__float_as_uint(r) & 0xffff0000u);
  p[2] = r - p[1];
}

// kTok tokens x 64 columns through LDS, transposed, a piece at a time.  A
// lane reads 8 columns of two neighbouring tokens and writes each column's
// pair as one 32-bit word; then each column's tokens leave as 128-byte lines.
// A tile row of kTok + 8 tokens is 4 banks (mod 64) longer than the last, so
// that a wave's writes (8 columns apart, two tokens apart) spread over the
// banks.  The workgroups behind the last columns write dY's part.
constexpr int kTok = 128;
// Quads of 4 columns of dY a workgroup cuts, each lane a 16-byte load, all in
// flight: 16384 x 4096 takes 100 us, 6.7 TB/s (8 columns a lane, one load at a
// time down a strided grid: 150; the pieces stored non-temporally: 119).
constexpr int kDy = 1024;

template <class T, int F, bool NORM, int TERMS>
__global__ __launch_bounds__(256) void k_wgrad_operands(WgradOperands w) {
  constexpr int LD = kTok + 8, PIECES = wgrad_pieces(TERMS).x;
  __shared__ __attribute__((aligned(16))) bf16 tile[64 * LD];
  const CkptArgs& a = w.a;
  const int tid = threadIdx.x;
  if ((int)blockIdx.y >= a.cols / 64) {
    // kDy quads of 4 neighbouring columns a workgroup, of all tokens (float32)
    // or of the last slab's, those padded among them: read as zeros
    const int cu = w.dy_cols / 4;
    const int64_t slab0 = TERMS == 1 ? w.slabs - 1 : 0, first = 64 * slab0 * cu;
    const int64_t q0 = ((int64_t)(blockIdx.y - a.cols / 64) * gridDim.x + blockIdx.x) * kDy;
    const int64_t quads = 64 * (w.slabs - slab0) * cu;
    if (q0 >= quads) return;
    const int64_t left = max((int64_t)0, w.dy_rows * cu - first - q0);
    const Win wy((const T*)w.dY + 4 * (first + q0), (uint32_t)min(left, (int64_t)kDy) * 4u * (uint32_t)sizeof(T));
    const int64_t row0 = q0 / cu;
    const uint32_t u0 = (uint32_t)(q0 - row0 * cu), n = (uint32_t)min(quads - q0, (int64_t)kDy);
    uint4 r[kDy / 256];
#pragma unroll
    for (int i = 0; i < kDy / 256; ++i) {
      const uint32_t u = tid + 256 * i;
      if constexpr (TERMS == 1) {
        const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(wy.r, (int)(8 * u), 0, 0);
        r[i] = make_uint4(v[0], v[1], 0u, 0u);
      } else {
        r[i] = win_load16(wy, 16 * u);
      }
    }
#pragma unroll
    for (int i = 0; i < kDy / 256; ++i) {
      const uint32_t u = tid + 256 * i;
      if (u >= n) break;
      if constexpr (TERMS == 1) {
        *reinterpret_cast<uint2*>(w.dYt + 4 * (q0 + u)) = make_uint2(r[i].x, r[i].y);
      } else {
        const uint32_t dr = (u0 + u) / (uint32_t)cu, row = (uint32_t)row0 + dr;
        const uint32_t col = u0 + u - dr * (uint32_t)cu;
        uint16_t* const dst = w.dYt + ((int64_t)(row / 64 * (64 * 3) + row % 64) * cu + col) * 4;
        float p[4][3];
        cut3(__uint_as_float(r[i].x), p[0]);
        cut3(__uint_as_float(r[i].y), p[1]);
        cut3(__uint_as_float(r[i].z), p[2]);
        cut3(__uint_as_float(r[i].w), p[3]);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          const u32x2_t v = {pack_bf16(p[0][j], p[1][j]), pack_bf16(p[2][j], p[3][j])};
          *reinterpret_cast<u32x2_t*>(dst + (int64_t)(64 * j) * w.dy_cols) = v;
        }
      }
    }
    return;
  }
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  const int c0 = blockIdx.y * 64;
  // the window of these rows (those past the end read as zeros)
  const uint32_t rows = (uint32_t)max((int64_t)0, min((int64_t)kTok, a.rows - t0));
  // 8 neighbouring columns a thread, for either type
  const HeldWin<bf16, F> wq(a.q, a.qs, t0 * a.cols, rows * (uint32_t)a.cols);
  const int c = tid & 7;
  Held<bf16, F> h[kTok / 64][2];
#pragma unroll
  for (int i = 0; i < kTok / 64; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      h[i][j].load(wq, unit_of<bf16>((uint32_t)((2 * (tid >> 3) + 64 * i + j) * a.cols + c0), c, 8));
  float v[kTok / 64][2][8];
  if constexpr (NORM) {
    const Win ww(a.weight ? a.weight + c0 : nullptr, 256), wc(a.bias ? a.bias + c0 : nullptr, 256);
    const Win wm(a.mean ? a.mean + t0 : nullptr, 4 * rows), wr(a.rstd ? a.rstd + t0 : nullptr, 4 * rows);
    Norm8 nm;
    nm.load(a, ww, wc, 8 * c);
    float mu[kTok / 64][2], r[kTok / 64][2];
#pragma unroll
    for (int i = 0; i < kTok / 64; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t row = 2 * (tid >> 3) + 64 * i + j;
        mu[i][j] = win_load_f32(wm, 4 * row);
        r[i][j] = a.rstd ? win_load_f32(wr, 4 * row) : 1.f;
      }
#pragma unroll
    for (int i = 0; i < kTok / 64; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        h[i][j].values(v[i][j]);
        nm.apply(v[i][j], mu[i][j], r[i][j]);
        // tokens past the end stay zeros (the bias would not)
        const bool in = 2 * (tid >> 3) + 64 * i + j < (int)rows;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][j][e] = in ? v[i][j][e] : 0.f;
      }
  } else {
#pragma unroll
    for (int i = 0; i < kTok / 64; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) h[i][j].values(v[i][j]);
  }
#pragma unroll
  for (int piece = 0; piece < PIECES; ++piece) {
    if (piece) __syncthreads();
#pragma unroll
    for (int i = 0; i < kTok / 64; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float x = v[i][0][e], y = v[i][1][e];
        if constexpr (PIECES == 3) {
          float p[3], q[3];
          cut3(x, p);
          cut3(y, q);
          x = p[piece];
          y = q[piece];
        }
        *reinterpret_cast<uint32_t*>(tile + (8 * c + e) * LD + 2 * (tid >> 3) + 64 * i) = pack_bf16(x, y);
      }
    __syncthreads();
    constexpr int CPC = kTok / 8;                    // 8-token pieces of a column
#pragma unroll
    for (int i = 0; i < 64 * CPC / 256; ++i) {
      const int u = tid + 256 * i, col = u / CPC, t8 = u % CPC;
      Row8<bf16> r;
      load_row8(r, tile + col * LD + 8 * t8, true);
      const int64_t slab = t0 / 64 + t8 / 8;
      if (slab < w.slabs)
        store_row8((bf16*)w.XT + ((int64_t)(c0 + col) * w.slabs + slab) * (64 * PIECES) + 64 * piece + 8 * (t8 % 8), r);
    }
  }
}

__global__ __launch_bounds__(256) void k_sum_parts(const float* __restrict__ part, int parts, float* __restrict__ out,
                                                   int64_t n, bool accumulate) {
  const int64_t i = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (i >= n) return;
  f32x4 s = accumulate ? *reinterpret_cast<const f32x4*>(out + i) : (f32x4){0.f, 0.f, 0.f, 0.f};
  int z = 0;
  for (; z + 8 <= parts; z += 8) {             // eight loads in flight
    f32x4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const f32x4*>(part + (int64_t)(z + j) * n + i);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += v[j][e];
  }
  for (; z < parts; ++z) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(part + (int64_t)z * n + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += v[e];
  }
  *reinterpret_cast<f32x4*>(out + i) = s;
}

dim3 flat_grid(int64_t units) { return dim3((unsigned)((units + kFlat - 1) / kFlat)); }

}  // namespace

hipError_t launch_ckpt_pack(Elt elt, int fmt, int64_t rows, int cols, const void* X, uint8_t* q, uint8_t* qs,
                            hipStream_t st) {
  const int64_t units = rows * cols / 8;
  if (units == 0) return hipSuccess;
  TraceScope ts("k_ckpt_pack", st);
  const dim3 g = flat_grid(units), b(256);
  if (elt == kBF16) {
    if (fmt == kQE4M3) hipLaunchKernelGGL((k_ckpt_pack<bf16, kQE4M3>), g, b, 0, st, (const bf16*)X, q, qs, units);
    else hipLaunchKernelGGL((k_ckpt_pack<bf16, kQI8>), g, b, 0, st, (const bf16*)X, q, qs, units);
  } else {
    if (fmt == kQE4M3) hipLaunchKernelGGL((k_ckpt_pack<float, kQE4M3>), g, b, 0, st, (const float*)X, q, qs, units);
    else hipLaunchKernelGGL((k_ckpt_pack<float, kQI8>), g, b, 0, st, (const float*)X, q, qs, units);
  }
  return hipGetLastError();
}

static bool has_norm(const CkptArgs& a) { return a.mean || a.rstd || a.weight || a.bias; }

hipError_t launch_ckpt_unpack(Elt elt, int fmt, const CkptArgs& a, void* X, hipStream_t st) {
  const int64_t units = a.rows * a.cols / 8;
  if (units == 0) return hipSuccess;
  TraceScope ts("k_ckpt_unpack", st);
  const int V = elt == kBF16 ? kUnit<bf16> : kUnit<float>, cu = a.cols / V, quad = 32 / V;
  int pieces = (cu + 255) / 256;
  const int width = ((cu + pieces - 1) / pieces + quad - 1) / quad * quad;
  pieces = (cu + width - 1) / width;
  const int rpt = pieces == 1 ? 256 / cu : 1;
  const int64_t per = has_norm(a) ? rpt * kNormRows : kFlat, n = has_norm(a) ? a.rows : a.rows * cu;
  const int64_t blocks = (n + per - 1) / per * (has_norm(a) ? pieces : 1);
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  const dim3 g((unsigned)blocks), bn((unsigned)(rpt * width));
#define MSR_UNPACK(T, F)                                                                                         \
  if (has_norm(a)) hipLaunchKernelGGL((k_ckpt_unpack_norm<T, F>), g, bn, 0, st, a, (T*)X, pieces, width);        \
  else hipLaunchKernelGGL((k_ckpt_unpack<T, F>), g, dim3(256), 0, st, a.q, a.qs, (T*)X, a.rows * a.cols);
  if (elt == kBF16) {
    if (fmt == kQE4M3) { MSR_UNPACK(bf16, kQE4M3) } else { MSR_UNPACK(bf16, kQI8) }
  } else {
    if (fmt == kQE4M3) { MSR_UNPACK(float, kQE4M3) } else { MSR_UNPACK(float, kQI8) }
  }
#undef MSR_UNPACK
  return hipGetLastError();
}

hipError_t launch_wgrad_operands(Elt elt, int fmt, int terms, const WgradOperands& w, hipStream_t st) {
  const CkptArgs& a = w.a;
  if (a.cols == 0 || w.slabs == 0) return hipSuccess;
  const int64_t tokens = 64 * w.slabs, gx = (tokens + kTok - 1) / kTok;
  const int64_t dy_wgs = w.dYt ? ((terms > 1 ? tokens : 64) * (w.dy_cols / 4) + kDy - 1) / kDy : 0;
  const int64_t gy = a.cols / 64 + (dy_wgs + gx - 1) / gx;
  if (a.cols % 64 || w.dy_cols % 8 || gx > INT32_MAX || gy > 65535) return hipErrorInvalidValue;
  TraceScope ts("k_wgrad_operands", st);
  const dim3 g((unsigned)gx, (unsigned)gy), b(256);
#define MSR_OPERANDS(T, N, TERMS)                                                                          \
  if (fmt == kQE4M3) hipLaunchKernelGGL((k_wgrad_operands<T, kQE4M3, N, TERMS>), g, b, 0, st, w);          \
  else hipLaunchKernelGGL((k_wgrad_operands<T, kQI8, N, TERMS>), g, b, 0, st, w);
  if (elt == kBF16 && terms == 1) {
    if (has_norm(a)) { MSR_OPERANDS(bf16, true, 1) } else { MSR_OPERANDS(bf16, false, 1) }
  } else if (elt == kF32 && terms == 3 && !has_norm(a)) {
    MSR_OPERANDS(float, false, 3)
  } else if (elt == kF32 && terms == 6) {
    MSR_OPERANDS(float, true, 6)
  } else {
    return hipErrorInvalidValue;
  }
#undef MSR_OPERANDS
  return hipGetLastError();
}

hipError_t launch_sum_parts(const float* part, int parts, float* out, int64_t n, bool accumulate, hipStream_t st) {
  if (n == 0) return hipSuccess;
  TraceScope ts("k_sum_parts", st);
  hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, st, part, parts, out, n,
                     accumulate);
  return hipGetLastError();
}

}  // namespace msr
