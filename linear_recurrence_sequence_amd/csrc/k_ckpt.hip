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

// A workgroup takes kFlat units of 8 values in a row, 256 at a time; four
// neighbouring lanes hold a group of 32 (the number of units is a multiple
// of 4, so a quad is on or off as one).
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
  for (int i = 0; i < kFlat / 256; ++i) win_load8(r[i], wx, 8 * (threadIdx.x + 256 * i));
#pragma unroll
  for (int i = 0; i < kFlat / 256; ++i) {
    float v[8];
    unpack_row8(v, r[i]);
    q_store8(v, wq, 8 * (threadIdx.x + 256 * i));
  }
}

// ((x - mean) rstd) weight + bias of 8 neighbouring values
struct Norm8 {
  const float* weight;
  const float* bias;
  __device__ __forceinline__ void apply(float* v, float mu, float r, int col) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = (v[e] - mu) * r;
      if (weight) v[e] *= weight[col + e];
      if (bias) v[e] += bias[col + e];
    }
  }
};

template <class T, int F, bool NORM>
__global__ __launch_bounds__(256) void k_ckpt_unpack(CkptArgs a, T* __restrict__ X) {
  const int cu = a.cols / 8;
  const int64_t unit0 = (int64_t)blockIdx.x * kFlat, at = unit0 * 8;
  const int n = (int)min((int64_t)kFlat, a.rows * cu - unit0);
  const HeldWin<T, F> wq(a.q, a.qs, at, 8u * (uint32_t)n);
  const Win wx(X + at, 8u * (uint32_t)n * (uint32_t)sizeof(T));
  Held<T, F> h[kFlat / 256];
#pragma unroll
  for (int i = 0; i < kFlat / 256; ++i) h[i].load(wq, 8 * (threadIdx.x + 256 * i));
#pragma unroll
  for (int i = 0; i < kFlat / 256; ++i) {
    const int u = threadIdx.x + 256 * i;
    float v[8];
    h[i].values(v);
    if constexpr (NORM) {
      if (u < n) {
        const int64_t row = (unit0 + u) / cu;
        const Norm8 nm{a.weight, a.bias};
        nm.apply(v, a.mean ? a.mean[row] : 0.f, a.rstd ? a.rstd[row] : 1.f, 8 * (int)(unit0 + u - row * cu));
      }
    }
    Row8<T> r;
    pack_row8(r, v);
    win_store8(wx, 8 * u, r);
  }
}

// tok() tokens (256 bytes of them) x 64 columns through LDS, transposed.  A lane reads 8 columns
// of two neighbouring tokens and writes each column's pair as one piece;
// then each column's tokens leave as one line.  A bf16 tile row of 136
// tokens is 4 banks (mod 64) longer than the last, so that a wave's 32-bit
// writes (8 columns apart, two tokens apart) spread over the banks.  The
// workgroups behind the last columns copy the rows of `pad`.
template <class T>
constexpr int tok() { return 256 / (int)sizeof(T); }

template <class T>
__device__ __forceinline__ void put_pair(T* p, float a, float b) {
  if constexpr (sizeof(T) == 2) *reinterpret_cast<uint32_t*>(p) = pack_bf16(a, b);
  else *reinterpret_cast<float2*>(p) = make_float2(a, b);
}

template <class T, int F, bool NORM>
__global__ __launch_bounds__(256) void k_ckpt_unpack_t(CkptArgs a, T* __restrict__ XT, int64_t ld, PadRows pad) {
  constexpr int kTok = tok<T>(), LD = kTok + 16 / (int)sizeof(T);
  __shared__ __attribute__((aligned(16))) T tile[64 * LD];
  if ((int)blockIdx.y >= a.cols / 64) {
    const int64_t n = pad.rows * (pad.cols / 8), out = pad.rows_out * (pad.cols / 8);
    const int64_t step = (int64_t)(gridDim.y - a.cols / 64) * gridDim.x * 256;
    for (int64_t u = ((int64_t)(blockIdx.y - a.cols / 64) * gridDim.x + blockIdx.x) * 256 + threadIdx.x; u < out;
         u += step) {
      Row8<T> r;
      load_row8(r, (const T*)pad.src + 8 * (u < n ? u : 0), u < n);
      store_row8((T*)pad.dst + 8 * u, r);
    }
    return;
  }
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  const int c0 = blockIdx.y * 64, tid = threadIdx.x;
  // the window of these rows (those past the end read as zeros)
  const uint32_t rows = (uint32_t)max((int64_t)0, min((int64_t)kTok, a.rows - t0));
  const HeldWin<T, F> wq(a.q, a.qs, t0 * a.cols, rows * (uint32_t)a.cols);
  const int c = tid & 7;
  Held<T, F> h[kTok / 64][2];
#pragma unroll
  for (int i = 0; i < kTok / 64; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) h[i][j].load(wq, (uint32_t)((2 * (tid >> 3) + 64 * i + j) * a.cols + c0 + 8 * c));
#pragma unroll
  for (int i = 0; i < kTok / 64; ++i) {
    const int r = 2 * (tid >> 3) + 64 * i;
    float v[2][8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      h[i][j].values(v[j]);
      if constexpr (NORM) {
        const int64_t row = t0 + r + j;
        if (row < a.rows) {
          const Norm8 n{a.weight, a.bias};
          n.apply(v[j], a.mean ? a.mean[row] : 0.f, a.rstd ? a.rstd[row] : 1.f, c0 + 8 * c);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) put_pair(tile + (8 * c + e) * LD + r, v[0][e], v[1][e]);
  }
  __syncthreads();
  constexpr int CPC = kTok / 8;                      // 8-token pieces of a column
#pragma unroll
  for (int i = 0; i < 64 * CPC / 256; ++i) {
    const int u = tid + 256 * i, col = u / CPC, t8 = u % CPC;
    Row8<T> r;
    load_row8(r, tile + col * LD + 8 * t8, true);
    if (t0 + 8 * t8 < ld) store_row8(XT + (int64_t)(c0 + col) * ld + t0 + 8 * t8, r);
  }
}

__global__ __launch_bounds__(256) void k_sum_parts(const float* __restrict__ part, int parts, float* __restrict__ out,
                                                   int64_t n, bool accumulate) {
  const int64_t i = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (i >= n) return;
  f32x4 s = accumulate ? *reinterpret_cast<const f32x4*>(out + i) : (f32x4){0.f, 0.f, 0.f, 0.f};
  for (int z = 0; z < parts; ++z) {
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
  const dim3 g = flat_grid(units), b(256);
#define MSR_UNPACK(T, F)                                                                               \
  if (has_norm(a)) hipLaunchKernelGGL((k_ckpt_unpack<T, F, true>), g, b, 0, st, a, (T*)X);             \
  else hipLaunchKernelGGL((k_ckpt_unpack<T, F, false>), g, b, 0, st, a, (T*)X);
  if (elt == kBF16) {
    if (fmt == kQE4M3) { MSR_UNPACK(bf16, kQE4M3) } else { MSR_UNPACK(bf16, kQI8) }
  } else {
    if (fmt == kQE4M3) { MSR_UNPACK(float, kQE4M3) } else { MSR_UNPACK(float, kQI8) }
  }
#undef MSR_UNPACK
  return hipGetLastError();
}

hipError_t launch_ckpt_unpack_t(Elt elt, int fmt, const CkptArgs& a, void* XT, int64_t ld, const PadRows& pad,
                                hipStream_t st) {
  if (a.cols == 0 || ld == 0) return hipSuccess;
  const int kTok = elt == kBF16 ? tok<bf16>() : tok<float>();
  const int64_t gx = (ld + kTok - 1) / kTok, padded = (pad.rows_out * (pad.cols / 8) + 255) / 256;
  const int64_t gy = a.cols / 64 + std::min<int64_t>((padded + gx - 1) / gx, 4096);
  if (a.cols % 64 || ld % 64 || pad.cols % 8 || gx > INT32_MAX || gy > 65535) return hipErrorInvalidValue;
  TraceScope ts("k_ckpt_unpack_t", st);
  const dim3 g((unsigned)gx, (unsigned)gy), b(256);
#define MSR_UNPACK(T, F)                                                                                    \
  if (has_norm(a)) hipLaunchKernelGGL((k_ckpt_unpack_t<T, F, true>), g, b, 0, st, a, (T*)XT, ld, pad);      \
  else hipLaunchKernelGGL((k_ckpt_unpack_t<T, F, false>), g, b, 0, st, a, (T*)XT, ld, pad);
  if (elt == kBF16) {
    if (fmt == kQE4M3) { MSR_UNPACK(bf16, kQE4M3) } else { MSR_UNPACK(bf16, kQI8) }
  } else {
    if (fmt == kQE4M3) { MSR_UNPACK(float, kQE4M3) } else { MSR_UNPACK(float, kQI8) }
  }
#undef MSR_UNPACK
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
