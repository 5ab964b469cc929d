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

// Units of 8 values, four neighbouring lanes to a group of 32; `units` is a
// multiple of 4 and so are the thread counts: a quad is on or off as one.
template <class T, int F>
__global__ __launch_bounds__(256) void k_ckpt_pack(const T* __restrict__ X, uint8_t* __restrict__ q,
                                                   uint8_t* __restrict__ qs, int64_t units) {
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    Row8<T> r;
    load_row8(r, X + 8 * u, true);
    float v[8];
    unpack_row8(v, r);
    q_store8<F>(v, q, qs, u);
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
  const int64_t units = a.rows * cu;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    Held<T, F> h;
    h.load(a.q, a.qs, u);
    float v[8];
    h.values(v);
    if constexpr (NORM) {
      const int64_t row = u / cu;
      const Norm8 n{a.weight, a.bias};
      n.apply(v, a.mean ? a.mean[row] : 0.f, a.rstd ? a.rstd[row] : 1.f, 8 * (int)(u - row * cu));
    }
    Row8<T> r;
    pack_row8(r, v);
    store_row8(X + 8 * u, r);
  }
}

// 64 tokens x 64 columns through LDS: 16 rows at a time are read (8 lanes a
// row), written to the tile transposed, and each column's 64 tokens stored
// as one line.
template <class T, int F, bool NORM>
__global__ __launch_bounds__(256) void k_ckpt_unpack_t(CkptArgs a, T* __restrict__ XT, int64_t ld) {
  constexpr int LD = 64 + 16 / (int)sizeof(T);       // tile row of 64 tokens, padded to keep 16-byte alignment
  __shared__ __attribute__((aligned(16))) T tile[64 * LD];
  const int64_t t0 = (int64_t)blockIdx.x * 64;
  const int c0 = blockIdx.y * 64, tid = threadIdx.x;
  const int cu = a.cols / 8;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (tid >> 3) + 32 * i, c = tid & 7;
    const int64_t row = t0 + r;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (row < a.rows) {
      Held<T, F> h;
      h.load(a.q, a.qs, row * cu + c0 / 8 + c);
      h.values(v);
      if constexpr (NORM) {
        const Norm8 n{a.weight, a.bias};
        n.apply(v, a.mean ? a.mean[row] : 0.f, a.rstd ? a.rstd[row] : 1.f, c0 + 8 * c);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[(8 * c + e) * LD + r] = (T)v[e];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int col = (tid >> 3) + 32 * i, t8 = tid & 7;
    Row8<T> r;
    load_row8(r, tile + col * LD + 8 * t8, true);
    store_row8(XT + (int64_t)(c0 + col) * ld + t0 + 8 * t8, r);
  }
}

template <class T>
__global__ __launch_bounds__(256) void k_pad_rows(const T* __restrict__ src, T* __restrict__ dst, int64_t units,
                                                  int64_t units_out) {
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= units_out) return;
  Row8<T> r;
  load_row8(r, src + 8 * (u < units ? u : 0), u < units);
  store_row8(dst + 8 * u, r);
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

// Workgroups of 256 threads over `units` units: enough to fill the card
// (2048 threads per CU), each walking with the grid's stride.
dim3 flat_grid(int64_t units) { return dim3((unsigned)std::min<int64_t>((units + 255) / 256, 256 * 8)); }

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

hipError_t launch_ckpt_unpack_t(Elt elt, int fmt, const CkptArgs& a, void* XT, int64_t ld, hipStream_t st) {
  if (a.cols == 0 || ld == 0) return hipSuccess;
  if (a.cols % 64 || ld % 64 || a.cols / 64 > 65535) return hipErrorInvalidValue;
  TraceScope ts("k_ckpt_unpack_t", st);
  const dim3 g((unsigned)(ld / 64), a.cols / 64), b(256);
#define MSR_UNPACK(T, F)                                                                               \
  if (has_norm(a)) hipLaunchKernelGGL((k_ckpt_unpack_t<T, F, true>), g, b, 0, st, a, (T*)XT, ld);      \
  else hipLaunchKernelGGL((k_ckpt_unpack_t<T, F, false>), g, b, 0, st, a, (T*)XT, ld);
  if (elt == kBF16) {
    if (fmt == kQE4M3) { MSR_UNPACK(bf16, kQE4M3) } else { MSR_UNPACK(bf16, kQI8) }
  } else {
    if (fmt == kQE4M3) { MSR_UNPACK(float, kQE4M3) } else { MSR_UNPACK(float, kQI8) }
  }
#undef MSR_UNPACK
  return hipGetLastError();
}

hipError_t launch_pad_rows(Elt elt, const void* src, void* dst, int64_t rows, int64_t rows_out, int cols,
                           hipStream_t st) {
  const int64_t units = rows * cols / 8, out = rows_out * cols / 8;
  if (out == 0) return hipSuccess;
  TraceScope ts("k_pad_rows", st);
  const dim3 g((unsigned)((out + 255) / 256)), b(256);
  if (elt == kBF16) hipLaunchKernelGGL((k_pad_rows<bf16>), g, b, 0, st, (const bf16*)src, (bf16*)dst, units, out);
  else hipLaunchKernelGGL((k_pad_rows<float>), g, b, 0, st, (const float*)src, (float*)dst, units, out);
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
