// Activations held in 8 bits, and the reductions of the row kernels that
// read and write them (internal; the format is described in include/msr.h).
//
// 32 neighbouring values of a row share a power of two 2^e; each is stored
// as q = x 2^-e rounded to nearest even, in e4m3 (|q| <= 448) or int8 (|q| <=
// 127), and e + 127 in one byte.  e is the smallest exponent that holds the
// group's largest magnitude, so nothing saturates.  A power of two: scaling
// is exact, q 2^e has 4 or 7 significant bits and is therefore exact in bf16
// too, and every value is a function of the group's inputs alone (the same
// bits from whichever kernel packs them).
#pragma once
#include "msr_device.h"

namespace msr {

enum : int { kQNone = 0, kQE4M3 = 1, kQI8 = 2 };
constexpr int kQGroup = 32;

// Sum over aligned groups of L lanes (8, 16, 32 or 64), returned to all of
// them: lane exchanges within a row of 16, then the gfx950 swaps of odd and
// even rows and of the wave's halves.  The lanes of a group have to be
// active together; other groups need not be.
template <int L>
__device__ __forceinline__ float group_sum(float x) {
  x = dpp_add<0xB1>(x);                        // quad_perm [1, 0, 3, 2]
  x = dpp_add<0x4E>(x);                        // quad_perm [2, 3, 0, 1]
  if constexpr (L >= 8) x = dpp_add<0x141>(x);   // row_half_mirror
  if constexpr (L >= 16) x = dpp_add<0x140>(x);  // row_mirror
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return x;
}

// Largest magnitude of the 4 lanes x 8 values of a group, as bits: magnitudes
// compare as integers, infinities and NaN above every number.
__device__ __forceinline__ uint32_t quad_amax(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
  return m;
}

// e + 127 for a largest magnitude 1.M 2^(E - 127): 448 = 1.75 * 2^8 and 127 =
// 1.984375 * 2^6, so e = E - 135 or E - 133, and one more when 1.M is above
// that significand.  At least 0; 255 for a group with an infinity or a NaN.
template <int F>
__device__ __forceinline__ int q_scale(uint32_t m) {
  const int E = (int)(m >> 23), M = (int)(m & 0x7fffffu);
  const int b = F == kQE4M3 ? E - 8 + (M > 0x600000) : E - 6 + (M > 0x7e0000);
  return m >= 0x7f800000u ? 255 : max(b, 0);
}
// 2^(127 - b) for b <= 248
__device__ __forceinline__ float q_inv(int b) { return __uint_as_float((uint32_t)(254 - b) << 23); }
// 2^(b - 127); NaN for b = 255.  b = 0 is the subnormal 2^-127.
__device__ __forceinline__ float q_pow2(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7fc00000u) : b == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

// 8 values times `inv`, rounded to codes.
template <int F>
__device__ __forceinline__ uint2 q_encode8(const float* v, float inv) {
  uint2 r;
  if constexpr (F == kQE4M3) {
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * inv, v[5] * inv, 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * inv, v[7] * inv, hi, true);
    r.x = (uint32_t)lo;
    r.y = (uint32_t)hi;
  } else {
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = (uint32_t)(int)rintf(v[e] * inv) & 0xffu;
    r.x = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
    r.y = b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24;
  }
  return r;
}

// 8 codes times `s`.
template <int F>
__device__ __forceinline__ void q_decode8(float* v, uint2 q, float s) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (F == kQE4M3) {
      const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
      const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
      v[4 * i] = a[0] * s;
      v[4 * i + 1] = a[1] * s;
      v[4 * i + 2] = b[0] * s;
      v[4 * i + 3] = b[1] * s;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] = (float)((int)(w[i] << (24 - 8 * e)) >> 24) * s;
    }
  }
}

// Packs this lane's 8 values (its quad holds a whole group) to q8[unit] and
// the group's byte to qs[unit / 4]; unit = flat index / 8.  All four lanes of
// the quad have to be active.
template <int F>
__device__ __forceinline__ void q_store8(const float* v, uint8_t* q, uint8_t* qs, int64_t unit) {
  const int b = q_scale<F>(quad_amax(v));
  uint2 c = q_encode8<F>(v, q_inv(b));
  if (b == 255) c = make_uint2(0u, 0u);        // the group reads back as NaN whatever its codes are
  reinterpret_cast<uint2*>(q)[unit] = c;
  if ((threadIdx.x & 3) == 0) qs[unit >> 2] = (uint8_t)b;
}

// 8 values of an activation held in T (F = kQNone) or in 8 bits, as loaded;
// values() converts when they are used.
template <class T, int F>
struct Held {
  uint2 q;
  uint32_t b;
  __device__ __forceinline__ void load(const void* x, const uint8_t* xs, int64_t unit) {
    q = reinterpret_cast<const uint2*>(x)[unit];
    b = xs[unit >> 2];
  }
  __device__ __forceinline__ void values(float* v) const { q_decode8<F>(v, q, q_pow2(b)); }
};
template <class T>
struct Held<T, kQNone> {
  Row8<T> r;
  __device__ __forceinline__ void load(const void* x, const uint8_t*, int64_t unit) {
    load_row8(r, reinterpret_cast<const T*>(x) + 8 * unit, true);
  }
  __device__ __forceinline__ void values(float* v) const { unpack_row8(v, r); }
};

}  // namespace msr
