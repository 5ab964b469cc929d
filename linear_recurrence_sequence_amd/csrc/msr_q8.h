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

typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

// Buffer access: a window of `bytes` bytes from a uniform address, and a
// lane's 32-bit byte offset in it.  Loads outside the window give zeros,
// stores outside are dropped (the hardware checks each lane), so that rows
// past the end, lanes past a row and tensors that are not given (a window of
// 0 bytes) need no branch -- a branch around a load would make the compiler
// wait for every load in flight where the paths meet, and the loads of the
// next rows are to stay in flight.
struct Win {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Win(const void* p, uint32_t bytes)
      : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, p ? (int)bytes : 0, 0x00027000)) {}
};
constexpr uint32_t kOutside = 0x7ffffff0u;     // beyond every window used
// Cache policies.  bf16 and 8-bit tensors: non-temporal (gated norm backward
// at 32768 x 16 x 512 from e4m3: 499 us, 514 with plain loads and stores;
// packing 32768 x 2560: 42 us, 56 plain).  float32: plain -- a lane's 8
// values are two 16-byte pieces, whose lines two instructions share (residual
// norm at 16384 x 4096: forward 206 us, 229 non-temporal; backward 307, 329).
constexpr int kStream = 2;

template <int POLICY = kStream>
__device__ __forceinline__ uint4 win_load16(const Win& w, uint32_t off) {
  const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(w.r, (int)off, 0, POLICY);
  return make_uint4(v[0], v[1], v[2], v[3]);
}
template <int POLICY = kStream>
__device__ __forceinline__ void win_store16(const Win& w, uint32_t off, uint4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(as_u32x4(v), w.r, (int)off, 0, POLICY);
}
__device__ __forceinline__ float win_load_f32(const Win& w, uint32_t off) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(w.r, (int)off, 0, 0));
}
__device__ __forceinline__ f32x4 win_load_f32x4(const Win& w, uint32_t off) {
  const uint4 u = win_load16<0>(w, off);
  return (f32x4){__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
}
__device__ __forceinline__ void win_store_f32(const Win& w, uint32_t off, float v) {
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), w.r, (int)off, 0, 0);
}
// 8 values at element offset `unit8` (a multiple of 8, or kOutside)
__device__ __forceinline__ void win_load8(Row8<bf16>& r, const Win& w, uint32_t unit8) {
  r.u = win_load16(w, unit8 == kOutside ? kOutside : 2 * unit8);
}
__device__ __forceinline__ void win_load8(Row8<float>& r, const Win& w, uint32_t unit8) {
  const uint32_t o = unit8 == kOutside ? kOutside : 4 * unit8;
  r.lo = win_load16<0>(w, o);
  r.hi = win_load16<0>(w, unit8 == kOutside ? kOutside : o + 16);
}
__device__ __forceinline__ void win_store8(const Win& w, uint32_t unit8, const Row8<bf16>& r) {
  win_store16(w, unit8 == kOutside ? kOutside : 2 * unit8, r.u);
}
__device__ __forceinline__ void win_store8(const Win& w, uint32_t unit8, const Row8<float>& r) {
  const uint32_t o = unit8 == kOutside ? kOutside : 4 * unit8;
  win_store16<0>(w, o, r.lo);
  win_store16<0>(w, unit8 == kOutside ? kOutside : o + 16, r.hi);
}

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
// 2^(b - 127) (b = 0: the subnormal 2^-127); NaN for b = 255.
__device__ __forceinline__ float q_pow2(uint32_t b) {
  const float s = __builtin_amdgcn_ldexpf(1.f, (int)b - 127);
  return b == 255u ? __builtin_nanf("") : s;
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

// The numbers that 8 codes stand for, without their scale.
template <int F>
__device__ __forceinline__ void q_decode8(float* v, uint2 q) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (F == kQE4M3) {
      const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
      const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
      v[4 * i] = a[0];
      v[4 * i + 1] = a[1];
      v[4 * i + 2] = b[0];
      v[4 * i + 3] = b[1];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] = (float)(int8_t)(w[i] >> (8 * e));
    }
  }
}

// The 8-bit form of this lane's 8 values (its quad holds a whole group):
// codes and the group's byte.  All four lanes of the quad have to be active.
template <int F>
__device__ __forceinline__ uint2 q_pack8(const float* v, int& b) {
  b = q_scale<F>(quad_amax(v));
  const uint2 c = q_encode8<F>(v, q_inv(b));
  return b == 255 ? make_uint2(0u, 0u) : c;    // the group reads back as NaN whatever its codes are
}

// A tensor's window held in T (F = kQNone: the values) or in 8 bits (codes
// and scale bytes): `rows` rows of d values from element `at` on.
template <class T, int F>
struct HeldWin {
  Win q, qs;
  __device__ __forceinline__ HeldWin(const void* x, const uint8_t* xs, int64_t at, uint32_t n)
      : q(x ? (const uint8_t*)x + at : nullptr, n), qs(xs ? xs + (at >> 5) : nullptr, n >> 5) {}
};
template <class T>
struct HeldWin<T, kQNone> {
  Win x;
  __device__ __forceinline__ HeldWin(const void* x_, const uint8_t*, int64_t at, uint32_t n)
      : x(x_ ? (const T*)x_ + at : nullptr, n * (uint32_t)sizeof(T)) {}
};
// Packs 8 values at element offset `off` of the window.
template <class T, int F>
__device__ __forceinline__ void q_store8(const float* v, const HeldWin<T, F>& w, uint32_t off) {
  int b;
  const uint2 c = q_pack8<F>(v, b);
  __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{c.x, c.y}, w.q.r, (int)off, 0, kStream);
  const uint32_t so = (threadIdx.x & 3) == 0 ? off >> 5 : kOutside;
  __builtin_amdgcn_raw_buffer_store_b8((uint8_t)b, w.qs.r, (int)so, 0, 0);
}

// 8 values of such a window, as loaded.  raw() gives them without their
// scale, times scale() they are the values: what multiplies them anyway
// takes it in.
template <class T, int F>
struct Held {
  uint2 q;
  uint32_t b;
  __device__ __forceinline__ void load(const HeldWin<T, F>& w, uint32_t off) {
    const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(w.q.r, (int)off, 0, kStream);
    q = make_uint2(v[0], v[1]);
    b = __builtin_amdgcn_raw_buffer_load_b8(w.qs.r, off == kOutside ? (int)kOutside : (int)(off >> 5), 0, 0);
  }
  __device__ __forceinline__ float scale() const { return q_pow2(b); }
  __device__ __forceinline__ void raw(float* v) const { q_decode8<F>(v, q); }
  __device__ __forceinline__ void values(float* v) const {
    raw(v);
    const float s = scale();
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= s;
  }
};
template <class T>
struct Held<T, kQNone> {
  Row8<T> r;
  __device__ __forceinline__ void load(const HeldWin<T, kQNone>& w, uint32_t off) { win_load8(r, w.x, off); }
  __device__ __forceinline__ float scale() const { return 1.f; }
  __device__ __forceinline__ void raw(float* v) const { unpack_row8(v, r); }
  __device__ __forceinline__ void values(float* v) const { unpack_row8(v, r); }
};

}  // namespace msr
