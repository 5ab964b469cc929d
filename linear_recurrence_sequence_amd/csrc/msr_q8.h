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
// Cache policy of the tensors that are read or written once: non-temporal
// (gated norm backward at 32768 x 16 x 512 from e4m3: 499 us, 514 with plain
// loads and stores; packing 32768 x 2560 bf16: 42 us, 56 plain).
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
// A lane's 8 values are two pieces of 4 neighbours, at element offsets lo and
// hi (multiples of 4; lo = kOutside: neither).  bf16: next to each other, one
// 16-byte access.  float32: hi a run of lanes further, so that neighbouring
// lanes' pieces are neighbours in memory and each access covers whole lines
// (16384 x 4096: residual norm forward 190 us, backward 135, gated norm
// backward 228; with 8 neighbours a lane each access touched every other 16
// bytes: 204, 150 and 252, and more non-temporal).
// A group of 32 of the 8-bit form is 4 lanes' units or 8 lanes' pieces.
struct Unit {
  uint32_t lo, hi;
  __device__ __forceinline__ bool on() const { return lo != kOutside; }
};
constexpr Unit kNoUnit = {kOutside, kOutside};
// Lane l's unit of L lanes that hold 8 L neighbouring values from `base` on.
template <class T>
__device__ __forceinline__ Unit unit_of(uint32_t base, int l, int L) {
  const uint32_t lo = base + (sizeof(T) == 2 ? 8u : 4u) * (uint32_t)l;
  return {lo, lo + (sizeof(T) == 2 ? 4u : 4u * (uint32_t)L)};
}
__device__ __forceinline__ void win_load8(Row8<bf16>& r, const Win& w, Unit u) {
  r.u = win_load16(w, u.on() ? 2 * u.lo : kOutside);
}
__device__ __forceinline__ void win_load8(Row8<float>& r, const Win& w, Unit u) {
  r.lo = win_load16(w, u.on() ? 4 * u.lo : kOutside);
  r.hi = win_load16(w, u.on() ? 4 * u.hi : kOutside);
}
__device__ __forceinline__ void win_store8(const Win& w, Unit u, const Row8<bf16>& r) {
  win_store16(w, u.on() ? 2 * u.lo : kOutside, r.u);
}
__device__ __forceinline__ void win_store8(const Win& w, Unit u, const Row8<float>& r) {
  win_store16(w, u.on() ? 4 * u.lo : kOutside, r.lo);
  win_store16(w, u.on() ? 4 * u.hi : kOutside, r.hi);
}
// A float32 vector's 8 values (def where there is no vector or no unit), and
// back.
__device__ __forceinline__ void load_vec8(float* v, const float* p, Unit u, float def) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = def;
  if (p && u.on()) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p + u.lo), b = *reinterpret_cast<const f32x4*>(p + u.hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
  }
}
__device__ __forceinline__ void store_vec8(float* p, Unit u, const float* v) {
  *reinterpret_cast<f32x4*>(p + u.lo) = (f32x4){v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + u.hi) = (f32x4){v[4], v[5], v[6], v[7]};
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

// Largest magnitude of a group, as bits: of N values of each of 32 / N lanes
// (all of them active).  Magnitudes compare as integers, infinities and NaN
// above every number.
template <int N>
__device__ __forceinline__ uint32_t group_amax(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
  if constexpr (N == 4) m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));
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

// 4 values of a group with byte b as codes.  A group with an infinity or a
// NaN reads back as NaN whatever its codes are: zeros.
template <int F>
__device__ __forceinline__ uint32_t q_encode4(const float* v, int b) {
  const float inv = q_inv(b);
  uint32_t r;
  if constexpr (F == kQE4M3) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
    r = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, lo, true);
  } else {
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = (uint32_t)(int)rintf(v[e] * inv) & 0xffu;
    r = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
  }
  return b == 255 ? 0u : r;
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
// Packs this lane's 8 values; the lanes of a group are active together.
template <class T, int F>
__device__ __forceinline__ void q_store8(const float* v, const HeldWin<T, F>& w, Unit u) {
  auto scale = [&](int b, uint32_t off, int lanes) {
    const uint32_t so = u.on() && (threadIdx.x & (lanes - 1)) == 0 ? off >> 5 : kOutside;
    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)b, w.qs.r, (int)so, 0, 0);
  };
  if constexpr (sizeof(T) == 2) {
    const int b = q_scale<F>(group_amax<8>(v));
    const u32x2_t c = {q_encode4<F>(v, b), q_encode4<F>(v + 4, b)};
    __builtin_amdgcn_raw_buffer_store_b64(c, w.q.r, (int)u.lo, 0, kStream);
    scale(b, u.lo, 4);
  } else {
    const int b0 = q_scale<F>(group_amax<4>(v)), b1 = q_scale<F>(group_amax<4>(v + 4));
    __builtin_amdgcn_raw_buffer_store_b32(q_encode4<F>(v, b0), w.q.r, (int)u.lo, 0, kStream);
    __builtin_amdgcn_raw_buffer_store_b32(q_encode4<F>(v + 4, b1), w.q.r, (int)u.hi, 0, kStream);
    scale(b0, u.lo, 8);
    scale(b1, u.hi, 8);
  }
}

// 8 values of such a window, as loaded.  raw() times scale() are the values:
// what multiplies them anyway takes the scale in (float32's pieces have one
// each, raw() has taken them in).
template <class T, int F>
struct Held {
  uint2 q;
  uint32_t b, b1;
  __device__ __forceinline__ void load(const HeldWin<T, F>& w, Unit u) {
    auto scale = [&](uint32_t off) {
      return __builtin_amdgcn_raw_buffer_load_b8(w.qs.r, u.on() ? (int)(off >> 5) : (int)kOutside, 0, 0);
    };
    if constexpr (sizeof(T) == 2) {
      const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(w.q.r, (int)u.lo, 0, kStream);
      q = make_uint2(v[0], v[1]);
    } else {
      q.x = __builtin_amdgcn_raw_buffer_load_b32(w.q.r, (int)u.lo, 0, kStream);
      q.y = __builtin_amdgcn_raw_buffer_load_b32(w.q.r, (int)u.hi, 0, kStream);
      b1 = scale(u.hi);
    }
    b = scale(u.lo);
  }
  __device__ __forceinline__ float scale() const { return sizeof(T) == 2 ? q_pow2(b) : 1.f; }
  __device__ __forceinline__ void raw(float* v) const {
    q_decode8<F>(v, q);
    if constexpr (sizeof(T) == 4) {
      const float s = q_pow2(b), s1 = q_pow2(b1);
#pragma unroll
      for (int e = 0; e < 4; ++e) { v[e] *= s; v[4 + e] *= s1; }
    }
  }
  __device__ __forceinline__ void values(float* v) const {
    raw(v);
    if constexpr (sizeof(T) == 2) {
      const float s = scale();
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= s;
    }
  }
};
template <class T>
struct Held<T, kQNone> {
  Row8<T> r;
  __device__ __forceinline__ void load(const HeldWin<T, kQNone>& w, Unit u) { win_load8(r, w.x, u); }
  __device__ __forceinline__ float scale() const { return 1.f; }
  __device__ __forceinline__ void raw(float* v) const { unpack_row8(v, r); }
  __device__ __forceinline__ void values(float* v) const { unpack_row8(v, r); }
};

}  // namespace msr
