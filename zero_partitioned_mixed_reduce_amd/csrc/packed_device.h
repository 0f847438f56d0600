// Device helpers of the packed-row kernels: the floating formats, eight elements at a time, and
// the packed format's rounding.
#pragma once
#include <hip/hip_runtime.h>

#include "packed.h"

namespace zs {
namespace packed {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int esize(int dt) { return dt == ZERO_F32 ? 4 : 2; }

template <class V>
__device__ __forceinline__ V load_any(const void* p) {  // at any alignment
  V v;
  __builtin_memcpy(&v, p, sizeof(V));
  return v;
}
template <class V>
__device__ __forceinline__ void store_any(void* p, V v) {
  __builtin_memcpy(p, &v, sizeof(V));
}

// Makes every NaN among x the positive quiet one, as which a 16-bit destination gets it; one comparison
// sees two values.
template <int N>
__device__ __forceinline__ void one_nan(float (&x)[N]) {
  static_assert(N % 2 == 0, "pairs");
  bool any = false;
#pragma unroll
  for (int i = 0; i < N; i += 2) any |= __builtin_isunordered(x[i], x[i + 1]);
  if (__builtin_expect(any, 0)) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __builtin_isnan(x[i]) ? __uint_as_float(0x7FC00000u) : x[i];
  }
}
// Two values rounded to nearest even into a 16-bit format.
template <int DT>
__device__ __forceinline__ uint32_t enc2(float a, float b) {
  if constexpr (DT == ZERO_BF16) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  } else {
    const f16x2 v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
}
template <int DT>
__device__ __forceinline__ float dec_lo(uint32_t x) {
  if constexpr (DT == ZERO_BF16) return __uint_as_float(x << 16);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)x);
}
template <int DT>
__device__ __forceinline__ float dec_hi(uint32_t x) {
  if constexpr (DT == ZERO_BF16) return __uint_as_float(x & 0xFFFF0000u);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(x >> 16));
}

// Eight consecutive elements as they lie in memory.
template <int DT>
struct Raw8 {
  u32x4 v[esize(DT) / 2];
};
template <int DT>
__device__ __forceinline__ float get(const Raw8<DT>& r, int i) {  // i known at compile time
  if constexpr (DT == ZERO_F32) return __uint_as_float(r.v[i >> 2][i & 3]);
  else return (i & 1) ? dec_hi<DT>(r.v[0][i >> 1]) : dec_lo<DT>(r.v[0][i >> 1]);
}
// Largest magnitude of the elements, and of m: for a 16-bit type two at a time, as bit patterns side by
// side, which are ordered as the magnitudes are.
template <int DT>
__device__ __forceinline__ uint32_t max_raw(const Raw8<DT>& r, uint32_t m) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 2 * esize(DT); ++i) {
    if constexpr (DT == ZERO_F32) {
      const uint32_t a = r.v[i >> 2][i & 3] & 0x7FFFFFFFu;
      m = m > a ? m : a;
    } else {
      const u16x2 a = __builtin_bit_cast(u16x2, r.v[0][i] & 0x7FFF7FFFu);
      m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m), a));
    }
  }
  return m;
}
// ... as the bits of a float.
template <int DT>
__device__ __forceinline__ uint32_t max_bits(uint32_t m) {
  if constexpr (DT == ZERO_F32) return m;
  const uint32_t a = m & 0xFFFFu, b = m >> 16;
  return __float_as_uint(dec_lo<DT>(a > b ? a : b));
}

// Elements [c, c + 8) of a row of `cols`; zeros past its end.  TAIL false: cols is a multiple of 8, and so
// there are all of them or none (the code for some of them costs the others registers).  ONCE: read past
// the caches' order of use, by who reads them only once.
template <int DT, bool TAIL = true, bool ONCE = false>
__device__ __forceinline__ Raw8<DT> load8(const char* row, int64_t c, int64_t cols) {
  constexpr int S = esize(DT);
  Raw8<DT> r;
  const char* p = row + c * S;
  if (TAIL ? c + 8 <= cols : c < cols) {
    if constexpr (ONCE) {
      typedef uint32_t any4 __attribute__((ext_vector_type(4), aligned(2)));
#pragma unroll
      for (int i = 0; i < S / 2; ++i) r.v[i] = __builtin_nontemporal_load((const any4*)(p + 16 * i));
    } else {
      r = load_any<Raw8<DT>>(p);
    }
    return r;
  }
#pragma unroll
  for (int i = 0; i < 2 * S; ++i) r.v[i >> 2][i & 3] = 0;
  if constexpr (TAIL) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) {
        if constexpr (DT == ZERO_F32) r.v[i >> 2][i & 3] = load_any<uint32_t>(p + 4 * i);
        else r.v[0][i >> 1] |= (uint32_t)load_any<uint16_t>(p + 2 * i) << (16 * (i & 1));
      }
  }
  return r;
}
// Stores x to elements [c, c + 8) of a row of `cols`, those within it (TAIL false: all are).
template <int DT, bool TAIL = true>
__device__ __forceinline__ void store8(char* row, int64_t c, int64_t cols, float (&x)[8]) {
  constexpr int S = esize(DT);
  char* p = row + c * S;
  if constexpr (DT == ZERO_F32) {
    if (!TAIL || c + 8 <= cols) {
      store_any(p, f32x4{x[0], x[1], x[2], x[3]});
      store_any(p + 16, f32x4{x[4], x[5], x[6], x[7]});
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < cols) store_any(p + 4 * i, x[i]);
    }
  } else {
    one_nan(x);
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = enc2<DT>(x[2 * i], x[2 * i + 1]);
    if (!TAIL || c + 8 <= cols) {
      store_any(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < cols) store_any(p + 2 * i, (uint16_t)(v[i >> 1] >> (16 * (i & 1))));
    }
  }
}

// Byte B of four 8-bit integers, signed, as a float in one instruction (the compiler takes two).
template <int B>
__device__ __forceinline__ float q_of(uint32_t four) {
  float x = 0.0f;
#ifdef __HIP_DEVICE_COMPILE__
  if constexpr (B == 0) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(x) : "v"(four));
  if constexpr (B == 1) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(x) : "v"(four));
  if constexpr (B == 2) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(x) : "v"(four));
  if constexpr (B == 3) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(x) : "v"(four));
#endif
  return x;
}
__device__ __forceinline__ void values4(uint32_t four, float scale, float* x) {
  x[0] = q_of<0>(four) * scale;
  x[1] = q_of<1>(four) * scale;
  x[2] = q_of<2>(four) * scale;
  x[3] = q_of<3>(four) * scale;
}

// How a row is rounded, from the bits of its largest magnitude.
struct Rounding {
  float scale, inv;  // inv: 1 / scale, exact for a power of two
  bool none;         // a row of zeros, or with an infinity or a NaN: q = 0
};
template <int RULE>
__device__ __forceinline__ Rounding rounding(uint32_t top) {
  Rounding r;
  r.none = top == 0 || top >= 0x7F800000u;
  if constexpr (RULE == ZERO_SCALE_POW2) {
    // top = f 2^e, 1 <= f < 2: top <= 127 s means s = 2^(e - 6) where f <= 127/64, else 2^(e - 5)
    int e = (int)(top >> 23) - 133 + ((top & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
    e = e < -126 ? -126 : e;
    r.scale = __uint_as_float((uint32_t)(e + 127) << 23);
    r.inv = __uint_as_float((uint32_t)(127 - e) << 23);
  } else {
    r.scale = fmaxf(__uint_as_float(top) / 127.0f, 0x1p-126f);
    r.inv = 1.0f / r.scale;
  }
  if (r.none) r.scale = top == 0 ? 0.0f : __uint_as_float(0x7FC00000u);
  return r;
}
// The nearest integer to x / scale, to even between two, in the last byte.  x * inv is exact for powers
// of two, and added to 1.5 * 2^23 is rounded once, to a whole number whose two's complement the
// result's low bits are.  For others it is within a step of the answer, and the sign of what is
// left over, an exact difference, says which: x and k * scale are multiples of half of scale's last
// place, and the difference is at most about scale / 2, which 24 bits hold.
template <int RULE>
__device__ __forceinline__ uint32_t quantise(float x, const Rounding& r) {
  constexpr float kWhole = 12582912.0f;
  if constexpr (RULE == ZERO_SCALE_POW2) return __float_as_uint(__builtin_fmaf(x, r.inv, kWhole));
  float k = rintf(x * r.inv);
  const float d = __builtin_fmaf(-k, r.scale, x);
  const float t = 2.0f * __builtin_fabsf(d);
  const bool odd = (int)k & 1;
  if (t > r.scale || (t == r.scale && odd)) k += __builtin_copysignf(1.0f, d);
  return __float_as_uint(fminf(fmaxf(k, -127.0f), 127.0f) + kWhole);
}
template <int RULE>
__device__ __forceinline__ u32x2 quantise8(const float (&x)[8], const Rounding& r) {
  u32x2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = quantise<RULE>(x[4 * h + i], r);
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0c);
    o[h] = r.none ? 0u : lo | hi;
  }
  return o;
}

}  // namespace packed
}  // namespace zs
