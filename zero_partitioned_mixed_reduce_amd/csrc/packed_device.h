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

// Two values rounded to nearest even into a 16-bit format; a NaN becomes the positive quiet one.
template <int DT>
__device__ __forceinline__ uint32_t enc2(float a, float b) {
  a = __builtin_isnan(a) ? __uint_as_float(0x7FC00000u) : a;
  b = __builtin_isnan(b) ? __uint_as_float(0x7FC00000u) : b;
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
// Elements [c, c + 8) of a row of `cols`; zeros past its end (and before its start, never read).
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const char* row, int64_t c, int64_t cols) {
  constexpr int S = esize(DT);
  Raw8<DT> r;
  const char* p = row + c * S;
  if (c + 8 <= cols) {
    r = load_any<Raw8<DT>>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 2 * S; ++i) r.v[i >> 2][i & 3] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) {
        if constexpr (DT == ZERO_F32) r.v[i >> 2][i & 3] = load_any<uint32_t>(p + 4 * i);
        else r.v[0][i >> 1] |= (uint32_t)load_any<uint16_t>(p + 2 * i) << (16 * (i & 1));
      }
  }
  return r;
}
// Stores x to elements [c, c + 8) of a row of `cols`, those within it.
template <int DT>
__device__ __forceinline__ void store8(char* row, int64_t c, int64_t cols, const float (&x)[8]) {
  constexpr int S = esize(DT);
  char* p = row + c * S;
  if constexpr (DT == ZERO_F32) {
    if (c + 8 <= cols) {
      store_any(p, f32x4{x[0], x[1], x[2], x[3]});
      store_any(p + 16, f32x4{x[4], x[5], x[6], x[7]});
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < cols) store_any(p + 4 * i, x[i]);
    }
  } else {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = enc2<DT>(x[2 * i], x[2 * i + 1]);
    if (c + 8 <= cols) {
      store_any(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < cols) store_any(p + 2 * i, (uint16_t)(v[i >> 1] >> (16 * (i & 1))));
    }
  }
}

// Value b (0 to 3) of four 8-bit integers.
__device__ __forceinline__ float q_of(uint32_t four, int b) { return (float)(int8_t)(four >> (8 * b)); }

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
// Nearest integer to x / scale, to even between two.  x * inv is exact for powers of two; for
// others it is within a step of the answer, and the sign of what is left over, an exact
// difference, says which: x and k * scale are multiples of half of scale's last place, and the
// difference is at most about scale / 2, which 24 bits hold.
template <int RULE>
__device__ __forceinline__ int quantise(float x, const Rounding& r) {
  if (r.none) return 0;
  float k = rintf(x * r.inv);
  if constexpr (RULE == ZERO_SCALE_MAX) {
    const float d = __builtin_fmaf(-k, r.scale, x);
    const float t = 2.0f * __builtin_fabsf(d);
    const bool odd = (int)k & 1;
    if (t > r.scale || (t == r.scale && odd)) k += __builtin_copysignf(1.0f, d);
    k = fminf(fmaxf(k, -127.0f), 127.0f);
  }
  return (int)k;
}
template <int RULE>
__device__ __forceinline__ u32x2 quantise8(const float (&x)[8], const Rounding& r) {
  u32x2 o = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i >> 2] |= ((uint32_t)quantise<RULE>(x[i], r) & 0xFFu) << (8 * (i & 3));
  return o;
}

}  // namespace packed
}  // namespace zs
