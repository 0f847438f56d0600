// Device helpers shared by the library's kernel sources: the 16-bit formats, block
// reductions and the device-scope stores of partial results.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zs_internal.h"

namespace zs {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// 16-bit formats

template <int DT>
__device__ __forceinline__ float dec16(uint32_t h) {
  if constexpr (DT == ZERO_BF16) {
    return __uint_as_float(h << 16);
  } else {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
  }
}

// Round to nearest even into the 16-bit format.  Every NaN, whatever its sign and
// payload, becomes the format's positive canonical quiet NaN (0x7FC0, 0x7E00): the
// sign and payload of an arithmetic NaN are not fixed by IEEE 754 and differ
// between machines, so keeping them would make the written bits machine-dependent.
template <int DT>
__device__ __forceinline__ uint32_t enc16(float x) {
  if constexpr (DT == ZERO_BF16) {
    uint32_t u = __float_as_uint(x);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FC0u;           // canonical quiet NaN
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;                   // round to nearest even
  } else {
    const uint32_t h = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x);  // v_cvt_f16_f32, RNE
    return __builtin_isnan(x) ? 0x7E00u : h;                         // canonical quiet NaN
  }
}

template <int DT>
__device__ __forceinline__ f32x4 dec16x4(u32x2 r) {
  f32x4 o;
  o.x = dec16<DT>(r.x & 0xFFFFu);
  o.y = dec16<DT>(r.x >> 16);
  o.z = dec16<DT>(r.y & 0xFFFFu);
  o.w = dec16<DT>(r.y >> 16);
  return o;
}

template <int DT>
__device__ __forceinline__ u32x2 enc16x4(f32x4 w) {
  u32x2 r;
  r.x = enc16<DT>(w.x) | (enc16<DT>(w.y) << 16);
  r.y = enc16<DT>(w.z) | (enc16<DT>(w.w) << 16);
  return r;
}

// ---------------------------------------------------------------------------
// deterministic block reductions (fixed butterfly, fixed cross-wave order)

__device__ __forceinline__ double block_sum(double x, double* lds) {
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, 64);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  __syncthreads();
  if (lane == 0) lds[wave] = x;
  __syncthreads();
  double r = lds[0];
  for (int w = 1; w < kBlock / 64; ++w) r += lds[w];
  return r;
}

__device__ __forceinline__ void store_part(uint64_t* p, double v) {
  __hip_atomic_store(p, (uint64_t)__double_as_longlong(v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double load_part(const uint64_t* p) {
  return __longlong_as_double((long long)__hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}
// Waits until this thread's device-scope stores have reached the device's coherence
// point, so that an arrival counted after it finds them there.
__device__ __forceinline__ void stores_complete() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

}  // namespace zs
