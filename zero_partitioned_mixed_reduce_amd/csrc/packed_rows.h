// Shared by the kernels that take whole rows of a matrix: a row's threads, and the launches' shapes.
#pragma once
#include <type_traits>

#include "packed_device.h"

namespace zs {
namespace packed {

constexpr int kWave = 64;

// Rows of a launch: blocks of T threads, a row each, or of four waves, a row each (T = 64).
template <int T>
constexpr int kRowBlock = T == kWave ? 4 * kWave : T;
template <int T>
constexpr int kRowsOf = kRowBlock<T> / T;

// Largest of the threads of a row.
template <int T>
__device__ __forceinline__ uint32_t row_max(uint32_t x, uint32_t* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t y = __shfl_xor(x, d);
    x = x > y ? x : y;
  }
  if constexpr (T > kWave) {
    __syncthreads();  // the values of the row before have been read
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = lds[0];
#pragma unroll
    for (int w = 1; w < T / kWave; ++w) x = x > lds[w] ? x : lds[w];
  }
  return x;
}
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t max8(const float (&x)[8], uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = magnitude(x[i]);
    m = m > a ? m : a;
  }
  return m;
}

// Elements of a q row that are stored: the columns and the zeros behind them.
__device__ __forceinline__ int64_t padded(int64_t cols) { return (cols + 15) & ~(int64_t)15; }

template <int DT>
__device__ __forceinline__ void decode8(const Raw8<DT>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = get<DT>(r, i);
}

// ---------------------------------------------------------------------------
// Launches

constexpr int64_t kMaxGrid = 1 << 20;  // blocks of a launch over rows, which loops beyond

template <int T>
static int64_t row_grid(int64_t rows) {
  const int64_t b = (rows + kRowsOf<T> - 1) / kRowsOf<T>;
  return b < kMaxGrid ? b : kMaxGrid;
}

template <class F>
static void by_dtype(int32_t dt, F fn) {
  if (dt == ZERO_F16) fn(std::integral_constant<int, ZERO_F16>());
  else if (dt == ZERO_BF16) fn(std::integral_constant<int, ZERO_BF16>());
  else fn(std::integral_constant<int, ZERO_F32>());
}

// Threads side by side in a row of groups of sixteen, and the blocks of the launch.
struct Tiles {
  int log_tx;
  int64_t col_blocks, row_blocks;
};
static Tiles tiles_of(int64_t rows, int64_t cols) {
  const int64_t groups = (cols + 15) / 16;
  Tiles t;
  t.log_tx = 0;
  while (t.log_tx < 8 && (int64_t)1 << t.log_tx < groups) ++t.log_tx;
  t.col_blocks = (groups + (1 << t.log_tx) - 1) >> t.log_tx;
  const int64_t ty = 256 >> t.log_tx;
  t.row_blocks = (rows + ty - 1) / ty;
  return t;
}

}  // namespace packed
}  // namespace zs
