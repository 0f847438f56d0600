// gfx950 kernels that pack rows and read them back.  Both are bound by memory.
//
// A row's scale has to be known before its first element is rounded, so the threads of a row hold
// it in registers between the two, eight elements (16 bytes of 16-bit data) to a load: one wave
// takes a row of up to 2048 elements, four rows to a block, and a block of 256 to 1024 threads one
// of up to 32 elements a thread.  Rows beyond 32768 elements are read twice, the second time
// mostly from the L2 cache.  16384 x 11008 in bf16: packed in 86 us (6.3 TB/s; 110 with ordinary
// loads), by ZERO_SCALE_MAX in 105 to 112 (5.0), whose rounding takes more instructions, read back in
// 108 (5.0); a copy reaches 6.4.
#include "packed_rows.h"

namespace zs {
namespace packed {

// U loads a thread keep a row of up to 8 T U elements; U = 0: any length, read twice.
template <int DT, int RULE, bool TAIL, int T, int U>
__global__ void __launch_bounds__(kRowBlock<T>) write_kernel(MatArg x, PackArg p, int64_t rows, int64_t cols) {
  __shared__ uint32_t lds[T / kWave];
  const int t = threadIdx.x % T;
  const int64_t wide = padded(cols);
  for (int64_t r = (int64_t)blockIdx.x * kRowsOf<T> + threadIdx.x / T; r < rows; r += (int64_t)gridDim.x * kRowsOf<T>) {
    const char* src = (const char*)x.p + r * x.pitch * esize(DT);
    int8_t* dst = p.q + r * p.pitch;
    uint32_t m = 0;
    float v[8];
    if constexpr (U > 0) {
      Raw8<DT> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t c = 8 * (int64_t)(t + u * T);
        raw[u] = load8<DT, TAIL, true>(src, c, cols);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) m = max_raw<DT>(raw[u], m);
      const Rounding k = rounding<RULE>(row_max<T>(max_bits<DT>(m), lds));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t c = 8 * (int64_t)(t + u * T);
        decode8<DT>(raw[u], v);
        if (c < wide) *(u32x2*)(dst + c) = quantise8<RULE>(v, k);
      }
      if (t == 0) p.scale[r] = k.scale;
    } else {
      for (int64_t c = 8 * t; c < cols; c += 8 * T) m = max_raw<DT>(load8<DT, TAIL>(src, c, cols), m);
      const Rounding k = rounding<RULE>(row_max<T>(max_bits<DT>(m), lds));
      for (int64_t c = 8 * t; c < wide; c += 8 * T) {
        decode8<DT>(load8<DT, TAIL>(src, c, cols), v);
        *(u32x2*)(dst + c) = quantise8<RULE>(v, k);
      }
      if (t == 0) p.scale[r] = k.scale;
    }
  }
}

// Sixteen values a thread: tx threads (a power of two) side by side in a row.
template <int DT, bool TAIL>
__global__ void __launch_bounds__(256) read_kernel(PackArg p, MatArg out, int64_t rows, int64_t cols, int log_tx,
                                                   int64_t col_blocks) {
  const int64_t rb = blockIdx.x / col_blocks, cb = blockIdx.x % col_blocks;
  const int64_t c = ((cb << log_tx) + (threadIdx.x & ((1 << log_tx) - 1))) * 16;
  const int64_t r = (rb << (8 - log_tx)) + (threadIdx.x >> log_tx);
  if (r >= rows || c >= cols) return;
  const u32x4 q = *(const u32x4*)(p.q + r * p.pitch + c);
  const float s = p.scale[r];
  char* dst = (char*)out.p + r * out.pitch * esize(DT);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) values4(q[2 * h + i], s, x + 4 * i);
    if (c + 8 * h < cols) store8<DT, TAIL>(dst, c + 8 * h, cols, x);
  }
}

// Calls fn with TAIL, T and U of rows of `cols` elements: as few idle threads as these allow, and for
// rows that end inside a group of eight some of the choices only.
template <class F>
static void by_length(int64_t cols, F fn) {
  const int64_t groups = (cols + 15) / 16 * 2;
  using std::integral_constant;
  if (cols % 8 == 0) {
    const std::false_type tail;
    if (groups <= 64) fn(tail, integral_constant<int, 64>(), integral_constant<int, 1>());
    else if (groups <= 128) fn(tail, integral_constant<int, 64>(), integral_constant<int, 2>());
    else if (groups <= 256) fn(tail, integral_constant<int, 64>(), integral_constant<int, 4>());
    else if (groups <= 512) fn(tail, integral_constant<int, 256>(), integral_constant<int, 2>());
    else if (groups <= 768) fn(tail, integral_constant<int, 256>(), integral_constant<int, 3>());
    else if (groups <= 1024) fn(tail, integral_constant<int, 256>(), integral_constant<int, 4>());
    else if (groups <= 1536) fn(tail, integral_constant<int, 512>(), integral_constant<int, 3>());
    else if (groups <= 2048) fn(tail, integral_constant<int, 512>(), integral_constant<int, 4>());
    else if (groups <= 4096) fn(tail, integral_constant<int, 1024>(), integral_constant<int, 4>());
    else fn(tail, integral_constant<int, 1024>(), integral_constant<int, 0>());
  } else {
    const std::true_type tail;
    if (groups <= 64) fn(tail, integral_constant<int, 64>(), integral_constant<int, 1>());
    else if (groups <= 256) fn(tail, integral_constant<int, 64>(), integral_constant<int, 4>());
    else if (groups <= 1024) fn(tail, integral_constant<int, 256>(), integral_constant<int, 4>());
    else if (groups <= 4096) fn(tail, integral_constant<int, 1024>(), integral_constant<int, 4>());
    else fn(tail, integral_constant<int, 1024>(), integral_constant<int, 0>());
  }
}

}  // namespace packed

using namespace packed;

hipError_t launch_write(const MatArg& x, const PackArg& p, int64_t rows, int64_t cols, hipStream_t st) {
  by_dtype(x.dtype, [&](auto dt) {
    by_length(cols, [&](auto tail, auto t, auto u) {
      constexpr int D = decltype(dt)::value, T = decltype(t)::value, U = decltype(u)::value;
      constexpr bool E = decltype(tail)::value;
      const dim3 grid((uint32_t)row_grid<T>(rows));
      if (p.rule == ZERO_SCALE_POW2) write_kernel<D, ZERO_SCALE_POW2, E, T, U><<<grid, kRowBlock<T>, 0, st>>>(x, p, rows, cols);
      else write_kernel<D, ZERO_SCALE_MAX, E, T, U><<<grid, kRowBlock<T>, 0, st>>>(x, p, rows, cols);
    });
  });
  return hipGetLastError();
}

hipError_t launch_read(const PackArg& p, const MatArg& out, int64_t rows, int64_t cols, hipStream_t st) {
  const Tiles t = tiles_of(rows, cols);
  // a launch has fewer than 2^32 threads
  const int64_t most = (((int64_t)1 << 24) - 1) / t.col_blocks;
  for (int64_t b = 0; b < t.row_blocks; b += most) {
    const int64_t r0 = b * (256 >> t.log_tx), nb = t.row_blocks - b < most ? t.row_blocks - b : most;
    PackArg q = p;
    q.q += r0 * p.pitch;
    q.scale += r0;
    MatArg o = out;
    o.p = (char*)out.p + r0 * out.pitch * (out.dtype == ZERO_F32 ? 4 : 2);
    by_dtype(out.dtype, [&](auto dt) {
      const uint32_t grid = (uint32_t)(nb * t.col_blocks);
      if (cols % 8 == 0) read_kernel<decltype(dt)::value, false><<<grid, 256, 0, st>>>(q, o, rows - r0, cols, t.log_tx, t.col_blocks);
      else read_kernel<decltype(dt)::value, true><<<grid, 256, 0, st>>>(q, o, rows - r0, cols, t.log_tx, t.col_blocks);
    });
  }
  return hipGetLastError();
}

}  // namespace zs
