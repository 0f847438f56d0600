// gfx950 kernels of the packed rows that go over each element once: packing, reading back, and the
// activation functions.  All are bound by memory.
//
// A row's scale has to be known before its first element is rounded, so the threads of a row hold
// it in registers between the two, eight elements (16 bytes of 16-bit data) to a load: one wave
// takes a row of up to 2048 elements, four rows to a block, and a block of 256 to 1024 threads one
// of up to 32 elements a thread.  Rows beyond 32768 elements are read twice, the second time
// mostly from the L2 cache.
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

// U loads a thread keep a row of up to 8 T U elements; U = 0: any length, read twice.
template <int DT, int RULE, int T, int U>
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
        raw[u] = load8<DT>(src, c, cols);
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
      for (int64_t c = 8 * t; c < cols; c += 8 * T) m = max_raw<DT>(load8<DT>(src, c, cols), m);
      const Rounding k = rounding<RULE>(row_max<T>(max_bits<DT>(m), lds));
      for (int64_t c = 8 * t; c < wide; c += 8 * T) {
        decode8<DT>(load8<DT>(src, c, cols), v);
        *(u32x2*)(dst + c) = quantise8<RULE>(v, k);
      }
      if (t == 0) p.scale[r] = k.scale;
    }
  }
}

// Sixteen values a thread: tx threads (a power of two) side by side in a row.
template <int DT>
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
    for (int i = 0; i < 8; ++i) x[i] = q_of(q[2 * h + (i >> 2)], i & 3) * s;
    if (c + 8 * h < cols) store8<DT>(dst, c + 8 * h, cols, x);
  }
}

// ---------------------------------------------------------------------------
// Activation functions

// f(x) = x g(h(x)), g the logistic function; f' = g + x g (1 - g) h'.
template <int KIND>
__device__ __forceinline__ void curve(float x, float& f, float& slope) {
  float h = x, dh = 1.0f;
  if constexpr (KIND == ZERO_ACT_GELU) {
    constexpr float a = 1.5957691216057308f, b = 0.044715f * 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float x2 = x * x;
    h = x * __builtin_fmaf(b, x2, a);
    dh = fminf(__builtin_fmaf(3.0f * b, x2, a), 1e30f);  // times 0 where it would be infinite
  }
  // e^-h; beyond 104 it is 0 or infinite, and g is 1 or 0.  The product with log2(e) in two parts, so
  // that the power is right to about a unit in the last place.
  h = __builtin_amdgcn_fmed3f(h, -104.0f, 104.0f);
  const float hi = h * -1.44269502162933349609375f;
  float lo = __builtin_fmaf(h, -1.44269502162933349609375f, -hi);
  lo = __builtin_fmaf(h, -1.925963033500011079e-08f, lo);
  const float e = __builtin_amdgcn_exp2f(hi) * __builtin_fmaf(lo, 0.693147182464599609375f, 1.0f);
  const float g = __builtin_amdgcn_rcpf(1.0f + e);
  f = x * g;
  // 1 - g = e g, without cancellation; e is infinite where g is 0
  const float rest = g > 0.0f ? e * g : 1.0f;
  slope = __builtin_fmaf(f * rest, dh, g);
}
template <int KIND>
__device__ __forceinline__ float value(float x) {
  float f, s;
  curve<KIND>(x, f, s);
  return f;
}

template <int DT>
__device__ __forceinline__ void load_row8(const char* row, int64_t c, int64_t cols, float (&x)[8]) {
  decode8<DT>(load8<DT>(row, c, cols), x);
}
__device__ __forceinline__ void store_y(const MatArg& y, int64_t r, int64_t c, int64_t cols, const float (&v)[8]) {
  char* row = (char*)y.p + r * y.pitch * (y.dtype == ZERO_F32 ? 4 : 2);
  if (y.dtype == ZERO_BF16) store8<ZERO_BF16>(row, c, cols, v);
  else if (y.dtype == ZERO_F16) store8<ZERO_F16>(row, c, cols, v);
  else store8<ZERO_F32>(row, c, cols, v);
}

// A row of x in its parts: one of n elements, or gate and factor of n each.  The packed x has them
// behind each other without a gap, so a part need not begin on one of q's vectors (n odd): its
// bytes are then stored one by one.
template <int DT, int KIND, bool GATED, int T, int U>
__global__ void __launch_bounds__(kRowBlock<T>) act_kernel(MatArg x, PackArg xp, MatArg y, PackArg yp, int64_t m,
                                                           int64_t n) {
  __shared__ uint32_t lds[T / kWave];
  constexpr int P = GATED ? 2 : 1;
  const int t = threadIdx.x % T;
  const int64_t wide = padded(n), xcols = P * n;
  const bool together = !GATED || n % 8 == 0;
  for (int64_t r = (int64_t)blockIdx.x * kRowsOf<T> + threadIdx.x / T; r < m; r += (int64_t)gridDim.x * kRowsOf<T>) {
    const char* src = (const char*)x.p + r * x.pitch * esize(DT);
    const char* src2 = src + n * esize(DT);
    uint32_t mx = 0, my = 0;
    // a thread's groups of eight: in registers (U > 0), or loaded anew
    constexpr int H = U > 0 ? U : 1;
    Raw8<DT> a[H], b[H];
    float vy[H][8];
    const auto fetch = [&](int u, int64_t c) __attribute__((always_inline)) {
      a[u] = load8<DT>(src, c, n);
      if constexpr (GATED) b[u] = load8<DT>(src2, c, n);
    };
    const auto compute = [&](int u) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        vy[u][i] = value<KIND>(get<DT>(a[u], i));
        if constexpr (GATED) vy[u][i] *= get<DT>(b[u], i);
      }
    };
    const auto first = [&](int u) __attribute__((always_inline)) {
      if (yp.q) my = max8(vy[u], my);
      mx = max_raw<DT>(a[u], mx);
      if constexpr (GATED) mx = max_raw<DT>(b[u], mx);
    };
    if constexpr (U > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) fetch(u, 8 * (int64_t)(t + u * T));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        compute(u);
        first(u);
      }
    } else if (xp.q || yp.q) {
      for (int64_t c = 8 * t; c < n; c += 8 * T) {
        fetch(0, c);
        compute(0);
        first(0);
      }
    }
    mx = max_bits<DT>(mx);
    Rounding kx{}, ky{};
    if (xp.q) kx = xp.rule == ZERO_SCALE_POW2 ? rounding<ZERO_SCALE_POW2>(row_max<T>(mx, lds))
                                              : rounding<ZERO_SCALE_MAX>(row_max<T>(mx, lds));
    if (yp.q) ky = yp.rule == ZERO_SCALE_POW2 ? rounding<ZERO_SCALE_POW2>(row_max<T>(my, lds))
                                              : rounding<ZERO_SCALE_MAX>(row_max<T>(my, lds));
    int8_t* qx = xp.q + r * xp.pitch;
    int8_t* qy = yp.q + r * yp.pitch;
    const auto put = [&](const float (&v)[8], const Rounding& k, int32_t rule) __attribute__((always_inline)) {
      return rule == ZERO_SCALE_POW2 ? quantise8<ZERO_SCALE_POW2>(v, k) : quantise8<ZERO_SCALE_MAX>(v, k);
    };
    const auto second = [&](int u, int64_t c) __attribute__((always_inline)) {
      if (c < n && y.p) store_y(y, r, c, n, vy[u]);
      if (xp.q) {
        float v[8];
        decode8<DT>(a[u], v);
        const u32x2 wa = put(v, kx, xp.rule);
        if (!GATED) {
          if (c < wide) *(u32x2*)(qx + c) = wa;
        } else {
          decode8<DT>(b[u], v);
          const u32x2 wb = put(v, kx, xp.rule);
          if (together) {
            if (c < n) *(u32x2*)(qx + c) = wa, *(u32x2*)(qx + n + c) = wb;
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c + i < n) {
                qx[c + i] = (int8_t)(wa[i >> 2] >> (8 * (i & 3)));
                qx[n + c + i] = (int8_t)(wb[i >> 2] >> (8 * (i & 3)));
              }
          }
        }
      }
      if (yp.q && c < wide) *(u32x2*)(qy + c) = put(vy[u], ky, yp.rule);
    };
    if constexpr (U > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) second(u, 8 * (int64_t)(t + u * T));
    } else {
      for (int64_t c = 8 * t; c < wide; c += 8 * T) {
        fetch(0, c);
        compute(0);
        second(0, c);
      }
    }
    if (t == 0) {
      if (xp.q) xp.scale[r] = kx.scale;
      if (yp.q) yp.scale[r] = ky.scale;
    }
    // the zeros behind a gated row
    if (GATED && xp.q && xcols + t < padded(xcols)) qx[xcols + t] = 0;
  }
}

// dx of dy and the packed x, sixteen results of each part a thread.
template <int DY, int DX, int KIND, bool GATED>
__global__ void __launch_bounds__(256) act_grad_kernel(PackArg xp, MatArg dy, MatArg dx, int64_t m, int64_t n, int log_tx,
                                                       int64_t col_blocks) {
  const int64_t rb = blockIdx.x / col_blocks, cb = blockIdx.x % col_blocks;
  const int64_t c = ((cb << log_tx) + (threadIdx.x & ((1 << log_tx) - 1))) * 16;
  const int64_t r = (rb << (8 - log_tx)) + (threadIdx.x >> log_tx);
  if (r >= m || c >= n) return;
  const int8_t* q = xp.q + r * xp.pitch;
  const u32x4 qa = *(const u32x4*)(q + c);
  u32x4 qb = {};
  if constexpr (GATED) {
    if (c + 16 <= n) {
      qb = load_any<u32x4>(q + n + c);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c + i < n) qb[i >> 2] |= (uint32_t)(uint8_t)q[n + c + i] << (8 * (i & 3));
    }
  }
  const float s = xp.scale[r];
  const char* src = (const char*)dy.p + r * dy.pitch * esize(DY);
  char* dst = (char*)dx.p + r * dx.pitch * esize(DX);
  float d[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h) load_row8<DY>(src, c + 8 * h, n, d[h]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float o[8], o2[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f, slope;
      curve<KIND>(q_of(qa[2 * h + (i >> 2)], i & 3) * s, f, slope);
      if constexpr (GATED) {
        const float u = q_of(qb[2 * h + (i >> 2)], i & 3) * s;
        o[i] = d[h][i] * u * slope;
        o2[i] = d[h][i] * f;
      } else {
        o[i] = d[h][i] * slope;
      }
    }
    if (c + 8 * h < n) {
      store8<DX>(dst, c + 8 * h, n, o);
      if constexpr (GATED) store8<DX>(dst + n * esize(DX), c + 8 * h, n, o2);
    }
  }
}

// ---------------------------------------------------------------------------
// Launches

constexpr int64_t kMaxGrid = 1 << 20;  // blocks of a launch over rows, which loops beyond

template <int T>
static int64_t row_grid(int64_t rows) {
  const int64_t b = (rows + kRowsOf<T> - 1) / kRowsOf<T>;
  return b < kMaxGrid ? b : kMaxGrid;
}

// Calls fn<T, U> with the threads and loads of rows of `cols` elements.
template <class F>
static void by_length(int64_t cols, F fn) {
  const int64_t groups = (cols + 15) / 16 * 2;
  using std::integral_constant;
  if (groups <= 64) fn(integral_constant<int, 64>(), integral_constant<int, 1>());
  else if (groups <= 128) fn(integral_constant<int, 64>(), integral_constant<int, 2>());
  else if (groups <= 256) fn(integral_constant<int, 64>(), integral_constant<int, 4>());
  else if (groups <= 512) fn(integral_constant<int, 256>(), integral_constant<int, 2>());
  else if (groups <= 768) fn(integral_constant<int, 256>(), integral_constant<int, 3>());
  else if (groups <= 1024) fn(integral_constant<int, 256>(), integral_constant<int, 4>());
  else if (groups <= 1536) fn(integral_constant<int, 512>(), integral_constant<int, 3>());
  else if (groups <= 2048) fn(integral_constant<int, 512>(), integral_constant<int, 4>());
  else if (groups <= 4096) fn(integral_constant<int, 1024>(), integral_constant<int, 4>());
  else fn(integral_constant<int, 1024>(), integral_constant<int, 0>());
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

using namespace packed;

hipError_t launch_write(const MatArg& x, const PackArg& p, int64_t rows, int64_t cols, hipStream_t st) {
  by_dtype(x.dtype, [&](auto dt) {
    by_length(cols, [&](auto t, auto u) {
      constexpr int D = decltype(dt)::value, T = decltype(t)::value, U = decltype(u)::value;
      const dim3 grid((uint32_t)row_grid<T>(rows));
      if (p.rule == ZERO_SCALE_POW2) write_kernel<D, ZERO_SCALE_POW2, T, U><<<grid, kRowBlock<T>, 0, st>>>(x, p, rows, cols);
      else write_kernel<D, ZERO_SCALE_MAX, T, U><<<grid, kRowBlock<T>, 0, st>>>(x, p, rows, cols);
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
      read_kernel<decltype(dt)::value><<<(uint32_t)(nb * t.col_blocks), 256, 0, st>>>(q, o, rows - r0, cols, t.log_tx, t.col_blocks);
    });
  }
  return hipGetLastError();
}

hipError_t launch_act(int kind, bool gated, const MatArg& x, const PackArg& xp, const MatArg& y, const PackArg& yp,
                      int64_t m, int64_t n, hipStream_t st) {
  by_dtype(x.dtype, [&](auto dt) {
    by_length(n, [&](auto t, auto u) {
      constexpr int D = decltype(dt)::value, T = decltype(t)::value, U = decltype(u)::value;
      const dim3 grid((uint32_t)row_grid<T>(m));
      if (kind == ZERO_ACT_GELU) {
        if (gated) act_kernel<D, ZERO_ACT_GELU, true, T, U><<<grid, kRowBlock<T>, 0, st>>>(x, xp, y, yp, m, n);
        else act_kernel<D, ZERO_ACT_GELU, false, T, U><<<grid, kRowBlock<T>, 0, st>>>(x, xp, y, yp, m, n);
      } else {
        if (gated) act_kernel<D, ZERO_ACT_SILU, true, T, U><<<grid, kRowBlock<T>, 0, st>>>(x, xp, y, yp, m, n);
        else act_kernel<D, ZERO_ACT_SILU, false, T, U><<<grid, kRowBlock<T>, 0, st>>>(x, xp, y, yp, m, n);
      }
    });
  });
  return hipGetLastError();
}

template <int KIND, bool GATED>
static void act_grad_typed(const PackArg& xp, const MatArg& dy, const MatArg& dx, int64_t m, int64_t n, const Tiles& t,
                           uint32_t grid, hipStream_t st) {
  by_dtype(dy.dtype, [&](auto a) {
    by_dtype(dx.dtype, [&](auto b) {
      act_grad_kernel<decltype(a)::value, decltype(b)::value, KIND, GATED><<<grid, 256, 0, st>>>(xp, dy, dx, m, n, t.log_tx, t.col_blocks);
    });
  });
}

hipError_t launch_act_grad(int kind, bool gated, const PackArg& xp, const MatArg& dy, const MatArg& dx, int64_t m,
                           int64_t n, hipStream_t st) {
  const Tiles t = tiles_of(m, n);
  const int64_t most = (((int64_t)1 << 24) - 1) / t.col_blocks;
  for (int64_t b = 0; b < t.row_blocks; b += most) {
    const int64_t r0 = b * (256 >> t.log_tx), nb = t.row_blocks - b < most ? t.row_blocks - b : most;
    PackArg q = xp;
    q.q += r0 * xp.pitch;
    q.scale += r0;
    MatArg s = dy, o = dx;
    s.p = (char*)dy.p + r0 * dy.pitch * (dy.dtype == ZERO_F32 ? 4 : 2);
    o.p = (char*)dx.p + r0 * dx.pitch * (dx.dtype == ZERO_F32 ? 4 : 2);
    const uint32_t grid = (uint32_t)(nb * t.col_blocks);
    if (kind == ZERO_ACT_GELU) {
      if (gated) act_grad_typed<ZERO_ACT_GELU, true>(q, s, o, m - r0, n, t, grid, st);
      else act_grad_typed<ZERO_ACT_GELU, false>(q, s, o, m - r0, n, t, grid, st);
    } else {
      if (gated) act_grad_typed<ZERO_ACT_SILU, true>(q, s, o, m - r0, n, t, grid, st);
      else act_grad_typed<ZERO_ACT_SILU, false>(q, s, o, m - r0, n, t, grid, st);
    }
  }
  return hipGetLastError();
}

}  // namespace zs
