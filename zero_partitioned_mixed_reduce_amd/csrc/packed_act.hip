// gfx950 kernels of the activation functions: forward, packing the input and the result, and backward
// from the packed input.  Each element is read and written once; the forward's rows stay in
// registers while their scales are found, as in packed_rows.hip (rows beyond 16384 elements are
// read twice).  8192 x 2 x 11008 in bf16, gated, both packed: 117 to 134 us (4.7 to 5.4 TB/s), backward
// 135 to 138 (5.2).  Both have 30 to 37 instructions an element, an exponential and a reciprocal among
// them, about as long as its bytes take: the vector units are busy 80% of the forward's time and 62% of
// the backward's, at 2048 x 6400, plain, 87 and 90%.
#include "packed_rows.h"

namespace zs {
namespace packed {

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

template <bool TAIL>
__device__ __forceinline__ void store_y(const MatArg& y, int64_t r, int64_t c, int64_t cols, float (&v)[8]) {
  char* row = (char*)y.p + r * y.pitch * (y.dtype == ZERO_F32 ? 4 : 2);
  if (y.dtype == ZERO_BF16) store8<ZERO_BF16, TAIL>(row, c, cols, v);
  else if (y.dtype == ZERO_F16) store8<ZERO_F16, TAIL>(row, c, cols, v);
  else store8<ZERO_F32, TAIL>(row, c, cols, v);
}

// A row of x in its parts: one of n elements, or gate and factor of n each.  The packed x has them
// behind each other without a gap, so a part need not begin on one of q's vectors (n odd): its
// bytes are then stored one by one.
template <int DT, int KIND, bool GATED, bool TAIL, int T, int U>
__global__ void __launch_bounds__(kRowBlock<T>, 4) act_kernel(MatArg x, PackArg xp, MatArg y, PackArg yp, int64_t m,
                                                           int64_t n) {
  __shared__ uint32_t lds[T / kWave];
  constexpr int P = GATED ? 2 : 1;
  const int t = threadIdx.x % T;
  const int64_t wide = padded(n), xcols = P * n;
  for (int64_t r = (int64_t)blockIdx.x * kRowsOf<T> + threadIdx.x / T; r < m; r += (int64_t)gridDim.x * kRowsOf<T>) {
    const char* src = (const char*)x.p + r * x.pitch * esize(DT);
    const char* src2 = src + n * esize(DT);
    uint32_t mx = 0, my = 0;
    // a thread's groups of eight: in registers (U > 0), or loaded anew
    constexpr int H = U > 0 ? U : 1;
    Raw8<DT> a[H], b[H];
    float vy[H][8];
    const auto fetch = [&](int u, int64_t c) __attribute__((always_inline)) {
      a[u] = load8<DT, TAIL>(src, c, n);
      if constexpr (GATED) b[u] = load8<DT, TAIL>(src2, c, n);
    };
    const auto compute = [&](int u) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        vy[u][i] = value<KIND>(get<DT>(a[u], i));
        if constexpr (GATED) vy[u][i] *= get<DT>(b[u], i);
      }
    };
    const auto first = [&](int u) __attribute__((always_inline)) {
      if (yp.scale) my = max8(vy[u], my);
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
    } else if (xp.scale || yp.scale) {
      for (int64_t c = 8 * t; c < n; c += 8 * T) {
        fetch(0, c);
        compute(0);
        first(0);
      }
    }
    mx = max_bits<DT>(mx);
    Rounding kx{}, ky{};
    if (xp.scale) kx = xp.rule == ZERO_SCALE_POW2 ? rounding<ZERO_SCALE_POW2>(row_max<T>(mx, lds))
                                                  : rounding<ZERO_SCALE_MAX>(row_max<T>(mx, lds));
    if (yp.scale) ky = yp.rule == ZERO_SCALE_POW2 ? rounding<ZERO_SCALE_POW2>(row_max<T>(my, lds))
                                                  : rounding<ZERO_SCALE_MAX>(row_max<T>(my, lds));
    int8_t* qx = xp.q + r * xp.pitch;
    int8_t* qy = yp.q + r * yp.pitch;
    const auto put = [&](const float (&v)[8], const Rounding& k, int32_t rule) __attribute__((always_inline)) {
      return rule == ZERO_SCALE_POW2 ? quantise8<ZERO_SCALE_POW2>(v, k) : quantise8<ZERO_SCALE_MAX>(v, k);
    };
    const auto second = [&](int u, int64_t c) __attribute__((always_inline)) {
      if (c < n && y.p) store_y<TAIL>(y, r, c, n, vy[u]);
      if (xp.scale) {
        float v[8];
        decode8<DT>(a[u], v);
        const u32x2 wa = put(v, kx, xp.rule);
        if (!GATED) {
          if (c < wide) *(u32x2*)(qx + c) = wa;
        } else {
          decode8<DT>(b[u], v);
          const u32x2 wb = put(v, kx, xp.rule);
          if constexpr (!TAIL) {
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
      if (yp.scale && c < wide) *(u32x2*)(qy + c) = put(vy[u], ky, yp.rule);
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
      if (xp.scale) xp.scale[r] = kx.scale;
      if (yp.scale) yp.scale[r] = ky.scale;
    }
    // the zeros behind a gated row
    if (GATED && xp.scale && xcols + t < padded(xcols)) qx[xcols + t] = 0;
  }
}

// dx of dy and the packed x, sixteen results of each part a thread.
template <int DY, int DX, int KIND, bool GATED, bool TAIL>
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
    } else if constexpr (!TAIL) {  // eight of them
      const u32x2 half = load_any<u32x2>(q + n + c);
      qb = u32x4{half.x, half.y, 0, 0};
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
  for (int h = 0; h < 2; ++h) decode8<DY>(load8<DY, TAIL>(src, c + 8 * h, n), d[h]);
  // all results before the first store, so that the two halves of a line follow each other (written
  // apart, 12% more went below the L2)
  float o[2][8], o2[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float xa[8], xb[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      values4(qa[2 * h + i], s, xa + 4 * i);
      if constexpr (GATED) values4(qb[2 * h + i], s, xb + 4 * i);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f, slope;
      curve<KIND>(xa[i], f, slope);
      if constexpr (GATED) {
        o[h][i] = d[h][i] * xb[i] * slope;
        o2[h][i] = d[h][i] * f;
      } else {
        o[h][i] = d[h][i] * slope;
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (c + 8 * h < n) store8<DX, TAIL>(dst, c + 8 * h, n, o[h]);
  if constexpr (GATED) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (c + 8 * h < n) store8<DX, TAIL>(dst + n * esize(DX), c + 8 * h, n, o2[h]);
  }
}

// Calls fn with TAIL, T and U of rows of `cols` elements.  Two blocks or more have to fit a compute unit, so
// that one loads while the other computes: 11008 elements gated take 134 us (117 at best) with 512
// threads of three groups, 185 with 768 of two, of which only one block fits.  The results stay beside
// the groups in registers: three gated groups spill 4 to 6 of them, whose stores add 0.1 GB to the 0.27
// that the case writes; four would spill 31 to 43.
template <class F>
static void by_length(int64_t cols, F fn) {
  const int64_t groups = (cols + 15) / 16 * 2;
  using std::integral_constant;
  if (cols % 8 == 0) {
    const std::false_type tail;
    if (groups <= 64) fn(tail, integral_constant<int, 64>(), integral_constant<int, 1>());
    else if (groups <= 128) fn(tail, integral_constant<int, 64>(), integral_constant<int, 2>());
    else if (groups <= 256) fn(tail, integral_constant<int, 256>(), integral_constant<int, 1>());
    else if (groups <= 512) fn(tail, integral_constant<int, 256>(), integral_constant<int, 2>());
    else if (groups <= 1024) fn(tail, integral_constant<int, 512>(), integral_constant<int, 2>());
    else if (groups <= 1536) fn(tail, integral_constant<int, 512>(), integral_constant<int, 3>());
    else if (groups <= 2048) fn(tail, integral_constant<int, 1024>(), integral_constant<int, 2>());
    else fn(tail, integral_constant<int, 1024>(), integral_constant<int, 0>());
  } else {
    const std::true_type tail;
    if (groups <= 128) fn(tail, integral_constant<int, 64>(), integral_constant<int, 2>());
    else if (groups <= 512) fn(tail, integral_constant<int, 256>(), integral_constant<int, 2>());
    else if (groups <= 2048) fn(tail, integral_constant<int, 1024>(), integral_constant<int, 2>());
    else fn(tail, integral_constant<int, 1024>(), integral_constant<int, 0>());
  }
}

}  // namespace packed

using namespace packed;

hipError_t launch_act(int kind, bool gated, const MatArg& x, const PackArg& xp, const MatArg& y, const PackArg& yp,
                      int64_t m, int64_t n, hipStream_t st) {
  by_dtype(x.dtype, [&](auto dt) {
    by_length(n, [&](auto tail, auto t, auto u) {
      constexpr int D = decltype(dt)::value, T = decltype(t)::value, U = decltype(u)::value;
      constexpr bool E = decltype(tail)::value;
      const dim3 grid((uint32_t)row_grid<T>(m));
      if (kind == ZERO_ACT_GELU) {
        if (gated) act_kernel<D, ZERO_ACT_GELU, true, E, T, U><<<grid, kRowBlock<T>, 0, st>>>(x, xp, y, yp, m, n);
        else act_kernel<D, ZERO_ACT_GELU, false, E, T, U><<<grid, kRowBlock<T>, 0, st>>>(x, xp, y, yp, m, n);
      } else {
        if (gated) act_kernel<D, ZERO_ACT_SILU, true, E, T, U><<<grid, kRowBlock<T>, 0, st>>>(x, xp, y, yp, m, n);
        else act_kernel<D, ZERO_ACT_SILU, false, E, T, U><<<grid, kRowBlock<T>, 0, st>>>(x, xp, y, yp, m, n);
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
      constexpr int A = decltype(a)::value, B = decltype(b)::value;
      if (n % 8 == 0) act_grad_kernel<A, B, KIND, GATED, false><<<grid, 256, 0, st>>>(xp, dy, dx, m, n, t.log_tx, t.col_blocks);
      else act_grad_kernel<A, B, KIND, GATED, true><<<grid, 256, 0, st>>>(xp, dy, dx, m, n, t.log_tx, t.col_blocks);
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
