// gfx950 kernels of the gradient-list operators.
//
// All of them walk the list's work table: one block per item of at most kGradsChunk
// elements, and four small tensors per block, one per wave.  Elements go four at a time --
// 8-byte accesses of 16-bit data, 16-byte accesses of fp32 -- with U groups per lane in
// flight.  The side that is written is brought to its vector alignment by peeling at most 3
// leading elements; the other side is read at whatever element alignment it has left (global
// loads take any), so tensors that lie back to back at odd offsets need no slow path.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "grads.h"
#include "zs_device.h"
#include "zs_internal.h"

namespace zs {

namespace {

// Addresses from the work table are global memory; said so, the accesses are global ones
// instead of flat ones, which would also occupy the LDS counter.
#define ZS_GLOBAL __attribute__((address_space(1)))
typedef const ZS_GLOBAL char* src_t;
typedef ZS_GLOBAL char* dst_t;
// Vectors at element alignment only.
typedef f32x4 f32x4_u __attribute__((aligned(4)));
typedef u32x2 u32x2_u __attribute__((aligned(2)));

template <int T>
constexpr int kSize = T == ZERO_F32 ? 4 : 2;

template <int T>
__device__ __forceinline__ float load1(src_t p) {
  if constexpr (T == ZERO_F32) return *(const ZS_GLOBAL float*)p;
  else return dec16<T>(*(const ZS_GLOBAL uint16_t*)p);
}
// Four consecutive elements as they lie in memory.
template <int T>
struct Raw4 {
  typename std::conditional<T == ZERO_F32, f32x4, u32x2>::type r;
};
template <int T>
__device__ __forceinline__ Raw4<T> load4(src_t p) {
  if constexpr (T == ZERO_F32) return {*(const ZS_GLOBAL f32x4_u*)p};
  else return {*(const ZS_GLOBAL u32x2_u*)p};
}
template <int T>
__device__ __forceinline__ f32x4 decode4(Raw4<T> x) {
  if constexpr (T == ZERO_F32) return x.r;
  else return dec16x4<T>(x.r);
}
// x as an fp32 value: keeps the compiler from joining the product that made it and an fp16
// conversion into one instruction, which rounds once where the definition rounds twice.
__device__ __forceinline__ float rounded(float x) {
  asm("" : "+v"(x));
  return x;
}
template <int T>
__device__ __forceinline__ void store1(dst_t p, float x) {
  if constexpr (T == ZERO_F32) *(ZS_GLOBAL float*)p = x;
  else *(ZS_GLOBAL uint16_t*)p = (uint16_t)enc16<T>(rounded(x));
}
template <int T>
__device__ __forceinline__ void store4(dst_t p, f32x4 x) {
  if constexpr (T == ZERO_F32) {
    *(ZS_GLOBAL f32x4*)p = x;
  } else {
    if constexpr (T == ZERO_F16) x = f32x4{rounded(x.x), rounded(x.y), rounded(x.z), rounded(x.w)};
    *(ZS_GLOBAL u32x2*)p = enc16x4<T>(x);
  }
}
// Elements before p reaches the alignment of a group of four (0..3).
template <int T>
__device__ __forceinline__ int lead4(src_t p) {
  constexpr uint32_t a = 4 * kSize<T>;
  return (int)(((a - ((uint32_t)(uintptr_t)p & (a - 1))) & (a - 1)) / kSize<T>);
}

// ---------------------------------------------------------------------------
// walking a work item

// First element of group g.  !FULL: g may lie beyond the run's ng groups, and the last one is
// read in its place, so that the loads of a run's end stay unconditional and in flight
// together.
template <bool FULL>
__device__ __forceinline__ int64_t group_at(int head, int g, int ng) {
  return head + 4 * (FULL || g < ng ? g : ng - 1);
}

// One run of `len` elements by W lanes of which this is lane t.
template <int W, int U, class Op>
__device__ __forceinline__ void walk_row(Op& op, int len, int t) {
  int head = op.lead();
  if (head > len) head = len;
  if (t < head) op.one(t);
  const int ng = (len - head) >> 2;  // whole groups; lane t takes t, t + W, ...
  int q = t;
  for (; q + (U - 1) * W < ng; q += U * W) op.template groups<U, W, true>(head, q, ng);
  if (q < ng) op.template groups<U, W, false>(head, q, ng);
  const int done = head + 4 * ng;
  if (t < len - done) op.one(done + t);
}

// A whole item by W lanes: one run; or rows -- a wave per row while a row fills one, else one
// element per lane.
template <int W, int U, class Op>
__device__ __forceinline__ void walk_item(Op& op, const GradsChunk& k, int t) {
  if (k.rows == 1) {
    op.row(0);
    walk_row<W, U>(op, k.cols, t);
  } else if (W > 64 && k.cols >= 256) {
    for (int r = t >> 6; r < k.rows; r += W / 64) {
      op.row(r);
      walk_row<64, U>(op, k.cols, t & 63);
    }
  } else {
    const uint32_t n = (uint32_t)k.rows * (uint32_t)k.cols, cols = (uint32_t)k.cols;
    for (uint32_t e = (uint32_t)t; e < n; e += W) {
      const uint32_t r = e / cols;
      op.row((int)r);
      op.one((int)(e - r * cols));
    }
  }
}

// ---------------------------------------------------------------------------
// norms

// What a norm accumulates.  L2: squares in fp64, where the square of a float is exact, so
// fma(d, d, s) rounds as s + d * d; four sums per lane keep the dependency chains short.  The
// sum is non-finite exactly when some u is: 2^60 squares of at most 1.2e77 stay finite, and
// nothing is subtracted.  MAX: the largest |u| as its bit pattern, whose order among
// non-negative floats is the floats' own, with infinity and then the NaNs on top -- so a NaN
// is never lost.
template <int KIND>
struct Acc;
template <>
struct Acc<ZERO_NORM_L2> {
  typedef double V;
  double s0 = 0.0, s1 = 0.0, s2 = 0.0, s3 = 0.0;
  static __device__ __forceinline__ double plus(double s, float u) {
    const double d = (double)u;
    return __builtin_fma(d, d, s);
  }
  __device__ __forceinline__ void add(float u) { s0 = plus(s0, u); }
  __device__ __forceinline__ void add4(f32x4 u) {
    s0 = plus(s0, u.x);
    s1 = plus(s1, u.y);
    s2 = plus(s2, u.z);
    s3 = plus(s3, u.w);
  }
  __device__ __forceinline__ V value() const { return ((s0 + s1) + s2) + s3; }
  static __device__ __forceinline__ V none() { return 0.0; }
  static __device__ __forceinline__ V join(V a, V b) { return a + b; }
  static __device__ __forceinline__ V load(const uint64_t* p) { return load_part(p); }
  static __device__ __forceinline__ void store(uint64_t* p, V v) { store_part(p, v); }
  static __device__ __forceinline__ double acc(V v) { return v; }
};
template <>
struct Acc<ZERO_NORM_MAX> {
  typedef uint32_t V;
  uint32_t s0 = 0, s1 = 0, s2 = 0, s3 = 0;
  static __device__ __forceinline__ uint32_t plus(uint32_t s, float u) {
    return join(s, __float_as_uint(u) & 0x7FFFFFFFu);
  }
  __device__ __forceinline__ void add(float u) { s0 = plus(s0, u); }
  __device__ __forceinline__ void add4(f32x4 u) {
    s0 = plus(s0, u.x);
    s1 = plus(s1, u.y);
    s2 = plus(s2, u.z);
    s3 = plus(s3, u.w);
  }
  __device__ __forceinline__ V value() const { return join(join(s0, s1), join(s2, s3)); }
  static __device__ __forceinline__ V none() { return 0; }
  static __device__ __forceinline__ V join(V a, V b) { return a > b ? a : b; }
  static __device__ __forceinline__ V load(const uint64_t* p) {
    return (uint32_t)__hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  static __device__ __forceinline__ void store(uint64_t* p, V v) {
    __hip_atomic_store(p, (uint64_t)v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  static __device__ __forceinline__ double acc(V v) { return (double)__uint_as_float(v); }
};

template <int KIND>
__device__ __forceinline__ double norm_of(double acc) {
  return KIND == ZERO_NORM_L2 ? sqrt(acc) : acc;
}

template <class A>
__device__ __forceinline__ typename A::V wave_join(typename A::V x) {
  for (int off = 32; off > 0; off >>= 1) x = A::join(x, __shfl_xor(x, off, 64));
  return x;
}
template <class A>
__device__ __forceinline__ typename A::V block_join(typename A::V x, typename A::V* lds) {
  x = wave_join<A>(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  typename A::V r = lds[0];
  for (int w = 1; w < kGradsWaves; ++w) r = A::join(r, lds[w]);
  return r;
}

template <int T, int KIND>
struct NormOp {
  src_t base;
  int64_t pitch;
  float inv;
  Acc<KIND> acc;
  src_t s;
  __device__ __forceinline__ void row(int r) { s = base + r * pitch; }
  __device__ __forceinline__ int lead() const { return lead4<T>(s); }
  __device__ __forceinline__ void one(int j) { acc.add(load1<T>(s + (int64_t)j * kSize<T>) * inv); }
  template <int U, int W, bool FULL>
  __device__ __forceinline__ void groups(int head, int q, int ng) {
    Raw4<T> x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) x[k] = load4<T>(s + group_at<FULL>(head, q + k * W, ng) * kSize<T>);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      f32x4 u = decode4<T>(x[k]) * inv;
      if (!FULL && q + k * W >= ng) u = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      acc.add4(u);
    }
  }
};

template <int T, int KIND, int W, int U>
__device__ __forceinline__ typename Acc<KIND>::V norm_typed(const GradsChunk& k, float inv, int t) {
  NormOp<T, KIND> op{(src_t)k.src, k.src_pitch, inv, {}, (src_t)k.src};
  walk_item<W, U>(op, k, t);
  return op.acc.value();
}
template <int KIND, int W>
__device__ __forceinline__ typename Acc<KIND>::V norm_item(const GradsChunk& k, float inv, int t) {
  constexpr int U16 = W == 64 ? 4 : 8;
  if (k.src_dtype == ZERO_F32) return norm_typed<ZERO_F32, KIND, W, 4>(k, inv, t);
  if (k.src_dtype == ZERO_BF16) return norm_typed<ZERO_BF16, KIND, W, U16>(k, inv, t);
  return norm_typed<ZERO_F16, KIND, W, U16>(k, inv, t);
}

// Joins the blocks' results in an order fixed by the grid, without float atomics: a block
// stores its own, arrives on its group's counter, and the group's last block joins the
// group's results one per lane; the last group joins the groups'.  Counters are re-armed by
// their last arrival.
template <int KIND>
__device__ void grads_finish(typename Acc<KIND>::V mine, const GradsArgs& a) {
  typedef Acc<KIND> A;
  __shared__ typename A::V lds[kGradsWaves];
  __shared__ int is_last;
  const typename A::V bsum = block_join<A>(mine, lds);
  const uint32_t b = blockIdx.x, nb = gridDim.x;
  const uint32_t g = b / kGradsGroup, g0 = g * kGradsGroup;
  const uint32_t gsize = nb - g0 < (uint32_t)kGradsGroup ? nb - g0 : (uint32_t)kGradsGroup;
  const uint32_t ngroups = (nb + kGradsGroup - 1) / kGradsGroup;
  if (threadIdx.x == 0) {
    A::store(a.part + b, bsum);
    stores_complete();
    const uint32_t prev =
        __hip_atomic_fetch_add(a.gcount + 16 * g, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    is_last = prev + 1 == gsize;
  }
  __syncthreads();
  if (!is_last) return;
  typename A::V total =
      block_join<A>(threadIdx.x < gsize ? A::load(a.part + g0 + threadIdx.x) : A::none(), lds);
  if (threadIdx.x == 0) __hip_atomic_store(a.gcount + 16 * g, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (ngroups > 1) {
    if (threadIdx.x == 0) {
      A::store(a.gpart + g, total);
      stores_complete();
      const uint32_t prev = __hip_atomic_fetch_add(&a.sc->counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      is_last = prev + 1 == ngroups;
    }
    __syncthreads();
    if (!is_last) return;
    typename A::V s = A::none();
    for (uint32_t i = threadIdx.x; i < ngroups; i += kGradsBlock) s = A::join(s, A::load(a.gpart + i));
    total = block_join<A>(s, lds);
    if (threadIdx.x == 0) __hip_atomic_store(&a.sc->counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (threadIdx.x == 0) {
    const double acc = A::acc(total);
    a.sc->acc = acc;
    a.sc->flag = !__builtin_isfinite(acc);
    a.sc->norm = (float)norm_of<KIND>(acc);
  }
}

template <int KIND>
__global__ void __launch_bounds__(kGradsBlock) grads_norm_kernel(GradsArgs a, float inv) {
  typename Acc<KIND>::V v = Acc<KIND>::none();
  const int b = (int)blockIdx.x;
  if (b < a.n_block_items) {
    const GradsChunk k = a.chunks[b];
    v = norm_item<KIND, kGradsBlock>(k, inv, (int)threadIdx.x);
  } else {
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int i = (b - a.n_block_items) * kGradsWaves + wave;
    if (i < a.n_chunks - a.n_block_items) {
      const GradsChunk k = a.chunks[a.n_block_items + i];
      v = norm_item<KIND, 64>(k, inv, (int)threadIdx.x & 63);
      const typename Acc<KIND>::V w = wave_join<Acc<KIND>>(v);
      if ((threadIdx.x & 63) == 0) Acc<KIND>::store(a.wave_part + i, w);
    }
  }
  grads_finish<KIND>(v, a);
}

// A list without elements: its norm is 0.
__global__ void grads_empty_kernel(GradsScalars* sc) {
  sc->acc = 0.0;
  sc->flag = 0;
  sc->norm = 0.0f;
}

// Each tensor's norm from its items' results, by W lanes per tensor, in an order fixed by
// the number of items.
template <int KIND, int W>
__global__ void __launch_bounds__(kGradsBlock) grads_tensor_norms_kernel(GradsArgs a) {
  typedef Acc<KIND> A;
  __shared__ typename A::V lds[kGradsWaves];
  const int i = (int)blockIdx.x * (kGradsBlock / W) + (int)threadIdx.x / W;
  const int t = (int)threadIdx.x % W;
  typename A::V s = A::none();
  if (i < a.n_tensors) {
    const GradsRange r = a.ranges[i];
    const uint64_t* p = r.first < a.n_block_items ? a.part + r.first : a.wave_part + (r.first - a.n_block_items);
    for (int c = t; c < r.count; c += W) s = A::join(s, A::load(p + c));
  }
  s = W == 64 ? wave_join<A>(s) : block_join<A>(s, lds);
  if (i < a.n_tensors && t == 0) {
    const double acc = A::acc(s);
    a.tensor_acc[i] = acc;
    a.norms[i] = (float)norm_of<KIND>(acc);
  }
}

// ---------------------------------------------------------------------------
// clip and scale

template <int S, int D>
struct ScaleOp {
  src_t sbase;
  dst_t dbase;
  int64_t spitch, dpitch;
  float inv, coef;
  src_t s;
  dst_t d;
  __device__ __forceinline__ void row(int r) {
    s = sbase + r * spitch;
    d = dbase + r * dpitch;
  }
  __device__ __forceinline__ int lead() const { return lead4<D>(d); }
  __device__ __forceinline__ void one(int j) {
    store1<D>(d + (int64_t)j * kSize<D>, (load1<S>(s + (int64_t)j * kSize<S>) * inv) * coef);
  }
  template <int U, int W, bool FULL>
  __device__ __forceinline__ void groups(int head, int q, int ng) {
    Raw4<S> x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) x[k] = load4<S>(s + group_at<FULL>(head, q + k * W, ng) * kSize<S>);
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (FULL || q + k * W < ng)
        store4<D>(d + (int64_t)(head + 4 * (q + k * W)) * kSize<D>, (decode4<S>(x[k]) * inv) * coef);
  }
};

template <int S, int D, int W>
__device__ __forceinline__ void scale_item(const GradsChunk& k, float inv, float coef, int t) {
  const src_t s = (src_t)k.src;
  const dst_t d = (dst_t)k.dst;
  ScaleOp<S, D> op{s, d, k.src_pitch, k.dst_pitch, inv, coef, s, d};
  walk_item<W, 4>(op, k, t);
}
template <int S, int W>
__device__ __forceinline__ void scale_to(const GradsChunk& k, float inv, float coef, int t) {
  if (k.dst_dtype == ZERO_F32) scale_item<S, ZERO_F32, W>(k, inv, coef, t);
  else if (k.dst_dtype == ZERO_BF16) scale_item<S, ZERO_BF16, W>(k, inv, coef, t);
  else scale_item<S, ZERO_F16, W>(k, inv, coef, t);
}
template <int W>
__device__ __forceinline__ void scale_any(const GradsChunk& k, float inv, float coef, int t) {
  if (inv == 1.0f && coef == 1.0f && k.src == k.dst) return;  // in place and nothing to change
  if (k.src_dtype == ZERO_F32) scale_to<ZERO_F32, W>(k, inv, coef, t);
  else if (k.src_dtype == ZERO_BF16) scale_to<ZERO_BF16, W>(k, inv, coef, t);
  else scale_to<ZERO_F16, W>(k, inv, coef, t);
}

struct ClipArgs {
  int32_t kind, scope;
  float inv, max_norm;
  int32_t other_flag;
  double other_acc;
};

__device__ __forceinline__ float coefficient(double norm, bool bad, float max_norm) {
  if (bad || !(max_norm > 0.0f)) return 1.0f;
  const double c = (double)max_norm / (norm + 1e-6);
  return c < 1.0 ? (float)c : 1.0f;
}

// CLIP: the coefficient from the device-resident results, computed alike by every block;
// else a plain scaling by c.inv.
template <bool CLIP>
__global__ void __launch_bounds__(kGradsBlock) grads_scale_kernel(GradsArgs a, ClipArgs c) {
  float coef = 1.0f;
  bool bad = false;
  if constexpr (CLIP) {
    double acc = a.sc->acc;
    if (c.kind == ZERO_NORM_L2) acc += c.other_acc;
    else acc = c.other_acc > acc || __builtin_isnan(c.other_acc) ? c.other_acc : acc;
    const double norm = c.kind == ZERO_NORM_L2 ? sqrt(acc) : acc;
    bad = (a.sc->flag | c.other_flag) != 0 || !__builtin_isfinite(acc);
    if (c.scope == ZERO_CLIP_GLOBAL) coef = coefficient(norm, bad, c.max_norm);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      a.sc->norm = (float)norm;
      a.sc->coef = coef;
      a.sc->clip_norm = norm;
      a.sc->clip_flag = bad;
    }
  }
  const int b = (int)blockIdx.x;
  int i = b;
  const bool by_wave = b >= a.n_block_items;
  if (by_wave)
    i = a.n_block_items + (b - a.n_block_items) * kGradsWaves +
        __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (i >= a.n_chunks) return;
  const GradsChunk k = a.chunks[i];
  if (CLIP && c.scope == ZERO_CLIP_EACH) {
    const double acc = a.tensor_acc[k.tensor];
    coef = coefficient(c.kind == ZERO_NORM_L2 ? sqrt(acc) : acc, bad, c.max_norm);
  }
  if (by_wave) scale_any<64>(k, c.inv, coef, (int)threadIdx.x & 63);
  else scale_any<kGradsBlock>(k, c.inv, coef, (int)threadIdx.x);
}

// New addresses for up to kGradsBind tensors, one block per tensor.
__global__ void __launch_bounds__(kGradsBlock) grads_bind_kernel(GradsBindArgs a) {
  const int b = (int)blockIdx.x;
  const GradsRange r = a.ranges[a.first + b];
  for (int c = (int)threadIdx.x; c < r.count; c += kGradsBlock) {
    GradsChunk* k = a.chunks + r.first + c;
    k->src = a.src[b] + (uint64_t)k->src_off;
    k->dst = a.dst[b] + (uint64_t)k->dst_off;
  }
}

// Zeroes the group counters.
__global__ void __launch_bounds__(kGradsBlock) grads_arm_kernel(uint32_t* gcount, int32_t n) {
  const int i = (int)blockIdx.x * kGradsBlock + (int)threadIdx.x;
  if (i < n) gcount[16 * i] = 0;
}

}  // namespace

// ---------------------------------------------------------------------------
// launchers (host)

hipError_t launch_grads_arm(const GradsArgs& a, hipStream_t st) {
  const int32_t n = (int32_t)grads_groups(a.n_blocks);
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(grads_arm_kernel, dim3((n + kGradsBlock - 1) / kGradsBlock), dim3(kGradsBlock), 0, st, a.gcount, n);
  return hipGetLastError();
}

template <int KIND>
static hipError_t launch_norm(const GradsArgs& a, float inv, bool per_tensor, hipStream_t st) {
  if (a.n_blocks == 0) hipLaunchKernelGGL(grads_empty_kernel, dim3(1), dim3(1), 0, st, a.sc);
  else hipLaunchKernelGGL(grads_norm_kernel<KIND>, dim3(a.n_blocks), dim3(kGradsBlock), 0, st, a, inv);
  if (per_tensor) {
    if (a.max_count <= 256)
      hipLaunchKernelGGL((grads_tensor_norms_kernel<KIND, 64>), dim3((a.n_tensors - 1) / kGradsWaves + 1), dim3(kGradsBlock),
                         0, st, a);
    else
      hipLaunchKernelGGL((grads_tensor_norms_kernel<KIND, kGradsBlock>), dim3(a.n_tensors), dim3(kGradsBlock), 0, st,
                         a);
  }
  return hipGetLastError();
}

hipError_t launch_grads_norm(const GradsArgs& a, int kind, float inv, bool per_tensor, hipStream_t st) {
  return kind == ZERO_NORM_MAX ? launch_norm<ZERO_NORM_MAX>(a, inv, per_tensor, st)
                               : launch_norm<ZERO_NORM_L2>(a, inv, per_tensor, st);
}

hipError_t launch_grads_clip(const GradsArgs& a, int kind, int scope, float inv, int other_flag, double other_acc,
                             float max_norm, hipStream_t st) {
  const ClipArgs c{kind, scope, inv, max_norm, other_flag, other_acc};
  const unsigned g = a.n_blocks > 0 ? (unsigned)a.n_blocks : 1u;
  hipLaunchKernelGGL(grads_scale_kernel<true>, dim3(g), dim3(kGradsBlock), 0, st, a, c);
  return hipGetLastError();
}

hipError_t launch_grads_scale(const GradsArgs& a, float factor, hipStream_t st) {
  if (a.n_blocks == 0) return hipSuccess;
  const ClipArgs c{0, 0, factor, 0.0f, 0, 0.0};
  hipLaunchKernelGGL(grads_scale_kernel<false>, dim3(a.n_blocks), dim3(kGradsBlock), 0, st, a, c);
  return hipGetLastError();
}

hipError_t launch_grads_bind(const GradsBindArgs& a, int n, hipStream_t st) {
  hipLaunchKernelGGL(grads_bind_kernel, dim3(n), dim3(kGradsBlock), 0, st, a);
  return hipGetLastError();
}

}  // namespace zs
