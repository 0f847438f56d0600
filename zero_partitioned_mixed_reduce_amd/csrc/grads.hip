// gfx950 kernels of the gradient-list operators (compiled behind kernels.hip, see device.hip).
//
// All of them walk the list's work table: one or more items of at most kGradsChunk elements
// per block, or a part of one, and four small tensors per block, one per wave.  They are
// bounded by memory traffic: a norm reads its list once, a clip reads it twice (the
// coefficient is known only after the first time) and writes it once.  Lanes take 16 bytes at
// a time of the wider side.  The side that is written is brought to its vector alignment by
// peeling its leading elements; the other is read at whatever element alignment that leaves
// (global loads take any), so tensors that lie back to back at odd offsets need no slow path.
//
// Measured (MI355X; a copy reaches 6.4 TB/s, pure reads 7.1): norm of 1.56e9 bf16 elements with
// per-tensor norms 478 us, 6.5 TB/s, without 465; scaling them into another buffer 1012 us,
// 6.1 TB/s, and 4.1e8 fp32 elements into bf16 361 us, 6.7 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "grads.h"
#include "zs_internal.h"

// Tuning knobs (each set to the value measured fastest on MI355X):
//   ZS_GRADS_NORM_U   groups per lane in flight in the norm kernel: 2 measured the same, and 2%
//                     slower in clips of 1.2e8 elements, 8 is 3-5% slower
//   ZS_GRADS_NT_BYTES a norm over a list of more bytes than this (the Infinity Cache) reads it
//                     with non-temporal loads: 1.56e9 bf16 elements 478 us and 536 without; 4.1e8
//                     fp32 clipped in 608 and 640.  Shorter ones stay cached for the clip behind
//                     (1.2e7 to 1e8 bf16 elements are clipped 2-5% faster without)
#ifndef ZS_GRADS_NORM_U
#define ZS_GRADS_NORM_U 4
#endif
#ifndef ZS_GRADS_NT_BYTES
#define ZS_GRADS_NT_BYTES (256ll << 20)
#endif

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
typedef u32x4 u32x4_u __attribute__((aligned(2)));

template <int T>
constexpr int kSize = T == ZERO_F32 ? 4 : 2;

// One element as it lies in memory, and its value.
template <int T>
__device__ __forceinline__ uint32_t load1(src_t p) {
  if constexpr (T == ZERO_F32) return *(const ZS_GLOBAL uint32_t*)p;
  else return *(const ZS_GLOBAL uint16_t*)p;
}
template <int T>
__device__ __forceinline__ float decode1(uint32_t x) {
  if constexpr (T == ZERO_F32) return __uint_as_float(x);
  else return dec16<T>(x);
}
// G consecutive elements as they lie in memory: 16 or 8 bytes.
template <int T, int G>
struct Raw {
  static_assert(G * kSize<T> == 16 || G * kSize<T> == 8, "one vector access");
  typedef typename std::conditional<T == ZERO_F32, f32x4, typename std::conditional<G == 8, u32x4, u32x2>::type>::type V;
  typedef typename std::conditional<
      T == ZERO_F32, f32x4_u, typename std::conditional<G == 8, u32x4_u, u32x2_u>::type>::type VU;
  V r;
};
template <int T, int G, bool NT>
__device__ __forceinline__ Raw<T, G> load(src_t p) {
  typedef const ZS_GLOBAL typename Raw<T, G>::VU* ptr;
  if constexpr (NT) return {__builtin_nontemporal_load((ptr)p)};
  else return {*(ptr)p};
}
template <int T, int G, bool NT, bool ALIGNED>
__device__ __forceinline__ void store(dst_t p, Raw<T, G> x) {
  typedef ZS_GLOBAL typename std::conditional<ALIGNED, typename Raw<T, G>::V, typename Raw<T, G>::VU>::type* ptr;
  if constexpr (NT) __builtin_nontemporal_store(x.r, (ptr)p);
  else *(ptr)p = x.r;
}
// Elements 4 * i to 4 * i + 3 of a group.
template <int T, int G>
__device__ __forceinline__ f32x4 decode4(Raw<T, G> x, int i) {
  if constexpr (T == ZERO_F32) return x.r;
  else return dec16x4<T>(u32x2{x.r[2 * i], x.r[2 * i + 1]});
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
// Four results in the form in which they are stored.
template <int T>
__device__ __forceinline__ u32x2 encode4(f32x4 x) {
  return enc16x4<T>(f32x4{rounded(x.x), rounded(x.y), rounded(x.z), rounded(x.w)});
}
// Elements before p reaches a multiple of `bytes`.
template <int T>
__device__ __forceinline__ int lead(src_t p, uint32_t bytes) {
  return (int)(((0u - (uint32_t)(uintptr_t)p) & (bytes - 1)) / kSize<T>);
}

// ---------------------------------------------------------------------------
// walking a work item

// An operator works on groups of kGroup consecutive elements and on single ones, named by their
// byte offsets from the item's first element in the source and in the destination:
//   head()                    elements before its side reaches its vector alignment
//   get(so), put(mine, do, x) one element: loaded, used
//   groups<U, ALIGNED>        U groups: all loaded, then used where ok

// One run of `len` elements by W lanes of which this is lane t, U groups per lane in flight.
// Where the run is part of a longer one, its ends are moved to the next vector boundary: it
// leaves its first elements to the part before it and takes those of the part behind it
// (`after` are there), so only the ends of a tensor take single elements (into a destination
// one element off, 3.4e7 bf16 elements take 24.7 us so and 26.3 otherwise; aligned ones 22.7).
// Single elements are loaded ahead of the groups and used after them, so a short run costs one
// memory latency and not three; lanes beyond the last group read it again, so that the loads of
// a run's end stay unconditional and in flight together.
template <int W, int U, class Op>
__device__ __forceinline__ void walk_run(Op& op, int len, bool before, int after, int t) {
  constexpr int G = Op::kGroup;
  int head = op.head();
  const int end = len + (head < after ? head : after);
  if (head > end) head = end;
  const int ng = (end - head) / G;  // whole groups; lane t takes t, t + W, ...
  const int done = head + G * ng;
  const bool first = !before && t < head, last = t < end - done;
  uint32_t x = 0, y = 0;
  if (first) x = op.get((int64_t)t * Op::kS);
  if (last) y = op.get((int64_t)(done + t) * Op::kS);
  int64_t so[U], to[U];
  bool ok[U];
  int q = t;
  for (; q + (U - 1) * W < ng; q += U * W) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t e = head + G * (q + k * W);
      so[k] = e * Op::kS;
      to[k] = e * Op::kD;
      ok[k] = true;
    }
    op.template groups<U, true>(so, to, ok);
  }
  if (q < ng) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      ok[k] = q + k * W < ng;
      const int64_t e = head + G * (ok[k] ? q + k * W : ng - 1);
      so[k] = e * Op::kS;
      to[k] = e * Op::kD;
    }
    op.template groups<U, true>(so, to, ok);
  }
  op.put(first, (int64_t)t * Op::kD, x);
  op.put(last, (int64_t)(done + t) * Op::kD, y);
}

// i / n for 0 <= i < 2^13, 1 <= n: the quotient is below 2^13 / n, so what fp32 loses of it is
// less than 2^13 * 2^-22 / n, and (i + 0.5) / n is 0.5 / n or more from any integer.
__device__ __forceinline__ int small_div(int i, float one_over_n) { return (int)(((float)i + 0.5f) * one_over_n); }

// Rows of `cols` elements: the groups of all rows in one sequence, whatever their alignment,
// then the elements that are left of each row.  The norm of 4.2e6 bf16 elements in rows of 64
// takes 6.4 us so and 10.8 at one element per lane, their scaling 5.0 and 8.8; in rows of 1000,
// 6.3 us, and 6.8 at a wave per row.
template <int W, int U, class Op>
__device__ __forceinline__ void walk_rows(Op& op, int rows, int cols, int64_t spitch, int64_t tpitch, int t) {
  constexpr int G = Op::kGroup;
  const int per_row = cols / G, ng = rows * per_row, left = cols - G * per_row, n = rows * left;
  if (ng > 0) {
    const float inv = 1.0f / (float)per_row;
    int64_t so[U], to[U];
    bool ok[U];
    for (int q = t; q < ng; q += U * W) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        ok[k] = q + k * W < ng;
        const int i = ok[k] ? q + k * W : ng - 1, r = small_div(i, inv), c = G * (i - r * per_row);
        so[k] = r * spitch + c * Op::kS;
        to[k] = r * tpitch + c * Op::kD;
      }
      op.template groups<U, false>(so, to, ok);
    }
  }
  if (n > 0) {
    const float inv = 1.0f / (float)left;
    for (int i = t; i < n; i += W) {
      const int r = small_div(i, inv), c = G * per_row + i - r * left;
      op.put(true, r * tpitch + c * Op::kD, op.get(r * spitch + c * Op::kS));
    }
  }
}

// A table entry's fields, each in a register of its own (a copied struct keeps a stack slot).
__device__ __forceinline__ GradsChunk entry(const GradsChunk* c) {
  GradsChunk k;
  k.src = c->src;
  k.dst = c->dst;
  k.src_pitch = c->src_pitch;
  k.dst_pitch = c->dst_pitch;
  k.rows = c->rows;
  k.cols = c->cols;
  k.tensor = c->tensor;
  k.src_dtype = c->src_dtype;
  k.dst_dtype = c->dst_dtype;
  k.first = c->first;
  k.count = c->count;
  k.join = c->join;
  k.before = c->before;
  k.after = c->after;
  return k;
}

// A whole item by W lanes.
template <int W, int U, class Op>
__device__ __forceinline__ void walk_item(Op& op, const GradsChunk& k, int t) {
  if (k.rows == 1) walk_run<W, U>(op, k.cols, k.before != 0, k.after, t);
  else walk_rows<W, U>(op, k.rows, k.cols, k.src_pitch, k.dst_pitch, t);
}

// ---------------------------------------------------------------------------
// norms

// A clip.  The coefficients are worked out once, on the device -- by the last block of the norm
// kernel when the clip follows in the same call (now), else by a kernel of their own -- and not
// by every block that scales: the square root and division in fp64 cost a block of 2048
// elements more than its memory traffic (1.56e9 bf16 elements: 1308 us instead of 1001).
struct ClipArgs {
  int32_t now;
  int32_t scope;
  float max_norm;
  int32_t other_flag;
  double other_acc;
};

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
template <int T, int KIND, bool NT>
struct NormOp {
  static constexpr int kGroup = 16 / kSize<T>, kS = kSize<T>, kD = 0;
  src_t s;
  float inv;
  Acc<KIND> acc;
  __device__ __forceinline__ int head() const { return lead<T>(s, 16); }
  __device__ __forceinline__ uint32_t get(int64_t so) const { return load1<T>(s + so); }
  __device__ __forceinline__ void put(bool, int64_t, uint32_t x) { acc.add(decode1<T>(x) * inv); }  // 0 adds nothing
  template <int U, bool ALIGNED>
  __device__ __forceinline__ void groups(const int64_t (&so)[U], const int64_t (&)[U], const bool (&ok)[U]) {
    Raw<T, kGroup> x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) x[k] = load<T, kGroup, NT>(s + so[k]);
#pragma unroll
    for (int k = 0; k < U; ++k) {
#pragma unroll
      for (int i = 0; i < kGroup / 4; ++i) {
        f32x4 u = decode4(x[k], i) * inv;
        if (!ok[k]) u = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        acc.add4(u);
      }
    }
  }
};

// Groups in flight of a wave item: all that a lane has of kGradsSmall elements.
constexpr int wave_groups(int group) { return kGradsSmall / 64 / group; }

template <int T, int KIND, bool NT, int W>
__device__ __forceinline__ typename Acc<KIND>::V norm_typed(const GradsChunk& k, float inv, int t) {
  NormOp<T, KIND, NT> op{(src_t)k.src, inv, {}};
  walk_item<W, W == 64 ? wave_groups(op.kGroup) : ZS_GRADS_NORM_U>(op, k, t);
  return op.acc.value();
}
template <int KIND, bool NT, int W>
__device__ __forceinline__ typename Acc<KIND>::V norm_item(const GradsChunk& k, float inv, int t) {
  if (k.src_dtype == ZERO_F32) return norm_typed<ZERO_F32, KIND, NT, W>(k, inv, t);
  if (k.src_dtype == ZERO_BF16) return norm_typed<ZERO_BF16, KIND, NT, W>(k, inv, t);
  return norm_typed<ZERO_F16, KIND, NT, W>(k, inv, t);
}

__device__ __forceinline__ float coefficient(double norm, bool bad, float max_norm) {
  if (bad || !(max_norm > 0.0f)) return 1.0f;
  const double c = (double)max_norm / (norm + 1e-6);
  return c < 1.0 ? (float)c : 1.0f;
}

// Records the global norm to clip by and its coefficient.
__device__ __forceinline__ void clip_by(GradsScalars* sc, double norm, bool bad, const ClipArgs& c) {
  sc->norm = (float)norm;
  sc->coef = c.scope == ZERO_CLIP_GLOBAL ? coefficient(norm, bad, c.max_norm) : 1.0f;
  sc->clip_norm = norm;
  sc->clip_flag = bad;
  sc->refused = 0;
  sc->clipped = 1;
}

// The list's results, once per pass.
template <int KIND>
__device__ __forceinline__ void finish_list(typename Acc<KIND>::V v, GradsScalars* sc, float inv, int per_tensor,
                                            const ClipArgs& clip) {
  const double acc = Acc<KIND>::acc(v), norm = norm_of<KIND>(acc);
  sc->acc = acc;
  sc->flag = !__builtin_isfinite(acc);
  sc->norm = (float)norm;
  sc->have = clip.now ? 0 : per_tensor ? kGradsNorm | kGradsPerTensor : kGradsNorm;
  sc->kind = KIND;
  sc->inv = inv;
  if (clip.now) clip_by(sc, norm, !__builtin_isfinite(acc), clip);
}
// A tensor's results.  The coefficient is the one without the flag, which another tensor may
// yet set; what reads it goes by the flag first.
template <int KIND>
__device__ __forceinline__ void finish_tensor(typename Acc<KIND>::V v, int tensor, const GradsArgs& a,
                                              const ClipArgs& clip) {
  const double acc = Acc<KIND>::acc(v), norm = norm_of<KIND>(acc);
  a.tensor_acc[tensor] = acc;
  a.norms[tensor] = (float)norm;
  if (clip.now && clip.scope == ZERO_CLIP_EACH) a.coefs[tensor] = coefficient(norm, false, clip.max_norm);
}

// Stores a result, counts its arrival, and returns how many had arrived before.  The store is
// complete (device scope) before the arrival is counted, so whoever arrives last finds every
// result of its group.
template <class A>
__device__ __forceinline__ uint32_t arrive(uint64_t* part, typename A::V v, uint32_t* count) {
  A::store(part, v);
  stores_complete();
  return __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void rearm(uint32_t* count) {
  __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The join of p[0 .. n) by one wave: ascending per lane, then a butterfly.  Beyond one result
// per lane eight loads are in flight (a load that is not needed repeats the last).
template <class A>
__device__ __forceinline__ typename A::V wave_join_of(const uint64_t* p, uint32_t n) {
  constexpr uint32_t kFlight = 8;
  const uint32_t lane = threadIdx.x & 63;
  typename A::V v = A::none();
  if (n <= 64) {
    if (lane < n) v = A::load(p + lane);
    return wave_join<A>(v);
  }
  for (uint32_t i0 = 0; i0 < n; i0 += 64 * kFlight) {
    typename A::V x[kFlight];
#pragma unroll
    for (uint32_t k = 0; k < kFlight; ++k) {
      const uint32_t i = i0 + 64 * k + lane;
      x[k] = A::load(p + (i < n ? i : n - 1));
    }
#pragma unroll
    for (uint32_t k = 0; k < kFlight; ++k) v = A::join(v, i0 + 64 * k + lane < n ? x[k] : A::none());
  }
  return wave_join<A>(v);
}

// Two levels above n results in groups, by the wave that found its group complete: whether it
// is the last of all, and then their join in *v.  Up to kGradsDirect results the group only
// arrives at the top, and the last one joins all of them at once; beyond, it leaves its own
// join.  (1e6 to 4.2e6 bf16 elements, 130 to 520 blocks: 5.7 to 6.6 us, and 6.4 to 7.0 with
// every group's join stored; 1000 small tensors the same either way.)
template <class A>
__device__ __forceinline__ bool join_level(uint32_t n, uint32_t groups, const uint64_t* part, uint32_t first,
                                           uint32_t size, uint64_t* gpart, uint32_t g, uint32_t* top,
                                           typename A::V* v) {
  const bool lead = (threadIdx.x & 63) == 0;
  const bool direct = n <= (uint32_t)kGradsDirect;
  uint32_t had = 0;
  if (!direct) *v = wave_join_of<A>(part + first, size);
  if (groups > 1) {
    if (lead)
      had = direct ? __hip_atomic_fetch_add(top, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                   : arrive<A>(gpart + g, *v, top);
    if (__shfl(had, 0, 64) + 1 != groups) return false;
    if (lead) rearm(top);
    if (!direct) *v = wave_join_of<A>(gpart, groups);
  }
  if (direct) *v = wave_join_of<A>(part, n);
  return true;
}

// What the end of a norm block knows of one of its items.
struct ItemEnd {
  int32_t tensor, first, count, join;
};

// The end of a norm block, by its first wave: lane j < n_items holds item first_item + j's
// result.  The block's own joins the list's in an order fixed by the grid, without float
// atomics: the block arrives on its group's counter, the group's last block joins the group's
// results, and the last group joins the groups'.  With per_tensor every item's result joins
// its tensor's in the same way, in groups of kGradsJoin items; a tensor of one item is
// finished at once.  All arrivals of a block are counted together, one per lane; items that share
// a counter arrive as one (their stores are the same wave's, complete before it).  Counters are
// re-armed by their last arrival.
template <int KIND>
__device__ void norm_block_end(typename Acc<KIND>::V item, int n_items, int first_item, const ItemEnd* ends,
                               const GradsArgs& a, float inv, int per_tensor, const ClipArgs& clip) {
  typedef Acc<KIND> A;
  const int lane = (int)threadIdx.x;
  typename A::V v = __shfl(item, 0, 64);
  for (int j = 1; j < n_items; ++j) v = A::join(v, __shfl(item, j, 64));
  const uint32_t b = blockIdx.x, nb = gridDim.x, group = (uint32_t)a.group;
  const uint32_t g = b / group, g0 = g * group;
  const uint32_t gsize = nb - g0 < group ? nb - g0 : group;
  const uint32_t ngroups = (nb + group - 1) / group;
  ItemEnd e = {0, 0, 0, 0};
  uint64_t* part = a.part + b;
  uint32_t* count = a.gcount + kGradsPitch / 4 * g;
  uint32_t jsize = 0, jgroup = 0;
  if (per_tensor && lane < n_items) {
    e = ends[lane];
    const uint32_t at = (uint32_t)(first_item + lane - e.first);  // among its tensor's items
    jgroup = at / kGradsJoin;
    jsize = (uint32_t)e.count - jgroup * kGradsJoin;
    if (jsize > (uint32_t)kGradsJoin) jsize = kGradsJoin;
    part = a.item_part + first_item + lane;
    count = a.join_count + kGradsPitch / 4 * (int64_t)(e.join + (int)jgroup);
    if (e.count == 1) finish_tensor<KIND>(item, e.tensor, a, clip);
  }
  const int at = e.count > 1 ? e.join + (int)jgroup : -1;
  const int left = __shfl_up(at, 1, 64);
  const bool own = lane == 63;  // the lane that arrives for the block
  const bool leads = at >= 0 && (lane == 0 || left != at);
  const uint64_t same = ~__ballot(at >= 0 && !leads) >> lane >> 1;  // bit 0: the next lane is not of this arrival
  const uint32_t weight = own ? 1 : 1 + (uint32_t)__builtin_ctzll(same);
  if (own || at >= 0) A::store(part, own ? v : item);
  stores_complete();
  uint32_t before = 0;
  if (own || leads) before = __hip_atomic_fetch_add(count, weight, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  uint64_t last = __ballot(leads && before + weight == jsize);
  while (last) {
    const int j = __builtin_ctzll(last);
    last &= last - 1;
    const int tensor = __shfl(e.tensor, j, 64), first = __shfl(e.first, j, 64), items = __shfl(e.count, j, 64);
    const int join = __shfl(e.join, j, 64);
    const uint32_t jg = __shfl(jgroup, j, 64), n = __shfl(jsize, j, 64);
    if (lane == 0) rearm(a.join_count + kGradsPitch / 4 * (int64_t)(join + (int)jg));
    const uint32_t groups = ((uint32_t)items + kGradsJoin - 1) / kGradsJoin;
    typename A::V t;
    if (join_level<A>((uint32_t)items, groups, a.item_part + first, jg * kGradsJoin, n, a.join_part + join, jg,
                      a.join_count + kGradsPitch / 4 * (int64_t)(join + (int)groups), &t) &&
        lane == 0)
      finish_tensor<KIND>(t, tensor, a, clip);
  }
  if (__shfl(before, 63, 64) + 1 != gsize) return;
  if (lane == 0) rearm(a.gcount + kGradsPitch / 4 * g);
  if (join_level<A>(nb, ngroups, a.part, g0, gsize, a.gpart, g, &a.sc->counter, &v) && lane == 0)
    finish_list<KIND>(v, a.sc, inv, per_tensor, clip);
}

// A block takes a.run consecutive block items, so that what ends a block -- its sum, a store, an
// arrival -- is paid once for them, or a wave item per wave.  Items that go on with one run of
// elements are streamed as one; the first of them has their sum, the others nothing.  Only the
// first wave stays for the end; the others leave their places to the blocks that wait.  The norm
// of 1.56e9 bf16 elements (with per-tensor norms) takes 524 us in runs of one item, 488 of 2, 477
// of 4, 473 of 8 and 470 of 16; the clip of 1.2e8 124, 124, 124, 134 and 129 (few blocks, and the
// last ones alone).
template <int KIND, bool NT>
__global__ void __launch_bounds__(kGradsBlock, 7) grads_norm_kernel(GradsArgs a, float inv, int per_tensor,
                                                                 ClipArgs clip) {
  typedef Acc<KIND> A;
  __shared__ typename A::V sums[kGradsRun][kGradsWaves];
  __shared__ ItemEnd ends[kGradsRun];
  static_assert(kGradsRun == kGradsWaves, "a block ends at most one item per wave");
  const int b = (int)blockIdx.x, runs = (a.n_block_items + a.run - 1) / a.run;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = (int)threadIdx.x & 63;
  typename A::V item = A::none();
  int first, n_items;
  if (b < runs) {
    first = b * a.run;
    n_items = a.n_block_items - first < a.run ? a.n_block_items - first : a.run;
    for (int j = 0; j < n_items;) {
      GradsChunk k = entry(a.chunks + first + j);
      int m = 1;
      if (a.run > 1) {  // all entries are requested together
        bool on = true;
#pragma unroll
        for (int i = 1; i < kGradsRun; ++i) {
          const GradsChunk* c = a.chunks + first + (j + i < n_items ? j + i : n_items - 1);
          const int cols = c->cols, before = c->before, after = c->after;
          on = on && j + i < n_items && before != 0;
          k.cols += on ? cols : 0;
          k.after = on ? (int16_t)after : k.after;
          m += on;
        }
      }
      const typename A::V x = wave_join<A>(norm_item<KIND, NT, kGradsBlock>(k, inv, (int)threadIdx.x));
      if (lane < m) sums[j + lane][wave] = lane == 0 ? x : A::none();
      if ((int)threadIdx.x < m) ends[j + threadIdx.x] = ItemEnd{k.tensor, k.first, k.count, k.join};
      j += m;
    }
    __syncthreads();
    if (wave != 0) return;
    if (lane < n_items) item = A::join(A::join(A::join(sums[lane][0], sums[lane][1]), sums[lane][2]), sums[lane][3]);
  } else {
    first = a.n_block_items + (b - runs) * kGradsWaves;
    n_items = a.n_chunks - first < kGradsWaves ? a.n_chunks - first : kGradsWaves;
    if (wave < n_items) {
      const GradsChunk k = entry(a.chunks + first + wave);
      const typename A::V x = wave_join<A>(norm_item<KIND, false, 64>(k, inv, lane));
      if (lane == 0) {
        sums[wave][0] = x;
        ends[wave] = ItemEnd{k.tensor, k.first, k.count, k.join};
      }
    }
    __syncthreads();
    if (wave != 0) return;
    if (lane < n_items) item = sums[lane][0];
  }
  norm_block_end<KIND>(item, n_items, first, ends, a, inv, per_tensor, clip);
}

// What no item finishes: the norms of tensors without elements, 0 in every pass (an exchange may
// have left other ranks' sums there), and that of a list without elements.  A launch of its own,
// for lists that have such tensors: looked for in the norm kernel they cost every list, 483 us
// for the 477 of 1.56e9 bf16 elements.
template <int KIND>
__global__ void __launch_bounds__(kGradsBlock) grads_empty_kernel(GradsArgs a, float inv, int per_tensor,
                                                                  int list, ClipArgs clip) {
  const int i = (int)blockIdx.x * kGradsBlock + (int)threadIdx.x;
  if (per_tensor && i < a.n_tensors && a.ranges[i].count == 0) {
    a.tensor_acc[i] = 0.0;
    a.norms[i] = 0.0f;
  }
  if (list && i == 0) finish_list<KIND>(Acc<KIND>::none(), a.sc, inv, per_tensor, clip);
}

// The coefficients of a clip from the results on the device, as the norm call and an exchange
// have left them, and other ranks'.  Which norm that was, and whether the values are still the
// ones it was taken of, is read here and not passed: a replay of captured calls may have come
// between.  The first thread decides for all; the other coefficients are not used if it refuses.
__global__ void __launch_bounds__(kGradsBlock) grads_coefs_kernel(GradsArgs a, ClipArgs c) {
  const bool l2 = a.sc->kind == ZERO_NORM_L2;
  const int i = (int)blockIdx.x * kGradsBlock + (int)threadIdx.x;
  if (i == 0) {
    const int32_t need = c.scope == ZERO_CLIP_EACH ? kGradsNorm | kGradsPerTensor : kGradsNorm;
    double acc = a.sc->acc;
    if (l2) acc += c.other_acc;
    else acc = c.other_acc > acc || __builtin_isnan(c.other_acc) ? c.other_acc : acc;
    const bool bad = (a.sc->flag | c.other_flag) != 0 || !__builtin_isfinite(acc);
    if ((a.sc->have & need) == need) clip_by(a.sc, l2 ? sqrt(acc) : acc, bad, c);
    else a.sc->refused = 1;
    a.sc->have = 0;
  }
  if (c.scope == ZERO_CLIP_EACH && i < a.n_tensors) {
    const double t = a.tensor_acc[i];
    a.coefs[i] = coefficient(l2 ? sqrt(t) : t, false, c.max_norm);
  }
}

// ---------------------------------------------------------------------------
// clip and scale

// NT (block items): loads and stores are non-temporal, as nothing reads either again here.
// 1.2e8 fp16 elements, which the Infinity Cache holds, are clipped in 138 us with them and
// 164 without; 4.1e8 fp32 ones in 636 and 665.
template <int S, int D, bool NT>
struct ScaleOp {
  // 16-byte accesses on the wider side; between two 16-bit types on both
  static constexpr int kGroup = S != ZERO_F32 && D != ZERO_F32 ? 8 : 4;
  static constexpr int kS = kSize<S>, kD = kSize<D>;
  src_t s;
  dst_t d;
  float inv, coef;
  __device__ __forceinline__ int head() const { return lead<D>(d, kGroup * kD); }
  __device__ __forceinline__ uint32_t get(int64_t so) const { return load1<S>(s + so); }
  __device__ __forceinline__ void put(bool mine, int64_t to, uint32_t x) {
    if (mine) store1<D>(d + to, (decode1<S>(x) * inv) * coef);
  }
  template <int U, bool ALIGNED>
  __device__ __forceinline__ void groups(const int64_t (&so)[U], const int64_t (&to)[U], const bool (&ok)[U]) {
    Raw<S, kGroup> x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) x[k] = load<S, kGroup, NT>(s + so[k]);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (!ok[k]) continue;
      Raw<D, kGroup> y;
      const f32x4 lo = (decode4(x[k], 0) * inv) * coef;
      if constexpr (D == ZERO_F32) {
        y.r = lo;
      } else if constexpr (kGroup == 4) {
        y.r = encode4<D>(lo);
      } else {
        const u32x2 a = encode4<D>(lo), b = encode4<D>((decode4(x[k], 1) * inv) * coef);
        y.r = u32x4{a.x, a.y, b.x, b.y};
      }
      store<D, kGroup, NT, ALIGNED>(d + to[k], y);
    }
  }
};

template <int S, int D, int W, bool NT>
__device__ __forceinline__ void scale_item(const GradsChunk& k, float inv, float coef, int t) {
  ScaleOp<S, D, NT> op{(src_t)k.src, (dst_t)k.dst, inv, coef};
  walk_item<W, W == 64 ? wave_groups(op.kGroup) : op.kGroup / 4>(op, k, t);
}
template <int S, int W, bool NT>
__device__ __forceinline__ void scale_to(const GradsChunk& k, float inv, float coef, int t) {
  if (k.dst_dtype == ZERO_F32) scale_item<S, ZERO_F32, W, NT>(k, inv, coef, t);
  else if (k.dst_dtype == ZERO_BF16) scale_item<S, ZERO_BF16, W, NT>(k, inv, coef, t);
  else scale_item<S, ZERO_F16, W, NT>(k, inv, coef, t);
}
template <int W, bool NT>
__device__ __forceinline__ void scale_any(const GradsChunk& k, float inv, float coef, int t) {
  if (k.src_dtype == ZERO_F32) scale_to<ZERO_F32, W, NT>(k, inv, coef, t);
  else if (k.src_dtype == ZERO_BF16) scale_to<ZERO_BF16, W, NT>(k, inv, coef, t);
  else scale_to<ZERO_F16, W, NT>(k, inv, coef, t);
}

// By what else than `inv` and the coefficients a list is scaled: nothing; nothing, and the norm
// that stands is ended; the inverse scale of the norm on the device, unless a clip was refused.
enum ScaleBy { kScaleByArgs = 0, kScaleEndsNorm = 1, kScaleByNorm = 2 };

// One of `parts` parts of a block item per block, or four wave items; by inv and, for a clip,
// the coefficients found for it.
__global__ void __launch_bounds__(kGradsBlock) grads_scale_kernel(GradsArgs a, float inv, int scope, int by, int parts) {
  const int b = (int)blockIdx.x;
  const int whole = a.n_block_items * parts;
  const bool by_wave = b >= whole;
  const int i = by_wave ? a.n_block_items + (b - whole) * kGradsWaves +
                              __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6)
                        : b / parts;
  if (i >= a.n_chunks) return;
  GradsChunk k = entry(a.chunks + i);
  const float coef = scope == ZERO_CLIP_GLOBAL                       ? a.sc->coef
                     : scope == ZERO_CLIP_EACH && !a.sc->clip_flag ? a.coefs[k.tensor]
                                                                   : 1.0f;
  if (by == kScaleByNorm) {
    inv = a.sc->inv;
    if (a.sc->refused) return;
  } else if (by == kScaleEndsNorm && b == 0 && threadIdx.x == 0) {
    a.sc->have = 0;  // behind the loads above, which would not be scalar ones after a store
  }
  if (inv == 1.0f && coef == 1.0f && k.src == k.dst) return;  // in place and nothing to change
  if (by_wave) {
    scale_any<64, false>(k, inv, coef, (int)threadIdx.x & 63);
    return;
  }
  // the part: of a run, or whole rows
  const int n = k.rows == 1 ? kGradsChunk / parts : (k.rows + parts - 1) / parts;
  const int lo = b % parts * n, have = (k.rows == 1 ? k.cols : k.rows) - lo;
  if (have <= 0) return;
  if (k.rows == 1) {
    k.cols = have < n ? have : n;
    k.before = lo > 0 || k.before;
    if (have > n) k.after = (int16_t)(have - n + k.after < 7 ? have - n + k.after : 7);
    k.src += (uint64_t)(lo * (k.src_dtype == ZERO_F32 ? 4 : 2));
    k.dst += (uint64_t)(lo * (k.dst_dtype == ZERO_F32 ? 4 : 2));
  } else {
    k.rows = have < n ? have : n;
    k.src += (uint64_t)(lo * k.src_pitch);
    k.dst += (uint64_t)(lo * k.dst_pitch);
  }
  scale_any<kGradsBlock, true>(k, inv, coef, (int)threadIdx.x);
}

// ---------------------------------------------------------------------------
// addresses

// New addresses for up to kGradsBind tensors, one block per tensor.
__global__ void __launch_bounds__(kGradsBlock) grads_bind_kernel(GradsBindArgs a) {
  const int b = (int)blockIdx.x;
  const GradsRange r = a.ranges[a.first + b];
  if (b == 0 && threadIdx.x == 0) a.sc->have = 0;
  for (int c = (int)threadIdx.x; c < r.count; c += kGradsBlock) {
    GradsChunk* k = a.chunks + r.first + c;
    const GradsOffset o = a.offsets[r.first + c];
    k->src = a.src[b] + (uint64_t)o.src;
    k->dst = a.dst[b] + (uint64_t)o.dst;
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// launchers (host)

template <int KIND>
static hipError_t launch_norm(const GradsArgs& a, float inv, bool per_tensor, const ClipArgs& c, hipStream_t st) {
  const unsigned g = (unsigned)((a.n_block_items + a.run - 1) / a.run + (a.n_blocks - a.n_block_items));
  if (g == 0 || (per_tensor && a.n_empty > 0)) {
    const unsigned ge = per_tensor ? (unsigned)((a.n_tensors - 1) / kGradsBlock + 1) : 1u;
    hipLaunchKernelGGL(grads_empty_kernel<KIND>, dim3(ge), dim3(kGradsBlock), 0, st, a, inv, (int)per_tensor,
                       (int)(g == 0), c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || g == 0) return e;
  }
  if (a.bytes_in > ZS_GRADS_NT_BYTES)
    hipLaunchKernelGGL((grads_norm_kernel<KIND, true>), dim3(g), dim3(kGradsBlock), 0, st, a, inv, (int)per_tensor, c);
  else
    hipLaunchKernelGGL((grads_norm_kernel<KIND, false>), dim3(g), dim3(kGradsBlock), 0, st, a, inv, (int)per_tensor, c);
  return hipGetLastError();
}

static hipError_t launch_norm_of(const GradsArgs& a, int norm, float inv, bool per_tensor, const ClipArgs& c,
                                 hipStream_t st) {
  return norm == ZERO_NORM_MAX ? launch_norm<ZERO_NORM_MAX>(a, inv, per_tensor, c, st)
                               : launch_norm<ZERO_NORM_L2>(a, inv, per_tensor, c, st);
}

// scope 0: by inv alone.
static hipError_t launch_scaling(const GradsArgs& a, float inv, int scope, ScaleBy by, hipStream_t st) {
  if (a.n_blocks == 0) return hipSuccess;
  // A block for 8 KiB of the wider side: short-lived blocks of one or two groups per lane keep
  // reads and writes in step (bf16 to bf16, 1.56e9 elements: 1156 us with whole items, 1012
  // with halves, 1030 with quarters; fp32 to bf16, 4.1e8: 445, 415 and 361; eighths 1350 and 450).
  const int parts = a.all16 ? 2 : 4;
  const unsigned g = (unsigned)(a.n_blocks + (int64_t)a.n_block_items * (parts - 1));
  hipLaunchKernelGGL(grads_scale_kernel, dim3(g), dim3(kGradsBlock), 0, st, a, inv, scope, (int)by, parts);
  return hipGetLastError();
}

hipError_t launch_grads_norm(const GradsArgs& a, int norm, float inv, bool per_tensor, hipStream_t st) {
  return launch_norm_of(a, norm, inv, per_tensor, ClipArgs{}, st);
}

hipError_t launch_grads_clip(const GradsArgs& a, int scope, int other_flag, double other_acc, float max_norm,
                             hipStream_t st) {
  const ClipArgs c{1, scope, max_norm, other_flag, other_acc};
  const unsigned g = scope == ZERO_CLIP_EACH ? (unsigned)((a.n_tensors - 1) / kGradsBlock + 1) : 1u;
  hipLaunchKernelGGL(grads_coefs_kernel, dim3(g), dim3(kGradsBlock), 0, st, a, c);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_scaling(a, 1.0f, scope, kScaleByNorm, st);
}

hipError_t launch_grads_clip_norm(const GradsArgs& a, int norm, float inv, bool per_tensor, int scope, float max_norm,
                                  hipStream_t st) {
  const ClipArgs c{1, scope, max_norm, 0, 0.0};
  hipError_t e = launch_norm_of(a, norm, inv, per_tensor, c, st);
  return e != hipSuccess ? e : launch_scaling(a, inv, scope, kScaleByArgs, st);
}

hipError_t launch_grads_scale(const GradsArgs& a, float factor, bool ends_norm, hipStream_t st) {
  return launch_scaling(a, factor, 0, ends_norm ? kScaleEndsNorm : kScaleByArgs, st);
}

hipError_t launch_grads_bind(const GradsBindArgs& a, int n, hipStream_t st) {
  hipLaunchKernelGGL(grads_bind_kernel, dim3(n), dim3(kGradsBlock), 0, st, a);
  return hipGetLastError();
}

}  // namespace zs
