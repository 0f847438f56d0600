// gfx950 kernels of the packed rows' products: the linear layer in 8-bit integers, and the products
// of a 16-bit matrix with packed rows whose scales lie along the sum (weight and input gradients).
#include <cmath>
#include <type_traits>

#include "packed_device.h"

namespace zs {
namespace packed {

#define ZS_LDS(T) __attribute__((address_space(3))) T

constexpr int kXcds = 8;  // consecutive blocks go to the XCDs in turn, each with an L2 cache of its own

// The tile of block b: each XCD takes a run of consecutive tiles, and a run goes down kDown tiles of
// i before it steps to the next j, so that what an XCD works on at a time shares rows and columns.
constexpr int kDown = 8;
struct Tile {
  int64_t i, j;
};
__device__ __forceinline__ Tile tile_of(uint32_t b, uint32_t ni, uint32_t nj) {
  const uint32_t n = ni * nj, per = n / kXcds, more = n % kXcds, x = b % kXcds;
  const uint32_t t = x * per + (x < more ? x : more) + b / kXcds;
  const uint32_t band = t / (kDown * nj), in = t % (kDown * nj);
  const uint32_t high = ni - band * kDown < kDown ? ni - band * kDown : kDown;
  return {band * kDown + in % high, in / high};
}

__device__ __forceinline__ float load1(const MatArg& a, int64_t at) {
  if (a.dtype == ZERO_F32) return ((const float*)a.p)[at];
  const uint32_t h = ((const uint16_t*)a.p)[at];
  return a.dtype == ZERO_BF16 ? dec_lo<ZERO_BF16>(h) : dec_lo<ZERO_F16>(h);
}
// N consecutive elements of a row, those before column n (N = 4 or 16), at any alignment.
template <int DT, int N>
__device__ __forceinline__ void store_run(char* row, int64_t col, int64_t n, float (&x)[N]) {
  constexpr int S = esize(DT);
  if constexpr (DT != ZERO_F32) one_nan(x);
  char* p = row + col * S;
  uint32_t w[N * S / 4];
#pragma unroll
  for (int i = 0; i < N * S / 4; ++i) {
    if constexpr (DT == ZERO_F32) w[i] = __float_as_uint(x[i]);
    else w[i] = enc2<DT>(x[2 * i], x[2 * i + 1]);
  }
  if (col + N <= n) {
    constexpr int V = N * S / 4 < 4 ? N * S / 4 : 4;
    typedef uint32_t vec __attribute__((ext_vector_type(V)));
#pragma unroll
    for (int i = 0; i < N * S / 4; i += V) {
      vec v;
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = w[i + k];
      store_any(p + 4 * i, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (col + i < n) {
        if constexpr (DT == ZERO_F32) store_any(p + 4 * i, w[i]);
        else store_any(p + 2 * i, (uint16_t)(w[i >> 1] >> (16 * (i & 1))));
      }
  }
}
template <int DT, int N>
__device__ __forceinline__ void load_run(const char* row, int64_t col, int64_t n, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    if (col + i + 4 <= n) {
      if constexpr (DT == ZERO_F32) {
        const f32x4 v = load_any<f32x4>(row + (col + i) * 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i + k] = v[k];
      } else {
        const u32x2 v = load_any<u32x2>(row + (col + i) * 2);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i + k] = (k & 1) ? dec_hi<DT>(v[k >> 1]) : dec_lo<DT>(v[k >> 1]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[i + k] = 0.0f;
        if (col + i + k < n) {
          if constexpr (DT == ZERO_F32) x[i + k] = load_any<float>(row + (col + i + k) * 4);
          else x[i + k] = dec_lo<DT>(load_any<uint16_t>(row + (col + i + k) * 2));
        }
      }
    }
  }
}
// Calls fn with the type of a matrix, which is the same for a whole launch.
template <class F>
__device__ __forceinline__ void with_type(int32_t dt, F fn) {
  if (dt == ZERO_BF16) fn(std::integral_constant<int, ZERO_BF16>());
  else if (dt == ZERO_F16) fn(std::integral_constant<int, ZERO_F16>());
  else fn(std::integral_constant<int, ZERO_F32>());
}
// N results of row r from column c, with what the matrix holds added if asked for.
template <int DT, int N>
__device__ __forceinline__ void finish_run(const MatArg& c, int64_t r, int64_t col, int64_t n, int32_t accumulate, float (&v)[N]) {
  char* row = (char*)c.p + r * c.pitch * esize(DT);
  if (accumulate) {
    float old[N];
    load_run<DT, N>(row, col, n, old);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += old[k];
  }
  store_run<DT, N>(row, col, n, v);
}

// ---------------------------------------------------------------------------
// Linear layer: y[m][n] = sum over k of x[m][k] w[n][k], 16x16x64 integer matrix instructions.

constexpr int kStepK = 64;  // k of a tile step: a row of 64 bytes

// A tile step of a wave has two phases: it reads its fragments from LDS and prepares later steps, and it
// multiplies.  In a block of eight waves, two to a SIMD, the second four are a phase behind, so
// that of a SIMD's waves one multiplies while the other reads and converts (all eight in step
// leave the matrix cores idle half of the time).  A phase ends for all waves of the block at once.
//
// Ends the first phase: at most N of the wave's loads are under way, all its LDS accesses done.
template <int N>
__device__ __forceinline__ void end_reading() {
  static_assert(N >= 0 && N < 64, "what the counter holds");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 7 << 4);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// What the sums of N channels from n become: scales and bias.
template <int N>
struct Channels {
  float s[N], b[N];
  bool bias;
  __device__ __forceinline__ Channels(const LinearArgs& a, int64_t n) : bias(a.bias.p != nullptr) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = n + i < a.n ? a.w.scale[n + i] : 0.0f;
      b[i] = bias && n + i < a.n ? load1(a.bias, n + i) : 0.0f;
    }
  }
  __device__ __forceinline__ float operator()(int i, int acc, float xs) const {
    const float v = (float)acc * xs * s[i];
    return bias ? v + b[i] : v;
  }
};

// A block makes a tile of BM x BN results with WM x WN waves.  256 x 256 reads each operand's byte for 512
// operations, so that loads and LDS stay within half of their rates, and eight waves of 128 x 64 fill
// the registers; smaller results take 128 x 128 with four waves, two blocks to a compute unit (20 us
// for 1024 x 1600 x 4800 either way).  16384 x 4096 x 11008 into bf16: 684 us, 2.16e15 operations a
// second, 2.45e15 at k = 8192; bound by the matrix cores within a tile, by its stores between two.
// kStages: tile steps in LDS, of which three are on their way while one is read.
template <int BM, int BN, int WM, int WN, int kStages>
__global__ void __launch_bounds__(WM* WN * 64, 2) linear_kernel(LinearArgs a, uint32_t tiles_m, uint32_t tiles_n, int64_t steps,
                                                            int64_t per_split) {
#ifdef __HIP_DEVICE_COMPILE__  // the host's compilation has no use for it, and stumbles over the builtins
  constexpr int W = WM * WN, T = W * 64;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16x16 results of a wave
  constexpr int LX = BM * 4 / T, LW = BN * 4 / T;      // 16-byte loads of a thread
  static_assert(BM * 4 % T == 0 && BN * 4 % T == 0, "whole loads");
  static_assert(TN == 4, "a lane's results of a row are 16 consecutive ones");
  __shared__ __attribute__((aligned(1024))) char lds[kStages][(BM + BN) * kStepK];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const Tile tile = tile_of(blockIdx.x, tiles_m, tiles_n);
  const int64_t m0 = tile.i * BM, n0 = tile.j * BN;
  const int first = (int)(blockIdx.y * per_split), last = (int)(first + per_split < steps ? first + per_split : steps);
  const int chunks = (int)((a.k + 15) >> 4);  // 16-byte chunks of a row

  // A wave's load fills 16 rows of 64 bytes; chunk c of row r lies in place c ^ (-r / 4 % 4): the LDS
  // serves a 16-byte read to lanes 0-3, 12-15, 20-23 and 24-27 at a time (and to the three other such
  // sets), whose rows and chunks then lie in different banks.  Rows past the end read the last one,
  // and their results are not stored.
  const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(a.x.q + m0 * a.x.pitch, 0, 0xFFFFFFFFu, 0x00020000);
  const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(a.w.q + n0 * a.w.pitch, 0, 0xFFFFFFFFu, 0x00020000);
  const int mlast = (int)(a.m - 1 - m0 < BM - 1 ? a.m - 1 - m0 : BM - 1);
  const int nlast = (int)(a.n - 1 - n0 < BN - 1 ? a.n - 1 - n0 : BN - 1);
  const int chunk = (lane & 3) ^ (-(lane >> 4) & 3);  // of this thread's loads: r / 4 % 4 is lane / 16
  uint32_t at[LX + LW];  // of a step's loads, from the step's first byte
#pragma unroll
  for (int u = 0; u < LX + LW; ++u) {
    int r = ((u < LX ? u : u - LX) * W + wave) * 16 + (lane >> 2);
    // Row 16 j + i of each 64 of w's tile holds channel 16 (i / 4) + 4 j + i % 4: a lane's results in
    // a wave's four products j, which are rows 4 (lane / 16) + 0..3 there, are then 16 channels in a
    // row, and two stores fill whole lines (runs of 8, and 64 bytes by each store, took 2% longer).
    if (u >= LX) r = (r & ~63) | (r & 12) << 2 | (r & 48) >> 2 | (r & 3);
    const int edge = u < LX ? mlast : nlast;
    at[u] = (uint32_t)(r < edge ? r : edge) * (uint32_t)(u < LX ? a.x.pitch : a.w.pitch) + chunk * 16u;
  }
  const auto fill = [&](int step) __attribute__((always_inline)) {
    // chunks past a row's end read its last one; run() leaves them out
    const int most = chunks - 1 - step * 4;
    const int back = chunk > most ? (most - chunk) * 16 : 0;
    char* to = lds[(unsigned)step % kStages];
#pragma unroll
    for (int u = 0; u < LX + LW; ++u)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(u < LX ? xr : wr, (ZS_LDS(void)*)(to + (u * W + wave) * 1024), 16, at[u] + back,
                                               step * kStepK, 0, 0);
  };

  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, l4 = lane >> 4;
  const int place = (l4 ^ (-(l16 >> 2) & 3)) * 16;
  const int xrow = (wm * TM * 16 + l16) * kStepK + place, wrow = (BM + wn * TN * 16 + l16) * kStepK + place;
  i32x4 acc[TM][TN] = {};
  i32x4 xf[TM], wf[TN];
  // Step s: the step kStages - 1 ahead is requested into the place of the step before, which the other
  // waves have read.
  const auto run = [&](auto inner, int s) __attribute__((always_inline)) {
    constexpr bool kInner = decltype(inner)::value;  // kStages - 1 steps or more follow
    const char* from = lds[s % kStages];
    if (kInner || s + kStages - 1 < last) fill(s + kStages - 1);
#pragma unroll
    for (int j = 0; j < TN; ++j) wf[j] = *(const i32x4*)(from + wrow + j * 16 * kStepK);
#pragma unroll
    for (int i = 0; i < TM; ++i) xf[i] = *(const i32x4*)(from + xrow + i * 16 * kStepK);
    if (kInner) end_reading<(kStages - 2) * (LX + LW)>();  // the next step's loads are done
    else end_reading<0>();
    if (!kInner && chunks - s * 4 < 4) {  // the end of the rows
#pragma unroll
      for (int j = 0; j < TN; ++j)
        if (l4 >= chunks - s * 4) wf[j] = i32x4{0, 0, 0, 0};
    }
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[j], xf[i], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
    meet();
  };
  const bool behind = W == 8 && wave >= 4;
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k)
    if (first + k < last) fill(first + k);
  end_reading<0>();
  if (behind) meet();
  int s = first;
  for (; s + kStages - 1 < last; ++s) run(std::true_type(), s);
  for (; s < last; ++s) run(std::false_type(), s);
  if (W == 8 && !behind) meet();

  // a lane has, of row m0 + lane % 16 of each 16, the channels n to n + 15
  const int64_t n = n0 + wn * 64 + l4 * 16;
  if (n >= a.n) return;
  if (a.part) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int64_t m = m0 + wm * TM * 16 + i * 16 + l16;
      if (m >= a.m) continue;
      int32_t* to = a.part + ((int64_t)blockIdx.y * a.m + m) * a.n4 + n;
#pragma unroll
      for (int j = 0; j < TN; ++j)
        if (n + 4 * j < a.n) *(i32x4*)(to + 4 * j) = acc[i][j];
    }
    return;
  }
  const Channels<16> ch(a, n);
  with_type(a.y.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int64_t m = m0 + wm * TM * 16 + i * 16 + l16;
      if (m >= a.m) continue;
      const float xs = a.x.scale[m];
      float v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = ch(k, acc[i][k >> 2][k & 3], xs);
      store_run<DT, 16>((char*)a.y.p + m * a.y.pitch * esize(DT), n, a.n, v);
    }
  });
#endif
}

// A few tokens (16 MT at most), bound by the bytes of w: a block takes 16 channels, and its W waves every
// W-th run of 128 of k, whose integer sums they join.  Nothing goes through LDS before that: a
// lane's 32 bytes of a run are the operands of two instructions, whose k are numbered alike in x
// and w.  One token, 4096 x 11008: 10.5 us with the weights in the Infinity Cache, 12.6 with others
// between (3.6 TB/s); 64 tokens of 4096 x 4096 12 us, 65 in tiles 14.5.
template <int MT, int W>
__global__ void __launch_bounds__(W * 64) linear_few_kernel(LinearArgs a) {
  __shared__ i32x4 lds[W][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, l4 = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int chunks = (int)((a.k + 15) >> 4), runs = (chunks + 7) >> 3;
  const int8_t* w = a.w.q + (n0 + l16 < a.n ? n0 + l16 : a.n - 1) * a.w.pitch;
  const int8_t* x[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) x[i] = a.x.q + (i * 16 + l16 < a.m ? i * 16 + l16 : a.m - 1) * a.x.pitch;
  i32x4 acc[MT] = {};
  constexpr int U = 4 / MT;  // runs whose loads are under way at once
  const auto take = [&](auto whole, int r0) __attribute__((always_inline)) {
    constexpr bool kWhole = decltype(whole)::value;  // U runs, no end of the rows among them
    i32x4 wf[U][2], xf[U][2][MT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int c = (r0 + u * W) * 8 + l4 * 2 + h;
        if (!kWhole) c = c < chunks ? c : chunks - 1;
        wf[u][h] = *(const i32x4*)(w + c * 16);
#pragma unroll
        for (int i = 0; i < MT; ++i) xf[u][h][i] = *(const i32x4*)(x[i] + c * 16);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!kWhole && (r0 + u * W) * 8 + l4 * 2 + h >= chunks) wf[u][h] = i32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[u][h], xf[u][h][i], acc[i], 0, 0, 0);
      }
  };
  int r = wave;
  for (; (r + (U - 1) * W + 1) * 8 <= chunks; r += U * W) take(std::true_type(), r);
  for (; r < runs; r += U * W) take(std::false_type(), r);
#pragma unroll
  for (int i = 0; i < MT; ++i) lds[wave][i][lane] = acc[i];
  __syncthreads();
  if (wave >= MT) return;
  i32x4 sum = lds[0][wave][lane];
#pragma unroll
  for (int k = 1; k < W; ++k) sum += lds[k][wave][lane];
  const int64_t m = wave * 16 + l16, n = n0 + l4 * 4;
  if (m >= a.m || n >= a.n) return;
  const Channels<4> ch(a, n);
  const float xs = a.x.scale[m];
  float v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = ch(k, sum[k], xs);
  with_type(a.y.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    store_run<DT, 4>((char*)a.y.p + m * a.y.pitch * esize(DT), n, a.n, v);
  });
}

// Adds the splits' integer sums, which no order changes.
__global__ void __launch_bounds__(256) linear_join_kernel(LinearArgs a, int splits) {
  const int64_t quads = a.n4 / 4;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < a.m * quads; q += (int64_t)gridDim.x * 256) {
    const int64_t m = q / quads, n = q % quads * 4;
    i32x4 acc = {0, 0, 0, 0};
    for (int s = 0; s < splits; ++s) acc += *(const i32x4*)(a.part + ((int64_t)s * a.m + m) * a.n4 + n);
    const Channels<4> ch(a, n);
    const float xs = a.x.scale[m];
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = ch(k, acc[k], xs);
    with_type(a.y.dtype, [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      store_run<DT, 4>((char*)a.y.p + m * a.y.pitch * esize(DT), n, a.n, v);
    });
  }
}

// ---------------------------------------------------------------------------
// Gradients: c[i][j] = sum over s of a[s][i] (or a[i][s]) scale[s] q[s][j], 16x16x32 bf16 matrix
// instructions.  Tiles lie in LDS as [s][..] (or [i][s]); the instruction wants each lane's
// values along s, which the transposing LDS read gives.

constexpr int kStepS = 32;  // s of a tile step: one matrix instruction's

// How a comes into LDS.
enum Feed : int {
  kDirect = 0,  // bf16 as it is, loaded into LDS: rows and columns on 16-byte boundaries
  kPlain = 1,   // bf16 as it is, through registers, at any alignment
  kTerms = 2,   // fp16 as two bf16 terms, through registers
  kScaled = 3,  // times the scales (see Factors), as two bf16 terms, through registers
};

// A scale that is no power of two does not fit into a bf16 value beside q: a is multiplied by it.  Outside
// [2^-32, 2^32) only by its significand, in [1, 2), and q by the power of two that is left, exactly, so that
// neither leaves its type's range at either end of the scales'.  A step with none of these leaves q
// alone: q multiplied in every step takes 7% longer (8192 x 4096 x 11008: 1920 for 1760 us).
struct Factors {
  float a, q;
};
__device__ __forceinline__ bool ordinary(float scale) { return __float_as_uint(scale) - 0x2F800000u < 0x20000000u; }
__device__ __forceinline__ Factors factors(float scale) {
  if (ordinary(scale)) return {scale, 1.0f};
  const uint32_t b = __float_as_uint(scale);
  const float power = __uint_as_float(b & 0xFF800000u);
  return {__uint_as_float((b & 0x007FFFFFu) | 0x3F800000u), __builtin_isnan(scale) ? scale : power};
}

// Place of 16-element segment g of row s in a tile [s][...] is g ^ this: the rows that a transposing
// read takes together lie in different banks.
__device__ __forceinline__ int seg_swizzle(int s) { return (s & 3) | ((s >> 1) & 4); }

// Splits two values into two bf16 values each whose sum is theirs to 16 bits: exactly fp16's eleven, and
// within 2^-17 of itself a product with a scale.  A third term would bring that to the product's own
// 2^-24, for half as many matrix instructions again; 16-bit results would not show it.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
  // what is left of an infinity is one of its sign
  constexpr float kMost = 0x1.fffffep127f;
  const float ha = __builtin_amdgcn_fmed3f(dec_lo<ZERO_BF16>(hi), -kMost, kMost);
  const float hb = __builtin_amdgcn_fmed3f(dec_hi<ZERO_BF16>(hi), -kMost, kMost);
  lo = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a - ha, b - hb}), bf16x2));
}

// A block makes a tile of BI x BJ results with WI x WJ waves: 256 x 256 with eight, or 128 x 256 where a
// comes through registers, and 128 x 128 with four for small results.  The weight gradient of
// 8192 x 4096 x 11008 takes 653 us, 1.13e15 FLOP/s (1.20e15 at 8192 cubed), the input gradient of that
// size 587, 1.26e15, whose a needs no transposing reads; in two terms 2047 x 4096 x 4096 takes 140 us,
// 0.99e15 of both.  Bound by the matrix cores and, a third of the instructions beside theirs, the
// conversion of q: each block converts its 32 x BJ values of a step once, two 16-byte loads ahead.
// (Conversion spread between the products by scheduling groups: 923 for 857 us then.)
template <int DT, bool TRANS, int FEED, int BI, int BJ, int WI, int WJ>
__global__ void __launch_bounds__(WI* WJ * 64, 2) grad_kernel(GradArgs g, uint32_t tiles_i, uint32_t tiles_j, int64_t steps,
                                                             int64_t per_split) {
#ifdef __HIP_DEVICE_COMPILE__  // the host's compilation has no use for it, and stumbles over the builtins
  constexpr int W = WI * WJ, T = W * 64, S = kStepS;
  constexpr int TI = BI / WI / 16, TJ = BJ / WJ / 16;
  constexpr int LA = BI * S / 8 / T, LQ = BJ * S / 16 / T;  // 16-byte chunks of a thread
  constexpr int TERMS = FEED == kTerms || FEED == kScaled ? 2 : 1;
  constexpr int ABYTES = BI * S * 2;
  constexpr int kStages = FEED == kDirect ? 4 : 2;  // tile steps in LDS
  static_assert(BI * S / 8 % T == 0 && BJ * S / 16 % T == 0, "whole chunks");
  static_assert(TJ == 4, "a lane's results of a row are 16 consecutive ones");
  // Each step's place is a variable of its own, named at compile time: the compiler would have a
  // transposing read wait for every load into the variable that it reads from.
  __shared__ __attribute__((aligned(1024))) char a0[ABYTES * TERMS], a1[ABYTES * TERMS], a2[kStages > 2 ? ABYTES : 16],
      a3[kStages > 2 ? ABYTES : 16], q0[BJ * S * 2], q1[BJ * S * 2];
  const auto a_place = [&](auto k) __attribute__((always_inline)) {
    constexpr int K = decltype(k)::value % kStages;
    if constexpr (K == 0) return (char*)a0;
    else if constexpr (K == 1) return (char*)a1;
    else if constexpr (K == 2) return (char*)a2;
    else return (char*)a3;
  };
  const auto q_place = [&](auto k) __attribute__((always_inline)) {
    if constexpr (decltype(k)::value % 2 == 0) return (char*)q0;
    else return (char*)q1;
  };
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const Tile tile = tile_of(blockIdx.x, tiles_i, tiles_j);
  const int64_t i0 = tile.i * BI, j0 = tile.j * BJ;
  const int first = (int)(blockIdx.y * per_split), last = (int)(first + per_split < steps ? first + per_split : steps);

  // --- a, loaded into LDS: a wave's load fills 1024 bytes in the order of the lanes
  uint32_t at[LA];  // from the step's first element
  if constexpr (FEED == kDirect) {
#pragma unroll
    for (int u = 0; u < LA; ++u) {
      const int id = (u * W + wave) * 64 + lane;
      if constexpr (TRANS) {  // columns past the end read the last ones, and their results are not stored
        const int s = id / (BI / 8), c = id % (BI / 8) ^ (seg_swizzle(s) << 1);
        const int64_t i = i0 + c * 8 < g.ni ? c * 8 : g.ni - 8 - i0;
        at[u] = (uint32_t)s * (uint32_t)(g.a.pitch * 2) + (uint32_t)(i * 2);
      } else {  // rows likewise; the chunks' order is that of the linear layer's tiles
        const int i = id / 4, c = id % 4 ^ (-(i >> 2) & 3);
        at[u] = (uint32_t)(i0 + i < g.ni ? i : g.ni - 1 - i0) * (uint32_t)(g.a.pitch * 2) + c * 16u;
      }
    }
  }
  const auto fill = [&](auto inner, auto k, int step) __attribute__((always_inline)) {
    const int64_t s0 = (int64_t)step * S;
    const char* base = (const char*)g.a.p + (TRANS ? s0 * g.a.pitch + i0 : i0 * g.a.pitch + s0) * 2;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, 0xFFFFFFFFu, 0x00020000);
    // past the end of s the last row or chunk is read; run() leaves it out
    const int over = (int)(s0 + S - g.nc);
    char* to = a_place(k);
#pragma unroll
    for (int u = 0; u < LA; ++u) {
      uint32_t o = at[u];
      if (!decltype(inner)::value && over > 0) {
        const int id = (u * W + wave) * 64 + lane;
        if constexpr (TRANS) {
          const int s = id / (BI / 8), end = S - 1 - over;
          if (s > end) o -= (uint32_t)(s - end) * (uint32_t)(g.a.pitch * 2);
        } else {
          const int i = id / 4, c = id % 4 ^ (-(i >> 2) & 3), end = (S - over) / 8 - 1;
          if (c > end) o -= (uint32_t)(c - end) * 16u;
        }
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (ZS_LDS(void)*)(to + (u * W + wave) * 1024), 16, o, 0, 0, 0);
    }
  };

  // --- through registers: two steps' worth, loaded two steps before they are written to LDS
  struct Held {
    Raw8<ZERO_BF16> a[FEED == kDirect ? 1 : LA];
    float as[FEED == kScaled ? (TRANS ? LA : LA * 8) : 1];
    float row;  // kScaled: the scale of row lane % 32 of the step
    u32x4 q[LQ];
    float qs[LQ];
  } held[2];
  // Row and segment of 16 columns of a thread's chunks of q: four lanes take 64 columns, the next ones
  // the same of the three following rows, which they write to different banks.
  const auto q_row = [&](int u) __attribute__((always_inline)) { return (u * T + t) / (BJ / 4) * 4 + (t >> 2 & 3); };
  const auto q_seg = [&](int u) __attribute__((always_inline)) { return (u * T + t) % (BJ / 4) / 16 * 4 + (t & 3); };
  uint32_t qat[LQ];  // of the chunks, from the step's first byte; columns past the end read the first ones
#pragma unroll
  for (int u = 0; u < LQ; ++u) {
    const int c = q_seg(u) * 16;
    qat[u] = (uint32_t)q_row(u) * (uint32_t)g.q.pitch + (j0 + c < g.nj ? (uint32_t)c : 0u);
  }
  const bool whole = TRANS ? i0 + BI <= g.ni : i0 + BI <= g.ni && g.nc >= S;  // the tile's rows or columns of a
  const auto load = [&](auto inner, int step, Held& h) __attribute__((always_inline)) {
    constexpr bool kInner = decltype(inner)::value;  // not the last step
    const int64_t s0 = (int64_t)step * S;
    const int left = kInner || g.nc - s0 > S ? S : (int)(g.nc - s0);
    if constexpr (FEED != kDirect) {
      const char* base = (const char*)g.a.p + (TRANS ? s0 * g.a.pitch + i0 : i0 * g.a.pitch + s0) * 2;
      const int64_t cols = TRANS ? g.ni - i0 : left;
#pragma unroll
      for (int u = 0; u < LA; ++u) {
        const int id = u * T + t;
        const int r = TRANS ? id / (BI / 8) : id / (S / 8), c = (TRANS ? id % (BI / 8) : id % (S / 8)) * 8;
        const char* row = base + (int64_t)r * g.a.pitch * 2;
        if (whole && (kInner || left == S)) {
          h.a[u] = load_any<Raw8<ZERO_BF16>>(row + c * 2);
        } else {
          const bool in = TRANS ? r < left : i0 + r < g.ni;
          h.a[u] = load8<ZERO_BF16>(in ? row : base, c, in ? cols : 0);
        }
        if constexpr (FEED == kScaled) {
          if constexpr (TRANS) {
            h.as[u] = g.q.scale[s0 + (r < left ? r : left - 1)];
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) h.as[u * 8 + k] = g.q.scale[s0 + (c + k < left ? c + k : left - 1)];
          }
        }
      }
    }
    const char* base = (const char*)g.q.q + s0 * g.q.pitch + j0;
    const float* scale = g.q.scale + s0;
    if constexpr (FEED == kScaled) h.row = scale[(lane & (S - 1)) < left ? lane & (S - 1) : left - 1];
#pragma unroll
    for (int u = 0; u < LQ; ++u) {
      const int r = q_row(u);
      if (kInner) {
        h.q[u] = *(const u32x4*)(base + qat[u]);
        if constexpr (FEED != kScaled) h.qs[u] = scale[r];
      } else {  // rows past the end read the last one, and count nothing
        const int back = r < left ? 0 : r - left + 1;
        h.q[u] = *(const u32x4*)(base + (qat[u] - (uint32_t)back * (uint32_t)g.q.pitch));
        if (back) h.q[u] = u32x4{0, 0, 0, 0};
        if constexpr (FEED != kScaled) h.qs[u] = back ? 0.0f : scale[r];
      }
    }
  };
  const auto stage = [&](auto k, Held& h) __attribute__((always_inline)) {
    [[maybe_unused]] char* la = a_place(k);
    char* lq = q_place(k);
    [[maybe_unused]] bool split = false;  // the same for all threads of the block
    if constexpr (FEED == kScaled) {
      split = __builtin_amdgcn_ballot_w64(!ordinary(h.row)) != 0;
      if (split) {
#pragma unroll
        for (float& s : h.as) s = factors(s).a;
      }
    }
    if constexpr (FEED != kDirect) {
#pragma unroll
      for (int u = 0; u < LA; ++u) {
        const int id = u * T + t;
        int to;
        if constexpr (TRANS) {
          const int s = id / (BI / 8), c = id % (BI / 8);
          to = s * BI * 2 + ((c ^ (seg_swizzle(s) << 1)) << 4);
        } else {
          const int i = id / (S / 8), c = id % (S / 8);
          to = i * S * 2 + ((c ^ (-(i >> 2) & 3)) << 4);
        }
        if constexpr (TERMS == 2) {
          u32x4 hi, lo;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float a = dec_lo<DT>(h.a[u].v[0][k]), b = dec_hi<DT>(h.a[u].v[0][k]);
            if constexpr (FEED == kScaled) {  // with an addend the conversion from fp16 is part of the instruction
              a = __builtin_fmaf(a, h.as[TRANS ? u : u * 8 + 2 * k], 0.0f);
              b = __builtin_fmaf(b, h.as[TRANS ? u : u * 8 + 2 * k + 1], 0.0f);
            }
            uint32_t x, y;
            split2(a, b, x, y);
            hi[k] = x;
            lo[k] = y;
          }
          *(u32x4*)(la + to) = hi;
          *(u32x4*)(la + ABYTES + to) = lo;
        } else {
          *(u32x4*)(la + to) = h.a[u].v[0];
        }
      }
    }
    // Quads k of a segment of 16 columns go to the four segments of its 64: position 16 k + 4 c + e holds
    // column 16 c + 4 k + e, so that a lane's results, rows 4 (lane / 16) + 0..3 of a wave's four
    // products, are 16 columns in a row.
#pragma unroll
    for (int u = 0; u < LQ; ++u) {
      const int s = q_row(u), c = q_seg(u);
      const auto put = [&](auto scaled, float qs) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          u32x2 o;
          float v[4] = {q_of<0>(h.q[u][k]), q_of<1>(h.q[u][k]), q_of<2>(h.q[u][k]), q_of<3>(h.q[u][k])};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f32x2 w = {v[2 * e], v[2 * e + 1]};
            if constexpr (decltype(scaled)::value) w = f32x2{w.x * qs, w.y * qs};
            o[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(w, bf16x2));
          }
          *(u32x2*)(lq + s * BJ * 2 + ((((c & ~3) + k) ^ seg_swizzle(s)) << 5) + (c & 3) * 8) = o;
        }
      };
      asm volatile("" : "+v"(h.q[u]));  // not taken apart before: its bytes in a register each would wait for it
      if constexpr (FEED == kScaled) {
        if (split) put(std::true_type(), factors(__shfl(h.row, s)).q);
        else put(std::false_type(), 1.0f);
      } else {
        put(std::true_type(), h.qs[u]);
      }
    }
  };

  // --- products
  const int wi = wave / WJ, wj = wave % WJ;
  const int l16 = lane & 15, l4 = lane >> 4;
  // a transposing read takes, in each sixteen lanes, four rows of sixteen columns
  const int trow = l4 * 8 + (l16 >> 2), tcol = (l16 & 3) * 8, tswz = seg_swizzle(trow);
  f32x4 acc[TI][TJ] = {};
  bf16x8 fa[TERMS][TI], fq[TJ];
  constexpr int NA = TRANS ? (TI < 8 ? TI : 8) : 1;
  int a_at[NA], q_at[TJ];  // of a wave's segments
#pragma unroll
  for (int k = 0; k < NA; ++k) a_at[k] = trow * BI * 2 + (((wi * TI + k) ^ tswz) << 5) + tcol;
#pragma unroll
  for (int k = 0; k < TJ; ++k) q_at[k] = trow * BJ * 2 + (((wj * TJ + k) ^ tswz) << 5) + tcol;
  static_assert(TI <= 8, "one address for each");
  const int a_row = ((wi * TI) * 16 + l16) * S * 2 + ((l4 ^ (-(l16 >> 2) & 3)) << 4);
  const auto frag_t = [&](char* base, int at, int width) __attribute__((always_inline)) {
    ZS_LDS(char)* p = (ZS_LDS(char)*)base + at;
    const bf16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((ZS_LDS(bf16x4)*)p);
    const bf16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((ZS_LDS(bf16x4)*)(p + 4 * width * 2));
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  const auto fetch_q = [&](auto k, int j) __attribute__((always_inline)) { return frag_t(q_place(k), q_at[j], BJ); };
  const auto fetch_a = [&](auto k, int h, int i) __attribute__((always_inline)) {
    char* la = a_place(k) + h * ABYTES;
    if constexpr (TRANS) return frag_t(la, a_at[i], BI);
    else return *(const bf16x8*)(la + a_row + i * 16 * S * 2);
  };
  // Step s: the step three ahead is requested into the place of the step before, which the other waves
  // have read (a, loaded into LDS), and into registers (the rest); the step ahead, requested two steps
  // before, is converted into its place.
  const auto run = [&](auto inner, auto k, int s) __attribute__((always_inline)) {
    constexpr bool kInner = decltype(inner)::value;  // four steps or more follow
    constexpr int K = decltype(k)::value;            // s - first, modulo 4
    Held& h = held[(K + 1) % 2];
    if constexpr (FEED == kDirect) {
      if (kInner || s + 3 < last) fill(inner, std::integral_constant<int, (K + 3) % 4>(), s + 3);
      asm volatile("" ::: "memory");  // requested before load()'s: end_reading() below counts by that order
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) fq[j] = fetch_q(k, j);
#pragma unroll
    for (int h2 = 0; h2 < TERMS; ++h2)
#pragma unroll
      for (int i = 0; i < TI; ++i) fa[h2][i] = fetch_a(k, h2, i);
    if (kInner || s + 1 < last) stage(std::integral_constant<int, (K + 1) % 4>(), h);
    if (kInner || s + 3 < last) load(inner, s + 3, h);
    if constexpr (FEED == kDirect) {  // the next step's loads into LDS are done
      if (kInner) end_reading<2 * (LA + 2 * LQ) + 2 * LQ>();
      else end_reading<0>();
    } else {
      end_reading<63>();
    }
    if constexpr (FEED == kDirect) {
      if (!kInner && (int64_t)(s + 1) * S > g.nc) {  // rows of s past the end
        const int left = (int)(g.nc - (int64_t)s * S) - l4 * 8;
#pragma unroll
        for (int i = 0; i < TI; ++i) {
          u32x4 w = __builtin_bit_cast(u32x4, fa[0][i]);
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] &= left >= 2 * k + 2 ? 0xFFFFFFFFu : left == 2 * k + 1 ? 0xFFFFu : 0u;
          fa[0][i] = __builtin_bit_cast(bf16x8, w);
        }
      }
    }
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int h2 = 0; h2 < TERMS; ++h2)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[j], fa[h2][i], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
    meet();
  };
  const bool behind = W == 8 && wave >= 4;
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  using Any = std::false_type;
  using Inner = std::true_type;
  if constexpr (FEED == kDirect) {
    if (first < last) fill(Any(), I0(), first);
    if (first + 1 < last) fill(Any(), I1(), first + 1);
    if (first + 2 < last) fill(Any(), I2(), first + 2);
  }
  if (first < last) {
    load(Any(), first, held[0]);
    stage(I0(), held[0]);
  }
  if (first + 1 < last) load(Any(), first + 1, held[1]);
  if (first + 2 < last) load(Any(), first + 2, held[0]);
  end_reading<0>();
  if (behind) meet();
  int s = first;
  for (; s + 7 < last; s += 4) {
    run(Inner(), I0(), s);
    run(Inner(), I1(), s + 1);
    run(Inner(), I2(), s + 2);
    run(Inner(), I3(), s + 3);
  }
  for (; s < last; s += 4) {
    run(Any(), I0(), s);
    if (s + 1 < last) run(Any(), I1(), s + 1);
    if (s + 2 < last) run(Any(), I2(), s + 2);
    if (s + 3 < last) run(Any(), I3(), s + 3);
  }
  if (W == 8 && !behind) meet();

  // a lane has, of row lane % 16 of each 16, the columns c to c + 15
  const int64_t c = j0 + wj * 64 + l4 * 16;
  if (c >= g.nj) return;
  with_type(g.c.dtype, [&](auto dt) {
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int64_t r = i0 + (wi * TI + i) * 16 + l16;
      if (r >= g.ni) continue;
      if (g.part) {
        float* to = g.part + ((int64_t)blockIdx.y * g.ni + r) * g.nj4 + c;
#pragma unroll
        for (int j = 0; j < TJ; ++j)
          if (c + 4 * j < g.nj) *(f32x4*)(to + 4 * j) = acc[i][j];
        continue;
      }
      float v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = acc[i][k >> 2][k & 3];
      finish_run<decltype(dt)::value, 16>(g.c, r, c, g.nj, g.accumulate, v);
    }
  });
#endif
}

// Adds the splits' sums, in their order.
__global__ void __launch_bounds__(256) grad_join_kernel(GradArgs g, int splits) {
  const int64_t quads = g.nj4 / 4;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < g.ni * quads; q += (int64_t)gridDim.x * 256) {
    const int64_t r = q / quads, c = q % quads * 4;
    f32x4 acc = {0, 0, 0, 0};
    for (int s = 0; s < splits; ++s) acc += *(const f32x4*)(g.part + ((int64_t)s * g.ni + r) * g.nj4 + c);
    float v[4] = {acc[0], acc[1], acc[2], acc[3]};
    with_type(g.c.dtype, [&](auto dt) { finish_run<decltype(dt)::value, 4>(g.c, r, c, g.nj, g.accumulate, v); });
  }
}

// ---------------------------------------------------------------------------
// Column sums: a block takes 512 columns (eight to a lane) and a run of rows, its waves every fourth.  Bound
// by memory: 4096 x 6400 10 us, 5.3 TB/s, and 4 us to join.  It reads dy past the caches' order of use,
// which leaves them to the products around it: two weight gradients of that size 275 us, 286 with ordinary loads.

template <int DT>
__global__ void __launch_bounds__(256) columns_kernel(MatArg dy, int64_t m, int64_t n, int64_t run, float* part) {
  __shared__ float lds[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 512 + lane * 8;
  const int64_t r0 = (int64_t)blockIdx.y * run, r1 = r0 + run < m ? r0 + run : m;
  float s[8] = {};
  for (int64_t r = r0 + wave; r < r1; r += 4) {
    const Raw8<DT> x = load8<DT, true, true>((const char*)dy.p + r * dy.pitch * 2, c, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += get<DT>(x, i);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) lds[wave][lane * 8 + i] = s[i];
  __syncthreads();
  for (int k = threadIdx.x; k < 512; k += 256) {
    const int64_t col = (int64_t)blockIdx.x * 512 + k;
    if (col < n) part[(int64_t)blockIdx.y * n + col] = (lds[0][k] + lds[1][k]) + (lds[2][k] + lds[3][k]);
  }
}
// Joins the runs' sums: four waves take every fourth run of 64 columns, eight of them in flight.
__global__ void __launch_bounds__(256) columns_join_kernel(const float* part, int splits, int64_t n, MatArg db, int accumulate) {
  __shared__ float lds[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane, at = c < n ? c : n - 1;
  float s = 0.0f;
  int k = wave;
  for (; k + 28 < splits; k += 32) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = part[(int64_t)(k + 4 * u) * n + at];
#pragma unroll
    for (int u = 0; u < 8; ++u) s += v[u];
  }
  for (; k < splits; k += 4) s += part[(int64_t)k * n + at];
  lds[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= n) return;
  float v = (lds[0][lane] + lds[1][lane]) + (lds[2][lane] + lds[3][lane]);
  if (accumulate) v += load1(db, c);
  if (db.dtype == ZERO_F32) {
    ((float*)db.p)[c] = v;
    return;
  }
  float x[2] = {v, 0.0f};
  one_nan(x);
  ((uint16_t*)db.p)[c] = (uint16_t)(db.dtype == ZERO_BF16 ? enc2<ZERO_BF16>(x[0], 0.0f) : enc2<ZERO_F16>(x[0], 0.0f));
}

}  // namespace packed

using namespace packed;

static int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
static int64_t join_grid(int64_t quads) {
  const int64_t b = up(quads, 256);
  return b < 4096 ? b : 4096;
}

// Tiles of `bi` x `bj` and a contraction of `steps`: split until the chip's 256 compute units have a
// block each (of the small tiles two), but no finer than four steps to a split, and not beyond where
// what the splits write and the join reads takes longer than the steps saved: a step takes `step_us`
// and a split about 2 ps for each result, so the sum is least at the root of their ratio (the
// linear layer of 128 tokens, 4096 x 4096: 16 splits 30 us, 4 splits 18).
static ProductPlan plan_product(int64_t ni, int64_t nj, int64_t steps, int64_t bi, int64_t bj, double step_us) {
  ProductPlan p{};
  p.tile = (int32_t)bi;
  p.tiles_i = up(ni, bi);
  p.tiles_j = up(nj, bj);
  p.steps = steps;
  const int64_t tiles = p.tiles_i * p.tiles_j;
  int64_t s = tiles > 0 ? (bi == 128 ? 512 : 256) / tiles : 1;  // of the small tiles two at a time
  if (s > steps / 4) s = steps / 4;
  const int64_t least = (int64_t)std::sqrt(step_us * 5e5 * (double)steps / ((double)ni * (double)nj + 1.0));
  if (s > least) s = least;
  if (s < 1) s = 1;
  p.splits = up(steps > 0 ? steps : 1, up(steps > 0 ? steps : 1, s));
  p.ws_bytes = p.splits > 1 ? p.splits * ni * (up(nj, 4) * 4) * 4 : 0;
  return p;
}

constexpr int64_t kFewTokens = 64;  // the most that linear_few_kernel takes
constexpr double kBigStep = 0.4, kLinearStep = 0.35, kGradStep = 1.0;  // us of a step of large and of small tiles

ProductPlan plan_linear(int64_t m, int64_t k, int64_t n) {
  if (m <= kFewTokens) {
    ProductPlan few = plan_product(m, n, 1, kFewTokens, 16, kLinearStep);
    few.tile = 16;
    few.splits = 1;
    few.ws_bytes = 0;
    return few;
  }
  // 256 large tiles fill the chip.  k = 1600 and 8192 in bf16: 128 tiles' worth of results in large tiles 28
  // and 86 us, in small ones 24 and 83; 256 34 and 115, 45 and 160; 272 54 and 188, 52 and 191.  (From 144 to
  // 255 the large ones would be ahead too: 224 31 and 104, 41 and 150.)
  const ProductPlan p = plan_product(m, n, up(k, kStepK), 256, 256, kBigStep);
  return p.tiles_i * p.tiles_j >= 256 ? p : plan_product(m, n, up(k, kStepK), 128, 128, kLinearStep);
}

// Four waves to 16 channels fill the chip from 8192 channels on; fewer channels take more waves each.
template <int MT>
static void launch_linear_few(const LinearArgs& a, hipStream_t st) {
  const uint32_t grid = (uint32_t)up(a.n, 16);
  if (a.n >= 8192) linear_few_kernel<MT, 4><<<grid, 256, 0, st>>>(a);
  else if (a.n >= 2048) linear_few_kernel<MT, 8><<<grid, 512, 0, st>>>(a);
  else linear_few_kernel<MT, 16><<<grid, 1024, 0, st>>>(a);
}

hipError_t launch_linear(const LinearArgs& a, const ProductPlan& p, hipStream_t st) {
  if (p.tile == 16) {
    if (a.m <= 16) launch_linear_few<1>(a, st);
    else if (a.m <= 32) launch_linear_few<2>(a, st);
    else launch_linear_few<4>(a, st);
    return hipGetLastError();
  }
  const dim3 grid((uint32_t)(p.tiles_i * p.tiles_j), (uint32_t)p.splits);
  if (p.tile == 256) linear_kernel<256, 256, 2, 4, 4><<<grid, 512, 0, st>>>(a, (uint32_t)p.tiles_i, (uint32_t)p.tiles_j, p.steps, up(p.steps, p.splits));
  else linear_kernel<128, 128, 2, 2, 4><<<grid, 256, 0, st>>>(a, (uint32_t)p.tiles_i, (uint32_t)p.tiles_j, p.steps, up(p.steps, p.splits));
  if (a.part) linear_join_kernel<<<(uint32_t)join_grid(a.m * a.n4 / 4), 256, 0, st>>>(a, (int)p.splits);
  return hipGetLastError();
}

// a goes straight into LDS if its 16-byte chunks are whole and on their boundaries; 256 rows lie within
// 32-bit offsets.
static bool direct(const GradArgs& g, bool trans) {
  const int64_t along = trans ? g.ni : g.nc;
  return g.a.dtype == ZERO_BF16 && g.q.rule == ZERO_SCALE_POW2 && (uintptr_t)g.a.p % 16 == 0 && g.a.pitch % 8 == 0 &&
         along % 8 == 0 && along > 0 && g.a.pitch <= (int64_t)1 << 22;
}
// Large tiles from half of what the chip takes at once.  Weight gradients over 1600 and 8192 rows: 64 large
// tiles 59 and 111 us, as many results in small tiles 43 and 105; 128 62 and 153, 46 and 159; 256 73 and 246,
// 80 and 308; 512 135 and 477, 143 and 588.  (From 257 to about 320 tiles the second round of large ones is
// nearly empty, and the small ones would be ahead: 272 120 and 442, 90 and 349.)
ProductPlan plan_grad(int64_t ni, int64_t nj, int64_t nc) {
  const ProductPlan p = plan_product(ni, nj, up(nc, kStepS), 256, 256, kBigStep);
  return p.tiles_i * p.tiles_j >= 128 ? p : plan_product(ni, nj, up(nc, kStepS), 128, 128, kGradStep);
}

template <int DT, bool TRANS, int FEED>
static void launch_grad_typed(const GradArgs& g, const ProductPlan& p, hipStream_t st) {
  const dim3 grid((uint32_t)(p.tiles_i * p.tiles_j), (uint32_t)p.splits);
  const uint32_t ti = (uint32_t)p.tiles_i, tj = (uint32_t)p.tiles_j;
  if (p.tile != 256) {
    grad_kernel<DT, TRANS, FEED, 128, 128, 2, 2><<<grid, 256, 0, st>>>(g, ti, tj, p.steps, up(p.steps, p.splits));
  } else if constexpr (FEED != kDirect) {  // 128 rows, whose values also lie in registers on their way
    const uint32_t t2 = (uint32_t)up(g.ni, 128);
    grad_kernel<DT, TRANS, FEED, 128, 256, 2, 4><<<dim3(t2 * tj, grid.y), 512, 0, st>>>(g, t2, tj, p.steps, up(p.steps, p.splits));
  } else {
    grad_kernel<DT, TRANS, FEED, 256, 256, 2, 4><<<grid, 512, 0, st>>>(g, ti, tj, p.steps, up(p.steps, p.splits));
  }
}

hipError_t launch_grad(const GradArgs& g, bool trans, const ProductPlan& p, hipStream_t st) {
  if (g.a.dtype == ZERO_F16 && g.q.rule == ZERO_SCALE_POW2) {
    trans ? launch_grad_typed<ZERO_F16, true, kTerms>(g, p, st) : launch_grad_typed<ZERO_F16, false, kTerms>(g, p, st);
  } else if (g.a.dtype == ZERO_F16) {
    trans ? launch_grad_typed<ZERO_F16, true, kScaled>(g, p, st) : launch_grad_typed<ZERO_F16, false, kScaled>(g, p, st);
  } else if (g.q.rule != ZERO_SCALE_POW2) {
    trans ? launch_grad_typed<ZERO_BF16, true, kScaled>(g, p, st) : launch_grad_typed<ZERO_BF16, false, kScaled>(g, p, st);
  } else if (direct(g, trans)) {
    trans ? launch_grad_typed<ZERO_BF16, true, kDirect>(g, p, st) : launch_grad_typed<ZERO_BF16, false, kDirect>(g, p, st);
  } else {
    trans ? launch_grad_typed<ZERO_BF16, true, kPlain>(g, p, st) : launch_grad_typed<ZERO_BF16, false, kPlain>(g, p, st);
  }
  if (g.part) grad_join_kernel<<<(uint32_t)join_grid(g.ni * g.nj4 / 4), 256, 0, st>>>(g, (int)p.splits);
  return hipGetLastError();
}

ColumnsPlan plan_columns(int64_t m, int64_t n) {
  ColumnsPlan p;
  const int64_t wide = up(n > 0 ? n : 1, 512);
  int64_t s = up(1024, wide);
  if (s > up(m, 32)) s = up(m, 32);
  if (s < 1) s = 1;
  p.run = up(m > 0 ? m : 1, s);
  p.splits = up(m > 0 ? m : 1, p.run);
  p.ws_bytes = p.splits * n * 4;
  return p;
}

hipError_t launch_columns(const MatArg& dy, int64_t m, int64_t n, const MatArg& db, bool accumulate, float* part,
                          const ColumnsPlan& p, hipStream_t st) {
  const dim3 grid((uint32_t)up(n, 512), (uint32_t)p.splits);
  if (dy.dtype == ZERO_BF16) columns_kernel<ZERO_BF16><<<grid, 256, 0, st>>>(dy, m, n, p.run, part);
  else columns_kernel<ZERO_F16><<<grid, 256, 0, st>>>(dy, m, n, p.run, part);
  columns_join_kernel<<<(uint32_t)up(n, 64), 256, 0, st>>>(part, (int)p.splits, n, db, accumulate);
  return hipGetLastError();
}

}  // namespace zs
