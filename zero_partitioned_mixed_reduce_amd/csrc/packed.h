// Internal layout of the packed-row operators, shared by their C ABI source and the kernels.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "zero_packed.h"

namespace zs {

// A matrix in floating point.
struct MatArg {
  void* p;
  int64_t pitch;  // elements
  int32_t dtype;
};

// Packed rows.
struct PackArg {
  int8_t* q;
  float* scale;
  int64_t pitch;
  int32_t rule;
};

// How a product is cut: tiles of bi x bj results, and the contraction into `splits` runs of
// `steps` tile steps, whose sums a second kernel joins.
struct ProductPlan {
  int64_t tiles_i, tiles_j;
  int64_t steps, splits;
  int64_t ws_bytes;
  int32_t tile;  // rows of a tile
};

// y [m][n] of x [m][k] and w [n][k].
struct LinearArgs {
  PackArg x, w;
  MatArg y, bias;  // bias.p null: none
  int64_t m, n, k;
  int32_t* part;   // splits > 1: integer sums [splits][m][n4]
  int64_t n4;      // n rounded up to a multiple of 4
};
ProductPlan plan_linear(int64_t m, int64_t k, int64_t n);
hipError_t launch_linear(const LinearArgs& a, const ProductPlan& p, hipStream_t st);

// c [ni][nj] of a, which is [nc][ni] (trans) or [ni][nc], and the packed rows q [nc][nj].
struct GradArgs {
  MatArg a, c;
  PackArg q;
  int64_t ni, nj, nc;
  int32_t accumulate;
  float* part;     // splits > 1: sums [splits][ni][nj4]
  int64_t nj4;
};
ProductPlan plan_grad(int64_t ni, int64_t nj, int64_t nc);
hipError_t launch_grad(const GradArgs& a, bool trans, const ProductPlan& p, hipStream_t st);

// db [n] of dy [m][n]: sums of runs of `run` rows, joined in order.
struct ColumnsPlan {
  int64_t run, splits;
  int64_t ws_bytes;
};
ColumnsPlan plan_columns(int64_t m, int64_t n);
hipError_t launch_columns(const MatArg& dy, int64_t m, int64_t n, const MatArg& db, bool accumulate, float* part,
                          const ColumnsPlan& p, hipStream_t st);

hipError_t launch_write(const MatArg& x, const PackArg& p, int64_t rows, int64_t cols, hipStream_t st);
hipError_t launch_read(const PackArg& p, const MatArg& out, int64_t rows, int64_t cols, hipStream_t st);
// xp.scale, y.p and yp.scale may be null: not asked for (a q without columns may be null as well)
hipError_t launch_act(int kind, bool gated, const MatArg& x, const PackArg& xp, const MatArg& y, const PackArg& yp,
                      int64_t m, int64_t n, hipStream_t st);
hipError_t launch_act_grad(int kind, bool gated, const PackArg& xp, const MatArg& dy, const MatArg& dx, int64_t m,
                           int64_t n, hipStream_t st);

}  // namespace zs
