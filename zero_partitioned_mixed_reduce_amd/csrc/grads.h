// Internal layout of the gradient-list operators, shared by the host plan and the kernels.
#pragma once
#include <stdint.h>

#include <string>
#include <vector>

#include "zero_grads.h"

namespace zs {

// Elements of a block's work item.
#ifndef ZS_GRADS_CHUNK
#define ZS_GRADS_CHUNK 8192
#endif
constexpr int kGradsChunk = ZS_GRADS_CHUNK;
static_assert(kGradsChunk % 8 == 0, "chunk starts keep a tensor's alignment");
// A tensor of at most this many elements is one work item of a single wave, so that a block of
// four waves takes four of them.
#ifndef ZS_GRADS_SMALL
#define ZS_GRADS_SMALL 1024
#endif
constexpr int kGradsSmall = ZS_GRADS_SMALL;
constexpr int kGradsBlock = 256;
constexpr int kGradsWaves = kGradsBlock / 64;
// Consecutive block items that a block of the norm kernel takes at most.
constexpr int kGradsRun = 4;
// Bytes from one arrival counter to the next.  An arrival is done by the memory, and while many
// of them meet in a few channels the reads of those channels wait: with counters 64 bytes apart
// in groups of 256 blocks the norm of 1.56e9 bf16 elements (without per-tensor norms, whose
// arrivals add 13 us) takes 498 us, with 256 bytes 467, in groups of 64 blocks 461 to 465; without
// any arrival the reads take 446.  512, 1024 and 4096 bytes measured the same as 256.
#ifndef ZS_GRADS_PITCH
#define ZS_GRADS_PITCH 256
#endif
constexpr int kGradsPitch = ZS_GRADS_PITCH;
static_assert(kGradsPitch % 64 == 0, "counters on lines of their own");
// Items of one tensor whose results a wave joins at once.
constexpr int kGradsJoin = 64;
// Results that one wave joins without their groups' (see join_level).
#ifndef ZS_GRADS_DIRECT
#define ZS_GRADS_DIRECT 1024
#endif
constexpr int kGradsDirect = ZS_GRADS_DIRECT;
// Limit of the blocks of work (each up to four blocks of a launch, whose limit is 2^32 - 1
// threads) and of the tensors.
constexpr int64_t kGradsMaxBlocks = (1 << 22) - 1;

// One work item: rows runs of cols elements.  The table holds the block items first, then the
// wave items, each in list order.
struct alignas(64) GradsChunk {
  uint64_t src, dst;              // addresses of the first element
  int64_t src_pitch, dst_pitch;   // bytes from row to row
  int32_t rows, cols;
  int32_t tensor;
  int16_t src_dtype, dst_dtype;
  int32_t first, count;           // the tensor's items: [first, first + count) of the table
  int32_t join;                   // index of the tensor's first counter and group result
  int16_t before, after;          // whether the item's run began before it, and how many of its elements
                                  // follow (at most 7): an item begins and ends on vector boundaries
                                  // inside a run, wherever the run itself begins
};
static_assert(sizeof(GradsChunk) == 64, "work item layout");

// An item's first element in its tensor, in bytes.
struct GradsOffset {
  int64_t src, dst;
};

// A tensor's items: [first, first + count) of the table.
struct GradsRange {
  int32_t first, count;
};

// What GradsScalars::have says of the results.
constexpr int32_t kGradsNorm = 1;       // acc and flag are those of the list's present values
constexpr int32_t kGradsPerTensor = 2;  // ... and tensor_acc with them

// Device-resident results (first 256 bytes of the workspace), and which of them a clip may use:
// only the device sees the replays of captured calls.
struct alignas(256) GradsScalars {
  double acc;        // sum of squares, or the largest magnitude
  int32_t flag;      // acc is not finite
  uint32_t counter;  // groups of blocks that have completed (re-armed by the last)
  float norm;        // in fp32; the one clipped by after a clip
  float coef;        // global coefficient of the last clip
  double clip_norm;  // global norm of the last clip
  int32_t clip_flag;
  int32_t have;      // kGradsNorm, kGradsPerTensor; 0 once the values have been written or bound anew
  int32_t kind;      // of the norm that ran last: zero_norm_t and inverse loss scale
  float inv;
  int32_t refused;   // the last clip found no norm that it could use, and wrote nothing
  int32_t clipped;   // a clip has left its norm here
};
static_assert(sizeof(GradsScalars) == 256, "scalar block");

// Where a tensor's results go: a destination of its own, itself because none was given, or
// itself as the destination given.
enum GradsInto : uint8_t { kInto = 0, kInPlace = 1, kInPlaceGiven = 2 };

struct GradsLayout {
  int64_t chunks, offsets, ranges, tensor_acc, norms, coefs, part, item_part, gcount, gpart, join_count, join_part, end;
};

struct GradsPlan {
  zero_grads_info_t info;
  std::vector<zero_grads_tensor_t> tensors;  // in-place destinations filled in, contiguous rows merged
  std::vector<uint8_t> in_place;             // kInto, kInPlace or kInPlaceGiven
  int64_t overlap;                           // a tensor with no destination that shares elements with another, or -1
  std::vector<GradsChunk> chunks;
  std::vector<GradsOffset> offsets;
  std::vector<GradsRange> ranges;
  int64_t n_block_items;  // the rest are wave items
  int64_t n_blocks;       // of one block item or kGradsWaves wave items each
  int64_t run;            // block items per block of the norm kernel
  int64_t norm_grid;      // blocks of the norm kernel
  int64_t group;          // blocks of the norm kernel whose results one group joins
  int64_t n_joins;        // counters of the tensors of several items
  int64_t bytes_in;       // of the sources
  int64_t n_empty;        // tensors without elements
  bool all16;             // every source and destination is 16-bit
  GradsLayout layout;
};

// Validates a list and sizes its work table.  ZERO_OK or ZERO_EINVAL with *err set.
zero_status_t build_grads_plan(const zero_grads_tensor_t* t, int64_t n, GradsPlan* out, std::string* err);
// Fills the work table of a validated plan (chunks, ranges).
void fill_grads_chunks(GradsPlan* p);
// Checks the addresses of a normalised list: null, misaligned or overlapping ones.  Tensors
// without a destination may repeat and overlap while only norms are taken; *overlap receives
// one of them, or -1.
zero_status_t check_grads_addresses(const std::vector<zero_grads_tensor_t>& t, const std::vector<uint8_t>& in_place,
                                    int64_t* overlap, std::string* err);

// Tensors whose new addresses one launch of the bind kernel carries (kernel arguments hold 4 KiB).
constexpr int kGradsBind = 240;
struct GradsBindArgs {
  GradsChunk* chunks;
  const GradsOffset* offsets;
  const GradsRange* ranges;
  GradsScalars* sc;
  int32_t first;  // index of the first tensor
  uint64_t src[kGradsBind], dst[kGradsBind];
};

struct GradsArgs {
  const GradsChunk* chunks;
  const GradsRange* ranges;
  GradsScalars* sc;
  double* tensor_acc;
  float* norms;
  float* coefs;          // of the last clip by each tensor's norm
  uint64_t* part;        // one per block of the norm kernel
  uint64_t* item_part;   // one per item
  uint32_t* gcount;      // one per group of blocks, kGradsPitch bytes apart
  uint64_t* gpart;       // one per group of blocks
  uint32_t* join_count;  // one per kGradsJoin items of a tensor, and one more per tensor of several; likewise
  uint64_t* join_part;   // beside them
  int64_t bytes_in;      // of the sources
  int32_t n_block_items, n_chunks, n_blocks, n_tensors, n_empty;
  int32_t run, group;
  int32_t all16;         // every source and destination is 16-bit
};

}  // namespace zs
