// Host-side work table of the gradient-list operators.
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "grads.h"
#include "zs_internal.h"

namespace zs {

namespace {

constexpr int64_t kMaxElems = int64_t{1} << 60;

int64_t size_of(int32_t dtype) { return dtype == ZERO_F32 ? 4 : 2; }
// Lists of at least this many block items take them in runs (see the norm kernel).
#ifndef ZS_GRADS_RUN_FROM
#define ZS_GRADS_RUN_FROM 8192
#endif
constexpr int64_t kGradsRunFrom = ZS_GRADS_RUN_FROM;

bool known(int32_t dtype) { return dtype == ZERO_F16 || dtype == ZERO_BF16 || dtype == ZERO_F32; }

// Counters (and group results) that join the results of a tensor of `count` items: one per
// kGradsJoin of them, and one for the tensor where those are several.
int64_t joins_of(int64_t count) {
  if (count <= 1) return 0;
  const int64_t groups = (count + kGradsJoin - 1) / kGradsJoin;
  return groups + (groups > 1 ? 1 : 0);
}

zero_status_t bad(std::string* err, int64_t i, const char* what) {
  *err = "tensor " + std::to_string(i) + ": " + what;
  return ZERO_EINVAL;
}

// The bytes a strided tensor covers: `rows` runs of `width` bytes, `pitch` bytes apart.
struct Span {
  uint64_t begin, end;
  uint64_t width, pitch;
  int64_t rows;
  int64_t tensor;
  int written;  // 0: read only; 1: written in place if anything is; 2: a destination
};

Span span_of(const zero_grads_tensor_t& t, int64_t i, bool dst) {
  const int64_t es = size_of(dst ? t.dst_dtype : t.src_dtype);
  Span s;
  s.begin = (uint64_t)(uintptr_t)(dst ? t.dst : t.src);
  s.width = (uint64_t)(t.cols * es);
  s.rows = t.rows;
  s.pitch = t.rows > 1 ? (uint64_t)((dst ? t.dst_pitch : t.src_pitch) * es) : s.width;
  s.end = s.begin + s.pitch * (uint64_t)(t.rows - 1) + s.width;
  s.tensor = i;
  s.written = 0;
  return s;
}

// Whether two spans share a byte.  Two runs-of-rows with one pitch (or one of them a single
// row no longer than the other's pitch) are told apart by their columns; others that
// interleave are taken to overlap.
bool share(const Span& a, const Span& b) {
  if (a.end <= b.begin || b.end <= a.begin) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  if (a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) return true;
  const uint64_t p = a.rows > 1 ? a.pitch : b.pitch;
  const Span& lo = a.begin <= b.begin ? a : b;
  const Span& hi = a.begin <= b.begin ? b : a;
  const uint64_t off = (hi.begin - lo.begin) % p;  // the later one's column in the earlier one's rows
  return !(off >= lo.width && off + hi.width <= p);
}

}  // namespace

zero_status_t check_grads_addresses(const std::vector<zero_grads_tensor_t>& t, const std::vector<uint8_t>& in_place,
                                    int64_t* overlap, std::string* err) {
  *overlap = -1;
  const int64_t n = (int64_t)t.size();
  uint64_t src_lo = UINT64_MAX, src_hi = 0, dst_lo = UINT64_MAX, dst_hi = 0;
  bool ordered = true;
  bool any_dst = false, any_in_place = false;
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].rows * t[i].cols == 0) continue;
    if (!t[i].src) return bad(err, i, "null address of a non-empty tensor");
    if ((uintptr_t)t[i].src % (uintptr_t)size_of(t[i].src_dtype)) return bad(err, i, "source not aligned to its element size");
    const Span s = span_of(t[i], i, false);
    if (s.end < s.begin) return bad(err, i, "addresses wrap around");
    src_lo = std::min(src_lo, s.begin);
    src_hi = std::max(src_hi, s.end);
    if (in_place[i]) {
      any_in_place = true;
      continue;
    }
    if (!t[i].dst) return bad(err, i, "null destination of a non-empty tensor");
    if ((uintptr_t)t[i].dst % (uintptr_t)size_of(t[i].dst_dtype))
      return bad(err, i, "destination not aligned to its element size");
    const Span d = span_of(t[i], i, true);
    if (d.end < d.begin) return bad(err, i, "addresses wrap around");
    if (any_dst && d.begin < dst_hi) ordered = false;
    any_dst = true;
    dst_lo = std::min(dst_lo, d.begin);
    dst_hi = std::max(dst_hi, d.end);
  }
  // destinations in ascending order apart from every source, as in a flat buffer
  if (!any_in_place && ordered && (!any_dst || dst_hi <= src_lo || src_hi <= dst_lo)) return ZERO_OK;
  // Any order: sweep over all spans by address.
  std::vector<Span> all;
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].rows * t[i].cols == 0) continue;
    all.push_back(span_of(t[i], i, false));
    all.back().written = in_place[i];
    if (in_place[i]) continue;
    all.push_back(span_of(t[i], i, true));
    all.back().written = 2;
  }
  std::sort(all.begin(), all.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
  // The spans that reach beyond the present one's begin, read and written ones apart: two that
  // are only read are not compared.  Once tensors without a destination have been found to
  // overlap, they count as read, and only destinations are looked for.
  std::vector<Span> open[2];
  for (const Span& s : all) {
    for (int w = s.written && !(s.written == 1 && *overlap >= 0) ? 0 : 1; w < 2; ++w) {
      size_t keep = 0;
      for (const Span& o : open[w]) {
        if (o.end <= s.begin) continue;
        if (share(o, s)) {
          const Span& d = s.written > o.written ? s : o;
          if (d.written == 2) return bad(err, d.tensor, "destination overlaps a source or another destination");
          *overlap = d.tensor;
        }
        open[w][keep++] = o;
      }
      open[w].resize(keep);
    }
    if (*overlap >= 0 && !open[1].empty()) {
      auto given = std::stable_partition(open[1].begin(), open[1].end(), [](const Span& o) { return o.written == 2; });
      open[0].insert(open[0].end(), given, open[1].end());
      open[1].erase(given, open[1].end());
    }
    open[s.written == 2 || (s.written == 1 && *overlap < 0)].push_back(s);
  }
  return ZERO_OK;
}

zero_status_t build_grads_plan(const zero_grads_tensor_t* tensors, int64_t n, GradsPlan* out, std::string* err) {
  if (!tensors || !out) {
    *err = "null list or output";
    return ZERO_EINVAL;
  }
  if (n < 1 || n > kGradsMaxBlocks) {
    *err = "need 1 <= n <= 2^22 - 1 tensors";
    return ZERO_EINVAL;
  }
  GradsPlan p;
  p.tensors.assign(tensors, tensors + n);
  p.in_place.resize((size_t)n);
  memset(&p.info, 0, sizeof(p.info));
  p.bytes_in = p.n_empty = 0;
  p.all16 = true;
  for (int64_t i = 0; i < n; ++i) {
    zero_grads_tensor_t& t = p.tensors[i];
    if (!known(t.src_dtype)) return bad(err, i, "src_dtype must be ZERO_F16, ZERO_BF16 or ZERO_F32");
    if (t.rows < 0 || t.cols < 0) return bad(err, i, "rows and cols must be >= 0");
    if (t.rows > 0 && t.cols > (kMaxElems - p.info.elems) / t.rows) {
      *err = "the list exceeds 2^60 elements";
      return ZERO_EINVAL;
    }
    const int64_t len = t.rows * t.cols;
    p.info.elems += len;
    if (t.rows > 1 && len > 0 && (t.src_pitch < t.cols || t.src_pitch > kMaxElems / t.rows))
      return bad(err, i, "src_pitch must be at least cols, and the tensor's span at most 2^60 elements");
    // a destination that is the source itself is in place
    const bool same = t.dst == t.src && t.dst_dtype == t.src_dtype && (t.rows <= 1 || t.dst_pitch == t.src_pitch);
    p.in_place[i] = !t.dst ? kInPlace : same ? kInPlaceGiven : kInto;
    if (p.in_place[i]) {
      t.dst = t.src;
      t.dst_dtype = t.src_dtype;
      t.dst_pitch = t.src_pitch;
    }
    if (!known(t.dst_dtype)) return bad(err, i, "dst_dtype must be ZERO_F16, ZERO_BF16 or ZERO_F32");
    if (t.rows > 1 && len > 0 && (t.dst_pitch < t.cols || t.dst_pitch > kMaxElems / t.rows))
      return bad(err, i, "dst_pitch must be at least cols, and the tensor's span at most 2^60 elements");
    if (len == 0) {
      ++p.n_empty;
      t.rows = 1;
      t.cols = 0;
    }
    if (t.rows == 1 || (t.src_pitch == t.cols && t.dst_pitch == t.cols)) {
      t.cols = len;
      t.rows = 1;
      t.src_pitch = t.dst_pitch = len;
    }
    p.bytes_in += len * size_of(t.src_dtype);
    p.all16 = p.all16 && (len == 0 || (t.src_dtype != ZERO_F32 && t.dst_dtype != ZERO_F32));
  }
  zero_status_t s = check_grads_addresses(p.tensors, p.in_place, &p.overlap, err);
  if (s != ZERO_OK) return s;

  // work items of a tensor: whole rows while one fits a block's item, else parts of a row
  auto count_of = [](const zero_grads_tensor_t& t) -> int64_t {
    if (t.rows * t.cols == 0) return 0;
    if (t.rows * t.cols <= kGradsSmall) return 1;
    if (t.cols >= kGradsChunk) return t.rows * ((t.cols + kGradsChunk - 1) / kGradsChunk);
    const int64_t per = kGradsChunk / t.cols;
    return (t.rows + per - 1) / per;
  };
  auto is_small = [](const zero_grads_tensor_t& t) { return t.rows * t.cols <= kGradsSmall; };
  int64_t n_block = 0, n_wave = 0;
  p.n_joins = 0;
  for (const auto& t : p.tensors) {
    const int64_t c = count_of(t);
    if (c > kGradsMaxBlocks || n_block > kGradsMaxBlocks) {
      *err = "the list needs more than 2^22 - 1 blocks of work";
      return ZERO_EINVAL;
    }
    (is_small(t) ? n_wave : n_block) += c;
    p.n_joins += joins_of(c);
  }
  const int64_t n_wave_blocks = (n_wave + kGradsWaves - 1) / kGradsWaves;
  const int64_t n_blocks = n_block + n_wave_blocks;
  if (n_blocks > kGradsMaxBlocks) {
    *err = "the list needs more than 2^22 - 1 blocks of work";
    return ZERO_EINVAL;
  }
  p.n_block_items = n_block;
  p.n_blocks = n_blocks;
  p.run = n_block >= kGradsRunFrom ? kGradsRun : 1;
  p.norm_grid = (n_block + p.run - 1) / p.run + n_wave_blocks;
  // Groups of about the square root of the blocks, at most 64: every arrival on one counter
  // takes about 10 ns, so groups of 256 made the norm of 4.2e6 bf16 elements (512 blocks) 9.1 us,
  // groups of 64 6.7.  1.56e9 elements (without per-tensor norms) take 467 us in groups of 256,
  // 461 of 64, 506 of 16, whose own arrivals crowd the top.  Up to 128 blocks one group is as fast as a second level.
  p.group = 128;
  if (p.norm_grid > 128)
    for (p.group = 16; p.group < 64 && p.group * p.group < p.norm_grid;) p.group *= 2;
  const int64_t n_groups = (p.norm_grid + p.group - 1) / p.group;
  p.info.num_chunks = n_block + n_wave;
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  GradsLayout& l = p.layout;
  l.chunks = sizeof(GradsScalars);
  l.offsets = up(l.chunks + p.info.num_chunks * (int64_t)sizeof(GradsChunk));
  l.ranges = up(l.offsets + p.info.num_chunks * (int64_t)sizeof(GradsOffset));
  l.tensor_acc = up(l.ranges + n * (int64_t)sizeof(GradsRange));
  l.norms = up(l.tensor_acc + 8 * n);
  l.coefs = up(l.norms + 4 * n);
  l.part = up(l.coefs + 4 * n);
  l.item_part = up(l.part + 8 * p.norm_grid);
  l.gpart = up(l.item_part + 8 * p.info.num_chunks);
  l.join_part = up(l.gpart + 8 * n_groups);
  l.gcount = up(l.join_part + 8 * p.n_joins);
  l.join_count = up(l.gcount + kGradsPitch * n_groups);
  l.end = up(l.join_count + kGradsPitch * p.n_joins);
  p.info.workspace_bytes = l.end;
  *out = std::move(p);
  return ZERO_OK;
}

void fill_grads_chunks(GradsPlan* p) {
  const int64_t n = (int64_t)p->tensors.size();
  p->chunks.resize((size_t)p->info.num_chunks);
  p->offsets.resize((size_t)p->info.num_chunks);
  p->ranges.resize((size_t)n);
  int64_t at[2] = {0, p->n_block_items};  // next block item, next wave item
  int64_t join = 0;
  for (int64_t i = 0; i < n; ++i) {
    const zero_grads_tensor_t& t = p->tensors[i];
    const int64_t len = t.rows * t.cols;
    const int64_t ss = size_of(t.src_dtype), ds = size_of(t.dst_dtype);
    int64_t& next = at[len <= kGradsSmall ? 1 : 0];
    const int64_t first = next;
    auto add = [&](int64_t r, int64_t c, int64_t rows, int64_t cols) {
      GradsOffset& o = p->offsets[(size_t)next];
      GradsChunk& k = p->chunks[(size_t)next++];
      o.src = (r * t.src_pitch + c) * ss;
      o.dst = (r * t.dst_pitch + c) * ds;
      k.src = (uint64_t)(uintptr_t)t.src + (uint64_t)o.src;
      k.dst = (uint64_t)(uintptr_t)t.dst + (uint64_t)o.dst;
      k.src_pitch = t.src_pitch * ss;
      k.dst_pitch = t.dst_pitch * ds;
      k.rows = (int32_t)rows;
      k.cols = (int32_t)cols;
      k.tensor = (int32_t)i;
      k.src_dtype = (int16_t)t.src_dtype;
      k.dst_dtype = (int16_t)t.dst_dtype;
      k.first = (int32_t)first;
      k.join = (int32_t)join;
      k.before = c > 0;
      k.after = (int16_t)std::min<int64_t>(7, t.cols - (c + cols));
    };
    if (len == 0) {
    } else if (len <= kGradsSmall) {
      add(0, 0, t.rows, t.cols);
    } else if (t.cols >= kGradsChunk) {
      for (int64_t r = 0; r < t.rows; ++r)
        for (int64_t c = 0; c < t.cols; c += kGradsChunk) add(r, c, 1, std::min<int64_t>(kGradsChunk, t.cols - c));
    } else {
      const int64_t per = kGradsChunk / t.cols;
      for (int64_t r = 0; r < t.rows; r += per) add(r, 0, std::min(per, t.rows - r), t.cols);
    }
    const int64_t count = next - first;
    for (int64_t c = first; c < next; ++c) p->chunks[(size_t)c].count = (int32_t)count;
    p->ranges[i] = GradsRange{(int32_t)first, (int32_t)count};
    join += joins_of(count);
  }
}

}  // namespace zs
