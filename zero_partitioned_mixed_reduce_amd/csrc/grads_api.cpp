// C ABI of the gradient-list operators.  Host side: argument checks, the order of calls and
// kernel launches.  The plan is in grads_plan.cpp, the arithmetic in grads.hip.
#include <hip/hip_runtime.h>

#include <cmath>
#include <exception>
#include <new>
#include <string>
#include <utility>

#include "grads.h"
#include "zero_grads.h"
#include "zs_host.h"

struct zero_grads {
  zs::GradsPlan plan;
  zs::GradsArgs args;
  int device;
  // Norms that a clip may find on the device (kGradsNorm, kGradsPerTensor).  What is captured runs
  // when its graph is replayed, unseen here: the device knows what has run (GradsScalars::have),
  // and the host refuses only what no replay can have made right.
  int32_t have;        // of the calls that were not captured
  int32_t graph_have;  // of all captured norms
  // Any captured call may meet any list that is bound later, and any later call a list bound in a graph.
  bool graph_writes;      // a call that writes has been captured
  int64_t graph_overlap;  // of lists bound in captures: as GradsPlan::overlap
};

namespace {

using zs::DeviceGuard;
using zs::set_error;

zero_status_t fail(zero_status_t s, const std::string& msg) { return set_error(s, msg); }
zero_status_t hip_fail(const char* what, hipError_t e) {
  return set_error(ZERO_EHIP, std::string(what) + ": " + hipGetErrorString(e));
}

// A stream that cannot tell is not captured: its calls fail by themselves.
bool capturing(hipStream_t st) {
  hipStreamCaptureStatus s = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(st, &s) != hipSuccess) {
    (void)hipGetLastError();
    return false;
  }
  return s != hipStreamCaptureStatusNone;
}

zero_status_t init(const zero_grads_tensor_t* tensors, int64_t n, void* workspace, int64_t workspace_capacity,
                   void* stream, zero_grads_t* out) {
  if (!out) return fail(ZERO_EINVAL, "null output handle");
  *out = nullptr;
  zs::GradsPlan p;
  std::string err;
  zero_status_t s = zs::build_grads_plan(tensors, n, &p, &err);
  if (s != ZERO_OK) return fail(s, err);
  if (!workspace) return fail(ZERO_EINVAL, "workspace must be non-null");
  if (((uintptr_t)workspace & 255u) != 0) return fail(ZERO_EINVAL, "workspace must be 256-byte aligned");
  if (workspace_capacity < p.info.workspace_bytes)
    return fail(ZERO_EINVAL, "workspace_capacity " + std::to_string(workspace_capacity) + " < workspace_bytes " +
                                 std::to_string(p.info.workspace_bytes));
  zs::fill_grads_chunks(&p);
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail("hipGetDevice", e);
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  zs::GradsArgs a;
  a.chunks = reinterpret_cast<zs::GradsChunk*>(ws + p.layout.chunks);
  a.ranges = reinterpret_cast<zs::GradsRange*>(ws + p.layout.ranges);
  a.sc = reinterpret_cast<zs::GradsScalars*>(ws);
  a.tensor_acc = reinterpret_cast<double*>(ws + p.layout.tensor_acc);
  a.norms = reinterpret_cast<float*>(ws + p.layout.norms);
  a.coefs = reinterpret_cast<float*>(ws + p.layout.coefs);
  a.part = reinterpret_cast<uint64_t*>(ws + p.layout.part);
  a.item_part = reinterpret_cast<uint64_t*>(ws + p.layout.item_part);
  a.gcount = reinterpret_cast<uint32_t*>(ws + p.layout.gcount);
  a.gpart = reinterpret_cast<uint64_t*>(ws + p.layout.gpart);
  a.join_count = reinterpret_cast<uint32_t*>(ws + p.layout.join_count);
  a.join_part = reinterpret_cast<uint64_t*>(ws + p.layout.join_part);
  a.bytes_in = p.bytes_in;
  a.n_block_items = (int32_t)p.n_block_items;
  a.n_chunks = (int32_t)p.info.num_chunks;
  a.n_blocks = (int32_t)p.n_blocks;
  a.n_tensors = (int32_t)n;
  a.n_empty = (int32_t)p.n_empty;
  a.run = (int32_t)p.run;
  a.group = (int32_t)p.group;
  a.all16 = p.all16;
  const zs::GradsScalars sc = {};
  zero_status_t rs = ZERO_OK;
  if ((e = hipMemcpyAsync(a.sc, &sc, sizeof(sc), hipMemcpyHostToDevice, st)) != hipSuccess)
    rs = hip_fail("hipMemcpyAsync(scalars)", e);
  else if (!p.chunks.empty() &&
           ((e = hipMemcpyAsync(ws + p.layout.chunks, p.chunks.data(), p.chunks.size() * sizeof(zs::GradsChunk),
                                hipMemcpyHostToDevice, st)) != hipSuccess ||
            (e = hipMemcpyAsync(ws + p.layout.offsets, p.offsets.data(), p.offsets.size() * sizeof(zs::GradsOffset),
                                hipMemcpyHostToDevice, st)) != hipSuccess))
    rs = hip_fail("hipMemcpyAsync(work table)", e);
  else if ((e = hipMemcpyAsync(ws + p.layout.ranges, p.ranges.data(), p.ranges.size() * sizeof(zs::GradsRange),
                               hipMemcpyHostToDevice, st)) != hipSuccess)
    rs = hip_fail("hipMemcpyAsync(tensor table)", e);
  // the counters start at zero (and are re-armed by every pass), the tensors' results until a first pass too
  else if ((e = zs::launch_fill_zero(reinterpret_cast<float*>(a.tensor_acc),
                                     (p.layout.part - p.layout.tensor_acc) / (int64_t)sizeof(float), st)) != hipSuccess ||
           (e = zs::launch_fill_zero(reinterpret_cast<float*>(a.gcount),
                                     (p.layout.end - p.layout.gcount) / (int64_t)sizeof(float), st)) != hipSuccess)
    rs = hip_fail("workspace fill", e);
  // copies already enqueued read the plan's tables
  e = hipStreamSynchronize(st);
  if (rs != ZERO_OK) return rs;
  if (e != hipSuccess) return hip_fail("hipStreamSynchronize(init)", e);
  p.chunks = std::vector<zs::GradsChunk>();
  p.offsets = std::vector<zs::GradsOffset>();
  p.ranges = std::vector<zs::GradsRange>();
  zero_grads* h = new (std::nothrow) zero_grads();
  if (!h) return fail(ZERO_ENOMEM, "out of host memory");
  h->plan = std::move(p);
  h->args = a;
  h->device = dev;
  h->have = h->graph_have = 0;
  h->graph_writes = false;
  h->graph_overlap = -1;
  *out = h;
  return ZERO_OK;
}

zero_status_t bind(zero_grads_t h, void* const* src, void* const* dst, hipStream_t st) {
  std::vector<zero_grads_tensor_t> t = h->plan.tensors;
  const int64_t n = (int64_t)t.size();
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].rows * t[i].cols == 0) continue;  // has no address
    t[i].src = src[i];
    if (h->plan.in_place[i]) {
      if (dst && dst[i] && dst[i] != src[i])
        return fail(ZERO_EINVAL, "tensor " + std::to_string(i) + ": planned in place, bound to another destination");
      t[i].dst = src[i];
    } else {
      if (!dst) return fail(ZERO_EINVAL, "tensor " + std::to_string(i) + ": planned with a destination, bound without");
      t[i].dst = dst[i];
    }
  }
  std::string err;
  int64_t overlap;
  zero_status_t s = zs::check_grads_addresses(t, h->plan.in_place, &overlap, &err);
  if (s != ZERO_OK) return fail(s, err);
  if (overlap >= 0 && h->graph_writes)
    return fail(ZERO_EINVAL, "tensor " + std::to_string(overlap) +
                                 ": shares elements with another tensor of the list, and a captured call writes in place");
  DeviceGuard dg(h->device);
  const bool graph = capturing(st);
  if (!graph) h->have = 0;
  zs::GradsBindArgs a;
  a.chunks = const_cast<zs::GradsChunk*>(h->args.chunks);
  a.offsets = reinterpret_cast<zs::GradsOffset*>(reinterpret_cast<char*>(h->args.sc) + h->plan.layout.offsets);
  a.ranges = h->args.ranges;
  a.sc = h->args.sc;
  for (int64_t i = 0; i < n; i += zs::kGradsBind) {
    const int m = (int)(n - i < zs::kGradsBind ? n - i : zs::kGradsBind);
    a.first = (int32_t)i;
    for (int k = 0; k < m; ++k) {
      a.src[k] = (uint64_t)(uintptr_t)t[i + k].src;
      a.dst[k] = (uint64_t)(uintptr_t)t[i + k].dst;
    }
    hipError_t e = zs::launch_grads_bind(a, m, st);
    if (e != hipSuccess) return hip_fail("bind kernel", e);
  }
  if (!graph)
    h->plan.overlap = overlap;
  else if (overlap >= 0)
    h->graph_overlap = overlap;
  return ZERO_OK;
}

// A call that writes the list's values has been enqueued: the norm is not theirs any more.
void written(zero_grads_t h, void* stream) {
  if (capturing(static_cast<hipStream_t>(stream))) h->graph_writes = true;
  else h->have = 0;
}

// Calls that write refuse a list in which tensors without a destination overlap.
zero_status_t check_writable(const zero_grads* h) {
  const int64_t overlap = h->plan.overlap >= 0 ? h->plan.overlap : h->graph_overlap;
  if (overlap < 0) return ZERO_OK;
  return fail(ZERO_EINVAL, "tensor " + std::to_string(overlap) +
                               ": shares elements with another tensor of the list, and would be written in place");
}

zero_status_t check_norm(zero_grads_t h, int32_t norm, float inv) {
  if (!h) return fail(ZERO_EINVAL, "null handle");
  if (norm != ZERO_NORM_L2 && norm != ZERO_NORM_MAX) return fail(ZERO_EINVAL, "norm must be ZERO_NORM_L2 or ZERO_NORM_MAX");
  if (!(inv > 0.0f) || !std::isfinite(inv)) return fail(ZERO_EINVAL, "inv_loss_scale must be finite and positive");
  return ZERO_OK;
}
zero_status_t check_clip(int32_t scope, float max_norm) {
  if (scope != ZERO_CLIP_GLOBAL && scope != ZERO_CLIP_EACH)
    return fail(ZERO_EINVAL, "scope must be ZERO_CLIP_GLOBAL or ZERO_CLIP_EACH");
  if (std::isnan(max_norm)) return fail(ZERO_EINVAL, "max_norm is NaN");
  return ZERO_OK;
}

}  // namespace

extern "C" {

// The plan's host tables may not fit in host memory: no exception leaves the C ABI.
zero_status_t zero_grads_plan(const zero_grads_tensor_t* tensors, int64_t n, zero_grads_info_t* out) {
  try {
    if (!out) return fail(ZERO_EINVAL, "null output");
    zs::GradsPlan p;
    std::string err;
    zero_status_t s = zs::build_grads_plan(tensors, n, &p, &err);
    if (s != ZERO_OK) return fail(s, err);
    *out = p.info;
    return ZERO_OK;
  } catch (const std::exception& e) {
    return fail(ZERO_ENOMEM, std::string("host resources: ") + e.what());
  }
}

zero_status_t zero_grads_init(const zero_grads_tensor_t* tensors, int64_t n, void* workspace,
                              int64_t workspace_capacity, void* stream, zero_grads_t* out) {
  try {
    return init(tensors, n, workspace, workspace_capacity, stream, out);
  } catch (const std::exception& e) {
    return fail(ZERO_ENOMEM, std::string("host resources: ") + e.what());
  }
}

zero_status_t zero_grads_info(zero_grads_t h, zero_grads_info_t* out) {
  if (!h || !out) return fail(ZERO_EINVAL, "null handle or output");
  *out = h->plan.info;
  return ZERO_OK;
}

zero_status_t zero_grads_bind(zero_grads_t h, void* const* src, void* const* dst, void* stream) {
  if (!h || !src) return fail(ZERO_EINVAL, "null handle or addresses");
  try {
    return bind(h, src, dst, static_cast<hipStream_t>(stream));
  } catch (const std::exception& e) {
    return fail(ZERO_ENOMEM, std::string("host resources: ") + e.what());
  }
}

zero_status_t zero_grads_norm(zero_grads_t h, int32_t norm, float inv_loss_scale, int32_t per_tensor, void* stream) {
  zero_status_t s = check_norm(h, norm, inv_loss_scale);
  if (s != ZERO_OK) return s;
  DeviceGuard dg(h->device);
  hipError_t e = zs::launch_grads_norm(h->args, norm, inv_loss_scale, per_tensor != 0, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("norm kernel", e);
  const int32_t have = per_tensor ? zs::kGradsNorm | zs::kGradsPerTensor : zs::kGradsNorm;
  if (capturing(static_cast<hipStream_t>(stream))) h->graph_have |= have;
  else h->have = have;
  return ZERO_OK;
}

zero_status_t zero_grads_device(zero_grads_t h, double** acc, int32_t** found_inf, float** norm, double** tensor_acc,
                                float** norms) {
  if (!h) return fail(ZERO_EINVAL, "null handle");
  if (acc) *acc = &h->args.sc->acc;
  if (found_inf) *found_inf = &h->args.sc->flag;
  if (norm) *norm = &h->args.sc->norm;
  if (tensor_acc) *tensor_acc = h->args.tensor_acc;
  if (norms) *norms = h->args.norms;
  return ZERO_OK;
}

zero_status_t zero_grads_clip(zero_grads_t h, int32_t scope, int32_t other_ranks_found_inf, double other_ranks_acc,
                              float max_norm, void* stream) {
  if (!h) return fail(ZERO_EINVAL, "null handle");
  zero_status_t s = check_clip(scope, max_norm);
  if (s != ZERO_OK) return s;
  if ((s = check_writable(h)) != ZERO_OK) return s;
  if (other_ranks_acc < 0.0) return fail(ZERO_EINVAL, "other_ranks_acc must not be negative");
  const int32_t have = h->have | h->graph_have;
  if (!have) return fail(ZERO_ESTATE, "zero_grads_clip must follow zero_grads_norm of the same values");
  if (scope == ZERO_CLIP_EACH && !(have & zs::kGradsPerTensor))
    return fail(ZERO_ESTATE, "ZERO_CLIP_EACH needs a zero_grads_norm with per_tensor");
  DeviceGuard dg(h->device);
  hipError_t e = zs::launch_grads_clip(h->args, scope, other_ranks_found_inf != 0, other_ranks_acc, max_norm,
                                       static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("clip kernel", e);
  written(h, stream);
  return ZERO_OK;
}

zero_status_t zero_grads_clip_norm(zero_grads_t h, int32_t norm, float inv_loss_scale, int32_t per_tensor,
                                   int32_t scope, float max_norm, void* stream) {
  zero_status_t s = check_norm(h, norm, inv_loss_scale);
  if (s == ZERO_OK) s = check_clip(scope, max_norm);
  if (s == ZERO_OK) s = check_writable(h);
  if (s != ZERO_OK) return s;
  DeviceGuard dg(h->device);
  hipError_t e = zs::launch_grads_clip_norm(h->args, norm, inv_loss_scale, per_tensor != 0 || scope == ZERO_CLIP_EACH,
                                            scope, max_norm, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("norm and clip kernels", e);
  written(h, stream);
  return ZERO_OK;
}

zero_status_t zero_grads_scale(zero_grads_t h, float factor, void* stream) {
  if (!h) return fail(ZERO_EINVAL, "null handle");
  if (!std::isfinite(factor)) return fail(ZERO_EINVAL, "factor must be finite");
  zero_status_t s = check_writable(h);
  if (s != ZERO_OK) return s;
  DeviceGuard dg(h->device);
  // the device has a norm to end if the host knows of one, or cannot know
  const bool ends_norm = h->have || h->graph_have || capturing(static_cast<hipStream_t>(stream));
  hipError_t e = zs::launch_grads_scale(h->args, factor, ends_norm, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("scale kernel", e);
  written(h, stream);
  return ZERO_OK;
}

zero_status_t zero_grads_query(zero_grads_t h, double* norm, int32_t* found_inf, float* coef, void* stream) {
  if (!h) return fail(ZERO_EINVAL, "null handle");
  DeviceGuard dg(h->device);
  zs::GradsScalars sc;
  hipError_t e = hipStreamSynchronize(static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("hipStreamSynchronize(query)", e);
  e = hipMemcpy(&sc, h->args.sc, sizeof(sc), hipMemcpyDeviceToHost);
  if (e != hipSuccess) return hip_fail("hipMemcpy(scalars)", e);
  if (sc.refused)
    return fail(ZERO_ESTATE, "the last zero_grads_clip found no norm of these values on the device, and wrote nothing");
  if (!sc.clipped) return fail(ZERO_ESTATE, "no zero_grads_clip has run yet");
  if (norm) *norm = sc.clip_norm;
  if (found_inf) *found_inf = sc.clip_flag ? 1 : 0;
  if (coef) *coef = sc.coef;
  return ZERO_OK;
}

zero_status_t zero_grads_destroy(zero_grads_t h) {
  delete h;
  return ZERO_OK;
}

}  // extern "C"
