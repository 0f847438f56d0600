"""Host side of the gradient-list operators, on the CPU: the plan, its refusals, the overlap rules, the Python
binding's description of strided tensors, and the planner under sanitizers."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import zero_partitioned_mixed_reduce_amd as zpm
from zero_partitioned_mixed_reduce_amd import _abi
from zero_partitioned_mixed_reduce_amd.grads import ZeroGrads, describe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F16, BF16, F32 = _abi.ZERO_F16, _abi.ZERO_BF16, _abi.ZERO_F32
BASE = 1 << 40      # fake addresses, never dereferenced


def entry(src=BASE, dst=None, rows=1, cols=100, sp=None, dp=None, sd=BF16, dd=BF16):
    return _abi.zero_grads_tensor_t(src, dst, rows, cols, cols if sp is None else sp, cols if dp is None else dp, sd, dd)


def listof(*entries):
    return (_abi.zero_grads_tensor_t * len(entries))(*entries)


def refused(*entries, needle=""):
    with pytest.raises(zpm.ZeroError) as e:
        zpm.zero_grads_plan(listof(*entries))
    assert e.value.status == _abi.ZERO_EINVAL and needle in str(e.value), str(e.value)


def test_plan_counts():
    i = zpm.zero_grads_plan(listof(entry(cols=8192 * 3 + 1), entry(cols=0, src=None), entry(cols=1000)))
    assert (i.elems, i.num_chunks) == (8192 * 3 + 1 + 1000, 5) and i.workspace_bytes % 256 == 0
    # a strided matrix whose pitch is its width is one run
    a = zpm.zero_grads_plan(listof(entry(rows=64, cols=1000)))
    b = zpm.zero_grads_plan(listof(entry(rows=1, cols=64000)))
    assert a.as_dict() == b.as_dict()
    # lists without elements are lists
    assert zpm.zero_grads_plan(listof(entry(cols=0, src=None), entry(rows=0, cols=7, src=None))).num_chunks == 0


def test_refusals():
    refused(entry(sd=0), needle="src_dtype")
    refused(entry(sd=4), needle="src_dtype")
    refused(entry(dst=BASE + 4096, dd=7), needle="dst_dtype")
    refused(entry(rows=-1), needle=">= 0")
    refused(entry(cols=-1), needle=">= 0")
    refused(entry(src=None), needle="null address")
    refused(entry(), entry(src=None), needle="tensor 1")
    refused(entry(src=BASE + 1), needle="aligned")
    refused(entry(src=BASE + 2, sd=F32), needle="aligned")
    refused(entry(dst=BASE + 4097), needle="destination not aligned")
    refused(entry(dst=BASE + 4098, dd=F32), needle="destination not aligned")
    refused(entry(rows=3, cols=10, sp=9), needle="src_pitch")
    refused(entry(rows=3, cols=10, sp=16, dst=BASE + 4096, dp=9), needle="dst_pitch")
    refused(entry(rows=3, cols=10, sp=1 << 62), needle="src_pitch")
    refused(entry(rows=1 << 31, cols=1 << 31), needle="2^60")
    refused(entry(cols=1 << 59), entry(cols=1 << 60), needle="2^60")
    refused(entry(cols=1 << 40), needle="blocks")
    refused(entry(src=2 ** 64 - 100, cols=100), needle="wrap")
    with pytest.raises(zpm.ZeroError):
        zpm.zero_grads_plan(listof())
    L, info = _abi.lib(), _abi.zero_grads_info_t()
    assert L.zero_grads_plan(None, 1, ctypes.byref(info)) == _abi.ZERO_EINVAL
    assert L.zero_grads_plan(listof(entry()), 1 << 22, ctypes.byref(info)) == _abi.ZERO_EINVAL  # nothing is read
    assert L.zero_grads_plan(listof(entry()), 1, None) == _abi.ZERO_EINVAL


def test_calls_refuse_null_handles():
    L = _abi.lib()
    assert L.zero_grads_norm(None, 1, 1.0, 0, None) == _abi.ZERO_EINVAL
    assert L.zero_grads_clip(None, 1, 0, 0.0, 1.0, None) == _abi.ZERO_EINVAL
    assert L.zero_grads_clip_norm(None, 1, 1.0, 0, 1, 1.0, None) == _abi.ZERO_EINVAL
    assert L.zero_grads_scale(None, 1.0, None) == _abi.ZERO_EINVAL
    assert L.zero_grads_bind(None, None, None, None) == _abi.ZERO_EINVAL
    assert L.zero_grads_query(None, None, None, None, None) == _abi.ZERO_EINVAL
    assert L.zero_grads_info(None, None) == _abi.ZERO_EINVAL
    assert L.zero_grads_device(None, None, None, None, None, None) == _abi.ZERO_EINVAL
    assert L.zero_grads_destroy(None) == _abi.ZERO_OK
    # init checks the workspace before any device work
    h = ctypes.c_void_p()
    t = listof(entry())
    need = zpm.zero_grads_plan(t).workspace_bytes
    for ws, cap, needle in ((None, need, "non-null"), (BASE + 128, need, "256-byte"), (BASE, need - 1, "capacity")):
        assert L.zero_grads_init(t, 1, ws, cap, None, ctypes.byref(h)) == _abi.ZERO_EINVAL
        assert needle in zpm.zero_last_error() and not h.value


def test_overlap_rules():
    far = BASE + (1 << 30)
    plan = lambda *e: zpm.zero_grads_plan(listof(*e))
    plan(entry(), entry())                                                   # nothing is written: sources repeat ...
    refused(entry(dst=far), entry(dst=far), needle="overlaps")               # ... destinations do not
    refused(entry(dst=far), entry(dst=far + 198), needle="overlaps")
    plan(entry(dst=far), entry(dst=far + 200))
    refused(entry(dst=BASE + 2), needle="overlaps")                          # partly onto itself
    refused(entry(dst=BASE, dd=F16), needle="overlaps")                      # onto itself as another type
    refused(entry(dst=far), entry(src=far + 100), needle="overlaps")         # onto another's source
    refused(entry(dst=BASE), entry(dst=far), needle="overlaps")              # a source written in place, read again
    plan(entry(dst=BASE), entry(src=BASE + 200, dst=far))
    # columns of one matrix, in place: q, k and v slices of a fused gradient
    cut = [entry(src=BASE + 2 * 40 * i, dst=BASE + 2 * 40 * i, rows=16, cols=40, sp=120, dp=120) for i in range(3)]
    plan(*cut)
    refused(*cut[:2], entry(src=BASE + 2 * 79, dst=BASE + 2 * 79, rows=16, cols=40, sp=120, dp=120), needle="overlaps")
    # a column that runs past the row's end reaches the next row's first columns
    refused(entry(src=BASE, dst=BASE, rows=16, cols=41, sp=120, dp=120),
            entry(src=BASE + 160, dst=BASE + 160, rows=15, cols=41, sp=120, dp=120), needle="overlaps")
    # one run inside another's gap
    plan(cut[0], entry(src=BASE + 2 * 40, dst=BASE + 2 * 40, cols=80))
    refused(cut[0], entry(src=BASE + 2 * 40, dst=BASE + 2 * 40, cols=81), needle="overlaps")
    # other pitches that interleave are refused
    refused(cut[0], entry(src=BASE + 2 * 40, dst=BASE + 2 * 40, rows=16, cols=40, sp=240, dp=240), needle="overlaps")


def test_overlap_rules_stay_fast():
    """A list that repeats one tensor many times is planned without comparing every pair."""
    import time
    n = 200_000
    t = listof(*[entry(cols=64)] * n)
    began = time.monotonic()
    assert zpm.zero_grads_plan(t).elems == 64 * n
    assert time.monotonic() - began < 5.0
    u = listof(*[entry(cols=64, dst=BASE + (1 << 40) + 128 * i) for i in range(n)])
    u[n - 1].dst = BASE + (1 << 40)            # out of order, so every pair of neighbours is compared
    with pytest.raises(zpm.ZeroError):
        zpm.zero_grads_plan(u)
    assert time.monotonic() - began < 10.0


def elements_of(t, dst=False):
    """Byte offsets from the tensor's first element, in list order."""
    es = 4 if (t.dst_dtype if dst else t.src_dtype) == F32 else 2
    pitch = t.dst_pitch if dst else t.src_pitch
    return [es * (r * pitch + c) for r in range(t.rows) for c in range(t.cols)]


def offsets(x):
    """Byte offsets of x's elements from its first, in logical order."""
    i = torch.zeros((), dtype=torch.int64)
    for k, n in enumerate(x.shape):
        i = i.unsqueeze(-1) + torch.arange(n) * x.stride(k)
    return (i.flatten() * x.element_size()).tolist()


CUTS = [lambda x: x, lambda x: x[:, :5], lambda x: x[1:, 2:], lambda x: x[::2], lambda x: x[:, ::2], lambda x: x[:, 3],
        lambda x: x.t(), lambda x: x[:, :5].t(), lambda x: x[2], lambda x: x[:1, :4], lambda x: x[3:3],
        lambda x: x.view(4, 3, 10), lambda x: x.view(4, 3, 10)[:, 1], lambda x: x.view(4, 3, 10)[:, :, :7],
        lambda x: x.view(4, 3, 10).permute(2, 0, 1), lambda x: x.view(4, 3, 10)[:, :2, :3],
        lambda x: x.view(4, 3, 10).permute(1, 0, 2), lambda x: x[0, 0]]


@pytest.mark.parametrize("cut", range(len(CUTS)))
def test_describe_matches_torch(cut):
    """Whatever description the binding gives covers exactly the tensor's elements; into another tensor, in logical
    order.  What it cannot describe it refuses."""
    x = CUTS[cut](torch.zeros(12, 10, dtype=torch.bfloat16))
    described = 0
    try:
        t = describe(0, x, None)
        assert sorted(elements_of(t)) == sorted(offsets(x))
        described += 1
    except ValueError as e:
        assert "rows of consecutive" in str(e)
    for y in (torch.zeros(x.numel()), torch.zeros(x.shape), torch.zeros(*x.shape, 2)[..., 0] if x.dim() else torch.zeros(()),
              torch.empty_strided(x.shape, x.stride(), dtype=torch.float16)):
        try:
            t = describe(0, x, y)
        except ValueError as e:
            assert "rows of consecutive" in str(e)
            continue
        described += 1
        pairs = list(zip(elements_of(t), elements_of(t, True)))
        assert sorted(pairs) == sorted(zip(offsets(x), offsets(y)))
    assert described >= 1 or cut == 15      # 15: three levels of strides, which no rows at one pitch describe


def test_described_cases():
    z = torch.zeros(12, 10, dtype=torch.bfloat16)
    flat = torch.zeros(120)
    for good, out in ((z[:, :5], flat[:60]), (z.t(), None), (z.view(4, 3, 10).permute(2, 0, 1), None), (z[:, 3], flat[:12]),
                      (z[::2], flat[:60]), (z.t(), torch.zeros(12, 10).t())):
        describe(0, good, out)
    for badly, out in ((z.t(), flat), (z.view(4, 3, 10)[:, :2, :3], None), (z[:1].expand(7, 10), None)):
        with pytest.raises(ValueError):
            describe(0, badly, out)
    with pytest.raises(ValueError, match="float64"):
        describe(3, torch.zeros(3, dtype=torch.float64), None)
    with pytest.raises(ValueError, match="elements"):
        describe(3, z, torch.zeros(119))
    with pytest.raises(ValueError, match="strided|dense"):
        describe(0, torch.zeros(4, 4).to_sparse(), None)


def test_class_refuses_on_the_host():
    with pytest.raises(ValueError, match="GPU"):
        ZeroGrads([torch.zeros(4)])
    with pytest.raises(ValueError, match="empty"):
        ZeroGrads([])
    assert zpm.ZeroGrads is ZeroGrads


def test_header_is_c99(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "use.c"
    src.write_text('#include "zero_grads.h"\nint main(void) { zero_grads_info_t i; zero_grads_tensor_t t = {0};\n'
                   "t.cols = 0; t.rows = 1; t.src_dtype = ZERO_F32;\n"
                   "return zero_grads_plan(&t, 1, &i) == ZERO_OK && i.elems == 0 ? 0 : 1; }\n")
    exe, lib_dir = tmp_path / "use", os.path.dirname(_abi.LIB_PATH)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe), "-L", lib_dir, "-lzero_shard", "-Wl,-rpath," + lib_dir], check=True, timeout=120)
    assert subprocess.run([str(exe)], timeout=120).returncode == 0


DRIVER = r'''
#include <stdio.h>
#include <string.h>
#include <set>
#include <string>
#include <vector>
#include "grads.h"
static unsigned long long seed = 777;
static unsigned rnd() { seed = seed * 6364136223846793005ULL + 1442695040888963407ULL; return (unsigned)(seed >> 33); }
static int es(int d) { return d == ZERO_F32 ? 4 : 2; }
// every (source byte, destination byte) pair of a tensor, by the definition
static void pairs_of(const zero_grads_tensor_t& t, std::vector<std::pair<uint64_t, uint64_t>>* v) {
  for (int64_t r = 0; r < t.rows; ++r)
    for (int64_t c = 0; c < t.cols; ++c)
      v->push_back({(uint64_t)(uintptr_t)t.src + es(t.src_dtype) * (r * t.src_pitch + c),
                    (uint64_t)(uintptr_t)t.dst + es(t.dst_dtype) * (r * t.dst_pitch + c)});
}
int main() {
  long tables = 0, overlaps = 0;
  for (int it = 0; it < 400; ++it) {   // tables: far-apart tensors, every element once
    int n = 1 + rnd() % 12;
    std::vector<zero_grads_tensor_t> t(n);
    uint64_t at = 1 << 20;
    int64_t elems = 0;
    for (auto& x : t) {
      memset(&x, 0, sizeof x);
      x.src_dtype = 1 + rnd() % 3;
      x.dst_dtype = 1 + rnd() % 3;
      int kind = rnd() % 5;
      x.rows = kind < 2 ? 1 : rnd() % 40;
      x.cols = kind == 0 ? rnd() % 70000 : kind == 1 ? rnd() % 2000 : kind == 2 ? rnd() % 10 : kind == 3 ? rnd() % 600 : 8000 + rnd() % 400;
      x.src_pitch = x.cols + (rnd() % 2 ? rnd() % 50 : 0);
      x.dst_pitch = x.cols + (rnd() % 2 ? rnd() % 50 : 0);
      x.src = (void*)(uintptr_t)(at + 4 * (rnd() % 8));
      at += 4 * (x.src_pitch * x.rows + 64);
      x.dst = rnd() % 4 ? (void*)(uintptr_t)(at + 4 * (rnd() % 8)) : nullptr;
      at += 4 * (x.dst_pitch * x.rows + 64);
      elems += x.rows * x.cols;
    }
    zs::GradsPlan p;
    std::string err;
    if (zs::build_grads_plan(t.data(), n, &p, &err) != ZERO_OK) { printf("refused: %s\n", err.c_str()); return 1; }
    zs::fill_grads_chunks(&p);
    if (p.info.elems != elems || (int64_t)p.chunks.size() != p.info.num_chunks) { printf("bad sizes\n"); return 1; }
    int64_t covered_items = 0, join = 0;
    auto joins = [](int64_t c) { return c <= 1 ? 0 : (c + 63) / 64 + (c > 64); };
    for (int i = 0; i < n; ++i) {
      zero_grads_tensor_t x = t[i];
      if (!x.dst) { x.dst = x.src; x.dst_pitch = x.src_pitch; x.dst_dtype = x.src_dtype; }
      std::vector<std::pair<uint64_t, uint64_t>> want, got;
      pairs_of(x, &want);
      const bool wave = x.rows * x.cols <= zs::kGradsSmall;
      for (int c = p.ranges[i].first; c < p.ranges[i].first + p.ranges[i].count; ++c) {
        const zs::GradsChunk& k = p.chunks[c];
        if ((c >= p.n_block_items) != wave || k.tensor != i || k.src_dtype != x.src_dtype || k.dst_dtype != x.dst_dtype) { printf("bad item\n"); return 1; }
        if (p.offsets[c].src != (int64_t)(k.src - (uint64_t)(uintptr_t)x.src) || p.offsets[c].dst != (int64_t)(k.dst - (uint64_t)(uintptr_t)x.dst)) { printf("bad offset\n"); return 1; }
        if (k.first != p.ranges[i].first || k.count != p.ranges[i].count || (k.count > 1 && (k.join != join || k.join + joins(k.count) > p.n_joins))) { printf("bad joins\n"); return 1; }
        if ((int64_t)k.rows * k.cols > zs::kGradsChunk || k.rows < 1 || k.cols < 1) { printf("bad size\n"); return 1; }
        for (int r = 0; r < k.rows; ++r)
          for (int e = 0; e < k.cols; ++e)
            got.push_back({k.src + r * k.src_pitch + (uint64_t)e * es(k.src_dtype), k.dst + r * k.dst_pitch + (uint64_t)e * es(k.dst_dtype)});
        ++covered_items;
      }
      join += joins(p.ranges[i].count);
      if (got != want) { printf("tensor %d not covered in order\n", i); return 1; }
    }
    if (join != p.n_joins) { printf("bad counters\n"); return 1; }
    const int64_t n_wave = p.info.num_chunks - p.n_block_items;
    if (covered_items != p.info.num_chunks || p.n_blocks != p.n_block_items + (n_wave + 3) / 4) { printf("bad blocks\n"); return 1; }
    ++tables;
  }
  for (int it = 0; it < 20000; ++it) {   // addresses in a narrow window, against a map of its bytes
    int n = 1 + rnd() % 3;
    std::vector<zero_grads_tensor_t> t(n);
    for (auto& x : t) {
      memset(&x, 0, sizeof x);
      x.src_dtype = rnd() % 2 ? ZERO_F32 : ZERO_BF16;
      x.dst_dtype = rnd() % 2 ? ZERO_F32 : ZERO_BF16;
      x.rows = 1 + rnd() % 3;
      x.cols = 1 + rnd() % 6;
      x.src_pitch = rnd() % 2 ? 8 : x.cols + rnd() % 4;
      x.dst_pitch = rnd() % 2 ? 8 : x.cols + rnd() % 4;
      x.src = (void*)(uintptr_t)(4096 + 4 * (rnd() % 40));
      if (rnd() % 3 == 0) { x.dst = nullptr; x.dst_dtype = x.src_dtype; }
      else x.dst = (void*)(uintptr_t)((rnd() % 4 ? 5000 : 4096) + 4 * (rnd() % 40));
    }
    bool truth = false;
    std::vector<int> written(4096, 0), read(4096, 0);
    for (int pass = 0; pass < 2; ++pass)
      for (auto x : t) {
        const bool in_place = !x.dst || (x.dst == x.src && x.dst_dtype == x.src_dtype && (x.rows <= 1 || x.dst_pitch == x.src_pitch));
        if (!x.dst) { x.dst = x.src; x.dst_pitch = x.src_pitch; x.dst_dtype = x.src_dtype; }
        std::vector<std::pair<uint64_t, uint64_t>> v;
        pairs_of(x, &v);
        for (auto& q : v) {
          for (int b = 0; b < es(x.dst_dtype); ++b) if (pass == 0 && written[q.second - 4096 + b]++) truth = true;
          for (int b = 0; b < es(x.src_dtype); ++b) if (pass == 1 && !in_place && written[q.first - 4096 + b]) truth = true;
        }
      }
    // a source read by another tensor in place is written: caught above as written + read
    zs::GradsPlan p;
    std::string err;
    const bool refused = zs::build_grads_plan(t.data(), n, &p, &err) != ZERO_OK || p.overlap >= 0;
    if (truth && !refused) { printf("overlap missed\n"); return 1; }
    // what is refused without sharing a byte interleaves rows of different pitch
    if (!truth && refused) {
      std::set<int64_t> pitches;
      for (auto& x : t) {
        if (x.rows > 1) pitches.insert(x.src_pitch * es(x.src_dtype));
        if (x.rows > 1 && x.dst) pitches.insert(x.dst_pitch * es(x.dst_dtype));
      }
      if (pitches.empty()) { printf("refused without reason: %s\n", err.c_str()); return 1; }
    }
    overlaps += truth;
  }
  zs::GradsPlan p;
  std::string err;
  if (zs::build_grads_plan(nullptr, 1, &p, &err) == ZERO_OK) return 1;
  printf("ok %ld tables, %s\n", tables, overlaps > 1000 ? "overlaps" : "few overlaps");
  return 0;
}
'''


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_planner_under_asan_ubsan(tmp_path):
    src, exe = tmp_path / "driver.cpp", tmp_path / "driver"
    src.write_text(DRIVER)
    csrc = os.path.join(ROOT, "zero_partitioned_mixed_reduce_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I",
                    os.path.join(ROOT, "include"), "-I", csrc, str(src), os.path.join(csrc, "grads_plan.cpp"), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1", UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.startswith("ok 400 tables, overlaps")
