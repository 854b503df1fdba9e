// C ABI of the gradient norm and clipping (poetx_grad_norm, _clip, _scale):
// validation of the tensor list, and the list as runs of contiguous memory
// for the kernels. Declarations and the contract are in include/poetx.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "api_util.h"
#include "kernels.h"
#include "poetx.h"

using poetx::DType;
using poetx::GradRun;
using namespace poetx::api;

namespace {

constexpr int64_t kMaxBytes = INT64_C(1) << 44;  // of one list: far above any memory

// The list's non-empty tensors as runs; neighbours in the list that are
// neighbours in memory (views of one flat buffer, in order, of one type, with
// their outputs likewise) are one run, so a whole flat buffer is one launch.
// `writes`: out is needed.
int make_runs(const poetx_grad_tensor* t, int32_t count, bool writes, std::vector<GradRun>& runs) {
  if (count < 0) return POETX_ERR_SHAPE;
  if (count > 0 && !t) return POETX_ERR_NULL;
  runs.reserve(count);
  int64_t bytes = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].dtype != POETX_F32 && t[i].dtype != POETX_BF16) return POETX_ERR_DTYPE;
    const int64_t es = (int64_t)act_size(t[i].dtype);
    if (t[i].n < 0 || t[i].n > kMaxBytes || t[i].reserved != 0) return POETX_ERR_SHAPE;
    if ((bytes += t[i].n * es) > kMaxBytes) return POETX_ERR_SHAPE;
    if (t[i].n == 0) continue;
    if (!t[i].grad || (writes && !t[i].out)) return POETX_ERR_NULL;
    const char* g = static_cast<const char*>(t[i].grad);
    char* o = static_cast<char*>(writes ? t[i].out : nullptr);
    if ((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(o)) % es)
      return POETX_ERR_ALIGN;
    const DType dt = t[i].dtype == POETX_BF16 ? DType::BF16 : DType::F32;
    if (!runs.empty()) {
      GradRun& b = runs.back();
      if (b.dtype == dt && static_cast<const char*>(b.grad) + b.n * es == g &&
          (!writes || static_cast<char*>(b.out) + b.n * es == o)) {
        b.n += t[i].n;
        continue;
      }
    }
    runs.push_back(GradRun{g, o, t[i].n, dt});
  }
  return POETX_OK;
}

// Large runs that start off a 16-byte boundary (views of a flat buffer, say),
// both ends alike: the values up to the boundary as a run of their own, so
// that the kernels read and write the rest 16 bytes at a time (the norm of
// 10^8 values that start one value off: float32 203 -> 76 us, bf16 119 -> 38;
// 20000 float32 5.7 -> 4.8, 20000 bf16 7.4 -> 4.8). A run within one
// workgroup's chunk, kPeelBytes, gains nothing from a second one.
constexpr int64_t kPeelBytes = 16384;
void peel_runs(std::vector<GradRun>& runs) {
  const auto head = [](const GradRun& r) -> int64_t {  // bytes, 0: as it is
    const uintptr_t g = reinterpret_cast<uintptr_t>(r.grad), o = reinterpret_cast<uintptr_t>(r.out);
    const int64_t es = r.dtype == DType::BF16 ? 2 : 4;
    if (g % 16 == 0 || (o && (g ^ o) % 16) || r.n * es <= kPeelBytes) return 0;
    return 16 - (int64_t)(g % 16);
  };
  if (std::all_of(runs.begin(), runs.end(), [&](const GradRun& r) { return head(r) == 0; })) return;
  std::vector<GradRun> peeled;
  peeled.reserve(2 * runs.size());
  for (const GradRun& r : runs) {
    const int64_t h = head(r), n = h / (r.dtype == DType::BF16 ? 2 : 4);
    if (h == 0) {
      peeled.push_back(r);
      continue;
    }
    peeled.push_back(GradRun{r.grad, r.out, n, r.dtype});
    peeled.push_back(GradRun{static_cast<const char*>(r.grad) + h,
                             r.out ? static_cast<char*>(r.out) + h : nullptr, r.n - n, r.dtype});
  }
  runs.swap(peeled);
}

Range grad_range(const GradRun& r) {
  return range_of(r.grad, (size_t)r.n * (r.dtype == DType::BF16 ? 2 : 4));
}
Range out_range(const GradRun& r) {
  return range_of(r.out, (size_t)r.n * (r.dtype == DType::BF16 ? 2 : 4));
}

// Every output range must be disjoint from every other output, from the
// gradients of other runs, and equal to or disjoint from its own gradient;
// the norm and the workspace (`extra`, written) disjoint from all. Sorted by
// address, a written range that overlaps anything overlaps a neighbour of
// the running maximum end.
int check_alias(const std::vector<GradRun>& runs, bool writes, const Range* extra, int nextra) {
  struct Item {
    Range r;
    bool written;
  };
  std::vector<Item> v;
  v.reserve(2 * runs.size() + nextra);
  for (const GradRun& r : runs) {
    const Range g = grad_range(r);
    if (!writes) {
      v.push_back(Item{g, false});
      continue;
    }
    v.push_back(Item{out_range(r), true});
    if (r.out != r.grad) v.push_back(Item{g, false});
  }
  for (int i = 0; i < nextra; ++i) v.push_back(Item{extra[i], true});
  std::sort(v.begin(), v.end(), [](const Item& a, const Item& b) { return a.r.lo < b.r.lo; });
  uintptr_t end_any = 0, end_written = 0;  // of the ranges that start earlier
  for (const Item& it : v) {
    if (it.r.lo < end_written || (it.written && it.r.lo < end_any)) return POETX_ERR_ALIAS;
    end_any = std::max(end_any, it.r.hi);
    if (it.written) end_written = std::max(end_written, it.r.hi);
  }
  return POETX_OK;
}

bool float_aligned(const float* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The three calls in one: norm only, norm and clip, scale by a given norm.
int run_list(const poetx_grad_tensor* t, int32_t count, bool measure, bool scale, float max_norm,
             float* norm_out, const float* norm_in, void* ws, size_t ws_bytes, void* stream) {
  if (scale && !(max_norm >= 0.0f)) return POETX_ERR_SHAPE;  // (NaN too)
  std::vector<GradRun> runs;
  int st = make_runs(t, count, scale, runs);
  if (st != POETX_OK) return st;
  const float* norm = measure ? norm_out : norm_in;
  if (!norm) return POETX_ERR_NULL;
  if (!float_aligned(norm)) return POETX_ERR_ALIGN;
  Range extra[2];
  int nextra = 0;
  size_t need = 0;
  if (measure) {
    need = poetx_grad_workspace_size(count);
    if (!ws || ws_bytes < need) return POETX_ERR_WORKSPACE;
    if (!aligned16(ws)) return POETX_ERR_ALIGN;
    extra[nextra++] = range_of(ws, need);
    extra[nextra++] = range_of(norm_out, sizeof(float));
  }
  st = check_alias(runs, scale, extra, nextra);
  if (st != POETX_OK) return st;
  if (!measure)  // the given norm is read while the outputs are written
    for (const GradRun& r : runs)
      if (overlap(out_range(r), range_of(norm_in, sizeof(float)))) return POETX_ERR_ALIAS;

  peel_runs(runs);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int n = (int)runs.size();
  double* part = static_cast<double*>(ws);
  int nparts = 0;
  if (measure) {
    hipError_t e = poetx::launch_grad_sumsq(runs.data(), n, part, &nparts, s);
    if (e == hipSuccess && (!scale || n == 0))
      e = poetx::launch_grad_norm(part, nparts, norm_out, s);
    if (e != hipSuccess) return POETX_ERR_HIP;
  }
  if (!scale || n == 0) return POETX_OK;
  return hip_status(poetx::launch_grad_scale(runs.data(), n, measure ? part : nullptr, nparts,
                                             norm_in, max_norm, norm_out, s));
}

}  // namespace

// (std::vector may throw; nothing leaves these calls but a status)
#define POETX_NOTHROW(expr)          \
  try {                              \
    return (expr);                   \
  } catch (const std::bad_alloc&) {  \
    return POETX_ERR_WORKSPACE;      \
  }

extern "C" {

size_t poetx_grad_workspace_size(int32_t count) {
  // (peel_runs makes two of a run at most)
  return count < 0 ? 0 : align_up(poetx::grad_partials_max(2 * (int64_t)count) * sizeof(double));
}

int poetx_grad_norm(const poetx_grad_tensor* tensors, int32_t count, float* norm, void* ws,
                    size_t ws_bytes, void* stream) {
  POETX_NOTHROW(run_list(tensors, count, true, false, 0.0f, norm, nullptr, ws, ws_bytes, stream))
}

int poetx_grad_clip(const poetx_grad_tensor* tensors, int32_t count, float max_norm, float* norm,
                    void* ws, size_t ws_bytes, void* stream) {
  POETX_NOTHROW(
      run_list(tensors, count, true, true, max_norm, norm, nullptr, ws, ws_bytes, stream))
}

int poetx_grad_scale(const poetx_grad_tensor* tensors, int32_t count, float max_norm,
                     const float* norm, void* stream) {
  POETX_NOTHROW(run_list(tensors, count, false, true, max_norm, nullptr, norm, nullptr, 0, stream))
}

}  // extern "C"
