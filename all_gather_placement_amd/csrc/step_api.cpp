// Entry points of libtide_step.so: argument checks, then kernel launches.  Nothing is allocated on
// the device and no state is kept, so every call may be captured into a graph.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "step_internal.h"

namespace tide_step {
namespace {

thread_local int g_last_hip_error = 0;

tide_status status_of(int hip_error) {
  if (hip_error == hipSuccess) return TIDE_OK;
  g_last_hip_error = hip_error;
  return TIDE_ERR_HIP;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool float_type(int t) { return t == TIDE_BF16 || t == TIDE_FP32; }
inline int size_of(int t) { return t == TIDE_BF16 ? 2 : t == TIDE_INT64 ? 8 : 4; }

struct Range {
  uintptr_t lo, hi;
  uintptr_t row = 0, stride = 0;  // bytes of each row and between rows' starts, where rows have gaps between them
};
inline Range range_of(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + uintptr_t(bytes)};
}
// `rows` rows of `row` elements, `stride` elements apart
inline Range range_of(const void* p, int64_t rows, int64_t row, int64_t stride, int size) {
  Range r = range_of(p, rows == 0 ? 0 : ((rows - 1) * stride + row) * size);
  if (rows > 1 && stride > row) {
    r.row = uintptr_t(row * size);
    r.stride = uintptr_t(stride * size);
  }
  return r;
}
inline Range opt_range(const void* p, int64_t bytes) { return p == nullptr ? Range{0, 0} : range_of(p, bytes); }
// Blocks of columns of one buffer do not overlap though one's rows lie between the other's: of equal strides,
// or of one whose gaps hold all of the other.  Rows of different strides are taken to meet somewhere.
inline bool overlap(const Range& a, const Range& b) {
  if (!(a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi)) return false;
  const uintptr_t stride = a.stride > b.stride ? a.stride : b.stride;
  if (stride == 0 || (a.stride != b.stride && a.stride != 0 && b.stride != 0)) return true;
  const uintptr_t arow = a.stride != 0 ? a.row : a.hi - a.lo, brow = b.stride != 0 ? b.row : b.hi - b.lo;
  // where a row of a starts, counted from the row of b that starts at or before it
  const uintptr_t from = a.lo >= b.lo ? (a.lo - b.lo) % stride : (stride - (b.lo - a.lo) % stride) % stride;
  return from < brow || from + arow > stride;
}
// Whether any output lies over another output or an input; empty ranges lie over nothing.
template <size_t N, size_t M>
bool outputs_overlap(const Range (&outs)[N], const Range (&ins)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
    for (const Range& in : ins)
      if (overlap(outs[i], in)) return true;
  }
  return false;
}

bool workspace_ok(const void* p, int64_t have, int64_t need) {
  return need >= 0 && have >= need && (need == 0 || (p != nullptr && aligned(p, 16)));
}

// ---------------------------------------------------------------------------------------------
// Gradient norm
// ---------------------------------------------------------------------------------------------

bool tensors_ok(int32_t n, const int64_t* numels, int32_t dtype) {
  if (n < 0 || (n > 0 && numels == nullptr) || !float_type(dtype)) return false;
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (numels[i] < 0 || numels[i] > kMaxNormElems - total) return false;
    total += numels[i];
  }
  return true;
}

bool pointers_ok(int32_t n, const void* const* ptrs, const int64_t* numels, int32_t dtype) {
  if (n > 0 && ptrs == nullptr) return false;
  for (int32_t i = 0; i < n; ++i)
    if (numels[i] > 0 && (ptrs[i] == nullptr || !aligned(ptrs[i], size_of(dtype)))) return false;
  return true;
}

// Chunks of a tensor, and the elements of its last one.
inline void cut(int64_t numel, int dtype, uint32_t* chunks, uint32_t* last) {
  const int64_t c = norm_chunk_elems(dtype), n = (numel + c - 1) / c;
  *chunks = uint32_t(n);
  *last = uint32_t(numel - (n - 1) * c);
}

inline int norm_grid(uint32_t chunks) { return int(std::min<uint32_t>(chunks, kNormWgs)); }
inline int clip_grid(uint32_t chunks) { return int(std::min<uint32_t>(chunks, kNormMaxWgs)); }

int64_t num_chunks(int32_t n, const int64_t* numels, int dtype) {
  const int64_t c = norm_chunk_elems(dtype);
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) total += (numels[i] + c - 1) / c;
  return total;
}
// Whether one workgroup does a whole call, in one launch.
bool one_workgroup(int64_t chunks) { return chunks > 0 && chunks <= kNormOneWgChunks; }

// Calls f(table) for every launch that the non-empty tensors need, stops at the first error.
template <typename Table, int kBatch, typename Fill, typename F>
int for_tables(int32_t n, const int64_t* numels, int dtype, Fill&& fill, F&& f) {
  Table t;
  t.count = 0;
  t.chunks = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (numels[i] == 0) continue;
    uint32_t chunks, last;
    cut(numels[i], dtype, &chunks, &last);
    auto& e = t.e[t.count++];
    fill(e, i);
    e.first = t.chunks;
    e.last = last;
    t.chunks += chunks;
    if (t.count == kBatch) {
      if (const int err = f(t)) return err;
      t.count = 0;
      t.chunks = 0;
    }
  }
  return t.count > 0 ? f(t) : 0;
}

int64_t num_partials(int32_t n, const int64_t* numels, int dtype) {
  int64_t total = 0;
  for_tables<NormTable, kNormBatch>(
      n, numels, dtype, [](NormEntry& e, int32_t) { e.p = nullptr; },
      [&](const NormTable& t) {
        total += norm_grid(t.chunks);
        return 0;
      });
  return total;
}

// Workspace: the sum of squares (for a clip that keeps it to itself), then the partial sums.
int64_t norm_workspace(int32_t n, const int64_t* numels, int dtype) {
  return 16 + (num_partials(n, numels, dtype) * 8 + 15) / 16 * 16;
}

// The partial sums of squares, `used` of them from workspace + 16 bytes on; one workgroup's calls write
// the results themselves.
int enqueue_partials(int32_t n, const void* const* grads, const int64_t* numels, int dtype, double* sumsq, float* norm,
                     double* partial, bool one, int* used, void* stream) {
  *used = 0;
  return for_tables<NormTable, kNormBatch>(
      n, numels, dtype, [&](NormEntry& t, int32_t i) { t.p = grads[i]; },
      [&](NormTable& t) {
        const int grid = one ? 1 : norm_grid(t.chunks);
        t.sumsq = one ? sumsq : nullptr;
        t.norm = one ? norm : nullptr;
        const int err = launch_norm_partial(t, dtype, partial + *used, grid, stream);
        *used += grid;
        return err;
      });
}
int enqueue_norm(int32_t n, const void* const* grads, const int64_t* numels, int dtype, double* sumsq, float* norm,
                 void* workspace, void* stream) {
  double* partial = static_cast<double*>(workspace) + 2;
  const bool one = one_workgroup(num_chunks(n, numels, dtype));
  int used;
  const int e = enqueue_partials(n, grads, numels, dtype, sumsq, norm, partial, one, &used, stream);
  return e != 0 ? e : launch_norm_finish(partial, used, one ? nullptr : sumsq, one ? nullptr : norm, stream);
}

// Clipping by *sumsq; or, where `sum_to` is given, by the sum of `partials` partial sums, or of one
// workgroup's own, which is written there.
int enqueue_clip(int32_t n, const void* const* grads, void* const* outs, const int64_t* numels, int dtype,
                 const double* sumsq, double* sum_to, const double* partial, int partials, double max_norm, float* norm,
                 void* stream) {
  bool first = true;
  const int e = for_tables<ClipTable, kClipBatch>(
      n, numels, dtype,
      [&](ClipEntry& t, int32_t i) {
        t.p = grads[i];
        t.out = outs[i];
      },
      [&](ClipTable& t) {
        t.sum_to = sum_to;
        t.partial = partial;
        t.partials = partials;
        const int grid = sum_to != nullptr && partial == nullptr ? 1 : clip_grid(t.chunks);
        const int err = launch_clip(t, dtype, sumsq, max_norm, first ? norm : nullptr, grid, stream);
        first = false;
        return err;
      });
  if (e != 0 || !first || norm == nullptr) return e;
  ClipTable none;  // no elements: the norm alone
  none.count = 0;
  none.chunks = 0;
  none.sum_to = nullptr;
  none.partial = nullptr;
  none.partials = 0;
  return launch_clip(none, dtype, sumsq, max_norm, norm, 1, stream);
}

// Each output may be its own gradient and lies over nothing else.  Throws std::bad_alloc.
bool clip_overlaps(int32_t n, const void* const* grads, void* const* outs, const int64_t* numels, int dtype,
                   const std::vector<Range>& scalars) {
  struct Tagged {
    Range r;
    int32_t tensor;
  };
  std::vector<Tagged> o;
  o.reserve(size_t(n));
  const int size = size_of(dtype);
  for (int32_t i = 0; i < n; ++i)
    if (numels[i] > 0) o.push_back({range_of(outs[i], numels[i] * size), i});
  const auto lower = [](const Tagged& a, const Tagged& b) { return a.r.lo < b.r.lo; };
  if (!std::is_sorted(o.begin(), o.end(), lower)) std::sort(o.begin(), o.end(), lower);
  for (size_t i = 1; i < o.size(); ++i)
    if (o[i].r.lo < o[i - 1].r.hi) return true;
  auto near = o.begin();  // where the last range was found: lists are mostly in order of address
  const auto hits = [&](const Range& in, int32_t own) {
    const auto first = [&](auto it) {  // whether `it` is the first output that ends after in.lo
      return (it == o.end() || in.lo < it->r.hi) && (it == o.begin() || std::prev(it)->r.hi <= in.lo);
    };
    if (near != o.end() && first(std::next(near)))
      ++near;
    else if (!first(near))
      near = std::upper_bound(o.begin(), o.end(), in.lo, [](uintptr_t v, const Tagged& t) { return v < t.r.hi; });
    auto it = near;
    for (; it != o.end() && it->r.lo < in.hi; ++it)
      if (it->tensor != own || it->r.lo != in.lo) return true;
    return false;
  };
  for (int32_t i = 0; i < n; ++i)
    if (numels[i] > 0 && hits(range_of(grads[i], numels[i] * size), i)) return true;
  for (const Range& s : scalars)
    if (hits(s, -1)) return true;
  return false;
}

// Whether one of the results or the workspace lies over another or over a gradient: a workgroup would write
// what others still read.
template <size_t N>
bool results_overlap(const Range (&results)[N], int32_t n, const void* const* grads, const int64_t* numels, int dtype) {
  const Range none[] = {{0, 0}};
  if (outputs_overlap(results, none)) return true;
  for (int32_t i = 0; i < n; ++i) {
    const Range g = range_of(grads[i], numels[i] * size_of(dtype));
    for (const Range& r : results)
      if (overlap(r, g)) return true;
  }
  return false;
}

bool max_norm_ok(double m) { return m >= 0; }  // false for NaN

}  // namespace
}  // namespace tide_step

using namespace tide_step;

extern "C" {

int64_t tide_grad_norm_workspace(int32_t num_tensors, const int64_t* numels, int32_t dtype) {
  if (!tensors_ok(num_tensors, numels, dtype)) return -1;
  return norm_workspace(num_tensors, numels, dtype);
}

tide_status tide_grad_norm(int32_t num_tensors, const void* const* grads, const int64_t* numels, int32_t dtype,
                           double* sumsq, float* norm, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!tensors_ok(num_tensors, numels, dtype) || !pointers_ok(num_tensors, grads, numels, dtype) ||
      !aligned(sumsq, 8) || !aligned(norm, 4))
    return TIDE_ERR_INVALID;
  const int64_t need = norm_workspace(num_tensors, numels, dtype);
  const Range results[] = {opt_range(sumsq, 8), opt_range(norm, 4), opt_range(workspace, need)};
  if (!workspace_ok(workspace, workspace_bytes, need) ||
      results_overlap(results, num_tensors, grads, numels, dtype))
    return TIDE_ERR_INVALID;
  return status_of(enqueue_norm(num_tensors, grads, numels, dtype, sumsq, norm, workspace, stream));
}

tide_status tide_grad_clip(int32_t num_tensors, const void* const* grads, void* const* outs, const int64_t* numels,
                           int32_t dtype, const double* sumsq, double max_norm, float* norm, void* stream) try {
  if (!tensors_ok(num_tensors, numels, dtype) || !pointers_ok(num_tensors, grads, numels, dtype) ||
      !pointers_ok(num_tensors, const_cast<const void* const*>(outs), numels, dtype) || sumsq == nullptr ||
      !aligned(sumsq, 8) || !aligned(norm, 4) || !max_norm_ok(max_norm))
    return TIDE_ERR_INVALID;
  const Range sum = range_of(sumsq, 8), results[] = {opt_range(norm, 4)};
  if (overlap(results[0], sum) || results_overlap(results, num_tensors, grads, numels, dtype) ||
      clip_overlaps(num_tensors, grads, outs, numels, dtype, {sum, results[0]}))
    return TIDE_ERR_INVALID;
  return status_of(enqueue_clip(num_tensors, grads, outs, numels, dtype, sumsq, nullptr, nullptr, 0, max_norm, norm, stream));
} catch (const std::bad_alloc&) {
  return TIDE_ERR_NOMEM;
}

tide_status tide_clip_grad_norm(int32_t num_tensors, const void* const* grads, void* const* outs,
                                const int64_t* numels, int32_t dtype, double max_norm, double* sumsq, float* norm,
                                void* workspace, int64_t workspace_bytes, void* stream) try {
  if (!tensors_ok(num_tensors, numels, dtype) || !pointers_ok(num_tensors, grads, numels, dtype) ||
      !pointers_ok(num_tensors, const_cast<const void* const*>(outs), numels, dtype) || !aligned(sumsq, 8) ||
      !aligned(norm, 4) || !max_norm_ok(max_norm))
    return TIDE_ERR_INVALID;
  const int64_t need = norm_workspace(num_tensors, numels, dtype);
  if (!workspace_ok(workspace, workspace_bytes, need)) return TIDE_ERR_INVALID;
  const Range results[] = {opt_range(sumsq, 8), opt_range(norm, 4), range_of(workspace, need)};
  if (results_overlap(results, num_tensors, grads, numels, dtype) ||
      clip_overlaps(num_tensors, grads, outs, numels, dtype, {results[0], results[1], results[2]}))
    return TIDE_ERR_INVALID;
  double* s = sumsq != nullptr ? sumsq : static_cast<double*>(workspace);
  const int64_t chunks = num_chunks(num_tensors, numels, dtype);
  if (one_workgroup(chunks))
    return status_of(
        enqueue_clip(num_tensors, grads, outs, numels, dtype, s, s, nullptr, 0, max_norm, norm, stream));
  int e;
  if (chunks > 0 && chunks <= kNormClipAddsChunks && num_tensors <= kClipBatch) {
    double* partial = static_cast<double*>(workspace) + 2;
    int used;
    e = enqueue_partials(num_tensors, grads, numels, dtype, nullptr, nullptr, partial, false, &used, stream);
    if (e == 0)
      e = enqueue_clip(num_tensors, grads, outs, numels, dtype, s, s, partial, used, max_norm, norm, stream);
  } else {
    e = enqueue_norm(num_tensors, grads, numels, dtype, s, norm, workspace, stream);
    if (e == 0) e = enqueue_clip(num_tensors, grads, outs, numels, dtype, s, nullptr, nullptr, 0, max_norm, nullptr, stream);
  }
  return status_of(e);
} catch (const std::bad_alloc&) {
  return TIDE_ERR_NOMEM;
}

}  // extern "C"

// ---------------------------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------------------------

namespace tide_step {
namespace {

constexpr int64_t kMaxElems = int64_t(1) << 44;

bool matrix_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 1 && cols < (int64_t(1) << 31) && rows <= kMaxElems / cols;
}
// A matrix argument: its rows do not lie over each other, and its last element's offset fits.
bool strided_ok(const void* p, int64_t rows, int64_t cols, int64_t stride, int dtype) {
  if (rows == 0) return true;
  return p != nullptr && aligned(p, size_of(dtype)) && (rows == 1 || (stride >= cols && stride <= kMaxElems / rows));
}
bool vector_ok(const void* p, int dtype) { return aligned(p, size_of(dtype)); }

int64_t layer_norm_bwd_bytes(int64_t rows, int64_t cols, int dtype) {
  return int64_t(layer_norm_bwd_groups(rows, cols, dtype)) * 2 * layer_norm_bwd_padded(cols) * 4;
}

}  // namespace
}  // namespace tide_step

extern "C" {

tide_status tide_layer_norm(int64_t rows, int64_t cols, const void* x, int64_t x_stride, int32_t dtype,
                            const void* weight, const void* bias, int32_t param_dtype, float eps, void* y,
                            int64_t y_stride, float* mean, float* rstd, void* stream) {
  if (!matrix_ok(rows, cols) || !float_type(dtype) || !float_type(param_dtype) ||
      !strided_ok(x, rows, cols, x_stride, dtype) || !strided_ok(y, rows, cols, y_stride, dtype) ||
      !vector_ok(weight, param_dtype) || !vector_ok(bias, param_dtype) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !(eps >= 0) || !std::isfinite(eps))
    return TIDE_ERR_INVALID;
  if (rows == 0) return TIDE_OK;
  const int64_t pbytes = cols * size_of(param_dtype);
  const Range outs[] = {range_of(y, rows, cols, y_stride, size_of(dtype)), opt_range(mean, rows * 4),
                        opt_range(rstd, rows * 4)};
  const Range ins[] = {range_of(x, rows, cols, x_stride, size_of(dtype)), opt_range(weight, pbytes),
                       opt_range(bias, pbytes)};
  if (outputs_overlap(outs, ins)) return TIDE_ERR_INVALID;
  const LayerNormArgs a{rows, cols, x, x_stride, weight, bias, eps, y, y_stride, mean, rstd};
  return status_of(launch_layer_norm(a, dtype, param_dtype, stream));
}

int64_t tide_layer_norm_bwd_workspace(int64_t rows, int64_t cols, int32_t dtype) {
  if (!matrix_ok(rows, cols) || !float_type(dtype)) return -1;
  return layer_norm_bwd_bytes(rows, cols, dtype);
}

tide_status tide_layer_norm_bwd(int64_t rows, int64_t cols, const void* dy, int64_t dy_stride, const void* x,
                                int64_t x_stride, int32_t dtype, const void* weight, int32_t param_dtype,
                                const float* mean, const float* rstd, void* dx, int64_t dx_stride, void* dweight,
                                void* dbias, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!matrix_ok(rows, cols) || !float_type(dtype) || !float_type(param_dtype) ||
      !strided_ok(dy, rows, cols, dy_stride, dtype) || !strided_ok(x, rows, cols, x_stride, dtype) ||
      (dx != nullptr && !strided_ok(dx, rows, cols, dx_stride, dtype)) || !vector_ok(weight, param_dtype) ||
      !vector_ok(dweight, param_dtype) || !vector_ok(dbias, param_dtype) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      (rows > 0 && (mean == nullptr || rstd == nullptr)))
    return TIDE_ERR_INVALID;
  const int64_t need = layer_norm_bwd_bytes(rows, cols, dtype), pbytes = cols * size_of(param_dtype);
  const bool params = dweight != nullptr || dbias != nullptr;
  if (params && !workspace_ok(workspace, workspace_bytes, need)) return TIDE_ERR_INVALID;
  const int size = size_of(dtype);
  const Range rdx = dx == nullptr ? Range{0, 0} : range_of(dx, rows, cols, dx_stride, size);
  const bool in_place = dx != nullptr && dx == dy && (dx_stride == dy_stride || rows <= 1);
  const Range outs[] = {rdx, opt_range(dweight, pbytes), opt_range(dbias, pbytes),
                        params ? opt_range(workspace, need) : Range{0, 0}};
  const Range rdy = range_of(dy, rows, cols, dy_stride, size);
  const Range ins[] = {in_place ? Range{0, 0} : rdy, range_of(x, rows, cols, x_stride, size),
                       opt_range(weight, pbytes), opt_range(mean, rows * 4), opt_range(rstd, rows * 4)};
  if (outputs_overlap(outs, ins)) return TIDE_ERR_INVALID;
  if (rows == 0 && !params) return TIDE_OK;
  const LayerNormBwdArgs a{rows, cols, dy, dy_stride, x,      x_stride, weight,
                           mean, rstd, dx, dx_stride, dweight, dbias,   static_cast<float*>(workspace)};
  return status_of(launch_layer_norm_bwd(a, dtype, param_dtype, stream));
}

}  // extern "C"

// ---------------------------------------------------------------------------------------------
// Embedding
// ---------------------------------------------------------------------------------------------

namespace tide_step {
namespace {

constexpr int64_t kInt31 = int64_t(1) << 31;

bool embedding_ok(int64_t tokens, const void* ids, int ids_dtype, int64_t vocab, int64_t dim, int dtype) {
  return tokens >= 0 && tokens < kInt31 && vocab >= 0 && vocab < kInt31 && dim >= 1 && dim < kInt31 &&
         float_type(dtype) && (ids_dtype == TIDE_INT32 || ids_dtype == TIDE_INT64) && tokens <= kMaxElems / dim &&
         vocab <= kMaxElems / dim && (tokens == 0 || (ids != nullptr && aligned(ids, size_of(ids_dtype))));
}
bool rows_ok(const void* p, int64_t rows, int dtype) { return rows == 0 || (p != nullptr && aligned(p, size_of(dtype))); }

struct EmbeddingPlan {
  int64_t token, row, count, last, runs, partial, bytes;  // offsets in the workspace
};
EmbeddingPlan embedding_plan(int64_t tokens, int64_t dim) {
  const auto up = [](int64_t n) { return (n + 15) / 16 * 16; };
  EmbeddingPlan p;
  p.count = 0;
  p.token = 16;
  p.row = p.token + up(tokens * 4);
  const int64_t pieces = (tokens + kPiece - 1) / kPiece;
  p.last = p.row + up(tokens * 4);
  p.runs = p.last + up(pieces * 4);
  p.partial = p.runs + up(pieces * int64_t(sizeof(EmbeddingRun)));
  p.bytes = p.partial + up(pieces * 2 * dim * 4);
  return p;
}

}  // namespace
}  // namespace tide_step

extern "C" {

tide_status tide_embedding(int64_t tokens, const void* ids, int32_t ids_dtype, int64_t vocab, int64_t dim,
                           const void* table, int32_t dtype, float scale, void* out, void* stream) {
  if (!embedding_ok(tokens, ids, ids_dtype, vocab, dim, dtype) || !rows_ok(table, vocab, dtype) ||
      !rows_ok(out, tokens, dtype))
    return TIDE_ERR_INVALID;
  if (tokens == 0) return TIDE_OK;
  const int size = size_of(dtype);
  const Range outs[] = {range_of(out, tokens * dim * size)};
  const Range ins[] = {range_of(ids, tokens * size_of(ids_dtype)), opt_range(table, vocab * dim * size)};
  if (outputs_overlap(outs, ins)) return TIDE_ERR_INVALID;
  return status_of(launch_embedding(tokens, ids, ids_dtype, vocab, dim, table, dtype, scale, out, stream));
}

int64_t tide_embedding_bwd_workspace(int64_t tokens, int64_t vocab, int64_t dim) {
  if (tokens < 0 || tokens >= kInt31 || vocab < 0 || vocab >= kInt31 || dim < 1 || dim >= kInt31 ||
      tokens > kMaxElems / dim)
    return -1;
  return embedding_plan(tokens, dim).bytes;
}

tide_status tide_embedding_bwd(int64_t tokens, const void* ids, int32_t ids_dtype, int64_t vocab, int64_t dim,
                               const void* dy, int32_t dtype, float scale, int32_t accumulate, void* dtable,
                               void* workspace, int64_t workspace_bytes, void* stream) {
  if (!embedding_ok(tokens, ids, ids_dtype, vocab, dim, dtype) || !rows_ok(dy, tokens, dtype) ||
      !rows_ok(dtable, vocab, dtype) || (accumulate != 0 && accumulate != 1))
    return TIDE_ERR_INVALID;
  const EmbeddingPlan p = embedding_plan(tokens, dim);
  if (!workspace_ok(workspace, workspace_bytes, p.bytes)) return TIDE_ERR_INVALID;
  const int size = size_of(dtype);
  const Range outs[] = {opt_range(dtable, vocab * dim * size), range_of(workspace, p.bytes)};
  const Range ins[] = {opt_range(ids, tokens * size_of(ids_dtype)), opt_range(dy, tokens * dim * size)};
  if (outputs_overlap(outs, ins)) return TIDE_ERR_INVALID;
  if (vocab == 0 || (accumulate && tokens == 0)) return TIDE_OK;
  char* ws = static_cast<char*>(workspace);
  const EmbeddingBwdArgs a{tokens,
                           vocab,
                           dim,
                           ids,
                           dy,
                           scale,
                           accumulate != 0,
                           dtable,
                           reinterpret_cast<int32_t*>(ws + p.token),
                           reinterpret_cast<int32_t*>(ws + p.row),
                           reinterpret_cast<int32_t*>(ws + p.count),
                           reinterpret_cast<int32_t*>(ws + p.last),
                           reinterpret_cast<EmbeddingRun*>(ws + p.runs),
                           reinterpret_cast<float*>(ws + p.partial)};
  return status_of(launch_embedding_bwd(a, dtype, ids_dtype, stream));
}

int32_t tide_step_last_hip_error(void) { return g_last_hip_error; }

#ifndef TIDE_BUILD_ID
#define TIDE_BUILD_ID "unknown"
#endif
const char* tide_step_build_id(void) { return TIDE_BUILD_ID; }

}  // extern "C"
