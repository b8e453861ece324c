// Entry points of libtide_step.so for what tokens pass through in a block -- experts, rotary positions,
// dropout --: argument checks, then kernel launches.  As in step_api.cpp nothing is allocated and no state
// is kept.
#include <cmath>

#include "step_checks.h"
#include "step_internal.h"

namespace tide_step {
namespace {

// ---------------------------------------------------------------------------------------------
// Experts
// ---------------------------------------------------------------------------------------------

bool pairs_ok(int64_t tokens, int32_t choices) {
  return tokens >= 0 && choices >= 1 && choices <= TIDE_MAX_CHOICES && tokens < kInt31 / choices;
}
bool experts_ok(int32_t experts) { return experts >= 1 && experts <= TIDE_MAX_EXPERTS; }
bool numbers_ok(const int32_t* p, int64_t n) { return n == 0 || (p != nullptr && aligned(p, 4)); }

int64_t sort_bytes(int64_t pairs, int32_t experts) {
  const int parts = expert_parts(pairs, experts);
  return parts > 1 ? (int64_t(parts) * experts * 4 + 15) / 16 * 16 : 0;
}
// What the calls on rows have in common: sizes, and both sides' matrices.
bool rows_args_ok(int64_t tokens, int32_t choices, int64_t dim, int64_t rows, int32_t dtype, const void* by_token,
                  int64_t token_stride, const void* sorted, int64_t sorted_stride, const int32_t* place) {
  return pairs_ok(tokens, choices) && rows >= 0 && rows < kInt31 && matrix_ok(tokens, dim) && matrix_ok(rows, dim) &&
         float_type(dtype) && strided_ok(by_token, tokens, dim, token_stride, dtype) &&
         strided_ok(sorted, rows, dim, sorted_stride, dtype) && numbers_ok(place, tokens);
}

}  // namespace
}  // namespace tide_step

using namespace tide_step;

extern "C" {

int64_t tide_expert_rows(int64_t tokens, int32_t choices, int32_t experts, int32_t align) {
  if (!pairs_ok(tokens, choices) || !experts_ok(experts) || align < 1) return -1;
  const int64_t pairs = tokens * choices, rows = pairs + (experts < pairs ? experts : pairs) * int64_t(align - 1);
  return rows < kInt31 ? rows : -1;
}

int64_t tide_expert_sort_workspace(int64_t tokens, int32_t choices, int32_t experts) {
  if (!pairs_ok(tokens, choices) || !experts_ok(experts)) return -1;
  return sort_bytes(tokens * choices, experts);
}

tide_status tide_expert_sort(int64_t tokens, int32_t choices, const void* ids, int32_t ids_dtype, int32_t experts,
                             int32_t align, int32_t* place, int32_t* source, int64_t rows, int32_t* offsets,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  const int64_t least = tide_expert_rows(tokens, choices, experts, align);
  if (least < 0 || rows < least || rows >= kInt31 || (ids_dtype != TIDE_INT32 && ids_dtype != TIDE_INT64) ||
      (tokens > 0 && (ids == nullptr || !aligned(ids, size_of(ids_dtype)))) || !numbers_ok(place, tokens) ||
      !numbers_ok(source, rows) || !numbers_ok(offsets, 1))
    return TIDE_ERR_INVALID;
  const int64_t pairs = tokens * choices, need = sort_bytes(pairs, experts);
  if (!workspace_ok(workspace, workspace_bytes, need)) return TIDE_ERR_INVALID;
  const Range outs[] = {range_of(place, pairs * 4), range_of(source, rows * 4),
                        range_of(offsets, (int64_t(experts) + 1) * 4), need > 0 ? range_of(workspace, need) : Range{0, 0}};
  const Range ins[] = {range_of(ids, pairs * size_of(ids_dtype))};
  if (outputs_overlap(outs, ins)) return TIDE_ERR_INVALID;
  const ExpertSortArgs a{pairs, ids, experts, align, place, source, rows, offsets, static_cast<int32_t*>(workspace)};
  return status_of(launch_expert_sort(a, ids_dtype, stream));
}

tide_status tide_expert_dispatch(int64_t tokens, int32_t choices, int64_t dim, const void* x, int64_t x_stride,
                                 int32_t dtype, const int32_t* place, const int32_t* source, int64_t rows, void* out,
                                 int64_t out_stride, void* stream) {
  if (!rows_args_ok(tokens, choices, dim, rows, dtype, x, x_stride, out, out_stride, place) ||
      !numbers_ok(source, rows))
    return TIDE_ERR_INVALID;
  if (rows == 0) return TIDE_OK;
  const int size = size_of(dtype);
  const Range outs[] = {range_of(out, rows, dim, out_stride, size)};
  const Range ins[] = {range_of(x, tokens, dim, x_stride, size), range_of(place, tokens * choices * 4),
                       range_of(source, rows * 4)};
  if (outputs_overlap(outs, ins)) return TIDE_ERR_INVALID;
  ExpertRowsArgs a{};
  a.tokens = tokens, a.dim = dim, a.rows = rows, a.choices = choices, a.place = place, a.source = source;
  a.x = x, a.x_stride = x_stride, a.out = out, a.out_stride = out_stride;
  return status_of(launch_expert_dispatch(a, dtype, stream));
}

tide_status tide_expert_combine(int64_t tokens, int32_t choices, int64_t dim, const void* x, int64_t x_stride,
                                int64_t rows, int32_t dtype, const void* weights, int32_t weight_dtype,
                                const int32_t* place, void* y, int64_t y_stride, void* stream) {
  if (!rows_args_ok(tokens, choices, dim, rows, dtype, y, y_stride, x, x_stride, place) || !float_type(weight_dtype) ||
      !vector_ok(weights, weight_dtype))
    return TIDE_ERR_INVALID;
  if (tokens == 0) return TIDE_OK;
  const int size = size_of(dtype);
  const Range outs[] = {range_of(y, tokens, dim, y_stride, size)};
  const Range ins[] = {range_of(x, rows, dim, x_stride, size), range_of(place, tokens * choices * 4),
                       opt_range(weights, tokens * choices * size_of(weight_dtype))};
  if (outputs_overlap(outs, ins)) return TIDE_ERR_INVALID;
  ExpertRowsArgs a{};
  a.tokens = tokens, a.dim = dim, a.rows = rows, a.choices = choices, a.place = place, a.weights = weights;
  a.x = x, a.x_stride = x_stride, a.out = y, a.out_stride = y_stride;
  return status_of(launch_expert_combine(a, dtype, weight_dtype, stream));
}

tide_status tide_expert_combine_bwd(int64_t tokens, int32_t choices, int64_t dim, const void* dy, int64_t dy_stride,
                                    const void* x, int64_t x_stride, int64_t rows, int32_t dtype, const void* weights,
                                    int32_t weight_dtype, const int32_t* place, const int32_t* source, void* dx,
                                    int64_t dx_stride, void* dweights, void* stream) {
  if (!rows_args_ok(tokens, choices, dim, rows, dtype, dy, dy_stride, x, x_stride, place) ||
      !strided_ok(dx, rows, dim, dx_stride, dtype) || !float_type(weight_dtype) || !vector_ok(weights, weight_dtype) ||
      !vector_ok(dweights, weight_dtype) || (tokens > 0 && (weights == nullptr || dweights == nullptr)) ||
      !numbers_ok(source, rows))
    return TIDE_ERR_INVALID;
  const int size = size_of(dtype);
  const int64_t wbytes = tokens * choices * size_of(weight_dtype);
  const Range rx = range_of(x, rows, dim, x_stride, size);
  const bool in_place = dx == x && (dx_stride == x_stride || rows <= 1);
  const Range outs[] = {range_of(dx, rows, dim, dx_stride, size), opt_range(dweights, wbytes)};
  const Range ins[] = {in_place ? Range{0, 0} : rx, range_of(dy, tokens, dim, dy_stride, size),
                       opt_range(weights, wbytes), range_of(place, tokens * choices * 4), range_of(source, rows * 4)};
  if (outputs_overlap(outs, ins)) return TIDE_ERR_INVALID;
  if (tokens == 0 && rows == 0) return TIDE_OK;
  ExpertRowsArgs a{};
  a.tokens = tokens, a.dim = dim, a.rows = rows, a.choices = choices, a.place = place, a.source = source;
  a.x = x, a.x_stride = x_stride, a.dy = dy, a.dy_stride = dy_stride, a.weights = weights;
  a.out = dx, a.out_stride = dx_stride, a.dweights = dweights;
  return status_of(launch_expert_combine_bwd(a, dtype, weight_dtype, stream));
}

}  // extern "C"

// ---------------------------------------------------------------------------------------------
// Rotary positions
// ---------------------------------------------------------------------------------------------

namespace tide_step {
namespace {

// Vectors of `dim` elements by token and head.
struct Heads {
  int64_t tokens, heads, dim, token, head;
  int64_t elems() const {  // from the first to behind the last
    return tokens == 0 || heads == 0 ? 0 : (tokens - 1) * token + (heads - 1) * head + dim;
  }
  bool strides_ok() const {
    const auto fits = [](int64_t n, int64_t stride) { return n <= 1 || (stride >= 0 && stride <= kMaxElems / n); };
    return fits(tokens, token) && fits(heads, head);
  }
  // No element lies over another: heads within a token's stride, or tokens within a head's.
  bool apart() const {
    const int64_t t = tokens <= 1 ? kMaxElems : token, h = heads <= 1 ? kMaxElems : head;
    return h >= dim && t >= dim && ((tokens <= 1 || t >= (heads - 1) * (heads <= 1 ? 0 : head) + dim) ||
                                    (heads <= 1 || h >= (tokens - 1) * (tokens <= 1 ? 0 : token) + dim));
  }
  // As rows with gaps between them where the heads of a token, or the tokens of a head, touch.
  Range range(const void* p, int size) const {
    if (heads <= 1 || head == dim) return range_of(p, tokens, heads * dim, tokens <= 1 ? 0 : token, size);
    if (tokens <= 1 || token == dim) return range_of(p, heads, tokens * dim, head, size);
    return range_of(p, elems() * size);
  }
};

}  // namespace
}  // namespace tide_step

extern "C" {

tide_status tide_rotary(int64_t tokens, int64_t heads, int64_t dim, const void* x, int64_t x_token_stride,
                        int64_t x_head_stride, int32_t dtype, const void* positions, int32_t positions_dtype,
                        int32_t axes, const int32_t* sections, const double* freqs, int32_t pairing, int32_t inverse,
                        void* out, int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  if (tokens < 0 || heads < 0 || tokens >= kInt31 || heads > TIDE_ROTARY_MAX_HEADS || dim < 1 || dim > TIDE_ROTARY_MAX_DIM ||
      (tokens > 0 && heads > kMaxElems / dim / tokens) || !float_type(dtype) ||
      (positions_dtype != TIDE_INT32 && positions_dtype != TIDE_INT64 && positions_dtype != TIDE_FP32) || axes < 1 ||
      axes > TIDE_ROTARY_MAX_AXES || sections == nullptr ||
      (pairing != TIDE_ROTARY_HALVES && pairing != TIDE_ROTARY_NEIGHBOURS) || (inverse != 0 && inverse != 1))
    return TIDE_ERR_INVALID;
  RotaryArgs a{};
  for (int32_t i = 0; i < axes; ++i) {
    if (sections[i] < 1 || sections[i] > dim / 2 - a.pairs) return TIDE_ERR_INVALID;
    a.pairs += sections[i];
    a.ends[i] = a.pairs;
  }
  if (tokens == 0 || heads == 0) return TIDE_OK;
  const Heads in{tokens, heads, dim, x_token_stride, x_head_stride}, to{tokens, heads, dim, out_token_stride, out_head_stride};
  const int size = size_of(dtype);
  if (x == nullptr || out == nullptr || positions == nullptr || freqs == nullptr || !aligned(x, size) ||
      !aligned(out, size) || !aligned(positions, size_of(positions_dtype)) || !aligned(freqs, 8) || !in.strides_ok() ||
      !to.strides_ok() || !to.apart())
    return TIDE_ERR_INVALID;
  const bool in_place = x == out && (tokens <= 1 || x_token_stride == out_token_stride) &&
                        (heads <= 1 || x_head_stride == out_head_stride);
  const Range outs[] = {to.range(out, size)};
  const Range ins[] = {in_place ? Range{0, 0} : in.range(x, size),
                       range_of(positions, axes * tokens * size_of(positions_dtype)), range_of(freqs, a.pairs * 8)};
  if (outputs_overlap(outs, ins)) return TIDE_ERR_INVALID;
  a.tokens = tokens, a.heads = heads, a.dim = int32_t(dim), a.axes = axes;
  a.x = x, a.x_token = x_token_stride, a.x_head = x_head_stride;
  a.positions = positions, a.freqs = freqs, a.sign = inverse ? -1.0f : 1.0f;
  a.out = out, a.out_token = out_token_stride, a.out_head = out_head_stride;
  return status_of(launch_rotary(a, dtype, positions_dtype, pairing, stream));
}

// ---------------------------------------------------------------------------------------------
// Dropout
// ---------------------------------------------------------------------------------------------

tide_status tide_dropout(int64_t rows, int64_t cols, const void* x, int64_t x_stride, int32_t dtype, double p,
                         uint64_t seed, const int64_t* seed_device, int64_t offset, const void* residual,
                         int64_t residual_stride, void* out, int64_t out_stride, void* stream) {
  if (rows < 0 || cols < 1 || cols > kMaxElems || rows > kMaxElems / cols || !float_type(dtype) || !(p >= 0 && p <= 1) ||
      !aligned(seed_device, 8) || offset < 0 || offset > (int64_t(1) << 62) - rows * cols ||
      !strided_ok(x, rows, cols, x_stride, dtype) || !strided_ok(out, rows, cols, out_stride, dtype) ||
      (residual != nullptr && !strided_ok(residual, rows, cols, residual_stride, dtype)))
    return TIDE_ERR_INVALID;
  if (rows == 0) return TIDE_OK;
  const int size = size_of(dtype);
  const auto same = [&](const void* q, int64_t stride) { return q == out && (stride == out_stride || rows == 1); };
  const Range none{0, 0}, outs[] = {range_of(out, rows, cols, out_stride, size)};
  const Range ins[] = {same(x, x_stride) ? none : range_of(x, rows, cols, x_stride, size),
                       residual == nullptr || same(residual, residual_stride)
                           ? none
                           : range_of(residual, rows, cols, residual_stride, size),
                       opt_range(seed_device, 8)};
  if (outputs_overlap(outs, ins)) return TIDE_ERR_INVALID;
  const double t = std::nearbyint(p * 65536.0);
  // the scale of an element that is kept: in 64 bits, rounded to fp32 (t = 65536 keeps none)
  const float scale = t < 65536.0 ? float(65536.0 / (65536.0 - t)) : 0.0f;
  const DropoutArgs a{rows, cols, x, x_stride, uint32_t(t), scale, seed, seed_device, offset,
                      residual, residual_stride, out, out_stride};
  return status_of(launch_dropout(a, dtype, stream));
}

}  // extern "C"
