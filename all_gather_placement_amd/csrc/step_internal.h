// Declarations shared by the entry points and the kernels of libtide_step.so.
#pragma once

#include <stdint.h>

#include "../../include/tide_step.h"

namespace tide_step {

// ---------------------------------------------------------------------------------------------
// Gradient norm and clipping
// ---------------------------------------------------------------------------------------------

// A tensor is cut into chunks of 16 KiB, four 16-byte vectors for each of 256 threads; the last
// chunk of a tensor holds what is left.  A launch walks the chunks of up to kNormBatch tensors in
// order.  Tensors are named in the kernel's arguments (4 KiB), so a call needs no device table, copy
// or event.
constexpr int kNormThreads = 256;
constexpr int kNormChunkBytes = 16384;
constexpr int kNormWgs = 1024;           // of a sum: workgroup b takes chunks b, b + grid, ... (196 us; 2048: 212)
constexpr int kNormMaxWgs = 1 << 20;     // of clipping: a workgroup lives for one chunk
// A call of up to so many chunks is one workgroup's, in one launch: as fast on the GPU (8 chunks: sum 3.7 us,
// clipping 7.1, in two and three launches 4.3 and 6.7; 16 chunks 5.3 and 11.4 against 4.4 and 6.7).
constexpr int kNormOneWgChunks = 8;
// Clipping of up to so many chunks (gradients and outputs fit the last-level cache) by one launch adds up
// the partial sums in each of its workgroups, instead of a launch for that: 160 chunks 6.6 us instead of
// 7.5, 1960 chunks 22.8 instead of 27.1, 7380 chunks 58.9 instead of 63.9.
constexpr int kNormClipAddsChunks = 8192;
constexpr int64_t kMaxNormElems = int64_t(1) << 42;
constexpr int norm_chunk_elems(int dtype) { return kNormChunkBytes / (dtype == TIDE_BF16 ? 2 : 4); }

struct NormEntry {
  const void* p;
  uint32_t first;  // chunk of the launch that the tensor begins with
  uint32_t last;   // elements of the tensor's last chunk
};
constexpr int kNormBatch = 250;
struct NormTable {
  int32_t count;
  uint32_t chunks;
  double* sumsq;  // not NULL (one of the two): the launch is one workgroup and its sum is the result
  float* norm;
  NormEntry e[kNormBatch];
};
static_assert(sizeof(NormTable) <= 4032, "kernel arguments stay within 4 KiB");

struct ClipEntry {
  const void* p;
  void* out;
  uint32_t first;
  uint32_t last;
};
constexpr int kClipBatch = 160;
struct ClipTable {
  int32_t count;
  uint32_t chunks;
  const double* partial;  // not NULL: each workgroup adds these `partials` sums; the first writes *sum_to
  int32_t partials;
  double* sum_to;  // not NULL without `partial`: the launch is one workgroup, which first forms that sum
  ClipEntry e[kClipBatch];
};
static_assert(sizeof(ClipTable) <= 4032, "kernel arguments stay within 4 KiB");

// Each returns a hipError_t.
int launch_norm_partial(const NormTable& t, int dtype, double* partial, int grid, void* stream);
int launch_norm_finish(const double* partial, int n, double* sumsq, float* norm, void* stream);  // nothing to write: no launch
int launch_clip(const ClipTable& t, int dtype, const double* sumsq, double max_norm, float* norm, int grid,
                void* stream);

// ---------------------------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------------------------

struct LayerNormArgs {
  int64_t rows, cols;
  const void* x;
  int64_t x_stride;
  const void* weight;
  const void* bias;
  float eps;
  void* y;
  int64_t y_stride;
  float* mean;
  float* rstd;
};
int launch_layer_norm(const LayerNormArgs& a, int dtype, int param_dtype, void* stream);

struct LayerNormBwdArgs {
  int64_t rows, cols;
  const void* dy;
  int64_t dy_stride;
  const void* x;
  int64_t x_stride;
  const void* weight;
  const float* mean;
  const float* rstd;
  void* dx;
  int64_t dx_stride;
  void* dweight;
  void* dbias;
  float* partial;  // [groups][2][layer_norm_bwd_padded(cols)]: each workgroup's sums over its rows
};
// Workgroups of the gradient's first kernel, each leaving a partial sum of every column.
int layer_norm_bwd_groups(int64_t rows, int64_t cols, int dtype);
// Columns of a partial sum: up to whole 16-byte vectors.
constexpr int64_t layer_norm_bwd_padded(int64_t cols) { return (cols + 3) / 4 * 4; }
int launch_layer_norm_bwd(const LayerNormBwdArgs& a, int dtype, int param_dtype, void* stream);

// ---------------------------------------------------------------------------------------------
// Embedding
// ---------------------------------------------------------------------------------------------

int launch_embedding(int64_t tokens, const void* ids, int ids_dtype, int64_t vocab, int64_t dim, const void* table,
                     int dtype, float scale, void* out, void* stream);

// The gradient's sort gives each of 2^shift workgroups the table rows v with v mod 2^shift its number;
// it finds their tokens by reading all ids.  There is one for each compute unit at least, and none has
// more than kSortMaxRows rows.
constexpr int kSortMaxRows = 512;
constexpr int kSortMinShift = 8;
inline int sort_shift(int64_t vocab) {
  int s = kSortMinShift;
  while (vocab > int64_t(kSortMaxRows) << s) ++s;
  return s;
}
// Sorted tokens are summed in pieces of kPiece.  A run of equal ids that crosses a border of pieces
// leaves fp32 partial sums, at most two for each piece, that a second kernel adds in order.
constexpr int kPiece = 32;
constexpr int kShortRun = 16;  // pieces of a run that one wave adds

struct EmbeddingRun {
  int32_t first, last, row;  // pieces, and the table's row
};
struct EmbeddingBwdArgs {
  int64_t tokens, vocab, dim;
  const void* ids;
  const void* dy;
  float scale;
  bool accumulate;
  void* dtable;
  int32_t* sorted_token;  // [tokens]
  int32_t* sorted_row;    // [tokens]
  int32_t* num_sorted;    // [3]: tokens inside the table, short and long runs that cross a border of pieces
  int32_t* last_piece;    // [pieces]: where such a run begins, the piece it ends in
  EmbeddingRun* runs;     // [pieces]: such runs in any order, the long ones from the end on
  float* partial;         // [pieces][2][dim]
};
int launch_embedding_bwd(const EmbeddingBwdArgs& a, int dtype, int ids_dtype, void* stream);

}  // namespace tide_step
