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

// ---------------------------------------------------------------------------------------------
// Experts
// ---------------------------------------------------------------------------------------------

// The sort cuts the pairs into parts, one for each workgroup; the first launch counts each part's pairs
// of every expert, the second places them.
// Times are of the call in a graph unless stated, of 128 experts unless stated.
constexpr int kExpertOnePart = 4096;         // pairs that one workgroup sorts, in one launch (8.3 us, and 8.1 by calls one after
                                             // another, which two launches make 9.0 to 10.5, though they take 7.9 in a graph)
constexpr int kExpertMinPart = 1024;         // of several parts (65536 pairs: 8.4 us; parts of 4096 11.2)
constexpr int kExpertMaxParts = 256;         // as many as there are compute units (1600000 pairs: 20.9 us; 128 parts 25.2, 512
                                             // 24.6; 524288 pairs: 13.0, 13.0, 17.7)
constexpr int kExpertMaxCounts = 1 << 16;    // parts * experts, all of which each workgroup reads (524288 pairs of 512
                                             // experts: 128 parts 17.6 us, 256 20.6; 65536 of 2048: 32 parts 30.8, 64 40.7, though
                                             // 524288 take 57.7 instead of 64.5 there)
inline int expert_parts(int64_t pairs, int experts) {
  if (pairs <= kExpertOnePart) return 1;
  const int64_t most = kExpertMaxCounts / experts < kExpertMaxParts ? kExpertMaxCounts / experts : kExpertMaxParts;
  const int64_t n = (pairs + kExpertMinPart - 1) / kExpertMinPart;
  return int(n < most ? n : most);
}

struct ExpertSortArgs {
  int64_t pairs;
  const void* ids;
  int32_t experts, align;
  int32_t* place;
  int32_t* source;
  int64_t rows;
  int32_t* offsets;
  int32_t* counts;  // [parts][experts]; none for one part
};
int launch_expert_sort(const ExpertSortArgs& a, int ids_dtype, void* stream);

struct ExpertRowsArgs {
  int64_t tokens, dim, rows;
  int32_t choices;
  const int32_t* place;
  const int32_t* source;
  const void* x;  // tokens' rows of dispatch, the sorted buffer of the others
  int64_t x_stride;
  const void* dy;
  int64_t dy_stride;
  const void* weights;
  void* out;  // the sorted buffer of dispatch and of combine's gradient
  int64_t out_stride;
  void* dweights;
};
int launch_expert_dispatch(const ExpertRowsArgs& a, int dtype, void* stream);
int launch_expert_combine(const ExpertRowsArgs& a, int dtype, int weight_dtype, void* stream);
int launch_expert_combine_bwd(const ExpertRowsArgs& a, int dtype, int weight_dtype, void* stream);

// ---------------------------------------------------------------------------------------------
// Rotary positions
// ---------------------------------------------------------------------------------------------

struct RotaryArgs {
  int64_t tokens, heads;
  int32_t dim, pairs, axes;
  int32_t ends[TIDE_ROTARY_MAX_AXES];  // the pair behind each axis's last
  const void* x;
  int64_t x_token, x_head;
  const void* positions;
  const double* freqs;
  float sign;
  void* out;
  int64_t out_token, out_head;
};
int launch_rotary(const RotaryArgs& a, int dtype, int positions_dtype, int pairing, void* stream);

// ---------------------------------------------------------------------------------------------
// Dropout
// ---------------------------------------------------------------------------------------------

struct DropoutArgs {
  int64_t rows, cols;
  const void* x;
  int64_t x_stride;
  uint32_t threshold;
  float scale;
  uint64_t seed;
  const int64_t* seed_device;
  int64_t offset;
  const void* residual;
  int64_t residual_stride;
  void* out;
  int64_t out_stride;
};
int launch_dropout(const DropoutArgs& a, int dtype, void* stream);

}  // namespace tide_step
