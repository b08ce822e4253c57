// Host/device interface of the decoding calls (topkp_decode.h): argument
// blocks and launchers, one per translation unit, as internal.h has them for
// the filter.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "topkp_decode.h"

namespace topkp {

// ------------------------------------------------------------ beam select
// One CTA scans a slice of a row, 256 threads of NV 16-byte vectors at a time.
constexpr int kBeamThreads = 256;

struct BeamArgs {
  const void* x;  // logits [B * K, ldx]
  int64_t ldx;
  const float* scores;
  const uint8_t* finished;  // or nullptr
  int64_t B;
  int32_t K, V, n, pad;
  int32_t nv;      // vectors of a chunk per thread: 1 or 4
  int32_t chunks;  // chunks of a slice
  int32_t slices;  // CTAs per row
  // workspace
  longlong2* stat;             // [rows][slices]: (c, sum of 2^(x log2 e - c) in 2^-38 units); sum 0 if nothing is finite
  uint32_t* units;             // [rows][unit_count]: order key of the largest logit of each 512 bytes
  uint32_t* pieces;            // [rows][unit_count / nv]: of each nv units; the units themselves if nv is 1
  int32_t unit_count;
  float* out_score;
  int32_t* out_parent;
  int32_t* out_token;
};

struct BeamPlan {
  int nv, chunks, slices;
  int unit_count;
  size_t stat_bytes, unit_bytes, piece_bytes;
};
BeamPlan plan_beam(int64_t rows, int64_t V, int esize, int num_sms);
cudaError_t launch_beam(topkp_dtype dt, const BeamArgs& a, cudaStream_t s);

// ---------------------------------------------------------------- reorder
constexpr int kReorderStates = 32;  // per launch (the descriptors travel as kernel parameters)

struct ReorderArgs {
  topkp_state st[kReorderStates];
  const int32_t* parent;
  const int32_t* lengths;  // or nullptr
  int64_t B;
  int32_t K;
  int32_t count;
  int32_t unit;   // bytes moved by a thread: 16, 4 or 1
  int32_t chunks; // grid.x
};
int32_t reorder_chunks(int64_t units, int64_t groups);
cudaError_t launch_reorder(const ReorderArgs& a, cudaStream_t s);

// ------------------------------------------------------------------ cache
struct CacheRowsArgs {
  const void* in[2];   // write: k, v rows
  void* out[2];        // read: k, v rows
  topkp_cache cache[2];
  const int64_t* slots;
  int64_t N, slots_end;
  int64_t token_stride[2], head_stride[2];  // of the dense rows, elements
  int32_t H, D, page_size;
  int32_t sides;  // 1 (keys alone) or 2
  int32_t vec;    // elements moved by a thread: 8 or 1
  // set by the launcher
  int32_t tokens;       // tokens of a CTA at a time
  uint32_t page_mul;    // reciprocal of page_size, 0: divide
  int32_t page_shift;
};
cudaError_t launch_cache_write(topkp_dtype dt, const CacheRowsArgs& a, cudaStream_t s);
cudaError_t launch_cache_read(topkp_dtype dt, const CacheRowsArgs& a, cudaStream_t s);

// ----------------------------------------------------------------- verify
constexpr int kVerifyThreads = 512;
enum { kVerifyRatio, kVerifyCertain, kVerifyGreedy };

struct VerifyArgs {
  const void* target;
  const void* draft;      // or nullptr
  int64_t t_batch, t_node, d_batch, d_node;
  const int32_t* tokens;  // [B, T]
  const int32_t* parent;  // [B, T], or nullptr (a chain)
  const int32_t* nodes;   // or nullptr
  const float* uniform;   // [B, T], or nullptr together with race (greedy)
  const float* race;
  int64_t ld_race;
  float eps;
  int64_t B;
  int32_t T, V;
  int32_t cs;     // CTAs of a request
  int32_t ahead;  // nodes of a step
  int32_t whole;  // rows and variates may be read 16 bytes at a time
  int32_t* count;
  int32_t* path;
  int32_t* token;
  float* logprob;  // or nullptr
};
void verify_plan(int64_t B, int64_t V, int esize, bool draft, int num_sms, int* cs, int* ahead);
cudaError_t launch_verify(topkp_dtype dt, const VerifyArgs& a, cudaStream_t s);

// ------------------------------------------------------------------ pages
constexpr int kPageStates = 128;  // per launch (the descriptors travel as kernel parameters)
constexpr int kForkThreads = 1024, kForkCtas = 8;

struct Reciprocal {
  uint32_t mul;  // 0: divide by 1
  int32_t shift;
};
struct ForkArgs {
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* source;
  const int32_t* grow;  // or nullptr: grow_all
  const int32_t* refs;
  int32_t* table_out;
  int32_t* refs_out;
  int32_t* missing;
  // workspace
  int32_t* hold;   // [pages] references that do not come from the old rows, or are carried over
  int32_t* claim;  // [pages] the first new row whose partial last page it is
  int32_t* fresh;  // [pages] free pages in the order they are given out
  int4* copies;    // [N] source page, its copy, tokens (0: none)
  int64_t ld, ld_out;
  int64_t pages;
  int32_t R, N, M, page_size, grow_all;
  Reciprocal by_page, by_columns;  // set by the launcher
};
struct PageState {
  char* data;
  int64_t page_stride, block_stride, blocks, entry_bytes;
  int32_t unit;  // bytes moved by a thread: 16, 4 or 1
};
struct CopyArgs {
  PageState st[kPageStates];
  const int4* copies;
  int32_t count, N, page_size;
  int32_t chunks;  // set by the launcher
};
struct CompactArgs {
  PageState st[kPageStates];
  const int32_t* table;  // or nullptr
  const int32_t* start;
  const int32_t* keep;
  const int32_t* kept;
  int64_t ld, pages;
  int32_t B, W, M, page_size, count;
  int32_t chunks;  // set by the launcher
};
size_t fork_workspace(int64_t N, int64_t pages);
cudaError_t launch_fork(const ForkArgs& a, cudaStream_t s);
cudaError_t launch_page_copy(const CopyArgs& a, cudaStream_t s);
cudaError_t launch_compact(const CompactArgs& a, cudaStream_t s);

// -------------------------------------------------------------- attention
struct AttnPlan {
  int splits;         // parts of a request's tokens
  int per;            // tiles of 64 tokens of a part
  size_t part_bytes;  // workspace: partial outputs and their (lse) rows
  double us;          // estimated
};
AttnPlan plan_attention(const topkp_tree_attention_args& a, int num_sms);
// part_o: [splits][B * T * Hq][D] float, part_l: [splits][B * T * Hq] float
cudaError_t launch_attention(const topkp_tree_attention_args& a, const AttnPlan& p, int* launches, cudaStream_t s);
struct SharedPlan {
  int64_t groups;       // 0: every request by itself
  AttnPlan front, own;  // splits and tiles of the shared tokens, and of each request's own
  size_t part_bytes;
};
SharedPlan plan_shared(const topkp_tree_attention_args& a, int64_t groups, int64_t max_shared, int num_sms);
cudaError_t launch_shared(const topkp_tree_attention_args& a, const int32_t* shared, const SharedPlan& p, int* launches, cudaStream_t s);

}  // namespace topkp
