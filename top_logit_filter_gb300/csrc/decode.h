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

// -------------------------------------------------------------- attention
struct AttnPlan {
  int splits;         // parts of a request's tokens
  int per;            // tiles of 64 tokens of a part
  size_t part_bytes;  // workspace: partial outputs and their (lse) rows
};
AttnPlan plan_attention(const topkp_tree_attention_args& a, int num_sms);
// part_o: [splits][B * T * Hq][D] float, part_l: [splits][B * T * Hq] float
cudaError_t launch_attention(const topkp_tree_attention_args& a, const AttnPlan& p, int* launches, cudaStream_t s);

}  // namespace topkp
