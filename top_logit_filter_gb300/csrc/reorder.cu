// topkp_beam_reorder: the rows of a request's states follow its beams.
//
// A thread owns one column (16 bytes, or fewer where alignment wants it) of
// all K rows of a request: it reads that column of every row that some other
// row wants, then writes it to those rows.  Because nobody else touches the
// column, the same code reorders in place, and each wanted row is read once
// however many children it has.
#include "common.cuh"
#include "decode.h"

namespace topkp {
namespace {

constexpr int kReorderThreads = 256;

template <typename U, int KMAX>
__global__ void __launch_bounds__(kReorderThreads) reorder_kernel(const __grid_constant__ ReorderArgs a) {
  __shared__ unsigned long long kids[TOPKP_MAX_BEAMS];  // rows that become row p
  __shared__ long long live[TOPKP_MAX_BEAMS];           // units of a block of row p that move
  __shared__ long long most;
  const topkp_state& st = a.st[blockIdx.z];
  const int64_t b = blockIdx.y;
  const int K = a.K, tid = threadIdx.x;
  const bool in_place = st.src == st.dst;
  if (tid < K) kids[tid] = 0ull;
  if (tid == 0) most = 0;
  __syncthreads();
  if (tid < K) {
    const int p = a.parent[b * K + tid];
    if (p >= 0 && p < K && !(in_place && p == tid)) atomicOr(&kids[p], 1ull << tid);
  }
  __syncthreads();
  const long long per_entry = st.entry_bytes / (long long)sizeof(U);
  if (tid < K) {
    long long n = kids[tid] ? st.entries : 0;
    if (n && a.lengths) n = min(n, (long long)max(a.lengths[b * K + tid], 0));
    live[tid] = n * per_entry;
    if (n) atomicMax(&most, n * per_entry);
  }
  __syncthreads();
  const long long width = most;
  if (width == 0) return;
  const long long total = width * st.blocks;
  const char* src = reinterpret_cast<const char*>(st.src) + b * K * st.src_row_stride;
  char* dst = reinterpret_cast<char*>(st.dst) + b * K * st.dst_row_stride;
  constexpr int COLS = KMAX <= 4 ? 4 : KMAX <= 8 ? 2 : 1;
  const long long step = (long long)gridDim.x * kReorderThreads;
  for (long long i0 = (long long)blockIdx.x * kReorderThreads + tid; i0 < total; i0 += step * COLS) {
    U r[COLS][KMAX];
    long long col[COLS], at[COLS];
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
      const long long i = i0 + c * step;
      long long blk = 0;
      if (st.blocks > 1) blk = total <= 0x7fffffffll ? (long long)((uint32_t)i / (uint32_t)width) : i / width;
      col[c] = i < total ? i - blk * width : width;  // a column past every live one moves nothing
      at[c] = blk;
#pragma unroll
      for (int p = 0; p < KMAX; ++p)
        if (p < K && col[c] < live[p])
          r[c][p] = *reinterpret_cast<const U*>(src + p * st.src_row_stride + blk * st.src_block_stride +
                                                col[c] * (long long)sizeof(U));
    }
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
      char* d = dst + at[c] * st.dst_block_stride + col[c] * (long long)sizeof(U);
#pragma unroll
      for (int p = 0; p < KMAX; ++p)
        if (p < K && col[c] < live[p]) {
          unsigned long long m = kids[p];
          while (m) {
            const int j = __ffsll((long long)m) - 1;
            m &= m - 1;
            *reinterpret_cast<U*>(d + j * st.dst_row_stride) = r[c][p];
          }
        }
    }
  }
}

template <typename U>
cudaError_t launch_unit(const ReorderArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.chunks, (unsigned)a.B, (unsigned)a.count);
  if (a.K <= 4) reorder_kernel<U, 4><<<grid, kReorderThreads, 0, s>>>(a);
  else if (a.K <= 8) reorder_kernel<U, 8><<<grid, kReorderThreads, 0, s>>>(a);
  else if (a.K <= 16) reorder_kernel<U, 16><<<grid, kReorderThreads, 0, s>>>(a);
  else reorder_kernel<U, 32><<<grid, kReorderThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

// CTAs of one request and state: enough for eight an SM over all of them, so
// that each has several rounds to spread the setup of its tables over.
int32_t reorder_chunks(int64_t units, int64_t groups) {
  const int64_t all = (units + kReorderThreads - 1) / kReorderThreads;
  const int64_t want = (8LL * 152 + groups - 1) / groups;
  const int64_t c = all < want ? all : want;
  return (int32_t)(c < 1 ? 1 : c);
}

cudaError_t launch_reorder(const ReorderArgs& a, cudaStream_t s) {
  if (a.K > 32) {  // registers for 64 rows: columns of 4 bytes at most
    const dim3 grid((unsigned)a.chunks, (unsigned)a.B, (unsigned)a.count);
    if (a.unit == 1) reorder_kernel<uint8_t, 64><<<grid, kReorderThreads, 0, s>>>(a);
    else reorder_kernel<uint32_t, 64><<<grid, kReorderThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  switch (a.unit) {
    case 16: return launch_unit<uint4>(a, s);
    case 4: return launch_unit<uint32_t>(a, s);
    default: return launch_unit<uint8_t>(a, s);
  }
}

}  // namespace topkp
