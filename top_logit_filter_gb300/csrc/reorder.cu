// topkp_beam_reorder: the rows of a request's states follow its beams.
//
// A thread owns one column (16 bytes, or fewer where alignment wants it) of
// all K rows of a request: it reads that column of every row that some other
// row wants, then writes it to those rows.  Because nobody else touches the
// column, the same code reorders in place, and each wanted row is read once
// however many children it has.  Bound by DRAM: 1.47 GB of bf16 caches
// [256, 1536, 8, 128] x 4 in place, ragged lengths, 251 us (5.9 TB/s).
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
  const long long step = (long long)gridDim.x * kReorderThreads;
  for (long long i = (long long)blockIdx.x * kReorderThreads + tid; i < total; i += step) {
    long long blk = 0;
    if (st.blocks > 1) blk = total <= 0x7fffffffll ? (long long)((uint32_t)i / (uint32_t)width) : i / width;
    const long long col = i - blk * width;
    const char* s = src + blk * st.src_block_stride + col * (long long)sizeof(U);
    char* d = dst + blk * st.dst_block_stride + col * (long long)sizeof(U);
    U r[KMAX];
#pragma unroll
    for (int p = 0; p < KMAX; ++p)
      if (p < K && col < live[p]) r[p] = *reinterpret_cast<const U*>(s + p * st.src_row_stride);
#pragma unroll
    for (int p = 0; p < KMAX; ++p)
      if (p < K && col < live[p]) {
        unsigned long long m = kids[p];
        while (m) {
          const int j = __ffsll((long long)m) - 1;
          m &= m - 1;
          *reinterpret_cast<U*>(d + j * st.dst_row_stride) = r[p];
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

// CTAs of one request and state, from the columns of a row and the number of
// (request, state) pairs.  A CTA sets up its tables (two dependent reads and
// four barriers) before it moves anything: eight columns a thread spread that
// where there is work for it.
int32_t reorder_chunks(int64_t units, int64_t groups) {
  int64_t rounds = 8;
  while (rounds > 1 && groups * units < rounds * kReorderThreads * 8 * 152) rounds /= 2;
  const int64_t c = (units + kReorderThreads * rounds - 1) / (kReorderThreads * rounds);
  return (int32_t)(c < 1 ? 1 : c > 65535 ? 65535 : c);
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
