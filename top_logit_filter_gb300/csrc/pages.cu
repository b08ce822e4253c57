// topkp_cache_fork and topkp_cache_compact: pages of a cache follow the
// requests that go on, and the accepted tokens of a drafted tree move up.
//
// Forking is bookkeeping, then copies.  The bookkeeping is one cluster of
// eight CTAs, since its steps depend on one another and a cluster barrier is
// the cheapest join there is: references that stay, with integer atomics
// (their order changes nothing); who claims a partly filled page; free pages
// counted and ranked in the order of their numbers; the new table.  Every CTA
// works out all rows' demands for itself rather than wait for another.  The
// copies, a CTA for a piece of a page of a state, are launched under the
// bookkeeping's tail and bound by DRAM.
//
// Compacting: a thread owns one column (16 bytes, or fewer where alignment
// wants it) of an entry and takes a request's kept tokens in order, eight
// reads before their eight writes.  A token only moves to a lower place, and
// every place that is read lies behind those written so far, so the same
// code is right in place.
#include <limits.h>

#include "common.cuh"
#include "decode.h"

namespace topkp {
namespace {

constexpr int kFW = kForkThreads / 32;

// Exclusive prefix sum over the CTA; *total gets the sum of all threads.
__device__ __forceinline__ int scan(int v, int* total, int* ws) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // ws may still be read from an earlier call
  if (lane == 31) ws[warp] = x;
  __syncthreads();
  const int w = ws[lane];  // kFW == 32
  int s = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  return __shfl_sync(0xffffffffu, s - w, warp) + x - v;
}
static_assert(kFW == 32, "a lane for each warp's sum");

__device__ __forceinline__ void all_sync() {
  __syncwarp();
  cluster_sync_all();
}

// What a new row takes over and asks for.
struct Taken {
  int source;  // old row, or -1
  int full;    // whole pages
  int part;    // tokens of the last page, where it is partly filled
  int last;    // that page, or -1
  int need;    // pages the row will have
};
__device__ __forceinline__ int clamped_length(const ForkArgs& a, int row) {
  const long long cap = (long long)a.M * a.page_size;
  return (int)min((long long)max(a.lengths[row], 0), cap);
}
__device__ __forceinline__ Taken take(const ForkArgs& a, int n) {
  Taken t;
  const int s = a.source[n];
  t.source = s >= 0 && s < a.R ? s : -1;
  const int len = t.source < 0 ? 0 : clamped_length(a, s);
  t.full = len / a.page_size;
  t.part = len - t.full * a.page_size;
  t.last = -1;
  if (t.part) {
    const int g = a.table[(int64_t)s * a.ld + t.full];
    if (g >= 0 && g < a.pages) t.last = g;
  }
  const long long want = (long long)len + max(a.grow ? a.grow[n] : a.grow_all, 0);
  t.need = (int)min((long long)a.M, (want + a.page_size - 1) / a.page_size);
  return t;
}
// Whether row n goes on with its partly filled page: the first to claim it,
// and nobody else holds it.
__device__ __forceinline__ bool keeps(const ForkArgs& a, const Taken& t, int n) {
  return t.last >= 0 && __ldcg(&a.claim[t.last]) == n && __ldcg(&a.hold[t.last]) == 0;
}

__global__ void __launch_bounds__(kForkThreads) fork_kernel(const __grid_constant__ ForkArgs a) {
  extern __shared__ int fork_smem[];
  int* children = fork_smem;       // [R] new rows of an old one
  int* base = fork_smem + a.R;     // [N] the first of a row's fresh pages
  __shared__ int ws[32], free_pages[kForkCtas];
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_ctarank();
  const int all = kForkThreads * kForkCtas, me = (int)rank * kForkThreads + tid;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int64_t p = me; p < a.pages; p += all) {
    __stcg(&a.hold[p], a.refs[p]);
    __stcg(&a.claim[p], INT_MAX);
  }
  for (int r = tid; r < a.R; r += kForkThreads) children[r] = 0;
  __syncthreads();
  for (int n = tid; n < a.N; n += kForkThreads) {
    const int s = a.source[n];
    if (s >= 0 && s < a.R) atomicAdd(&children[s], 1);
  }
  all_sync();
  // what the old rows held goes, what the new ones share comes
  const int entries = a.R * a.M;
  for (int x = me; x < entries; x += all) {
    const int r = x / a.M, i = x - r * a.M;
    const int p = a.table[(int64_t)r * a.ld + i];
    if (p < 0 || p >= a.pages) continue;
    const int change = (i < clamped_length(a, r) / a.page_size ? children[r] : 0) - 1;
    if (change) atomicAdd(&a.hold[p], change);
  }
  for (int n = me; n < a.N; n += all) {
    const Taken t = take(a, n);
    if (t.last >= 0) atomicMin(&a.claim[t.last], n);
  }
  all_sync();
  // every row's demand, and the free pages of this CTA's part of the pool
  int total = 0;
  for (int n0 = 0; n0 < a.N; n0 += kForkThreads) {
    const int n = n0 + tid;
    int want = 0;
    if (n < a.N) {
      const Taken t = take(a, n);
      want = max(t.need - t.full - (t.part > 0), 0) + (t.last >= 0 && !keeps(a, t, n));
    }
    int sum;
    const int before = scan(want, &sum, ws);
    if (n < a.N) base[n] = total + before;
    total += sum;
  }
  const int64_t per = ((a.pages + kForkCtas - 1) / kForkCtas + 3) / 4 * 4;
  const int64_t first = min(per * (int64_t)rank, a.pages), last = min(first + per, a.pages);
  int many = 0;
  for (int64_t p = first + tid; p < last; p += kForkThreads) many += __ldcg(&a.hold[p]) == 0 && __ldcg(&a.claim[p]) == INT_MAX;
  int here;
  scan(many, &here, ws);
  if (tid < kForkCtas) {
    const uint32_t to = dsmem_addr(&free_pages[rank], (uint32_t)tid);
    dsmem_st_u32(to, (uint32_t)here);
  }
  all_sync();
  int before = 0, most = 0;
  for (int c = 0; c < kForkCtas; ++c) {
    if (c < (int)rank) before += free_pages[c];
    most += free_pages[c];
  }
  const int lacking = max(total - most, 0);
  if (me == 0) a.missing[0] = lacking;
  // ranks of the free pages, and the references as they will be
  for (int64_t p0 = first; p0 < last; p0 += 4 * kForkThreads) {
    const int64_t p = p0 + 4 * tid;
    int h[4], mine = 0;
    bool is_free[4], kept[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = p + k < last;
      h[k] = in ? __ldcg(&a.hold[p + k]) : 1;
      const bool claimed = in && __ldcg(&a.claim[p + k]) != INT_MAX;
      is_free[k] = h[k] == 0 && !claimed;
      kept[k] = h[k] == 0 && claimed;
      mine += is_free[k];
    }
    int sum;
    int k0 = before + scan(mine, &sum, ws);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (p + k >= last) continue;
      const bool given = is_free[k] && k0 < total;
      if (given) __stcg(&a.fresh[k0], (int)(p + k));
      k0 += is_free[k];
      a.refs_out[p + k] = lacking ? a.refs[p + k] : h[k] + kept[k] + given;
    }
    before += sum;
  }
  all_sync();
  // the new table, and the pages to copy
  for (int n = me; n < a.N; n += all) {
    const Taken t = take(a, n);
    const bool copy = !lacking && t.last >= 0 && !keeps(a, t, n);
    a.copies[n] = make_int4(t.last, copy ? __ldcg(&a.fresh[base[n]]) : -1, copy ? t.part : 0, 0);
  }
  const int slots = a.N * a.M;
  for (int x = me; x < slots; x += all) {
    const int n = x / a.M, i = x - n * a.M;
    int p = -1;
    if (!lacking) {
      const Taken t = take(a, n);
      if (i < t.full) {
        p = a.table[(int64_t)t.source * a.ld + i];
        if (p < 0 || p >= a.pages) p = -1;
      } else {
        const bool copy = t.last >= 0 && !keeps(a, t, n);
        const int k = i - t.full - (t.part > 0);  // among the grown ones
        if (k < 0) p = copy ? __ldcg(&a.fresh[base[n]]) : t.last;
        else if (i < t.need) p = __ldcg(&a.fresh[base[n] + copy + k]);
      }
    }
    a.table_out[(int64_t)n * a.ld_out + i] = p;
  }
  // no CTA leaves while another may still write its count here
  all_sync();
}

// --------------------------------------------------------------------- copies
constexpr int kCopyThreads = 256, kCopyDepth = 8;

template <typename U>
__device__ __forceinline__ void copy_units(const PageState& st, const int4& c, int chunks) {
  const int64_t live = (int64_t)c.z * st.entry_bytes / (int64_t)sizeof(U);  // of a block
  const int64_t total = live * st.blocks;
  const char* src = st.data + c.x * st.page_stride;
  char* dst = st.data + c.y * st.page_stride;
  for (int64_t i0 = (int64_t)blockIdx.x * kCopyThreads * kCopyDepth + threadIdx.x; i0 < total; i0 += (int64_t)chunks * kCopyThreads * kCopyDepth) {
    U r[kCopyDepth];
    int64_t at[kCopyDepth];
#pragma unroll
    for (int k = 0; k < kCopyDepth; ++k) {
      const int64_t i = i0 + k * kCopyThreads;
      const int64_t blk = st.blocks > 1 ? (total <= 0x7fffffffll ? (int64_t)((uint32_t)i / (uint32_t)live) : i / live) : 0;
      at[k] = blk * st.block_stride + (i - blk * live) * (int64_t)sizeof(U);
      if (i < total) r[k] = *reinterpret_cast<const U*>(src + at[k]);
    }
#pragma unroll
    for (int k = 0; k < kCopyDepth; ++k)
      if (i0 + k * kCopyThreads < total) *reinterpret_cast<U*>(dst + at[k]) = r[k];
  }
}
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ CopyArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 c = a.copies[blockIdx.y];
  if (c.z <= 0) return;
  const PageState& st = a.st[blockIdx.z];
  if (st.unit == 16) copy_units<uint4>(st, c, a.chunks);
  else if (st.unit == 4) copy_units<uint32_t>(st, c, a.chunks);
  else copy_units<uint8_t>(st, c, a.chunks);
}

// ----------------------------------------------------------------- compaction
constexpr int kCompactThreads = 128, kAtOnce = 8;

template <typename U>
__device__ __forceinline__ void compact_units(const PageState& st, const int64_t* from, const int64_t* to, int n, int chunks) {
  const int64_t per = st.entry_bytes / (int64_t)sizeof(U), total = per * st.blocks;
  for (int64_t i = (int64_t)blockIdx.x * kCompactThreads + threadIdx.x; i < total; i += (int64_t)chunks * kCompactThreads) {
    const int64_t blk = st.blocks > 1 ? (total <= 0x7fffffffll ? (int64_t)((uint32_t)i / (uint32_t)per) : i / per) : 0;
    char* p = st.data + blk * st.block_stride + (i - blk * per) * (int64_t)sizeof(U);
    for (int j0 = 0; j0 < n; j0 += kAtOnce) {
      U r[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (j0 + j < n) r[j] = *reinterpret_cast<const U*>(p + from[j0 + j]);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (j0 + j < n) *reinterpret_cast<U*>(p + to[j0 + j]) = r[j];
    }
  }
}
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ int64_t from[TOPKP_MAX_TREE], to[TOPKP_MAX_TREE];
  __shared__ int moves;
  const PageState& st = a.st[blockIdx.z];
  const int b = blockIdx.y;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const long long cap = (long long)a.M * a.page_size;
    const int count = min(max(a.kept[b], 0), a.W);
    const long long start = a.start[b];
    const int32_t* table = a.table ? a.table + (int64_t)b * a.ld : nullptr;
    // the byte a token's entry begins at, or -1
    auto place = [&](long long t) -> int64_t {
      if (t < 0 || t >= cap) return -1;
      const int pg = (int)(t / a.page_size);
      const int page = table ? table[pg] : b;
      if (page < 0 || page >= a.pages) return -1;
      return page * st.page_stride + (t - (long long)pg * a.page_size) * st.entry_bytes;
    };
    int n = 0;
    for (int j0 = 0; j0 < count; j0 += 32) {
      const int j = j0 + lane;
      int64_t f = -1, t = -1;
      if (j < count && start >= 0) {
        const int k = a.keep[(int64_t)b * a.W + j];
        if (k > j) {
          f = place(start + k);
          t = place(start + j);
        }
      }
      const bool move = f >= 0 && t >= 0;
      const uint32_t who = __ballot_sync(0xffffffffu, move);
      if (move) {
        const int at = n + __popc(who & ((1u << lane) - 1u));
        from[at] = f;
        to[at] = t;
      }
      n += __popc(who);
    }
    if (lane == 0) moves = n;
  }
  __syncthreads();
  const int n = moves;
  if (n == 0) return;
  if (st.unit == 16) compact_units<uint4>(st, from, to, n, a.chunks);
  else if (st.unit == 4) compact_units<uint32_t>(st, from, to, n, a.chunks);
  else compact_units<uint8_t>(st, from, to, n, a.chunks);
}

int64_t widest(const PageState* st, int count, int64_t entries) {
  int64_t w = 1;
  for (int i = 0; i < count; ++i) {
    const int64_t units = st[i].blocks * entries * st[i].entry_bytes / st[i].unit;
    w = units > w ? units : w;
  }
  return w;
}

}  // namespace

size_t fork_workspace(int64_t N, int64_t pages) {
  const size_t p = ((size_t)pages * sizeof(int32_t) + 255) / 256 * 256;
  return 3 * p + ((size_t)N * sizeof(int4) + 255) / 256 * 256;
}

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t s) {
  const size_t smem = ((size_t)a.R + a.N) * sizeof(int);
  const cudaError_t e = cudaFuncSetAttribute(fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * TOPKP_MAX_ROWS * (int)sizeof(int));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kForkCtas);
  cfg.blockDim = dim3(kForkThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kForkCtas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fork_kernel, a);
}

// The copies' launch overlaps the bookkeeping (or the states before); they
// wait for it themselves.
cudaError_t launch_page_copy(const CopyArgs& in, cudaStream_t s) {
  CopyArgs a = in;
  const int64_t c = (widest(a.st, a.count, a.page_size) + kCopyThreads * kCopyDepth - 1) / (kCopyThreads * kCopyDepth);
  a.chunks = (int32_t)(c > 65535 ? 65535 : c);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.chunks, (unsigned)a.N, (unsigned)a.count);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_copy_kernel, a);
}

cudaError_t launch_compact(const CompactArgs& in, cudaStream_t s) {
  CompactArgs a = in;
  const int64_t c = (widest(a.st, a.count, 1) + kCompactThreads - 1) / kCompactThreads;
  a.chunks = (int32_t)(c > 65535 ? 65535 : c);
  compact_kernel<<<dim3((unsigned)a.chunks, (unsigned)a.B, (unsigned)a.count), kCompactThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace topkp
