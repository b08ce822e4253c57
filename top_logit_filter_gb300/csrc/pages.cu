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
// bookkeeping's tail.
//
// Measured: one row of 253 pages to eight, 12.4 us, about 8.5 of them the
// bookkeeping's four phases (a barrier about 1 us, a phase one to two reads
// that depend on one another); 32 x 8 beams of 74 pages, 8 states, 21.5; 64
// rows to 1024, 503 MB of copies, 108: 4.7 TB/s of writes over the whole
// call, where filling memory alone reaches 4.0 (part of these stay in L2).
//
// Compacting: a thread owns one column (16 bytes, or fewer where alignment
// wants it) of an entry and takes a request's kept tokens in order, eight
// reads before their eight writes.  A token only moves to a lower place, and
// every place that is read lies behind those written so far, so the same
// code is right in place.  64 requests, 16 states of 2 KB entries: 8.3 us, a
// launch and four reads that depend on one another; 4.2 for one request.
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

__device__ __forceinline__ int divided(uint32_t x, const Reciprocal& r) { return r.mul ? (int)(__umulhi(x, r.mul) >> r.shift) : (int)x; }

// What a new row takes over and asks for.
struct Taken {
  int source;     // old row
  int full;       // whole pages
  int last;       // the partly filled page behind them; -1: none, -2: an entry that holds nothing
  int need;       // pages the row will have
};
__device__ __forceinline__ int clamped_length(const ForkArgs& a, int row) {
  const long long cap = (long long)a.M * a.page_size;
  return (int)min((long long)max(a.lengths[row], 0), cap);
}
__device__ __forceinline__ Taken take(const ForkArgs& a, int n, int* part) {
  Taken t;
  const int s = a.source[n];
  const int grow = max(a.grow ? a.grow[n] : a.grow_all, 0);
  const bool in = s >= 0 && s < a.R;
  t.source = in ? s : -1;
  const int len = in ? clamped_length(a, s) : 0;
  t.full = divided(len, a.by_page);
  *part = len - t.full * a.page_size;
  t.last = -1;
  if (*part) {
    const int g = a.table[(int64_t)s * a.ld + t.full];
    t.last = g >= 0 && g < a.pages ? g : -2;
  }
  const int tokens = len + min(grow, a.M * a.page_size - len);
  t.need = tokens ? divided(tokens - 1, a.by_page) + 1 : 0;
  return t;
}

__global__ void __launch_bounds__(kForkThreads, 1) fork_kernel(const __grid_constant__ ForkArgs a) {
  extern __shared__ int4 fork_smem[];
  Taken* taken = reinterpret_cast<Taken*>(fork_smem);          // [N]
  int* base = reinterpret_cast<int*>(fork_smem + a.N);         // [N] the first of a row's fresh pages; complemented if it is a copy
  int* children = base + a.N;                                  // [R] new rows of an old one
  int* whole = children + a.R;                                 // [R] whole pages of an old row
  __shared__ int ws[32], free_pages[kForkCtas];
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_ctarank();
  constexpr int all = kForkThreads * kForkCtas;
  const int me = (int)rank * kForkThreads + tid;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int64_t p = me; p < a.pages; p += all) {
    __stcg(&a.hold[p], a.refs[p]);
    __stcg(&a.claim[p], INT_MAX);
  }
  for (int r = tid; r < a.R; r += kForkThreads) {
    children[r] = 0;
    whole[r] = divided(clamped_length(a, r), a.by_page);
  }
  __syncthreads();
  // every CTA looks at every new row: rather than wait for another's answer
  for (int n = tid; n < a.N; n += kForkThreads) {
    int part;
    const Taken t = take(a, n, &part);
    taken[n] = t;
    base[n] = part;
    if (t.source >= 0) atomicAdd(&children[t.source], 1);
  }
  all_sync();
  // what the old rows held goes, what the new ones share comes; several
  // entries a thread at once
  const int entries = a.R * a.M;
  for (int x0 = me; x0 < entries; x0 += 4 * all) {
    int p[4], change[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int x = x0 + k * all;
      p[k] = -1;
      change[k] = 0;
      if (x < entries) {
        const int r = divided(x, a.by_columns), i = x - r * a.M;
        p[k] = a.table[(int64_t)r * a.ld + i];
        change[k] = (i < whole[r] ? children[r] : 0) - 1;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (change[k] && p[k] >= 0 && p[k] < a.pages) atomicAdd(&a.hold[p[k]], change[k]);
  }
  for (int n = me; n < a.N; n += all)
    if (taken[n].last >= 0) atomicMin(&a.claim[taken[n].last], n);
  all_sync();
  // the free pages of this CTA's part of the pool, ranked: a thread four pages
  const int64_t per = ((a.pages + kForkCtas - 1) / kForkCtas + 3) / 4 * 4;
  const int64_t first = min(per * (int64_t)rank, a.pages), last = min(first + per, a.pages);
  int h[4];
  uint32_t free4 = 0, kept4 = 0;  // bit k: of page k
  auto look = [&](int64_t p) {
    // (both arrays go on to a multiple of 256 bytes)
    const int4 x = p < last ? __ldcg(reinterpret_cast<const int4*>(a.hold + p)) : make_int4(1, 1, 1, 1);
    const int4 y = p < last ? __ldcg(reinterpret_cast<const int4*>(a.claim + p)) : make_int4(0, 0, 0, 0);
    const int c[4] = {y.x, y.y, y.z, y.w};
    h[0] = x.x, h[1] = x.y, h[2] = x.z, h[3] = x.w;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (p + k >= last) h[k] = 1;
    free4 = kept4 = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      free4 |= (uint32_t)(h[k] == 0 && c[k] == INT_MAX) << k;
      kept4 |= (uint32_t)(h[k] == 0 && c[k] != INT_MAX) << k;
    }
  };
  look(first + 4 * tid);
  // Every row's demand.  A row goes on with its partly filled page if it is
  // the first to claim it, and nobody else holds it.
  int total = 0;
  for (int n0 = 0; n0 < a.N; n0 += kForkThreads) {
    const int n = n0 + tid;
    int want = 0;
    bool copy = false;
    if (n < a.N) {
      const Taken t = taken[n];
      if (t.last >= 0) {
        const int claim = __ldcg(&a.claim[t.last]), hold = __ldcg(&a.hold[t.last]);
        copy = claim != n || hold != 0;
      }
      want = max(t.need - t.full - (t.last != -1), 0) + copy;
    }
    int sum;
    const int before = total + scan(want, &sum, ws);
    total += sum;
    if (n < a.N) {
      if (n % kForkCtas == (int)rank) a.copies[n] = make_int4(taken[n].last, before, copy ? base[n] : 0, 0);
      base[n] = copy ? ~before : before;
    }
  }
  int here, sum, sum0;
  int k0 = scan(__popc(free4), &sum0, ws);  // of the first chunk; further ones are only counted now
  here = sum0;
  for (int64_t p0 = first + 4 * kForkThreads; p0 < last; p0 += 4 * kForkThreads) {
    const int h0 = h[0], h1 = h[1], h2 = h[2], h3 = h[3];
    const uint32_t f = free4, g = kept4;
    look(p0 + 4 * tid);
    const int mine = __popc(free4);
    scan(mine, &sum, ws);
    here += sum;
    h[0] = h0, h[1] = h1, h[2] = h2, h[3] = h3;
    free4 = f;
    kept4 = g;
  }
  if (tid < kForkCtas) dsmem_st_u32(dsmem_addr(&free_pages[rank], (uint32_t)tid), (uint32_t)here);
  all_sync();
  int before = 0, most = 0;
  for (int c = 0; c < kForkCtas; ++c) {
    if (c < (int)rank) before += free_pages[c];
    most += free_pages[c];
  }
  const int lacking = max(total - most, 0);
  if (me == 0) a.missing[0] = lacking;
  // the first `total` free pages are given out; the references as they will be
  for (int64_t p0 = first; p0 < last; p0 += 4 * kForkThreads) {
    const int64_t p = p0 + 4 * tid;
    if (p0 > first) {
      look(p);
      k0 = scan(__popc(free4), &sum0, ws);
    }
    int rank_of = before + k0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (p + k >= last) continue;
      const bool is_free = free4 >> k & 1, given = is_free && rank_of < total;
      if (given) __stcg(&a.fresh[rank_of], (int)(p + k));
      rank_of += is_free;
      a.refs_out[p + k] = lacking ? a.refs[p + k] : h[k] + (int)(kept4 >> k & 1) + given;
    }
    before += sum0;
  }
  all_sync();
  // the new table, and where copies go
  for (int n = me; n < a.N; n += all) {
    // (written above by this cluster's CTA n mod 8: a release and acquire ago)
    int4 c = __ldcg(&a.copies[n]);
    if (lacking) c.z = 0;
    if (c.z) c.y = __ldcg(&a.fresh[c.y]);
    a.copies[n] = c;
  }
  const int slots = a.N * a.M;
  for (int x0 = me; x0 < slots; x0 += 4 * all) {
    int p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int x = x0 + k * all;
      p[k] = -1;
      if (x < slots && !lacking) {
        const int n = divided(x, a.by_columns), i = x - n * a.M;
        const Taken t = taken[n];
        const int b = base[n], g = i - t.full - (t.last != -1);  // g: among the grown pages
        if (i < t.full) p[k] = a.table[(int64_t)t.source * a.ld + i];
        else if (g < 0) p[k] = b < 0 ? __ldcg(&a.fresh[~b]) : t.last;
        else if (i < t.need) p[k] = __ldcg(&a.fresh[b < 0 ? ~b + 1 + g : b + g]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int x = x0 + k * all;
      if (x < slots) {
        const int n = divided(x, a.by_columns), i = x - n * a.M;
        a.table_out[(int64_t)n * a.ld_out + i] = p[k] >= 0 && p[k] < a.pages ? p[k] : -1;
      }
    }
  }
}

// --------------------------------------------------------------------- copies
constexpr int kCopyThreads = 256, kCopyDepth = 8;

template <typename U>
__device__ __noinline__ void copy_blocks(const PageState& st, const int4& c, int chunks) {
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
template <typename U>
__device__ __forceinline__ void copy_units(const PageState& st, const int4& c, int chunks) {
  if (st.blocks == 1 && (int64_t)c.z * st.entry_bytes <= INT_MAX / 2) {  // the usual page: bytes one after another
    const U* from = reinterpret_cast<const U*>(st.data + c.x * st.page_stride);
    U* to = reinterpret_cast<U*>(st.data + c.y * st.page_stride);
    const int n = (int)(c.z * st.entry_bytes / (int64_t)sizeof(U));
    for (int i = blockIdx.x * (kCopyThreads * kCopyDepth) + threadIdx.x; i < n; i += chunks * (kCopyThreads * kCopyDepth)) {
      U r[kCopyDepth];
#pragma unroll
      for (int k = 0; k < kCopyDepth; ++k)
        if (i + k * kCopyThreads < n) r[k] = from[i + k * kCopyThreads];
#pragma unroll
      for (int k = 0; k < kCopyDepth; ++k)
        if (i + k * kCopyThreads < n) to[i + k * kCopyThreads] = r[k];
    }
    return;
  }
  copy_blocks<U>(st, c, chunks);
}
__global__ void __launch_bounds__(kCopyThreads, 4) page_copy_kernel(const __grid_constant__ CopyArgs a) {
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

static_assert(7 * TOPKP_MAX_ROWS * sizeof(int) <= 226 * 1024, "the rows do not fit shared memory");
// x / d = (x * mul) >> (32 + shift), exact for x below 2^31
Reciprocal reciprocal(int64_t d) {
  if (d <= 1) return {0u, 0};
  int l = 1;
  while ((1LL << l) < d) ++l;
  return {(uint32_t)(((1ull << (31 + l)) + d - 1) / d), l - 1};
}

size_t fork_workspace(int64_t N, int64_t pages) {
  const size_t p = ((size_t)pages * sizeof(int32_t) + 255) / 256 * 256;
  return 3 * p + ((size_t)N * sizeof(int4) + 255) / 256 * 256;
}

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t s) {
  ForkArgs b = a;
  b.by_page = reciprocal(a.page_size);
  b.by_columns = reciprocal(a.M);
  const size_t smem = (size_t)a.R * 2 * sizeof(int) + (size_t)a.N * 5 * sizeof(int);
  if (smem > 40 << 10) {  // beyond what a kernel has unasked
    const cudaError_t e = cudaFuncSetAttribute(fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 7 * TOPKP_MAX_ROWS * (int)sizeof(int));
    if (e != cudaSuccess) return e;
  }
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
  return cudaLaunchKernelEx(&cfg, fork_kernel, b);
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
