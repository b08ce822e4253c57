// topkp_beam_select: the best continuations of each request's beams.
//
// Within one row the candidates' order is the order of the logits, since
// score and normaliser shift a row as a whole.  So one pass over the logits
// gives everything: each CTA holds a slice of a row in registers, sums its
// exponentials, and lists the slice's n largest logits; a second kernel, one
// CTA per request, turns those into scores and takes the n best.
//
// The sum.  exp(x) = 2^(x log2 e).  A slice sums 2^(x log2 e - c) with c the
// integer ceil(max x log2 e): slices (and rows) then combine by exact powers
// of two, and the largest term is in (1/2, 1].
//
// The n largest of a slice.  The slice goes through the CTA in chunks, each
// thread four 16-byte vectors at a time, the next chunk on its way.  In the
// first chunk, disjoint units of elements (those of one or of a few threads)
// each have a maximum; the n-th largest of the maxima is reached by at least
// n elements, and hardly any more when there are many units.  Every element
// not below it is listed; later elements are listed if they are above the
// bound.  When the list has outgrown 3 n, a bisection over the listed keys
// (value, then index: no two are equal) finds one with n keys not below it:
// those stay, and the bound moves up to it.  What is left at the end goes to
// the second kernel in any order.  A chunk that overflows the list (rows of
// many equal values) takes n rounds of a block-wide maximum instead.
#include <limits.h>

#include "common.cuh"
#include "decode.h"

namespace topkp {
namespace {

constexpr int kList = 1024;   // listed candidates of a slice
constexpr int kPool = 2560;   // of a request
constexpr int kFew = 288;     // of a request, once cut
constexpr float kLog2eHi = 1.44268798828125f;  // log2 e to 16 bits
constexpr float kLog2eLo = 7.0526077e-06f;     // the rest
// Logits beyond this magnitude count as this magnitude in the normaliser and
// the score (a mask may have put the type's lowest value there); their order
// within the row stays their own.
constexpr float kFar = 60000.0f;
// Sums are kept in 64-bit fixed point: a chunk's few fp32 terms, each at most
// 1, are added up in 2^-38 units (2^23 elements of a row stay below 2^61), so
// a long row loses nothing behind a large term and the order does not matter.
constexpr float kSumScale = 274877906944.0f;  // 2^38

template <int DT>
__device__ __forceinline__ float elem(const uint4& q, int j) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if (DT == TOPKP_F32) return __uint_as_float(w[j]);
  return DType<DT>::to_float((typename DType<DT>::raw)(w[j >> 1] >> (16 * (j & 1))));
}
template <int DT>
__device__ __forceinline__ typename DType<DT>::raw elem_raw(const uint4& q, int j) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if (DT == TOPKP_F32) return (typename DType<DT>::raw)w[j];
  return (typename DType<DT>::raw)(w[j >> 1] >> (16 * (j & 1)));
}

// Scores are compared in 64-bit fixed point, 2^-40 a unit (FP64 runs on a
// narrow pipe here).  A score as an unsigned key of the same order; 0 stands
// for no candidate.
__device__ __forceinline__ long long fixed_of(float x) {
  x = fminf(fmaxf(x, -kFar), kFar);
  const long long f = (long long)f2ull_rn(fabsf(x) * kMassScaleF);
  return x < 0.0f ? -f : f;
}
__device__ __forceinline__ unsigned long long fixed_key(long long f) {
  return (unsigned long long)f ^ 0x8000000000000000ull;
}
__device__ __forceinline__ float key_score(unsigned long long k) {
  return (float)(long long)(k ^ 0x8000000000000000ull) * (1.0f / kMassScaleF);
}

constexpr int kBW = kBeamThreads / 32;

// The sum of one value of each thread, with one barrier: `slots` has two
// alternating rows, so that the next sum does not wait for this one's readers.
__device__ __forceinline__ int block_count(int v, int (*slots)[kBW], int& phase) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) slots[phase][threadIdx.x >> 5] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int i = 0; i < kBW; ++i) t += slots[phase][i];
  phase ^= 1;
  return t;
}
// A key with exactly `want` of list[0 .. found) not below it; want < found,
// all keys different, all at least lo and below hi.  Every thread gets it.
__device__ __forceinline__ unsigned long long bisect_keys(const unsigned long long* list, int found, int want,
                                                          unsigned long long lo, unsigned long long hi,
                                                          int (*slots)[kBW], int& phase) {
  for (;;) {  // more than `want` keys are >= lo, fewer are >= hi: at most 64 halvings
    const unsigned long long mid = lo + (hi - lo) / 2;
    int c = 0;
    for (int i = threadIdx.x; i < found; i += kBeamThreads) c += list[i] >= mid ? 1 : 0;
    c = block_count(c, slots, phase);
    if (c == want) return mid;
    if (c > want) lo = mid;
    else hi = mid;
  }
}

// Two fp32 lanes in a 64-bit register, one instruction for both.
__device__ __forceinline__ unsigned long long f32x2(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ unsigned long long fma_x2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long add_x2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float ex2(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}
// 2^(x log2 e - c) of two logits.
__device__ __forceinline__ unsigned long long terms(float x0, float x1, unsigned long long c2) {
  const unsigned long long x = f32x2(x0, x1);
  const unsigned long long t =
      fma_x2(x, f32x2(kLog2eLo, kLog2eLo), fma_x2(x, f32x2(kLog2eHi, kLog2eHi), c2));
  float t0, t1;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(t0), "=f"(t1) : "l"(t));
  return f32x2(ex2(t0), ex2(t1));
}
// The largest element of a vector (packed 16-bit maxima; NaN is passed over).
template <int DT>
__device__ __forceinline__ float vec_max(const uint4& q) {
  if (DT == TOPKP_F32)
    return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
  uint32_t m;
  if (DT == TOPKP_F16)
    asm("{.reg .b32 a, b;\n\tmax.f16x2 a, %1, %2;\n\tmax.f16x2 b, %3, %4;\n\tmax.f16x2 %0, a, b;}"
        : "=r"(m) : "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w));
  else
    asm("{.reg .b32 a, b;\n\tmax.bf16x2 a, %1, %2;\n\tmax.bf16x2 b, %3, %4;\n\tmax.bf16x2 %0, a, b;}"
        : "=r"(m) : "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w));
  return fmaxf(elem<DT>(make_uint4(m, 0, 0, 0), 0), elem<DT>(make_uint4(m, 0, 0, 0), DT == TOPKP_F32 ? 0 : 1));
}

// Candidates that a slice may hand on.
__host__ __device__ inline int beam_keep(int n) { return n < 16 ? 48 : 3 * n; }

// The NV vectors of chunk elements [e, e + 256 * NV * VEC) that this thread
// holds; a vector that sticks out of the row is read element by element, and
// what lies outside reads as -inf.
template <int DT, int NV>
__device__ __forceinline__ void load_chunk(uint4 (&q)[NV], const typename DType<DT>::raw* xr, int e0, int V) {
  using raw = typename DType<DT>::raw;
  constexpr int VEC = 16 / (int)sizeof(raw);
  if (e0 >= 0 && e0 + kBeamThreads * NV * VEC <= V) {
    const uint4* p = reinterpret_cast<const uint4*>(xr + e0) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < NV; ++u) q[u] = __ldcs(p + u * kBeamThreads);
    return;
  }
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int e = e0 + (u * kBeamThreads + (int)threadIdx.x) * VEC;
    if (e >= 0 && e + VEC <= V) {
      q[u] = __ldcs(reinterpret_cast<const uint4*>(xr + e));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = DT == TOPKP_F32 ? 0xff800000u : DType<DT>::kNegInf * 0x10001u;
      if (e < V && e + VEC > 0) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          if (e + j >= 0 && e + j < V) {
            const uint32_t r = xr[e + j];
            if (DT == TOPKP_F32) w[j] = r;
            else w[j >> 1] = (j & 1) ? ((w[j >> 1] & 0xffffu) | (r << 16)) : ((w[j >> 1] & 0xffff0000u) | r);
          }
        }
      }
      q[u] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

struct ScanShared {
  unsigned long long list[2][kList];  // the current list, and where its first n go
  __align__(16) float unit[kBeamThreads];
  float wmax[kBW];
  unsigned long long wkey[kBW];
  unsigned long long wsum[kBW];
  int slots[2][kBW];
  float tau;
  int count;
};

template <int DT, int NV>
__global__ void __launch_bounds__(kBeamThreads, 3) beam_scan(const BeamArgs a) {
  using raw = typename DType<DT>::raw;
  constexpr int VEC = 16 / (int)sizeof(raw);
  constexpr int CHUNK = kBeamThreads * NV * VEC;
  __shared__ ScanShared s;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t part = blockIdx.x;
  const uint32_t row = part / (uint32_t)a.slices;
  const int slice = (int)(part - row * (uint32_t)a.slices);
  const int keep = beam_keep(a.n);
  unsigned long long* out = a.cand + (int64_t)part * keep;

  const float score = a.scores[row];
  if ((a.finished && a.finished[row]) || score == -INFINITY) {
    if (tid == 0) a.stat[part] = make_longlong2(0, 0);
    return;
  }

  // 16-byte vectors of the row's aligned window
  const raw* xr = reinterpret_cast<const raw*>(a.x) + row * a.ldx;
  const int lead = (int)((reinterpret_cast<uintptr_t>(xr) & 15) / sizeof(raw));
  const int e_first = slice * a.chunks * CHUNK - lead;  // row index of this slice's first element
  const int e_end = min(e_first + a.chunks * CHUNK, a.V);

  uint4 q[NV], nx[NV];
  load_chunk<DT, NV>(q, xr, e_first, a.V);
  int cur = 0;             // which list is current
  int phase = 0;
  int held = 0;            // entries of it
  float tau = -INFINITY;   // an element is listed if it is above (in the first chunk: not below)
  float c = -INFINITY;     // this thread's shift: an integer, or -inf before its first finite element
  unsigned long long acc = 0ull;  // this thread's sum in units of 2^(c - 38)
  if (tid == 0) s.count = 0;

#pragma unroll 1
  for (int e0 = e_first; e0 < e_end; e0 += CHUNK) {
    const bool first = e0 == e_first, last = e0 + CHUNK >= e_end;
    if (!last) load_chunk<DT, NV>(nx, xr, e0 + CHUNK, a.V);
    float vm[NV], m = -INFINITY;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      vm[u] = vec_max<DT>(q[u]);
      m = fmaxf(m, vm[u]);
    }
    if (first) {
      // units of 1, 2 or 4 threads, at least 2 n of them
      const int per = a.n <= 32 ? 4 : a.n <= 64 ? 2 : 1;
      float um = m;
      if (per >= 2) um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 1));
      if (per >= 4) um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 2));
      if (tid % per == 0) s.unit[tid / per] = um;
      if (tid == 0) s.tau = -INFINITY;
      __syncthreads();
      const int units = kBeamThreads / per;
      if (tid < units) {
        const float mine = s.unit[tid];
        int rank = 0;
        for (int i = 0; i < units; i += 4) {
          const float4 o = *reinterpret_cast<const float4*>(&s.unit[i]);
          rank += (o.x > mine || (o.x == mine && i < tid)) + (o.y > mine || (o.y == mine && i + 1 < tid)) +
                  (o.z > mine || (o.z == mine && i + 2 < tid)) + (o.w > mine || (o.w == mine && i + 3 < tid));
        }
        if (rank == a.n - 1) s.tau = mine;
      }
    }
    // the sum, in 2^c units of this thread's own
    const float mc = fminf(fmaxf(m, -kFar), kFar);
    if (m > -INFINITY && mc * (kLog2eHi + kLog2eLo) > c) {
      const float nc = ceilf(mc * (kLog2eHi + kLog2eLo));
      acc = c == -INFINITY ? 0ull : acc >> min((int)(nc - c), 63);
      c = nc;
    }
    const unsigned long long c2 = f32x2(-c, -c);
    if (m > -INFINITY) {
      unsigned long long sum2 = 0ull;
      if (fabsf(m) <= kFar) {
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
          for (int j = 0; j < VEC; j += 2) sum2 = add_x2(sum2, terms(elem<DT>(q[u], j), elem<DT>(q[u], j + 1), c2));
      } else {
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
          for (int j = 0; j < VEC; j += 2) {
            // -inf stays -inf
            const float x0 = elem<DT>(q[u], j), x1 = elem<DT>(q[u], j + 1);
            sum2 = add_x2(sum2, terms(x0 > -INFINITY ? fminf(fmaxf(x0, -kFar), kFar) : x0,
                                      x1 > -INFINITY ? fminf(fmaxf(x1, -kFar), kFar) : x1, c2));
          }
      }
      float s0, s1;
      asm("mov.b64 {%0, %1}, %2;" : "=f"(s0), "=f"(s1) : "l"(sum2));
      acc += f2ull_rn(s0 * kSumScale) + f2ull_rn(s1 * kSumScale);
    }
    if (first) {
      __syncthreads();
      tau = s.tau;
    }
    int mine = 0;
    auto wanted = [&](float x) { return first ? x >= tau && x > -INFINITY : x > tau; };
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (wanted(vm[u])) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float x = elem<DT>(q[u], j);
          if (wanted(x)) {
            ++mine;
            const int at = atomicAdd(&s.count, 1);
            const uint32_t idx = (uint32_t)(e0 + (u * kBeamThreads + tid) * VEC + j);
            if (at < kList)
              s.list[cur][at] = ((unsigned long long)order_key<DT>(elem_raw<DT>(q[u], j)) << 32) | (uint32_t)~idx;
          }
        }
      }
    // the count is summed, not read from s.count: a fast thread may be adding
    // the next chunk's already
    const int found = held + block_count(mine, s.slots, phase);
    if (found > kList) {
      // many equal or rising values: the next one in order, n times, of this
      // chunk and of what was kept (entries listed by this chunk are in q)
      unsigned long long prev = ~0ull;
#pragma unroll 1
      for (int r = 0; r < a.n; ++r) {
        unsigned long long best = 0ull;
#pragma unroll
        for (int u = 0; u < NV; ++u)  // the keys are made anew each round, not held
          asm volatile("" : "+r"(q[u].x), "+r"(q[u].y), "+r"(q[u].z), "+r"(q[u].w));
        for (int i = tid; i < held; i += kBeamThreads) {
          const unsigned long long k = s.list[cur][i];
          if (k < prev && k > best) best = k;
        }
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float x = elem<DT>(q[u], j);
            const uint32_t idx = (uint32_t)(e0 + (u * kBeamThreads + tid) * VEC + j);
            const unsigned long long k =
                ((unsigned long long)order_key<DT>(elem_raw<DT>(q[u], j)) << 32) | (uint32_t)~idx;
            if (wanted(x) && k < prev && k > best) best = k;
          }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const unsigned long long w = __shfl_xor_sync(0xffffffffu, best, o);
          best = w > best ? w : best;
        }
        if (lane == 0) s.wkey[warp] = best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kBW; ++i) best = s.wkey[i] > best ? s.wkey[i] : best;
        __syncthreads();
        if (tid == 0) s.list[cur ^ 1][r] = best;
        prev = best;
      }
      if (tid == 0) s.count = a.n;
      __syncthreads();
      cur ^= 1;
      held = a.n;
      tau = value_of_key<DT>((uint32_t)(s.list[cur][a.n - 1] >> 32));
    } else if (found > keep) {
      const unsigned long long bound =
          bisect_keys(s.list[cur], found, a.n, 0ull, DT == TOPKP_F32 ? ~0ull : 1ull << 48, s.slots, phase);
      if (tid == 0) s.count = 0;
      __syncthreads();
      for (int i = tid; i < found; i += kBeamThreads) {
        const unsigned long long k = s.list[cur][i];
        if (k >= bound) s.list[cur ^ 1][atomicAdd(&s.count, 1)] = k;
      }
      cur ^= 1;
      // the bound lies above the largest key dropped, so a later element
      // (of a larger index) with that key's value is not wanted either
      tau = value_of_key<DT>((uint32_t)(bound >> 32));
      held = a.n;
    } else {
      held = found;
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) q[u] = nx[u];
  }

  // the slice's sum: the threads' at the largest of their shifts, exact and in no order
  float top = c;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s.wmax[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBW; ++i) top = fmaxf(top, s.wmax[i]);
  unsigned long long total = c == -INFINITY ? 0ull : acc >> min((int)(top - c), 63);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) s.wsum[warp] = total;
  __syncthreads();
  if (tid == 0) {
    total = 0;
    for (int i = 0; i < kBW; ++i) total += s.wsum[i];
    // shift in the low half, number of candidates in the high one
    a.stat[part] = make_longlong2((long long)(((unsigned long long)held << 32) | (uint32_t)(top == -INFINITY ? 0 : (int)top)),
                                  (long long)total);
  }
  for (int i = tid; i < held; i += kBeamThreads) out[i] = s.list[cur][i];
}

// One CTA per request: the candidates of its beams' slices become scores in
// shared memory, a bisection leaves n of them, and each one's rank among
// those is its place.  More candidates than the pool holds are cut first by
// the n-th largest of the threads' own maxima.
template <int DT>
__global__ void __launch_bounds__(kBeamThreads) beam_merge(const BeamArgs a) {
  __shared__ unsigned long long key[kPool];
  __shared__ uint32_t flat[kPool];  // ~(k * V + v): larger is earlier
  __shared__ unsigned long long key2[kFew];
  __shared__ uint32_t flat2[kFew];
  __shared__ __align__(16) unsigned long long unit[kBeamThreads];
  __shared__ long long shift[TOPKP_MAX_BEAMS];  // score - normaliser; the score itself where finished
  __shared__ int top[TOPKP_MAX_BEAMS];
  __shared__ uint8_t state[TOPKP_MAX_BEAMS];  // 0: no candidate, 1: live, 2: finished
  __shared__ int slots[2][kBW];
  __shared__ unsigned long long tau_s, wk[kBW];
  __shared__ uint32_t wf[kBW];
  __shared__ int count, few;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.x;
  const int n = a.n, S = a.slices, keep = beam_keep(a.n);
  int phase = 0;

  if (tid == 0) {
    count = few = 0;
    tau_s = 1ull;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int k = warp; k < a.K; k += kBW) {
    const int64_t row = b * a.K + k;
    int c = INT_MIN;
    for (int s = lane; s < S; s += 32) {
      const longlong2 st = a.stat[row * S + s];
      if (st.y > 0) c = max(c, (int)st.x);
    }
    c = __reduce_max_sync(0xffffffffu, c);
    long long l = 0;
    for (int s = lane; s < S; s += 32) {
      const longlong2 st = a.stat[row * S + s];
      if (st.y > 0) l += st.y >> min(c - (int)st.x, 63);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      shift[k] = l;
      top[k] = c;
    }
  }
  __syncthreads();
  if (tid < a.K) {
    const int64_t row = b * a.K + tid;
    const float score = a.scores[row];
    const bool done = a.finished && a.finished[row];
    const long long l = shift[tid];
    const bool live = !done && score != -INFINITY && l > 0;
    state[tid] = done ? (score != -INFINITY ? 2 : 0) : live ? 1 : 0;
    // the 38 fractional bits of l go with its shift
    const double lse = live ? log((double)l) + (double)(top[tid] - 38) * 0.693147180559945309417 : 0.0;
    shift[tid] = state[tid] ? llrint(((double)score - lse) * 1099511627776.0) : 0;
  }
  __syncthreads();

  const int lists = a.K * S;
  const unsigned long long* cand = a.cand + b * lists * (int64_t)keep;
  // every candidate of the request: a warp takes a list, its lanes the entries
  auto each = [&](auto&& f) {
    for (int l = warp; l < lists; l += kBW) {
      const int k = l / S;
      const int st = state[k];
      if (st == 2) {
        if (l == k * S && lane == 0) f(fixed_key(shift[k]), ~(uint32_t)(k * a.V + a.pad));
      } else if (st == 1) {
        const int m = (int)(a.stat[b * lists + l].x >> 32);
        for (int i = lane; i < m; i += 32) {
          const unsigned long long e = cand[(int64_t)l * keep + i];
          f(fixed_key(shift[k] + fixed_of(value_of_key<DT>((uint32_t)(e >> 32)))), ~(uint32_t)(k * a.V + (int)~(uint32_t)e));
        }
      }
    }
  };
  auto pool = [&](unsigned long long e, uint32_t f) {
    const int at = atomicAdd(&count, 1);
    if (at < kPool) {
      key[at] = e;
      flat[at] = f;
    }
  };
  unsigned long long mine = 0ull;
  each([&](unsigned long long e, uint32_t f) {
    mine = e > mine ? e : mine;
    pool(e, f);
  });
  __syncthreads();
  int found = count;
  unsigned long long tau = 1ull;
  if (found > kPool) {
    unit[tid] = mine;
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < kBeamThreads; ++i) rank += (unit[i] > mine || (unit[i] == mine && i < tid)) ? 1 : 0;
    if (rank == n - 1 && mine) tau_s = mine;
    if (tid == 0) count = 0;  // read by all before the barrier above
    __syncthreads();
    tau = tau_s;
    each([&](unsigned long long e, uint32_t f) {
      if (e >= tau) pool(e, f);
    });
    __syncthreads();
    found = count;
  }
  float* os = a.out_score + b * n;
  int32_t* op = a.out_parent + b * n;
  int32_t* ot = a.out_token + b * n;
  auto put = [&](int r, unsigned long long e, uint32_t f) {
    const uint32_t p = ~f;
    os[r] = key_score(e);
    op[r] = (int32_t)(p / (uint32_t)a.V);
    ot[r] = (int32_t)(p % (uint32_t)a.V);
  };
  auto none = [&](int r) {
    os[r] = -INFINITY;
    op[r] = r % a.K;
    ot[r] = -1;
  };
  if (found <= kPool) {
    // lo: a bound with at least n candidates not below it, hardly more
    const unsigned long long* ks = key;
    const uint32_t* fs = flat;
    if (found > 2 * n + 32) {
      unit[tid] = mine;
      __syncthreads();
      unsigned long long hi = 0ull;
      for (int i = lane; i < kBeamThreads; i += 32) hi = unit[i] > hi ? unit[i] : hi;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long w = __shfl_xor_sync(0xffffffffu, hi, o);
        hi = w > hi ? w : hi;
      }
      unsigned long long lo = 1ull;
      unsigned long long mid = hi > (1ull << 44) ? hi - (1ull << 43) : 1ull;  // 8 below the best: often the first half
      ++hi;
      while (hi - lo > 1) {
        int c = 0;
        for (int i = tid; i < found; i += kBeamThreads) c += key[i] >= mid ? 1 : 0;
        c = block_count(c, slots, phase);
        if (c >= n) lo = mid;
        else hi = mid;
        if (c >= n && c <= n + 32) break;
        mid = lo + (hi - lo) / 2;
      }
      for (int i = tid; i < found; i += kBeamThreads)
        if (key[i] >= lo) {
          const int at = atomicAdd(&few, 1);
          if (at < kFew) {
            key2[at] = key[i];
            flat2[at] = flat[i];
          }
        }
      __syncthreads();
      if (few <= kFew) {  // else many equal candidates: ranked among all
        found = few;
        ks = key2;
        fs = flat2;
      }
    }
    for (int i = tid; i < found; i += kBeamThreads) {
      const unsigned long long e = ks[i];
      const uint32_t f = fs[i];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < found; ++j) rank += (ks[j] > e || (ks[j] == e && fs[j] > f)) ? 1 : 0;
      if (rank < n) put(rank, e, f);
    }
    for (int r = found + tid; r < n; r += kBeamThreads) none(r);
    return;
  }
  // many equal candidates: the next one in order, n times
  unsigned long long le = ~0ull;
  uint32_t lf = ~0u;
  for (int r = 0; r < n; ++r) {
    unsigned long long be = 0ull;
    uint32_t bf = 0;
    each([&](unsigned long long e, uint32_t f) {
      if (e >= tau && (e < le || (e == le && f < lf)) && (e > be || (e == be && f > bf))) {
        be = e;
        bf = f;
      }
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long e = __shfl_xor_sync(0xffffffffu, be, o);
      const uint32_t f = __shfl_xor_sync(0xffffffffu, bf, o);
      if (e > be || (e == be && f > bf)) {
        be = e;
        bf = f;
      }
    }
    if (lane == 0) {
      wk[warp] = be;
      wf[warp] = bf;
    }
    __syncthreads();
    be = wk[0];
    bf = wf[0];
    for (int i = 1; i < kBW; ++i)
      if (wk[i] > be || (wk[i] == be && wf[i] > bf)) {
        be = wk[i];
        bf = wf[i];
      }
    __syncthreads();
    if (tid == 0) {
      if (be) put(r, be, bf);
      else none(r);
    }
    le = be;
    lf = bf;
  }
}

template <int DT>
cudaError_t launch_dt(const BeamArgs& a, cudaStream_t s) {
  const unsigned int grid = (unsigned int)(a.B * a.K * a.slices);
  if (a.nv == 1) beam_scan<DT, 1><<<grid, kBeamThreads, 0, s>>>(a);
  else beam_scan<DT, 4><<<grid, kBeamThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the merge's launch overlaps the scan; it waits for the scan's results itself
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned int)a.B);
  cfg.blockDim = dim3(kBeamThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_merge<DT>, a);
}

}  // namespace

// A row is cut into slices of whole chunks so that the device has about
// three waves of three CTAs an SM, and into single short chunks when there
// are too few rows for that.
BeamPlan plan_beam(int64_t rows, int64_t V, int esize, int32_t n, int num_sms) {
  BeamPlan p;
  const int vec = 16 / esize;
  // the aligned window may start up to vec - 1 elements before the row
  auto chunks = [&](int nv) { return (V + vec - 1 + (int64_t)kBeamThreads * nv * vec - 1) / ((int64_t)kBeamThreads * nv * vec); };
  const int64_t wave = 3LL * num_sms;
  p.nv = rows * chunks(4) >= wave ? 4 : 1;
  const int64_t all = chunks(p.nv);
  int64_t slices = (3 * wave + rows - 1) / rows;
  if (slices > all) slices = all;
  p.chunks = (int)((all + slices - 1) / slices);
  p.slices = (int)((all + p.chunks - 1) / p.chunks);
  p.stat_bytes = ((size_t)rows * p.slices * sizeof(longlong2) + 255) / 256 * 256;
  p.cand_bytes = (size_t)rows * p.slices * beam_keep(n) * sizeof(unsigned long long);
  return p;
}

cudaError_t launch_beam(topkp_dtype dt, const BeamArgs& a, cudaStream_t s) {
  switch (dt) {
    case TOPKP_F32: return launch_dt<TOPKP_F32>(a, s);
    case TOPKP_F16: return launch_dt<TOPKP_F16>(a, s);
    default: return launch_dt<TOPKP_BF16>(a, s);
  }
}

}  // namespace topkp
