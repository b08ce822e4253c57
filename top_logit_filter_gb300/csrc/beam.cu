// topkp_beam_select: the best continuations of each request's beams.
//
// Within one row the candidates' order is the order of the logits, since
// score and normaliser shift a row as a whole.  One pass over the logits
// leaves what the choice needs: each row's sum of exponentials, and the
// largest logit of every unit of 512 bytes.  An element of the best n lies in
// one of the n units with the best maxima (a unit before it in that order has
// a maximum that beats it), so a second kernel, one CTA per request, takes
// the n best units by (score of the maximum, position), reads those again,
// 512 n bytes, and ranks their elements.  Nothing is selected in the pass
// over the logits, and rows of equal values cost no more than others there.
//
// The sum.  exp(x) = 2^(x log2 e).  A warp sums 2^(x log2 e - c) with c the
// integer ceil(max x log2 e) of what it has seen: sums then combine by exact
// powers of two, and the largest term is in (1/2, 1].
//
// Measured: 32 x 32 x 151936 fp32, n = 64, scan 99 us (6.3 TB/s, bound by
// DRAM), both kernels 129; 64 x 4 x 128256 bf16, n = 8, scan 17 us (3.8 TB/s:
// issue, and the latency of CTAs that live for a few loads), both 27.5, the
// merge being a chain of dependent steps on one CTA a request; one request of
// 4 x 32000 10.5, two such chains.
#include <limits.h>

#include "common.cuh"
#include "decode.h"

namespace topkp {
namespace {

// (64 x 4 x 128256 bf16, 32 x 32 x 151936 fp32: 28.7, 148 us with 256
// threads, 27.5, 129 with 512, 31.6, 135 with 1024)
constexpr int kMergeThreads = 512;
constexpr int kMW = kMergeThreads / 32;
constexpr int kPool = 1024;  // units, then elements, of a request that may be chosen
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

// The float of a float_order_key, and the key of -inf (0: no element).
__device__ __forceinline__ float order_key_float(uint32_t k) {
  return k ? __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k) : -INFINITY;
}
constexpr uint32_t kNegInfKey = 0x007fffffu;

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

// Vector `i` of a row's aligned window, which starts `lead` elements before
// the row; one that sticks out of the row is read element by element, and
// what lies outside reads as -inf.
template <int DT>
__device__ __forceinline__ uint4 edge_vector(const typename DType<DT>::raw* xr, int e, int V) {
  using raw = typename DType<DT>::raw;
  constexpr int VEC = 16 / (int)sizeof(raw);
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
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// A warp's NV * 32 vectors from row element e0 on.
template <int DT, int NV>
__device__ __forceinline__ void load_vectors(uint4 (&q)[NV], const typename DType<DT>::raw* xr, int e0, int V) {
  constexpr int VEC = 16 / (int)sizeof(typename DType<DT>::raw);
  const int lane = threadIdx.x & 31;
  if (e0 >= 0 && e0 + NV * 32 * VEC <= V) {
    const uint4* p = reinterpret_cast<const uint4*>(xr + e0) + lane;
#pragma unroll
    for (int u = 0; u < NV; ++u) q[u] = __ldcs(p + u * 32);
    return;
  }
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int e = e0 + (u * 32 + lane) * VEC;
    q[u] = e >= 0 && e + VEC <= V ? __ldcs(reinterpret_cast<const uint4*>(xr + e)) : edge_vector<DT>(xr, e, V);
  }
}

template <int DT, int NV>
__global__ void __launch_bounds__(kBeamThreads, 4) beam_scan(const BeamArgs a) {
  using raw = typename DType<DT>::raw;
  constexpr int VEC = 16 / (int)sizeof(raw);
  constexpr int PIECE = NV * 32 * VEC;     // elements a warp takes at a time
  constexpr int CHUNK = kBW * PIECE;
  __shared__ float wtop[kBW];
  __shared__ unsigned long long wsum[kBW];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t part = blockIdx.x;
  const uint32_t row = part / (uint32_t)a.slices;
  const int slice = (int)(part - row * (uint32_t)a.slices);
  const float score = a.scores[row];
  if ((a.finished && a.finished[row]) || score == -INFINITY) {
    if (threadIdx.x == 0) a.stat[part] = make_longlong2(0, 0);
    return;
  }

  const raw* xr = reinterpret_cast<const raw*>(a.x) + row * a.ldx;
  const int lead = (int)((reinterpret_cast<uintptr_t>(xr) & 15) / sizeof(raw));
  // row element of this warp's first piece, and the end of the slice
  const int c_first = slice * a.chunks;
  int e0 = c_first * CHUNK + warp * PIECE - lead;
  const int e_end = min((c_first + a.chunks) * CHUNK - lead, a.V);
  uint32_t* units = a.units + (int64_t)row * a.unit_count + (c_first * kBW + warp) * NV;
  uint32_t* pieces = a.pieces + (int64_t)row * (a.unit_count / NV) + c_first * kBW + warp;

  uint4 q[NV], nx[NV];
  load_vectors<DT, NV>(q, xr, e0, a.V);
  float c = -INFINITY;            // the warp's shift: an integer, or -inf before its first finite element
  unsigned long long acc = 0ull;  // this thread's sum in units of 2^(c - 38)
#pragma unroll 1
  for (; e0 < e_end; e0 += CHUNK, units += kBW * NV, pieces += kBW) {
    if (e0 + CHUNK < e_end) load_vectors<DT, NV>(nx, xr, e0 + CHUNK, a.V);
    uint32_t key = 0;  // of unit `lane`, for lane < NV
    uint32_t kmax = 0;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const float v = vec_max<DT>(q[u]);
      const uint32_t k = __reduce_max_sync(0xffffffffu, float_order_key(v));
      key = lane == u ? k : key;
      kmax = max(kmax, k);
    }
    if (lane < NV) units[lane] = key;
    if (NV > 1 && lane == 0) *pieces = kmax;
    const float m = order_key_float(kmax);
    if (m > -INFINITY) {
      const float mc = fminf(fmaxf(m, -kFar), kFar) * (kLog2eHi + kLog2eLo);
      if (mc > c) {
        const float nc = ceilf(mc);
        acc = c == -INFINITY ? 0ull : acc >> min((int)(nc - c), 63);
        c = nc;
      }
      const unsigned long long c2 = f32x2(-c, -c);
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
      acc += f2ull_rn((s0 + s1) * kSumScale);
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) q[u] = nx[u];
  }

  // the slice's sum: the warps' at the largest of their shifts, exact and in no order
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) {
    wtop[warp] = c;
    wsum[warp] = acc;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float top = -INFINITY;
    for (int i = 0; i < kBW; ++i) top = fmaxf(top, wtop[i]);
    unsigned long long total = 0ull;
    for (int i = 0; i < kBW; ++i)
      if (wtop[i] > -INFINITY) total += wsum[i] >> min((int)(top - wtop[i]), 63);
    a.stat[part] = make_longlong2(top == -INFINITY ? 0 : (long long)(int)top, (long long)total);
  }
}

// (key, place) pairs in shared memory: larger key first, then larger place.
struct Pool {
  unsigned long long key[kPool];
  uint32_t place[kPool];
  int count;
};
// 1 if pair a comes before pair b, without a branch.
__device__ __forceinline__ int before(unsigned long long ak, uint32_t ap, unsigned long long bk, uint32_t bp) {
  return (int)(ak > bk) | ((int)(ak == bk) & (int)(ap > bp));
}
__device__ __forceinline__ void pool_add(Pool& p, unsigned long long key, uint32_t place) {
  const int at = atomicAdd(&p.count, 1);
  if (at < kPool) {
    p.key[at] = key;
    p.place[at] = place;
  }
}
// f(item, rank) for m <= kMergeThreads items by one thread of each; the pairs
// before an item are counted by several threads where there are enough.
// Warps whose threads hold no item skip it.
template <class F>
__device__ __forceinline__ void rank_items(const unsigned long long* key, const uint32_t* place, int m, F&& f) {
  int parts = 32;
  while (parts > 1 && kMergeThreads / parts < m) parts /= 2;
  for (int i0 = 0; i0 < m; i0 += kMergeThreads / parts) {
    const int i = i0 + (int)threadIdx.x / parts, part = threadIdx.x % parts;
    const unsigned long long k = i < m ? key[i] : 0ull;
    const uint32_t p = i < m ? place[i] : 0u;
    int rank = 0;
    if (i < m) {
#pragma unroll 4
      for (int j = part; j < m; j += parts) rank += before(key[j], place[j], k, p);
    }
    for (int o = parts / 2; o > 0; o /= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (i < m && part == 0) f(i, rank);
  }
}
// The best pair below (lk, lp) that `each` hands out, over the CTA.
template <class F>
__device__ __forceinline__ void next_best(F&& each, unsigned long long& lk, uint32_t& lp, unsigned long long* wk,
                                          uint32_t* wp) {
  unsigned long long bk = 0ull;
  uint32_t bp = 0;
  each([&](unsigned long long k, uint32_t p) {
    if ((k < lk || (k == lk && p < lp)) && (k > bk || (k == bk && p > bp))) {
      bk = k;
      bp = p;
    }
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long k = __shfl_xor_sync(0xffffffffu, bk, o);
    const uint32_t p = __shfl_xor_sync(0xffffffffu, bp, o);
    if (k > bk || (k == bk && p > bp)) {
      bk = k;
      bp = p;
    }
  }
  __syncthreads();  // the slots may still be read from the last round
  if ((threadIdx.x & 31) == 0) {
    wk[threadIdx.x >> 5] = bk;
    wp[threadIdx.x >> 5] = bp;
  }
  __syncthreads();
  for (int i = 0; i < kMW; ++i)
    if (wk[i] > bk || (wk[i] == bk && wp[i] > bp)) {
      bk = wk[i];
      bp = wp[i];
    }
  lk = bk;
  lp = bp;
}

// One CTA per request, its launch under the scan's end.  Launched alone and
// from a cold cache 16 us at n = 8, K = 4, 38 at n = 64, K = 32.
template <int DT>
__global__ void __launch_bounds__(kMergeThreads) beam_merge(const BeamArgs a) {
  using raw = typename DType<DT>::raw;
  constexpr int VEC = 16 / (int)sizeof(raw);
  __shared__ Pool pool;
  __shared__ unsigned long long best[kMergeThreads];
  __shared__ uint32_t bplace[kMergeThreads];
  __shared__ unsigned long long ukey[TOPKP_MAX_CANDIDATES];  // the chosen units, in order
  __shared__ uint32_t uplace[TOPKP_MAX_CANDIDATES];
  __shared__ long long shift[TOPKP_MAX_BEAMS];  // score - normaliser; the score itself where finished
  __shared__ int top[TOPKP_MAX_BEAMS];
  __shared__ uint8_t state[TOPKP_MAX_BEAMS];  // 0: no candidate, 1: live, 2: finished
  __shared__ unsigned long long tau_s, wk[kMW];
  __shared__ uint32_t wp[kMW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.x;
  const int n = a.n, S = a.slices, U = a.unit_count;

  if (tid == 0) {
    pool.count = 0;
    tau_s = 1ull;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int k = warp; k < a.K; k += kMW) {
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

  // ---- the n best units.  Place of unit u of beam k: ~(k U + u) ----
  const uint32_t* units = a.units + b * a.K * (int64_t)U;
  const int share = max(1, kMW / a.K);  // warps to a beam
  // pieces of nv units, and how many of them hold an element of the beam's row
  const int P = U / a.nv;
  const uint32_t* pieces = a.pieces + b * a.K * (int64_t)P;
  auto row_pieces = [&](int k) {
    const raw* xr = reinterpret_cast<const raw*>(a.x) + (b * a.K + k) * a.ldx;
    const int lead = (int)((reinterpret_cast<uintptr_t>(xr) & 15) / sizeof(raw));
    return (a.V + lead + a.nv * 32 * VEC - 1) / (a.nv * 32 * VEC);
  };
  // a thread reads four pieces at once, or one where that leaves no thread idle
  const int wide = P >= 256 * share ? 4 : 1, step = wide * 32 * share;
  auto some_pieces = [&](const uint32_t* pr, int i, int end) {
    if (i >= end) return make_uint4(0, 0, 0, 0);
    return wide == 4 ? *reinterpret_cast<const uint4*>(pr + i) : make_uint4(pr[i], 0, 0, 0);
  };
  auto unit_key = [&](int k, uint32_t fk) { return fixed_key(shift[k] + fixed_of(order_key_float(fk))); };
  // every unit whose key may reach `least` (0: all); finished beams are a unit of their own
  auto each_unit = [&](unsigned long long least, auto&& f) {
    for (int i = warp; i < a.K * share; i += kMW) {
      const int k = i / share, from = (i - k * share) * 32 + lane;
      if (state[k] == 2) {
        const unsigned long long e = fixed_key(shift[k]);
        if (from == 0 && e >= least) f(e, ~(uint32_t)(k * U));
      } else if (state[k] == 1) {
        // the bound as a logit of this beam, one part in 10^6 lower
        uint32_t low = kNegInfKey + 1;
        if (least > 1ull) {
          const float x = (float)((long long)(least ^ 0x8000000000000000ull) - shift[k]) * (1.0f / kMassScaleF);
          if (x > -0.999f * kFar) low = float_order_key(x - fabsf(x) * 1e-6f - 1e-6f);
        }
        const uint32_t* ur = units + (int64_t)k * U;
        const uint32_t* pr = pieces + (int64_t)k * P;
        const int end = row_pieces(k);
        auto take = [&](uint32_t fk, int u) {
          if (fk >= low) {
            const unsigned long long e = unit_key(k, fk);
            if (e >= least) f(e, ~(uint32_t)(k * U + u));
          }
        };
        auto open = [&](uint32_t fk, int i) {
          if (fk < low || i >= end) return;
          if (a.nv == 1) return take(fk, i);
          const uint4 v = *reinterpret_cast<const uint4*>(ur + 4 * i);
          take(v.x, 4 * i);
          take(v.y, 4 * i + 1);
          take(v.z, 4 * i + 2);
          take(v.w, 4 * i + 3);
        };
        for (int i0 = wide * from; i0 < end; i0 += step) {
          const uint4 v = some_pieces(pr, i0, end);
          if (max(max(v.x, v.y), max(v.z, v.w)) < low) continue;
          open(v.x, i0);
          open(v.y, i0 + 1);
          open(v.z, i0 + 2);
          open(v.w, i0 + 3);
        }
      }
    }
  };
  {
    // the n-th largest of the threads' own maxima bounds the n-th unit
    unsigned long long mine = 0ull;
    for (int i = warp; i < a.K * share; i += kMW) {
      const int k = i / share, from = (i - k * share) * 32 + lane;
      if (state[k] == 2 && from == 0) mine = max(mine, fixed_key(shift[k]));
      if (state[k] != 1) continue;
      uint32_t fk = 0;
      const uint32_t* pr = pieces + (int64_t)k * P;
      const int end = row_pieces(k);
#pragma unroll 4
      for (int i2 = wide * from; i2 < end; i2 += step) {
        const uint4 v = some_pieces(pr, i2, end);
        fk = max(fk, max(max(v.x, i2 + 1 < end ? v.y : 0u), max(i2 + 2 < end ? v.z : 0u, i2 + 3 < end ? v.w : 0u)));
      }
      if (fk > kNegInfKey) mine = max(mine, unit_key(k, fk));
    }
    // groups of lanes, at least 2 n of them; few beams leave warps without a
    // row, whose maxima are 0
    const int used = min(a.K * share, kMW) * 32;
    int group = 1;
    while (group < 32 && used / (2 * group) >= max(2 * n, 32)) {
      const unsigned long long o = __shfl_xor_sync(0xffffffffu, mine, group);
      mine = o > mine ? o : mine;
      group *= 2;
    }
    const int groups = used / group;
    if (tid % group == 0 && tid < used) {
      best[tid / group] = mine;
      bplace[tid / group] = (uint32_t)tid;
    }
    __syncthreads();
    rank_items(best, bplace, groups, [&](int i, int rank) {
      if (rank == n - 1 && best[i]) tau_s = best[i];
    });
    __syncthreads();
  }
  unsigned long long least = tau_s;
  each_unit(least, [&](unsigned long long k, uint32_t p) { pool_add(pool, k, p); });
  __syncthreads();
  const int listed = pool.count;
  int chosen = min(listed, n);
  if (listed <= kPool) {
    rank_items(pool.key, pool.place, listed, [&](int i, int rank) {
      if (rank < n) {
        ukey[rank] = pool.key[i];
        uplace[rank] = pool.place[i];
      }
    });
  } else {  // many equal maxima: the next unit in order, n times
    unsigned long long lk = ~0ull;
    uint32_t lp = ~0u;
    for (int r = 0; r < n; ++r) {
      next_best([&](auto&& f) { each_unit(least, f); }, lk, lp, wk, wp);
      if (tid == 0) {
        ukey[r] = lk;
        uplace[r] = lp;
      }
    }
  }
  __syncthreads();
  if (tid == 0) pool.count = 0;  // its readers are past the barrier above
  __syncthreads();

  // ---- their elements.  Place of token v of beam k: ~(k V + v) ----
  least = chosen == n ? ukey[n - 1] : 1ull;  // n maxima reach it
  auto each_element = [&](auto&& f) {
    for (int i = warp; i < chosen; i += kMW) {
      const uint32_t p = ~uplace[i];
      const int k = (int)(p / (uint32_t)U), u = (int)(p - (uint32_t)k * U);
      if (state[k] == 2) {
        if (lane == 0) f(fixed_key(shift[k]), ~(uint32_t)(k * a.V + a.pad));
        continue;
      }
      const raw* xr = reinterpret_cast<const raw*>(a.x) + (b * a.K + k) * a.ldx;
      const int lead = (int)((reinterpret_cast<uintptr_t>(xr) & 15) / sizeof(raw));
      uint4 q[1];
      const int e = u * 32 * VEC - lead;
      load_vectors<DT, 1>(q, xr, e, a.V);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float x = elem<DT>(q[0], j);
        if (x > -INFINITY) {
          const unsigned long long key = fixed_key(shift[k] + fixed_of(x));
          if (key >= least) f(key, ~(uint32_t)(k * a.V + e + lane * VEC + j));
        }
      }
    }
  };
  each_element([&](unsigned long long k, uint32_t p) { pool_add(pool, k, p); });
  __syncthreads();
  const int found = pool.count;
  float* os = a.out_score + b * n;
  int32_t* op = a.out_parent + b * n;
  int32_t* ot = a.out_token + b * n;
  auto put = [&](int r, unsigned long long k, uint32_t place) {
    const uint32_t p = ~place;
    os[r] = k ? key_score(k) : -INFINITY;
    op[r] = k ? (int32_t)(p / (uint32_t)a.V) : r % a.K;
    ot[r] = k ? (int32_t)(p % (uint32_t)a.V) : -1;
  };
  if (found <= kPool) {
    rank_items(pool.key, pool.place, found, [&](int i, int rank) {
      if (rank < n) put(rank, pool.key[i], pool.place[i]);
    });
    for (int r = found + tid; r < n; r += kMergeThreads) put(r, 0ull, 0u);
    return;
  }
  // many equal elements: the next one in order, n times
  unsigned long long lk = ~0ull;
  uint32_t lp = ~0u;
  for (int r = 0; r < n; ++r) {
    next_best(each_element, lk, lp, wk, wp);
    if (tid == 0) put(r, lk, lp);
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
  cfg.blockDim = dim3(kMergeThreads);
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
// three waves of four CTAs an SM, and into single short chunks when there
// are too few rows for that.
BeamPlan plan_beam(int64_t rows, int64_t V, int esize, int num_sms) {
  BeamPlan p;
  const int vec = 16 / esize;
  // the aligned window may start up to vec - 1 elements before the row
  auto chunks = [&](int nv) { return (V + vec - 1 + (int64_t)kBeamThreads * nv * vec - 1) / ((int64_t)kBeamThreads * nv * vec); };
  const int64_t wave = 4LL * num_sms;
  p.nv = rows * chunks(4) >= wave ? 4 : 1;
  const int64_t all = chunks(p.nv);
  int64_t slices = (3 * wave + rows - 1) / rows;
  if (slices > all) slices = all;
  p.chunks = (int)((all + slices - 1) / slices);
  p.slices = (int)((all + p.chunks - 1) / p.chunks);
  p.stat_bytes = ((size_t)rows * p.slices * sizeof(longlong2) + 255) / 256 * 256;
  p.unit_count = p.slices * p.chunks * kBW * p.nv;
  p.unit_bytes = ((size_t)rows * p.unit_count * sizeof(uint32_t) + 255) / 256 * 256;
  p.piece_bytes = p.nv > 1 ? p.unit_bytes / p.nv + 256 : 0;
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
