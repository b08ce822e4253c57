// topkp_beam_select: the best continuations of each request's beams.
//
// Within one row the candidates' order is the order of the logits, since
// score and normaliser shift a row as a whole.  One pass over the logits
// leaves what the choice needs: each row's sum of exponentials, and the
// largest logit of every unit of 512 bytes.  An element of the best n lies in
// one of the n units with the best maxima (a unit before it in that order has
// a maximum that beats it), so a second kernel, one CTA per request, takes
// those units (and a few more where fp32 cannot tell), reads them again,
// 512 n bytes, and ranks their elements.  Nothing is selected in the pass
// over the logits, and rows of equal values cost no more than others there.
//
// The sum.  exp(x) = 2^(x log2 e).  A warp sums 2^(x log2 e - c) with c the
// integer ceil(max x log2 e) of what it has seen: sums then combine by exact
// powers of two, and the largest term is in (1/2, 1].  Where the largest logit
// lies beyond +-60000 fp32 has no room for that: there it is exp(x - r) with r
// that logit (x - r is exact for every term that counts), and sums combine by
// factors from 64 bits.
//
// The order.  A candidate is score + ((x - base) - less) in 64-bit floating
// point, (base, less) = (normaliser, 0), or (r, log of the sum) beyond +-60000:
// no finite score or logit leaves its range, a dead beam's -1e9 or a mask's
// lowest value included.  Behind it go the beam, the logit itself and the
// index, so that one beam's candidates follow their logits even where 64 bits
// round two of them alike.  FP64 is narrow here (two lanes a clock and SM), so
// the bound that most units and elements fail is in fp32, with its roundings
// taken off; what passes gets a 64-bit key, one thread each.
//
// Measured: 32 x 32 x 151936 fp32, n = 64, scan 99 us (6.3 TB/s, bound by
// DRAM), both kernels 124; 64 x 4 x 128256 bf16, n = 8, scan 17 us (3.8 TB/s:
// issue, and the latency of CTAs that live for a few loads), both 26.5, the
// merge being a chain of dependent steps on one CTA a request; one request of
// 4 x 32000 11.0, two such chains.  Logits beyond +-60000 throughout: 135 and
// 28; 31 of 32 beams marked with -1e9 (nth_unit() is called for): 258.
#include <float.h>
#include <limits.h>

#include "common.cuh"
#include "decode.h"

namespace topkp {
namespace {

// (one request, 64 x 4 x 128256 bf16, 32 x 32 x 151936 fp32: 10.2, 28.0, 149
// us with 256 threads, 11.0, 26.5, 124 with 512, 12.6, 30.1, 113 with 1024)
constexpr int kMergeThreads = 512;
constexpr int kMW = kMergeThreads / 32;
constexpr int kPool = 1024;  // units, then elements, of a request that may be chosen
constexpr float kLog2eHi = 1.44268798828125f;  // log2 e to 16 bits
constexpr float kLog2eLo = 7.0526077e-06f;     // the rest
// Largest magnitude of the largest logit for sums by powers of two: x log2 e
// in two fp32 products is then off by less than 2^-25.
constexpr float kFar = 60000.0f;
constexpr double kLog2e = 1.4426950408889634074, kLn2 = 0.693147180559945309417;
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

// A candidate as an unsigned key of the same order; 0 stands for no candidate.
__device__ __forceinline__ unsigned long long value_key(double v) {
  const long long b = __double_as_longlong(v + 0.0);  // -0 is 0
  return (unsigned long long)b ^ (b < 0 ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value(unsigned long long k) {
  return __longlong_as_double((long long)(k ^ (k >> 63 ? 0x8000000000000000ull : ~0ull)));
}

constexpr int kBW = kBeamThreads / 32;

// The float of a float_order_key, and the key of -inf (0: no element).
__device__ __forceinline__ float order_key_float(uint32_t k) {
  return k ? __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k) : -INFINITY;
}
constexpr uint32_t kNegInfKey = 0x007fffffu;

// Where a unit or an element stands: beam, order key of its (largest) logit,
// index in the row; of two with equal candidates the larger place comes first.
constexpr unsigned long long kIndexMask = (1ull << 26) - 1;
static_assert(TOPKP_MAX_V <= 1ll << 26 && TOPKP_MAX_BEAMS <= 64, "a place has 64 bits");
__device__ __forceinline__ unsigned long long place_of(int k, uint32_t logit_key, uint32_t index) {
  return (unsigned long long)(63 - k) << 58 | (unsigned long long)logit_key << 26 | (kIndexMask - index);
}
__device__ __forceinline__ int place_beam(unsigned long long p) { return 63 - (int)(p >> 58); }
__device__ __forceinline__ uint32_t place_index(unsigned long long p) { return (uint32_t)(kIndexMask - (p & kIndexMask)); }
__device__ __forceinline__ float place_logit(unsigned long long p) { return order_key_float((uint32_t)(p >> 26)); }

// A slice's reference in its statistics: the integer c, or a logit beyond +-60000.
constexpr long long kFarMark = 1ll << 40;
__device__ __forceinline__ long long reference_code(float c, bool far) {
  return far ? kFarMark | (long long)__float_as_uint(c) : (long long)(int)c;
}
__device__ __forceinline__ bool is_far(long long code) { return (code >> 40) == 1; }
__device__ __forceinline__ double reference_of(long long code) {  // as a natural logarithm
  return is_far(code) ? (double)__uint_as_float((uint32_t)code) : (double)(int)code * kLn2;
}
// A sum in units of another reference, 2^d of the first.  Out of line, and
// only where a unit is left: this takes the narrow FP64 pipe.
__device__ __noinline__ unsigned long long rescaled(unsigned long long sum, double d) {
  return d < -64.0 ? 0ull : (unsigned long long)((double)sum * exp2(d));
}
// Logits below this are nothing beside one of -60000 or more.
constexpr float kNothing = -60200.0f;

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
  __shared__ uint8_t wfar[kBW];
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
  bool far = false;               // c is a logit beyond +-60000 instead
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
      if (far || m > kFar || (m < -kFar && c == -INFINITY)) {
        // a new reference; what a hundred lies below it comes to less than a unit
        if (!far || m > c) {
          const float was = far ? c : c * (float)kLn2;
          const float nc = fabsf(m) > kFar ? m : ceilf(m * (kLog2eHi + kLog2eLo));
          if (was - m < -100.0f) acc = 0ull;
          else acc = rescaled(acc, (far ? (double)c * kLog2e : (double)c) - (fabsf(m) > kFar ? (double)m * kLog2e : (double)nc));
          c = nc;
          far = fabsf(m) > kFar;
        }
      }
      unsigned long long sum2 = 0ull;
      if (!far) {
        const float mc = m * (kLog2eHi + kLog2eLo);
        if (mc > c) {
          const float nc = ceilf(mc);
          acc = c == -INFINITY ? 0ull : acc >> min((int)(nc - c), 63);
          c = nc;
        }
        const unsigned long long c2 = f32x2(-c, -c);
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
          for (int j = 0; j < VEC; j += 2) sum2 = add_x2(sum2, terms(elem<DT>(q[u], j), elem<DT>(q[u], j + 1), c2));
      } else {
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
          for (int j = 0; j < VEC; j += 2)
            sum2 = add_x2(sum2, terms(elem<DT>(q[u], j) - c, elem<DT>(q[u], j + 1) - c, 0ull));
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
    wfar[warp] = far;
  }
  __syncthreads();
  if (warp == 0) {
    const float own = lane < kBW ? wtop[lane] : -INFINITY;
    const bool own_far = lane < kBW && wfar[lane];
    unsigned long long sum = lane < kBW ? wsum[lane] : 0ull;
    // the largest shift; another reference counts where it is not far below
    // it, or where there is no shift
    const int shift = own > -INFINITY && !own_far ? (int)own : INT_MIN;
    const int top = __reduce_max_sync(0xffffffffu, shift);
    long long code = top == INT_MIN ? 0 : (long long)top;
    if (!__any_sync(0xffffffffu, own_far && (own >= kNothing || top == INT_MIN))) {
      sum = shift == INT_MIN ? 0ull : sum >> min(top - shift, 63);
    } else {
      code = reference_code(own, own_far);
      double ref = own > -INFINITY ? reference_of(code) : -INFINITY;
      const double mine = ref;
#pragma unroll
      for (int o = kBW / 2; o > 0; o >>= 1) {
        const double r = __shfl_xor_sync(0xffffffffu, ref, o);
        const long long c2 = __shfl_xor_sync(0xffffffffu, code, o);
        if (r > ref || (r == ref && c2 > code)) {
          ref = r;
          code = c2;
        }
      }
      sum = own == -INFINITY ? 0ull : mine == ref ? sum : rescaled(sum, (mine - ref) * kLog2e);
    }
#pragma unroll
    for (int o = kBW / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) a.stat[part] = make_longlong2(code, (long long)sum);
  }
}

// (key, place) pairs in shared memory: larger key first, then larger place.
struct Pool {
  unsigned long long key[kPool];
  unsigned long long place[kPool];
  int count;
};
__device__ __forceinline__ void pool_add(Pool& p, unsigned long long place) {
  const int at = atomicAdd(&p.count, 1);
  if (at < kPool) p.place[at] = place;
}
// f(item, rank) for m <= kPool items by one thread of each; the items before
// one, as `precedes` says without a branch, are counted by several threads
// where there are enough.  Warps whose threads hold no item skip it.
template <class P, class F>
__device__ __forceinline__ void rank_items(int m, P&& precedes, F&& f) {
  int parts = 32;
  while (parts > 1 && kMergeThreads / parts < m) parts /= 2;
  for (int i0 = 0; i0 < m; i0 += kMergeThreads / parts) {
    const int i = i0 + (int)threadIdx.x / parts, part = threadIdx.x % parts;
    int rank = 0;
    if (i < m) {
      auto own = precedes(i);
#pragma unroll 4
      for (int j = part; j < m; j += parts) rank += own(j);
    }
    for (int o = parts / 2; o > 0; o /= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (i < m && part == 0) f(i, rank);
  }
}
// Larger key first, then larger place.
template <class F>
__device__ __forceinline__ void rank_pool(const Pool& p, int m, F&& f) {
  rank_items(m, [&](int i) {
    return [&p, k = p.key[i], at = p.place[i]](int j) {
      return (int)(p.key[j] > k) | ((int)(p.key[j] == k) & (int)(p.place[j] > at));
    };
  }, f);
}
// Larger word first; no two are equal.
template <class F>
__device__ __forceinline__ void rank_words(const unsigned long long* w, int m, F&& f) {
  rank_items(m, [&](int i) { return [w, own = w[i]](int j) { return (int)(w[j] > own); }; }, f);
}
// The next place in order, over the CTA, of those that `each` hands out a
// thread's beams one after another.  Within a beam places are ordered as their
// keys are: what is left of one lies below its last place taken, and a thread
// takes one key a beam.
template <class F, class G>
__device__ __forceinline__ void next_best(F&& each, G&& key_of, unsigned long long* last, unsigned long long& bk,
                                          unsigned long long& bp, unsigned long long* wk, unsigned long long* wp) {
  unsigned long long best = 0ull;  // place of the present beam
  bk = bp = 0ull;
  auto against = [&](unsigned long long k, unsigned long long p) {
    if (k > bk || (k == bk && p > bp)) {
      bk = k;
      bp = p;
    }
  };
  each([&](unsigned long long p) {
    if (p >= last[place_beam(p)]) return;
    if (best && place_beam(p) != place_beam(best)) {
      against(key_of(best), best);
      best = 0ull;
    }
    best = p > best ? p : best;
  });
  if (best) against(key_of(best), best);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) against(__shfl_xor_sync(0xffffffffu, bk, o), __shfl_xor_sync(0xffffffffu, bp, o));
  if ((threadIdx.x & 31) == 0) {
    wk[threadIdx.x >> 5] = bk;
    wp[threadIdx.x >> 5] = bp;
  }
  __syncthreads();
  for (int i = 0; i < kMW; ++i) against(wk[i], wp[i]);
  if (threadIdx.x == 0 && bk) last[place_beam(bp)] = bp;
  __syncthreads();
}

// One CTA per request, its launch under the scan's end.  Launched alone and
// from a cold cache 17 us at n = 8, K = 4, 30 at n = 64, K = 32.
template <int DT>
__global__ void __launch_bounds__(kMergeThreads) beam_merge(const BeamArgs a) {
  using raw = typename DType<DT>::raw;
  constexpr int VEC = 16 / (int)sizeof(raw);
  __shared__ Pool pool;
  __shared__ unsigned long long unit[kPool];  // places of the units whose elements are looked at
  __shared__ long long total[TOPKP_MAX_BEAMS];
  __shared__ double score[TOPKP_MAX_BEAMS], base[TOPKP_MAX_BEAMS], less[TOPKP_MAX_BEAMS];  // candidate = score + ((x - base) - less)
  __shared__ int top[TOPKP_MAX_BEAMS];
  __shared__ float score32[TOPKP_MAX_BEAMS], base32[TOPKP_MAX_BEAMS], less32[TOPKP_MAX_BEAMS];
  __shared__ uint8_t state[TOPKP_MAX_BEAMS];  // 0: no candidate, 1: live, 2: finished
  __shared__ unsigned long long last[TOPKP_MAX_BEAMS];  // of a beam, where places are taken one by one
  __shared__ unsigned long long wk[kMW], wp[kMW];
  __shared__ uint32_t tau_s;
  __shared__ int tau_want, units_taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.x;
  const int n = a.n, S = a.slices, U = a.unit_count;

  if (tid == 0) {
    pool.count = 0;
    tau_s = 0u;
    units_taken = 0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int k = warp; k < a.K; k += kMW) {
    const int64_t row = b * a.K + k;
    int c = INT_MIN;
    bool odd = false, other = false;  // a reference beyond +-60000 that counts in any case, or where there is no other
    for (int s = lane; s < S; s += 32) {
      const longlong2 st = a.stat[row * S + s];
      if (st.y <= 0) continue;
      if (!is_far(st.x)) {
        c = max(c, (int)st.x);
      } else {
        other = true;
        odd = odd || __uint_as_float((uint32_t)st.x) >= kNothing;
      }
    }
    c = __reduce_max_sync(0xffffffffu, c);
    odd = odd || (other && c == INT_MIN);
    if (!__any_sync(0xffffffffu, odd)) {
      long long l = 0;
      for (int s = lane; s < S; s += 32) {
        const longlong2 st = a.stat[row * S + s];
        if (st.y > 0 && !is_far(st.x)) l += st.y >> min(c - (int)st.x, 63);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (lane == 0) {
        total[k] = l;
        top[k] = c;
      }
    } else {
      double ref = -INFINITY, sum = 0.0;
      for (int s = lane; s < S; s += 32) {
        const longlong2 st = a.stat[row * S + s];
        if (st.y > 0) ref = fmax(ref, reference_of(st.x));
      }
      for (int o = 16; o > 0; o >>= 1) ref = fmax(ref, __shfl_xor_sync(0xffffffffu, ref, o));
      for (int s = lane; s < S; s += 32) {
        const longlong2 st = a.stat[row * S + s];
        if (st.y > 0) {
          const double d = (reference_of(st.x) - ref) * kLog2e;
          if (d > -64.0) sum += d == 0.0 ? (double)st.y : (double)st.y * exp2(d);
        }
      }
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) {
        total[k] = (long long)sum;
        top[k] = INT_MIN;
        base[k] = ref;
      }
    }
  }
  __syncthreads();
  if (tid < a.K) {
    const float own = a.scores[b * a.K + tid];
    const bool done = a.finished && a.finished[b * a.K + tid];
    const long long l = total[tid];
    score[tid] = (double)own;
    last[tid] = ~0ull;
    state[tid] = own == -INFINITY ? 0 : done ? 2 : l > 0 ? 1 : 0;
    // the 38 fractional bits of l go with its reference
    const double lg = l > 0 ? log((double)l) - 38.0 * kLn2 : 0.0;
    if (top[tid] != INT_MIN) base[tid] = lg + (double)top[tid] * kLn2;
    less[tid] = top[tid] != INT_MIN ? 0.0 : lg;
    score32[tid] = own;
    base32[tid] = (float)base[tid];
    less32[tid] = (float)less[tid];
  }
  __syncthreads();
  auto key_of = [&](unsigned long long place) {
    const int k = place_beam(place);
    if (state[k] == 2) return value_key(score[k]);
    double d = (double)place_logit(place) - base[k];
    if (less32[k] != 0.0f) d -= less[k];
    return value_key(score[k] + d);
  };
  // keys of the pool's places
  auto fill_keys = [&](int m) {
    for (int i = tid; i < m; i += kMergeThreads) pool.key[i] = key_of(pool.place[i]);
  };
  // Bounds in fp32, each with twice what four of its roundings can amount to
  // (and never 0, which as a key lies above -0): a candidate is at least
  // at_least(k, x), and one of t or more has a logit of at least low_of(k, t).
  auto slack = [&](int k, float x) {
    return 1e-30f + 4.8e-7f * (fabsf(score32[k]) + fabsf(base32[k]) + fabsf(less32[k]) + fabsf(x));
  };
  auto at_least = [&](int k, float x) {
    return state[k] == 2 ? score32[k] : score32[k] + ((x - base32[k]) - less32[k]) - slack(k, x);
  };
  auto low_of = [&](int k, float t) {
    const float x = fminf(((t - score32[k]) + less32[k]) + base32[k], FLT_MAX) - slack(k, t);
    return x > -FLT_MAX ? x : -FLT_MAX;
  };

  // ---- the n best units ----
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
  // every unit whose candidates may reach `bound`; finished beams are a unit of their own
  float bound = -INFINITY;
  auto each_unit = [&](auto&& f) {
    for (int i = warp; i < a.K * share; i += kMW) {
      const int k = i / share, from = (i - k * share) * 32 + lane;
      if (state[k] == 2) {
        if (from == 0) f(place_of(k, 0u, 0u));
      } else if (state[k] == 1) {
        const uint32_t least = float_order_key(low_of(k, bound));
        const uint32_t* ur = units + (int64_t)k * U;
        const uint32_t* pr = pieces + (int64_t)k * P;
        const int end = row_pieces(k);
        auto take = [&](uint32_t fk, int u) {
          // -0 and 0 are one logit
          if (fk >= least) f(place_of(k, float_order_key(order_key_float(fk) + 0.0f), (uint32_t)u));
        };
        for (int i0 = wide * from; i0 < end; i0 += step) {
          const uint4 v = some_pieces(pr, i0, end);
          if (max(max(v.x, v.y), max(v.z, v.w)) < least) continue;
          const uint32_t p[4] = {v.x, i0 + 1 < end ? v.y : 0u, i0 + 2 < end ? v.z : 0u, i0 + 3 < end ? v.w : 0u};
          if (a.nv == 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) take(p[j], i0 + j);
            continue;
          }
          uint4 w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = p[j] >= least ? *reinterpret_cast<const uint4*>(ur + 4 * (i0 + j)) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            take(w[j].x, 4 * (i0 + j));
            take(w[j].y, 4 * (i0 + j) + 1);
            take(w[j].z, 4 * (i0 + j) + 2);
            take(w[j].w, 4 * (i0 + j) + 3);
          }
        }
      }
    }
  };
  {
    // the n-th largest maximum of groups of a beam's units bounds the n-th unit
    const int all = a.K * share * 32;
    int group = 1;  // lanes; at least 3 n groups, at most kMergeThreads
    while (all / group > kMergeThreads || (group < 32 && all / (2 * group) >= max(3 * n, 32))) group *= 2;
    const int per = 32 / group, groups = all / group;
    for (int i = warp; i < a.K * share; i += kMW) {
      const int k = i / share, from = (i - k * share) * 32 + lane;
      uint32_t fk = 0;
      if (state[k] == 1) {
        const uint32_t* pr = pieces + (int64_t)k * P;
        const int end = row_pieces(k);
#pragma unroll 4
        for (int i2 = wide * from; i2 < end; i2 += step) {
          const uint4 v = some_pieces(pr, i2, end);
          fk = max(fk, max(max(v.x, i2 + 1 < end ? v.y : 0u), max(i2 + 2 < end ? v.z : 0u, i2 + 3 < end ? v.w : 0u)));
        }
      }
      for (int o = 1; o < group; o *= 2) fk = max(fk, __shfl_xor_sync(0xffffffffu, fk, o));
      if (lane % group == 0) {
        const int g = i * per + lane / group;
        // a finished beam is one maximum; kNegInfKey and below: none
        const bool one = state[k] == 2 ? g == k * share * per : fk > kNegInfKey;
        pool.key[g] = (unsigned long long)(one ? float_order_key(at_least(k, order_key_float(fk))) : 0u) << 32 | (unsigned)g;
      }
    }
    __syncthreads();
    rank_words(pool.key, groups, [&](int i, int rank) {
      if (rank == n - 1) tau_s = (uint32_t)(pool.key[i] >> 32);
    });
    __syncthreads();
    bound = order_key_float(tau_s);
  }
  auto approximate = [&](unsigned long long p) { return float_order_key(at_least(place_beam(p), place_logit(p))); };
  // The n-th largest at_least() of all units that may reach the bound, digit by
  // digit: where one beam holds the best n, its few groups bound them badly.
  auto nth_unit = [&]() {
    uint32_t* bins = reinterpret_cast<uint32_t*>(pool.key);
    constexpr int kBins = 2048;
    static_assert(sizeof(pool.key) >= kBins * sizeof(uint32_t), "the bins lie in the pool");
    uint32_t prefix = 0, mask = 0;
    int want = n;
    for (int bit = 21; bit >= 0; bit -= bit == 21 ? 11 : 10) {
      const uint32_t digits = bit ? 2047u : 1023u;
      for (int i = tid; i < kBins; i += kMergeThreads) bins[i] = 0;
      __syncthreads();
      uint32_t bin = 0, count = 0;  // runs of one bin are counted before they are added
      each_unit([&](unsigned long long p) {
        const uint32_t key = approximate(p);
        if ((key & mask) != prefix) return;
        const uint32_t to = (key >> bit) & digits;
        if (to != bin && count) {
          atomicAdd(&bins[bin], count);
          count = 0;
        }
        bin = to;
        ++count;
      });
      if (count) atomicAdd(&bins[bin], count);
      __syncthreads();
      if (warp == 0) {  // from the largest bin on; a lane sums 64 of them
        int sum = 0;
        const int first = kBins - 1 - lane * (kBins / 32);
        for (int i = 0; i < kBins / 32; ++i) sum += (int)bins[first - i];
        int before = sum;
        for (int o = 1; o < 32; o *= 2) {
          const int v = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += v;
        }
        before -= sum;
        if (before < want && before + sum >= want) {
          int i = first;
          while (before + (int)bins[i] < want) before += (int)bins[i--];
          tau_s = prefix | (uint32_t)i << bit;
          tau_want = want - before;
        }
      }
      __syncthreads();
      prefix = tau_s;
      want = tau_want;
      mask |= digits << bit;
    }
    return order_key_float(prefix);
  };
  each_unit([&](unsigned long long p) { pool_add(pool, p); });
  __syncthreads();
  int listed = pool.count;
  if (listed > kPool) {  // at least n of them
    __syncthreads();
    if (tid == 0) pool.count = 0;
    bound = nth_unit();
    each_unit([&](unsigned long long p) { pool_add(pool, p); });
    __syncthreads();
    listed = pool.count;
  }
  // Units are taken by their bounds: those that may reach the n-th, n or a few more.
  if (listed <= kPool) {
    for (int i = tid; i < listed; i += kMergeThreads) pool.key[i] = (unsigned long long)approximate(pool.place[i]) << 32 | (unsigned)i;
    __syncthreads();
    if (tid == 0) pool.count = 0;  // its readers are past the barrier above
    rank_words(pool.key, listed, [&](int i, int rank) {
      if (rank == n - 1) tau_s = (uint32_t)(pool.key[i] >> 32);
    });
    __syncthreads();
    bound = order_key_float(tau_s);
    for (int i = tid; i < listed; i += kMergeThreads) {
      const unsigned long long p = pool.place[i];
      if (state[place_beam(p)] == 2 || place_logit(p) >= low_of(place_beam(p), bound)) unit[atomicAdd(&units_taken, 1)] = p;
    }
    __syncthreads();
    if (units_taken > 2 * n) {  // many that fp32 cannot tell apart
      fill_keys(listed);
      __syncthreads();
      rank_pool(pool, listed, [&](int i, int rank) {
        if (rank < n) unit[rank] = pool.place[i];
      });
      if (tid == 0) units_taken = n;
    }
  } else {  // many equal maxima: the next unit in order, n times
    unsigned long long k, p;
    for (int r = 0; r < n; ++r) {
      next_best(each_unit, key_of, last, k, p, wk, wp);
      if (tid == 0) unit[r] = p;
    }
    bound = (float)key_value(k);
    if (tid == 0) {
      pool.count = 0;
      units_taken = n;
    }
  }
  __syncthreads();
  // ---- their elements ----
  const int chosen = units_taken;
  auto each_element = [&](auto&& f) {
    for (int i = warp; i < chosen; i += kMW) {
      const int k = place_beam(unit[i]), u = (int)place_index(unit[i]);
      if (state[k] == 2) {
        if (lane == 0) f(place_of(k, 0u, (uint32_t)a.pad));
        continue;
      }
      const raw* xr = reinterpret_cast<const raw*>(a.x) + (b * a.K + k) * a.ldx;
      const int lead = (int)((reinterpret_cast<uintptr_t>(xr) & 15) / sizeof(raw));
      const float low = low_of(k, bound);
      uint4 q[1];
      const int e = u * 32 * VEC - lead;
      load_vectors<DT, 1>(q, xr, e, a.V);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float x = elem<DT>(q[0], j);
        if (x >= low) f(place_of(k, float_order_key(x + 0.0f), (uint32_t)(e + lane * VEC + j)));
      }
    }
  };
  each_element([&](unsigned long long p) { pool_add(pool, p); });
  __syncthreads();
  const int found = pool.count;
  float* os = a.out_score + b * n;
  int32_t* op = a.out_parent + b * n;
  int32_t* ot = a.out_token + b * n;
  auto put = [&](int r, unsigned long long k, unsigned long long place) {
    os[r] = k ? (float)key_value(k) : -INFINITY;
    op[r] = k ? place_beam(place) : r % a.K;
    ot[r] = k ? (int32_t)place_index(place) : -1;
  };
  if (found <= kPool) {
    fill_keys(found);
    __syncthreads();
    rank_pool(pool, found, [&](int i, int rank) {
      if (rank < n) put(rank, pool.key[i], pool.place[i]);
    });
    for (int r = found + tid; r < n; r += kMergeThreads) put(r, 0ull, 0ull);
    return;
  }
  // many equal elements: the next one in order, n times
  if (tid < a.K) last[tid] = ~0ull;
  __syncthreads();
  for (int r = 0; r < n; ++r) {
    unsigned long long k, p;
    next_best(each_element, key_of, last, k, p, wk, wp);
    if (tid == 0) put(r, k, p);
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
