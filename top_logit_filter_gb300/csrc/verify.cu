// topkp_draft_verify: drafted tokens against the target's probabilities.
//
// A request is walked down from its root by one cluster of CTAs.  At node n
// the children are tried in turn.  With p and q the target's and the draft's
// distributions after n, what is left of p after k rejected children is
//   p_k = norm(max(p_{k-1} - q, 0)) = max(p - a_k q, 0) / W_k,
//   a_{k+1} = a_k + W_k,   W_k = sum max(p - a_k q, 0),   a_0 = 0, W_0 = 1,
// so a child costs two probabilities, and a further child one pass over the
// node's two rows.  The token drawn when no child is accepted is the largest
// of max(p - a q, 0) / (race + eps): no normaliser, no prefix sums.  Where
// children are certain what is left is the row less the tokens tried: W loses
// p(x), and is summed afresh, by a pass over the row without them, when less
// than half of the last sum is left and another child asks for it.  (Carried
// on as a difference W keeps the sum's error: off by 12% of itself after a
// token of 1 - 3e-7.)
//
// Only rows down the accepted path are needed (about four of a tree of 64
// nodes).  Rows are cut over the cluster's CTAs; a row's second reading comes
// from L2.  Each warp hands its maximum and sum to every CTA of the cluster
// through distributed shared memory, so that a pass ends in one barrier and
// every CTA takes the same decision by itself.  A step reads the rows of
// several nodes, each the first child of the one before, unless that alone
// keeps DRAM busy: a chain whose tokens are accepted is then decided at once.
//
// Sums are fp32: a thread's batches of up to 64 terms, then its batches, warps,
// and the cluster's warps.  Probabilities that decide are fp32 with the
// exponent's rounding put back (exp_one).
//
// Measured (one call in a graph): one request of 5 x 32000 fp16 12.4 us, a chain
// of launch, one step and the draw; 64 chains of 6 x 128256 bf16 47.6, 189 MB
// from DRAM at 4.0 TB/s where 144 are needed, bound by the latency of a step
// (scan 5 to 6 us, barrier and decision 2) and by the few requests that go to
// the end; 128 chains of 8 x 152064 fp32 159, 4.3 TB/s over what is needed; 32
// trees of 64 x 151936 bf16 51, a chain of short steps; 64 x 6 x 128255, whose
// rows are unaligned, 52.
#include <limits.h>
#include <type_traits>

#include "common.cuh"
#include "decode.h"

namespace topkp {
namespace {

constexpr int kVW = kVerifyThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;   // (off by 2^-26 of itself: a sum whose terms lie e^-20 below the largest by 3e-7)
constexpr float kLog2eHi = 1.44268798828125f;  // log2 e to 16 bits
constexpr float kLog2eLo = 7.0526077e-06f;     // the rest

__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void apart(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t add_two(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_two(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_two(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float ex2(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}
// exp(t), t <= 0, with log2 e to 40 bits: the exponent is off by half a step
// of its own, which evens out over a sum.
__device__ __forceinline__ float exp_fast(float t) { return ex2(fmaf(t, kLog2eHi, t * kLog2eLo)); }
// exp(x - m), x <= m, where a single one decides: the rounding of x - m and
// of the exponent go into a factor 1 + d.
__device__ __forceinline__ float exp_one(float x, float m) {
  const float t = fmaxf(x - m, -200.0f);  // (2^-288 is zero)
  const float back = t + m;
  const float lost = t > -200.0f ? (x - back) + ((back - t) - m) : 0.0f;  // x - m - t
  const float y = t * kLog2eHi;  // 16 bits by 24: rounded
  const float d = fmaf(t, kLog2eHi, -y) + fmaf(t, kLog2eLo, lost * 1.4426950f);
  const float e = ex2(y);
  return fmaf(e, d * 0.69314718f, e);
}

// A thread's share of a row: its largest element and the sum of exp(x - m).
struct Sum {
  float m, s;
};

// A row as vectors of 16 bytes: `head` elements before the first of them, and
// what is left behind the last.
template <int DT>
struct Row {
  using raw = typename DType<DT>::raw;
  static constexpr int VEC = 16 / (int)sizeof(raw);
  const raw* x;
  int V, head, vectors;
  __device__ __forceinline__ Row(const raw* p, int n) : x(p), V(n) {
    head = min((int)((16 - ((uintptr_t)p & 15)) % 16 / sizeof(raw)), n);
    vectors = (n - head) / VEC;
  }
  __device__ __forceinline__ const uint4* at(int v) const { return reinterpret_cast<const uint4*>(x + head) + v; }
  // element k of those that lie in no vector, up to 2 VEC - 2 of them: its place, or -1
  __device__ __forceinline__ int loose(int k) const {
    const int i = k < head ? k : k + vectors * VEC;
    return i < V ? i : -1;
  }
};
template <int DT>
__device__ __forceinline__ uint4 nothing() {
  constexpr uint32_t n = DType<DT>::kNegInf;
  constexpr uint32_t w = DT == TOPKP_F32 ? n : n | n << 16;
  return make_uint4(w, w, w, w);
}
// Pair j of a vector.
template <int DT>
__device__ __forceinline__ void pair_of(const uint4& q, int j, float& a, float& b) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if (DT == TOPKP_F32) {
    a = __uint_as_float(w[2 * j % 4]);
    b = __uint_as_float(w[(2 * j + 1) % 4]);
  } else if (DT == TOPKP_BF16) {
    a = __uint_as_float(w[j] << 16);
    b = __uint_as_float(w[j] & 0xffff0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
    a = f.x;
    b = f.y;
  }
}

// The largest element of U vectors; 16-bit types two at a time.
template <int DT, int U>
__device__ __forceinline__ float largest(const uint4 (&q)[U]) {
  if constexpr (DT == TOPKP_F32) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(q[u].x), __uint_as_float(q[u].y)), fmaxf(__uint_as_float(q[u].z), __uint_as_float(q[u].w))));
    return m;
  } else {
    using pair = typename std::conditional<DT == TOPKP_F16, __half2, __nv_bfloat162>::type;
    auto as = [](const uint32_t& w) { return *reinterpret_cast<const pair*>(&w); };
    pair m = __hmax2(__hmax2(as(q[0].x), as(q[0].y)), __hmax2(as(q[0].z), as(q[0].w)));
#pragma unroll
    for (int u = 1; u < U; ++u) m = __hmax2(m, __hmax2(__hmax2(as(q[u].x), as(q[u].y)), __hmax2(as(q[u].z), as(q[u].w))));
    if constexpr (DT == TOPKP_F16) {
      const float2 f = __half22float2(m);
      return fmaxf(f.x, f.y);
    } else {
      const float2 f = __bfloat1622float2(m);
      return fmaxf(f.x, f.y);
    }
  }
}
// U vectors into a thread's share.
template <int DT, int U>
__device__ __forceinline__ void absorb(const uint4 (&q)[U], Sum& s) {
  constexpr int PAIRS = Row<DT>::VEC / 2;
  const float mx = largest<DT, U>(q);
  if (mx > s.m) {
    s.s *= s.m == -INFINITY ? 0.0f : exp_fast(s.m - mx);
    s.m = mx;
  }
  if (s.m == -INFINITY) return;
  const uint64_t less = two(-s.m, -s.m), scale = two(kLog2e, kLog2e);
  uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      float a, b;
      pair_of<DT>(q[u], j, a, b);
      apart(mul_two(add_two(two(a, b), less), scale), a, b);
      sum[j & 1] = add_two(sum[j & 1], two(ex2(a), ex2(b)));
    }
  float a, b;
  apart(add_two(sum[0], sum[1]), a, b);
  s.s += a + b;
}

__device__ __forceinline__ void prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

constexpr int kAhead = 4;  // nodes of a step, at most
enum { kGo, kPass, kDraw };

// What the warps of a cluster hand to each other, and what a step leaves.
struct Shared {
  float4 part[2][kAhead][16 * kVW];
  int32_t parent[TOPKP_MAX_TREE], tokens[TOPKP_MAX_TREE], path[TOPKP_MAX_TREE], tried[TOPKP_MAX_TREE];
  float uniform[TOPKP_MAX_TREE];
  float xt[TOPKP_MAX_TREE], xd[TOPKP_MAX_TREE];    // the children's logits
  float gap[TOPKP_MAX_TREE], sum[TOPKP_MAX_TREE];  // of the emitted tokens: logit less the row's largest, the row's sum
  // the node that the walk has come to
  float mt, md, st, sd;     // the rows' largest logits and sums of exponentials
  float weight, factor;     // W and a of the comment above, times st and st / sd
  unsigned long long open;  // children to be tried
  unsigned long long bloom;  // of the tokens tried, eight neighbours to a bit
  unsigned long long best;
  uint32_t bound;  // a candidate's key of the draw
  int state, node, depth, tries, top, token;
  int n;                    // nodes of the request
  const void *target, *draft;  // its rows
};

struct Team {
  int cs;
  uint32_t rank;
  int at;  // which of the two sets of parts
};

__device__ __forceinline__ void team_sync(const Team& t) {
  __syncwarp();
  if (t.cs > 1) cluster_sync_all();
  else __syncthreads();
}
// This warp's part to all CTAs, a lane a CTA.
__device__ __forceinline__ void hand_out(const Team& t, Shared& sh, int set, int place, const float4& v) {
  const int lane = threadIdx.x & 31;
  if (lane < t.cs) {
    float4* to = &sh.part[t.at][set][place];
    if (t.cs == 1) {
      *to = v;
    } else {
      const uint32_t a = dsmem_addr(to, (uint32_t)lane);
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
    }
  }
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v ? w : v;
  }
  return v;
}
// Maxima and sums of both rows over the warps' n parts, by one warp: a lane's
// up to eight parts side by side, since one after another their latency was
// most of a step's time.
template <bool DRAFT>
__device__ __forceinline__ void join_sums(const float4* part, int n, float& mt, float& st, float& md, float& sd) {
  constexpr int E = 16 * kVW / 32;
  const int lane = threadIdx.x & 31;
  float4 v[E];
#pragma unroll
  for (int k = 0; k < E; ++k) v[k] = lane + 32 * k < n ? part[lane + 32 * k] : make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
  mt = v[0].x;
  md = v[0].z;
#pragma unroll
  for (int k = 1; k < E; ++k) {
    mt = fmaxf(mt, v[k].x);
    md = fmaxf(md, v[k].z);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    if (DRAFT) md = fmaxf(md, __shfl_xor_sync(0xffffffffu, md, o));
  }
  const float rt = mt == -INFINITY ? 0.0f : mt, rd = md == -INFINITY ? 0.0f : md;
  st = sd = 0.0f;
#pragma unroll
  for (int k = 0; k < E; ++k) {
    if (k > 0 && 32 * k >= n) break;
    st = fmaf(v[k].y, exp_fast(v[k].x - rt), st);
    if (DRAFT) sd = fmaf(v[k].w, exp_fast(v[k].z - rd), sd);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    st += __shfl_xor_sync(0xffffffffu, st, o);
    if (DRAFT) sd += __shfl_xor_sync(0xffffffffu, sd, o);
  }
}
// A warp's shares as one.
__device__ __forceinline__ Sum warp_join(const Sum& s) {
  Sum r;
  r.m = s.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r.m = fmaxf(r.m, __shfl_xor_sync(0xffffffffu, r.m, o));
  r.s = warp_sum(s.m == -INFINITY ? 0.0f : s.s * exp_fast(s.m - r.m));
  return r;
}

// Largest element and sum of this CTA's part of a row, by `threads` threads,
// of which this is `who`; a warp's joined.  Rows are given to warps rather
// than both to each: two rows' loads in flight did not fit the registers
// (53 against 45 thousand cycles a step of 128 x 152064 fp32).  With GREEDY
// `first` is the place of the largest.
template <int DT, bool GREEDY>
__device__ __forceinline__ Sum scan(const typename DType<DT>::raw* x, int V, int rank, int cs, int threads, int who, uint32_t& first) {
  constexpr int VEC = Row<DT>::VEC;
  Sum s = {-INFINITY, 0.0f}, loose = {-INFINITY, 0.0f};
  uint32_t at_loose = 0;
  first = 0xffffffffu;
  const Row<DT> r(x, V);
  const int per = (r.vectors + cs - 1) / cs, begin = min(per * rank, r.vectors), n = min(per, r.vectors - begin);
  if (rank == 0 && who < 2 * VEC - 2) {  // what lies in no vector
    const int i = r.loose(who);
    if (i >= 0) {
      // (greedy: apart, since it may lie behind the vectors, and of equal elements the first counts)
      Sum& one = GREEDY ? loose : s;
      one.m = DType<DT>::to_float(x[i]);
      one.s = one.m > -INFINITY ? 1.0f : 0.0f;
      at_loose = (uint32_t)i;
    }
  }
  const uint4* p = r.at(begin) + who;
  const int place = (begin + who) * VEC + r.head;
  // U vectors, all read before the first is used; `all`: none is beyond the end
  auto take = [&](auto count, auto all, int at) {
    constexpr int U = decltype(count)::value;
    constexpr bool ALL = decltype(all)::value;
    uint4 q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) q[u] = ALL || at + u * threads + who < n ? __ldg(p + at + u * threads) : nothing<DT>();
    const float before = s.m;
    absorb<DT, U>(q, s);
    if (GREEDY && s.m > before) {  // its first place
#pragma unroll
      for (int u = U - 1; u >= 0; --u)
#pragma unroll
        for (int j = VEC / 2 - 1; j >= 0; --j) {
          float a, b;
          pair_of<DT>(q[u], j, a, b);
          const uint32_t e = (uint32_t)(place + (at + u * threads) * VEC + 2 * j);
          if (b == s.m) first = e + 1;
          if (a == s.m) first = e;
        }
    }
  };
  using One = std::integral_constant<int, 1>;
  using Eight = std::integral_constant<int, 8>;
  int at = 0;
  for (; at + 8 * threads <= n; at += 8 * threads) take(Eight(), std::true_type(), at);
  if (n - at > threads) {
    take(Eight(), std::false_type(), at);
  } else if (n > at) {
    take(One(), std::false_type(), at);
  }
  if (GREEDY && loose.m > -INFINITY) {
    if (loose.m > s.m) {
      s.s = s.m == -INFINITY ? 0.0f : s.s * exp_fast(s.m - loose.m);
      s.m = loose.m;
      first = at_loose;
    } else if (loose.m == s.m) {
      first = min(first, at_loose);
    }
    s.s += exp_fast(loose.m - s.m);
  }
  const Sum w = warp_join(s);
  if (GREEDY) first = __reduce_min_sync(0xffffffffu, s.m == w.m ? first : 0xffffffffu);
  return w;
}

// A candidate of the draw: the larger key, the lower index.
__device__ __forceinline__ unsigned long long candidate(float key, int i) {
  return (unsigned long long)__float_as_uint(key) << 32 | (uint32_t)~i;
}
// The children of a node, by a whole warp.
__device__ __forceinline__ unsigned long long children(const Shared& sh, int node, int n) {
  const int lane = threadIdx.x & 31;
  const bool lo = lane > node && lane < n && sh.parent[lane] == node;
  const bool hi = lane + 32 > node && lane + 32 < n && sh.parent[lane + 32] == node;
  return __ballot_sync(0xffffffffu, lo) | (unsigned long long)__ballot_sync(0xffffffffu, hi) << 32;
}

// This CTA's elements of a row.
template <int DT>
__device__ __forceinline__ void part_of(const VerifyArgs& a, const Team& team, int& first, int& last) {
  constexpr int VEC = Row<DT>::VEC;
  const int per = ((a.V + a.cs - 1) / a.cs + VEC - 1) / VEC * VEC;
  first = min(per * (int)team.rank, a.V);
  last = min(first + per, a.V);
}

// A thread's sum of max(exp(x - mt) - factor exp(y - md), 0).
template <int DT>
__device__ __forceinline__ float weigh(const VerifyArgs& a, const Team& team, const typename DType<DT>::raw* t,
                                       const typename DType<DT>::raw* d, float mt, float md, float factor) {
  constexpr int VEC = Row<DT>::VEC, U = 4;
  int first, last;
  part_of<DT>(a, team, first, last);
  float sum = 0.0f;
  if (mt == -INFINITY) return 0.0f;
  const bool drafted = md > -INFINITY;
  const uint64_t hi = two(kLog2eHi, kLog2eHi), lo = two(kLog2eLo, kLog2eLo);
  const uint64_t lt = two(-mt, -mt), ld = drafted ? two(-md, -md) : 0ull;
  auto exps = [&](float& x, float& y, uint64_t less) {
    const uint64_t v = add_two(two(x, y), less);
    apart(fma_two(v, hi, mul_two(v, lo)), x, y);
    x = ex2(x);
    y = ex2(y);
  };
  auto add = [&](float x, float y, float c, float g) {
    exps(x, y, lt);
    exps(c, g, ld);
    sum += fmaxf(fmaf(-factor, c, x), 0.0f) + fmaxf(fmaf(-factor, g, y), 0.0f);
  };
  if (a.whole) {
    for (int i0 = first + (int)threadIdx.x * VEC; i0 < last; i0 += U * kVerifyThreads * VEC) {
      uint4 qt[U], qd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kVerifyThreads * VEC;
        qt[u] = i < last ? __ldg(reinterpret_cast<const uint4*>(t + i)) : nothing<DT>();
        qd[u] = i < last ? __ldg(reinterpret_cast<const uint4*>(d + i)) : nothing<DT>();
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          float x, y, c, g;
          pair_of<DT>(qt[u], j, x, y);
          pair_of<DT>(qd[u], j, c, g);
          add(x, y, c, g);
        }
    }
  } else {
    for (int i = first + (int)threadIdx.x; i < last; i += 2 * kVerifyThreads) {
      const bool two_of = i + kVerifyThreads < last;
      add(DType<DT>::to_float(t[i]), two_of ? DType<DT>::to_float(t[i + kVerifyThreads]) : -INFINITY, DType<DT>::to_float(d[i]),
          two_of ? DType<DT>::to_float(d[i + kVerifyThreads]) : -INFINITY);
    }
  }
  return sum;
}

// Eight neighbouring tokens to a bit.
__device__ __forceinline__ unsigned long long bloom_bit(int x) { return 1ull << ((x >> 3) & 63); }

// A thread's sum of exp(x - mt) over the tokens that have not been tried.  It
// is asked for where the tried ones held most of the row, and few elements may
// be all that counts: each is worked out with care, and what the rounding of a
// sum of vectors drops is kept.  One request of 128256 bf16 that needs it
// takes 6 us more, 64 of them 12.5 (22.5 an element at a time).
template <int DT>
__device__ __forceinline__ float weigh_rest(const VerifyArgs& a, const Team& team, const Shared& sh, const typename DType<DT>::raw* t) {
  constexpr int VEC = Row<DT>::VEC, U = 4;
  int first, last;
  part_of<DT>(a, team, first, last);
  const float mt = sh.mt;
  const unsigned long long bloom = sh.bloom;
  const int tries = sh.tries;
  float sum = 0.0f, low = 0.0f;
  if (mt == -INFINITY) return 0.0f;
  auto add = [&](float e) {
    e -= low;
    const float next = sum + e;
    low = (next - sum) - e;
    sum = next;
  };
  if (a.whole) {
    for (int i0 = first + (int)threadIdx.x * VEC; i0 < last; i0 += U * kVerifyThreads * VEC) {
      uint4 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kVerifyThreads * VEC;
        q[u] = i < last ? __ldg(reinterpret_cast<const uint4*>(t + i)) : nothing<DT>();
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kVerifyThreads * VEC;  // a multiple of VEC, as V is: a vector's elements share a bit
        const bool some = (bloom & bloom_bit(i)) != 0;
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          float x, y;
          pair_of<DT>(q[u], j, x, y);
          if (some)
            for (int k = 0; k < tries; ++k) {
              x = sh.tried[k] == i + 2 * j ? -INFINITY : x;
              y = sh.tried[k] == i + 2 * j + 1 ? -INFINITY : y;
            }
          part += exp_one(x, mt) + exp_one(y, mt);
        }
        add(part);
      }
    }
  } else {
    for (int i0 = first + (int)threadIdx.x; i0 < last; i0 += 2 * U * kVerifyThreads) {
      float x[2 * U];
#pragma unroll
      for (int u = 0; u < 2 * U; ++u) {
        const int i = i0 + u * kVerifyThreads;
        x[u] = i < last ? DType<DT>::to_float(t[i]) : -INFINITY;
      }
      float part = 0.0f;
#pragma unroll
      for (int u = 0; u < 2 * U; ++u) {
        const int i = i0 + u * kVerifyThreads;
        if (bloom & bloom_bit(i))
          for (int k = 0; k < tries; ++k) x[u] = sh.tried[k] == i ? -INFINITY : x[u];
        part += exp_one(x[u], mt);
      }
      add(part);
    }
  }
  return sum;
}

// The best candidate of this warp's elements: the largest
// (exp(x - mt) - factor exp(y - md)) / (variate + eps), of equal ones the
// first.  No element can be better than exp(x - mt) / (variate + eps), which
// a few instructions tell to 2^-14; what that leaves in the race, few
// elements of a row, is worked out with care, a lane's best first, so that
// the bound rises fast.  (With care for every element: 33 thousand cycles a
// CTA for 4 x 128256 bf16 over 64 requests, and the draft's row read again.)
template <int DT, int MODE>
__device__ __forceinline__ unsigned long long draw(const VerifyArgs& a, const Team& team, Shared& sh, const typename DType<DT>::raw* t,
                                                   const typename DType<DT>::raw* d, const float* race, float factor, int tries) {
  constexpr int VEC = Row<DT>::VEC, K = 16, U = K / VEC;
  const float mt = sh.mt, md = sh.md, eps = a.eps;
  int first, last;
  part_of<DT>(a, team, first, last);
  unsigned long long best = 0ull;
  if (mt == -INFINITY) return 0ull;
  for (int base = first; base < last; base += K * kVerifyThreads) {
    // element k of this thread; about what it is in the race
    auto place = [&](int k) {
      return base + (a.whole ? ((k / VEC) * kVerifyThreads + (int)threadIdx.x) * VEC + k % VEC : k * kVerifyThreads + (int)threadIdx.x);
    };
    float r[K];
    auto rough = [&](int k, float x, float y, float v, float w) {
      const uint64_t e = mul_two(add_two(two(x, y), two(-mt, -mt)), two(1.4426950408889634f, 1.4426950408889634f));
      float p, q, g, h;
      apart(e, p, q);
      apart(add_two(two(v, w), two(eps, eps)), g, h);
      asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(g));
      asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(h));
      r[k] = ex2(p) * g;
      r[k + 1] = ex2(q) * h;
    };
    if (a.whole) {
      uint4 q[U];
      float4 v[U][VEC / 4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = place(u * VEC);
        q[u] = i < last ? __ldg(reinterpret_cast<const uint4*>(t + i)) : nothing<DT>();
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) v[u][k] = i < last ? __ldg(reinterpret_cast<const float4*>(race + i) + k) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          float x, y;
          pair_of<DT>(q[u], j, x, y);
          rough(u * VEC + 2 * j, x, y, j & 1 ? v[u][j / 2].z : v[u][j / 2].x, j & 1 ? v[u][j / 2].w : v[u][j / 2].y);
        }
    } else {
#pragma unroll
      for (int k = 0; k < K; k += 2) {
        const int i = place(k), j = place(k + 1);
        rough(k, i < last ? DType<DT>::to_float(t[i]) : -INFINITY, j < last ? DType<DT>::to_float(t[j]) : -INFINITY,
              i < last ? race[i] : 1.0f, j < last ? race[j] : 1.0f);
      }
    }
    for (;;) {
      float top = r[0];
#pragma unroll
      for (int k = 1; k < K; ++k) top = fmaxf(top, r[k]);
      const uint32_t bound = *(volatile uint32_t*)&sh.bound;
      const bool go = top > 0.0f && top * 1.00006103515625f >= __uint_as_float(bound);
      if (!__any_sync(0xffffffffu, go)) break;
      if (go) {
        int at = 0;
        bool found = false;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const bool me = !found && r[k] == top;
          if (me) {
            at = k;
            r[k] = 0.0f;
          }
          found = found || me;
        }
        const int i = place(at);
        float e = exp_one(DType<DT>::to_float(t[i]), mt);
        if (MODE == kVerifyRatio && factor > 0.0f) {
          const float y = DType<DT>::to_float(d[i]);
          if (y > -INFINITY) e = fmaxf(fmaf(-factor, exp_one(y, md), e), 0.0f);
        }
        if (MODE == kVerifyCertain)
          for (int k = 0; k < tries; ++k)
            if (sh.tried[k] == i) e = 0.0f;
        if (e > 0.0f) {
          const float key = __fdiv_rn(e, race[i] + eps);
          const unsigned long long c = candidate(key, i);
          best = c > best ? c : best;
          if (__float_as_uint(key) > bound) atomicMax(&sh.bound, __float_as_uint(key));
        }
      }
      __syncwarp();
    }
  }
  return warp_max(best);
}

// The walk as far as the rows that were read go, by one warp: children in
// turn, on to the next node of the step where its token is accepted.  `set`
// is the node's among the step's, of `parts` parts each; resumed: after a pass for the weight of
// what is left at sh.node.
template <int DT, int MODE>
__device__ __forceinline__ void decide(const VerifyArgs& a, const Team& team, Shared& sh, int n, int sets, int parts, bool resumed) {
  constexpr bool DRAFT = MODE == kVerifyRatio, GREEDY = MODE == kVerifyGreedy;
  const int lane = threadIdx.x & 31;
  int node = sh.node, depth = sh.depth, state = kDraw, tries = resumed ? sh.tries : 0, top = -1;
  float mt = sh.mt, md = sh.md, st = sh.st, sd = sh.sd, weight = sh.weight, factor = sh.factor;
  unsigned long long open = sh.open, bloom = resumed ? sh.bloom : 0ull;
  float whole = 0.0f;
  if (resumed) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 16 * kVW / 32; ++k)
      if (lane + 32 * k < parts) sum += sh.part[team.at][0][lane + 32 * k].x;
    weight = whole = warp_sum(sum);
  }
  float inverse = 1.0f / sd;
  for (int set = 0;;) {
    if (!resumed) {
      join_sums<DRAFT>(sh.part[team.at][set], parts, mt, st, md, sd);
      if (GREEDY) {
        uint32_t f = 0xffffffffu;
        for (int i = lane; i < parts; i += 32) {
          const float4 v = sh.part[team.at][set][i];
          if (v.x == mt) f = min(f, __float_as_uint(v.z));
        }
        top = (int)__reduce_min_sync(0xffffffffu, f);
        if (mt == -INFINITY || top < 0 || top >= a.V) top = -1;
      }
      inverse = 1.0f / sd;
      open = children(sh, node, n);
      weight = whole = st;
      factor = 0.0f;
      tries = 0;
      bloom = 0ull;
    }
    const int next = open ? __ffsll((long long)open) - 1 : -1;  // the step's next node, where this is not resumed
    int chosen = -1;
    state = kDraw;
    while (open) {
      const int c = __ffsll((long long)open) - 1;
      open &= open - 1;
      const int x = sh.tokens[c];
      if (x < 0 || x >= a.V) continue;
      if (GREEDY) {
        if (x == top) chosen = c;
      } else {
        float left = exp_one(sh.xt[c], mt), q = 1.0f;
        if (sh.xt[c] == -INFINITY) left = 0.0f;
        if (DRAFT) {
          q = sd > 0.0f && sh.xd[c] > -INFINITY ? exp_one(sh.xd[c], md) : 0.0f;
          if (sh.uniform[c] * (q * inverse) * weight < fmaf(-factor, q, left) || (q == 0.0f && left > 0.0f)) {
            chosen = c;
          } else {
            if (sd > 0.0f) factor += weight * inverse;
            if (open) {
              state = kPass;
              break;
            }
          }
        } else {
          if (bloom & bloom_bit(x))
            for (int i = 0; i < tries; ++i)
              if (sh.tried[i] == x) left = 0.0f;
          if (sh.uniform[c] * weight < left) {
            chosen = c;
          } else if (left > 0.0f) {
            weight = fmaxf(weight - left, 0.0f);
            if (lane == 0) sh.tried[tries] = x;
            __syncwarp();
            ++tries;
            bloom |= bloom_bit(x);
            if (open && weight < 0.5f * whole) {
              state = kPass;
              break;
            }
          }
        }
      }
      if (chosen >= 0) break;
    }
    if (chosen < 0) break;
    if (lane == 0) {
      sh.gap[depth] = GREEDY ? 0.0f : sh.xt[chosen] - mt;
      sh.sum[depth] = st;
      sh.path[depth + 1] = chosen;
    }
    ++depth;
    node = chosen;
    state = kGo;
    if (resumed || chosen != next || ++set >= sets) break;
  }
  if (lane == 0) {
    sh.state = state;
    sh.node = node;
    sh.depth = depth;
    sh.mt = mt;
    sh.md = md;
    sh.st = st;
    sh.sd = sd;
    sh.weight = weight;
    sh.factor = factor;
    sh.open = open;
    sh.bloom = bloom;
    sh.tries = tries;
    sh.top = top;
  }
}

template <int DT, int MODE>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const __grid_constant__ VerifyArgs a) {
  using raw = typename DType<DT>::raw;
  constexpr bool DRAFT = MODE == kVerifyRatio, GREEDY = MODE == kVerifyGreedy;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Team team = {a.cs, a.cs > 1 ? cluster_ctarank() : 0u, 0};
  if (a.cs > 1) cluster_arrive();
  {
    const int64_t b = blockIdx.x / a.cs;
    const int n = a.nodes ? min(max(a.nodes[b], 0), a.T) : a.T;
    if (tid < a.T) {
      const int64_t i = b * a.T + tid;
      sh.parent[tid] = a.parent ? a.parent[i] : tid - 1;
      sh.tokens[tid] = a.tokens[i];
      sh.uniform[tid] = a.uniform ? a.uniform[i] : 0.0f;
      sh.path[tid] = tid == 0 && n > 0 ? 0 : -1;
    }
    if (tid == 0) {
      sh.node = sh.depth = sh.bound = 0;
      sh.token = -1;
      sh.n = n;
      sh.target = reinterpret_cast<const raw*>(a.target) + b * a.t_batch;
      sh.draft = reinterpret_cast<const raw*>(a.draft) + (DRAFT ? b * a.d_batch : 0);
    }
  }
  __syncthreads();
  // every CTA of the cluster has started before one writes into another's memory
  if (a.cs > 1) cluster_wait();
  // (what a pass does not need waits in shared memory: its loads take half the registers)
  auto target = [&](int node) { return reinterpret_cast<const raw*>(sh.target) + node * a.t_node; };
  auto draft = [&](int node) { return reinterpret_cast<const raw*>(sh.draft) + (DRAFT ? node * a.d_node : 0); };
  while (sh.n > 0) {
    // Largest elements and sums of the node's rows, and of its first child's
    // and so on: all warps a node, or half or a quarter of them.
    int sets = 0;
    {
      int list[kAhead], next = sh.node, node = -1;
#pragma unroll
      for (int g = 0; g < kAhead; ++g) {
        list[g] = next;
        if (next >= 0 && g < a.ahead) {
          ++sets;
          const unsigned long long kids = children(sh, next, sh.n);
          next = kids ? __ffsll((long long)kids) - 1 : -1;
        }
      }
      const int parts = kVW / (sets > 2 ? 4 : sets), which = warp / parts, threads = 32 * parts, who = tid & (threads - 1);
#pragma unroll
      for (int g = 0; g < kAhead; ++g)
        if (g == which && g < sets) node = list[g];
      if (node >= 0) {
        auto token_of = [&]() {  // a child's token; none of the vocabulary for other threads
          return !GREEDY && who < TOPKP_MAX_TREE && (children(sh, node, sh.n) >> (who & 63) & 1) ? sh.tokens[who] : -1;
        };
        const bool drafted = DRAFT && children(sh, node, sh.n) != 0;
        int x = token_of();
        if (x >= 0 && x < a.V) {  // the children's logits: asked for early, read once the row is through
          prefetch(target(node) + x);
          if (DRAFT) prefetch(draft(node) + x);
        }
        // the second half of the warps takes the draft's row, where there are children
        const int half = threads / 2;
        const bool second = drafted && who >= half;
        uint32_t first;
        const Sum got = scan<DT, GREEDY>(second ? draft(node) : target(node), a.V, (int)team.rank, a.cs, drafted ? half : threads,
                                         drafted ? who & (half - 1) : who, first);
        float4 mine = make_float4(got.m, got.s, -INFINITY, 0.0f);
        if (DRAFT && second) mine = make_float4(-INFINITY, 0.0f, got.m, got.s);
        if (GREEDY) mine.z = __uint_as_float(first);
        x = token_of();
        if (x >= 0 && x < a.V) {
          sh.xt[who] = DType<DT>::to_float(target(node)[x]);
          if (DRAFT) sh.xd[who] = DType<DT>::to_float(draft(node)[x]);
        }
        hand_out(team, sh, which, (int)team.rank * parts + warp % parts, mine);
      }
    }
    team_sync(team);
    for (bool resumed = false;; resumed = true) {
      if (warp == 0) decide<DT, MODE>(a, team, sh, sh.n, sets, (resumed ? kVW : kVW / (sets > 2 ? 4 : sets)) * a.cs, resumed);
      team.at ^= 1;
      __syncthreads();
      if (GREEDY || sh.state != kPass) break;
      // the weight of what is left: the sum of max(p - a q, 0), or of p but for the tokens tried
      float sum;
      if constexpr (DRAFT) sum = weigh<DT>(a, team, target(sh.node), draft(sh.node), sh.mt, sh.md, sh.factor);
      else sum = weigh_rest<DT>(a, team, sh, target(sh.node));
      sum = warp_sum(sum);
      hand_out(team, sh, 0, (int)team.rank * kVW + warp, make_float4(sum, 0.0f, 0.0f, 0.0f));
      team_sync(team);
    }
    if (sh.state == kGo) continue;
    // the draw, from what is left; from the whole where nothing is
    if (GREEDY) {
      if (tid == 0) sh.token = sh.top;
    } else {
      float factor = DRAFT ? sh.factor : 0.0f;
      int tries = sh.tries;
      for (int round = 0;; ++round) {
        unsigned long long best =
            draw<DT, MODE>(a, team, sh, target(sh.node), draft(sh.node), a.race + (blockIdx.x / a.cs) * a.ld_race, factor, tries);
        hand_out(team, sh, 0, (int)team.rank * kVW + warp, make_float4(__uint_as_float((uint32_t)best), __uint_as_float((uint32_t)(best >> 32)), 0.0f, 0.0f));
        team_sync(team);
        if (warp == 0) {
          best = 0ull;
          for (int i = lane; i < a.cs * kVW; i += 32) {
            const float4 v = sh.part[team.at][0][i];
            const unsigned long long c = (unsigned long long)__float_as_uint(v.y) << 32 | __float_as_uint(v.x);
            best = c > best ? c : best;
          }
          best = warp_max(best);
          if (lane == 0) {
            sh.best = best;
            sh.token = best ? (int)~(uint32_t)best : -1;
          }
        }
        team.at ^= 1;
        __syncthreads();
        if (sh.best || round || (factor == 0.0f && tries == 0)) break;
        factor = 0.0f;
        tries = 0;
        __syncthreads();
      }
    }
    if (tid == 0) {
      const int token = sh.token;
      sh.gap[sh.depth] = token >= 0 ? DType<DT>::to_float(target(sh.node)[token]) - sh.mt : 0.0f;
      sh.sum[sh.depth] = token >= 0 ? sh.st : 1.0f;
    }
    __syncthreads();
    break;
  }
  if (team.rank == 0) {
    const int64_t b = blockIdx.x / a.cs;
    if (tid < a.T) {
      a.path[b * a.T + tid] = sh.path[tid];
      if (a.logprob) a.logprob[b * a.T + tid] = sh.n > 0 && tid <= sh.depth ? sh.gap[tid] - logf(sh.sum[tid]) : 0.0f;
    }
    if (tid == 0) {
      a.count[b] = sh.n > 0 ? sh.depth + 1 : 0;
      a.token[b] = sh.token;
    }
  }
  // none leaves while another may still write into its memory
  __syncwarp();
  if (a.cs > 1) cluster_sync_all();
}

template <int DT, int MODE>
cudaError_t launch_mode(const VerifyArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * a.cs));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)a.cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.cs > 1 ? 1 : 0;
  if (a.cs > 8) {
    const cudaError_t e = cudaFuncSetAttribute(verify_kernel<DT, MODE>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, verify_kernel<DT, MODE>, a);
}
template <int DT>
cudaError_t launch_dt(const VerifyArgs& a, cudaStream_t s) {
  if (!a.race) return launch_mode<DT, kVerifyGreedy>(a, s);
  return a.draft ? launch_mode<DT, kVerifyRatio>(a, s) : launch_mode<DT, kVerifyCertain>(a, s);
}

}  // namespace

// CTAs of a request: as many as two an SM allow, but none with fewer than 256
// vectors of a row, and 16 (whose barriers take longer) only while they leave
// half the SMs alone: 4 requests of 128256 bf16 17.5 us with 16 and 19.6 with
// 8, 16 requests 31.3 and 25.7; 64 requests 48 with 4, 60 with 8, 55 with 2.
//
// Nodes of a step, ahead of what is known to be accepted: with the draft's
// probabilities most children are, so four, unless a node's rows alone keep
// DRAM busy (128 x 152064 fp32: one 158 us, four 168; 64 chains over 128256
// bf16: one 57.5, four 48; one request of 32000 fp16 19.8 and 13.4); two where
// children are certain or greedy, which fewer are (64 x 128256 bf16, greedy:
// one 19.6, two 17.5, four 20.0).
void verify_plan(int64_t B, int64_t V, int esize, bool draft, int num_sms, int* cs, int* ahead) {
  const int64_t vectors = (V * esize + 15) / 16;
  *cs = 1;
  while (*cs < 16 && B * *cs * 2 <= (*cs == 8 ? num_sms / 2 : 2LL * num_sms) && vectors >= 256LL * *cs * 2) *cs *= 2;
  const int64_t bytes = B * V * esize * (draft ? 2 : 1);
  *ahead = bytes > 64 << 20 ? 1 : draft ? kAhead : 2;
}

cudaError_t launch_verify(topkp_dtype dt, const VerifyArgs& a, cudaStream_t s) {
  switch (dt) {
    case TOPKP_F32: return launch_dt<TOPKP_F32>(a, s);
    case TOPKP_F16: return launch_dt<TOPKP_F16>(a, s);
    default: return launch_dt<TOPKP_BF16>(a, s);
  }
}

}  // namespace topkp
