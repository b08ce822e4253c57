// topkp_draft_verify: drafted tokens against the target's probabilities.
//
// A request is walked down from its root by one cluster of CTAs.  At node n
// the children are tried in turn.  With p and q the target's and the draft's
// distributions after n, what is left of p after k rejected children is
//   p_k = norm(max(p_{k-1} - q, 0)) = max(p - a_k q, 0) / W_k,
//   a_{k+1} = a_k + W_k,   W_k = sum max(p - a_k q, 0),   a_0 = 0, W_0 = 1,
// so a child costs two probabilities, and a further child one pass over the
// node's two rows.  The token drawn when no child is accepted is the largest
// of max(p - a q, 0) / (race + eps): no normaliser, no prefix sums.
//
// Only the rows of the accepted path are read (a tree of 64 nodes has about
// four).  Rows are cut over the cluster's CTAs; a row's second reading comes
// from L2.  Each warp hands its maximum and sum to every CTA of the cluster
// through distributed shared memory, so that a pass ends in one barrier and
// every CTA takes the same decision by itself.
//
// Sums are fp32 in a thread (at most a few tens of terms of a batch, then a
// few tens of batches), 64 bits from the warps' sums on.
#include <limits.h>

#include "common.cuh"
#include "decode.h"

namespace topkp {
namespace {

constexpr int kVW = kVerifyThreads / 32;
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

// Vectors of 16 bytes; the first and last of a row may stick out of it.
template <int DT>
struct Row {
  using raw = typename DType<DT>::raw;
  static constexpr int VEC = 16 / (int)sizeof(raw);
  const raw* x;
  int V, off, vectors;  // elements that the first vector begins before the row
  __device__ __forceinline__ Row(const raw* p, int n)
      : x(p), V(n), off((int)(((uintptr_t)p & 15) / sizeof(raw))), vectors((int)(((long long)off + n + VEC - 1) / VEC)) {}
  __device__ __forceinline__ uint4 load(int v) const {
    const int e = v * VEC - off;
    if (e >= 0 && e <= V - VEC) return __ldg(reinterpret_cast<const uint4*>(x + e));
    return edge(e);
  }
  __device__ __noinline__ uint4 edge(int e) const {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const uint32_t r = e + j >= 0 && e + j < V ? (uint32_t)x[e + j] : (uint32_t)DType<DT>::kNegInf;
      if (sizeof(raw) == 4) w[j % 4] = r;
      else w[(j >> 1) % 4] |= r << (16 * (j & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
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

// U vectors into a thread's share.
template <int DT, int U>
__device__ __forceinline__ void absorb(const uint4 (&q)[U], Sum& s) {
  constexpr int PAIRS = Row<DT>::VEC / 2;
  float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      float a, b;
      pair_of<DT>(q[u], j, a, b);
      top[j & 1] = fmaxf(top[j & 1], fmaxf(a, b));
    }
  const float mx = fmaxf(top[0], top[1]);
  if (mx > s.m) {
    s.s *= s.m == -INFINITY ? 0.0f : exp_fast(s.m - mx);
    s.m = mx;
  }
  if (s.m == -INFINITY) return;
  const uint64_t less = two(-s.m, -s.m), hi = two(kLog2eHi, kLog2eHi), lo = two(kLog2eLo, kLog2eLo);
  uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      float a, b;
      pair_of<DT>(q[u], j, a, b);
      const uint64_t t = add_two(two(a, b), less);
      apart(fma_two(t, hi, mul_two(t, lo)), a, b);
      sum[j & 1] = add_two(sum[j & 1], two(ex2(a), ex2(b)));
    }
  float a, b;
  apart(add_two(sum[0], sum[1]), a, b);
  s.s += a + b;
}

// What a warp hands to every CTA of its cluster, and what a step leaves there.
struct Shared {
  float4 part[2][16 * kVW];
  int32_t parent[TOPKP_MAX_TREE], tokens[TOPKP_MAX_TREE], path[TOPKP_MAX_TREE], tried[TOPKP_MAX_TREE];
  float uniform[TOPKP_MAX_TREE], logprob[TOPKP_MAX_TREE];
  float xt[TOPKP_MAX_TREE], xd[TOPKP_MAX_TREE];  // the children's logits
  double px[TOPKP_MAX_TREE], qx[TOPKP_MAX_TREE];
  float mt, md, factor;
  double st, sd, weight, less;
  unsigned long long bloom, best;
  int chosen, next, tries, again;
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
// This warp's part to all CTAs (lane 0's value).
__device__ __forceinline__ void hand_out(const Team& t, Shared& sh, const float4& v) {
  const int lane = threadIdx.x & 31;
  if (lane < t.cs) {
    float4* to = &sh.part[t.at][t.rank * kVW + (threadIdx.x >> 5)];
    if (t.cs == 1) {
      *to = v;
    } else {
      const uint32_t a = dsmem_addr(to, (uint32_t)lane);
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
    }
  }
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
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
// Maximum and sum over the warps' parts, by one warp.
__device__ __forceinline__ void join_sums(const Team& t, const Shared& sh, bool second, float& m, double& s) {
  const int lane = threadIdx.x & 31, n = t.cs * kVW;
  m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, second ? sh.part[t.at][i].z : sh.part[t.at][i].x);
  m = warp_max(m);
  s = 0.0;
  for (int i = lane; i < n; i += 32) {
    const float4 v = sh.part[t.at][i];
    const float pm = second ? v.z : v.x, ps = second ? v.w : v.y;
    if (pm > -INFINITY) s += (double)(ps * exp_one(pm, m));
  }
  s = warp_sum(s);
}
__device__ __forceinline__ Sum warp_join(const Sum& s) {
  Sum r;
  r.m = warp_max(s.m);
  r.s = warp_sum(s.m == -INFINITY ? 0.0f : s.s * exp_fast(s.m - r.m));
  return r;
}

// A candidate of the draw: the larger key, the lower index.
__device__ __forceinline__ unsigned long long candidate(float key, int i) {
  return (unsigned long long)__float_as_uint(key) << 32 | (uint32_t)~i;
}

// A CTA's elements of a node's rows, once more: f(i, target's logit, draft's,
// the race's variate) for each, -inf and 0 for what is not read.
template <int DT, bool DRAFT, bool RACE, typename F>
__device__ __forceinline__ void each_element(const VerifyArgs& a, const Team& team, const typename DType<DT>::raw* t,
                                             const typename DType<DT>::raw* d, bool draft, const float* race, F f) {
  constexpr int VEC = Row<DT>::VEC, U = 2;
  const int per = ((a.V + a.cs - 1) / a.cs + VEC - 1) / VEC * VEC;
  const int first = min(per * (int)team.rank, a.V), last = min(first + per, a.V);
  if (a.whole) {  // all rows 16 bytes at a time
    for (int i0 = first + (int)threadIdx.x * VEC; i0 < last; i0 += U * kVerifyThreads * VEC) {
      uint4 qt[U], qd[U];
      float4 e[U][VEC / 4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kVerifyThreads * VEC;
        const bool in = i < last;
        qt[u] = in ? __ldg(reinterpret_cast<const uint4*>(t + i)) : nothing<DT>();
        qd[u] = DRAFT && draft && in ? __ldg(reinterpret_cast<const uint4*>(d + i)) : nothing<DT>();
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k)
          e[u][k] = RACE && in ? __ldg(reinterpret_cast<const float4*>(race + i) + k) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          const int i = i0 + u * kVerifyThreads * VEC + 2 * j;
          float x, y, c = -INFINITY, g = -INFINITY;
          pair_of<DT>(qt[u], j, x, y);
          if (DRAFT) pair_of<DT>(qd[u], j, c, g);
          f(i, x, c, j & 1 ? e[u][j / 2].z : e[u][j / 2].x);
          f(i + 1, y, g, j & 1 ? e[u][j / 2].w : e[u][j / 2].y);
        }
    }
  } else {
    for (int i = first + (int)threadIdx.x; i < last; i += kVerifyThreads)
      f(i, DType<DT>::to_float(t[i]), DRAFT && draft ? DType<DT>::to_float(d[i]) : -INFINITY, RACE ? race[i] : 0.0f);
  }
}

template <int DT, int MODE>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const __grid_constant__ VerifyArgs a) {
  using raw = typename DType<DT>::raw;
  constexpr bool DRAFT = MODE == kVerifyRatio, GREEDY = MODE == kVerifyGreedy;
  constexpr int VEC = Row<DT>::VEC;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Team team = {a.cs, a.cs > 1 ? cluster_ctarank() : 0u, 0};
  const int64_t b = blockIdx.x / a.cs;
  const int n = a.nodes ? min(max(a.nodes[b], 0), a.T) : a.T;
  if (tid < a.T) {
    const int64_t i = b * a.T + tid;
    sh.parent[tid] = a.parent ? a.parent[i] : tid - 1;
    sh.tokens[tid] = a.tokens[i];
    sh.uniform[tid] = a.uniform ? a.uniform[i] : 0.0f;
    sh.path[tid] = -1;
    sh.logprob[tid] = 0.0f;
  }
  // every CTA of the cluster has started before one writes into another's memory
  team_sync(team);
  int node = 0, depth = 0, token = -1;
  const raw* target = reinterpret_cast<const raw*>(a.target) + b * a.t_batch;
  const raw* draft = reinterpret_cast<const raw*>(a.draft) + (DRAFT ? b * a.d_batch : 0);
  if (n > 0) {
    if (tid == 0) sh.path[0] = 0;
    for (;;) {
      // the children, and their logits
      unsigned long long kids = 0;
      {
        const bool lo = lane > node && lane < n && sh.parent[lane] == node;
        const bool hi = lane + 32 > node && lane + 32 < n && sh.parent[lane + 32] == node;
        kids = __ballot_sync(0xffffffffu, lo) | (unsigned long long)__ballot_sync(0xffffffffu, hi) << 32;
      }
      const raw* t = target + node * a.t_node;
      const raw* d = draft + (DRAFT ? node * a.d_node : 0);
      const bool drafted = DRAFT && kids != 0;
      if (!GREEDY && warp < 2) {
        const int c = warp * 32 + lane;
        if (kids >> c & 1) {
          const int x = sh.tokens[c];
          const bool in = x >= 0 && x < a.V;
          sh.xt[c] = in ? DType<DT>::to_float(t[x]) : -INFINITY;
          sh.xd[c] = DRAFT && in ? DType<DT>::to_float(d[x]) : -INFINITY;
        }
      }
      // largest elements and sums of both rows
      Sum st = {-INFINITY, 0.0f}, sd = {-INFINITY, 0.0f};
      uint32_t first = 0xffffffffu;  // of the largest element
      const Row<DT> rt(t, a.V), rd(DRAFT ? d : t, a.V);
      {
        constexpr int U = 4;
        const int per = (max(rt.vectors, rd.vectors) + a.cs - 1) / a.cs;
        const int begin = per * (int)team.rank, te = min(begin + per, rt.vectors), de = min(begin + per, rd.vectors);
        for (int v = begin + tid; v < begin + per; v += U * kVerifyThreads) {
          uint4 q[U], r[U];
#pragma unroll
          for (int u = 0; u < U; ++u) q[u] = v + u * kVerifyThreads < te ? rt.load(v + u * kVerifyThreads) : nothing<DT>();
          if (DRAFT && drafted) {
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = v + u * kVerifyThreads < de ? rd.load(v + u * kVerifyThreads) : nothing<DT>();
          }
          const float before = st.m;
          absorb<DT, U>(q, st);
          if (GREEDY && st.m > before) {  // its first place
#pragma unroll
            for (int u = U - 1; u >= 0; --u)
#pragma unroll
              for (int j = VEC / 2 - 1; j >= 0; --j) {
                float x, y;
                pair_of<DT>(q[u], j, x, y);
                const uint32_t e = (uint32_t)((v + u * kVerifyThreads) * VEC - rt.off + 2 * j);
                if (y == st.m) first = e + 1;
                if (x == st.m) first = e;
              }
          }
          if (DRAFT && drafted) absorb<DT, U>(r, sd);
        }
      }
      {
        const Sum w = warp_join(st);
        float4 part = make_float4(w.m, w.s, -INFINITY, 0.0f);
        if (DRAFT) {
          const Sum x = warp_join(sd);
          part.z = x.m;
          part.w = x.s;
        }
        if (GREEDY) part.z = __uint_as_float(__reduce_min_sync(0xffffffffu, st.m == w.m ? first : 0xffffffffu));
        hand_out(team, sh, part);
      }
      team_sync(team);
      if (warp == 0) {
        float mt, md = -INFINITY;
        double zt, zd = 0.0;
        join_sums(team, sh, false, mt, zt);
        if (DRAFT) join_sums(team, sh, true, md, zd);
        int top = 0;
        if (GREEDY) {
          uint32_t f = 0xffffffffu;
          for (int i = lane; i < a.cs * kVW; i += 32) {
            const float4 v = sh.part[team.at][i];
            if (v.x == mt) f = min(f, __float_as_uint(v.z));
          }
          top = (int)__reduce_min_sync(0xffffffffu, f);
          if (mt == -INFINITY || top < 0 || top >= a.V) top = -1;
        } else {
          for (int c = lane; c < TOPKP_MAX_TREE; c += 32)
            if (kids >> c & 1) {
              sh.px[c] = sh.xt[c] > -INFINITY ? exp((double)sh.xt[c] - mt) / zt : 0.0;
              if (DRAFT) sh.qx[c] = sh.xd[c] > -INFINITY ? exp((double)sh.xd[c] - md) / zd : 0.0;
            }
        }
        if (lane == 0) {
          sh.mt = mt;
          sh.md = md;
          sh.st = zt;
          sh.sd = zd;
          sh.less = 0.0;
          sh.weight = 1.0;
          sh.tries = 0;
          sh.bloom = 0ull;
          sh.best = (unsigned long long)(long long)top;
        }
      }
      team.at ^= 1;
      // the children in turn, by one thread; a pass of all where the weight of what is left is wanted
      unsigned long long open = kids;
      int chosen = -1;
      for (;;) {
        if (tid == 0) {
          chosen = -1;
          bool pass = false;
          while (open && chosen < 0 && !pass) {
            const int c = __ffsll((long long)open) - 1;
            open &= open - 1;
            const int x = sh.tokens[c];
            if (x < 0 || x >= a.V) continue;
            if (GREEDY) {
              if (x == (int)(long long)sh.best) chosen = c;
              continue;
            }
            double left = sh.px[c], q = 1.0;
            if (DRAFT) {
              q = sh.qx[c];
              left -= sh.less * q;
            } else if (sh.bloom >> ((x >> 3) & 63) & 1) {
              for (int i = 0; i < sh.tries; ++i)
                if (sh.tried[i] == x) left = 0.0;
            }
            if ((double)sh.uniform[c] * q * sh.weight < left) {
              chosen = c;
            } else if (DRAFT) {
              sh.less += sh.weight;
              pass = open != 0;
            } else if (left > 0.0) {
              sh.weight = fmax(sh.weight - left, 0.0);
              sh.tried[sh.tries++] = x;
              sh.bloom |= 1ull << ((x >> 3) & 63);
            }
          }
          if (chosen >= 0 && a.logprob) sh.logprob[depth] = (float)((double)(GREEDY ? sh.mt : sh.xt[chosen]) - sh.mt - log(sh.st));
          sh.chosen = chosen;
          sh.again = pass;
          if (DRAFT) sh.factor = sh.sd > 0.0 ? (float)(sh.less * sh.st / sh.sd) : 0.0f;
        }
        __syncthreads();
        chosen = sh.chosen;
        if (!DRAFT || !sh.again) break;
        // the weight of max(p - less q, 0)
        float sum = 0.0f;
        const float mt = sh.mt, md = sh.md, factor = sh.factor;
        each_element<DT, DRAFT, false>(a, team, t, d, true, nullptr, [&](int, float x, float y, float) {
          const float e = x > -INFINITY ? exp_fast(x - mt) : 0.0f, g = y > -INFINITY ? exp_fast(y - md) : 0.0f;
          sum += fmaxf(fmaf(-factor, g, e), 0.0f);
        });
        sum = warp_sum(sum);
        hand_out(team, sh, make_float4(sum, 0.0f, 0.0f, 0.0f));
        team_sync(team);
        if (warp == 0) {
          double w = 0.0;
          for (int i = lane; i < a.cs * kVW; i += 32) w += (double)sh.part[team.at][i].x;
          w = warp_sum(w);
          if (lane == 0) sh.weight = w / sh.st;
        }
        team.at ^= 1;
        __syncthreads();
      }
      if (chosen >= 0) {
        node = chosen;
        ++depth;
        if (tid == 0) sh.path[depth] = node;
        __syncthreads();
        continue;
      }
      // the draw, from what is left; from the whole where nothing is
      if (GREEDY) {
        token = (int)(long long)sh.best;
      } else {
        const float* race = a.race + b * a.ld_race;
        const float mt = sh.mt, md = sh.md, eps = a.eps;
        float factor = DRAFT ? sh.factor : 0.0f;
        unsigned long long bloom = sh.bloom;
        const int tries = sh.tries;
        for (int round = 0;; ++round) {
          unsigned long long best = 0ull;
          const bool less = DRAFT && factor > 0.0f;
          each_element<DT, DRAFT, true>(a, team, t, d, less, race, [&](int i, float x, float y, float variate) {
            float e = x > -INFINITY ? exp_one(x, mt) : 0.0f;
            if (less && y > -INFINITY) e = fmaxf(fmaf(-factor, exp_one(y, md), e), 0.0f);
            if (!DRAFT && (bloom >> ((i >> 3) & 63) & 1))
              for (int k = 0; k < tries; ++k)
                if (sh.tried[k] == i) e = 0.0f;
            if (e > 0.0f) {
              const unsigned long long c = candidate(__fdiv_rn(e, variate + eps), i);
              best = c > best ? c : best;
            }
          });
          best = warp_max(best);
          hand_out(team, sh, make_float4(__uint_as_float((uint32_t)best), __uint_as_float((uint32_t)(best >> 32)), 0.0f, 0.0f));
          team_sync(team);
          if (warp == 0) {
            best = 0ull;
            for (int i = lane; i < a.cs * kVW; i += 32) {
              const float4 v = sh.part[team.at][i];
              const unsigned long long c = (unsigned long long)__float_as_uint(v.y) << 32 | __float_as_uint(v.x);
              best = c > best ? c : best;
            }
            best = warp_max(best);
            if (lane == 0) sh.best = best;
          }
          team.at ^= 1;
          __syncthreads();
          if (sh.best || round || (factor == 0.0f && bloom == 0ull)) break;
          factor = 0.0f;
          bloom = 0ull;
          __syncthreads();
        }
        token = sh.best ? (int)~(uint32_t)sh.best : -1;
      }
      if (tid == 0 && a.logprob && token >= 0)
        sh.logprob[depth] = (float)((double)DType<DT>::to_float(t[token]) - sh.mt - log(sh.st));
      break;
    }
    __syncthreads();
  }
  if (team.rank == 0) {
    if (tid < a.T) {
      a.path[b * a.T + tid] = sh.path[tid];
      if (a.logprob) a.logprob[b * a.T + tid] = sh.logprob[tid];
    }
    if (tid == 0) {
      a.count[b] = n > 0 ? depth + 1 : 0;
      a.token[b] = token;
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

// CTAs of a request: as many as two an SM allow, but none with fewer than
// 256 vectors of a row.
int verify_cluster(int64_t B, int64_t V, int esize, int num_sms) {
  const int64_t vectors = (V * esize + 15) / 16;
  int cs = 1;
  while (cs < 16 && B * cs * 2 <= 2LL * num_sms && vectors >= 256LL * cs * 2) cs *= 2;
  return cs;
}

cudaError_t launch_verify(topkp_dtype dt, const VerifyArgs& a, cudaStream_t s) {
  switch (dt) {
    case TOPKP_F32: return launch_dt<TOPKP_F32>(a, s);
    case TOPKP_F16: return launch_dt<TOPKP_F16>(a, s);
    default: return launch_dt<TOPKP_BF16>(a, s);
  }
}

}  // namespace topkp
