// topkp_tree_attention: one token, a drafted chain or a drafted tree of each
// request attends to the request's cache.
//
// With G = Hq / Hkv query heads to a head of the cache, the T nodes of a
// request make T * G rows that share one head's keys and values.  Each key
// and value is read once for a tile of rows, with the running maximum and
// sum of the softmax; a request's tokens are split over CTAs when there are
// few rows, and the parts joined by their log-sums.  With up to 128 rows the
// cache's bytes bound the work (64 single tokens, 32 query and 8 cache heads
// of 128, contexts to 8192: 251 to 263 us, 6.1 to 6.4 TB/s; 2 x 131000 tokens: 153 us, 5.3,
// in one round of CTAs), with more the products and exponentials.
//
// topkp_shared_attention: what requests share is one launch in which a group
// is a request with the nodes of all its requests, so its keys and values are
// read once a group; each request's own tokens are another, beside it; the
// join takes the parts of both.  64 samples under 8192 tokens (32 query and 8
// cache heads of 128, bf16) 51 us, 258 each by itself; 32 trees of 16 under
// 65500 547 us (1.03 PFLOP/s; bound by the tensor pipe, whose products of 64
// tokens cost what 128 would, and by the rounds of CTAs); 16 x 8 beams under
// 32000 over e4m3 400 us (bound by the chain of one tile's roles).
#include <string.h>

#include <algorithm>

#include "attention_launch.cuh"

namespace topkp {

// attention_shared.cu
cudaError_t launch_grouped(const AttnDev& front, const AttnDev& own, cudaStream_t s);
cudaError_t grouped_take_device_error(unsigned int* out);

namespace {

// Joins the parts of a row: weights exp(lse_i - lse).  One warp per row; a
// lane holds the log-sums of four parts and four elements of the row, and the
// parts' elements are read four parts at a time.  Four parts of 65536 rows
// of 128: 37 us from a cold cache, less where the parts are still in L2.
constexpr int kMaxParts = 128;
template <bool BF>
__global__ void __launch_bounds__(128) attn_join(const __grid_constant__ AttnDev p) {
  const topkp_tree_attention_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t rows = a.B * a.T * a.Hq;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= rows) return;
  float l[kMaxParts / 32], m = -INFINITY, total = 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxParts / 32; ++i) {
    const int s = i * 32 + lane;
    l[i] = s < p.splits ? p.part_l[s * rows + row] : -INFINITY;
    m = fmaxf(m, l[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
  for (int i = 0; i < kMaxParts / 32; ++i) {
    l[i] = l[i] == -INFINITY ? 0.0f : exp2f((l[i] - m) * kLog2e);  // from here on the part's weight
    total += l[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const float inv = total > 0.0f ? 1.0f / total : total;
  const int64_t bt = row / a.Hq;
  const int64_t hq = row - bt * a.Hq, b = bt / a.T, t = bt - b * a.T;
  uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + b * a.out_batch_stride + t * a.out_token_stride + hq * a.out_head_stride;
  for (int d0 = 0; d0 < a.D; d0 += 128) {
    const int d = d0 + lane * 4;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kMaxParts / 32; ++i) {
      const int count = min(32, p.splits - i * 32);
#pragma unroll 4
      for (int k = 0; k < count; ++k) {
        const float w = __shfl_sync(0xffffffffu, l[i], k);
        // a part that saw nothing was not written
        if (w != 0.0f && d < a.D) {
          const float4 x = *reinterpret_cast<const float4*>(p.part_o + ((int64_t)(i * 32 + k) * rows + row) * a.D + d);
          acc.x += w * x.x;
          acc.y += w * x.y;
          acc.z += w * x.z;
          acc.w += w * x.w;
        }
      }
    }
    if (d < a.D)
      *reinterpret_cast<uint2*>(out + d) = make_uint2(pack2<BF>(acc.x * inv, acc.y * inv), pack2<BF>(acc.z * inv, acc.w * inv));
  }
  if (lane == 0 && a.lse) a.lse[row] = total > 0.0f ? m + log2f(total) * kLn2 : total == 0.0f ? -INFINITY : total;
}

}  // namespace

cudaError_t attention_take_device_error(unsigned int* out) {
  const unsigned int zero = 0;
  unsigned int grouped = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_attention_error, sizeof(*out));
  if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_attention_error, &zero, sizeof(zero));
  if (e == cudaSuccess) e = grouped_take_device_error(&grouped);
  *out |= grouped;
  return e;
}

namespace {

// What a tile of a CTA's costs and how many CTAs the device holds.
struct Cost {
  double base;   // CTAs of one part
  double slots;  // resident ones
  double tile;   // us a tile
  int64_t tiles;
};
Cost cost_of(const topkp_tree_attention_args& a, int64_t tokens, bool lone, int num_sms) {
  const int64_t nt = row_tiles(a), rows = a.T * (a.Hq / a.Hkv);
  const bool pair = !lone && few_rows(a) && a.dtype == TOPKP_BF16;
  Cost c;
  c.slots = (nt == 2 || a.D > (a.k.dtype == TOPKP_E4M3 && !pair ? 64 : 128) ? 1.0 : 2.0) * num_sms;
  c.base = (double)(a.B * a.Hkv * ((rows + nt * kTcRows - 1) / (nt * kTcRows)));
  // a tile takes a CTA about 0.9 us (1.3 with two of them on an SM)
  c.tile = c.slots > num_sms ? 1.3 : 0.9;
  c.tiles = (tokens + kTile - 1) / kTile;
  return c;
}
int64_t bounded_context(const topkp_tree_attention_args& a) {
  const int64_t cap = a.max_pages * a.page_size;
  return a.max_context < cap ? (a.max_context > 0 ? a.max_context : 0) : cap;
}
// The shared tokens' launch: a group's requests are one, its nodes theirs.
topkp_tree_attention_args as_groups(const topkp_tree_attention_args& a, int64_t groups) {
  topkp_tree_attention_args g = a;
  const int64_t size = a.B / groups;
  g.B = groups;
  g.T = a.T * size;
  g.q_batch_stride *= size;
  g.ld_table *= size;
  g.tree = nullptr;
  g.lse = nullptr;
  return g;
}

}  // namespace

AttnPlan plan_attention(const topkp_tree_attention_args& a, int num_sms) {
  AttnPlan p;
  const Cost c = cost_of(a, bounded_context(a) + a.T, false, num_sms);
  // Parts of equal size, whatever a request's length, so that the CTAs of
  // ragged requests even out.  In units of a tile's time: the rounds of CTAs
  // (between whole ones, as for equal requests, and what ragged ones average
  // to), four tiles for a CTA's start and end, and writing and reading the
  // partial outputs.
  // A part of every row costs 8 bytes an element at the copy's rate.
  const double join = (double)(a.B * a.T * a.Hq * a.D) * 8.0 / 6.8e6 / c.tile;
  double best = -1.0;
  p.splits = 1;
  p.per = (int)c.tiles;
  for (int64_t n = 1; n <= kMaxParts && n <= c.tiles; ++n) {
    const int64_t per = (c.tiles + n - 1) / n;
    if ((c.tiles + per - 1) / per != n) continue;
    const double part = (double)per + 4.0;
    const double rounds = c.base * n / c.slots;
    double cost = rounds <= 1.0 ? part : 0.5 * (ceil(rounds) + rounds + 0.5) * part;
    if (n > 1) cost += 3.0 + join * n;
    if (best < 0 || cost < best) {
      best = cost;
      p.splits = (int)n;
      p.per = (int)per;
    }
  }
  p.us = best * c.tile;
  p.part_bytes = p.splits > 1 ? (size_t)p.splits * (size_t)(a.B * a.T * a.Hq) * (a.D + 1) * sizeof(float) : 0;
  return p;
}

// Parts of the shared tokens and of the requests' own, which run side by
// side: both kernels' CTAs fill the device together.
namespace {
SharedPlan choose_shared(const topkp_tree_attention_args& a, int64_t groups, int64_t max_shared, int num_sms) {
  SharedPlan s;
  const AttnPlan alone = plan_attention(a, num_sms);
  s.groups = 0;  // every request by itself
  s.own = alone;
  s.part_bytes = alone.part_bytes;
  const int64_t context = bounded_context(a), front = std::min(max_shared, context) / kTile * kTile;
  if (groups >= a.B || front <= 0) return s;
  const Cost x = cost_of(as_groups(a, groups), front, true, num_sms), y = cost_of(a, context - front + a.T + kTile - 1, false, num_sms);
  // As fitted to 15 x 4 choices of parts of seven cases (8 to 512 rows a
  // group's head, 4000 to 65500 shared tokens, both kinds of cache; the choice
  // made is at worst 10% slower than the best, in six cases at most 6%): a
  // tile takes a CTA of 256 rows 1.1 us, another one that has its SM for
  // itself 1.0, one of two 1.1; a CTA's start and end are four tiles, a part of
  // every row 16 bytes an element at the copy's rate, the launches 8 us.
  const double cx = row_tiles(as_groups(a, groups)) == 2 ? 1.1 : x.slots > num_sms ? 1.1 : 1.0;
  const double cy = row_tiles(a) == 2 ? 1.1 : y.slots > num_sms ? 1.1 : 1.0;
  const double join = (double)(a.B * a.T * a.Hq * a.D) * 16.0 / 6.8e6;
  static const int counts[] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 20, 24, 32, 40, 48, 64, 80, 96};
  double best = -1.0;
  for (const int i : counts) {
    const int64_t px = (x.tiles + i - 1) / i, nx = (x.tiles + px - 1) / px;
    if (i > x.tiles) break;
    for (const int j : counts) {
      const int64_t py = (y.tiles + j - 1) / j, ny = (y.tiles + py - 1) / py;
      if (j > y.tiles || nx + ny > kMaxParts) break;
      const double tx = ((double)px + 4.0) * cx, ty = ((double)py + 4.0) * cy;
      const double fx = x.base * nx / x.slots, fy = y.base * ny / y.slots;
      // rounds of the shared parts (of one group they are alike, of several
      // ragged), beside which the others find their place, or all the work
      const double rounds = fx <= 1.0 ? 1.0 : groups == 1 ? ceil(fx) : 0.5 * (ceil(fx) + fx + 0.5);
      double us = std::max(rounds * tx, ty);
      if (fx + fy > 1.0) us = std::max(us, fx * tx + (fy + 0.25) * ty);
      us += 8.0 + join * (nx + ny);
      if (best < 0 || us < best) {
        best = us;
        s.front.splits = (int)nx;
        s.front.per = (int)px;
        s.own.splits = (int)ny;
        s.own.per = (int)py;
      }
    }
  }
  if (alone.us <= best) {  // little is shared: not worth another launch
    s.own = alone;
    return s;
  }
  s.groups = groups;
  s.part_bytes = (size_t)(s.front.splits + s.own.splits) * (size_t)(a.B * a.T * a.Hq) * (a.D + 1) * sizeof(float);
  return s;
}
}  // namespace

// (The choice takes longer than a launch, and a program asks for it twice a
// call and for the same shapes call after call: the last one is kept.)
SharedPlan plan_shared(const topkp_tree_attention_args& a, int64_t groups, int64_t max_shared, int num_sms) {
  struct Shapes {
    int64_t v[14];
  };
  const Shapes shapes = {{a.B, a.T, a.Hq, a.Hkv, a.D, a.page_size, a.max_pages, a.max_context, a.dtype, a.k.dtype, groups, max_shared, num_sms, 1}};
  static thread_local Shapes last = {};
  static thread_local SharedPlan plan;
  if (memcmp(&last, &shapes, sizeof(shapes))) {
    plan = choose_shared(a, groups, max_shared, num_sms);
    last = shapes;
  }
  return plan;
}

namespace {

AttnDev device_args(const topkp_tree_attention_args& a) {
  AttnDev p = {};
  p.a = a;
  if (a.page_size > 1) {  // t / page_size = (t * mul) >> (32 + shift), exact below 2^31
    int l = 1;
    while ((1LL << l) < a.page_size) ++l;
    p.page_mul = (uint32_t)(((1ull << (31 + l)) + a.page_size - 1) / a.page_size);
    p.page_shift = l - 1;
  }
  auto by16 = [](const topkp_cache& c) {
    return ((uintptr_t)c.data | (uintptr_t)c.page_stride | (uintptr_t)c.token_stride | (uintptr_t)c.head_stride) % 16 == 0;
  };
  p.wide = a.D % 16 == 0 && by16(a.k) && by16(a.v);
  return p;
}
// Room for the partial outputs of all parts: their rows, then their log-sums.
void give_parts(AttnDev& p, int parts) {
  const size_t all = (size_t)(p.a.B * p.a.T * p.a.Hq);
  p.part_o = reinterpret_cast<float*>(p.a.workspace);
  p.part_l = p.part_o + (parts > 1 ? (size_t)parts * all * p.a.D : 0);
}
// The join's launch overlaps the parts; it waits for them itself.
cudaError_t launch_join(const AttnDev& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.a.B * p.a.T * p.a.Hq + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return p.a.dtype == TOPKP_BF16 ? cudaLaunchKernelEx(&cfg, attn_join<true>, p) : cudaLaunchKernelEx(&cfg, attn_join<false>, p);
}

}  // namespace

cudaError_t launch_attention(const topkp_tree_attention_args& a, const AttnPlan& plan, int* launches, cudaStream_t s) {
  AttnDev p = device_args(a);
  p.splits = plan.splits;
  p.per = plan.per;
  give_parts(p, plan.splits);
  Maps maps;
  const cudaError_t e = launch_parts<false>(p, maps, s);
  *launches = 1;
  if (e != cudaSuccess || plan.splits <= 1) return e;
  *launches = 2;
  return launch_join(p, s);
}

cudaError_t launch_shared(const topkp_tree_attention_args& a, const int32_t* shared, const SharedPlan& plan, int* launches, cudaStream_t s) {
  if (!plan.groups) return launch_attention(a, plan.own, launches, s);
  const int parts = plan.front.splits + plan.own.splits;
  const size_t all = (size_t)(a.B * a.T * a.Hq);
  AttnDev own = device_args(a);
  give_parts(own, parts);
  own.size = (int)(a.B / plan.groups);
  own.shared = shared;
  AttnDev front = own;
  front.a = as_groups(a, plan.groups);
  front.stage = 1;
  front.inner = (int)a.T;
  front.q_member = a.q_batch_stride;
  front.ld_member = a.ld_table;
  front.splits = plan.front.splits;
  front.per = plan.front.per;
  AttnDev join = own;
  join.splits = parts;
  own.stage = 2;
  own.splits = plan.own.splits;
  own.per = plan.own.per;
  own.part_o += (size_t)front.splits * all * a.D;
  own.part_l += (size_t)front.splits * all;
  const cudaError_t e = launch_grouped(front, own, s);
  *launches = 3;
  return e != cudaSuccess ? e : launch_join(join, s);
}

}  // namespace topkp
