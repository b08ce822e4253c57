// topkp_tree_attention: one token, a drafted chain or a drafted tree of each
// request attends to the request's cache.
//
// With G = Hq / Hkv query heads to a head of the cache, the T nodes of a
// request make T * G rows that share one head's keys and values.  Each key
// and value is read once for a tile of rows, with the running maximum and
// sum of the softmax; a request's tokens are split over CTAs when there are
// few rows, and the parts joined by their log-sums.  With up to 128 rows the
// cache's bytes bound the work (64 single tokens, 32 query and 8 cache heads
// of 128, contexts to 8192: 251 us, 6.4 TB/s; 2 x 131000 tokens: 153 us, 5.3,
// in one round of CTAs), with more the products and exponentials.
#include <cuda.h>
#include <math.h>

#include "common.cuh"
#include "decode.h"
#include "internal.h"

namespace topkp {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnDev {
  topkp_tree_attention_args a;
  int splits;
  int per;        // tiles of a part; the last part takes what is left
  float* part_o;  // [splits][B * T * Hq][D]
  float* part_l;  // [splits][B * T * Hq]
  uint32_t page_mul;  // reciprocal of page_size below 2^31, 0: divide
  int page_shift;
  int wide;           // an e4m3 row may be read 16 bytes at a time
  int box;            // tokens of a TMA box, 0: plain copies
};

// Tokens of request b that its nodes may see: the context, and the end of
// the drafted nodes.
__device__ __forceinline__ void request_span(const topkp_tree_attention_args& a, int64_t b, int* ctx, int* len,
                                             int* nodes) {
  const long long cap = a.max_pages * a.page_size;
  const long long c = min((long long)max(a.context[b], 0), cap);
  const int n = a.nodes ? min(max(a.nodes[b], 0), (int)a.T) : (int)a.T;
  *ctx = (int)c;
  *len = (int)min(c + n, cap);
  *nodes = n;
}

constexpr int kTile = 64;  // tokens

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float exponent_scale(uint32_t e) { return __uint_as_float(e ? e << 23 : 0x400000u); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  const int n = in ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

}  // namespace
}  // namespace topkp

#include "attention_tc.cuh"

namespace topkp {
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

// The driver's encoder of tensor maps, looked up once (null where it is missing).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}
// A cache as (element, head, token, page); false where TMA cannot take it.
bool make_map(CUtensorMap* map, const topkp_cache& c, const topkp_tree_attention_args& a, int box, int width,
              CUtensorMapSwizzle swizzle) {
  const bool q8 = c.dtype == TOPKP_E4M3;
  const uint64_t es = q8 ? 1 : 2;
  // a dimension of one entry may have any stride: give it one that is valid
  auto stride = [&](int64_t s, int64_t count) { return count > 1 ? (uint64_t)s * es : ((uint64_t)a.D * es + 15) / 16 * 16; };
  const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.Hkv, (cuuint64_t)a.page_size, (cuuint64_t)a.pages};
  const cuuint64_t strides[3] = {stride(c.head_stride, a.Hkv), stride(c.token_stride, a.page_size), stride(c.page_stride, a.pages)};
  for (const cuuint64_t s : strides)
    if (s % 16 || s >= (1ull << 40)) return false;
  if ((uintptr_t)c.data % 16) return false;
  const cuuint32_t boxes[4] = {(cuuint32_t)width, 1, (cuuint32_t)box, 1}, steps[4] = {1, 1, 1, 1};
  const EncodeTiled encode = encoder();
  return encode && encode(map, q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, c.data, dims, strides,
                          boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, int NT, bool BF, bool Q8, int SH = 1>
cudaError_t launch_tc(AttnDev p, cudaStream_t s) {
  using Shape = TcShape<DP, NT, BF, Q8, SH>;
  const topkp_tree_attention_args& a = p.a;
  cudaError_t e = cudaFuncSetAttribute(attn_tc<DP, NT, BF, Q8, SH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape::kSmem);
  if (e != cudaSuccess) return e;
  // tokens of a box: they lie in one page, and eight rows make a swizzle's group
  CUtensorMap km = {}, vm = {};
  p.box = kTile;
  if (a.table)
    while (p.box > 4 && a.page_size % p.box) p.box /= 2;
  // operands are swizzled (rows of 128 bytes, or of 64 e4m3); raw values are not
  constexpr auto by128 = CU_TENSOR_MAP_SWIZZLE_128B, by64 = CU_TENSOR_MAP_SWIZZLE_64B, plain = CU_TENSOR_MAP_SWIZZLE_NONE;
  if (p.box < 8 || !make_map(&km, a.k, a, p.box, !Q8 ? 64 : DP < 128 ? DP : 128, Q8 && DP == 64 ? by64 : by128) ||
      !make_map(&vm, a.v, a, p.box, Q8 ? DP : 64, Q8 ? plain : by128))
    p.box = 0;
  const int64_t rows = a.T * (a.Hq / a.Hkv);
  const dim3 grid((unsigned)((rows + NT * kTcRows - 1) / (NT * kTcRows)), (unsigned)p.splits, (unsigned)(a.B * a.Hkv));
  attn_tc<DP, NT, BF, Q8, SH><<<grid, Shape::kThreads, Shape::kSmem, s>>>(p, km, vm);
  return cudaGetLastError();
}

// Tiles of 128 rows of a CTA (256 dims leave tensor memory for one).
int row_tiles(const topkp_tree_attention_args& a) { return a.T * (a.Hq / a.Hkv) > kTcRows && a.D <= 128 ? 2 : 1; }

// Whether four warps share each row's tokens: up to 32 rows over e4m3, at 65 to
// 128 dims.  64 single tokens to 8000, in us with and without: 303 / 350 (fp16
// 340 / 365); it gives nothing at 64 dims (217 / 218) or 256 (313 / 311).
bool few_rows(const topkp_tree_attention_args& a) {
  return a.k.dtype == TOPKP_E4M3 && a.D > 64 && a.D <= 128 && a.T * (a.Hq / a.Hkv) <= 32;
}

template <bool BF, bool Q8>
cudaError_t launch_dim(const AttnDev& p, cudaStream_t s) {
  if constexpr (Q8) {
    if (few_rows(p.a)) return launch_tc<128, 1, BF, true, 4>(p, s);
  }
  const bool two = row_tiles(p.a) == 2;
  if (p.a.D <= 64) return two ? launch_tc<64, 2, BF, Q8>(p, s) : launch_tc<64, 1, BF, Q8>(p, s);
  if (p.a.D <= 128) return two ? launch_tc<128, 2, BF, Q8>(p, s) : launch_tc<128, 1, BF, Q8>(p, s);
  return launch_tc<256, 1, BF, Q8>(p, s);
}

}  // namespace

cudaError_t attention_take_device_error(unsigned int* out) {
  const unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_attention_error, sizeof(*out));
  if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_attention_error, &zero, sizeof(zero));
  return e;
}

AttnPlan plan_attention(const topkp_tree_attention_args& a, int num_sms) {
  AttnPlan p;
  const int64_t rows = a.T * (a.Hq / a.Hkv);
  const int64_t cap = a.max_pages * a.page_size;
  const int64_t len = (a.max_context < cap ? (a.max_context > 0 ? a.max_context : 0) : cap) + a.T;
  const int64_t tiles = (len + kTile - 1) / kTile;
  // Parts of equal size, whatever a request's length, so that the CTAs of
  // ragged requests even out.  In units of a tile's time: the rounds of CTAs
  // (between whole ones, as for equal requests, and what ragged ones average
  // to), four tiles for a CTA's start and end, and writing and reading the
  // partial outputs.
  const int64_t nt = row_tiles(a);
  const bool pair = few_rows(a) && a.dtype == TOPKP_BF16;
  const double slots = (nt == 2 || a.D > (a.k.dtype == TOPKP_E4M3 && !pair ? 64 : 128) ? 1.0 : 2.0) * num_sms;
  const double base = (double)(a.B * a.Hkv * ((rows + nt * kTcRows - 1) / (nt * kTcRows)));
  // a tile takes a CTA about 0.9 us (1.3 with two of them on an SM); a part
  // of every row costs 8 bytes an element at the copy's rate
  const double join = (double)(a.B * a.T * a.Hq * a.D) * 8.0 / 6.8e6 / (slots > num_sms ? 1.3 : 0.9);
  double best = -1.0;
  p.splits = 1;
  p.per = (int)tiles;
  for (int64_t n = 1; n <= kMaxParts && n <= tiles; ++n) {
    const int64_t per = (tiles + n - 1) / n;
    if ((tiles + per - 1) / per != n) continue;
    const double part = (double)per + 4.0;
    const double rounds = base * n / slots;
    double cost = rounds <= 1.0 ? part : 0.5 * (ceil(rounds) + rounds + 0.5) * part;
    if (n > 1) cost += 3.0 + join * n;
    if (best < 0 || cost < best) {
      best = cost;
      p.splits = (int)n;
      p.per = (int)per;
    }
  }
  p.part_bytes = p.splits > 1 ? (size_t)p.splits * (size_t)(a.B * a.T * a.Hq) * (a.D + 1) * sizeof(float) : 0;
  return p;
}

cudaError_t launch_attention(const topkp_tree_attention_args& a, const AttnPlan& plan, int* launches, cudaStream_t s) {
  AttnDev p;
  p.a = a;
  p.splits = plan.splits;
  p.per = plan.per;
  const size_t all = (size_t)(a.B * a.T * a.Hq);
  p.part_o = reinterpret_cast<float*>(a.workspace);
  p.part_l = p.part_o + (plan.splits > 1 ? (size_t)plan.splits * all * a.D : 0);
  p.page_mul = 0;
  p.page_shift = 0;
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
  const bool bf = a.dtype == TOPKP_BF16, q8 = a.k.dtype == TOPKP_E4M3;
  cudaError_t e = bf ? (q8 ? launch_dim<true, true>(p, s) : launch_dim<true, false>(p, s))
                     : (q8 ? launch_dim<false, true>(p, s) : launch_dim<false, false>(p, s));
  *launches = 1;
  if (e != cudaSuccess || plan.splits <= 1) return e;
  // the join's launch overlaps the parts; it waits for them itself
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((all + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  *launches = 2;
  return bf ? cudaLaunchKernelEx(&cfg, attn_join<true>, p) : cudaLaunchKernelEx(&cfg, attn_join<false>, p);
}

}  // namespace topkp
