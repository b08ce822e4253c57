// topkp_tree_attention: one token, a drafted chain or a drafted tree of each
// request attends to the request's cache.
//
// With G = Hq / Hkv query heads to a head of the cache, the T nodes of a
// request make T * G rows that share one head's keys and values.  Each key
// and value is read once for a tile of rows, with the running maximum and
// sum of the softmax; a request's tokens are split over CTAs when there are
// few rows, and the parts joined by their log-sums.
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

// ------------------------------------------------------------- mma.sync
// One CTA: 16 rows, four warps; each warp takes 16 of the 64 tokens of a
// tile with a softmax of its own, and the four are joined at the end.
constexpr int kTile = 64;
constexpr int kRowTile = 16;
constexpr int kMmaThreads = 128;

template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Eight e4m3 of a cache, scaled, in the rows' type (exact in bf16).
template <bool BF>
__device__ __forceinline__ uint4 widen8(uint2 w, float scale) {
  const uint32_t two[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two[i]));
    r[i] = pack2<BF>(__half2float(__ushort_as_half((uint16_t)h)) * scale,
                     __half2float(__ushort_as_half((uint16_t)(h >> 16))) * scale);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ float exponent_scale(uint32_t e) { return __uint_as_float(e ? e << 23 : 0x400000u); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  const int n = in ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

template <int DP>
constexpr size_t mma_smem() {
  return (size_t)2 * 2 * kTile * (DP + 8) * 2;
}

template <int DP, bool BF, bool Q8>
__global__ void __launch_bounds__(kMmaThreads) attn_mma(const __grid_constant__ AttnDev p) {
  constexpr int LD = DP + 8;  // a padded row: eight consecutive rows fall into different banks
  constexpr int KS = DP / 16;
  extern __shared__ __align__(16) unsigned char smem[];
  uint16_t* sk = reinterpret_cast<uint16_t*>(smem);  // [2][kTile][LD]
  uint16_t* sv = sk + 2 * kTile * LD;
  const topkp_tree_attention_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = (int)(a.Hq / a.Hkv);
  const int rows = (int)a.T * G;
  const int64_t bh = blockIdx.y;
  const int64_t b = bh / a.Hkv;
  const int h = (int)(bh - b * a.Hkv);
  const int row0 = blockIdx.z * kRowTile;
  const int split = blockIdx.x;
  int ctx, len, nodes;
  request_span(a, b, &ctx, &len, &nodes);
  const int tiles = (len + kTile - 1) / kTile;
  const int t_begin = min(split * p.per, tiles);
  const int t_end = split == p.splits - 1 ? tiles : min(t_begin + p.per, tiles);

  // the two rows of this thread (lane / 4 and that plus 8)
  int node[2];
  uint64_t bits[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row0 + (lane >> 2) + 8 * i;
    node[i] = r / G;
    bits[i] = 0;
    if (node[i] >= nodes) node[i] = -1;
    else if (a.tree) bits[i] = a.tree[b * a.T + node[i]];
  }
  // Q in registers, as the left operand's 16 x 16 pieces
  uint32_t qf[KS][4];
  {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q) + b * a.q_batch_stride;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = row0 + (lane >> 2) + 8 * i;
      const bool in = r < rows;
      const uint16_t* qr = q + (in ? (r / G) * a.q_token_stride + (h * G + r % G) * a.q_head_stride : 0);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int d = k * 16 + j * 8 + (lane & 3) * 2;
          qf[k][i + 2 * j] = in && d < a.D ? *reinterpret_cast<const uint32_t*>(qr + d) : 0u;
        }
    }
  }

  float o[DP / 8][4];
#pragma unroll
  for (int i = 0; i < DP / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  const float sc = a.scale * kLog2e;
  const int32_t* table = a.table ? a.table + b * a.ld_table : nullptr;

  auto load = [&](int tile, int buf) {
    constexpr int CH = DP / 8;  // 8-element pieces of a row
#pragma unroll 4
    for (int i = tid; i < kTile * CH; i += kMmaThreads) {
      const int r = i / CH, c = i - r * CH;
      const int t = tile * kTile + r;
      bool in = t < len && c * 8 < a.D;
      int64_t page = b, at = t;
      if (table && in) {
        const int pg = t / (int)a.page_size;
        at = t - pg * (int)a.page_size;
        page = table[pg];
        in = page >= 0 && page < a.pages;
      }
      if (!in) page = at = 0;
      const int cc = in ? c * 8 : 0;
      const int64_t ko = page * a.k.page_stride + at * a.k.token_stride + h * a.k.head_stride + cc;
      const int64_t vo = page * a.v.page_stride + at * a.v.token_stride + h * a.v.head_stride + cc;
      uint16_t* dk = sk + (buf * kTile + r) * LD + c * 8;
      uint16_t* dv = sv + (buf * kTile + r) * LD + c * 8;
      if (Q8) {
        uint4 kk = make_uint4(0, 0, 0, 0), vv = kk;
        if (in) {
          const float ks = exponent_scale(
              a.k.exponents[page * a.k.exp_page_stride + at * a.k.exp_token_stride + h * a.k.exp_head_stride]);
          const float vs = exponent_scale(
              a.v.exponents[page * a.v.exp_page_stride + at * a.v.exp_token_stride + h * a.v.exp_head_stride]);
          kk = widen8<BF>(*reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(a.k.data) + ko), ks);
          vv = widen8<BF>(*reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(a.v.data) + vo), vs);
        }
        *reinterpret_cast<uint4*>(dk) = kk;
        *reinterpret_cast<uint4*>(dv) = vv;
      } else {
        cp16(smem_u32(dk), reinterpret_cast<const uint16_t*>(a.k.data) + ko, in);
        cp16(smem_u32(dv), reinterpret_cast<const uint16_t*>(a.v.data) + vo, in);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  if (t_begin < t_end) load(t_begin, 0);
  for (int tile = t_begin; tile < t_end; ++tile) {
    const int buf = (tile - t_begin) & 1;
    if (tile + 1 < t_end) {
      load(tile + 1, buf ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const uint16_t* kt = sk + (buf * kTile + warp * 16) * LD;
    const uint16_t* vt = sv + (buf * kTile + warp * 16) * LD;
    float s[2][4] = {};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t f[4];
      // matrices: tokens 0-7 and 8-15, each of 16 elements in two halves
      ldsm4(f, smem_u32(kt + ((lane & 7) + (lane >> 4) * 8) * LD + k * 16 + ((lane >> 3) & 1) * 8));
      mma16816<BF>(s[0], qf[k], f[0], f[1]);
      mma16816<BF>(s[1], qf[k], f[2], f[3]);
    }
    const int t0 = tile * kTile + warp * 16;
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t0 + n * 8 + (lane & 3) * 2 + (e & 1);
        const int i = e >> 1;
        bool see = node[i] >= 0 && t < len;
        if (t >= ctx) see = see && (a.tree ? (bits[i] >> (t - ctx)) & 1 : t - ctx <= node[i]);
        s[n][e] = see ? s[n][e] * sc : -INFINITY;
        mx[i] = fmaxf(mx[i], s[n][e]);
      }
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
      const float base = mx[i] == -INFINITY ? 0.0f : mx[i];
      f[i] = exp2f(m[i] - base);
      m[i] = mx[i];
      l[i] *= f[i];
      mx[i] = base;
    }
    uint32_t pf[4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      float e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e[j] = exp2f(s[n][j] - mx[j >> 1]);
        l[j >> 1] += e[j];
      }
      pf[2 * n] = pack2<BF>(e[0], e[1]);
      pf[2 * n + 1] = pack2<BF>(e[2], e[3]);
    }
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[2 * d][j] *= f[j >> 1];
        o[2 * d + 1][j] *= f[j >> 1];
      }
      uint32_t v[4];
      ldsm4t(v, smem_u32(vt + ((lane & 7) + ((lane >> 3) & 1) * 8) * LD + d * 16 + (lane >> 4) * 8));
      mma16816<BF>(o[2 * d], pf, v[0], v[1]);
      mma16816<BF>(o[2 * d + 1], pf, v[2], v[3]);
    }
    __syncthreads();
  }

  // join the four warps: row statistics, then the weighted outputs through
  // shared memory (the tiles are done with)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
  }
  float* so = reinterpret_cast<float*>(smem);  // [4 warps][16][DP + 4]
  __shared__ float sm[4][16], sl[4][16];
  if ((lane & 3) == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sm[warp][(lane >> 2) + 8 * i] = m[i];
      sl[warp][(lane >> 2) + 8 * i] = l[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (lane >> 2) + 8 * i;
    const float all = fmaxf(fmaxf(sm[0][r], sm[1][r]), fmaxf(sm[2][r], sm[3][r]));
    const float f = m[i] == -INFINITY ? 0.0f : exp2f(m[i] - all);
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) {
      float* at = so + (warp * 16 + r) * (DP + 4) + d * 8 + (lane & 3) * 2;
      at[0] = o[d][2 * i] * f;
      at[1] = o[d][2 * i + 1] * f;
    }
  }
  __syncthreads();
  const int64_t all_rows = a.B * a.T * a.Hq;
  for (int i = tid; i < kRowTile * (DP / 2); i += kMmaThreads) {
    const int rr = i / (DP / 2), d = (i - rr * (DP / 2)) * 2;
    const int r = row0 + rr;
    if (r >= rows || d >= a.D) continue;
    const float all = fmaxf(fmaxf(sm[0][rr], sm[1][rr]), fmaxf(sm[2][rr], sm[3][rr]));
    float total = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (sm[w][rr] == -INFINITY) continue;
      total += sl[w][rr] * exp2f(sm[w][rr] - all);
      x += so[(w * 16 + rr) * (DP + 4) + d];
      y += so[(w * 16 + rr) * (DP + 4) + d + 1];
    }
    const float inv = total > 0.0f ? 1.0f / total : total;
    const float lse = total > 0.0f ? (all + log2f(total)) * kLn2 : total == 0.0f ? -INFINITY : total;
    const int node_r = r / G, hq = h * G + r % G;
    const int64_t row = (b * a.T + node_r) * a.Hq + hq;
    if (p.splits > 1) {
      float* po = p.part_o + (split * all_rows + row) * a.D + d;
      *reinterpret_cast<float2*>(po) = make_float2(x * inv, y * inv);
      if (d == 0) p.part_l[split * all_rows + row] = lse;
    } else {
      uint16_t* po = reinterpret_cast<uint16_t*>(a.out) + b * a.out_batch_stride + node_r * a.out_token_stride +
                     hq * a.out_head_stride + d;
      *reinterpret_cast<uint32_t*>(po) = pack2<BF>(x * inv, y * inv);
      if (d == 0 && a.lse) a.lse[row] = lse;
    }
  }
}

}  // namespace
}  // namespace topkp

#include "attention_tc.cuh"

namespace topkp {
namespace {

// Joins the parts of a row: weights exp(lse_i - lse).  One warp per row.
template <bool BF>
__global__ void __launch_bounds__(128) attn_join(const __grid_constant__ AttnDev p) {
  const topkp_tree_attention_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t rows = a.B * a.T * a.Hq;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= rows) return;
  float m = -INFINITY;
  for (int s = lane; s < p.splits; s += 32) m = fmaxf(m, p.part_l[s * rows + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float acc[TOPKP_MAX_HEAD_DIM / 32] = {};
  float total = 0.0f;
  for (int s = 0; s < p.splits; ++s) {
    const float li = p.part_l[s * rows + row];
    if (li == -INFINITY) continue;
    const float w = exp2f((li - m) * kLog2e);
    total += w;
    const float* po = p.part_o + (s * rows + row) * a.D;
#pragma unroll
    for (int i = 0; i < TOPKP_MAX_HEAD_DIM / 32; ++i)
      if (i * 32 + lane < a.D) acc[i] += w * po[i * 32 + lane];
  }
  const float inv = total > 0.0f ? 1.0f / total : total;
  const int64_t bt = row / a.Hq;
  const int64_t hq = row - bt * a.Hq, b = bt / a.T, t = bt - b * a.T;
  uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + b * a.out_batch_stride + t * a.out_token_stride + hq * a.out_head_stride;
#pragma unroll
  for (int i = 0; i < TOPKP_MAX_HEAD_DIM / 32; ++i)
    if (i * 32 + lane < a.D) out[i * 32 + lane] = (uint16_t)pack2<BF>(acc[i] * inv, 0.0f);
  if (lane == 0 && a.lse) a.lse[row] = total > 0.0f ? m + log2f(total) * kLn2 : total == 0.0f ? -INFINITY : total;
}

template <int DP, bool BF, bool Q8>
cudaError_t launch_mma(const AttnDev& p, cudaStream_t s) {
  const topkp_tree_attention_args& a = p.a;
  constexpr size_t tiles = mma_smem<DP>(), join = (size_t)4 * 16 * (DP + 4) * 4;
  constexpr size_t smem = tiles > join ? tiles : join;
  cudaError_t e = cudaFuncSetAttribute(attn_mma<DP, BF, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t rows = a.T * (a.Hq / a.Hkv);
  const dim3 grid((unsigned)p.splits, (unsigned)(a.B * a.Hkv), (unsigned)((rows + kRowTile - 1) / kRowTile));
  attn_mma<DP, BF, Q8><<<grid, kMmaThreads, smem, s>>>(p);
  return cudaGetLastError();
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
bool make_map(CUtensorMap* map, const topkp_cache& c, const topkp_tree_attention_args& a, int box, int width) {
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
                          boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          q8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, int NT, bool BF, bool Q8>
cudaError_t launch_tc(AttnDev p, cudaStream_t s) {
  using Shape = TcShape<DP, NT, Q8>;
  const topkp_tree_attention_args& a = p.a;
  cudaError_t e = cudaFuncSetAttribute(attn_tc<DP, NT, BF, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape::kSmem);
  if (e != cudaSuccess) return e;
  // tokens of a box: they lie in one page, and eight rows make a swizzle's group
  CUtensorMap km = {}, vm = {};
  p.box = kTile;
  if (a.table)
    while (p.box > 4 && a.page_size % p.box) p.box /= 2;
  const int width = Q8 ? DP : 64;
  if (p.box < 8 || !make_map(&km, a.k, a, p.box, width) || !make_map(&vm, a.v, a, p.box, width)) p.box = 0;
  const int64_t rows = a.T * (a.Hq / a.Hkv);
  const dim3 grid((unsigned)((rows + NT * kTcRows - 1) / (NT * kTcRows)), (unsigned)p.splits, (unsigned)(a.B * a.Hkv));
  attn_tc<DP, NT, BF, Q8><<<grid, Shape::kThreads, Shape::kSmem, s>>>(p, km, vm);
  return cudaGetLastError();
}

// Tensor memory's 128 rows pay from here on.
bool on_tensor_cores(const topkp_tree_attention_args& a) { return a.T * (a.Hq / a.Hkv) > 0; }
// Tiles of 128 rows of a CTA (256 dims leave tensor memory for one).
int row_tiles(const topkp_tree_attention_args& a) { return a.T * (a.Hq / a.Hkv) > kTcRows && a.D <= 128 ? 2 : 1; }

template <bool BF, bool Q8>
cudaError_t launch_dim(const AttnDev& p, cudaStream_t s) {
  if (on_tensor_cores(p.a)) {
    const bool two = row_tiles(p.a) == 2;
    if (p.a.D <= 64) return two ? launch_tc<64, 2, BF, Q8>(p, s) : launch_tc<64, 1, BF, Q8>(p, s);
    if (p.a.D <= 128) return two ? launch_tc<128, 2, BF, Q8>(p, s) : launch_tc<128, 1, BF, Q8>(p, s);
    return launch_tc<256, 1, BF, Q8>(p, s);
  }
  if (p.a.D <= 64) return launch_mma<64, BF, Q8>(p, s);
  if (p.a.D <= 128) return launch_mma<128, BF, Q8>(p, s);
  return launch_mma<256, BF, Q8>(p, s);
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
  const int64_t ctas = a.B * a.Hkv * ((rows + kRowTile - 1) / kRowTile);
  const int64_t cap = a.max_pages * a.page_size;
  const int64_t len = (a.max_context < cap ? (a.max_context > 0 ? a.max_context : 0) : cap) + a.T;
  const int64_t tiles = (len + kTile - 1) / kTile;
  if (on_tensor_cores(a)) {
    // Parts of equal size, whatever a request's length, so that the CTAs of
    // ragged requests even out.  In units of a tile's time: the rounds of CTAs
    // (between whole ones, as for equal requests, and what ragged ones average
    // to), four tiles for a CTA's start and end, and writing and reading the
    // partial outputs.
    const int64_t nt = row_tiles(a);
    const double slots = (a.D > 128 || nt == 2 || a.k.dtype == TOPKP_E4M3 ? 1.0 : 2.0) * num_sms;
    const double base = (double)(a.B * a.Hkv * ((rows + nt * kTcRows - 1) / (nt * kTcRows)));
    // a tile takes a CTA about 0.9 us (1.3 with two of them on an SM); a part
    // of every row costs 8 bytes an element at the copy's rate
    const double join = (double)(a.B * a.T * a.Hq * a.D) * 8.0 / 6.8e6 / (slots > num_sms ? 1.3 : 0.9);
    double best = -1.0;
    p.splits = 1;
    p.per = (int)tiles;
    for (int64_t n = 1; n <= 128 && n <= tiles; ++n) {
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
  int64_t splits = (3LL * num_sms + ctas - 1) / ctas;
  if (splits > (tiles + 1) / 2) splits = (tiles + 1) / 2;
  if (splits < 1) splits = 1;
  if (splits > 256) splits = 256;
  p.per = (int)((tiles + splits - 1) / splits);
  p.splits = (int)((tiles + p.per - 1) / p.per);
  splits = p.splits;
  const size_t all = (size_t)(a.B * a.T * a.Hq);
  p.part_bytes = splits > 1 ? (size_t)splits * all * (a.D + 1) * sizeof(float) : 0;
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
  const unsigned grid = (unsigned)((all + 3) / 4);
  if (bf) attn_join<true><<<grid, 128, 0, s>>>(p);
  else attn_join<false><<<grid, 128, 0, s>>>(p);
  *launches = 2;
  return cudaGetLastError();
}

}  // namespace topkp
