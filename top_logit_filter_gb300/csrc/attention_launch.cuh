// Launching the tensor-memory kernel of the attention calls: its arguments,
// its tensor maps, and the rule by which an instantiation is picked.  Included
// by attention.cu (each request by itself) and attention_shared.cu (requests
// that share a prefix), so that the two compile side by side.
#pragma once

#include <cuda.h>
#include <math.h>

#include "common.cuh"
#include "decode.h"
#include "internal.h"

namespace topkp {

struct AttnDev {
  topkp_tree_attention_args a;
  int splits;
  int per;        // tiles of a part (in the grouped kernel at least); the last part takes what is left
  float* part_o;  // [splits][B * T * Hq][D]
  float* part_l;  // [splits][B * T * Hq]
  uint32_t page_mul;  // reciprocal of page_size below 2^31, 0: divide
  int page_shift;
  int wide;           // an e4m3 row may be read 16 bytes at a time
  int box;            // tokens of a TMA box, 0: plain copies
  // Requests that share a prefix (the grouped kernel; its outputs are always
  // partial ones, to be joined).  stage 1: the shared tokens; a request of
  // `a` is then a group, its nodes those of all its requests in turn.  Stage
  // 2: each request's own tokens.
  int stage;
  int size;                // requests of a group
  int inner;               // stage 1: nodes of a request
  int64_t q_member;        // stage 1: from request to request in q
  int64_t ld_member;       // and in the block table
  const int32_t* shared;   // [groups]
};

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

// Tokens that group g's requests read together: whole tiles within what they
// share and within the context of each that has a node; and the first of
// those, whose block table they are read through.  By a whole warp.
__device__ __forceinline__ int shared_span(const AttnDev& p, int64_t g, int* first) {
  const topkp_tree_attention_args& a = p.a;
  int most = p.shared[g], who = p.size;
  for (int i = threadIdx.x & 31; i < p.size; i += 32) {
    const int64_t r = g * p.size + i;
    if (!a.nodes || a.nodes[r] > 0) {
      most = min(most, a.context[r]);
      who = min(who, i);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    most = min(most, __shfl_xor_sync(0xffffffffu, most, o));
    who = min(who, __shfl_xor_sync(0xffffffffu, who, o));
  }
  *first = who;
  if (who == p.size) return 0;
  return (int)min((long long)max(most, 0), (long long)(a.max_pages * a.page_size)) / kTile * kTile;
}

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

// What a launch leaves for the next one of the same call: the maps of the
// same caches (a box's shape depends on the kernel's head dimension only).
struct Maps {
  CUtensorMap k, v;
  int box = -1;  // tokens of a box, 0: TMA cannot take the caches, -1: not made
};

template <bool GROUPED, int DP, int NT, bool BF, bool Q8, int SH = 1, bool LONE = false>
cudaError_t launch_tc(AttnDev p, Maps& maps, cudaStream_t s) {
  using Shape = TcShape<DP, NT, BF, Q8, SH, LONE>;
  const topkp_tree_attention_args& a = p.a;
  // (asked for once a device and thread)
  static thread_local int configured = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured != dev) {
    const cudaError_t e = cudaFuncSetAttribute(attn_tc<GROUPED, DP, NT, BF, Q8, SH, LONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape::kSmem);
    if (e != cudaSuccess) return e;
    configured = dev;
  }
  if (maps.box < 0) {
    // tokens of a box: they lie in one page, and eight rows make a swizzle's group
    maps.box = kTile;
    if (a.table)
      while (maps.box > 4 && a.page_size % maps.box) maps.box /= 2;
    // operands are swizzled (rows of 128 bytes, or of 64 e4m3); raw values are not
    constexpr auto by128 = CU_TENSOR_MAP_SWIZZLE_128B, by64 = CU_TENSOR_MAP_SWIZZLE_64B, plain = CU_TENSOR_MAP_SWIZZLE_NONE;
    if (maps.box < 8 || !make_map(&maps.k, a.k, a, maps.box, !Q8 ? 64 : DP < 128 ? DP : 128, Q8 && DP == 64 ? by64 : by128) ||
        !make_map(&maps.v, a.v, a, maps.box, Q8 ? DP : 64, Q8 ? plain : by128))
      maps.box = 0;
  }
  p.box = maps.box;
  const int64_t rows = a.T * (a.Hq / a.Hkv);
  const dim3 grid((unsigned)((rows + NT * kTcRows - 1) / (NT * kTcRows)), (unsigned)p.splits, (unsigned)(a.B * a.Hkv));
  if (!GROUPED || p.stage != 2) {
    attn_tc<GROUPED, DP, NT, BF, Q8, SH, LONE><<<grid, Shape::kThreads, Shape::kSmem, s>>>(p, maps.k, maps.v);
    return cudaGetLastError();
  }
  // the requests' own tokens run beside the shared ones
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(Shape::kThreads);
  cfg.dynamicSmemBytes = Shape::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_tc<GROUPED, DP, NT, BF, Q8, SH, LONE>, p, maps.k, maps.v);
}

// Tiles of 128 rows of a CTA (256 dims leave tensor memory for one).
int row_tiles(const topkp_tree_attention_args& a) { return a.T * (a.Hq / a.Hkv) > kTcRows && a.D <= 128 ? 2 : 1; }

// Whether four warps share each row's tokens: up to 32 rows over e4m3, at 65 to
// 128 dims.  64 single tokens to 8000, in us with and without: 303 / 350 (fp16
// 340 / 365 with one loading warp; 276 with a warp each for keys, values and
// scales); it gives nothing at 64 dims (217 / 218) or 256 (313 / 311).
bool few_rows(const topkp_tree_attention_args& a) {
  return a.k.dtype == TOPKP_E4M3 && a.D > 64 && a.D <= 128 && a.T * (a.Hq / a.Hkv) <= 32;
}

// Two warps to a row for 33 to 64 of them, where requests share a prefix (16
// groups of 8 single tokens of 64 query and 8 cache heads, prefixes to 32000:
// 399 us, the own tokens' kernel alike; with one warp a row the softmax takes
// 1520 of a tile's 1650 cycles, with two 1030).
bool some_rows(const topkp_tree_attention_args& a) {
  const int64_t rows = a.T * (a.Hq / a.Hkv);
  return a.k.dtype == TOPKP_E4M3 && a.D > 64 && a.D <= 128 && rows > 32 && rows <= 64;
}

template <bool GROUPED, bool BF, bool Q8>
cudaError_t launch_dim(const AttnDev& p, Maps& maps, cudaStream_t s) {
  if constexpr (Q8) {
    if constexpr (GROUPED && BF) {
      if (few_rows(p.a) && p.stage == 1) return launch_tc<GROUPED, 128, 1, BF, true, 4, true>(p, maps, s);
    }
    if (few_rows(p.a)) return launch_tc<GROUPED, 128, 1, BF, true, 4>(p, maps, s);
    if constexpr (GROUPED) {
      if (some_rows(p.a)) return launch_tc<GROUPED, 128, 1, BF, true, 2>(p, maps, s);
    }
  }
  const bool two = row_tiles(p.a) == 2;
  if (p.a.D <= 64) return two ? launch_tc<GROUPED, 64, 2, BF, Q8>(p, maps, s) : launch_tc<GROUPED, 64, 1, BF, Q8>(p, maps, s);
  if (p.a.D <= 128) return two ? launch_tc<GROUPED, 128, 2, BF, Q8>(p, maps, s) : launch_tc<GROUPED, 128, 1, BF, Q8>(p, maps, s);
  return launch_tc<GROUPED, 256, 1, BF, Q8>(p, maps, s);
}

template <bool GROUPED>
cudaError_t launch_parts(const AttnDev& p, Maps& maps, cudaStream_t s) {
  const bool bf = p.a.dtype == TOPKP_BF16, q8 = p.a.k.dtype == TOPKP_E4M3;
  return bf ? (q8 ? launch_dim<GROUPED, true, true>(p, maps, s) : launch_dim<GROUPED, true, false>(p, maps, s))
            : (q8 ? launch_dim<GROUPED, false, true>(p, maps, s) : launch_dim<GROUPED, false, false>(p, maps, s));
}

}  // namespace
}  // namespace topkp
