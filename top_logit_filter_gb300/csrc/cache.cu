// topkp_cache_write and topkp_cache_read: rows of keys and values into a
// cache, in its own type or as e4m3 with a power of two for each (token,
// head), and back.
//
// The scale.  With amax the largest finite magnitude of the row, 2^e is the
// smallest power of two with amax <= 448 * 2^e; 448 = 1.75 * 2^8, so from
// amax = 1.f * 2^x it is e = x - 8, plus one if 1.f > 1.75: two integer
// operations on the bits.  Scaling by 2^-e is exact, so the stored value has
// one rounding, and reading back has none: 4 significant bits always fit the
// row's type.  A scale that is not a power of two would use up to one more
// binade of e4m3's sixteen, and add a rounding on either side.
#include "common.cuh"
#include "decode.h"

namespace topkp {
namespace {

constexpr int kCacheThreads = 256;

// Lanes of a row: a power of two, each lane VEC elements.
__host__ __device__ inline int row_lanes(int D, int vec) {
  int l = 1;
  while (l < 32 && l * vec < D) l *= 2;
  return l;
}

template <int DT, int VEC>
struct alignas(16) Rows {
  using raw = typename DType<DT>::raw;
  raw v[VEC];
};

template <int DT, int VEC>
__device__ __forceinline__ Rows<DT, VEC> load_rows(const void* p) {
  Rows<DT, VEC> r;
  using raw = typename DType<DT>::raw;
  if (VEC == 1) {
    r.v[0] = *reinterpret_cast<const raw*>(p);
  } else if (sizeof(raw) == 2) {
    *reinterpret_cast<uint4*>(&r.v[0]) = *reinterpret_cast<const uint4*>(p);
  } else {
    *reinterpret_cast<uint4*>(&r.v[0]) = reinterpret_cast<const uint4*>(p)[0];
    *reinterpret_cast<uint4*>(&r.v[VEC / 2]) = reinterpret_cast<const uint4*>(p)[1];
  }
  return r;
}
template <int DT, int VEC>
__device__ __forceinline__ void store_rows(void* p, const Rows<DT, VEC>& r) {
  using raw = typename DType<DT>::raw;
  if (VEC == 1) {
    *reinterpret_cast<raw*>(p) = r.v[0];
  } else if (sizeof(raw) == 2) {
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&r.v[0]);
  } else {
    reinterpret_cast<uint4*>(p)[0] = *reinterpret_cast<const uint4*>(&r.v[0]);
    reinterpret_cast<uint4*>(p)[1] = *reinterpret_cast<const uint4*>(&r.v[VEC / 2]);
  }
}

// Two floats to two e4m3 (lo in the low byte), to nearest even, infinities
// and larger values to 448, NaN kept.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return make_float2(__half2float(__ushort_as_half((uint16_t)h)), __half2float(__ushort_as_half((uint16_t)(h >> 16))));
}
template <int DT>
__device__ __forceinline__ typename DType<DT>::raw from_float(float f) {
  if (DT == TOPKP_F32) return (typename DType<DT>::raw)__float_as_uint(f);
  if (DT == TOPKP_F16) return (typename DType<DT>::raw)__half_as_ushort(__float2half_rn(f));
  return (typename DType<DT>::raw)__bfloat16_as_ushort(__float2bfloat16_rn(f));
}

// One group of lanes moves one row; a lane moves elements lane * VEC + i *
// lanes * VEC of it.
template <int DT, int VEC, bool QUANT>
__global__ void __launch_bounds__(kCacheThreads) write_kernel(const __grid_constant__ CacheRowsArgs a) {
  using D_ = DType<DT>;
  using raw = typename D_::raw;
  const int lanes = row_lanes(a.D, VEC);
  const int64_t rows = a.N * a.H * a.sides;
  const int64_t r = ((int64_t)blockIdx.x * kCacheThreads + threadIdx.x) / lanes;
  const int lane = threadIdx.x & (lanes - 1);
  const unsigned mask = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << (threadIdx.x & 31 & ~(lanes - 1));
  if (r >= rows) return;
  const int64_t th = r / a.sides;
  const int side = (int)(r - th * a.sides);
  const int64_t tok = th / a.H;
  const int h = (int)(th - tok * a.H);
  const int64_t slot = a.slots[tok];
  if (slot < 0 || slot >= a.slots_end) return;
  const int64_t page = slot / a.page_size;
  const int64_t at = slot - page * a.page_size;
  const raw* x = reinterpret_cast<const raw*>(a.in[side]) + tok * a.token_stride[side] + h * a.head_stride[side];
  const topkp_cache& c = a.cache[side];
  const int64_t off = page * c.page_stride + at * c.token_stride + h * c.head_stride;
  if (!QUANT) {
    raw* o = reinterpret_cast<raw*>(c.data) + off;
    for (int d = lane * VEC; d < a.D; d += lanes * VEC) store_rows<DT, VEC>(o + d, load_rows<DT, VEC>(x + d));
    return;
  }
  uint32_t amax = 0;
  constexpr int kKeep = VEC == 8 ? 1 : TOPKP_MAX_HEAD_DIM / 32;
  Rows<DT, VEC> keep[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int d = (i * lanes + lane) * VEC;
    if (d < a.D) {
      keep[i] = load_rows<DT, VEC>(x + d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const uint32_t m = __float_as_uint(D_::to_float(keep[i].v[j])) & 0x7fffffffu;
        if (m < 0x7f800000u) amax = max(amax, m);
      }
    }
  }
  for (int o = lanes / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(mask, amax, o));
  // below the normal range (and for zeros) e stays at its lowest
  const int e = max((int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0), -126);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
  uint8_t* o = reinterpret_cast<uint8_t*>(c.data) + off;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int d = (i * lanes + lane) * VEC;
    if (d < a.D) {
      if (VEC == 1) {
        o[d] = (uint8_t)to_e4m3x2(D_::to_float(keep[i].v[0]) * inv, 0.0f);
      } else {
        uint32_t w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w[j] = to_e4m3x2(D_::to_float(keep[i].v[4 * j]) * inv, D_::to_float(keep[i].v[4 * j + 1]) * inv) |
                 (to_e4m3x2(D_::to_float(keep[i].v[4 * j + 2]) * inv, D_::to_float(keep[i].v[4 * j + 3]) * inv) << 16);
        *reinterpret_cast<uint2*>(o + d) = make_uint2(w[0], w[1]);
      }
    }
  }
  if (lane == 0) c.exponents[page * c.exp_page_stride + at * c.exp_token_stride + h * c.exp_head_stride] = (uint8_t)(e + 127);
}

template <int DT, int VEC, bool QUANT>
__global__ void __launch_bounds__(kCacheThreads) read_kernel(const __grid_constant__ CacheRowsArgs a) {
  using raw = typename DType<DT>::raw;
  const int lanes = row_lanes(a.D, VEC);
  const int64_t rows = a.N * a.H * a.sides;
  const int64_t r = ((int64_t)blockIdx.x * kCacheThreads + threadIdx.x) / lanes;
  const int lane = threadIdx.x & (lanes - 1);
  if (r >= rows) return;
  const int64_t th = r / a.sides;
  const int side = (int)(r - th * a.sides);
  const int64_t tok = th / a.H;
  const int h = (int)(th - tok * a.H);
  raw* o = reinterpret_cast<raw*>(a.out[side]) + tok * a.token_stride[side] + h * a.head_stride[side];
  const int64_t slot = a.slots[tok];
  const bool in = slot >= 0 && slot < a.slots_end;
  const int64_t page = in ? slot / a.page_size : 0;
  const int64_t at = in ? slot - page * a.page_size : 0;
  const topkp_cache& c = a.cache[side];
  const int64_t off = page * c.page_stride + at * c.token_stride + h * c.head_stride;
  float scale = 0.0f;
  if (QUANT && in) {
    const uint32_t e = c.exponents[page * c.exp_page_stride + at * c.exp_token_stride + h * c.exp_head_stride];
    scale = __uint_as_float(e ? e << 23 : 0x400000u);
  }
  for (int d = lane * VEC; d < a.D; d += lanes * VEC) {
    Rows<DT, VEC> v;
#pragma unroll
    for (int j = 0; j < VEC; ++j) v.v[j] = 0;
    if (in) {
      if (!QUANT) {
        v = load_rows<DT, VEC>(reinterpret_cast<const raw*>(c.data) + off + d);
      } else if (VEC == 1) {
        v.v[0] = from_float<DT>(from_e4m3x2(reinterpret_cast<const uint8_t*>(c.data)[off + d]).x * scale);
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(c.data) + off + d);
        const uint32_t two[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = from_e4m3x2(two[j]);
          v.v[2 * j % VEC] = from_float<DT>(f.x * scale);
          v.v[(2 * j + 1) % VEC] = from_float<DT>(f.y * scale);
        }
      }
    }
    store_rows<DT, VEC>(o + d, v);
  }
}

template <int DT>
cudaError_t launch_dt(const CacheRowsArgs& a, bool write, cudaStream_t s) {
  const int64_t threads = a.N * a.H * a.sides * row_lanes(a.D, a.vec);
  const unsigned int grid = (unsigned int)((threads + kCacheThreads - 1) / kCacheThreads);
  const bool q = a.cache[0].dtype == TOPKP_E4M3;
#define TOPKP_CACHE_GO(KERNEL)                                             \
  if (a.vec == 8) {                                                        \
    if (q) KERNEL<DT, 8, true><<<grid, kCacheThreads, 0, s>>>(a);          \
    else KERNEL<DT, 8, false><<<grid, kCacheThreads, 0, s>>>(a);           \
  } else {                                                                 \
    if (q) KERNEL<DT, 1, true><<<grid, kCacheThreads, 0, s>>>(a);          \
    else KERNEL<DT, 1, false><<<grid, kCacheThreads, 0, s>>>(a);           \
  }
  if (write) {
    TOPKP_CACHE_GO(write_kernel)
  } else {
    TOPKP_CACHE_GO(read_kernel)
  }
#undef TOPKP_CACHE_GO
  return cudaGetLastError();
}

cudaError_t launch_any(topkp_dtype dt, const CacheRowsArgs& a, bool write, cudaStream_t s) {
  switch (dt) {
    case TOPKP_F32: return launch_dt<TOPKP_F32>(a, write, s);
    case TOPKP_F16: return launch_dt<TOPKP_F16>(a, write, s);
    default: return launch_dt<TOPKP_BF16>(a, write, s);
  }
}

}  // namespace

cudaError_t launch_cache_write(topkp_dtype dt, const CacheRowsArgs& a, cudaStream_t s) { return launch_any(dt, a, true, s); }
cudaError_t launch_cache_read(topkp_dtype dt, const CacheRowsArgs& a, cudaStream_t s) { return launch_any(dt, a, false, s); }

}  // namespace topkp
