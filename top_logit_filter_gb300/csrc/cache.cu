// topkp_cache_write and topkp_cache_read: rows of keys and values into a
// cache, in its own type or as e4m3 with a power of two for each (token,
// head), and back.
//
// The scale.  With amax the largest finite magnitude of the row, 2^e is the
// smallest power of two with amax <= 448 * 2^e; 448 = 1.75 * 2^8, so from
// amax = 1.f * 2^x it is e = x - 8, plus one if 1.f > 1.75: two integer
// operations on the bits.  Scaling by 2^-e is exact, so the stored value has
// one rounding, and reading back has none within the type's range, where 4
// significant bits always fit.  That one rounding goes past the range at its
// very top: fp16 magnitudes from 63488 become 65536, bf16 and fp32 ones from
// 1.9375 * 2^127 become 2^128, and both read back as infinities.  A scale that is not a power of two would use up to one more
// binade of e4m3's sixteen, and add a rounding on either side.
//
// Measured, heads of 8 x 128, bf16 and e4m3: 65501 tokens written in 102 us
// (4.0 TB/s; bound by instructions, 172 a thread for eight elements: maxima
// over the row, scaling, conversion, addresses), 32749 read in 37 (5.5 TB/s),
// 64 written in 2.2 (a launch).
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

// A thread's place is fixed for its life: a side (keys or values), a head and
// a lane of the row, and a token of each group of `tokens` tokens that the
// CTA takes; it moves kTokens tokens at once, so that as many reads are on
// their way.  Only the slot is divided, by a multiplication.
struct Place {
  int side, head, lane, token;
  bool on;
};
__device__ __forceinline__ Place place_of(const CacheRowsArgs& a, int lanes) {
  Place p;
  const int per_token = a.sides * a.H * lanes;           // threads of a token
  const int base = (int)blockIdx.y * kCacheThreads;      // first of them in this CTA, where a token has several CTAs
  const int t = base + (int)threadIdx.x;
  p.token = per_token < kCacheThreads ? (int)((uint32_t)t / (uint32_t)per_token) : 0;
  const int c = t - p.token * per_token;
  p.on = c < per_token && p.token < a.tokens;
  p.lane = c & (lanes - 1);
  const int row = p.on ? c >> (31 - __clz(lanes)) : 0;
  p.side = row >= a.H ? 1 : 0;
  p.head = row - p.side * a.H;
  return p;
}
struct Spot {
  uint32_t page;
  int at;
  bool in;
};
__device__ __forceinline__ Spot spot_of(const CacheRowsArgs& a, int64_t slot) {
  Spot s;
  s.in = slot >= 0 && slot < a.slots_end;
  if (!s.in) slot = 0;
  // slots below 2^31 go through a 32-bit reciprocal (exact there)
  s.page = a.page_mul ? __umulhi((uint32_t)slot, a.page_mul) >> a.page_shift : (uint32_t)(slot / a.page_size);
  s.at = (int)(slot - (int64_t)s.page * a.page_size);
  return s;
}

// base + i * x + j * y, one instruction a product where the strides (in
// bytes) have 32 bits: the eight-element kernels, whose 64-bit products
// would be a third of their instructions.
template <int VEC>
__device__ __forceinline__ char* at_bytes(const void* base, uint32_t i, int64_t x, uint32_t j, int64_t y) {
  uint64_t r = reinterpret_cast<uint64_t>(base);
  if (VEC == 8) {
    asm("mad.wide.u32 %0, %1, %2, %0;" : "+l"(r) : "r"(i), "r"((uint32_t)x));
    asm("mad.wide.u32 %0, %1, %2, %0;" : "+l"(r) : "r"(j), "r"((uint32_t)y));
  } else {
    r += (uint64_t)i * (uint64_t)x + (uint64_t)j * (uint64_t)y;
  }
  return reinterpret_cast<char*>(r);
}

template <int DT, int VEC, bool QUANT, int TOK>
__global__ void __launch_bounds__(kCacheThreads) write_kernel(const __grid_constant__ CacheRowsArgs a) {
  using D_ = DType<DT>;
  using raw = typename D_::raw;
  constexpr int kKeep = VEC == 8 ? 1 : TOPKP_MAX_HEAD_DIM / 32;
  const int lanes = row_lanes(a.D, VEC);
  const Place p = place_of(a, lanes);
  const unsigned mask = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << (threadIdx.x & 31 & ~(lanes - 1));
  const topkp_cache& c = a.cache[p.side];
  constexpr int ES = QUANT ? 1 : (int)sizeof(raw);
  const char* x = reinterpret_cast<const char*>(a.in[p.side]) + (p.head * a.head_stride[p.side] + p.lane * VEC) * (int64_t)sizeof(raw);
  char* o0 = reinterpret_cast<char*>(c.data) + (p.head * c.head_stride + p.lane * VEC) * ES;
  uint8_t* e0 = QUANT ? c.exponents + p.head * c.exp_head_stride : nullptr;
  const uint32_t tok0 = blockIdx.x * (uint32_t)(a.tokens * TOK) + p.token;
  const bool own = p.lane * VEC < a.D;  // this lane's first piece lies in the row

  Spot spot[TOK];
  Rows<DT, VEC> keep[TOK][kKeep];
  // every read is of a row that exists, wanted or not: a branch around each
  // would make the reads wait for one another
  int64_t slot[TOK];
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    const uint32_t tok = min(tok0 + u * a.tokens, (uint32_t)a.N - 1u);
    slot[u] = a.slots[tok];
    const char* xt = at_bytes<VEC>(x, tok, a.token_stride[p.side] * (int64_t)sizeof(raw), 0, 0);
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (VEC == 8 ? own : (i * lanes + p.lane) * VEC < a.D) keep[u][i] = load_rows<DT, VEC>(xt + i * lanes * VEC * sizeof(raw));
  }
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    spot[u] = spot_of(a, p.on && tok0 + u * a.tokens < a.N ? slot[u] : -1);
    if (!spot[u].in) continue;  // all lanes of the row alike
    char* o = at_bytes<VEC>(o0, spot[u].page, c.page_stride * ES, (uint32_t)spot[u].at, c.token_stride * ES);
    if (!QUANT) {
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (VEC == 8 ? own : (i * lanes + p.lane) * VEC < a.D) store_rows<DT, VEC>(o + i * lanes * VEC * sizeof(raw), keep[u][i]);
      continue;
    }
    uint32_t amax = 0;  // magnitude bits as fp32's
    if (VEC == 8 && sizeof(raw) == 2) {
      // two 16-bit magnitudes at once; a row with an infinity or NaN is gone
      // through again for its finite ones
      uint32_t two = 0;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&keep[u][0].v[0]);
      if (own) {
#pragma unroll
        for (int j = 0; j < 4; ++j) two = __vmaxu2(two, w[j % (VEC / 2 > 0 ? VEC / 2 : 1)] & 0x7fff7fffu);
      }
      uint32_t top = max(two & 0xffffu, two >> 16);
      for (int o = lanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(mask, top, o));
      constexpr uint32_t kInf = DT == TOPKP_F16 ? 0x7c00u : 0x7f80u;
      if (top >= kInf) {
        top = 0;
        if (own) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const uint32_t m = (uint32_t)keep[u][0].v[j] & 0x7fffu;
            if (m < kInf) top = max(top, m);
          }
        }
        for (int o = lanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(mask, top, o));
      }
      amax = __float_as_uint(D_::to_float((raw)top));
    } else {
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if ((i * lanes + p.lane) * VEC < a.D) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const uint32_t m = __float_as_uint(D_::to_float(keep[u][i].v[j])) & 0x7fffffffu;
            if (m < 0x7f800000u) amax = max(amax, m);
          }
        }
      for (int o = lanes / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(mask, amax, o));
    }
    // below the normal range (and for zeros) e stays at its lowest
    const int e = max((int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0), -126);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      if (VEC == 8 ? !own : (i * lanes + p.lane) * VEC >= a.D) continue;
      const Rows<DT, VEC>& r = keep[u][i];
      if (VEC == 1) {
        o[i * lanes] = (char)to_e4m3x2(D_::to_float(r.v[0]) * inv, 0.0f);
      } else {
        uint32_t w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w[j] = to_e4m3x2(D_::to_float(r.v[4 * j % VEC]) * inv, D_::to_float(r.v[(4 * j + 1) % VEC]) * inv) |
                 (to_e4m3x2(D_::to_float(r.v[(4 * j + 2) % VEC]) * inv, D_::to_float(r.v[(4 * j + 3) % VEC]) * inv) << 16);
        *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
      }
    }
    if (p.lane == 0)
      *at_bytes<VEC>(e0, spot[u].page, c.exp_page_stride, (uint32_t)spot[u].at, c.exp_token_stride) = (char)(e + 127);
  }
}

template <int DT, int VEC, bool QUANT, int TOK>
__global__ void __launch_bounds__(kCacheThreads) read_kernel(const __grid_constant__ CacheRowsArgs a) {
  using raw = typename DType<DT>::raw;
  constexpr int kKeep = VEC == 8 ? 1 : TOPKP_MAX_HEAD_DIM / 32;
  const int lanes = row_lanes(a.D, VEC);
  const Place p = place_of(a, lanes);
  if (!p.on) return;
  const topkp_cache& c = a.cache[p.side];
  constexpr int ES = QUANT ? 1 : (int)sizeof(raw);
  char* out = reinterpret_cast<char*>(a.out[p.side]) + (p.head * a.head_stride[p.side] + p.lane * VEC) * (int64_t)sizeof(raw);
  const char* c0 = reinterpret_cast<const char*>(c.data) + (p.head * c.head_stride + p.lane * VEC) * ES;
  const uint8_t* e0 = QUANT ? c.exponents + p.head * c.exp_head_stride : nullptr;
  const uint32_t tok0 = blockIdx.x * (uint32_t)(a.tokens * TOK) + p.token;

  Spot spot[TOK];
  Rows<DT, VEC> v[TOK][kKeep];
  uint2 w[TOK][kKeep];
  uint32_t e[TOK];
  int64_t slot[TOK];
#pragma unroll
  for (int u = 0; u < TOK; ++u) slot[u] = a.slots[min(tok0 + u * a.tokens, (uint32_t)a.N - 1u)];
  // a slot outside reads the cache's first row, and drops it
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    spot[u] = spot_of(a, slot[u]);
    const char* from = at_bytes<VEC>(c0, spot[u].page, c.page_stride * ES, (uint32_t)spot[u].at, c.token_stride * ES);
    e[u] = QUANT ? (uint32_t)*reinterpret_cast<const uint8_t*>(
                       at_bytes<VEC>(e0, spot[u].page, c.exp_page_stride, (uint32_t)spot[u].at, c.exp_token_stride))
                 : 0u;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      w[u][i] = make_uint2(0, 0);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[u][i].v[j] = 0;
      if ((i * lanes + p.lane) * VEC >= a.D) continue;
      const char* f = from + i * lanes * VEC * ES;
      if (!QUANT) v[u][i] = load_rows<DT, VEC>(f);
      else if (VEC == 1) w[u][i].x = *reinterpret_cast<const uint8_t*>(f);
      else w[u][i] = *reinterpret_cast<const uint2*>(f);
    }
  }
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    const uint32_t tok = tok0 + u * a.tokens;
    if (tok >= a.N) continue;
    char* to = at_bytes<VEC>(out, tok, a.token_stride[p.side] * (int64_t)sizeof(raw), 0, 0);
    const float scale = spot[u].in ? __uint_as_float(e[u] ? e[u] << 23 : 0x400000u) : 0.0f;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const int d = (i * lanes + p.lane) * VEC;
      if (d >= a.D) continue;
      if (!QUANT && !spot[u].in) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[u][i].v[j] = 0;
      }
      if (QUANT && !spot[u].in) w[u][i] = make_uint2(0, 0);
      if (QUANT && VEC == 1) {
        v[u][i].v[0] = from_float<DT>(from_e4m3x2(w[u][i].x).x * scale);
      } else if (QUANT) {
        const uint32_t two[4] = {w[u][i].x & 0xffffu, w[u][i].x >> 16, w[u][i].y & 0xffffu, w[u][i].y >> 16};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = from_e4m3x2(two[j]);
          v[u][i].v[2 * j % VEC] = from_float<DT>(f.x * scale);
          v[u][i].v[(2 * j + 1) % VEC] = from_float<DT>(f.y * scale);
        }
      }
      store_rows<DT, VEC>(to + i * lanes * VEC * sizeof(raw), v[u][i]);
    }
  }
}

template <int DT>
cudaError_t launch_dt(const CacheRowsArgs& args, bool write, cudaStream_t s) {
  CacheRowsArgs a = args;
  const int lanes = row_lanes(a.D, a.vec);
  const int64_t per_token = (int64_t)a.sides * a.H * lanes;
  a.tokens = per_token < kCacheThreads ? (int)(kCacheThreads / per_token) : 1;
  // page = slot / page_size = (slot * mul) >> (32 + shift), exact below 2^31
  a.page_mul = 0;
  a.page_shift = 0;
  if (a.slots_end <= (1LL << 31) && a.page_size > 1) {
    int l = 1;
    while ((1LL << l) < a.page_size) ++l;
    a.page_mul = (uint32_t)(((1ull << (31 + l)) + a.page_size - 1) / a.page_size);
    a.page_shift = l - 1;
  }
  const bool q = a.cache[0].dtype == TOPKP_E4M3;
  // four tokens a thread where that still leaves every SM its 2048 threads,
  // one where there are fewer
  const unsigned gy = (unsigned)((per_token + kCacheThreads - 1) / kCacheThreads);
  const bool many = a.vec == 8 && a.N * per_token >= 4LL * 152 * 2048;
  const int64_t per_cta = (int64_t)a.tokens * (many ? 4 : 1);
  const dim3 grid((unsigned)((a.N + per_cta - 1) / per_cta), gy);
#define TOPKP_CACHE_GO(KERNEL)                                             \
  if (a.vec == 8) {                                                        \
    if (many) {                                                            \
      if (q) KERNEL<DT, 8, true, 4><<<grid, kCacheThreads, 0, s>>>(a);     \
      else KERNEL<DT, 8, false, 4><<<grid, kCacheThreads, 0, s>>>(a);      \
    } else {                                                               \
      if (q) KERNEL<DT, 8, true, 1><<<grid, kCacheThreads, 0, s>>>(a);     \
      else KERNEL<DT, 8, false, 1><<<grid, kCacheThreads, 0, s>>>(a);      \
    }                                                                      \
  } else {                                                                 \
    if (q) KERNEL<DT, 1, true, 1><<<grid, kCacheThreads, 0, s>>>(a);       \
    else KERNEL<DT, 1, false, 1><<<grid, kCacheThreads, 0, s>>>(a);        \
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
