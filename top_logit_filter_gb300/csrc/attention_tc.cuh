// The tensor-memory kernel of topkp_tree_attention (included by attention.cu).
//
// One CTA: NT tiles of 128 rows against tiles of 64 tokens.  Warps 0 .. 4 NT - 1
// do the softmax, a thread a row (TMEM lane i is row i of its tile); the next
// warps bring keys and values into shared memory; the last warp issues
// the matrix instructions:
//   S = Q K^T   Q in TMEM (or shared memory), K in shared memory, K-major,
//               128-byte swizzle
//   O += P V    P in TMEM over its S, V in shared memory as it lies (tokens
//               by dims), read with the dims as the major direction
// (issued from uniform code: behind a branch to one lane every descriptor went
// through general registers, about 100 cycles an instruction).
// S is double-buffered, so the product of tile j + 1 runs under the softmax
// of tile j.  Up to 128 rows, two CTAs share an SM (eight warps each leave
// 128 registers a thread), and one's products run under the other's softmax;
// beyond, one CTA takes 256 rows, so that keys and values are brought (and
// values widened from e4m3) once for both tiles.  O stays in TMEM; a row's reference
// maximum moves only when a tile's maximum exceeds it by 2^8, which spares
// the rescaling of O but for the first few tiles (probabilities up to 2^8
// lose nothing in floating point).
//
// Probabilities are rounded to the rows' 16-bit type for their product with
// the values (tensor instructions take both operands alike; their sum, the
// denominator, is of the unrounded ones in fp32).  A probability is off by
// half a step of that type, as each value is, and the errors of a row's
// tokens are independent: outputs are off by little more than their own
// rounding (0.0023 against 0.0017 of a plain fp32 softmax over bf16, 0.00023
// against 0.00021 over fp16).  fp16 has no steps below 2^-24, so its
// probabilities stand 2^7 above the reference, up to 2^15, and weights down to
// 2^-32 still count (without that, 2^18 tokens of weight 2^-26, a thousandth
// of a row, went missing from O and not from the denominator).
//
// Keys and values come by TMA, a box of tokens that lie in one page at a
// time; in 16 bits straight into the swizzled operands (the last, ragged tile
// by plain copies that zero what no token fills), as e4m3 into a raw ring
// that the feeder warps widen from: sixteen values a thread, by shifts and
// two exact products with powers of two.  Layouts TMA cannot take (pages of a
// size that is no multiple of 8, e4m3 rows off 16 bytes) are copied plainly.
//
// An e4m3 key is an operand as it lies, against Q as a sum of e4m3 terms (two
// for bf16, three for fp16, both exact but for what lies 2^18 below a row's
// largest element); its scale is a factor of its column of S.  Values have to
// meet probabilities, which two or three e4m3 do not hold (a far tail of
// small ones matters together), so they are widened.
//
// 512 rows a head (64 nodes, 64 query and 8 cache heads of 128), 16 requests
// to 16000 tokens: 404 us over bf16 (1.0 PFLOP/s), 505 over e4m3 (0.80).  The
// softmax warps bound both: an exponential for every 256 multiply-adds, and
// the waits of the two products and the softmax of a tile on one another.
#pragma once

namespace topkp {
namespace {

constexpr int kTcRows = 128;
constexpr int kRun = 4;  // tiles that a loading warp looks up at once
constexpr float kSlack = 8.0f;
// what a maximum stands above the reference that is subtracted, in powers of two
template <bool BF>
constexpr float kLift = BF ? 0.0f : 7.0f;
constexpr uint64_t kWaitNs = 2000000000ull;

// bit 0: a wait of this translation unit gave up
__device__ unsigned int g_attention_error;

__device__ __forceinline__ float exp2_approx(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}
// Two fp32 in 64 bits, one instruction for both.
__device__ __forceinline__ uint64_t two_f32(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void of_two(uint64_t v, uint32_t& lo, uint32_t& hi) { asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v)); }
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
__device__ __forceinline__ uint64_t add_two(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The next three are called by a whole warp and executed by one thread of it
// (the same each time), so that the code around them stays uniform and the
// operands' descriptors stay in uniform registers.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
template <bool F8>
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  if (F8)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((int)acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((int)acc)
        : "memory");
}
template <bool F8>
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  if (F8)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((int)acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((int)acc)
        : "memory");
}
// 32 columns of this thread's lane.
__device__ __forceinline__ void tc_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
      "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr));
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand of a matrix instruction, 128-byte swizzle.  K-major:
// groups of eight rows are `stride` bytes apart.  Major in the other
// direction: groups of eight k are `stride` apart, blocks of 64 elements of
// the major direction `lead`.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)((lead >> 4) & 0x3fff) << 16) |
         ((uint64_t)((stride >> 4) & 0x3fff) << 32) | (1ull << 46) | (2ull << 61);
}
// Where 16-byte piece c of row r lies in a swizzled operand of ROWS rows.
template <int ROWS>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return (uint32_t)((c >> 3) * (ROWS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull; }

// Among the softmax warps of one row tile.
__device__ __forceinline__ void softmax_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// SH warps share a row's tokens.  With up to 32 rows over e4m3 the four softmax
// warps hold a copy of the rows each and take a quarter of every tile's tokens
// (for O's product the others' are zeros); their O, maxima and sums are joined
// at the end.  With up to 64 rows two pairs of warps take a half.
template <int DP, int NT, bool BF, bool Q8, int SH, bool LONE>
struct TcShape {
  static constexpr int kSoftWarps = 4 * NT;
  // 16 bits: one warp for keys, one for values; e4m3: one loads, the others widen
  // then bf16's 128 dims leave room for two CTAs an SM, which short requests
  // are better for (128 single tokens of 64 query and 8 cache heads to 500:
  // 64 us, fp16 with one CTA 87), LONE: one all the same, for a long prefix
  static constexpr bool kPair = SH == 4 && BF && !LONE;
  // Where there are registers for it, keys, values and their scales are brought
  // by a warp each, and two groups of warps widen values in turn: a single
  // loading warp, with the latency of its own instructions and loads, was what
  // a tile waited for (1845 of 2107 cycles), then the widening (1300 of 1620).
  // Heads of 256 gain nothing (8 / 2 heads over bf16, with and without: 64 single
  // tokens to 8000 173 / 170 us, 4 x 64 nodes to 16000 61.5 / 60.0).
  static constexpr bool kSplit = Q8 && NT == 1 && DP == 128 && !kPair;
  static constexpr int kFeedWarps = !Q8 ? 2 : NT == 2 ? 7 : kPair ? 5 : kSplit ? 11 : DP >= 128 ? 9 : 3;
  static constexpr int kWiden = kFeedWarps - (kSplit ? 3 : 1);  // warps that widen e4m3 values
  static constexpr int kThreads = 32 * (kSoftWarps + kFeedWarps + 1);
  // with a warp to a row two CTAs leave room for two warps that widen, enough for 64 dims only
  // (128 rows of 128 dims over e4m3: 258 us with two CTAs, 228 with one)
  static constexpr int kPerSm = NT == 1 && DP <= (Q8 && !kPair ? 64 : 128) ? 2 : 1;
  // e4m3 keys are operands as they lie: Q is then a sum of terms in e4m3
  static constexpr int kTerms = !Q8 ? 1 : BF ? 2 : 3;
  static constexpr int kKeyBytes = kTile * DP * (Q8 ? 1 : 2), kValueBytes = kTile * DP * 2, kRawBytes = kTile * DP;
  // Q as a shared-memory operand would be read again for every product (4 KB
  // a step, twice what a step of 64 tokens' keys is), so it sits in TMEM
  // where there is room; the second S is worth more (with one S a row tile,
  // its two products and its softmax take turns).  TMEM columns: S, Q, O.
  static constexpr int kQColumns = DP / 2 * (Q8 ? kTerms : 2) / 2;
  static constexpr bool kQInTmem = NT * (128 + kQColumns + DP) <= 512 / kPerSm;
  static constexpr int kQBytes = kQInTmem ? 0 : NT * kTcRows * DP * (Q8 ? kTerms : 2);
  // stages of keys, of values, and of raw e4m3 values.  Keys free theirs as
  // soon as their product is done, well before the softmax
  static constexpr int kKeys = Q8 ? (kPair ? 3 : DP <= 128 ? 4 : 2) : DP == 64 || (DP == 128 && NT == 2) ? 4 : DP == 256 ? 3 : 2;
  static constexpr int kValues = !Q8 ? kKeys : kPair ? 2 : DP == 256 ? (BF ? 3 : 1) : DP == 128 && NT == 2 ? 2 : 3;
  static constexpr int kRaw = !Q8 ? 0 : DP == 256 || kPair ? 2 : 4;
  // A group of warps widens every kGroups-th tile.  A wait on a stage's
  // barrier must not pass by the phase before the one that it is for: the
  // tiles between two uses of a stage see to that, so two groups need two stages.
  static constexpr int kGroups = kSplit ? 2 : 1;
  static_assert(kGroups == 1 || kValues >= 2, "a stage of values for each group");
  static constexpr uint32_t kQ = NT * 128;  // after two S of 64 columns a row tile
  static constexpr uint32_t kO = kQ + (kQInTmem ? NT * kQColumns : 0);
  static constexpr int kColumns = kO + NT * DP <= 256 ? 256 : 512;
  static constexpr size_t kSmem = 1024 + kQBytes + (size_t)kKeys * kKeyBytes + (size_t)kValues * kValueBytes + (size_t)kRaw * kRawBytes;
  static_assert(kO + NT * DP <= 512, "O does not fit tensor memory");
  static_assert(kSmem * kPerSm <= 225 * 1024, "the rings do not fit shared memory");
};
// Tiles of keys' scales kept: a softmax reads those of a tile whose keys'
// stage may have been filled again since, by at most kKeys + 2 tiles.
constexpr int kScales = 8;

// A box of tokens of one page: element x, head, token and page.
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int head, int token, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(head), "r"(token), "r"(page)
      : "memory");
}

// A stage of a ring and the parity of its round.
struct Ring {
  int at;
  uint32_t phase;
  template <int N>
  __device__ __forceinline__ void step() {
    if (++at == N) {
      at = 0;
      phase ^= 1;
    }
  }
};

// A bounded wait; once one has given up, none of the CTA waits any more.
__device__ __forceinline__ void tc_wait(uint64_t* bar, uint32_t parity, volatile int* dead) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*dead) return;
    if (globaltimer_ns() - t0 > kWaitNs) {
      *dead = 1;
      atomicOr(&g_attention_error, 1u);
      return;
    }
  }
}

// Sixteen e4m3 by the conversion instruction: fp16 rows, and what the shifts
// below do not take.
template <bool BF>
__device__ __noinline__ void widen16_slow(const uint4& w, uint32_t e, uint4& lo, uint4& hi) {
  uint32_t r[8];
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  const float s = exponent_scale(e);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(in[i >> 1] >> (16 * (i & 1)))));
    r[i] = pack2<BF>(__half2float(__ushort_as_half((uint16_t)h)) * s, __half2float(__ushort_as_half((uint16_t)(h >> 16))) * s);
  }
  lo = make_uint4(r[0], r[1], r[2], r[3]);
  hi = make_uint4(r[4], r[5], r[6], r[7]);
}
// Sixteen e4m3 times 2^(e - 127) in the rows' type.  bf16: two bytes go to
// the high bytes of two halves; sign, then exponent and mantissa four bits
// down, read as the value times 2^-120 (subnormals too), and one exact
// product with 2^(e - 7) brings it to its size.  That factor is a bf16 up to
// e = 134 (rows up to 57344), and the code 0x7f of either sign is NaN, which
// the shift would read as 480: both are left to the conversion.
template <bool BF>
__device__ __forceinline__ void widen16(const uint4& w, uint32_t e, uint4& lo, uint4& hi) {
  if (!BF) {
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t r[8];
    // fp16 holds the values themselves; the scale in two exact steps where one leaves fp16's range
    const float s = exponent_scale(e);
    const bool one = e >= 112 && e <= 142;
    const uint32_t s2 = one ? pack2<false>(s, s) : 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(in[i >> 1] >> (16 * (i & 1)))));
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r[i]) : "r"(h), "r"(s2));
    }
    lo = make_uint4(r[0], r[1], r[2], r[3]);
    hi = make_uint4(r[4], r[5], r[6], r[7]);
    if (!one) widen16_slow<BF>(w, e, lo, hi);
    return;
  }
  const uint32_t sc = (e + 120) << 7, s2 = sc | (sc << 16);
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t r[8], most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t t = __byte_perm(in[i >> 1], 0u, i & 1 ? 0x3424 : 0x1404);
    const uint32_t u = (t >> 4) & 0x07f007f0u;
    most = __vmaxu2(most, u);
    r[i] = (t & 0x80008000u) | u;
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(r[i]) : "r"(s2));
  }
  lo = make_uint4(r[0], r[1], r[2], r[3]);
  hi = make_uint4(r[4], r[5], r[6], r[7]);
  if (e > 134 || (most & 0xffffu) == 0x07f0u || (most >> 16) == 0x07f0u) widen16_slow<BF>(w, e, lo, hi);
}
// Sixteen e4m3 of a row, in two pieces where the row's alignment or end asks for it.
__device__ __forceinline__ uint4 fetch16(const uint8_t* p, int wide, bool both) {
  if (wide) return __ldg(reinterpret_cast<const uint4*>(p));
  const uint2 lo = __ldg(reinterpret_cast<const uint2*>(p));
  const uint2 hi = both ? __ldg(reinterpret_cast<const uint2*>(p) + 1) : make_uint2(0, 0);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// Element i of a pair of the rows' type.
template <bool BF>
__device__ __forceinline__ float half_of(uint32_t w, int i) {
  const uint16_t r = (uint16_t)(i ? w >> 16 : w);
  return BF ? __uint_as_float((uint32_t)r << 16) : __half2float(__ushort_as_half(r));
}
// Two floats rounded to e4m3, and what they leave (exact: both have the
// rounding's exponents).
__device__ __forceinline__ uint32_t e4m3_of(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ void e4m3_away(uint32_t two, float& x, float& y) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  x -= __half2float(__ushort_as_half((uint16_t)h));
  y -= __half2float(__ushort_as_half((uint16_t)(h >> 16)));
}

template <bool GROUPED, int DP, int NT, bool BF, bool Q8, int SH, bool LONE>
__global__ void __launch_bounds__(TcShape<DP, NT, BF, Q8, SH, LONE>::kThreads, TcShape<DP, NT, BF, Q8, SH, LONE>::kPerSm)
    attn_tc(const __grid_constant__ AttnDev p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using Shape = TcShape<DP, NT, BF, Q8, SH, LONE>;
  static_assert(SH == 1 || ((SH == 4 || SH == 2) && NT == 1 && DP == 128 && Q8), "a row's tokens go to one warp, two or four");
  constexpr int H = 32 / SH;     // half of a thread's columns of S
  constexpr int kOwn = 128 / SH;  // rows, each held by SH warps
  constexpr int KS = Shape::kKeys, VS = Shape::kValues;
  constexpr int RS = Shape::kRaw > 0 ? Shape::kRaw : 1;
  constexpr int kFeed = Shape::kFeedWarps;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ unsigned char tc_smem[];
  unsigned char* smem = tc_smem + ((1024 - (smem_u32(tc_smem) & 1023)) & 1023);
  unsigned char* sq = smem;
  unsigned char* sk = smem + Shape::kQBytes;
  unsigned char* sv = sk + KS * Shape::kKeyBytes;
  unsigned char* raw = sv + VS * Shape::kValueBytes;
  __shared__ uint64_t k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], raw_full[RS], raw_empty[RS], s_full[NT][2], p_full[NT][2], pv_done[NT], q_full;
  __shared__ uint32_t tmem_base, sexp[RS][kTile];               // values' exponents
  __shared__ __align__(16) float sscale[Q8 ? kScales : 1][kTile];  // keys' scales
  __shared__ volatile int dead;
  const topkp_tree_attention_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int G = (int)(a.Hq / a.Hkv);
  const int rows = (int)a.T * G;
  const int64_t bh = blockIdx.z;
  const int64_t b = bh / a.Hkv;
  const int h = (int)(bh - b * a.Hkv);
  const int row0 = blockIdx.x * (NT * kTcRows);
  const int split = blockIdx.y;
  int ctx, len, nodes, tile0 = 0, first = 0;
  const bool front = GROUPED && p.stage == 1;
  if (front) {
    ctx = len = shared_span(p, b, &first);
    nodes = 0;  // asked for row by row
  } else {
    request_span(a, b, &ctx, &len, &nodes);
    if (GROUPED) tile0 = shared_span(p, b / p.size, &first) / kTile;
  }
  const int tiles = (len + kTile - 1) / kTile;
  // Tiles of a part, as planned; more where what is shared, or what is a
  // request's own, is longer than the bounds that it was planned by (groups
  // with prefixes of different lengths), so that the last part is not left
  // with all the rest (4 groups of 8 requests of 32000 tokens, planned for
  // 28000 shared, of which one group shares 8000: 262 us, 358 without).
  const int per = GROUPED ? max(p.per, (tiles - tile0 + p.splits - 1) / p.splits) : p.per;
  const int t_begin = min(tile0 + split * per, tiles);
  const int n = (split == p.splits - 1 ? tiles : min(t_begin + per, tiles)) - t_begin;

  if (tid == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(&k_full[i], Q8 ? 2 : 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&v_full[i], Q8 ? Shape::kWiden / Shape::kGroups : 1);  // warps that fill a stage
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < RS; ++i) {
      mbar_init(&raw_full[i], 2);
      mbar_init(&raw_empty[i], Shape::kWiden / Shape::kGroups);
    }
    for (int t = 0; t < NT; ++t) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s_full[t][i], 1);
        mbar_init(&p_full[t][i], 128);
      }
      mbar_init(&pv_done[t], 1);
    }
    mbar_init(&q_full, NT * 128);
    fence_mbar_init();
    dead = 0;
  }
  if (warp == Shape::kSoftWarps + kFeed) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "n"(Shape::kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;

  if (warp < Shape::kSoftWarps) {
    // ---- softmax: thread = row ----
    const int tile = NT == 1 ? 0 : warp >> 2;
    const int r = SH == 1 ? row0 + tid : tid & (kOwn - 1);
    const int quarter = SH == 1 ? 0 : tid / kOwn;  // which of the warps that hold the row
    const int node = r / G;
    const int hq = h * G + (r - node * G);
    const bool in = r < rows;
    // the node's request within its group, and its place there
    const int member = front ? node / p.inner : 0, place_in = front ? node - member * p.inner : node;
    float q_scale = 1.0f;
    {
      // the row of Q into its place
      const uint16_t* qr = reinterpret_cast<const uint16_t*>(a.q) + b * a.q_batch_stride +
                           (in ? (front ? member * p.q_member : 0) + place_in * a.q_token_stride + hq * a.q_head_stride : 0);
      auto piece = [&](int c) {
        return in && c * 8 < a.D ? *reinterpret_cast<const uint4*>(qr + c * 8) : make_uint4(0, 0, 0, 0);
      };
      const uint32_t q_tmem = tm + ((uint32_t)((warp & 3) * 32) << 16) + Shape::kQ + tile * Shape::kQColumns;
      if constexpr (Q8) {
        // The row times a power of two that brings its largest magnitude to
        // e4m3's top binade, as kTerms e4m3 that add up to it: 8 significant
        // bits are two times 4, fp16's 11 three times.  What e4m3's smallest
        // step of 2^-9 cuts off lies 2^18 below the largest.
        uint32_t amax = 0;
        bool finite = true;
#pragma unroll 2
        for (int c = 0; c < DP / 8; ++c) {
          const uint4 v = piece(c);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t m = __float_as_uint(half_of<BF>(w[i >> 1], i & 1)) & 0x7fffffffu;
            finite = finite && m < 0x7f800000u;
            amax = max(amax, m);
          }
        }
        const int e = max((int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0), -126);
        const float inv = finite ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.0f;
        q_scale = finite ? __uint_as_float((uint32_t)(127 + e) << 23) : __uint_as_float(0x7fc00000u);
#pragma unroll 1
        for (int c = 0; c < DP / 64; ++c) {
          uint32_t t[Shape::kTerms][16];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 v = piece(c * 8 + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float x[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) x[u] = half_of<BF>(w[2 * k + (u >> 1)], u & 1) * inv;
#pragma unroll
              for (int term = 0; term < Shape::kTerms; ++term) {
                const uint32_t lo = e4m3_of(x[0], x[1]), hi = e4m3_of(x[2], x[3]);
                t[term][2 * i + k] = lo | (hi << 16);
                e4m3_away(lo, x[0], x[1]);
                e4m3_away(hi, x[2], x[3]);
              }
            }
          }
#pragma unroll
          for (int term = 0; term < Shape::kTerms; ++term) {
            if constexpr (Shape::kQInTmem) {
              tc_st16(q_tmem + term * (DP / 4) + c * 16, t[term]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4*>(sq + (tile * Shape::kTerms + term) * (kTcRows * DP) + swizzled<kTcRows>(tid & 127, c * 4 + i)) =
                    make_uint4(t[term][4 * i], t[term][4 * i + 1], t[term][4 * i + 2], t[term][4 * i + 3]);
            }
          }
        }
        if constexpr (Shape::kQInTmem) {
          tc_wait_st();
          tc_fence_before();
        } else {
          fence_proxy_async_shared();
        }
      } else if constexpr (Shape::kQInTmem) {
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 v = piece(c * 8 + i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
          }
          tc_st32(q_tmem + c * 32, w);
        }
        tc_wait_st();
        tc_fence_before();
      } else {
#pragma unroll 4
        for (int c = 0; c < DP / 8; ++c)
          *reinterpret_cast<uint4*>(sq + tile * (kTcRows * DP * 2) + swizzled<kTcRows>(tid & 127, c)) = piece(c);
        fence_proxy_async_shared();
      }
      mbar_arrive(&q_full);
    }
    // rows past the last (their Q is zero) and of missing nodes go along as
    // if they saw the context; what they get is not written
    if (front && in) nodes = a.nodes ? a.nodes[b * p.size + member] : p.inner;
    const bool seen = in && place_in < nodes;
    const uint64_t bits = seen && a.tree ? a.tree[b * a.T + node] : 0;
    const bool idle = SH == 1 && row0 + warp * 32 >= rows;  // the whole warp
    const int c0 = quarter * 2 * H;                 // the thread's first column of S
    const float sc0 = a.scale * kLog2e * q_scale;
    const float sc = sc0 > 0.0f ? sc0 : 1.0f;  // a scale of zero or less is applied to the products first
    const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ocol = lanes + Shape::kO + tile * DP;
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j < n; ++j) {
      const int buf = j & 1;
      const uint32_t sb = lanes + (tile * 2 + buf) * 64;
      tc_wait(&s_full[tile][buf], (j >> 1) & 1, &dead);
      if (idle) {
        if (j == n - 1 && j > 0) tc_wait(&pv_done[tile], (j - 1) & 1, &dead);
        mbar_arrive(&p_full[tile][buf]);
        continue;
      }
      __syncwarp();
      tc_fence_after();
      uint32_t s0[H], s1[H];
      if constexpr (SH == 1) {
        tc_ld32(s0, sb);
        tc_ld32(s1, sb + 32);
        tc_wait_ld();
      } else {
        uint32_t both[2 * H];
        if constexpr (SH == 4) tc_ld16(both, sb + c0);
        else tc_ld32(both, sb + c0);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < H; ++i) {
          s0[i] = both[i];
          s1[i] = both[H + i];
        }
      }
      const int t0 = (t_begin + j) * kTile;
      if (Q8) {  // the keys' scales, powers of two
        const ulonglong2* f = reinterpret_cast<const ulonglong2*>(sscale[j % kScales] + c0);
#pragma unroll
        for (int i = 0; i < H / 4; ++i) {
          const ulonglong2 x = f[i], y = f[H / 4 + i];
          of_two(mul_two(two_f32(s0[4 * i], s0[4 * i + 1]), x.x), s0[4 * i], s0[4 * i + 1]);
          of_two(mul_two(two_f32(s0[4 * i + 2], s0[4 * i + 3]), x.y), s0[4 * i + 2], s0[4 * i + 3]);
          of_two(mul_two(two_f32(s1[4 * i], s1[4 * i + 1]), y.x), s1[4 * i], s1[4 * i + 1]);
          of_two(mul_two(two_f32(s1[4 * i + 2], s1[4 * i + 3]), y.y), s1[4 * i + 2], s1[4 * i + 3]);
        }
      }
      if (!(sc0 > 0.0f)) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
          s0[i] = __float_as_uint(__uint_as_float(s0[i]) * sc0);
          s1[i] = __float_as_uint(__uint_as_float(s1[i]) * sc0);
        }
      }
      if (t0 + kTile > ctx) {  // a tile with drafted nodes in it, or past the end
        // bit i: whether the row sees token t0 + i
        const int d = t0 - ctx;
        uint64_t vis;
        if (a.tree) vis = d >= 64 ? 0 : d >= 0 ? bits >> d : (bits << -d) | low_bits(-d);
        else vis = low_bits(node + 1 - d);
        vis = (vis & low_bits(len - t0)) >> c0;
        const uint32_t v0 = (uint32_t)vis, v1 = (uint32_t)(vis >> H);
#pragma unroll
        for (int i = 0; i < H; ++i) {
          s0[i] = v0 & (1u << i) ? s0[i] : 0xff800000u;
          s1[i] = v1 & (1u << i) ? s1[i] : 0xff800000u;
        }
      }
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // four chains
#pragma unroll
      for (int i = 0; i < H; ++i) m4[i & 3] = fmaxf(m4[i & 3], fmaxf(__uint_as_float(s0[i]), __uint_as_float(s1[i])));
      const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      const float top = mx == -INFINITY ? -INFINITY : mx * sc;
      if (j == 0) {
        m = top - kLift<BF>;
      } else {
        const bool up = top > m + (kSlack + kLift<BF>) || (m == -INFINITY && top > -INFINITY);
        if (__any_sync(0xffffffffu, up)) {
          const float ref = top - kLift<BF>;
          const float f = up ? exp2f(m - ref) : 1.0f;
          if (up) {
            m = ref;
            l *= f;
          }
          tc_wait(&pv_done[tile], (j - 1) & 1, &dead);
          __syncwarp();
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < DP; c += 16) {
            uint32_t o[16];
            tc_ld16(o, ocol + c);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tc_st16(ocol + c, o);
          }
        }
      }
      const float base = m == -INFINITY ? 0.0f : m;
      const uint64_t sc2 = two_f32(__float_as_uint(sc), __float_as_uint(sc)), base2 = two_f32(__float_as_uint(-base), __float_as_uint(-base));
      uint64_t sum0 = 0ull, sum1 = 0ull;
      uint32_t pk[H];
#pragma unroll
      for (int i = 0; i < H; i += 2) {
        uint32_t x0, x1, y0, y1;
        of_two(fma_two(two_f32(s0[i], s0[i + 1]), sc2, base2), x0, x1);
        of_two(fma_two(two_f32(s1[i], s1[i + 1]), sc2, base2), y0, y1);
        const float p0 = exp2_approx(__uint_as_float(x0)), p1 = exp2_approx(__uint_as_float(x1));
        const float r0 = exp2_approx(__uint_as_float(y0)), r1 = exp2_approx(__uint_as_float(y1));
        sum0 = add_two(sum0, two_f32(__float_as_uint(p0), __float_as_uint(p1)));
        sum1 = add_two(sum1, two_f32(__float_as_uint(r0), __float_as_uint(r1)));
        pk[i / 2] = pack2<BF>(p0, p1);
        pk[H / 2 + i / 2] = pack2<BF>(r0, r1);
      }
      {
        uint32_t x0, x1;
        of_two(add_two(sum0, sum1), x0, x1);
        l += __uint_as_float(x0) + __uint_as_float(x1);
      }
      if constexpr (SH == 1) {
        tc_st32(sb, pk);
      } else {  // zeros for the tokens of the other warps
        uint32_t row[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) row[i] = i / H == quarter ? pk[i % H] : 0u;
        tc_st32(sb, row);
      }
      tc_wait_st();
      tc_fence_before();
      // a parity tells one phase from the next only: product n - 2 is seen done
      // before product n - 1, which needs this arrival, can be
      if (j == n - 1 && j > 0) tc_wait(&pv_done[tile], (j - 1) & 1, &dead);
      mbar_arrive(&p_full[tile][buf]);
    }
    if (n > 0) {
      tc_wait(&pv_done[tile], (n - 1) & 1, &dead);
      __syncwarp();
      tc_fence_after();
    }
    const int64_t all_rows = a.B * a.T * a.Hq;
    const int64_t row = (b * a.T + node) * a.Hq + hq;
    float part = 1.0f;  // this warp's weight in the row
    if constexpr (SH > 1) {
      // the warps' maxima and sums, then O in blocks of 64 dims, by way of the
      // rings, which are done with: every tile has been through its products
      float* sums = reinterpret_cast<float*>(sk);
      sums[tid] = m;
      sums[128 + tid] = l;
      softmax_barrier();
      float all_m = -INFINITY, all_l = 0.0f;
#pragma unroll
      for (int w = 0; w < SH; ++w) all_m = fmaxf(all_m, sums[w * kOwn + r]);
      const float ref = all_m == -INFINITY ? 0.0f : all_m;
#pragma unroll
      for (int w = 0; w < SH; ++w) all_l += sums[128 + w * kOwn + r] * exp2f(sums[w * kOwn + r] - ref);
      part = exp2f(m - ref);
      m = all_m;
      l = all_l;
    }
    if (!seen) l = 0.0f;
    const float inv = l > 0.0f ? 1.0f / l : l;
    const float lse = l > 0.0f ? (m + log2f(l)) * kLn2 : l == 0.0f ? -INFINITY : l;
    const bool write = in && !dead;
    if constexpr (SH > 1) {
      constexpr int kLine = 68;  // floats from row to row, 16 bytes off a multiple of the banks
      static_assert(KS * Shape::kKeyBytes + VS * Shape::kValueBytes >= 128 * kLine * 4, "the rings hold a block of O");
      constexpr int DW = 2 * H;  // dims of a block of 64 that a thread writes
      float* ring = reinterpret_cast<float*>(sk);
#pragma unroll 1
      for (int c = 0; c < DP; c += 64) {
        softmax_barrier();  // what the last block, or the sums, left has been read
#pragma unroll
        for (int k = 0; k < 64; k += 32) {
          uint32_t o[32];
          if (n > 0) {
            tc_ld32(o, ocol + c + k);
            tc_wait_ld();
          }
          float4* to = reinterpret_cast<float4*>(ring + tid * kLine + k);
          const float f = part * inv;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            to[i] = n > 0 && l != 0.0f ? make_float4(__uint_as_float(o[4 * i]) * f, __uint_as_float(o[4 * i + 1]) * f,
                                                     __uint_as_float(o[4 * i + 2]) * f, __uint_as_float(o[4 * i + 3]) * f)
                                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        softmax_barrier();
        const int d = c + c0;
        float x[DW];
#pragma unroll
        for (int i = 0; i < DW / 4; ++i) {
          float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < SH; ++w) {
            const float4 u = *reinterpret_cast<const float4*>(ring + (w * kOwn + r) * kLine + c0 + 4 * i);
            t = make_float4(t.x + u.x, t.y + u.y, t.z + u.z, t.w + u.w);
          }
          x[4 * i] = t.x;
          x[4 * i + 1] = t.y;
          x[4 * i + 2] = t.z;
          x[4 * i + 3] = t.w;
        }
        if (write) {
          if (GROUPED || p.splits > 1) {
            float4* po = reinterpret_cast<float4*>(p.part_o + ((int64_t)split * all_rows + row) * a.D + d);
#pragma unroll
            for (int i = 0; i < DW / 4; ++i)
              if (d + i * 4 < a.D) po[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          } else {
            uint4* po = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + b * a.out_batch_stride +
                                                 node * a.out_token_stride + hq * a.out_head_stride + d);
#pragma unroll
            for (int i = 0; i < DW / 8; ++i)
              if (d + i * 8 < a.D)
                po[i] = make_uint4(pack2<BF>(x[8 * i], x[8 * i + 1]), pack2<BF>(x[8 * i + 2], x[8 * i + 3]),
                                   pack2<BF>(x[8 * i + 4], x[8 * i + 5]), pack2<BF>(x[8 * i + 6], x[8 * i + 7]));
          }
        }
        __syncwarp();
      }
    }
#pragma unroll 1
    for (int c = 0; SH == 1 && c < DP; c += 32) {
      uint32_t o[32];
      if (n > 0) {
        tc_ld32(o, ocol + c);
        tc_wait_ld();
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = n > 0 && l != 0.0f ? __float_as_uint(__uint_as_float(o[i]) * inv) : 0u;
      if (write) {
        if (GROUPED || p.splits > 1) {
          uint4* po = reinterpret_cast<uint4*>(p.part_o + ((int64_t)split * all_rows + row) * a.D + c);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i * 4 < a.D) po[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else {
          uint4* po = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + b * a.out_batch_stride +
                                               node * a.out_token_stride + hq * a.out_head_stride + c);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i * 8 < a.D) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack2<BF>(__uint_as_float(o[8 * i + 2 * k]), __uint_as_float(o[8 * i + 2 * k + 1]));
              po[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
      }
      __syncwarp();
    }
    if (write && quarter == 0) {
      if (GROUPED || p.splits > 1) p.part_l[(int64_t)split * all_rows + row] = lse;
      else if (a.lse) a.lse[row] = lse;
    }
    tc_fence_before();
  } else if (warp < Shape::kSoftWarps + kFeed) {
    // ---- keys and values ----
    const int feeder = warp - Shape::kSoftWarps;
    const int32_t* table = a.table ? a.table + b * a.ld_table + (front ? first * p.ld_member : 0) : nullptr;
    // the page and place of token t; the page may lie outside the pool
    auto place = [&](int t, int& page, int& at) {
      page = (int)b;
      at = t;
      if (table) {
        const int pg = p.page_mul ? (int)(__umulhi((uint32_t)t, p.page_mul) >> p.page_shift) : t / (int)a.page_size;
        at = t - pg * (int)a.page_size;
        page = table[pg];
      }
    };
    // the same of a token that this thread reads itself; page -1: nothing to read
    auto find = [&](int t, int& page, int& at) {
      page = -1;
      at = 0;
      if (t < len) {
        place(t, page, at);
        if (page < 0 || page >= a.pages) page = -1;
      }
    };
    auto hand_over = [&](uint64_t* bar) {  // this warp's part of a stage, written by plain stores
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    const int per_tile = p.box ? kTile / p.box : 0;  // boxes of a tile (and of each 64 dims in 16 bits)
    if constexpr (!Q8) {
      // one warp for keys, one for values; a lane a box, its page looked up a tile ahead
      const topkp_cache& ca = feeder == 0 ? a.k : a.v;
      const CUtensorMap* map = feeder == 0 ? &kmap : &vmap;
      unsigned char* ring = feeder == 0 ? sk : sv;
      uint64_t* full = feeder == 0 ? k_full : v_full;
      uint64_t* empty = feeder == 0 ? k_empty : v_empty;
      const int S = feeder == 0 ? KS : VS;  // the stages are of one size here
      const uint16_t* base = reinterpret_cast<const uint16_t*>(ca.data) + h * ca.head_stride;
      const int blk = per_tile ? lane / per_tile : 0, piece = per_tile ? lane - blk * per_tile : 0;
      const bool boxed = lane < per_tile * (DP / 64);
      int page = -1, at = 0;
      if (boxed && n > 0) place(min(t_begin * kTile + piece * p.box, len - 1), page, at);
      int st = 0, phase = 1;  // the first round finds every stage empty
      for (int j = 0; j < n; ++j) {
        unsigned char* dst = ring + st * Shape::kValueBytes;
        tc_wait(&empty[st], phase, &dead);
        __syncwarp();
        if (p.box && (t_begin + j + 1) * kTile <= len) {
          if (lane == 0) mbar_arrive_expect_tx(&full[st], Shape::kValueBytes);
          __syncwarp();
          if (boxed) {
            tma_box(dst + blk * (kTile * 128) + piece * p.box * 128, map, &full[st], blk * 64, h, at, page);
            if (j + 1 < n) place(min((t_begin + j + 1) * kTile + piece * p.box, len - 1), page, at);
          }
        } else {
          // the ragged tile, and layouts TMA cannot take: zeros where no token is
          constexpr int CH = DP / 8;
          for (int i = lane; i < kTile * CH; i += 32) {
            const int r = i / CH, c = i - r * CH;
            int pg = -1, to = 0;
            if (c * 8 < a.D) find((t_begin + j) * kTile + r, pg, to);
            const bool in = pg >= 0;
            cp16(smem_u32(dst) + swizzled<kTile>(r, c),
                 in ? base + (int64_t)pg * ca.page_stride + (int64_t)to * ca.token_stride + c * 8 : reinterpret_cast<const uint16_t*>(ca.data), in);
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          hand_over(&full[st]);
        }
        if (++st == S) {
          st = 0;
          phase ^= 1;
        }
      }
    } else {
      // The first warp (or the first two) brings keys, which are operands as
      // they lie, values into the raw ring, and the scales of both (a fence of
      // a warp that widens would wait for such loads); the others widen values.
      constexpr uint32_t kToken = 1u << 16;  // beside a value's exponent: there is a token
      if (Shape::kSplit && feeder < 2) {
        // Keys, or values; a lane a box, its page (outside the pool past the
        // last token, which reads as zeros) looked up a tile ahead.
        const bool val = feeder == 1, boxed = lane < per_tile;
        const int piece = boxed ? lane : 0;
        const int t_end = min(len, (t_begin + n) * kTile);
        int pg = -1, to = 0;
        auto look = [&](int j) {
          const int t = (t_begin + j) * kTile + piece * p.box;
          place(min(t, len - 1), pg, to);
          if (!boxed || t >= t_end) pg = -1;
        };
        if (n > 0) look(0);
        Ring ring = {0, 1};
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          uint64_t* full = val ? &raw_full[ring.at] : &k_full[ring.at];
          unsigned char* to_smem = val ? raw + ring.at * Shape::kRawBytes : sk + ring.at * Shape::kKeyBytes;
          // each full barrier takes two arrivals: this one, and that of the warp with the scales
          tc_wait(val ? &raw_empty[ring.at] : &k_empty[ring.at], ring.phase, &dead);
          __syncwarp();
          if (p.box) {
            if (lane == 0) mbar_arrive_expect_tx(full, val ? Shape::kRawBytes : Shape::kKeyBytes);
            __syncwarp();
            if (boxed) {
              tma_box(to_smem + piece * p.box * DP, val ? &vmap : &kmap, full, 0, h, to, pg);
            }
          } else {
            if (!val) {  // (values are read by the warps that widen them)
              constexpr int CH = DP / 16;
              for (int x = lane; x < kTile * CH; x += 32) {
                const int r = x / CH, c = x - r * CH;
                int page1 = -1, at1 = 0;
                if (c * 16 < a.D) find((t_begin + j) * kTile + r, page1, at1);
                uint4 w = make_uint4(0, 0, 0, 0);
                if (page1 >= 0)
                  w = fetch16(reinterpret_cast<const uint8_t*>(a.k.data) + h * a.k.head_stride + (int64_t)page1 * a.k.page_stride +
                                  (int64_t)at1 * a.k.token_stride + c * 16,
                              p.wide, c * 16 + 8 < a.D);
                *reinterpret_cast<uint4*>(to_smem + swizzled<kTile>(r, c)) = w;
              }
              fence_proxy_async_shared();
              __syncwarp();
            }
            if (lane == 0) mbar_arrive(full);
          }
          if (j + 1 < n) look(j + 1);
          if (val) ring.template step<RS>();
          else ring.template step<KS>();
        }
      } else if (Shape::kSplit && feeder == 2) {
        // This warp brings the scales: all pages of a run are asked for at
        // once, then all its exponents, this lane's two tokens of each tile.
        const uint8_t* ke = a.k.exponents + h * a.k.exp_head_stride;
        const uint8_t* ve = a.v.exponents + h * a.v.exp_head_stride;
        Ring kr = {0, 1}, rr = {0, 1};
#pragma unroll 1
        for (int j0 = 0; j0 < n; j0 += kRun) {
          // (unconditional reads, at places that exist: a branch around each would make them wait for one another)
          int page[2 * kRun], at[2 * kRun];
          uint32_t e[2 * kRun], ek[2 * kRun], ev[2 * kRun];
          const int t0 = (t_begin + j0) * kTile, t_end = min(len, (t_begin + n) * kTile);
#pragma unroll
          for (int i = 0; i < 2 * kRun; ++i) place(min(t0 + i * 32 + lane, len - 1), page[i], at[i]);
#pragma unroll
          for (int i = 0; i < 2 * kRun; ++i) {
            const bool in = (uint32_t)page[i] < (uint32_t)a.pages && t0 + i * 32 + lane < t_end;
            const uint32_t q = in ? page[i] : 0, t = in ? at[i] : 0;  // strides have 32 bits
            e[i] = in ? kToken : 0;
            ek[i] = __ldg(ke + (uint64_t)q * (uint32_t)a.k.exp_page_stride + (uint64_t)t * (uint32_t)a.k.exp_token_stride);
            ev[i] = __ldg(ve + (uint64_t)q * (uint32_t)a.v.exp_page_stride + (uint64_t)t * (uint32_t)a.v.exp_token_stride);
          }
#pragma unroll 1
          for (int i = 0; i < kRun && j0 + i < n; ++i) {
            // the run's registers are indexed by selects, not unrolled code
            uint32_t k2[2] = {0, 0}, v2[2] = {0, 0};
#pragma unroll
            for (int u = 0; u < kRun; ++u)
              if (u == i) {
                k2[0] = e[2 * u] ? ek[2 * u] : 127;
                k2[1] = e[2 * u + 1] ? ek[2 * u + 1] : 127;
                v2[0] = e[2 * u] ? kToken | ev[2 * u] : 0;
                v2[1] = e[2 * u + 1] ? kToken | ev[2 * u + 1] : 0;
              }
            // an arrival of a later round must not be taken for the other warp's of this one
            tc_wait(&k_empty[kr.at], kr.phase, &dead);
            float* f = sscale[(j0 + i) % kScales];
            f[lane] = exponent_scale(k2[0]);
            f[lane + 32] = exponent_scale(k2[1]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_full[kr.at]);
            tc_wait(&raw_empty[rr.at], rr.phase, &dead);
            sexp[rr.at][lane] = v2[0];
            sexp[rr.at][lane + 32] = v2[1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_full[rr.at]);
            kr.template step<KS>();
            rr.template step<RS>();
          }
        }
      } else if (!Shape::kSplit && feeder == 0) {
        const uint8_t* ke = a.k.exponents + h * a.k.exp_head_stride;
        const uint8_t* ve = a.v.exponents + h * a.v.exp_head_stride;
        // boxes: lanes 0-15 keys (blocks of 128 dims), 16-31 values
        constexpr int KW = DP < 128 ? DP : 128;  // bytes of a row of a keys' block
        const bool val = lane >= 16;
        const int blk = per_tile && !val ? lane / per_tile : 0, piece = per_tile ? (val ? lane - 16 : lane - blk * per_tile) : 0;
        const bool boxed = val ? piece < per_tile : lane < per_tile * (DP / KW);
        Ring kr = {0, 1}, rr = {0, 1};
        // All pages of a run are asked for at once, then all its exponents,
        // so that a run waits for each once: this lane's two rows of each
        // tile, and its box (outside the pool past the last token, which
        // reads as zeros).
#pragma unroll 1
        for (int j0 = 0; j0 < n; j0 += kRun) {
          // The reads are unconditional, at places that exist, and what is not
          // wanted is dropped after: a branch around each would make them wait
          // for one another.
          int page[2 * kRun], at[2 * kRun], bpage[kRun], bat[kRun];
          uint32_t e[2 * kRun];
          const int t0 = (t_begin + j0) * kTile, t_end = min(len, (t_begin + n) * kTile);
#pragma unroll
          for (int i = 0; i < 2 * kRun; ++i) place(min(t0 + i * 32 + lane, len - 1), page[i], at[i]);
#pragma unroll
          for (int i = 0; i < kRun; ++i) place(min(t0 + i * kTile + piece * p.box, len - 1), bpage[i], bat[i]);
#pragma unroll
          for (int i = 0; i < kRun; ++i)
            if (!boxed || t0 + i * kTile + piece * p.box >= t_end) bpage[i] = -1;
          uint32_t ek[2 * kRun], ev[2 * kRun];
#pragma unroll
          for (int i = 0; i < 2 * kRun; ++i) {
            const bool in = (uint32_t)page[i] < (uint32_t)a.pages && t0 + i * 32 + lane < t_end;
            const uint32_t q = in ? page[i] : 0, t = in ? at[i] : 0;  // strides have 32 bits
            e[i] = in ? kToken : 0;
            ek[i] = __ldg(ke + (uint64_t)q * (uint32_t)a.k.exp_page_stride + (uint64_t)t * (uint32_t)a.k.exp_token_stride);
            ev[i] = __ldg(ve + (uint64_t)q * (uint32_t)a.v.exp_page_stride + (uint64_t)t * (uint32_t)a.v.exp_token_stride);
          }
#pragma unroll 1
          for (int i = 0; i < kRun && j0 + i < n; ++i) {
            // the run's registers are indexed by selects, not unrolled code:
            // the roles of this kernel share the instruction cache
            uint32_t k2[2] = {0, 0}, v2[2] = {0, 0};
            int pg = -1, to = 0;
#pragma unroll
            for (int u = 0; u < kRun; ++u)
              if (u == i) {
                k2[0] = e[2 * u] ? ek[2 * u] : 127;
                k2[1] = e[2 * u + 1] ? ek[2 * u + 1] : 127;
                v2[0] = e[2 * u] ? kToken | ev[2 * u] : 0;
                v2[1] = e[2 * u + 1] ? kToken | ev[2 * u + 1] : 0;
                pg = bpage[u];
                to = bat[u];
              }
            unsigned char* kd = sk + kr.at * Shape::kKeyBytes;
            unsigned char* vd = raw + rr.at * Shape::kRawBytes;
            // each full barrier takes two arrivals: the boxes on their way, and what is stored here
            tc_wait(&k_empty[kr.at], kr.phase, &dead);
            __syncwarp();
            if (p.box) {
              if (lane == 0) mbar_arrive_expect_tx(&k_full[kr.at], Shape::kKeyBytes);
              __syncwarp();
              if (boxed && !val) tma_box(kd + blk * (kTile * 128) + piece * p.box * KW, &kmap, &k_full[kr.at], blk * 128, h, to, pg);
            } else {
              if (lane == 0) mbar_arrive(&k_full[kr.at]);
              constexpr int CH = DP / 16;
              for (int x = lane; x < kTile * CH; x += 32) {
                const int r = x / CH, c = x - r * CH;
                int page1 = -1, at1 = 0;
                if (c * 16 < a.D) find((t_begin + j0 + i) * kTile + r, page1, at1);
                uint4 w = make_uint4(0, 0, 0, 0);
                if (page1 >= 0)
                  w = fetch16(reinterpret_cast<const uint8_t*>(a.k.data) + h * a.k.head_stride + (int64_t)page1 * a.k.page_stride +
                                  (int64_t)at1 * a.k.token_stride + c * 16,
                              p.wide, c * 16 + 8 < a.D);
                const uint32_t off = DP == 64 ? (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)) : swizzled<kTile>(r, c);
                *reinterpret_cast<uint4*>(kd + off) = w;
              }
              fence_proxy_async_shared();
            }
            float* f = sscale[(j0 + i) % kScales];
            f[lane] = exponent_scale(k2[0]);
            f[lane + 32] = exponent_scale(k2[1]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_full[kr.at]);
            tc_wait(&raw_empty[rr.at], rr.phase, &dead);
            __syncwarp();
            if (lane == 0) {
              if (p.box) mbar_arrive_expect_tx(&raw_full[rr.at], Shape::kRawBytes);
              else mbar_arrive(&raw_full[rr.at]);
            }
            __syncwarp();
            if (boxed && val) tma_box(vd + piece * p.box * DP, &vmap, &raw_full[rr.at], 0, h, to, pg);
            sexp[rr.at][lane] = v2[0];
            sexp[rr.at][lane + 32] = v2[1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_full[rr.at]);
            kr.template step<KS>();
            rr.template step<RS>();
          }
        }
      } else {
        constexpr int GROUPS = Shape::kGroups, kTeam = Shape::kWiden / GROUPS;  // warps that share a tile
        const int pw = warp - (Shape::kSoftWarps + kFeed - Shape::kWiden), group = pw / kTeam;
        const int pt = (pw - group * kTeam) * 32 + lane;
        constexpr int CH = DP / 16;                  // 16-byte pieces of a cached row
        constexpr int STEP = 32 * kTeam / CH;  // rows between a thread's rows
        const int c = pt % CH, r0 = pt / CH;
        const bool c_in = c * 16 < a.D;
        // This thread's pieces of the values of tile j; rows without a token
        // become zeros whatever the box held.  Two or
        // three are read before the first is widened.
        constexpr int NR = (kTile + STEP - 1) / STEP;
        constexpr int NB = NR % 3 == 0 ? 3 : NR % 2 == 0 ? 2 : 1;  // at a time
        Ring vr = {0, 1}, rr = {0, 0};  // an empty stage's wait starts passed
        if (group) {
          vr.template step<VS>();
          rr.template step<RS>();
        }
#pragma unroll 1
        for (int j = group; j < n; j += GROUPS) {
          tc_wait(&raw_full[rr.at], rr.phase, &dead);
          tc_wait(&v_empty[vr.at], vr.phase, &dead);
          const unsigned char* from = raw + rr.at * Shape::kRawBytes + c * 16;
          unsigned char* dst = sv + vr.at * Shape::kValueBytes;
#pragma unroll 1
          for (int i0 = 0; i0 < NR; i0 += NB) {
            uint4 w[NB];
            uint32_t e[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              const int r = min(r0 + (i0 + i) * STEP, kTile - 1);
              e[i] = sexp[rr.at][r];
              w[i] = *reinterpret_cast<const uint4*>(from + r * DP);
            }
            if (!p.box) {
#pragma unroll 1
              for (int i = 0; i < NB; ++i) {
                uint4 x = make_uint4(0, 0, 0, 0);
                const int r = min(r0 + (i0 + i) * STEP, kTile - 1);
                if ((sexp[rr.at][r] & kToken) && c_in) {
                  int page, at;
                  find((t_begin + j) * kTile + r, page, at);
                  x = fetch16(reinterpret_cast<const uint8_t*>(a.v.data) + h * a.v.head_stride + (int64_t)page * a.v.page_stride +
                                  (int64_t)at * a.v.token_stride + c * 16,
                              p.wide, c * 16 + 8 < a.D);
                }
#pragma unroll
                for (int k = 0; k < NB; ++k)
                  if (k == i) w[k] = x;
              }
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              const int r = r0 + (i0 + i) * STEP;
              if (r0 >= STEP || (NR * STEP != kTile && r >= kTile)) continue;
              if (!(e[i] & kToken)) w[i] = make_uint4(0, 0, 0, 0);
              uint4 lo, hi;
              widen16<BF>(w[i], e[i] & 0xff, lo, hi);
              *reinterpret_cast<uint4*>(dst + swizzled<kTile>(r, 2 * c)) = lo;
              *reinterpret_cast<uint4*>(dst + swizzled<kTile>(r, 2 * c + 1)) = hi;
            }
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&v_full[vr.at]);
            mbar_arrive(&raw_empty[rr.at]);
          }
#pragma unroll
          for (int i = 0; i < GROUPS; ++i) {
            vr.template step<VS>();
            rr.template step<RS>();
          }
        }
      }
    }
  } else {
    // ---- matrix instructions ----
    constexpr uint32_t kind = BF ? 1u : 0u;
    constexpr uint32_t common = (1u << 4) | (kind << 7) | (kind << 10) | ((uint32_t)(kTcRows / 16) << 24);
    // e4m3 by e4m3 takes 32 dims a step: both formats are code 0
    constexpr uint32_t i_qk = (Q8 ? (1u << 4) | ((uint32_t)(kTcRows / 16) << 24) : common) | ((uint32_t)(kTile / 8) << 17);
    constexpr uint32_t i_pv = common | (1u << 16) | ((uint32_t)(DP / 8) << 17);
    const uint32_t q0 = smem_u32(sq), k0 = smem_u32(sk), v0 = smem_u32(sv);
    Ring kr = {0, 0}, vr = {0, 0};
    // S of row tile t against the keys of stage kr, into buffer `buf`
    auto product_s = [&](int t, int buf) {
      const uint32_t d = tm + (t * 2 + buf) * 64;
      const uint32_t ka = k0 + kr.at * Shape::kKeyBytes;
      // rows of 128 bytes swizzled over eight, or (64 e4m3) of 64 bytes
      const uint64_t kd = Q8 && DP == 64 ? (operand(ka, 16, 512) & ~(7ull << 61)) | (4ull << 61) : operand(ka, 16, 1024);
      constexpr int STEPS = DP / (Q8 ? 32 : 16);
      // in 16-byte units a step is 2, a block of 128 bytes of the tile's rows kTile * 8
      if constexpr (Shape::kQInTmem) {
        const uint32_t qa = tm + Shape::kQ + t * Shape::kQColumns;
#pragma unroll
        for (int term = 0; term < Shape::kTerms; ++term)
#pragma unroll
          for (int kk = 0; kk < STEPS; ++kk)
            tc_mma_ts<Q8>(d, qa + (term * STEPS + kk) * 8, kd + (kk / 4) * (kTile * 8) + (kk % 4) * 2, i_qk, term + kk > 0);
      } else {
        const uint64_t qd = operand(q0 + t * (Shape::kQBytes / NT), 16, 1024);
#pragma unroll
        for (int term = 0; term < Shape::kTerms; ++term)
#pragma unroll
          for (int kk = 0; kk < STEPS; ++kk)
            tc_mma_ss<Q8>(d, qd + term * (kTcRows * DP / 16) + (kk / 4) * (kTcRows * 8) + (kk % 4) * 2,
                          kd + (kk / 4) * (kTile * 8) + (kk % 4) * 2, i_qk, term + kk > 0);
      }
      if (t == NT - 1) tc_commit(&k_empty[kr.at]);
      tc_commit(&s_full[t][buf]);
    };
    if (n > 0) {
      tc_wait(&q_full, 0, &dead);
      tc_wait(&k_full[0], 0, &dead);
      tc_fence_after();
      for (int t = 0; t < NT; ++t) product_s(t, 0);
      kr.template step<KS>();
    }
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const int buf = j & 1;
      if (j + 1 < n) {
        tc_wait(&k_full[kr.at], kr.phase, &dead);
        for (int t = 0; t < NT; ++t) {
          // the other S still holds P of tile j - 1 until its product is done
          if (j > 0) tc_wait(&pv_done[t], (j - 1) & 1, &dead);
          tc_fence_after();
          product_s(t, buf ^ 1);
        }
        kr.template step<KS>();
      }
      for (int t = 0; t < NT; ++t) {
        tc_wait(&p_full[t][buf], (j >> 1) & 1, &dead);
        if (t == 0) tc_wait(&v_full[vr.at], vr.phase, &dead);
        tc_fence_after();
        const uint64_t vd = operand(v0 + vr.at * Shape::kValueBytes, kTile * 128, 1024);
        const uint32_t pa = tm + (t * 2 + buf) * 64;
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          tc_mma_ts<false>(tm + Shape::kO + t * DP, pa + kk * 8, vd + kk * 128, i_pv, j > 0 || kk > 0);
        if (t == NT - 1) tc_commit(&v_empty[vr.at]);
        tc_commit(&pv_done[t]);
      }
      vr.template step<VS>();
    }
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (dead) {  // products and copies may still be in flight: time for them to end
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 10000000ull) __nanosleep(1000);
  }
  if (warp == Shape::kSoftWarps + kFeed) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(Shape::kColumns) : "memory");
    // A join that waits for this launch waits for the one before it, too: its
    // last CTA does not end before that has.  (All of them waiting would hold
    // the SMs that the rest of this launch is to run on.)  Its tensor memory
    // is free by then: a CTA of the launch before may be on this SM and still
    // be asking for it, and neither would ever go on.
    if (GROUPED && p.stage == 2 && blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1)
      asm volatile("griddepcontrol.wait;" ::: "memory");
  }
}

}  // namespace
}  // namespace topkp
