// C ABI of the decoding calls (topkp_decode.h): argument checks (host only,
// no device sync) and launches, in the order of api.cu: null pointers, then
// dtypes, then shapes.
#include <algorithm>
#include <climits>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>

#include "decode.h"
#include "internal.h"

using namespace topkp;

namespace {

topkp_status fail(topkp_status code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
topkp_status fail(topkp_status code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return report_error(code, buf);
}

int esize(int dt) { return dt == TOPKP_F32 ? 4 : dt == TOPKP_F16 || dt == TOPKP_BF16 ? 2 : dt == TOPKP_E4M3 ? 1 : 0; }
bool row_type(int dt) { return dt == TOPKP_F32 || dt == TOPKP_F16 || dt == TOPKP_BF16; }

struct Range {
  const void* p;
  size_t n;
};
bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + b.n && y < x + a.n;
}

topkp_status launched(const char* fn, cudaError_t e, int launches) {
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(TOPKP_ERR_LAUNCH, "%s: launch failed (%s)", fn, cudaGetErrorString(e));
  }
  report_launches(launches);
  return TOPKP_SUCCESS;
}

// One side of a state of the reordering: rows of blocks of bytes.
struct Region {
  uintptr_t at;
  int64_t row, block;    // strides
  int64_t blocks, len;   // of a row; bytes of a block
  int64_t extent;        // bytes from a row's first to its last
  int64_t state;
  bool written;
  uintptr_t end(int64_t rows) const { return at + (uintptr_t)((rows - 1) * row + extent); }
  uintptr_t residue() const { return at % (uintptr_t)row; }
};
int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }
// Whether two regions of `rows` rows share a byte.  Exact where their strides
// are equal; with two block strides a row counts as one block from its first
// byte to its last, and with two row strides the whole regions do.
bool share(const Region& a, const Region& b, int64_t rows) {
  if (a.at >= b.end(rows) || b.at >= a.end(rows)) return false;
  if (rows > 1 && a.row != b.row) return true;
  const bool whole = (a.blocks > 1 || b.blocks > 1) && !(a.blocks > 1 && b.blocks > 1 && a.block == b.block);
  const int64_t na = whole ? 1 : a.blocks, nb = whole ? 1 : b.blocks, la = whole ? a.extent : a.len, lb = whole ? b.extent : b.len;
  // block p of row i and block q of row j share one iff -lb < d - (i - j) row - (p - q) block < la
  const int64_t d = (int64_t)(b.at - a.at), m0 = floor_div(d, a.row);
  for (int64_t m = std::max(m0 - 1, 1 - rows); m <= std::min(m0 + 2, rows - 1); ++m) {
    const int64_t e = d - m * a.row;
    if (na == 1 && nb == 1) {
      if (-lb < e && e < la) return true;
      continue;
    }
    const int64_t low = std::max(floor_div(e - la, a.block) + 1, 1 - nb), high = std::min(floor_div(e + lb - 1, a.block), na - 1);
    if (low <= high) return true;
  }
  return false;
}
// Two regions that share a byte, one of them written; false if there are none.
// Regions are sorted by address and, where a cluster of them lies interleaved
// (views of one tensor), by their place within a row.
bool clash(Region* r, int64_t n, int64_t rows, const Region** one, const Region** other) {
  std::sort(r, r + n, [](const Region& a, const Region& b) { return a.at < b.at; });
  auto bad = [&](const Region& a, const Region& b) {
    if (!(a.written || b.written) || !share(a, b, rows)) return false;
    *one = &a;
    *other = &b;
    return true;
  };
  for (int64_t first = 0, last; first < n; first = last) {
    uintptr_t end = r[first].end(rows);
    bool alike = true;
    for (last = first + 1; last < n && r[last].at < end; ++last) {
      end = std::max(end, r[last].end(rows));
      alike = alike && r[last].row == r[first].row;
    }
    if (last - first == 1) continue;
    if (!alike) {
      for (int64_t i = first; i < last; ++i)
        for (int64_t j = i + 1; j < last && r[j].at < r[i].end(rows); ++j)
          if (bad(r[i], r[j])) return true;
      continue;
    }
    std::sort(r + first, r + last, [](const Region& a, const Region& b) { return a.residue() < b.residue(); });
    const uintptr_t row = (uintptr_t)r[first].row;
    for (int64_t i = first; i < last; ++i) {
      const uintptr_t to = r[i].residue() + (uintptr_t)r[i].extent;
      for (int64_t j = i + 1; j < last && r[j].residue() < to; ++j)
        if (bad(r[i], r[j])) return true;
      for (int64_t j = first; to > row && j < i && r[j].residue() < to - row; ++j)  // past the row's end
        if (bad(r[i], r[j])) return true;
    }
  }
  return false;
}

// The slices are planned for this many SMs whatever the device, so that the
// workspace's size does not depend on it.
constexpr int kPlanSms = 152;

// The attention's places of tokens are 32 bits, and its loads look ahead by up
// to a run of tiles: the largest capacity, so that none of them wraps.
constexpr int64_t kMostTokens = INT_MAX - 1023;

}  // namespace

extern "C" {

size_t topkp_beam_select_workspace_size(int64_t B, int64_t K, int64_t V, topkp_dtype dtype, int32_t n) {
  if (B <= 0 || K <= 0 || K > TOPKP_MAX_BEAMS || V <= 0 || V > TOPKP_MAX_V || n <= 0 || n > TOPKP_MAX_CANDIDATES ||
      !row_type(dtype))
    return 0;
  const BeamPlan p = plan_beam(B * K, V, esize(dtype), kPlanSms);
  return p.stat_bytes + p.unit_bytes + p.piece_bytes;
}

topkp_status topkp_beam_select(const void* logits, int64_t B, int64_t K, int64_t V, int64_t ld_logits,
                               topkp_dtype dtype, const float* scores, const uint8_t* finished, int32_t pad_token,
                               int32_t n, float* out_score, int32_t* out_parent, int32_t* out_token, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const char* fn = "topkp_beam_select";
  report_launches(0);
  if (!row_type(dtype)) return fail(TOPKP_ERR_PARAM_INVALID, "%s: unknown dtype %d", fn, (int)dtype);
  if (B < 0 || V < 1 || V > TOPKP_MAX_V)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: B=%lld V=%lld (V is 1 to %lld)", fn, (long long)B, (long long)V,
                (long long)TOPKP_MAX_V);
  if (K < 1 || K > TOPKP_MAX_BEAMS)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: %lld beams (1 to %d)", fn, (long long)K, TOPKP_MAX_BEAMS);
  if (n < 1 || n > TOPKP_MAX_CANDIDATES)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: %d candidates (1 to %d)", fn, (int)n, TOPKP_MAX_CANDIDATES);
  if (pad_token < 0 || pad_token >= V) return fail(TOPKP_ERR_PARAM_INVALID, "%s: pad_token %d outside [0, V)", fn, (int)pad_token);
  if (B == 0) return TOPKP_SUCCESS;
  if (!logits || !scores || !out_score || !out_parent || !out_token || !workspace)
    return fail(TOPKP_ERR_PARAM_NULLPTR, "%s: logits, scores, an output or the workspace is NULL", fn);
  if (ld_logits < V) return fail(TOPKP_ERR_PARAM_INVALID, "%s: row stride %lld below V=%lld", fn, (long long)ld_logits, (long long)V);
  const int es = esize(dtype);
  if ((uintptr_t)logits % es || (uintptr_t)scores % 4 || (uintptr_t)out_score % 4 || (uintptr_t)out_parent % 4 ||
      (uintptr_t)out_token % 4)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: a pointer is not aligned to its element size", fn);
  if (B > INT_MAX / TOPKP_MAX_BEAMS) return fail(TOPKP_ERR_PARAM_INVALID, "%s: B=%lld is too large", fn, (long long)B);
  const BeamPlan p = plan_beam(B * K, V, es, kPlanSms);
  if (B * K * p.slices > INT_MAX) return fail(TOPKP_ERR_PARAM_INVALID, "%s: B * K * V is too large", fn);
  const size_t need = p.stat_bytes + p.unit_bytes + p.piece_bytes;
  if ((uintptr_t)workspace % 256 || workspace_bytes < need)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: the workspace needs %zu bytes, 256-byte aligned", fn, need);
  const Range ins[3] = {{logits, (size_t)((B * K - 1) * ld_logits + V) * es}, {scores, (size_t)(B * K) * 4}, {finished, (size_t)(B * K)}};
  const Range outs[4] = {{out_score, (size_t)B * n * 4}, {out_parent, (size_t)B * n * 4}, {out_token, (size_t)B * n * 4}, {workspace, need}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 3; ++j)
      if (overlap(outs[i], ins[j])) return fail(TOPKP_ERR_PARAM_INVALID, "%s: an output or the workspace overlaps an input", fn);
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i], outs[j])) return fail(TOPKP_ERR_PARAM_INVALID, "%s: two outputs (or the workspace) overlap", fn);
  }
  int dev = 0;
  if (device_sms(&dev) <= 0) return fail(TOPKP_ERR_LAUNCH, "%s: no usable CUDA device", fn);
  BeamArgs a = {};
  a.x = logits;
  a.ldx = ld_logits;
  a.scores = scores;
  a.finished = finished;
  a.B = B;
  a.K = (int32_t)K;
  a.V = (int32_t)V;
  a.n = n;
  a.pad = pad_token;
  a.nv = p.nv;
  a.chunks = p.chunks;
  a.slices = p.slices;
  a.stat = reinterpret_cast<longlong2*>(workspace);
  a.units = reinterpret_cast<uint32_t*>((char*)workspace + p.stat_bytes);
  a.pieces = p.nv > 1 ? a.units + p.unit_bytes / sizeof(uint32_t) : a.units;
  a.unit_count = p.unit_count;
  a.out_score = out_score;
  a.out_parent = out_parent;
  a.out_token = out_token;
  return launched(fn, launch_beam(dtype, a, (cudaStream_t)stream), 2);
}

topkp_status topkp_beam_reorder(const topkp_state* states, int64_t count, int64_t B, int64_t K, const int32_t* parent,
                                const int32_t* lengths, void* stream) {
  const char* fn = "topkp_beam_reorder";
  report_launches(0);
  if (count < 0 || B < 0) return fail(TOPKP_ERR_PARAM_INVALID, "%s: negative count or B", fn);
  if (K < 1 || K > TOPKP_MAX_BEAMS)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: %lld beams (1 to %d)", fn, (long long)K, TOPKP_MAX_BEAMS);
  if (count == 0 || B == 0) return TOPKP_SUCCESS;
  if (B > 65535) return fail(TOPKP_ERR_PARAM_INVALID, "%s: B=%lld above 65535", fn, (long long)B);
  if (!states || !parent) return fail(TOPKP_ERR_PARAM_NULLPTR, "%s: states or parent is NULL", fn);
  if ((uintptr_t)parent % 4 || (uintptr_t)lengths % 4)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: a pointer is not aligned to its element size", fn);
  const Range index[2] = {{parent, (size_t)(B * K) * 4}, {lengths, (size_t)(B * K) * 4}};
  auto span = [&](const topkp_state& s, bool dst) -> Range {
    const int64_t row = dst ? s.dst_row_stride : s.src_row_stride, blk = dst ? s.dst_block_stride : s.src_block_stride;
    return {dst ? s.dst : s.src, (size_t)((B * K - 1) * row + (s.blocks - 1) * blk + s.entries * s.entry_bytes)};
  };
  for (int64_t i = 0; i < count; ++i) {
    const topkp_state& s = states[i];
    if (s.blocks < 0 || s.entries < 0 || s.entry_bytes < 0)
      return fail(TOPKP_ERR_PARAM_INVALID, "%s: state %lld has a negative size", fn, (long long)i);
    if (s.blocks == 0 || s.entries == 0 || s.entry_bytes == 0) continue;
    if (!s.src || !s.dst) return fail(TOPKP_ERR_PARAM_NULLPTR, "%s: state %lld has a NULL pointer", fn, (long long)i);
    const int64_t block = s.entries * s.entry_bytes;
    if ((s.blocks > 1 && (s.src_block_stride < block || s.dst_block_stride < block)) ||
        s.src_row_stride < (s.blocks - 1) * s.src_block_stride + block ||
        s.dst_row_stride < (s.blocks - 1) * s.dst_block_stride + block)
      return fail(TOPKP_ERR_PARAM_INVALID, "%s: state %lld has rows or blocks that overlap", fn, (long long)i);
    if (s.src == s.dst && (s.src_row_stride != s.dst_row_stride || (s.blocks > 1 && s.src_block_stride != s.dst_block_stride)))
      return fail(TOPKP_ERR_PARAM_INVALID, "%s: state %lld is in place with two layouts", fn, (long long)i);
  }
  Region few[64];
  Region* regions = few;
  if (count > 32) regions = count <= (int64_t)(SIZE_MAX / 2 / sizeof(Region)) ? (Region*)malloc((size_t)count * 2 * sizeof(Region)) : nullptr;
  if (!regions) return fail(TOPKP_ERR_PARAM_INVALID, "%s: no memory for %lld states", fn, (long long)count);
  int64_t n = 0;
  topkp_status st = TOPKP_SUCCESS;
  for (int64_t i = 0; i < count && !st; ++i) {
    const topkp_state& s = states[i];
    if (s.blocks == 0 || s.entries == 0 || s.entry_bytes == 0) continue;
    const Range d = span(s, true);
    if (overlap(d, index[0]) || overlap(d, index[1]))
      st = fail(TOPKP_ERR_PARAM_INVALID, "%s: state %lld overlaps parent or lengths", fn, (long long)i);
    const int64_t len = s.entries * s.entry_bytes;
    regions[n++] = {(uintptr_t)s.dst, s.dst_row_stride, s.dst_block_stride, s.blocks, len, (s.blocks - 1) * s.dst_block_stride + len, i, true};
    if (s.src != s.dst)
      regions[n++] = {(uintptr_t)s.src, s.src_row_stride, s.src_block_stride, s.blocks, len, (s.blocks - 1) * s.src_block_stride + len, i, false};
  }
  const Region *one, *other;
  if (!st && clash(regions, n, B * K, &one, &other)) {
    if (one->written && other->written)
      st = fail(TOPKP_ERR_PARAM_INVALID, "%s: states %lld and %lld are written to one place", fn, (long long)std::min(one->state, other->state),
                (long long)std::max(one->state, other->state));
    else
      st = fail(TOPKP_ERR_PARAM_INVALID, "%s: state %lld is written over state %lld", fn, (long long)(one->written ? one : other)->state,
                (long long)(one->written ? other : one)->state);
  }
  if (regions != few) free(regions);
  if (st) return st;
  int dev = 0;
  if (device_sms(&dev) <= 0) return fail(TOPKP_ERR_LAUNCH, "%s: no usable CUDA device", fn);
  int launches = 0;
  // states of one unit travel together
  for (const int unit : {16, 4, 1}) {
    ReorderArgs a;
    a.parent = parent;
    a.lengths = lengths;
    a.B = B;
    a.K = (int32_t)K;
    a.unit = unit;
    a.count = 0;
    int64_t widest = 0;
    for (int64_t i = 0; i <= count; ++i) {
      if (i < count) {
        const topkp_state& s = states[i];
        if (s.blocks == 0 || s.entries == 0 || s.entry_bytes == 0) continue;
        uint64_t all = (uint64_t)(uintptr_t)s.src | (uint64_t)(uintptr_t)s.dst | (uint64_t)s.src_row_stride |
                       (uint64_t)s.dst_row_stride | (uint64_t)s.entry_bytes;
        if (s.blocks > 1) all |= (uint64_t)s.src_block_stride | (uint64_t)s.dst_block_stride;
        int own = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
        if (own == 16 && K > 32) own = 4;
        if (own != unit) continue;
        a.st[a.count++] = s;
        const int64_t bytes = s.blocks * s.entries * s.entry_bytes;
        widest = bytes > widest ? bytes : widest;
      }
      if (a.count == kReorderStates || (i == count && a.count)) {
        a.chunks = reorder_chunks(widest / unit, B * a.count);
        const cudaError_t e = launch_reorder(a, (cudaStream_t)stream);
        if (e != cudaSuccess) return launched(fn, e, 0);
        ++launches;
        a.count = 0;
        widest = 0;
      }
    }
  }
  return launched(fn, cudaSuccess, launches);
}

}  // extern "C"

namespace {

// What both cache calls check of a descriptor.
topkp_status check_cache(const char* fn, const char* name, const topkp_cache* c, int64_t H, int64_t D, int64_t pages,
                         int64_t page_size, int row_dtype) {
  if (!c->data) return fail(TOPKP_ERR_PARAM_NULLPTR, "%s: %s has no data", fn, name);
  if (c->dtype != row_dtype && c->dtype != TOPKP_E4M3)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: %s has dtype %d; the rows' own or e4m3 is wanted", fn, name, (int)c->dtype);
  if (c->dtype == TOPKP_E4M3 && !c->exponents)
    return fail(TOPKP_ERR_PARAM_NULLPTR, "%s: %s is e4m3 and has no exponents", fn, name);
  if (c->dtype != TOPKP_E4M3 && c->exponents)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: %s has exponents and is not e4m3", fn, name);
  if ((uintptr_t)c->data % esize(c->dtype)) return fail(TOPKP_ERR_PARAM_INVALID, "%s: %s is not aligned to its element size", fn, name);
  if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0 || c->exp_page_stride < 0 ||
      c->exp_token_stride < 0 || c->exp_head_stride < 0)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: %s has a negative stride", fn, name);
  if ((H > 1 && c->head_stride < D) || (page_size > 1 && c->token_stride < D) || (pages > 1 && c->page_stride < D))
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: %s has a stride below D", fn, name);
  return TOPKP_SUCCESS;
}
Range cache_span(const topkp_cache& c, int64_t H, int64_t D, int64_t pages, int64_t page_size) {
  return {c.data, (size_t)((pages - 1) * c.page_stride + (page_size - 1) * c.token_stride + (H - 1) * c.head_stride + D) *
                      esize(c.dtype)};
}
Range exp_span(const topkp_cache& c, int64_t H, int64_t pages, int64_t page_size) {
  return {c.exponents,
          (size_t)((pages - 1) * c.exp_page_stride + (page_size - 1) * c.exp_token_stride + (H - 1) * c.exp_head_stride + 1)};
}
// Whether a cache may be read and written 8 elements at a time.
bool cache_by_8(const topkp_cache& c) {
  const int64_t unit = c.dtype == TOPKP_E4M3 ? 8 : 16 / esize(c.dtype);
  return (uintptr_t)c.data % (unit * esize(c.dtype)) == 0 && c.page_stride % unit == 0 && c.token_stride % unit == 0 &&
         c.head_stride % unit == 0;
}
// Whether every stride (in bytes) that a row's place is multiplied with has 32 bits.
bool strides_32(const topkp_cache& c) {
  const int64_t most = 0xffffffffll / esize(c.dtype);
  return c.page_stride <= most && c.token_stride <= most && c.exp_page_stride <= most && c.exp_token_stride <= most;
}

topkp_status cache_shapes(const char* fn, int64_t N, int64_t H, int64_t D, int64_t pages, int64_t page_size, int dtype) {
  if (!row_type(dtype)) return fail(TOPKP_ERR_PARAM_INVALID, "%s: unknown dtype %d", fn, dtype);
  if (N < 0 || H < 0 || H > INT_MAX) return fail(TOPKP_ERR_PARAM_INVALID, "%s: N=%lld H=%lld", fn, (long long)N, (long long)H);
  if (D < 1 || D > TOPKP_MAX_HEAD_DIM)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: head dimension %lld (1 to %d)", fn, (long long)D, TOPKP_MAX_HEAD_DIM);
  if (pages < 1 || page_size < 1 || page_size > INT_MAX || pages > INT_MAX)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: pages=%lld page_size=%lld", fn, (long long)pages, (long long)page_size);
  if (H > 65535LL * 4 || N > INT_MAX) return fail(TOPKP_ERR_PARAM_INVALID, "%s: N * H is too large", fn);
  return TOPKP_SUCCESS;
}

}  // namespace

extern "C" {

topkp_status topkp_cache_write(const void* k, const void* v, int64_t N, int64_t H, int64_t D, int64_t k_token_stride,
                               int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                               topkp_dtype dtype, const int64_t* slots, const topkp_cache* k_cache,
                               const topkp_cache* v_cache, int64_t pages, int64_t page_size, void* stream) {
  const char* fn = "topkp_cache_write";
  report_launches(0);
  topkp_status st = cache_shapes(fn, N, H, D, pages, page_size, dtype);
  if (st) return st;
  if (N == 0 || H == 0) return TOPKP_SUCCESS;
  if (!k || !slots || !k_cache) return fail(TOPKP_ERR_PARAM_NULLPTR, "%s: k, slots or k_cache is NULL", fn);
  if (!v != !v_cache) return fail(TOPKP_ERR_PARAM_NULLPTR, "%s: v and v_cache go together", fn);
  CacheRowsArgs a = {};
  a.sides = v ? 2 : 1;
  const void* in[2] = {k, v};
  const topkp_cache* cs[2] = {k_cache, v_cache};
  const int64_t ts[2] = {k_token_stride, v_token_stride}, hs[2] = {k_head_stride, v_head_stride};
  const int es = esize(dtype);
  bool by8 = D % 8 == 0;
  if ((uintptr_t)slots % 8) return fail(TOPKP_ERR_PARAM_INVALID, "%s: slots is not aligned to its element size", fn);
  Range spans[2][3] = {};
  for (int i = 0; i < a.sides; ++i) {
    st = check_cache(fn, i ? "v_cache" : "k_cache", cs[i], H, D, pages, page_size, dtype);
    if (st) return st;
    if ((uintptr_t)in[i] % es || ts[i] < 0 || hs[i] < 0)
      return fail(TOPKP_ERR_PARAM_INVALID, "%s: %s is not aligned to its element size or has a negative stride", fn, i ? "v" : "k");
    by8 = by8 && cache_by_8(*cs[i]) && strides_32(*cs[i]) && ts[i] <= 0xffffffffll / es && ((uintptr_t)in[i] | (uint64_t)ts[i] * es | (uint64_t)hs[i] * es) % 16 == 0;
    a.in[i] = in[i];
    a.cache[i] = *cs[i];
    a.token_stride[i] = ts[i];
    a.head_stride[i] = hs[i];
    spans[i][0] = {in[i], (size_t)((N - 1) * ts[i] + (H - 1) * hs[i] + D) * es};
    spans[i][1] = cache_span(*cs[i], H, D, pages, page_size);
    spans[i][2] = exp_span(*cs[i], H, pages, page_size);
  }
  if (a.sides == 2 && k_cache->dtype != v_cache->dtype)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: the caches have two dtypes", fn);
  // the two caches may share an allocation (interleaved by their strides), so only the rows are held apart from them
  for (int i = 0; i < a.sides; ++i)
    for (int j = 0; j < a.sides; ++j)
      for (int w = 1; w < 3; ++w)
        if (overlap(spans[i][0], spans[j][w]) || overlap({slots, (size_t)N * 8}, spans[j][w]))
          return fail(TOPKP_ERR_PARAM_INVALID, "%s: a cache overlaps the rows or the slots", fn);
  int dev = 0;
  if (device_sms(&dev) <= 0) return fail(TOPKP_ERR_LAUNCH, "%s: no usable CUDA device", fn);
  a.slots = slots;
  a.N = N;
  a.slots_end = pages * page_size;
  a.H = (int32_t)H;
  a.D = (int32_t)D;
  a.page_size = (int32_t)page_size;
  a.vec = by8 ? 8 : 1;
  return launched(fn, launch_cache_write(dtype, a, (cudaStream_t)stream), 1);
}

topkp_status topkp_cache_read(const int64_t* slots, int64_t N, int64_t H, int64_t D, const topkp_cache* k_cache,
                              const topkp_cache* v_cache, int64_t pages, int64_t page_size, topkp_dtype dtype, void* k,
                              void* v, void* stream) {
  const char* fn = "topkp_cache_read";
  report_launches(0);
  topkp_status st = cache_shapes(fn, N, H, D, pages, page_size, dtype);
  if (st) return st;
  if (N == 0 || H == 0) return TOPKP_SUCCESS;
  if (!k || !slots || !k_cache) return fail(TOPKP_ERR_PARAM_NULLPTR, "%s: k, slots or k_cache is NULL", fn);
  if (!v != !v_cache) return fail(TOPKP_ERR_PARAM_NULLPTR, "%s: v and v_cache go together", fn);
  CacheRowsArgs a = {};
  a.sides = v ? 2 : 1;
  void* out[2] = {k, v};
  const topkp_cache* cs[2] = {k_cache, v_cache};
  const int es = esize(dtype);
  bool by8 = D % 8 == 0;
  if ((uintptr_t)slots % 8) return fail(TOPKP_ERR_PARAM_INVALID, "%s: slots is not aligned to its element size", fn);
  const size_t bytes = (size_t)(N * H * D) * es;
  for (int i = 0; i < a.sides; ++i) {
    st = check_cache(fn, i ? "v_cache" : "k_cache", cs[i], H, D, pages, page_size, dtype);
    if (st) return st;
    if ((uintptr_t)out[i] % es) return fail(TOPKP_ERR_PARAM_INVALID, "%s: an output is not aligned to its element size", fn);
    by8 = by8 && cache_by_8(*cs[i]) && strides_32(*cs[i]) && H * D <= 0xffffffffll / es && (uintptr_t)out[i] % 16 == 0;
    a.out[i] = out[i];
    a.cache[i] = *cs[i];
    a.token_stride[i] = H * D;
    a.head_stride[i] = D;
  }
  if (a.sides == 2 && k_cache->dtype != v_cache->dtype)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: the caches have two dtypes", fn);
  if (overlap({k, bytes}, {v, v ? bytes : 0})) return fail(TOPKP_ERR_PARAM_INVALID, "%s: the outputs overlap", fn);
  for (int i = 0; i < a.sides; ++i) {
    const Range o = {out[i], bytes};
    if (overlap(o, {slots, (size_t)N * 8})) return fail(TOPKP_ERR_PARAM_INVALID, "%s: an output overlaps the slots", fn);
    for (int j = 0; j < a.sides; ++j)
      if (overlap(o, cache_span(*cs[j], H, D, pages, page_size)) || overlap(o, exp_span(*cs[j], H, pages, page_size)))
        return fail(TOPKP_ERR_PARAM_INVALID, "%s: an output overlaps a cache", fn);
  }
  int dev = 0;
  if (device_sms(&dev) <= 0) return fail(TOPKP_ERR_LAUNCH, "%s: no usable CUDA device", fn);
  a.slots = slots;
  a.N = N;
  a.slots_end = pages * page_size;
  a.H = (int32_t)H;
  a.D = (int32_t)D;
  a.page_size = (int32_t)page_size;
  a.vec = by8 ? 8 : 1;
  return launched(fn, launch_cache_read(dtype, a, (cudaStream_t)stream), 1);
}

size_t topkp_tree_attention_workspace_size(const topkp_tree_attention_args* args) {
  if (!args || args->B <= 0 || args->T <= 0 || args->Hkv <= 0 || args->Hq < args->Hkv || args->D <= 0 ||
      args->max_pages <= 0 || args->page_size <= 0)
    return 0;
  return plan_attention(*args, kPlanSms).part_bytes;
}

topkp_status topkp_tree_attention(const topkp_tree_attention_args* args, void* stream) {
  const char* fn = "topkp_tree_attention";
  report_launches(0);
  if (!args) return fail(TOPKP_ERR_PARAM_NULLPTR, "%s: args is NULL", fn);
  const topkp_tree_attention_args& a = *args;
  if (a.dtype != TOPKP_F16 && a.dtype != TOPKP_BF16)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: dtype %d (fp16 or bf16 is wanted)", fn, (int)a.dtype);
  if (a.B < 0 || a.T < 0 || a.Hkv < 1 || a.Hq < 1 || a.Hq % a.Hkv)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: B=%lld T=%lld Hq=%lld Hkv=%lld (Hq a multiple of Hkv)", fn, (long long)a.B,
                (long long)a.T, (long long)a.Hq, (long long)a.Hkv);
  if (a.D < 8 || a.D > TOPKP_MAX_HEAD_DIM || a.D % 8)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: head dimension %lld (a multiple of 8 up to %d)", fn, (long long)a.D, TOPKP_MAX_HEAD_DIM);
  if (a.tree && a.T > TOPKP_MAX_TREE)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: a tree of %lld nodes (up to %d)", fn, (long long)a.T, TOPKP_MAX_TREE);
  if (a.B == 0 || a.T == 0) return TOPKP_SUCCESS;
  if (a.pages < 1 || a.page_size < 1 || a.max_pages < 1 || a.pages > INT_MAX || a.page_size > INT_MAX ||
      a.max_pages > kMostTokens / a.page_size || (a.table && a.ld_table < a.max_pages) ||
      (!a.table && (a.max_pages != 1 || a.pages != a.B)))
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: pages=%lld page_size=%lld max_pages=%lld ld_table=%lld", fn, (long long)a.pages,
                (long long)a.page_size, (long long)a.max_pages, (long long)a.ld_table);
  if (!a.q || !a.out || !a.context) return fail(TOPKP_ERR_PARAM_NULLPTR, "%s: q, out or context is NULL", fn);
  if (a.B * a.Hkv > 65535 || a.T * (a.Hq / a.Hkv) > 65535LL * 16 || a.Hq > INT_MAX || a.T > INT_MAX)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: B * Hkv above 65535, or too many rows", fn);
  topkp_status st = check_cache(fn, "k", &a.k, a.Hkv, a.D, a.pages, a.page_size, a.dtype);
  if (!st) st = check_cache(fn, "v", &a.v, a.Hkv, a.D, a.pages, a.page_size, a.dtype);
  if (st) return st;
  if (a.k.dtype != a.v.dtype) return fail(TOPKP_ERR_PARAM_INVALID, "%s: the caches have two dtypes", fn);
  for (const topkp_cache* c : {&a.k, &a.v})
    if (c->exponents && ((a.pages > 1 && c->exp_page_stride > UINT32_MAX) || (a.page_size > 1 && c->exp_token_stride > UINT32_MAX)))
      return fail(TOPKP_ERR_PARAM_INVALID, "%s: a stride of exponents has more than 32 bits", fn);
  if (!cache_by_8(a.k) || !cache_by_8(a.v))
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: a cache's pointer or strides are not multiples of 8 elements", fn);
  for (const int64_t s : {a.q_batch_stride, a.q_token_stride, a.q_head_stride, a.out_batch_stride, a.out_token_stride, a.out_head_stride})
    if (s < 0 || s % 8) return fail(TOPKP_ERR_PARAM_INVALID, "%s: a stride of q or out is not a multiple of 8", fn);
  if ((uintptr_t)a.q % 16 || (uintptr_t)a.out % 16 || (uintptr_t)a.lse % 4 || (uintptr_t)a.table % 4 ||
      (uintptr_t)a.context % 4 || (uintptr_t)a.nodes % 4 || (uintptr_t)a.tree % 8)
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: a pointer is not aligned (q and out to 16 bytes, others to their element)", fn);
  if ((a.B > 1 && a.out_batch_stride < a.D) || (a.T > 1 && a.out_token_stride < a.D) || (a.Hq > 1 && a.out_head_stride < a.D))
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: a stride of out is below D", fn);
  const AttnPlan p = plan_attention(a, kPlanSms);
  if (p.part_bytes && (!a.workspace || (uintptr_t)a.workspace % 256 || a.workspace_bytes < p.part_bytes))
    return fail(TOPKP_ERR_PARAM_INVALID, "%s: the workspace needs %zu bytes, 256-byte aligned", fn, p.part_bytes);
  const Range ins[9] = {
      {a.q, (size_t)((a.B - 1) * a.q_batch_stride + (a.T - 1) * a.q_token_stride + (a.Hq - 1) * a.q_head_stride + a.D) * 2},
      cache_span(a.k, a.Hkv, a.D, a.pages, a.page_size),
      cache_span(a.v, a.Hkv, a.D, a.pages, a.page_size),
      exp_span(a.k, a.Hkv, a.pages, a.page_size),
      exp_span(a.v, a.Hkv, a.pages, a.page_size),
      {a.context, (size_t)a.B * 4},
      {a.table, (size_t)((a.B - 1) * a.ld_table + a.max_pages) * 4},
      {a.tree, (size_t)(a.B * a.T) * 8},
      {a.nodes, (size_t)a.B * 4}};
  const Range outs[3] = {
      {a.out, (size_t)((a.B - 1) * a.out_batch_stride + (a.T - 1) * a.out_token_stride + (a.Hq - 1) * a.out_head_stride + a.D) * 2},
      {a.lse, (size_t)(a.B * a.T * a.Hq) * 4},
      {a.workspace, p.part_bytes}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 9; ++j)
      if (overlap(outs[i], ins[j])) return fail(TOPKP_ERR_PARAM_INVALID, "%s: an output or the workspace overlaps an input", fn);
    for (int j = i + 1; j < 3; ++j)
      if (overlap(outs[i], outs[j])) return fail(TOPKP_ERR_PARAM_INVALID, "%s: two outputs (or the workspace) overlap", fn);
  }
  int dev = 0;
  if (device_sms(&dev) <= 0) return fail(TOPKP_ERR_LAUNCH, "%s: no usable CUDA device", fn);
  int launches = 0;
  const cudaError_t e = launch_attention(a, p, &launches, (cudaStream_t)stream);
  return launched(fn, e, launches);
}

}  // extern "C"
