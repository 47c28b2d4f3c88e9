// Host entry points of include/serving/rhtq_serving.h: argument checks, workspace sizes, launches.
// Every check happens before the first HIP call, so a rejected call enqueues nothing.
#include <stdint.h>

#include <climits>

#include "rhtq_internal.h"
#include "rhtq_paging.h"
#include "rhtq_serving_internal.h"

namespace {

bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int from_hip(hipError_t e) { return e == hipSuccess ? RHTQ_OK : RHTQ_EHIP; }
int log2_of(int32_t v) { return 31 - __builtin_clz((unsigned)v); }
bool in_type(int t) { return t == RHTQ_IN_BF16 || t == RHTQ_IN_F16 || t == RHTQ_IN_F32; }
constexpr int64_t kMostTokens = 1 << 20;
constexpr int64_t kMostQueries = ((int64_t)1 << 26) - 64;   // heads of all sequences: a join's 64 threads each stay below 2^32
int64_t round16(int64_t v) { return (v + 15) & ~(int64_t)15; }
uintptr_t scale_size(int t) { return t == RHTQ_SCALE_F32 ? 4 : (t == RHTQ_SCALE_F16 ? 2 : 1); }

// Shape of a cache, without its pointers: RHTQ_OK or the status.
int check_cache(const rhtq_cache_t* c) {
  if (!c) return RHTQ_EINVAL;
  if (c->layers < 1 || c->pages < 0 || c->kv_heads < 1) return RHTQ_EINVAL;
  if (c->scale_dtype != RHTQ_SCALE_F32 && c->scale_dtype != RHTQ_SCALE_F16) return RHTQ_EUNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return RHTQ_EUNSUPPORTED;
  if (!is_pow2(c->page) || c->page < 16 || c->page > 256) return RHTQ_EUNSUPPORTED;
  return RHTQ_OK;
}

int check_table(int32_t width, int32_t seqs, int32_t page) {
  if (width < 0 || seqs < 0) return RHTQ_EINVAL;
  // positions and the tiles beyond them stay 32-bit numbers
  if ((int64_t)width * page > INT32_MAX - 256) return RHTQ_EINVAL;
  return RHTQ_OK;
}

bool cache_pointers(const rhtq_cache_t* c, uintptr_t scale_alignment) {
  return c->k_codes && c->v_codes && c->k_scales && c->v_scales && aligned(c->k_codes, 16) && aligned(c->v_codes, 16) &&
         aligned(c->k_scales, scale_alignment) && aligned(c->v_scales, scale_alignment);
}

int cache_rows(const rhtq_cache_t* c, int64_t tokens, const int32_t* table, int32_t width, const int32_t* lengths,
               const int32_t* starts, int32_t seqs, const int8_t* k_signs, const int8_t* v_signs, rhtq::CacheArgs& a) {
  int st = check_cache(c);
  if (st == RHTQ_OK) st = check_table(width, seqs, c->page);
  if (st != RHTQ_OK) return st;
  if (tokens < 0 || tokens > rhtq::kMostRows || (!starts && tokens != seqs) || c->layers != 1) return RHTQ_EINVAL;
  if (c->kv_heads > 65535) return RHTQ_EUNSUPPORTED;   // a grid's limit
  if (tokens == 0) return RHTQ_OK;
  if (c->pages > 0 && !cache_pointers(c, scale_size(c->scale_dtype))) return RHTQ_EINVAL;
  if (seqs > 0 && ((width > 0 && !table) || !lengths)) return RHTQ_EINVAL;
  if (!aligned(table, 4) || !aligned(lengths, 4) || !aligned(starts, 4) || !aligned(k_signs, 4) || !aligned(v_signs, 4))
    return RHTQ_EINVAL;
  a.tokens = tokens;
  a.codes[0] = c->k_codes;
  a.codes[1] = c->v_codes;
  a.scales[0] = c->k_scales;
  a.scales[1] = c->v_scales;
  a.signs[0] = k_signs;
  a.signs[1] = v_signs;
  a.table = table;
  a.lengths = lengths;
  a.starts = starts;
  a.seqs = seqs;
  a.width = width;
  a.pages = c->pages;
  a.kv_heads = c->kv_heads;
  a.page_log = log2_of(c->page);
  a.head_dim = c->head_dim;
  a.scale_dtype = c->scale_dtype;
  return RHTQ_OK;
}

// Fields every page call shares; RHTQ_OK or the status.
int page_args(int32_t* table, int32_t width, int32_t* lengths, int32_t seqs, int32_t* refs, int32_t pages, int32_t page,
              rhtq::PagesArgs& a) {
  if (pages < 0 || !is_pow2(page) || page < 16 || page > 256) return RHTQ_EINVAL;
  const int st = check_table(width, seqs, page);
  if (st != RHTQ_OK) return st;
  if (!aligned(table, 4) || !aligned(lengths, 4) || !aligned(refs, 4)) return RHTQ_EINVAL;
  a.table = table;
  a.width = width;
  a.lengths = lengths;
  a.seqs = seqs;
  a.refs = refs;
  a.pages = pages;
  a.page = page;
  return RHTQ_OK;
}

int page_data(const rhtq_cache_t* c, rhtq::PagesArgs& a) {
  const int st = check_cache(c);
  if (st != RHTQ_OK) return st;
  if (c->kv_heads > 65535) return RHTQ_EUNSUPPORTED;   // 16-byte words of a page's slots are counted in 32 bits
  if (c->pages > 0 && !cache_pointers(c, 16)) return RHTQ_EINVAL;
  a.data[0] = c->k_codes;
  a.data[1] = static_cast<uint8_t*>(c->k_scales);
  a.data[2] = c->v_codes;
  a.data[3] = static_cast<uint8_t*>(c->v_scales);
  a.row_bytes[0] = a.row_bytes[2] = c->head_dim / 2;
  a.row_bytes[1] = a.row_bytes[3] = (int32_t)scale_size(c->scale_dtype);
  a.layers = c->layers;
  a.kv_heads = c->kv_heads;
  a.pages = c->pages;
  a.page = c->page;
  return RHTQ_OK;
}

bool workspace_ok(const void* w, int64_t bytes, int64_t need) { return need == 0 || (w && aligned(w, 16) && bytes >= need); }

}  // namespace

extern "C" {

int rhtq_serving_version(void) { return RHTQ_SERVING_VERSION; }

// The operands of x, an exponent for each padded token, the sums of split k, and the rotated rows.
int64_t rhtq_matvec_workspace(int64_t tokens, int32_t n, int64_t rows) {
  if (tokens <= 0 || n <= 0 || rows <= 0 || tokens > kMostTokens || rows > rhtq::kMostWeightRows || n > (1 << 20)) return 0;
  const int64_t parts = rhtq::matvec_splits(tokens, n, rows);
  return rhtq::matvec_halves_bytes(tokens, n) + round16(4 * rhtq::matvec_padded(tokens)) +
         (parts > 1 ? round16(4 * parts * tokens * rows) : 0) + 4 * tokens * n;
}

int rhtq_matvec(const void* x, int in_dtype, int64_t tokens, int32_t n, int32_t block, const int8_t* signs, int rotated,
                const uint8_t* packed, const void* scales, const float* tensor_scale, int64_t rows, int fmt, int32_t group,
                int scale_dtype, void* y_out, int out_dtype, void* workspace, int64_t workspace_bytes,
                rhtq_stream_t stream) {
  if (!in_type(in_dtype) || !in_type(out_dtype) || tokens < 0 || rows < 0) return RHTQ_EINVAL;
  if (fmt != RHTQ_FMT_INT4 && fmt != RHTQ_FMT_NVFP4 && fmt != RHTQ_FMT_MXFP4) return RHTQ_EINVAL;
  if (n < 32 || n % 32 || n > (1 << 20)) return RHTQ_EUNSUPPORTED;
  if (fmt == RHTQ_FMT_INT4) {
    if (group != 0 && (!is_pow2(group) || group < 16 || n % group)) return RHTQ_EUNSUPPORTED;
    if (scale_dtype != RHTQ_SCALE_F32 && scale_dtype != RHTQ_SCALE_F16) return RHTQ_EUNSUPPORTED;
  } else if (fmt == RHTQ_FMT_NVFP4) {
    if (group != 16 || scale_dtype != RHTQ_SCALE_E4M3) return RHTQ_EUNSUPPORTED;
  } else if (group != 32 || scale_dtype != RHTQ_SCALE_E8M0) {
    return RHTQ_EUNSUPPORTED;
  }
  if (tokens > kMostTokens || rows > rhtq::kMostWeightRows) return RHTQ_EINVAL;
  if (!rotated) {
    // the rotation's own checks of n and block, with no rows: nothing is enqueued
    const int st = block == n ? rhtq_rotate(x, in_dtype, 0, n, signs, nullptr, stream)
                              : rhtq_rotate_blocked(x, in_dtype, 0, n, block, signs, nullptr, stream);
    if (st != RHTQ_OK) return st;
  }
  if (tokens == 0 || rows == 0) return RHTQ_OK;
  if (!x || !packed || !scales || !y_out || (fmt == RHTQ_FMT_NVFP4 && !tensor_scale)) return RHTQ_EINVAL;
  const uintptr_t scale_alignment = fmt == RHTQ_FMT_NVFP4 ? 2 : scale_size(scale_dtype);   // E4M3 bytes are loaded in pairs
  if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(y_out, 16) || !aligned(scales, scale_alignment) ||
      !aligned(tensor_scale, 4) || (!rotated && !aligned(signs, 16)))
    return RHTQ_EINVAL;
  if (!workspace_ok(workspace, workspace_bytes, rhtq_matvec_workspace(tokens, n, rows))) return RHTQ_EINVAL;
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  rhtq::MatvecArgs a{};
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.halves = w;
  w += rhtq::matvec_halves_bytes(tokens, n);
  a.exponents = reinterpret_cast<int32_t*>(w);
  w += round16(4 * rhtq::matvec_padded(tokens));
  a.k_splits = rhtq::matvec_splits(tokens, n, rows);
  a.partial = reinterpret_cast<float*>(w);
  if (a.k_splits > 1) w += round16(4 * (int64_t)a.k_splits * tokens * rows);
  a.x = x;
  if (!rotated) {
    float* y = reinterpret_cast<float*>(w);
    const int st = block == n ? rhtq_rotate(x, in_dtype, tokens, n, signs, y, stream)
                              : rhtq_rotate_blocked(x, in_dtype, tokens, n, block, signs, y, stream);
    if (st != RHTQ_OK) return st;
    a.x = y;
    in_dtype = RHTQ_IN_F32;
  }
  a.packed = packed;
  a.scales = scales;
  a.tensor_scale = fmt == RHTQ_FMT_NVFP4 ? tensor_scale : nullptr;
  a.y = y_out;
  a.tokens = tokens;
  a.rows = rows;
  a.n = n;
  a.groups = group ? n / group : 1;
  a.group_log = group ? log2_of(group) : -1;
  a.fmt = fmt;
  a.scale_dtype = scale_dtype;
  a.out_dtype = out_dtype;
  return from_hip(rhtq::launch_matvec(in_dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

int rhtq_cache_append(const rhtq_cache_t* cache, const void* k, const void* v, int in_dtype, int64_t tokens,
                      int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                      const int32_t* table, int32_t width, const int32_t* lengths, const int32_t* starts, int32_t seqs,
                      const int8_t* k_signs, const int8_t* v_signs, rhtq_stream_t stream) {
  if (!in_type(in_dtype)) return RHTQ_EINVAL;
  rhtq::CacheArgs a{};
  const int st = cache_rows(cache, tokens, table, width, lengths, starts, seqs, k_signs, v_signs, a);
  if (st != RHTQ_OK || tokens == 0) return st;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return RHTQ_EINVAL;
  const int64_t per16 = in_dtype == RHTQ_IN_F32 ? 4 : 8;   // elements in 16 bytes
  const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  for (int64_t x : strides)
    if (x < 0 || x % per16) return RHTQ_EINVAL;
  a.x[0] = k;
  a.x[1] = v;
  a.token_stride[0] = k_token_stride;
  a.token_stride[1] = v_token_stride;
  a.head_stride[0] = k_head_stride;
  a.head_stride[1] = v_head_stride;
  if (seqs == 0) return RHTQ_OK;   // no row belongs to a sequence
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  return from_hip(rhtq::launch_cache_append(in_dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

int rhtq_cache_read(const rhtq_cache_t* cache, void* k_out, void* v_out, int out_dtype, int64_t tokens,
                    const int32_t* table, int32_t width, const int32_t* lengths, const int32_t* starts, int32_t seqs,
                    const int8_t* k_signs, const int8_t* v_signs, rhtq_stream_t stream) {
  if (!in_type(out_dtype)) return RHTQ_EINVAL;
  rhtq::CacheArgs a{};
  const int st = cache_rows(cache, tokens, table, width, lengths, starts, seqs, k_signs, v_signs, a);
  if (st != RHTQ_OK || tokens == 0 || (!k_out && !v_out)) return st;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return RHTQ_EINVAL;
  a.y[0] = k_out;
  a.y[1] = v_out;
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  return from_hip(rhtq::launch_cache_read(out_dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

int64_t rhtq_paged_attention_workspace(int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t width,
                                       int32_t page, int32_t window, int32_t sinks) {
  if (seqs <= 0 || kv_heads <= 0 || q_heads < kv_heads || head_dim <= 0 || width < 0 || page <= 0 || window < 0 || sinks < 0) return 0;
  const int32_t splits = rhtq::attention_splits(seqs, q_heads, kv_heads, width, page, window, sinks);
  return splits == 1 ? 0 : (int64_t)seqs * q_heads * splits * (head_dim + 2) * 4;
}

int rhtq_paged_attention(const void* q, int in_dtype, int32_t seqs, int32_t q_heads, int64_t q_seq_stride,
                         int64_t q_head_stride, const rhtq_cache_t* cache, const int32_t* table, int32_t width,
                         const int32_t* lengths, const int8_t* k_signs, const int8_t* v_signs, float scale, int32_t window,
                         int32_t sinks, void* out, void* workspace, int64_t workspace_bytes, rhtq_stream_t stream) {
  if (in_dtype != RHTQ_IN_BF16 && in_dtype != RHTQ_IN_F16) return in_dtype == RHTQ_IN_F32 ? RHTQ_EUNSUPPORTED : RHTQ_EINVAL;
  int st = check_cache(cache);
  if (st == RHTQ_OK) st = check_table(width, seqs, cache->page);
  if (st != RHTQ_OK) return st;
  if (q_heads < 1 || cache->layers != 1 || window < 0 || sinks < 0 || !(scale - scale == 0.0f)) return RHTQ_EINVAL;
  if (q_heads % cache->kv_heads) return RHTQ_EUNSUPPORTED;
  if (q_seq_stride < 0 || q_head_stride < 0 || q_seq_stride % 8 || q_head_stride % 8) return RHTQ_EINVAL;
  if (seqs == 0) return RHTQ_OK;
  const int32_t splits = rhtq::attention_splits(seqs, q_heads, cache->kv_heads, width, cache->page, window, sinks);
  if (seqs > 65535 || (int64_t)cache->kv_heads * rhtq::attention_head_tiles(q_heads / cache->kv_heads) > 65535 ||
      (int64_t)seqs * q_heads * splits > INT32_MAX || (int64_t)seqs * q_heads > kMostQueries)
    return RHTQ_EUNSUPPORTED;   // a grid's limits
  if (!q || !out || !lengths || !aligned(q, 16) || !aligned(out, 16) || !aligned(lengths, 4) || !aligned(k_signs, 4) ||
      !aligned(v_signs, 4))
    return RHTQ_EINVAL;
  if (width > 0 && (!table || !aligned(table, 4))) return RHTQ_EINVAL;
  if (cache->pages > 0 && !cache_pointers(cache, 2 * scale_size(cache->scale_dtype))) return RHTQ_EINVAL;   // loaded in pairs
  const int64_t need =
      rhtq_paged_attention_workspace(seqs, q_heads, cache->kv_heads, cache->head_dim, width, cache->page, window, sinks);
  if (!workspace_ok(workspace, workspace_bytes, need)) return RHTQ_EINVAL;
  rhtq::AttentionArgs a{};
  a.q = q;
  a.q_seq_stride = q_seq_stride;
  a.q_head_stride = q_head_stride;
  a.out = out;
  a.partial = static_cast<float*>(workspace);
  a.k_codes = cache->k_codes;
  a.v_codes = cache->v_codes;
  a.k_scales = cache->k_scales;
  a.v_scales = cache->v_scales;
  a.k_signs = k_signs;
  a.v_signs = v_signs;
  a.table = table;
  a.lengths = lengths;
  a.seqs = seqs;
  a.q_heads = q_heads;
  a.kv_heads = cache->kv_heads;
  a.each = q_heads / cache->kv_heads;
  a.head_tiles = rhtq::attention_head_tiles(a.each);
  a.width = width;
  a.pages = cache->pages;
  a.page_log = log2_of(cache->page);
  a.head_dim = cache->head_dim;
  a.scale_dtype = cache->scale_dtype;
  a.window = window;
  a.sinks = sinks;
  a.splits = splits;
  a.scale = scale;
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  return from_hip(rhtq::launch_paged_attention(in_dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

// The largest of what the calls lay out: a fork's fresh pages, marks and three words a pair; a compaction's moves and places.
int64_t rhtq_pages_workspace(int32_t pages, int32_t seqs, int32_t count) {
  if (pages < 0 || seqs < 0 || count < 0) return 0;
  const int64_t fork = (int64_t)pages + seqs + 3 * (int64_t)count;
  const int64_t compact = 1 + 2 * ((int64_t)pages / 2 + 1) + pages;
  return 4 * (fork > compact ? fork : compact);
}

int rhtq_pages_reserve(int32_t* table, int32_t width, int32_t* lengths, int32_t seqs, int32_t* refs, int32_t pages,
                       int32_t page, const int32_t* add, int32_t* status, void* workspace, int64_t workspace_bytes,
                       rhtq_stream_t stream) {
  rhtq::PagesArgs a{};
  const int st = page_args(table, width, lengths, seqs, refs, pages, page, a);
  if (st != RHTQ_OK) return st;
  if (!status || !aligned(status, 4)) return RHTQ_EINVAL;
  if (pages > 0 && !refs) return RHTQ_EINVAL;      // free pages are counted whatever the sequences
  if (seqs > 0 && (!lengths || !add || !aligned(add, 4) || (width > 0 && !table))) return RHTQ_EINVAL;
  if (!workspace_ok(workspace, workspace_bytes, rhtq_pages_workspace(pages, seqs, 0))) return RHTQ_EINVAL;
  a.add = add;
  a.status = status;
  a.work = static_cast<int32_t*>(workspace);
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  return from_hip(rhtq::launch_pages_reserve(a, reinterpret_cast<hipStream_t>(stream)));
}

int rhtq_pages_free(int32_t* table, int32_t width, int32_t* lengths, int32_t seqs, int32_t* refs, int32_t pages,
                    const int32_t* list, int32_t count, rhtq_stream_t stream) {
  rhtq::PagesArgs a{};
  const int st = page_args(table, width, lengths, seqs, refs, pages, 16, a);
  if (st != RHTQ_OK) return st;
  if (count < 0) return RHTQ_EINVAL;
  if (count == 0 || seqs == 0) return RHTQ_OK;
  if (!list || !aligned(list, 4) || !lengths || (width > 0 && !table) || (pages > 0 && !refs)) return RHTQ_EINVAL;
  a.src = list;
  a.count = count;
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  return from_hip(rhtq::launch_pages_free(a, reinterpret_cast<hipStream_t>(stream)));
}

int rhtq_pages_trim(int32_t* table, int32_t width, const int32_t* lengths, int32_t seqs, int32_t* refs, int32_t pages,
                    int32_t page, int32_t window, int32_t sinks, rhtq_stream_t stream) {
  rhtq::PagesArgs a{};
  const int st = page_args(table, width, const_cast<int32_t*>(lengths), seqs, refs, pages, page, a);
  if (st != RHTQ_OK) return st;
  if (window < 1 || sinks < 0) return RHTQ_EINVAL;
  if (seqs == 0 || width == 0) return RHTQ_OK;
  if (!lengths || !table || (pages > 0 && !refs)) return RHTQ_EINVAL;
  a.window = window;
  a.sinks = sinks;
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  return from_hip(rhtq::launch_pages_trim(a, reinterpret_cast<hipStream_t>(stream)));
}

int rhtq_pages_fork(const rhtq_cache_t* cache, int32_t* table, int32_t width, int32_t* lengths, int32_t seqs, int32_t* refs,
                    const int32_t* src, const int32_t* dst, int32_t count, int32_t* status, void* workspace,
                    int64_t workspace_bytes, rhtq_stream_t stream) {
  rhtq::PagesArgs a{};
  int st = page_data(cache, a);
  if (st == RHTQ_OK) st = page_args(table, width, lengths, seqs, refs, a.pages, a.page, a);
  if (st != RHTQ_OK) return st;
  if (count < 0 || !status || !aligned(status, 4)) return RHTQ_EINVAL;
  if (count > 0 && (!src || !dst || !aligned(src, 4) || !aligned(dst, 4))) return RHTQ_EINVAL;
  if (a.pages > 0 && !refs) return RHTQ_EINVAL;
  if (seqs > 0 && (!lengths || (width > 0 && !table))) return RHTQ_EINVAL;
  if (!workspace_ok(workspace, workspace_bytes, rhtq_pages_workspace(a.pages, seqs, count))) return RHTQ_EINVAL;
  a.src = src;
  a.dst = dst;
  a.count = count;
  a.status = status;
  a.work = static_cast<int32_t*>(workspace);
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  return from_hip(rhtq::launch_pages_fork(a, reinterpret_cast<hipStream_t>(stream)));
}

int rhtq_pages_copy(const rhtq_cache_t* cache, const int32_t* src, const int32_t* dst, int32_t count, rhtq_stream_t stream) {
  rhtq::PagesArgs a{};
  const int st = page_data(cache, a);
  if (st != RHTQ_OK) return st;
  if (count < 0) return RHTQ_EINVAL;
  if (count == 0) return RHTQ_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return RHTQ_EINVAL;
  a.src = src;
  a.dst = dst;
  a.count = count;
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  return from_hip(rhtq::launch_pages_copy(a, reinterpret_cast<hipStream_t>(stream)));
}

int rhtq_pages_compact(const rhtq_cache_t* cache, int32_t* table, int32_t width, int32_t seqs, int32_t* refs, int32_t* live,
                       void* workspace, int64_t workspace_bytes, rhtq_stream_t stream) {
  rhtq::PagesArgs a{};
  int st = page_data(cache, a);
  if (st == RHTQ_OK) st = page_args(table, width, nullptr, seqs, refs, a.pages, a.page, a);
  if (st != RHTQ_OK) return st;
  if (!live || !aligned(live, 4)) return RHTQ_EINVAL;
  if (seqs > 0 && width > 0 && !table) return RHTQ_EINVAL;
  if (a.pages > 0 && !refs) return RHTQ_EINVAL;
  if (!workspace_ok(workspace, workspace_bytes, rhtq_pages_workspace(a.pages, seqs, 0))) return RHTQ_EINVAL;
  a.status = live;
  a.work = static_cast<int32_t*>(workspace);
  if (rhtq::getenv_test_fail_launch()) return RHTQ_EHIP;
  return from_hip(rhtq::launch_pages_compact(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
