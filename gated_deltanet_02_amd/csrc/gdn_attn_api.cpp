// C ABI of the attention over a paged key-value cache (declared in
// include/gdn.h): block tables and slot maps, the store of new rows, and the
// attention of prompts and of single tokens.  Host side only: every argument
// is validated before any HIP call, then the kernels are enqueued on the
// caller's stream.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gdn.h"
#include "gdn_api_check.h"
#include "gdn_api_common.h"
#include "gdn_attn.h"

using namespace gdn;

namespace {

constexpr int64_t kMaxThreads = (int64_t)1 << 32;  // of one launch
constexpr size_t kAlign = 256;
constexpr int64_t kMaxRequests = (int64_t)1 << 20;
constexpr int64_t kMaxRowStride = (int64_t)1 << 24;  // keys' and values': 32-bit offsets inside a tile

bool attn_dim(int64_t d) { return d == 64 || d == 128 || d == 256; }

// A 1-D integer array of n values.
int check_ints(const gdn_tensor* t, const char* name, int64_t n, int32_t dtype = GDN_DTYPE_I32) {
  if (t->dtype != dtype)
    return api_fail(GDN_ERR_DTYPE, "%s must be %s", name, dtype == GDN_DTYPE_I32 ? "int32" : "int64");
  int rc;
  if ((rc = check_tensor(t, name, 1, 1))) return rc;
  if (n >= 0 && t->shape[0] != n) return api_fail(GDN_ERR_SHAPE, "%s must have %lld entries", name, (long long)n);
  return GDN_OK;
}

// A block table [n, width].
int check_table(const gdn_tensor* t, int64_t n) {
  if (t->dtype != GDN_DTYPE_I32) return api_fail(GDN_ERR_DTYPE, "block_table must be int32");
  int rc;
  if ((rc = check_tensor(t, "block_table", 2, 2))) return rc;
  if (t->shape[0] != n)
    return api_fail(GDN_ERR_SHAPE, "block_table must have a row for each of %lld requests", (long long)n);
  return GDN_OK;
}

int check_page(int64_t page, int64_t width) {
  if (page < 1 || page > kMaxCount) return api_fail(GDN_ERR_SHAPE, "page_size must be 1 .. 2^31 - 2^21");
  if ((__int128)page * width > kMaxCount)
    return api_fail(GDN_ERR_SHAPE, "a block table's row holds at most 2^31 - 2^21 tokens");
  return GDN_OK;
}

// Rows [.., heads, d] that 16-byte accesses fit: every stride that is taken.
int check_granules(const gdn_tensor* t, const char* name) {
  if (is_empty(t)) return GDN_OK;
  if (!aligned16(t->data)) return api_fail(GDN_ERR_LAYOUT, "%s must be 16-byte aligned", name);
  const int64_t epg = 16 / element_size(t->dtype);
  for (int i = 0; i + 1 < t->ndim; ++i)
    if (t->shape[i] > 1 && t->stride[i] % epg)
      return api_fail(GDN_ERR_LAYOUT, "%s: strides must be multiples of %lld elements", name, (long long)epg);
  return GDN_OK;
}

// Two outputs, or one output's own elements: no place twice.  Two arrays of
// the same shape and strides may interleave (the halves of one allocation).
int check_distinct(const gdn_tensor* a, const char* name) {
  if (!is_empty(a) && !distinct(a->shape, a->stride, a->ndim))
    return api_fail(GDN_ERR_LAYOUT, "%s: rows overlap", name);
  return GDN_OK;
}

bool interleaved(const gdn_tensor* a, const gdn_tensor* b) {
  if (a->ndim != b->ndim || a->dtype != b->dtype) return false;
  int64_t shape[5], stride[5];
  for (int i = 0; i < a->ndim; ++i) {
    if (a->shape[i] != b->shape[i] || (a->shape[i] > 1 && a->stride[i] != b->stride[i])) return false;
    shape[i] = a->shape[i];
    stride[i] = a->stride[i];
  }
  const uintptr_t lo = std::min((uintptr_t)a->data, (uintptr_t)b->data);
  const uintptr_t hi = std::max((uintptr_t)a->data, (uintptr_t)b->data);
  const int64_t es = element_size(a->dtype);
  if ((hi - lo) % (uintptr_t)es) return false;
  shape[a->ndim] = 2;
  stride[a->ndim] = (int64_t)((hi - lo) / (uintptr_t)es);
  return distinct(shape, stride, a->ndim + 1);
}

int attn_options(const gdn_attn_options* opts, gdn_attn_options* o) {
  gdn_attn_default_options(o);
  if (opts) *o = *opts;
  if (!(std::fabs(o->scale) <= 0x1p64f)) return api_fail(GDN_ERR_SHAPE, "scale must be within +-2^64");
  if (o->window < 0) return api_fail(GDN_ERR_SHAPE, "window must be >= 0 (got %d)", o->window);
  if (o->sinks < 0) return api_fail(GDN_ERR_SHAPE, "sinks must be >= 0 (got %d)", o->sinks);
  return GDN_OK;
}

// What prompts and single tokens have in common once q's rank is known.
struct Attn {
  int64_t T = 0, H = 0, K = 0, D = 0;
  int64_t pages = 0, page = 0, width = 0;
  gdn_attn_options opts;
};

// Caches [pages, page, kv, d] with a block table of n rows and lengths.
int parse_caches(const gdn_tensor* k, const gdn_tensor* v, const gdn_tensor* table, const gdn_tensor* lens, int64_t n,
                 Attn* A) {
  int rc;
  if ((rc = check_tensor(k, "k", 4, 4)) || (rc = check_tensor(v, "v", 4, 4))) return rc;
  A->pages = k->shape[0];
  A->page = k->shape[1];
  A->K = k->shape[2];
  if (k->shape[3] != A->D) return api_fail(GDN_ERR_SHAPE, "the caches' d differs from q's");
  if ((rc = check_table(table, n)) || (rc = check_ints(lens, "seq_lens", n))) return rc;
  A->width = table->shape[1];
  return check_page(A->page, A->width);
}

int check_heads(const Attn& A, const gdn_tensor* q, const gdn_tensor* k, const gdn_tensor* v, const gdn_tensor* out) {
  if (k->ndim != v->ndim) return api_fail(GDN_ERR_SHAPE, "k and v must have one shape");
  for (int i = 0; i < k->ndim; ++i)
    if (k->shape[i] != v->shape[i]) return api_fail(GDN_ERR_SHAPE, "k and v must have one shape");
  if (A.H < 1 || A.K < 1 || A.H % A.K)
    return api_fail(GDN_ERR_SHAPE, "query heads (%lld) must be a positive multiple of key heads (%lld)", (long long)A.H,
                    (long long)A.K);
  if (A.H > 65535) return api_fail(GDN_ERR_UNSUPPORTED, "at most 65535 heads");
  const int row = k->ndim - 3;
  if (!is_empty(k) && k->shape[row] > 1 && std::max(k->stride[row], v->stride[row]) > kMaxRowStride)
    return api_fail(GDN_ERR_LAYOUT, "tokens of k and v lie at most 2^24 elements apart");
  int rc;
  if ((rc = check_granules(q, "q")) || (rc = check_granules(k, "k")) || (rc = check_granules(v, "v")) ||
      (rc = check_granules(out, "out")))
    return rc;
  return check_distinct(out, "out");
}

int check_types(const gdn_tensor* q, const gdn_tensor* k, const gdn_tensor* v, const gdn_tensor* out) {
  if (!is_float(q->dtype)) return api_fail(GDN_ERR_DTYPE, "q must be bf16 or f32");
  if (k->dtype != q->dtype || v->dtype != q->dtype || out->dtype != q->dtype)
    return api_fail(GDN_ERR_DTYPE, "q, k, v and out must share one dtype");
  return GDN_OK;
}

// out must match q, of a rank between lo and hi.
int check_rows_of(const gdn_tensor* q, const gdn_tensor* out, int lo, int hi) {
  int rc;
  if ((rc = check_tensor(q, "q", lo, hi)) || (rc = check_tensor(out, "out", lo, hi))) return rc;
  if (out->ndim != q->ndim) return api_fail(GDN_ERR_SHAPE, "out must match q");
  for (int i = 0; i < q->ndim; ++i)
    if (out->shape[i] != q->shape[i]) return api_fail(GDN_ERR_SHAPE, "out must match q");
  const int64_t d = q->shape[q->ndim - 1];
  if (!attn_dim(d)) return api_fail(GDN_ERR_UNSUPPORTED, "d must be 64, 128 or 256 (got %lld)", (long long)d);
  return GDN_OK;
}

// The bytes of a stride that is taken, else 0 (of one row it may be anything).
int64_t step(const gdn_tensor* t, int i) {
  return !is_empty(t) && t->shape[i] > 1 ? t->stride[i] * element_size(t->dtype) : 0;
}

void fill(const Attn& A, const gdn_tensor* q, const gdn_tensor* k, const gdn_tensor* v, const gdn_tensor* table,
          const gdn_tensor* lens, const gdn_tensor* out, AttnParams* p) {
  const int r = q->ndim, c = k->ndim;
  p->q = q->data;
  p->k = k->data;
  p->v = v->data;
  p->out = out->data;
  p->q_sh = step(q, r - 2);
  p->o_sh = step(out, r - 2);
  p->k_st = step(k, c - 3);
  p->k_sh = step(k, c - 2);
  p->v_st = step(v, c - 3);
  p->v_sh = step(v, c - 2);
  if (table) {
    p->k_sp = step(k, 0);
    p->v_sp = step(v, 0);
    // (a table of no pages may have no address; none of it is read then, but
    // that there is one tells the caches from rows)
    p->table = (const int32_t*)(table->data ? table->data : lens->data);
    p->table_st = step(table, 0) / 4;
    p->lens = (const int32_t*)lens->data;
    p->width = (int32_t)A.width;
    p->pages = (int32_t)A.pages;
    p->max_len = (int32_t)(A.width * A.page);
  }
  p->page = divide_by((uint32_t)std::max<int64_t>(A.page, 1));
  p->heads = (int32_t)A.H;
  p->kv = (int32_t)A.K;
  p->group = (int32_t)(A.H / A.K);
  p->window = A.opts.window;
  p->sinks = A.opts.sinks;
  const double scale = A.opts.scale != 0.f ? (double)A.opts.scale : 1.0 / std::sqrt((double)A.D);
  p->scale = (float)(scale * 1.4426950408889634);
}

// Shapes of gdn_attn_decode that its workspace depends on.
size_t decode_workspace(bool bf16, int64_t d) {
  const size_t waves = (size_t)attn_decode_waves(bf16, (int)d);
  const size_t parts = (2 * waves * attn_part_floats((int)d) * 4 + kAlign - 1) / kAlign * kAlign;
  return parts + (waves * 16 + kAlign - 1) / kAlign * kAlign;
}

}  // namespace

extern "C" {

int gdn_cache_plan(const gdn_tensor* ctx_lens, const gdn_tensor* cu_seqlens, gdn_tensor* block_table,
                   const gdn_tensor* free_pages, const gdn_tensor* n_free, int32_t page_size, gdn_tensor* seq_lens,
                   gdn_tensor* slots, gdn_tensor* n_free_out, void* stream) {
  if (!ctx_lens || !block_table || !free_pages || !n_free || !seq_lens || !slots || !n_free_out)
    return api_fail(GDN_ERR_NULL_ARG,
                    "ctx_lens, block_table, free_pages, n_free, seq_lens, slots and n_free_out are required");
  int rc;
  if ((rc = check_ints(ctx_lens, "ctx_lens", -1))) return rc;
  const int64_t n = ctx_lens->shape[0];
  if (n > kMaxRequests) return api_fail(GDN_ERR_SHAPE, "at most 2^20 requests");
  if ((rc = check_table(block_table, n)) || (rc = check_ints(free_pages, "free_pages", -1)) ||
      (rc = check_ints(n_free, "n_free", 1)) || (rc = check_ints(seq_lens, "seq_lens", n)) ||
      (rc = check_ints(slots, "slots", -1, GDN_DTYPE_I64)) || (rc = check_ints(n_free_out, "n_free_out", 1)) ||
      (rc = check_page(page_size, block_table->shape[1])))
    return rc;
  const int64_t t = slots->shape[0];
  if (t > kMaxCount) return api_fail(GDN_ERR_SHAPE, "slots: at most 2^31 - 2^21 tokens");
  Sequences seq;
  if (cu_seqlens) {
    if ((rc = parse_sequences(cu_seqlens, 1, t, &seq))) return rc;
    if (seq.n != n) return api_fail(GDN_ERR_SHAPE, "cu_seqlens must have a sequence for each of %lld requests", (long long)n);
  } else if (t != n) {
    return api_fail(GDN_ERR_SHAPE, "without cu_seqlens there is one token for each of %lld requests", (long long)n);
  }
  if ((rc = check_distinct(block_table, "block_table"))) return rc;
  const Range outs[4] = {range_of(block_table, "block_table"), range_of(seq_lens, "seq_lens"), range_of(slots, "slots"),
                         range_of(n_free_out, "n_free_out")};
  const Range ins[4] = {same_view(ctx_lens, seq_lens) ? Range{} : range_of(ctx_lens, "ctx_lens"),
                        range_of(cu_seqlens, "cu_seqlens"), range_of(free_pages, "free_pages"),
                        same_view(n_free, n_free_out) ? Range{} : range_of(n_free, "n_free")};
  if ((rc = check_overlaps(outs, 4, ins, 4))) return rc;
  const hipStream_t s = (hipStream_t)stream;
  api_clear_error();
  if (cu_seqlens && (rc = api_debug_check_cu(cu_seqlens, n, t, s))) return rc;
  PlanParams p{};
  p.ctx = (const int32_t*)ctx_lens->data;
  p.cu = cu_seqlens ? cu_seqlens->data : nullptr;
  p.cu_i64 = cu_seqlens && cu_seqlens->dtype == GDN_DTYPE_I64;
  p.table = (int32_t*)block_table->data;
  p.table_st = step(block_table, 0) / 4;
  p.free = (const int32_t*)free_pages->data;
  p.free_max = (int32_t)free_pages->shape[0];
  p.n_free = (const int32_t*)n_free->data;
  p.lens = (int32_t*)seq_lens->data;
  p.slots = (int64_t*)slots->data;
  p.n_free_out = (int32_t*)n_free_out->data;
  p.n = (int32_t)n;
  p.t = (int32_t)t;
  p.width = (int32_t)block_table->shape[1];
  p.page = divide_by((uint32_t)page_size);
  const hipError_t e = launch_cache_plan(p, s);
  if (e != hipSuccess) return api_fail(GDN_ERR_HIP, "cache plan launch: %s", hipGetErrorString(e));
  return GDN_OK;
}

int gdn_cache_release(const gdn_tensor* done, gdn_tensor* seq_lens, gdn_tensor* block_table, gdn_tensor* free_pages,
                      gdn_tensor* n_free, int32_t page_size, void* stream) {
  if (!done || !seq_lens || !block_table || !free_pages || !n_free)
    return api_fail(GDN_ERR_NULL_ARG, "done, seq_lens, block_table, free_pages and n_free are required");
  int rc;
  if ((rc = check_ints(done, "done", -1))) return rc;
  const int64_t n = done->shape[0];
  if (n > kMaxRequests) return api_fail(GDN_ERR_SHAPE, "at most 2^20 requests");
  if ((rc = check_table(block_table, n)) || (rc = check_ints(seq_lens, "seq_lens", n)) ||
      (rc = check_ints(free_pages, "free_pages", -1)) || (rc = check_ints(n_free, "n_free", 1)) ||
      (rc = check_page(page_size, block_table->shape[1])) || (rc = check_distinct(block_table, "block_table")))
    return rc;
  const Range outs[4] = {range_of(block_table, "block_table"), range_of(seq_lens, "seq_lens"),
                         range_of(free_pages, "free_pages"), range_of(n_free, "n_free")};
  const Range ins[1] = {range_of(done, "done")};
  if ((rc = check_overlaps(outs, 4, ins, 1))) return rc;
  api_clear_error();
  if (n == 0) return GDN_OK;
  ReleaseParams p{};
  p.done = (const int32_t*)done->data;
  p.lens = (int32_t*)seq_lens->data;
  p.table = (int32_t*)block_table->data;
  p.table_st = step(block_table, 0) / 4;
  p.free = (int32_t*)free_pages->data;
  p.n_free = (int32_t*)n_free->data;
  p.n = (int32_t)n;
  p.width = (int32_t)block_table->shape[1];
  p.free_max = (int32_t)free_pages->shape[0];
  p.page = divide_by((uint32_t)page_size);
  const hipError_t e = launch_cache_release(p, (hipStream_t)stream);
  if (e != hipSuccess) return api_fail(GDN_ERR_HIP, "cache release launch: %s", hipGetErrorString(e));
  return GDN_OK;
}

int gdn_cache_store(const gdn_tensor* k, const gdn_tensor* v, const gdn_tensor* slots, gdn_tensor* k_cache,
                    gdn_tensor* v_cache, void* stream) {
  if (!k || !v || !slots || !k_cache || !v_cache)
    return api_fail(GDN_ERR_NULL_ARG, "k, v, slots, k_cache and v_cache are required");
  if (!is_float(k->dtype)) return api_fail(GDN_ERR_DTYPE, "k must be bf16 or f32");
  if (v->dtype != k->dtype || k_cache->dtype != k->dtype || v_cache->dtype != k->dtype)
    return api_fail(GDN_ERR_DTYPE, "k, v and the caches must share one dtype");
  int rc;
  if ((rc = check_tensor(k, "k", 3, 3)) || (rc = check_tensor(v, "v", 3, 3)) ||
      (rc = check_tensor(k_cache, "k_cache", 4, 4)) || (rc = check_tensor(v_cache, "v_cache", 4, 4)))
    return rc;
  const int64_t t = k->shape[0], kv = k->shape[1], d = k->shape[2];
  if (t > kMaxCount) return api_fail(GDN_ERR_SHAPE, "k: at most 2^31 - 2^21 tokens");
  if (!attn_dim(d)) return api_fail(GDN_ERR_UNSUPPORTED, "d must be 64, 128 or 256 (got %lld)", (long long)d);
  if (kv < 1 || kv > 65535) return api_fail(GDN_ERR_SHAPE, "1 to 65535 key heads (got %lld)", (long long)kv);
  for (int i = 0; i < 3; ++i)
    if (v->shape[i] != k->shape[i]) return api_fail(GDN_ERR_SHAPE, "k and v must have one shape");
  for (int i = 0; i < 4; ++i)
    if (v_cache->shape[i] != k_cache->shape[i]) return api_fail(GDN_ERR_SHAPE, "the caches must have one shape");
  if (k_cache->shape[2] != kv || k_cache->shape[3] != d)
    return api_fail(GDN_ERR_SHAPE, "the caches must be [pages, page_size, %lld, %lld]", (long long)kv, (long long)d);
  if ((rc = check_ints(slots, "slots", t, GDN_DTYPE_I64))) return rc;
  if ((rc = check_granules(k, "k")) || (rc = check_granules(v, "v")) || (rc = check_granules(k_cache, "k_cache")) ||
      (rc = check_granules(v_cache, "v_cache")) || (rc = check_distinct(k_cache, "k_cache")) ||
      (rc = check_distinct(v_cache, "v_cache")))
    return rc;
  const Range outs[2] = {range_of(k_cache, "k_cache"), range_of(v_cache, "v_cache")};
  const Range ins[3] = {range_of(k, "k"), range_of(v, "v"), range_of(slots, "slots")};
  if ((rc = check_overlaps(&outs[0], 1, ins, 3)) || (rc = check_overlaps(&outs[1], 1, ins, 3))) return rc;
  if (overlap(outs[0], outs[1]) && !interleaved(k_cache, v_cache))
    return api_fail(GDN_ERR_LAYOUT, "k_cache overlaps v_cache");
  api_clear_error();
  if (t == 0 || is_empty(k_cache)) return GDN_OK;
  StoreParams p{};
  p.k = k->data;
  p.v = v->data;
  p.k_cache = k_cache->data;
  p.v_cache = v_cache->data;
  p.slots = (const int64_t*)slots->data;
  p.k_st = step(k, 0);
  p.k_sh = step(k, 1);
  p.v_st = step(v, 0);
  p.v_sh = step(v, 1);
  p.kc_sp = step(k_cache, 0);
  p.kc_st = step(k_cache, 1);
  p.kc_sh = step(k_cache, 2);
  p.vc_sp = step(v_cache, 0);
  p.vc_st = step(v_cache, 1);
  p.vc_sh = step(v_cache, 2);
  p.n_slots = k_cache->shape[0] * k_cache->shape[1];
  p.t = (int32_t)t;
  p.kv = (int32_t)kv;
  for (p.row_shift = 0; (16 << p.row_shift) < d * element_size(k->dtype);) ++p.row_shift;
  p.page = divide_by((uint32_t)k_cache->shape[1]);
  const hipError_t e = launch_cache_store(p, (hipStream_t)stream);
  if (e != hipSuccess) return api_fail(GDN_ERR_HIP, "cache store launch: %s", hipGetErrorString(e));
  return GDN_OK;
}

void gdn_attn_default_options(gdn_attn_options* opts) {
  if (!opts) return;
  opts->scale = 0.f;
  opts->window = 0;
  opts->sinks = 0;
}

int gdn_attn_prefill(const gdn_tensor* q, const gdn_tensor* k, const gdn_tensor* v, const gdn_tensor* cu_seqlens,
                     const gdn_tensor* block_table, const gdn_tensor* seq_lens, gdn_tensor* out,
                     const gdn_attn_options* opts, void* stream) {
  if (!q || !k || !v || !out) return api_fail(GDN_ERR_NULL_ARG, "q, k, v and out are required");
  if (!block_table != !seq_lens) return api_fail(GDN_ERR_NULL_ARG, "block_table and seq_lens go together");
  Attn A;
  int rc;
  if ((rc = attn_options(opts, &A.opts)) || (rc = check_types(q, k, v, out)) || (rc = check_rows_of(q, out, 3, 4)))
    return rc;
  Tokens tq, to, tk, tv;
  if ((rc = parse_tokens(q, "q", 2, &tq)) || (rc = parse_tokens(out, "out", 2, &to))) return rc;
  const int r = q->ndim;
  A.T = tq.T;
  A.H = q->shape[r - 2];
  A.D = q->shape[r - 1];
  Sequences seq;
  if ((rc = parse_sequences(cu_seqlens, tq.B, A.T, &seq))) return rc;
  if (block_table) {
    if ((rc = parse_caches(k, v, block_table, seq_lens, seq.n, &A))) return rc;
  } else {
    if ((rc = check_tensor(k, "k", 3, 4)) || (rc = check_tensor(v, "v", 3, 4)) ||
        (rc = parse_tokens(k, "k", 2, &tk)) || (rc = parse_tokens(v, "v", 2, &tv)))
      return rc;
    if (k->ndim != r || v->ndim != r) return api_fail(GDN_ERR_SHAPE, "q, k and v must have one rank");
    if (tk.T != A.T || tk.B != tq.B || tv.T != A.T || tv.B != tq.B)
      return api_fail(GDN_ERR_SHAPE, "k and v must have a row for each of q's");
    A.K = k->shape[r - 2];
    if (k->shape[r - 1] != A.D) return api_fail(GDN_ERR_SHAPE, "k's d differs from q's");
  }
  if ((rc = check_heads(A, q, k, v, out))) return rc;
  const bool bf16 = q->dtype == GDN_DTYPE_BF16;
  const int64_t rows = attn_tile_rows(bf16, (int)A.D);
  const int64_t tiles = seq.packed ? A.T / rows + seq.n : (int64_t)seq.n * ((seq.len + rows - 1) / rows);
  if (tiles * A.H * 512 >= kMaxThreads) return api_fail(GDN_ERR_SHAPE, "too many (tile, head) pairs");
  const Range outs[1] = {range_of(out, "out")};
  const Range ins[6] = {range_of(q, "q"), range_of(k, "k"), range_of(v, "v"), range_of(cu_seqlens, "cu_seqlens"),
                        range_of(block_table, "block_table"), range_of(seq_lens, "seq_lens")};
  if ((rc = check_overlaps(outs, 1, ins, 6))) return rc;
  const hipStream_t s = (hipStream_t)stream;
  api_clear_error();
  if (seq.packed && (rc = api_debug_check_cu(cu_seqlens, seq.n, A.T, s))) return rc;
  if (A.T == 0) return GDN_OK;
  AttnParams p{};
  fill(A, q, k, v, block_table, seq_lens, out, &p);
  const int64_t es = element_size(q->dtype);
  p.q_st = A.T > 1 ? tq.st * es : 0;
  p.o_st = A.T > 1 ? to.st * es : 0;
  if (!block_table) {
    p.k_st = A.T > 1 ? tk.st * es : 0;
    p.v_st = A.T > 1 ? tv.st * es : 0;
  }
  p.cu = cu_seqlens ? cu_seqlens->data : nullptr;
  p.cu_i64 = cu_seqlens && cu_seqlens->dtype == GDN_DTYPE_I64;
  p.n_seq = seq.n;
  p.seq_len = seq.len;
  p.t_total = (int32_t)A.T;
  const hipError_t e = launch_attn_prefill(bf16, (int)A.D, p, s);
  if (e != hipSuccess) return api_fail(GDN_ERR_HIP, "attention launch: %s", hipGetErrorString(e));
  return GDN_OK;
}

int gdn_attn_workspace_size(const gdn_tensor* q, size_t* bytes) {
  if (!q || !bytes) return api_fail(GDN_ERR_NULL_ARG, "q and bytes are required");
  if (!is_float(q->dtype)) return api_fail(GDN_ERR_DTYPE, "q must be bf16 or f32");
  if (q->ndim != 3) return api_fail(GDN_ERR_SHAPE, "q must be [N, H, d]");
  if (!attn_dim(q->shape[2]))
    return api_fail(GDN_ERR_UNSUPPORTED, "d must be 64, 128 or 256 (got %lld)", (long long)q->shape[2]);
  *bytes = decode_workspace(q->dtype == GDN_DTYPE_BF16, q->shape[2]);
  return GDN_OK;
}

int gdn_attn_decode(const gdn_tensor* q, const gdn_tensor* k_cache, const gdn_tensor* v_cache,
                    const gdn_tensor* block_table, const gdn_tensor* seq_lens, gdn_tensor* out,
                    const gdn_attn_options* opts, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out)
    return api_fail(GDN_ERR_NULL_ARG, "q, k_cache, v_cache, block_table, seq_lens and out are required");
  Attn A;
  int rc;
  if ((rc = attn_options(opts, &A.opts)) || (rc = check_types(q, k_cache, v_cache, out)) ||
      (rc = check_rows_of(q, out, 3, 3)))
    return rc;
  const int64_t n = q->shape[0];
  A.T = n;
  A.H = q->shape[1];
  A.D = q->shape[2];
  if (n > kMaxRequests) return api_fail(GDN_ERR_SHAPE, "at most 2^20 sequences");
  if ((rc = parse_caches(k_cache, v_cache, block_table, seq_lens, n, &A)) ||
      (rc = check_heads(A, q, k_cache, v_cache, out)))
    return rc;
  const bool bf16 = q->dtype == GDN_DTYPE_BF16;
  const size_t need = decode_workspace(bf16, A.D);
  if (!workspace || workspace_bytes < need)
    return api_fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, workspace_bytes);
  if ((uintptr_t)workspace % kAlign) return api_fail(GDN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const Range outs[2] = {range_of(out, "out"), range_of(workspace, (int64_t)need, "workspace")};
  const Range ins[5] = {range_of(q, "q"), range_of(k_cache, "k_cache"), range_of(v_cache, "v_cache"),
                        range_of(block_table, "block_table"), range_of(seq_lens, "seq_lens")};
  if ((rc = check_overlaps(outs, 2, ins, 5))) return rc;
  api_clear_error();
  if (n == 0) return GDN_OK;
  AttnParams p{};
  fill(A, q, k_cache, v_cache, block_table, seq_lens, out, &p);
  p.q_st = step(q, 0);
  p.o_st = step(out, 0);
  p.n_seq = (int32_t)n;
  p.t_total = (int32_t)n;
  p.waves = attn_decode_waves(bf16, (int)A.D);
  p.parts = (float*)workspace;
  p.chains = (int32_t*)((char*)workspace + need - ((size_t)p.waves * 16 + kAlign - 1) / kAlign * kAlign);
  const hipError_t e = launch_attn_decode(bf16, (int)A.D, p, (hipStream_t)stream);
  if (e != hipSuccess) return api_fail(GDN_ERR_HIP, "attention launch: %s", hipGetErrorString(e));
  return GDN_OK;
}

}  // extern "C"
