// Checks of descriptors that the sources of the C ABI share (host only): ranks,
// sizes, strides, packed sequences and overlaps.
#pragma once

#include <cstdint>

#include "gdn.h"
#include "gdn_api_common.h"

namespace gdn {

constexpr int64_t kMax32 = (int64_t)1 << 31;
// Tokens, sequences and channels: the kernels' 32-bit counters may run past
// the last one by a tile, a segment or a round of threads.
constexpr int64_t kMaxCount = kMax32 - ((int64_t)1 << 21);
constexpr int64_t kMaxElements = (int64_t)1 << 48;

inline int64_t element_size(int32_t dtype) {
  switch (dtype) {
    case GDN_DTYPE_BF16: return 2;
    case GDN_DTYPE_F32: case GDN_DTYPE_I32: return 4;
    case GDN_DTYPE_I64: return 8;
    case GDN_E4M3: return 1;
  }
  return 0;
}

inline bool is_float(int32_t dtype) { return dtype == GDN_DTYPE_BF16 || dtype == GDN_DTYPE_F32; }

// Rank, sizes and strides of a tensor whose last dimension has unit stride
// (or any stride, for per-head scalars).  An empty tensor's strides carry no
// layout and its data may be NULL.
inline int check_tensor(const gdn_tensor* t, const char* name, int lo_rank, int hi_rank, bool unit_last = true) {
  if (t->ndim < lo_rank || t->ndim > hi_rank)
    return api_fail(GDN_ERR_SHAPE, "%s: expected %d to %d dimensions, got %d", name, lo_rank, hi_rank, t->ndim);
  if (element_size(t->dtype) == 0) return api_fail(GDN_ERR_DTYPE, "%s: unknown dtype", name);
  bool empty = false;
  __int128 elements = 1, extent = 0;
  for (int i = 0; i < t->ndim; ++i) {
    if (t->shape[i] < 0 || t->shape[i] >= kMax32) return api_fail(GDN_ERR_SHAPE, "%s: size out of range", name);
    empty = empty || t->shape[i] == 0;
    elements *= t->shape[i];
  }
  if (empty) return GDN_OK;
  for (int i = 0; i < t->ndim; ++i) {
    if (t->stride[i] < 0) return api_fail(GDN_ERR_LAYOUT, "%s: negative stride", name);
    extent += (__int128)(t->shape[i] - 1) * t->stride[i];
  }
  if (elements >= kMaxElements || extent >= kMaxElements)
    return api_fail(GDN_ERR_SHAPE, "%s: larger than any memory", name);
  if (unit_last && t->shape[t->ndim - 1] > 1 && t->stride[t->ndim - 1] != 1)
    return api_fail(GDN_ERR_LAYOUT, "%s: last dimension must have unit stride", name);
  if (!t->data) return api_fail(GDN_ERR_NULL_ARG, "%s data is NULL", name);
  if ((uintptr_t)t->data % (uintptr_t)element_size(t->dtype))
    return api_fail(GDN_ERR_LAYOUT, "%s: misaligned data", name);
  return GDN_OK;
}

inline bool is_empty(const gdn_tensor* t) {
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] == 0) return true;
  return false;
}

inline bool contiguous(const gdn_tensor* t) {
  int64_t acc = 1;
  for (int i = t->ndim - 1; i >= 0; --i) {
    if (t->shape[i] != 1 && t->stride[i] != acc) return false;
    acc *= t->shape[i];
  }
  return true;
}

// The bytes between a tensor's first and last element.
struct Range {
  uintptr_t lo = 0, hi = 0;  // empty: lo == hi
  const char* name = "";
};

inline Range range_of(const gdn_tensor* t, const char* name) {
  Range r;
  r.name = name;
  if (!t || !t->data || is_empty(t)) return r;
  int64_t last = 0;
  for (int i = 0; i < t->ndim; ++i) last += (t->shape[i] - 1) * t->stride[i];
  r.lo = (uintptr_t)t->data;
  r.hi = r.lo + (uintptr_t)((last + 1) * element_size(t->dtype));
  return r;
}

inline Range range_of(const void* p, int64_t bytes, const char* name) {
  Range r;
  r.name = name;
  if (!p || bytes <= 0) return r;
  r.lo = (uintptr_t)p;
  r.hi = r.lo + (uintptr_t)bytes;
  return r;
}

inline bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

// The same elements in the same places (an output an input may share).
inline bool same_view(const gdn_tensor* a, const gdn_tensor* b) {
  if (!a || !b || a->data != b->data || a->ndim != b->ndim || a->dtype != b->dtype) return false;
  for (int i = 0; i < a->ndim; ++i)
    if (a->shape[i] != b->shape[i] || (a->shape[i] > 1 && a->stride[i] != b->stride[i])) return false;
  return true;
}

// Token-major views: [T, ...] or [B, L, ...] flattened.
struct Tokens {
  int64_t B = 1, T = 0, st = 0;  // sequences, tokens, token stride
};

// rank: dimensions after the tokens.
inline int parse_tokens(const gdn_tensor* t, const char* name, int rank, Tokens* v) {
  const bool batched = t->ndim == rank + 2;
  if (!batched && t->ndim != rank + 1)
    return api_fail(GDN_ERR_SHAPE, "%s: expected %d or %d dimensions, got %d", name, rank + 1, rank + 2, t->ndim);
  v->B = batched ? t->shape[0] : 1;
  v->T = batched ? t->shape[0] * t->shape[1] : t->shape[0];
  v->st = t->stride[batched ? 1 : 0];
  if (batched && t->shape[1] == 1) v->st = t->stride[0];
  if (v->T > kMaxCount) return api_fail(GDN_ERR_SHAPE, "%s: T must be at most 2^31 - 2^21", name);
  if (batched && !is_empty(t) && t->shape[0] > 1 && t->shape[1] > 1 && t->stride[0] != (__int128)t->shape[1] * t->stride[1])
    return api_fail(GDN_ERR_LAYOUT, "%s: batch stride must equal seq_len * token stride", name);
  return GDN_OK;
}

// cu_seqlens, or the uniform sequences of a batch.
struct Sequences {
  bool packed = false;
  int n = 0;
  int len = 0;  // uniform
};

inline int parse_sequences(const gdn_tensor* cu, int64_t batch, int64_t tokens, Sequences* s) {
  if (!cu) {
    if (batch < 1) return api_fail(GDN_ERR_SHAPE, "at least one sequence is required");
    if (batch > kMaxCount) return api_fail(GDN_ERR_SHAPE, "too many sequences");
    s->packed = false;
    s->n = (int)batch;
    s->len = (int)(tokens / batch);
    return GDN_OK;
  }
  if (cu->dtype != GDN_DTYPE_I32 && cu->dtype != GDN_DTYPE_I64)
    return api_fail(GDN_ERR_DTYPE, "cu_seqlens must be int32 or int64");
  if (cu->ndim != 1 || cu->shape[0] < 2) return api_fail(GDN_ERR_SHAPE, "cu_seqlens must be 1-D with N+1 >= 2 entries");
  if (cu->shape[0] - 1 > kMaxCount) return api_fail(GDN_ERR_SHAPE, "too many sequences");
  if (cu->stride[0] != 1) return api_fail(GDN_ERR_LAYOUT, "cu_seqlens must be contiguous");
  if (!cu->data) return api_fail(GDN_ERR_NULL_ARG, "cu_seqlens data is NULL");
  if ((uintptr_t)cu->data % (uintptr_t)element_size(cu->dtype))
    return api_fail(GDN_ERR_LAYOUT, "cu_seqlens: misaligned data");
  if (batch != 1) return api_fail(GDN_ERR_SHAPE, "with cu_seqlens the batch dimension must be 1");
  s->packed = true;
  s->n = (int)(cu->shape[0] - 1);
  s->len = 0;
  return GDN_OK;
}

// Whether a strided array's elements all lie in different places: sorted by
// stride, every dimension steps past all that the smaller ones span.
inline bool distinct(const int64_t* shape, const int64_t* stride, int n) {
  bool done[8] = {};
  __int128 span = 0;  // of the dimensions so far
  for (int k = 0; k < n; ++k) {
    int at = -1;
    for (int i = 0; i < n; ++i)
      if (!done[i] && (at < 0 || stride[i] < stride[at])) at = i;
    done[at] = true;
    if (shape[at] <= 1) continue;
    if (stride[at] <= span) return false;
    span += (__int128)(shape[at] - 1) * stride[at];
  }
  return true;
}

inline bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

// Rows [tokens][heads][row] of an output that overlap each other would race.
inline int check_rows(const char* name, int64_t tokens, int64_t st, int64_t heads, int64_t sh, int64_t row) {
  const bool token_major = (heads <= 1 || sh >= row) && (tokens <= 1 || st >= (heads - 1) * sh + row);
  const bool head_major = (tokens <= 1 || st >= row) && (heads <= 1 || sh >= (tokens - 1) * st + row);
  if (tokens > 0 && !token_major && !head_major) return api_fail(GDN_ERR_LAYOUT, "%s: rows overlap", name);
  return GDN_OK;
}

// Every output against every input and the other outputs.
inline int check_overlaps(const Range* outs, int n_out, const Range* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(outs[i], ins[j])) return api_fail(GDN_ERR_LAYOUT, "%s overlaps %s", outs[i].name, ins[j].name);
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(outs[i], outs[j])) return api_fail(GDN_ERR_LAYOUT, "%s overlaps %s", outs[i].name, outs[j].name);
  }
  return GDN_OK;
}

}  // namespace gdn
