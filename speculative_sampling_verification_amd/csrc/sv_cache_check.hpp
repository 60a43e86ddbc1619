// Host-side checks shared by the C entry points of the paged-cache operators: a cache's
// description, strides of dense and strided tensors, arrays that must not share memory.
#pragma once

#include <climits>
#include <cstdint>

#include "sv_cache.hpp"

namespace sv {

constexpr int kMaxHeads = 1024;
constexpr int kMaxHeadBytes = 1024;
constexpr int kMaxLayers = 8192;

inline bool aligned_to(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) % n) == 0;
}

// Whether [a, a + n) and [b, b + m) (bytes) share memory; a null pointer shares none.
inline bool overlap(const void* a, uint64_t n, const void* b, uint64_t m) {
  const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + m && y < x + n;
}

// Whether the rows of a dense or strided tensor lie apart: with the dimensions in order of
// stride, each stride clears everything the smaller ones span.  `row` is the innermost extent.
// Sizes of one do not move anything, so their strides do not matter.
template <int Dims>
bool rows_apart(int64_t row, const int64_t (&stride)[Dims], const int64_t (&size)[Dims]) {
  int64_t span = row;
  bool used[Dims] = {};
  for (int n = 0; n < Dims; ++n) {
    int best = -1;
    for (int i = 0; i < Dims; ++i)
      if (!used[i] && size[i] > 1 && (best < 0 || stride[i] < stride[best])) best = i;
    if (best < 0) return true;
    used[best] = true;
    if (stride[best] < span) return false;
    int64_t step;
    if (__builtin_mul_overflow(stride[best], size[best] - 1, &step) ||
        __builtin_add_overflow(span, step, &span))
      return false;
  }
  return true;
}

// Checks a cache description and fills the kernels' view of layers [layer, layer + count).
inline int view_of(const sv_cache* c, int layer, int count, CacheView* v) {
  if (!c) return SV_ERR_INVALID_ARG;
  if (c->dtype != SV_DTYPE_F32 && c->dtype != SV_DTYPE_BF16) return SV_ERR_UNSUPPORTED_DTYPE;
  const int es = c->dtype == SV_DTYPE_BF16 ? 2 : 4;
  if (!c->k || !c->v || !c->page_table || !c->seq_lens) return SV_ERR_INVALID_ARG;
  if (c->layers < 1 || c->layers > kMaxLayers || c->pages < 1 || c->page_size < 1 ||
      c->kv_heads < 1 || c->kv_heads > kMaxHeads || c->head_dim < 1)
    return SV_ERR_INVALID_ARG;
  if (c->head_dim > kMaxHeadBytes / es || (c->head_dim * es) % 16 != 0) return SV_ERR_INVALID_ARG;
  if (c->seqs < 1 || c->seqs > kCacheMaxSeqs || c->table_width < 1) return SV_ERR_INVALID_ARG;
  if ((int64_t)c->table_width * c->page_size > kCacheMaxTokens) return SV_ERR_INVALID_ARG;
  if ((int64_t)c->seqs * c->table_width > INT_MAX) return SV_ERR_INVALID_ARG;
  if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16)) return SV_ERR_INVALID_ARG;
  if (!aligned_to(c->page_table, 4) || !aligned_to(c->seq_lens, 4) ||
      !aligned_to(c->seq_pages, 4) || !aligned_to(c->refcount, 4))
    return SV_ERR_INVALID_ARG;
  const int64_t stride[4] = {c->layer_stride, c->page_stride, c->token_stride, c->head_stride};
  const int64_t size[4] = {c->layers, c->pages, c->page_size, c->kv_heads};
  for (int i = 0; i < 4; ++i)
    if (size[i] > 1 &&
        (stride[i] < 0 || stride[i] > INT64_MAX / 4 || (stride[i] * es) % 16 != 0))
      return SV_ERR_INVALID_ARG;
  if (!rows_apart(c->head_dim, stride, size)) return SV_ERR_INVALID_ARG;
  if (layer < 0 || layer >= c->layers) return SV_ERR_INVALID_ARG;
  auto bytes = [&](int i) { return size[i] > 1 ? stride[i] * es : 0; };
  v->layer_stride = bytes(0);
  v->page_stride = bytes(1);
  v->token_stride = bytes(2);
  v->head_stride = bytes(3);
  v->k = static_cast<char*>(c->k) + layer * v->layer_stride;
  v->v = static_cast<char*>(c->v) + layer * v->layer_stride;
  v->esize = es;
  v->layers = count;
  v->pages = c->pages;
  v->page_size = c->page_size;
  v->kv_heads = c->kv_heads;
  v->head_dim = c->head_dim;
  v->seqs = c->seqs;
  v->width = c->table_width;
  v->cap = c->table_width * c->page_size;
  v->page_div = make_fast_div((uint32_t)c->page_size);
  v->table = c->page_table;
  v->lens = c->seq_lens;
  v->held = c->seq_pages;
  v->refcount = c->refcount;
  return SV_OK;
}

// Whether no row of the keys is one of the values: of two tensors apart, or two parts of one.
inline bool values_apart(const sv_cache* c) {
  const int64_t k = (int64_t)reinterpret_cast<uintptr_t>(c->k);
  const int64_t v = (int64_t)reinterpret_cast<uintptr_t>(c->v);
  const int es = c->dtype == SV_DTYPE_BF16 ? 2 : 4;
  const int64_t stride[5] = {c->layer_stride, c->page_stride, c->token_stride, c->head_stride,
                             (k < v ? v - k : k - v) / es};
  const int64_t size[5] = {c->layers, c->pages, c->page_size, c->kv_heads, 2};
  return rows_apart(c->head_dim, stride, size);
}

// Strides (elements) of a [B, N, H, D] tensor, dense where `given` is null; false if a row does
// not start on 16 bytes.
inline bool row_strides(const int64_t* given, int N, int H, int D, int es, int64_t (&s)[3]) {
  if (given) {
    for (int i = 0; i < 3; ++i) {
      if (given[i] < 0 || given[i] > INT64_MAX / 8 || (given[i] * es) % 16 != 0) return false;
      s[i] = given[i] * es;
    }
  } else {
    s[2] = (int64_t)D * es;
    s[1] = s[2] * H;
    s[0] = s[1] * N;
  }
  return true;
}

// Bytes from a tensor's first element to behind its last (strides in bytes), false where no address
// space holds them.
template <int Dims>
bool extent_of(int64_t row, const int64_t (&stride)[Dims], const int64_t (&size)[Dims],
               uint64_t* bytes) {
  int64_t span = row, step;
  for (int i = 0; i < Dims; ++i)
    if (__builtin_mul_overflow(stride[i], size[i] - 1, &step) ||
        __builtin_add_overflow(span, step, &span))
      return false;
  *bytes = (uint64_t)span;
  return true;
}

struct Range {
  const void* at;  // null: an array that is not given
  uint64_t bytes;
};

// Whether what a call writes (the first `outs` of the ranges) shares memory with
// anything else that it reads or writes.
template <int Count>
bool outputs_apart(const Range (&r)[Count], int outs) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < Count; ++j)
      if (overlap(r[i].at, r[i].bytes, r[j].at, r[j].bytes)) return false;
  return true;
}

// Whether attention, and what follows it, takes N nodes of q_heads heads.
inline bool attn_shape(const sv_cache* c, int N, int q_heads) {
  if (N < 1 || N > kCacheMaxNodes) return false;
  if (q_heads < 1 || q_heads > 64 * kMaxHeads || q_heads % c->kv_heads != 0) return false;
  const int D = c->head_dim;
  if (D != 64 && D != 96 && D != 128 && D != 256) return false;
  return (int64_t)N * (q_heads / c->kv_heads) <= INT_MAX / 2;
}

inline int status_of(hipError_t e) { return e == hipSuccess ? SV_OK : SV_ERR_LAUNCH; }

}  // namespace sv
