// extern "C" entry points of the paged-cache operators: host-side argument checks, workspace
// layout and dispatch.  No allocation, no synchronisation; everything is enqueued on the
// caller's stream.  See include/spec_verify.h for the contract of each function.

#include <climits>
#include <cmath>
#include <cstdint>

#include "sv_cache.hpp"

using namespace sv;

namespace {

constexpr int kMaxHeads = 1024;
constexpr int kMaxHeadBytes = 1024;
constexpr int kMaxLayers = 8192;

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// Whether [a, a + n) and [b, b + m) (bytes) share memory; a null pointer shares none.
bool overlap(const void* a, uint64_t n, const void* b, uint64_t m) {
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
int view_of(const sv_cache* c, int layer, int count, CacheView* v) {
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
bool values_apart(const sv_cache* c) {
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
bool row_strides(const int64_t* given, int N, int H, int D, int es, int64_t (&s)[3]) {
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

// Whether what an attention call writes (the first `outs` of the ranges) shares memory with
// anything else that it reads or writes.
template <int Count>
bool outputs_apart(const Range (&r)[Count], int outs) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < Count; ++j)
      if (overlap(r[i].at, r[i].bytes, r[j].at, r[j].bytes)) return false;
  return true;
}

bool attn_shape(const sv_cache* c, int N, int q_heads) {
  if (N < 1 || N > kCacheMaxNodes) return false;
  if (q_heads < 1 || q_heads > 64 * kMaxHeads || q_heads % c->kv_heads != 0) return false;
  const int D = c->head_dim;
  if (D != 64 && D != 96 && D != 128 && D != 256) return false;
  return (int64_t)N * (q_heads / c->kv_heads) <= INT_MAX / 2;
}

int status_of(hipError_t e) { return e == hipSuccess ? SV_OK : SV_ERR_LAUNCH; }

}  // namespace

extern "C" {

size_t spec_tree_attention_workspace_size(const sv_cache* cache, int N, int q_heads) {
  CacheView v{};
  if (view_of(cache, 0, 1, &v) != SV_OK || !attn_shape(cache, N, q_heads)) return 0;
  return plan_tree_attention(v, cache->dtype, N, q_heads / cache->kv_heads).bytes;
}

int spec_tree_attention(const void* q, const int64_t* q_strides, int N, int q_heads,
                        const sv_cache* cache, int layer, const uint8_t* mask,
                        const int32_t* num_nodes, float scale, void* out, float* out_lse,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
  AttnArgs a{};
  const int st = view_of(cache, layer, 1, &a.c);
  if (st != SV_OK) return st;
  if (!q || !out || !attn_shape(cache, N, q_heads)) return SV_ERR_INVALID_ARG;
  // the kernel multiplies scores by scale * log2(e)
  if (!(scale > 0.0f) || !std::isfinite(scale * 1.44269504088896340736f)) return SV_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(out_lse, 4) ||
      !aligned_to(num_nodes, 4))
    return SV_ERR_INVALID_ARG;
  int64_t s[3];
  if (!row_strides(q_strides, N, q_heads, cache->head_dim, a.c.esize, s))
    return SV_ERR_INVALID_ARG;
  a.G = q_heads / cache->kv_heads;
  a.N = N;
  const AttnPlan p = plan_tree_attention(a.c, cache->dtype, N, a.G);
  if (!workspace || workspace_bytes < p.bytes) return SV_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned_to(workspace, 16)) return SV_ERR_INVALID_ARG;
  // workgroups write while others still read
  const CacheView& v = a.c;
  const int64_t row = (int64_t)v.head_dim * v.esize;
  const int64_t cache_stride[3] = {v.page_stride, v.token_stride, v.head_stride};
  const int64_t cache_size[3] = {v.pages, v.page_size, v.kv_heads};
  const int64_t q_size[3] = {v.seqs, N, q_heads};
  uint64_t layer_bytes, q_bytes;
  if (!extent_of(row, cache_stride, cache_size, &layer_bytes) ||
      !extent_of(row, s, q_size, &q_bytes))
    return SV_ERR_INVALID_ARG;
  const uint64_t rows = (uint64_t)v.seqs * N * q_heads, word = sizeof(int32_t);
  const Range ranges[] = {{out, rows * row}, {out_lse, rows * sizeof(float)},
                          {workspace, p.bytes}, {q, q_bytes},
                          {v.k, layer_bytes}, {v.v, layer_bytes},
                          {mask, (uint64_t)v.seqs * N * N}, {num_nodes, word * v.seqs},
                          {v.table, word * v.seqs * v.width}, {v.lens, word * v.seqs},
                          {v.held, word * v.seqs}, {v.refcount, word * v.pages}};
  if (!outputs_apart(ranges, 3)) return SV_ERR_INVALID_ARG;
  a.q = static_cast<const char*>(q);
  a.q_seq = s[0];
  a.q_node = s[1];
  a.q_head = s[2];
  a.mask = mask;
  a.nodes = num_nodes;
  a.mts = p.mts;
  a.scale = scale;
  a.out = static_cast<char*>(out);
  a.lse = out_lse;
  a.workers = p.workers;
  char* ws = static_cast<char*>(workspace);
  a.part = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + p.o_ml);
  a.tail = reinterpret_cast<int4*>(ws + p.o_tail);
  return status_of(launch_tree_attention(a, cache->dtype, p, stream));
}

int spec_cache_append(const void* k_new, const void* v_new, const int64_t* new_strides, int N,
                      const sv_cache* cache, int layer, const int32_t* num_nodes,
                      hipStream_t stream) {
  CacheView v{};
  const int st = view_of(cache, layer, 1, &v);
  if (st != SV_OK) return st;
  if (!values_apart(cache) || !k_new || !v_new || N < 1 || N > kCacheMaxNodes) return SV_ERR_INVALID_ARG;
  if (!aligned_to(k_new, 16) || !aligned_to(v_new, 16) || !aligned_to(num_nodes, 4))
    return SV_ERR_INVALID_ARG;
  int64_t s[3];
  if (!row_strides(new_strides, N, v.kv_heads, v.head_dim, v.esize, s)) return SV_ERR_INVALID_ARG;
  return status_of(launch_cache_append(v, static_cast<const char*>(k_new),
                                       static_cast<const char*>(v_new), s[0], s[1], s[2],
                                       num_nodes, N, stream));
}

int spec_cache_commit(const sv_cache* cache, const int32_t* last_node, const int32_t* parent,
                      int N, int32_t* out_lens, hipStream_t stream) {
  CacheView v{};
  const int st = view_of(cache, 0, cache ? cache->layers : 0, &v);
  if (st != SV_OK) return st;
  if (!values_apart(cache) || !last_node || !out_lens || N < 1 || N > kCacheMaxNodes)
    return SV_ERR_INVALID_ARG;
  if (!aligned_to(last_node, 4) || !aligned_to(parent, 4) || !aligned_to(out_lens, 4))
    return SV_ERR_INVALID_ARG;
  // every workgroup of a sequence reads these while one of them stores the new length
  const uint64_t row = (uint64_t)v.seqs * sizeof(int32_t);
  if (overlap(out_lens, row, v.lens, row) || overlap(out_lens, row, last_node, row) ||
      overlap(out_lens, row, parent, row * N) || overlap(out_lens, row, v.table, row * v.width) ||
      overlap(out_lens, row, v.held, row) ||
      overlap(out_lens, row, v.refcount, (uint64_t)v.pages * sizeof(int32_t)))
    return SV_ERR_INVALID_ARG;
  return status_of(launch_cache_commit(v, parent, last_node, N, out_lens, stream));
}

int spec_cache_resize(const sv_cache* cache, const int32_t* want, const int32_t* new_lens,
                      int32_t* out_ok, hipStream_t stream) {
  CacheView v{};
  const int st = view_of(cache, 0, 1, &v);
  if (st != SV_OK) return st;
  if (!v.held || !v.refcount || !want || !out_ok) return SV_ERR_INVALID_ARG;
  if (!aligned_to(want, 4) || !aligned_to(new_lens, 4) || !aligned_to(out_ok, 4))
    return SV_ERR_INVALID_ARG;
  // the cache's arrays and the results are written while the others are read; seq_lens itself may
  // be given (a thread reads a sequence's values before it stores its length)
  const uint64_t row = (uint64_t)v.seqs * sizeof(int32_t);
  const uint64_t counts = (uint64_t)v.pages * sizeof(int32_t);
  for (const int32_t* x : {want, new_lens, static_cast<const int32_t*>(out_ok)})
    if ((overlap(x, row, v.lens, row) && (x == out_ok || x != v.lens)) || overlap(x, row, v.held, row) ||
        overlap(x, row, v.refcount, counts) || overlap(x, row, v.table, row * v.width))
      return SV_ERR_INVALID_ARG;
  if (overlap(out_ok, row, want, row) || overlap(out_ok, row, new_lens, row))
    return SV_ERR_INVALID_ARG;
  return status_of(launch_cache_resize(v, want, new_lens, out_ok, stream));
}

int spec_cache_fork(const sv_cache* cache, const int32_t* src, const int32_t* dst, int F,
                    int32_t* out_ok, hipStream_t stream) {
  CacheView v{};
  const int st = view_of(cache, 0, cache ? cache->layers : 0, &v);
  if (st != SV_OK) return st;
  if (!values_apart(cache) || !v.held || !v.refcount || F < 0 || F > v.seqs)
    return SV_ERR_INVALID_ARG;
  if (F == 0) return SV_OK;
  if (!src || !dst || !out_ok) return SV_ERR_INVALID_ARG;
  if (!aligned_to(src, 4) || !aligned_to(dst, 4) || !aligned_to(out_ok, 4))
    return SV_ERR_INVALID_ARG;
  const uint64_t row = (uint64_t)v.seqs * sizeof(int32_t), some = (uint64_t)F * sizeof(int32_t);
  const uint64_t counts = (uint64_t)v.pages * sizeof(int32_t);
  for (const int32_t* x : {src, dst, static_cast<const int32_t*>(out_ok)})
    if (overlap(x, some, v.lens, row) || overlap(x, some, v.held, row) ||
        overlap(x, some, v.refcount, counts) || overlap(x, some, v.table, row * v.width))
      return SV_ERR_INVALID_ARG;
  if (overlap(out_ok, some, src, some) || overlap(out_ok, some, dst, some))
    return SV_ERR_INVALID_ARG;
  return status_of(launch_cache_fork(v, src, dst, F, out_ok, stream));
}

}  // extern "C"
