// extern "C" entry points of the paged-cache operators: host-side argument checks, workspace
// layout and dispatch.  No allocation, no synchronisation; everything is enqueued on the
// caller's stream.  See include/spec_verify.h for the contract of each function.

#include <climits>
#include <cmath>
#include <cstdint>

#include "sv_cache_check.hpp"

using namespace sv;

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
