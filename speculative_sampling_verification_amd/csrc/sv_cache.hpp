// Shared declarations of the paged-cache operators: tree attention (sv_tree_attn.hip), the
// cache's row and page movement (sv_cache.hip) and their C entry points (sv_cache_abi.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "spec_verify.h"

namespace sv {

constexpr int kCacheMaxSeqs = 8192;          // sequences of a cache (the page pool keeps three
                                             // words of each in LDS)
constexpr int kCacheMaxNodes = 2048;         // nodes per sequence (as spec_verify_tree)
constexpr int kCacheMaxTokens = 1 << 30;     // table_width * page_size
constexpr int kAttnCus = 256;                // compute units of a gfx950 GPU

// t / d for 0 <= t < 2^31 by a multiplication (d >= 1), after Granlund and Montgomery, "Division by
// Invariant Integers using Multiplication" (1994): with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, t / d = (hi32(m t) + t) >> s; the sum stays below 2^32.
struct FastDiv {
  uint32_t d, m, s;
};

inline FastDiv make_fast_div(uint32_t d) {
  FastDiv f{d, 0u, 0u};
  while ((1ull << f.s) < d) ++f.s;
  f.m = (uint32_t)((((1ull << f.s) - d) << 32) / d + 1);
  return f;
}

__device__ __forceinline__ uint32_t fast_div(const FastDiv& f, uint32_t t) {
  return (__umulhi(f.m, t) + t) >> f.s;
}

// One layer's view (attention, append) or all layers' (commit, fork) of a paged cache.
struct CacheView {
  char* k;  // layer offset applied
  char* v;
  int esize;                                        // bytes per element
  int layers, pages, page_size, kv_heads, head_dim;
  int64_t layer_stride, page_stride, token_stride, head_stride;  // bytes
  int seqs, width, cap;                             // table rows, entries a row, width * page_size
  FastDiv page_div;
  int32_t* table;
  int32_t* lens;
  int32_t* held;
  int32_t* refcount;
};

// Positions of sequence b in the pages that it holds; all there can be for a cache without books.
__device__ __forceinline__ int positions_held(const CacheView& c, int b) {
  if (!c.held || !c.refcount) return INT32_MAX;
  const int n = c.held[b];
  return (n < 0 ? 0 : n > c.width ? c.width : n) * c.page_size;
}

// Whether a page that the table names for position `pos` is its sequence's, which holds `held`
// positions.  Entries behind those keep what they named before pages were given back, and such a
// page may have gone to another sequence: its count says so (one load, and only there).
__device__ __forceinline__ bool names_page(const CacheView& c, int held, int pos, int page) {
  if (page < 0 || page >= c.pages) return false;
  return pos < held || c.refcount[page] == 0;
}

// Byte offset of a position's row in the pages of sequence b, which holds `held` of them; -1 where
// it has no page.
__device__ __forceinline__ int64_t row_offset(const CacheView& c, int b, int held, int pos) {
  if (pos < 0 || pos >= c.cap) return -1;
  const uint32_t pi = fast_div(c.page_div, (uint32_t)pos);
  const int page = c.table[(size_t)b * c.width + pi];
  if (!names_page(c, held, pos, page)) return -1;
  return (int64_t)page * c.page_stride + (int64_t)(pos - (int)(pi * c.page_div.d)) * c.token_stride;
}

__device__ __forceinline__ int clamp_len(const CacheView& c, int len) {
  return len < 0 ? 0 : len > c.cap ? c.cap : len;
}

struct AttnArgs {
  CacheView c;
  const char* q;
  int64_t q_seq, q_node, q_head;  // bytes
  const uint8_t* mask;            // [B, N, N] or null (a chain)
  const int32_t* nodes;           // [B] or null (N each)
  int N, G;                       // nodes a sequence, query heads per kv head
  int mts;                        // row tiles of a (sequence, kv head)
  float scale;                    // > 0
  char* out;                      // [B, N, Hq, D]
  float* lse;                     // [B, N, Hq] or null
  int workers;                    // workgroups that share the key tiles
  float* part;                    // [workers][2][MT][D] unnormalised partial outputs
  float2* part_ml;                // [workers][2][MT] running maximum and sum of each row
  int4* tail;                     // [workers] the group whose first part is a worker's last
};

// What spec_tree_attention launches for a problem: rows per workgroup and workgroups.
struct AttnPlan {
  int row_tile;   // rows (node, query head) per workgroup
  int key_tile;   // keys per step
  int mts, workers;
  size_t o_ml, o_tail, bytes;  // workspace: part at 0
};

AttnPlan plan_tree_attention(const CacheView& c, sv_dtype dt, int N, int G);
hipError_t launch_tree_attention(const AttnArgs& a, sv_dtype dt, const AttnPlan& p,
                                 hipStream_t stream);

hipError_t launch_cache_append(const CacheView& c, const char* k_new, const char* v_new,
                               int64_t new_seq, int64_t new_node, int64_t new_head,
                               const int32_t* nodes, int N, hipStream_t stream);
hipError_t launch_cache_commit(const CacheView& c, const int32_t* parent, const int32_t* last,
                               int N, int32_t* out_lens, hipStream_t stream);
hipError_t launch_cache_resize(const CacheView& c, const int32_t* want, const int32_t* new_lens,
                               int32_t* out_ok, hipStream_t stream);
hipError_t launch_cache_fork(const CacheView& c, const int32_t* src, const int32_t* dst, int F,
                             int32_t* out_ok, hipStream_t stream);

}  // namespace sv
