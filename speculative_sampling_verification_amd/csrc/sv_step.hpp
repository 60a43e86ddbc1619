// Declarations of what a decoding step does around tree attention: rotary positions
// (sv_rotary.hip), attention weights of the committed tokens and their eviction (sv_evict.hip).
// The C entry points are in sv_step_abi.hip.
#pragma once

#include "sv_cache.hpp"

namespace sv {

// Rows of one tensor [seqs, N, heads, head_dim]: strides in bytes.
struct RowView {
  const char* at;
  int64_t seq, node, head;
};

struct RotaryArgs {
  RowView q, k, v;       // sources; v is only copied
  RowView q_out, k_out;  // targets (k_out unused where keys go to the cache)
  int q_heads, k_heads;  // 0: not given
  int row;               // bytes of a head
  int half;              // pairs turned
  int seqs, N;
  const double* freq;    // [half]: radians a position
  float amplitude;
  const int32_t* base;       // [seqs] or null: 0
  const int32_t* positions;  // [seqs, N] or null: 0 .. N - 1
  const int32_t* nodes;      // [seqs] or null: N each
  CacheView c;               // where keys and values go (to_cache)
};

hipError_t launch_rotary(const RotaryArgs& a, sv_dtype dt, bool interleaved, bool to_cache,
                         hipStream_t stream);

struct WeighArgs {
  CacheView c;  // one layer
  RowView q;
  const float* lse;      // [seqs, N, G kv_heads]
  const int32_t* seen;   // [seqs, N] or null: every committed token
  const int32_t* nodes;  // [seqs] or null: N each
  int N, G;
  FastDiv g_div;         // by G
  float scale, decay;
  float* w;              // [seqs, kv_heads, length]
  int length;
};

hipError_t launch_cache_weigh(const WeighArgs& a, sv_dtype dt, hipStream_t stream);

struct EvictArgs {
  CacheView c;  // all layers
  const float* w;  // [layers, seqs, kv_heads, length]
  float* out_w;    // w itself, or apart from it
  int length;
  const int32_t* keep;  // [seqs]
  int max_keep, sinks, recent;
  int32_t* out_lens;  // [seqs]
  int32_t* kept;      // [layers, seqs, kv_heads, max_keep]
};

hipError_t launch_cache_evict(const EvictArgs& a, hipStream_t stream);

}  // namespace sv
