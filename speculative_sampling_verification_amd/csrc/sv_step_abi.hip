// extern "C" entry points of what a decoding step does around tree attention: rotary positions,
// attention weights of the committed tokens, eviction.  Host-side argument checks and dispatch; no
// allocation, no synchronisation.  See include/spec_verify.h for the contract of each function.

#include <cmath>

#include "sv_cache_check.hpp"
#include "sv_step.hpp"

using namespace sv;

namespace {

constexpr uint64_t kMaxWeights = (uint64_t)1 << 60;  // an array of attention weights
constexpr double kTurn = 6.283185307179586476925;  // 2 pi

bool dtype_ok(sv_dtype dt) { return dt == SV_DTYPE_F32 || dt == SV_DTYPE_BF16; }

// Strided rows [seqs, N, heads, head_dim] of an argument and the bytes from the first to behind the last.
struct Rows {
  int64_t s[3];
  int64_t size[3];
  int64_t row;
  uint64_t bytes;
};

bool rows_of(const int64_t* strides, int seqs, int N, int heads, int D, int es, Rows* r) {
  if (!row_strides(strides, N, heads, D, es, r->s)) return false;
  r->size[0] = seqs;
  r->size[1] = N;
  r->size[2] = heads;
  r->row = (int64_t)D * es;
  return extent_of(r->row, r->s, r->size, &r->bytes);
}

RowView view_rows(const void* at, const Rows& r) {
  return RowView{static_cast<const char*>(at), r.s[0], r.s[1], r.s[2]};
}

// Whether rows that are written in place share no memory with other rows.  Apart as a whole, or
// parts of one tensor whose tokens lie alike (queries, keys and values made by one product): then
// a token's part of either has to end before the other's begins.
bool parts_apart(const void* a, const Rows& x, const void* b, const Rows& y) {
  if (!a || !b || !overlap(a, x.bytes, b, y.bytes)) return true;
  for (int i = 0; i < 2; ++i)
    if (x.size[i] > 1 && x.s[i] != y.s[i]) return false;
  const int64_t p = (int64_t)reinterpret_cast<uintptr_t>(a);
  const int64_t q = (int64_t)reinterpret_cast<uintptr_t>(b);
  const int64_t span_x = x.s[2] * (x.size[2] - 1) + x.row, span_y = y.s[2] * (y.size[2] - 1) + y.row;
  const int64_t gap = p < q ? q - p : p - q;
  if (gap < (p < q ? span_x : span_y)) return false;
  const int64_t stride[2] = {x.s[0], x.s[1]}, size[2] = {x.size[0], x.size[1]};
  int64_t both;
  return !__builtin_add_overflow(gap, p < q ? span_y : span_x, &both) &&
         rows_apart(both, stride, size);
}

bool in_place_ok(const Rows& x) {
  return rows_apart(x.row, x.s, x.size);
}

struct RotaryCall {
  const void* q;
  const int64_t* q_strides;
  int q_heads;
  void* q_out;
  const void* k;
  const int64_t* k_strides;
  int k_heads;
  void* k_out;
  const void* v;
  sv_dtype dtype;
  int seqs, N, head_dim;
  const double* freq;
  int rot_dim, interleaved;
  float amplitude;
  const int32_t *base, *positions, *nodes;
};

// Checks that both entry points share and the kernel's arguments.  `more` are arrays that the call
// reads besides, written[] what it writes besides.
int rotary_args(const RotaryCall& r, const Range (&written)[2], const Range (&more)[4],
                RotaryArgs* a) {
  if (!dtype_ok(r.dtype)) return SV_ERR_UNSUPPORTED_DTYPE;
  const int es = r.dtype == SV_DTYPE_BF16 ? 2 : 4;
  if (r.seqs < 1 || r.N < 1 || (int64_t)r.seqs * r.N > INT_MAX) return SV_ERR_INVALID_ARG;
  if (r.head_dim < 1 || r.head_dim > kMaxHeadBytes / es || (r.head_dim * es) % 16 != 0)
    return SV_ERR_INVALID_ARG;
  if (!r.freq || r.rot_dim < 2 || r.rot_dim % 2 != 0 || r.rot_dim > r.head_dim)
    return SV_ERR_INVALID_ARG;
  if (r.interleaved != 0 && r.interleaved != 1) return SV_ERR_INVALID_ARG;
  if (!std::isfinite(r.amplitude)) return SV_ERR_INVALID_ARG;
  if (r.q_heads < 0 || r.k_heads < 0 || r.q_heads > 64 * kMaxHeads || r.k_heads > 64 * kMaxHeads ||
      r.q_heads + r.k_heads < 1)
    return SV_ERR_INVALID_ARG;
  if ((r.q_heads > 0) != (r.q != nullptr) || (r.q_heads > 0) != (r.q_out != nullptr) ||
      (r.k_heads > 0) != (r.k != nullptr))
    return SV_ERR_INVALID_ARG;
  if (!aligned_to(r.q, 16) || !aligned_to(r.q_out, 16) || !aligned_to(r.k, 16) ||
      !aligned_to(r.k_out, 16) || !aligned_to(r.v, 16) || !aligned_to(r.freq, 8) ||
      !aligned_to(r.base, 4) || !aligned_to(r.positions, 4) || !aligned_to(r.nodes, 4))
    return SV_ERR_INVALID_ARG;
  Rows q{}, k{}, v{}, dense_q{}, dense_k{};
  if (r.q_heads && (!rows_of(r.q_strides, r.seqs, r.N, r.q_heads, r.head_dim, es, &q) ||
                    !rows_of(nullptr, r.seqs, r.N, r.q_heads, r.head_dim, es, &dense_q)))
    return SV_ERR_INVALID_ARG;
  if (r.k_heads && (!rows_of(r.k_strides, r.seqs, r.N, r.k_heads, r.head_dim, es, &k) ||
                    !rows_of(nullptr, r.seqs, r.N, r.k_heads, r.head_dim, es, &dense_k)))
    return SV_ERR_INVALID_ARG;
  v = k;
  // what is written lies apart from all else, or is the rows that are read, in place
  const bool q_here = r.q && r.q_out == r.q, k_here = r.k && r.k_out == r.k;
  const Rows& qo = q_here ? q : dense_q;
  const Rows& ko = k_here ? k : dense_k;
  if ((q_here && !in_place_ok(q)) || (k_here && !in_place_ok(k))) return SV_ERR_INVALID_ARG;
  if (!parts_apart(r.q_out, qo, r.k_out, ko)) return SV_ERR_INVALID_ARG;
  if ((!q_here && !parts_apart(r.q_out, qo, r.q, q)) || !parts_apart(r.q_out, qo, r.k, k) ||
      !parts_apart(r.q_out, qo, r.v, v))
    return SV_ERR_INVALID_ARG;
  if ((!k_here && !parts_apart(r.k_out, ko, r.k, k)) || !parts_apart(r.k_out, ko, r.q, q))
    return SV_ERR_INVALID_ARG;
  const uint64_t word = sizeof(int32_t);
  const Range ranges[] = {{r.q_out, qo.bytes}, {r.k_out, ko.bytes}, written[0], written[1],
                          {r.freq, sizeof(double) * (uint64_t)(r.rot_dim / 2)},
                          {r.base, word * r.seqs}, {r.positions, word * r.seqs * r.N},
                          {r.nodes, word * r.seqs}, more[0], more[1], more[2], more[3]};
  // the first four are written; q_out and k_out against each other are looked at above
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 12; ++j)
      if (!(i == 0 && j == 1) && overlap(ranges[i].at, ranges[i].bytes, ranges[j].at, ranges[j].bytes))
        return SV_ERR_INVALID_ARG;
  for (const Range& w : written)
    if (overlap(w.at, w.bytes, r.q, q.bytes) || overlap(w.at, w.bytes, r.k, k.bytes) ||
        overlap(w.at, w.bytes, r.v, v.bytes))
      return SV_ERR_INVALID_ARG;
  a->q = view_rows(r.q, q);
  a->k = view_rows(r.k, k);
  a->v = view_rows(r.v, v);
  a->q_out = view_rows(r.q_out, qo);
  a->k_out = view_rows(r.k_out, ko);
  a->q_heads = r.q_heads;
  a->k_heads = r.k_heads;
  a->row = r.head_dim * es;
  a->half = r.rot_dim / 2;
  a->seqs = r.seqs;
  a->N = r.N;
  a->freq = r.freq;
  a->amplitude = r.amplitude;
  a->base = r.base;
  a->positions = r.positions;
  a->nodes = r.nodes;
  return SV_OK;
}

}  // namespace

extern "C" {

int spec_rotary(const void* q, const int64_t* q_strides, int q_heads, void* out_q, const void* k,
                const int64_t* k_strides, int k_heads, void* out_k, sv_dtype dtype, int seqs, int N,
                int head_dim, const double* inv_freq, int rot_dim, int interleaved, float amplitude,
                const int32_t* base, const int32_t* positions, hipStream_t stream) {
  if ((k_heads > 0) != (out_k != nullptr)) return SV_ERR_INVALID_ARG;
  const RotaryCall r{q, q_strides, q_heads, out_q, k, k_strides, k_heads, out_k, nullptr, dtype,
                     seqs, N, head_dim, inv_freq, rot_dim, interleaved, amplitude, base, positions,
                     nullptr};
  RotaryArgs a{};
  const int st = rotary_args(r, {}, {}, &a);
  if (st != SV_OK) return st;
  return status_of(launch_rotary(a, dtype, interleaved != 0, false, stream));
}

int spec_rotary_append(const void* q, const int64_t* q_strides, int q_heads, void* out_q,
                       const void* k_new, const void* v_new, const int64_t* new_strides, int N,
                       const sv_cache* cache, int layer, const int32_t* num_nodes,
                       const double* inv_freq, int rot_dim, int interleaved, float amplitude,
                       const int32_t* base, const int32_t* positions, hipStream_t stream) {
  RotaryArgs a{};
  const int st = view_of(cache, layer, 1, &a.c);
  if (st != SV_OK) return st;
  if (!values_apart(cache) || !k_new || !v_new || N > kCacheMaxNodes) return SV_ERR_INVALID_ARG;
  const CacheView& v = a.c;
  const int64_t row = (int64_t)v.head_dim * v.esize;
  const int64_t stride[3] = {v.page_stride, v.token_stride, v.head_stride};
  const int64_t size[3] = {v.pages, v.page_size, v.kv_heads};
  uint64_t bytes;
  if (!extent_of(row, stride, size, &bytes)) return SV_ERR_INVALID_ARG;
  const RotaryCall r{q, q_strides, q_heads, out_q, k_new, new_strides, cache->kv_heads, nullptr,
                     v_new, cache->dtype, v.seqs, N, v.head_dim, inv_freq, rot_dim, interleaved,
                     amplitude, base ? base : v.lens, positions, num_nodes};
  const uint64_t word = sizeof(int32_t);
  // keys and values may be parts of one tensor, whose rows lie apart
  const Range written[2] = {{v.k, bytes}, {nullptr, 0}};
  const Range more[4] = {{v.table, word * v.seqs * v.width}, {v.lens, word * v.seqs},
                         {v.held, word * v.seqs}, {v.refcount, word * v.pages}};
  const int bad = rotary_args(r, written, more, &a);
  if (bad != SV_OK) return bad;
  RotaryArgs unused{};
  const Range values[2] = {{v.v, bytes}, {nullptr, 0}};
  const int bad_values = rotary_args(r, values, more, &unused);
  if (bad_values != SV_OK) return bad_values;
  return status_of(launch_rotary(a, cache->dtype, interleaved != 0, true, stream));
}

int spec_cache_weigh(const void* q, const int64_t* q_strides, int N, int q_heads, const float* lse,
                     const sv_cache* cache, int layer, const int32_t* seen,
                     const int32_t* num_nodes, float scale, float decay, float* weights, int length,
                     hipStream_t stream) {
  WeighArgs a{};
  const int st = view_of(cache, layer, 1, &a.c);
  if (st != SV_OK) return st;
  const CacheView& v = a.c;
  if (!q || !lse || !weights || !attn_shape(cache, N, q_heads)) return SV_ERR_INVALID_ARG;
  if (length < 1 || length > kCacheMaxTokens) return SV_ERR_INVALID_ARG;
  // the kernel multiplies scores by scale * log2(e)
  if (!(scale > 0.0f) || !std::isfinite(scale * 1.44269504088896340736f)) return SV_ERR_INVALID_ARG;
  if (!(decay >= 0.0f && decay <= 1.0f)) return SV_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(lse, 4) || !aligned_to(weights, 4) ||
      !aligned_to(seen, 4) || !aligned_to(num_nodes, 4))
    return SV_ERR_INVALID_ARG;
  Rows r{};
  if (!rows_of(q_strides, v.seqs, N, q_heads, v.head_dim, v.esize, &r)) return SV_ERR_INVALID_ARG;
  const int64_t row = (int64_t)v.head_dim * v.esize;
  const int64_t stride[3] = {v.page_stride, v.token_stride, v.head_stride};
  const int64_t size[3] = {v.pages, v.page_size, v.kv_heads};
  uint64_t bytes;
  if (!extent_of(row, stride, size, &bytes)) return SV_ERR_INVALID_ARG;
  const uint64_t word = sizeof(int32_t);
  const uint64_t slab = (uint64_t)v.seqs * v.kv_heads * length;  // at most 2^53
  if (slab > kMaxWeights / cache->layers) return SV_ERR_INVALID_ARG;
  const Range ranges[] = {{weights + slab * layer, word * slab}, {q, r.bytes},
                          {lse, word * v.seqs * N * q_heads}, {seen, word * v.seqs * N},
                          {num_nodes, word * v.seqs}, {v.k, bytes},
                          {v.table, word * v.seqs * v.width}, {v.lens, word * v.seqs},
                          {v.held, word * v.seqs}, {v.refcount, word * v.pages}};
  if (!outputs_apart(ranges, 1)) return SV_ERR_INVALID_ARG;
  a.q = view_rows(q, r);
  a.lse = lse;
  a.seen = seen;
  a.nodes = num_nodes;
  a.N = N;
  a.G = q_heads / v.kv_heads;
  a.g_div = make_fast_div((uint32_t)a.G);
  a.scale = scale;
  a.decay = decay;
  a.w = weights + slab * layer;
  a.length = length;
  return status_of(launch_cache_weigh(a, cache->dtype, stream));
}

int spec_cache_evict(const sv_cache* cache, const float* weights, int length, const int32_t* keep,
                     int max_keep, int sinks, int recent, float* out_weights, int32_t* out_lens,
                     int32_t* out_kept, hipStream_t stream) {
  EvictArgs a{};
  const int st = view_of(cache, 0, cache ? cache->layers : 0, &a.c);
  if (st != SV_OK) return st;
  const CacheView& v = a.c;
  if (!values_apart(cache) || !weights || !keep || !out_weights || !out_lens || !out_kept)
    return SV_ERR_INVALID_ARG;
  if (length < 1 || length > kCacheMaxTokens || max_keep < 1 || max_keep > length || sinks < 0 ||
      recent < 0)
    return SV_ERR_INVALID_ARG;
  if (!aligned_to(weights, 4) || !aligned_to(keep, 4) || !aligned_to(out_weights, 4) ||
      !aligned_to(out_lens, 4) || !aligned_to(out_kept, 4))
    return SV_ERR_INVALID_ARG;
  const int64_t row = (int64_t)v.head_dim * v.esize;
  const int64_t stride[4] = {v.layer_stride, v.page_stride, v.token_stride, v.head_stride};
  const int64_t size[4] = {v.layers, v.pages, v.page_size, v.kv_heads};
  uint64_t bytes, groups;
  if (!extent_of(row, stride, size, &bytes)) return SV_ERR_INVALID_ARG;
  groups = (uint64_t)v.layers * v.seqs * v.kv_heads;  // at most 2^36
  if (groups > kMaxWeights / length) return SV_ERR_INVALID_ARG;
  const uint64_t word = sizeof(int32_t), all = word * groups * length;
  const bool in_place = out_weights == weights;
  const Range ranges[] = {{out_weights, all}, {out_lens, word * v.seqs},
                          {out_kept, word * groups * max_keep}, {v.k, bytes}, {keep, word * v.seqs},
                          {in_place ? nullptr : weights, all},
                          {v.table, word * v.seqs * v.width}, {v.lens, word * v.seqs},
                          {v.held, word * v.seqs}, {v.refcount, word * v.pages}};
  const Range values[] = {{v.v, bytes}, {out_weights, all}, {out_lens, word * v.seqs},
                          {out_kept, word * groups * max_keep}, {keep, word * v.seqs},
                          {weights, all}, {v.table, word * v.seqs * v.width},
                          {v.lens, word * v.seqs}, {v.held, word * v.seqs},
                          {v.refcount, word * v.pages}};
  // keys and values may be parts of one tensor, whose rows lie apart
  if (!outputs_apart(ranges, 4) || !outputs_apart(values, 1)) return SV_ERR_INVALID_ARG;
  a.w = weights;
  a.out_w = out_weights;
  a.length = length;
  a.keep = keep;
  a.max_keep = max_keep;
  a.sinks = sinks;
  a.recent = recent;
  a.out_lens = out_lens;
  a.kept = out_kept;
  return status_of(launch_cache_evict(a, stream));
}

int spec_rotary_frequencies(int rot_dim, double theta, int scaling, double factor,
                            double original_length, double beta_fast, double beta_slow,
                            double* out_inv_freq, float* out_amplitude) {
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 4096 || !out_inv_freq) return SV_ERR_INVALID_ARG;
  if (!(theta > 0.0) || !std::isfinite(theta)) return SV_ERR_INVALID_ARG;
  if (scaling < SV_ROTARY_PLAIN || scaling > SV_ROTARY_YARN) return SV_ERR_INVALID_ARG;
  if (scaling != SV_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return SV_ERR_INVALID_ARG;
  if (scaling == SV_ROTARY_YARN &&
      (!(original_length > 0.0) || !std::isfinite(original_length) || !(beta_slow >= 0.0) ||
       !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
    return SV_ERR_INVALID_ARG;
  const int half = rot_dim / 2;
  // the slowest pair is stretched by the factor, the fastest not at all
  if (scaling == SV_ROTARY_NTK && half > 1) theta *= std::pow(factor, (double)half / (half - 1));
  for (int p = 0; p < half; ++p) {
    double f = std::pow(theta, -(double)p / half);
    if (scaling == SV_ROTARY_LINEAR) {
      f /= factor;
    } else if (scaling == SV_ROTARY_YARN) {
      const double turns = original_length * f / kTurn;
      const double keep = std::fmin(1.0, std::fmax(0.0, (turns - beta_slow) / (beta_fast - beta_slow)));
      f = (1.0 - keep) * f / factor + keep * f;
    }
    out_inv_freq[p] = f;
  }
  if (out_amplitude)
    *out_amplitude = scaling == SV_ROTARY_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return SV_OK;
}

}  // extern "C"
