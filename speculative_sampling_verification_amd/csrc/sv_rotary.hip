// Rotary positions on gfx950: pairs of columns of every query and key head turned by an angle
// proportional to the token's position, in place, into tensors, or (keys, with the values beside
// them) into a paged cache.
//
//   a = t w_p,  x' = s (x cos a - y sin a),  y' = s (x sin a + y cos a)
//
// for position t, pair p with frequency w_p and amplitude s; columns (p, p + half) are a pair, or
// (2 p, 2 p + 1) where they interleave.  Columns behind the 2 half turned ones are copied.
//
// Angles grow with the position, and what counts is their remainder: t w_p / (2 pi) is formed in
// 64 bits and brought to an eighth of a turn around a quarter there; sine and cosine of the rest
// (at most pi / 4) are Taylor sums in 32 bits.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "sv_step.hpp"

namespace sv {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotMaxBlocks = 1 << 20;

// sin and cos of `quarters` quarter turns.  |f| <= 1/2, so the sums end where the next term is
// below 2^-28: x^11 / 11! and x^12 / 12! at x = pi / 4 are 2e-9 and 2e-10.
__device__ __forceinline__ float2 turn(double quarters) {
  const double whole = rint(quarters);
  const float x = (float)(quarters - whole) * 1.57079632679489661923f, x2 = x * x;
  float s = fmaf(x2, 2.75573192e-6f, -1.98412698e-4f);  // 1/9!, 1/7!
  s = fmaf(x2, s, 8.33333333e-3f);
  s = fmaf(x2, s, -1.66666667e-1f);
  s = fmaf(x * x2, s, x);
  float c = fmaf(x2, -2.75573192e-7f, 2.48015873e-5f);  // 1/10!, 1/8!
  c = fmaf(x2, c, -1.38888889e-3f);
  c = fmaf(x2, c, 4.16666667e-2f);
  c = fmaf(x2, c, -0.5f);
  c = fmaf(x2, c, 1.0f);
  const int q = (int)(whole - 4.0 * floor(whole * 0.25));  // 0 .. 3
  const float sq = q & 1 ? c : s, cq = q & 1 ? s : c;
  return make_float2(q == 1 || q == 2 ? -cq : cq, q >= 2 ? -sq : sq);  // cos, sin
}

// A piece of W bytes of a row, and its elements as floats.
template <int W>
struct Bytes;
template <>
struct Bytes<16> { typedef uint32_t T __attribute__((ext_vector_type(4))); };
template <>
struct Bytes<8> { typedef uint32_t T __attribute__((ext_vector_type(2))); };
template <>
struct Bytes<4> { typedef uint32_t T; };
template <>
struct Bytes<2> { typedef uint16_t T; };

template <bool BF16, int W>
struct Piece {
  static constexpr int kN = W / (BF16 ? 2 : 4);
  union {
    typename Bytes<W>::T raw;
    __bf16 h[W / 2];
    float f[W >= 4 ? W / 4 : 1];
  };
  __device__ __forceinline__ float get(int i) const { return BF16 ? (float)h[i] : f[i]; }
  __device__ __forceinline__ void set(int i, float x) {
    if constexpr (BF16) h[i] = (__bf16)x;  // to the nearest, once
    else f[i] = x;
  }
};

template <int W>
__device__ __forceinline__ typename Bytes<W>::T load_bytes(const char* p) {
  return *reinterpret_cast<const typename Bytes<W>::T*>(p);
}
template <int W>
__device__ __forceinline__ void store_bytes(char* p, typename Bytes<W>::T x) {
  *reinterpret_cast<typename Bytes<W>::T*>(p) = x;
}

__device__ __forceinline__ int64_t row_in(const RowView& x, int b, int i, int h) {
  return (int64_t)b * x.seq + (int64_t)i * x.node + (int64_t)h * x.head;
}

// How a launch cuts the tokens' rows into a thread's units of work.
struct RotaryPlan {
  int tokens;            // of a workgroup
  int pair_units;        // units of a turned head that hold pairs ...
  int units;             // ... and all of them, the copied rest included
  int value_units;       // of a value head (16 bytes each)
  FastDiv token_div;     // units of a token: q_heads, k_heads, then v heads
  FastDiv unit_div, value_div, half_div, node_div;
};

// Units of W bytes: where a pair's columns lie `half` apart, one thread loads and stores the units of
// both, so that rows may be turned in place.  Sines and cosines of a workgroup's tokens are formed
// once for all heads and lie in LDS.
//
// Bound by memory, and by latency where there are few tokens: 16000 tokens of 32 + 8 heads of 128 in
// bf16 take 58 us, 5.7 TB/s; 64 tokens into the cache 4.9 us.  Rows loaded before the angles are there,
// in batches, took 15.7 -> 18.6 us for 2048 nodes into the cache (registers leave fewer waves), loads
// past the caches 15.6 -> 19.3; 512 threads 60 -> 73 us for the 16000 tokens.
template <bool BF16, int W, bool Inter, bool ToCache>
__global__ __launch_bounds__(kRotThreads) void k_rotary(RotaryArgs a, RotaryPlan p) {
  extern __shared__ float2 turns[];  // [tokens][half]: s cos, s sin
  __shared__ long long row_at[kRotThreads];
  constexpr int kES = BF16 ? 2 : 4;
  const int tid = threadIdx.x, all = a.seqs * a.N;
  for (int64_t first = (int64_t)blockIdx.x * p.tokens; first < all;
       first += (int64_t)gridDim.x * p.tokens) {
  const int token0 = (int)first, count = all - token0 < p.tokens ? all - token0 : p.tokens;
  for (int x = tid; x < count * a.half; x += kRotThreads) {
    const int t = (int)fast_div(p.half_div, (uint32_t)x), pair = x - t * a.half;
    const int b = (int)fast_div(p.node_div, (uint32_t)(token0 + t)), i = token0 + t - b * a.N;
    const int64_t at = (a.base ? (int64_t)a.base[b] : 0) +
                       (a.positions ? a.positions[token0 + t] : i);
    const float2 cs = turn((double)at * (a.freq[pair] * 0.63661977236758134308));  // 2 / pi
    turns[x] = make_float2(a.amplitude * cs.x, a.amplitude * cs.y);
  }
  // rows that the tokens' keys and values go to: -1 none, -2 a token that is not there
  for (int t = tid; t < count; t += kRotThreads) {
    const int b = (int)fast_div(p.node_div, (uint32_t)(token0 + t)), i = token0 + t - b * a.N;
    long long row = 0;
    if (a.nodes && i >= a.nodes[b]) row = -2;
    if constexpr (ToCache)
      if (row == 0) row = row_offset(a.c, b, positions_held(a.c, b), clamp_len(a.c, a.c.lens[b]) + i);
    row_at[t] = row;
  }
  __syncthreads();
  const uint32_t work = (uint32_t)count * p.token_div.d;
  for (uint32_t x = tid; x < work; x += kRotThreads) {
    const int t = (int)fast_div(p.token_div, x);
    const long long row = row_at[t];
    if (row == -2) continue;
    const int b = (int)fast_div(p.node_div, (uint32_t)(token0 + t)), i = token0 + t - b * a.N;
    uint32_t u = x - (uint32_t)t * p.token_div.d;
    const int turned = (a.q_heads + a.k_heads) * p.units;
    if (ToCache && (int)u >= turned) {  // values
      u -= turned;
      const int h = (int)fast_div(p.value_div, u), at = (int)(u - h * p.value_div.d) * 16;
      if (row < 0) continue;
      store_bytes<16>(a.c.v + row + (int64_t)h * a.c.head_stride + at,
                      load_bytes<16>(a.v.at + row_in(a.v, b, i, h) + at));
      continue;
    }
    int h = (int)fast_div(p.unit_div, u);
    const int unit = (int)(u - h * p.unit_div.d);
    const bool key = h >= a.q_heads;
    h -= key ? a.q_heads : 0;
    const RowView& from = key ? a.k : a.q;
    const char* src = from.at + row_in(from, b, i, h);
    char* dst;
    if (ToCache && key) {
      if (row < 0) continue;
      dst = a.c.k + row + (int64_t)h * a.c.head_stride;
    } else {
      const RowView& to = key ? a.k_out : a.q_out;
      dst = const_cast<char*>(to.at) + row_in(to, b, i, h);
    }
    const float2* cs = turns + t * a.half;
    Piece<BF16, W> lo, hi;
    if (unit >= p.pair_units) {  // behind the turned columns
      if (src == dst) continue;
      const int at = Inter ? unit * W : (unit + p.pair_units) * W;
      lo.raw = load_bytes<W>(src + at);
      store_bytes<W>(dst + at, lo.raw);
    } else if constexpr (Inter) {
      lo.raw = load_bytes<W>(src + unit * W);
      const int pair = unit * (W / kES / 2);
#pragma unroll
      for (int e = 0; e + 1 < lo.kN; e += 2) {
        if (pair + e / 2 >= a.half) break;
        const float2 w = cs[pair + e / 2];
        const float fx = lo.get(e), fy = lo.get(e + 1);
        lo.set(e, fmaf(fx, w.x, -fy * w.y));
        lo.set(e + 1, fmaf(fx, w.y, fy * w.x));
      }
      store_bytes<W>(dst + unit * W, lo.raw);
    } else {
      const int apart = a.half * kES;
      lo.raw = load_bytes<W>(src + unit * W);
      hi.raw = load_bytes<W>(src + unit * W + apart);
      const int pair = unit * (W / kES);
#pragma unroll
      for (int e = 0; e < lo.kN; ++e) {
        const float2 w = cs[pair + e];
        const float fx = lo.get(e), fy = hi.get(e);
        lo.set(e, fmaf(fx, w.x, -fy * w.y));
        hi.set(e, fmaf(fx, w.y, fy * w.x));
      }
      store_bytes<W>(dst + unit * W, lo.raw);
      store_bytes<W>(dst + unit * W + apart, hi.raw);
    }
  }
  __syncthreads();  // before the next tokens' turns
  }
}

template <bool BF16, int W, bool Inter>
void launch(const RotaryArgs& a, bool to_cache, hipStream_t stream) {
  constexpr int kES = BF16 ? 2 : 4;
  RotaryPlan p{};
  const int turned = 2 * a.half * kES;  // bytes
  if (Inter) {
    p.units = a.row / W;
    p.pair_units = (turned + W - 1) / W;
  } else {
    p.pair_units = turned / 2 / W;
    p.units = p.pair_units + (a.row - turned) / W;
  }
  p.value_units = a.row / 16;
  const int units = (a.q_heads + a.k_heads) * p.units + (to_cache ? a.k_heads * p.value_units : 0);
  // two tokens where 1024 workgroups remain: 2048 nodes into the cache 15.6 -> 14.4 us, 16000 tokens
  // 60.0 -> 57.7; 64 tokens 10.5 -> 11.0, and with four of them 2048 nodes take 18.2
  p.tokens = (int64_t)a.seqs * a.N >= 2048 ? 2 : 1;
  p.token_div = make_fast_div((uint32_t)units);
  p.unit_div = make_fast_div((uint32_t)p.units);
  p.value_div = make_fast_div((uint32_t)p.value_units);
  p.half_div = make_fast_div((uint32_t)a.half);
  p.node_div = make_fast_div((uint32_t)a.N);
  const int64_t groups = ((int64_t)a.seqs * a.N + p.tokens - 1) / p.tokens;
  const unsigned blocks = (unsigned)(groups < kRotMaxBlocks ? groups : kRotMaxBlocks);
  const size_t lds = (size_t)p.tokens * a.half * sizeof(float2);
  if (to_cache)
    hipLaunchKernelGGL((k_rotary<BF16, W, Inter, true>), dim3(blocks), dim3(kRotThreads), lds,
                       stream, a, p);
  else
    hipLaunchKernelGGL((k_rotary<BF16, W, Inter, false>), dim3(blocks), dim3(kRotThreads), lds,
                       stream, a, p);
}

template <bool BF16>
void launch_for(const RotaryArgs& a, bool interleaved, bool to_cache, hipStream_t stream) {
  const int apart = a.half * (BF16 ? 2 : 4);  // bytes between the halves
  if (interleaved) launch<BF16, 16, true>(a, to_cache, stream);
  else if (apart % 16 == 0) launch<BF16, 16, false>(a, to_cache, stream);
  else if (apart % 8 == 0) launch<BF16, 8, false>(a, to_cache, stream);
  else if (apart % 4 == 0) launch<BF16, 4, false>(a, to_cache, stream);
  else if constexpr (BF16) launch<BF16, 2, false>(a, to_cache, stream);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, sv_dtype dt, bool interleaved, bool to_cache,
                         hipStream_t stream) {
  if (dt == SV_DTYPE_BF16) launch_for<true>(a, interleaved, to_cache, stream);
  else launch_for<false>(a, interleaved, to_cache, stream);
  return hipGetLastError();
}

}  // namespace sv
