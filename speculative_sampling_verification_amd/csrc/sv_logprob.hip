// Log probabilities of given tokens on gfx950, with the entropy of their distributions, the tokens'
// ranks and the most probable alternatives, in one pass over the logits.
//
// With x = z log2(e) / T, a shift k and S = sum 2^(x - k), X = sum 2^(x - k) (x - k):
//   log p(t) = ln2 (x_t - k) - ln S,   H = ln S - ln2 X / S
// k is never far below the largest x so far: H is the difference of two numbers that both grow with
// that distance, and S and X take their rounding errors from it.  Sums are in fp32 a lane, joined in
// 64 bits.
//
// Alternatives: the top n elements (larger first, ties to the lower index) lie in the n vectors of
// 16 bytes that come first by (their largest element, position): an element of another vector comes
// behind the largest of each of these.  So the pass only keeps vectors whose maximum, which the
// shift needs anyway, beats the wave's n-th so far; a wave meets its vectors in order of position,
// so a tie never does.  The kept vectors' elements are ranked at the end.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "sv_logprob.hpp"

namespace sv {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kVecs = 4;              // vectors a thread and tile
constexpr int kTile = kThreads * kVecs;
constexpr int kSpare = 48;            // vectors a wave keeps beyond n until it cuts its list
constexpr int kList = kLogprobMaxTop + kSpare + 64 * kVecs;
constexpr int kMaxParts = 64;         // of a row: one a lane of the join
constexpr int64_t kMaxBlocks = 1 << 20;
constexpr float kRise = 2.0f;         // how far x may lie above the shift
constexpr double kLn2 = 0.69314718055994530942;

// Every lambda of the kernel is part of its loop: the captures of one that the compiler calls
// instead are kept in memory.
#define SV_INLINE __attribute__((always_inline))

// Order-preserving key of a logit (the two zeros alike) and its inverse.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t u = __float_as_uint(z == 0.0f ? 0.0f : z);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

template <bool BF16>
struct Row {
  static constexpr int kES = BF16 ? 2 : 4;
  static constexpr int kPer = 16 / kES;  // elements a vector
  const char* at;    // aligned start: vector 0 may begin before the row
  int phase;         // elements of vector 0 that lie before the row
  int V;
  int first, last;   // vectors first .. last - 1 lie in the row as a whole
  int head;          // elements of the row before them; behind them: from tail() on

  __device__ __forceinline__ Row(const char* row, int V_) : V(V_) {
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
    at = row - off;
    phase = (int)off / kES;
    first = phase ? 1 : 0;
    last = (int)(((int64_t)phase + V) / kPer);
    head = !phase ? 0 : V < kPer - phase ? V : kPer - phase;
    if (last < first) last = first;
  }
  __device__ __forceinline__ int64_t tail() const {
    const int64_t i = (int64_t)last * kPer - phase;
    return i > head ? i : head;
  }
  __device__ __forceinline__ float load(int64_t i) const {
    const char* p = at + (i + phase) * kES;
    if constexpr (BF16)
      return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
    else
      return *reinterpret_cast<const float*>(p);
  }
  static __device__ __forceinline__ float elem(const u32x4& v, int e) {
    if constexpr (BF16) return __uint_as_float(e & 1 ? v[e >> 1] & 0xFFFF0000u : v[e >> 1] << 16);
    else return __uint_as_float(v[e]);
  }
};

// A value of the lane that a DPP control names, and of a given lane.
template <int Control, class T>
__device__ __forceinline__ T across(T x) {
  int w[sizeof(T) / 4];
  __builtin_memcpy(w, &x, sizeof(T));
#pragma unroll
  for (int& y : w) y = __builtin_amdgcn_update_dpp(y, y, Control, 0xF, 0xF, false);
  __builtin_memcpy(&x, w, sizeof(T));
  return x;
}
template <class T>
__device__ __forceinline__ T of_lane(T x, int lane) {
  int w[sizeof(T) / 4];
  __builtin_memcpy(w, &x, sizeof(T));
#pragma unroll
  for (int& y : w) y = __builtin_amdgcn_readlane(y, lane);
  __builtin_memcpy(&x, w, sizeof(T));
  return x;
}

// op over four neighbouring lanes, and over the wave (all lanes active): within rows of 16 lanes
// by DPP (neighbours, pairs, then halves mirrored), the four rows as scalars.
template <class T, class Op>
__device__ __forceinline__ T quad_all(T x, Op op) {
  x = op(x, across<0xB1>(x));  // lanes 1 0 3 2
  return op(x, across<0x4E>(x));  // lanes 2 3 0 1
}
template <class T, class Op>
__device__ __forceinline__ T wave_all(T x, Op op) {
  x = quad_all(x, op);
  x = op(x, across<0x141>(x));  // 7 .. 0 of each 8
  x = op(x, across<0x140>(x));  // 15 .. 0 of each 16
  return op(op(of_lane(x, 0), of_lane(x, 16)), op(of_lane(x, 32), of_lane(x, 48)));
}

// The n-th largest of the wave's keys, several a lane (the largest k with n keys >= k).  Keys of
// bf16 are told apart by their upper halves: half as many steps.
template <bool BF16, int Keys>
__device__ __forceinline__ uint32_t nth_key(const uint32_t (&k)[Keys], int n) {
  uint32_t t = 0;
#pragma unroll 1
  for (uint32_t bit = 0x80000000u; bit >= (BF16 ? 0x10000u : 1u); bit >>= 1) {
    const uint32_t c = t | bit;
    int count = 0;
#pragma unroll
    for (int i = 0; i < Keys; ++i) count += __popcll(__ballot(k[i] >= c));
    if (count >= n) t = c;
  }
  return BF16 && !(t & 0x80000000u) && t ? t | 0xFFFFu : t;  // a negative number's lower half
}

struct Lds {
  float val[kWaves][kList];
  uint32_t pos[kWaves][kList];
  unsigned long long keys[kWaves][kLogprobMaxTop];
  unsigned long long edge[2];  // the row's first and last vector where they are not whole
  unsigned long long picked[kLogprobMaxTop];
  unsigned long long elems[kLogprobMaxTop * 8];
  LogprobPart stat[kWaves];
  int count[kWaves];
  int found, near;
};

// Vectors that a wave keeps, in order of position.
template <bool BF16>
struct Kept {
  float* val;
  uint32_t* pos;
  int count;
  float tau;  // vectors count only above it

  // keeps the n first by (value, position)
  template <int Keys>
  __device__ __forceinline__ void cut_some(int n) {
    const int lane = threadIdx.x & 63;
    uint32_t k[Keys], p[Keys];
#pragma unroll
    for (int i = 0; i < Keys; ++i) {
      const int at = lane + 64 * i;
      k[i] = at < count ? key_of(val[at]) : 0u;
      p[i] = at < count ? pos[at] : 0u;
    }
    const uint32_t t = nth_key<BF16>(k, n);
    const unsigned long long below = (1ull << lane) - 1;
    int quota = n;
#pragma unroll
    for (int i = 0; i < Keys; ++i) quota -= __popcll(__ballot(k[i] > t));
    __builtin_amdgcn_wave_barrier();
    int at = 0, level_before = 0;
#pragma unroll
    for (int i = 0; i < Keys; ++i) {
      const unsigned long long level = __ballot(k[i] == t);
      const bool take = k[i] > t || (k[i] == t && level_before + __popcll(level & below) < quota);
      const unsigned long long m = __ballot(take);
      if (take) {
        val[at + __popcll(m & below)] = of_key(k[i]);
        pos[at + __popcll(m & below)] = p[i];
      }
      at += __popcll(m);
      level_before += __popcll(level);
    }
    __builtin_amdgcn_wave_barrier();
    count = n;
    tau = of_key(t);
  }
  __device__ __forceinline__ void cut(int n) {
    __builtin_amdgcn_wave_barrier();
    if (count <= 128) cut_some<2>(n);
    else cut_some<(kList + 63) / 64>(n);
  }

  __device__ __forceinline__ void add(bool hit, float v, uint32_t p) {
    const unsigned long long m = __ballot(hit);
    if (!m) return;
    const int at = count + __popcll(m & ((1ull << (threadIdx.x & 63)) - 1));
    if (hit) {
      val[at] = v;
      pos[at] = p;
    }
    count += __popcll(m);
  }
};

// Parts, one a lane, on one shift: all(x, op) is op over the lanes that hold them.  In 64 bits, as 1
// less a row's largest probability may be far below half a step of fp32.
template <class All>
__device__ __forceinline__ LogprobPart joined(LogprobPart r, All all) {
  const double own = r.shift;
  r.shift = all(own, [](double x, double y) { return x > y ? x : y; });
  double sum = 0.0, sum_x = 0.0;
  if (own > -INFINITY) {  // there is a finite logit
    const double d = own - r.shift;
    const double f = exp2(d);
    sum = f * r.sum;
    if (f > 0.0) sum_x = f * (r.sum_x + d * r.sum);
  }
  auto add = [](auto x, auto y) { return x + y; };
  r.sum = all(sum, add);
  r.sum_x = all(sum_x, add);
  r.top = all(r.top, [](float x, float y) { return fmaxf(x, y); });
  r.above = all(r.above, add);
  return r;
}

// A row's results from its statistics and, in s.picked, the keys (largest element, ~position) of
// its first s.found vectors.
template <bool BF16>
__device__ __forceinline__ void finish(const LogprobArgs& a, Lds& s, const Row<BF16>* row, int r,
                       const LogprobPart& st, int token) {
  const int tid = threadIdx.x;
  const bool some = row && st.top > -INFINITY;
  const double ln_s = some ? log(st.sum) : 0.0;
  auto logprob = [&](float z) -> float {
    return some ? (float)(kLn2 * ((double)a.c * z - st.shift) - ln_s) : -INFINITY;
  };
  if (tid == 0) {
    const bool valid = row && token >= 0 && token < a.V;
    if (a.logprob) a.logprob[r] = valid ? logprob(row->load(token)) : -INFINITY;
    if (a.rank) a.rank[r] = valid ? st.above : -1;
    if (a.entropy) {
      const double h = some ? ln_s - kLn2 * st.sum_x / st.sum : 0.0;
      a.entropy[r] = (float)(h > 0.0 ? h : 0.0);
    }
  }
  if (!a.n) return;
  const int vecs = some ? s.found : 0, all = vecs * Row<BF16>::kPer;
  if (tid == 0) s.near = 0;
  __syncthreads();
  // elements that may be among the first: no less than the last vector's largest where there are n
  // vectors; in no order, as their keys are all different
  const unsigned long long least = vecs == a.n ? s.picked[vecs - 1] >> 32 << 32 : 0ull;
  for (int e = tid; e < all; e += kThreads) {
    const uint32_t v = ~(uint32_t)s.picked[e / Row<BF16>::kPer];
    const int64_t i = (int64_t)v * Row<BF16>::kPer - row->phase + e % Row<BF16>::kPer;
    const float z = i >= 0 && i < a.V ? row->load(i) : -INFINITY;
    const unsigned long long key = (unsigned long long)key_of(z) << 32 | (uint32_t)~(uint32_t)i;
    if (z > -INFINITY && key >= least) s.elems[atomicAdd(&s.near, 1)] = key;
  }
  __syncthreads();
  const int near = s.near;
  for (int e = tid; e < near; e += kThreads) {
    const unsigned long long me = s.elems[e];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < near; ++j) rank += s.elems[j] > me;
    if (rank < a.n) {
      a.top_tokens[(int64_t)r * a.n + rank] = (int32_t) ~(uint32_t)me;
      a.top_logprobs[(int64_t)r * a.n + rank] = logprob(of_key((uint32_t)(me >> 32)));
    }
  }
  for (int j = near + tid; j < a.n; j += kThreads) {
    a.top_tokens[(int64_t)r * a.n + j] = -1;
    a.top_logprobs[(int64_t)r * a.n + j] = -INFINITY;
  }
}

__device__ __forceinline__ int row_index(const LogprobArgs& a, int r) {
  const int i = a.rows ? a.rows[r] : r;
  return i >= 0 && i < a.num_rows ? i : -1;
}

// One workgroup a row, or part of one.  Bound by memory: 2048 rows of 128256 bf16 logits (525 MB) take
// 96 us, 5.5 TB/s, 512 rows of 256000 in fp32 87 us, 6.0 (a large copy runs at 5.2, a sum over 2 GiB
// at 4.0).  Loads pass the caches, as nothing is read twice (else 110 and 101 us).  4 KB on their way a
// wave and eight waves a SIMD, all 2048 rows at once (seven, with 71 registers: 102); 2 KB 101 and 120
// us, 8 KB at four waves 100 and 95, loads of a whole tile ahead of its arithmetic 103.  Rows in
// stretches an XCD: no difference.  In bf16 the instructions, an exponential and five more a logit,
// weigh nearly as much (waves wait for 25% of their cycles, in fp32 for 52%): 2048 rows of 32000, 1200
// different ones, take 26 us.  With logits decoded again for the maximum, the sums, the rank and the
// alternatives the same pass took 464 us.  Where there is about one row a compute unit, the alternatives
// cost 10 of 38 us (300 rows), as nothing else runs.
//
// The shift follows the maximum vector by vector, kRise = 2.  A tile that is only read again where a
// logit lies 24 above it takes 95 us, and 36 for the 300 rows, but the entropy of a row with one token of
// 2^18 to 2^23 times any other's weight is then off by up to 3e-6, here by 2e-7; 2 or 4: no difference in
// time; a tile read again at 2: 108 us, a vector read again 98 (loads come back in order, so it waits
// for the next tile's); the maximum before the exponentials 97, and 105 in fp32.
template <bool BF16, bool Entropy, bool Rank, bool Top>
__global__ __launch_bounds__(kThreads, 8) void k_logprob(LogprobArgs a) {
  using R = Row<BF16>;
  constexpr int kPer = R::kPer;
  __shared__ Lds s;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t unit = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int r = (int)(unit / a.parts), part = (int)(unit - (int64_t)r * a.parts);
  if (r >= a.R) return;
  const int at = row_index(a, r);
  const int token = a.tokens ? a.tokens[r] : -1;
  if (at < 0) {  // no such row
    if (part == 0) finish<BF16>(a, s, nullptr, r, LogprobPart{}, -1);
    return;
  }
  const R row(a.logits + (int64_t)at * a.V * R::kES, a.V);
  const int v0 = row.first + part * a.part_vecs;
  const int v1 = row.last - v0 < a.part_vecs ? row.last : v0 + a.part_vecs;
  // a vector's elements come first if they are >= `level` (it lies before the token's) or
  // >= `beyond`, the next number; those level with the token in its own vector are counted below
  const bool ranked = Rank && token >= 0 && token < a.V;
  const float level = ranked ? row.load(token) : INFINITY;
  const float beyond = ranked ? of_key(key_of(level) + 1) : INFINITY;
  const int token_vec = ranked ? (int)(((int64_t)row.phase + token) / kPer) : 0;

  float sum = 0.0f, sum_x = 0.0f, top = -INFINITY;
  float m0 = -INFINITY, k = 0.0f;  // the shift as a logit (wave-wide), and as c m0
  float limit = -INFINITY;         // logits above it move the shift
  bool far = false;                // |c m0| is 2^22 or more, and its rounding (then over
                                   // 1/8) shows in x - k: differences of logits first
  int above = 0;
  Kept<BF16> kept{s.val[wave], s.pos[wave], 0, -INFINITY};

  // pass<true>: logits of -inf, far ones, or a temperature that brings -1e30 near to 0
  bool clamp = a.c < 0x1p-77f;

  const float rise = kRise / a.c;

  // Where a lane's `most` lies above the limit: moves the shift to the wave's largest, with the sums so
  // far and those of a tile, f and fx.
  auto raise = [&](float most, float& f, float& fx) SV_INLINE {
    if (__builtin_expect(!__any(most > limit), 1)) return false;
    const float m = wave_all(most, [](float x, float y) { return fmaxf(x, y); });
    const float kn = a.c * m;
    const bool far_n = !(fabsf(kn) < 4194304.0f);
    if (m0 > -INFINITY) {
      const float d = far || far_n ? (m0 - m) * a.c : k - kn;
      const float w = exp2f(d);
      sum_x = w > 0.0f ? w * fmaf(d, sum, sum_x) : 0.0f;
      sum *= w;
      fx = w > 0.0f ? w * fmaf(d, f, fx) : 0.0f;
      f *= w;
    }
    m0 = m;
    k = kn;
    asm("" : "+v"(m0), "+v"(k));  // in vector registers: the loop's products have a scalar, a.c
    limit = m + rise;
    far = far_n;
    clamp |= far;
    return true;
  };
  float none = 0.0f, none_x = 0.0f;  // no tile's sums
  // one logit, whatever it is
  auto take = [&](float z) SV_INLINE {
    const float x = fmaxf(far ? (z - m0) * a.c : fmaf(z, a.c, -k), -200.0f);
    const float w = __builtin_amdgcn_exp2f(x);
    sum += w;
    sum_x = fmaf(w, x, sum_x);
  };
  auto vec_max = [&](const u32x4& v) SV_INLINE {
    float m = R::elem(v, 0);
#pragma unroll
    for (int e = 1; e < kPer; ++e) m = fmaxf(m, R::elem(v, e));
    return m;
  };

  // behind the last vector: that one again
  const u32x4* vecs = reinterpret_cast<const u32x4*>(row.at);
  auto load_vec = [&](int t, int u) SV_INLINE {
    const int j = t + u * kThreads + tid;
    return __builtin_nontemporal_load(&vecs[j < v1 ? j : v1 - 1]);
  };

  // One tile.  A vector's registers take the next tile's as soon as it is done, so that 4 KB a wave
  // are always on their way.  A vector's sums are formed at the shift as it is, and again where one
  // of its logits lies above the limit; the whole tile's (`redo`) where that turns out to need the
  // other form.  Clamp: logits of -inf, or of no weight at all, do not count as 0 * inf, and far
  // shifts are subtracted first.
  auto pass = [&](auto clamped, int t, u32x4 (&v)[kVecs], float (&vm)[kVecs],
                  float& most) SV_INLINE {
    constexpr bool Clamp = decltype(clamped)::value;
    float f = 0.0f, fx = 0.0f;
    most = -INFINITY;
    auto add = [&](const u32x4& y, float& m) SV_INLINE {
      const float z0 = Clamp && far ? m0 : 0.0f, k0 = Clamp && far ? 0.0f : k;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const float z = R::elem(y, e);
        float x = fmaf(Clamp ? z - z0 : z, a.c, -k0);
        if constexpr (Clamp) x = fmaxf(x, -200.0f);
        const float w = __builtin_amdgcn_exp2f(x);
        m = fmaxf(m, z);
        f += w;
        if constexpr (Entropy) fx = fmaf(w, x, fx);
      }
    };
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int j = t + u * kThreads + tid;
      float m = -INFINITY, before = f, before_x = fx;
      add(v[u], m);
      vm[u] = j < v1 ? m : -INFINITY;
      if (raise(vm[u], before, before_x)) {
        f = before;
        fx = before_x;
        add(v[u], m);
      }
      most = fmaxf(most, vm[u]);
      if constexpr (Rank) {
        const float th = j >= v1 ? INFINITY : j < token_vec ? level : beyond;
        if (__any(m >= th)) {
#pragma unroll
          for (int e = 0; e < kPer; ++e) above += __popcll(__ballot(R::elem(v[u], e) >= th));
        }
      }
      v[u] = load_vec(t + kTile, u);
      // few decoded logits at a time: nothing moves over this
      asm volatile("" : "+v"(f), "+v"(fx), "+v"(vm[u]));
      __builtin_amdgcn_sched_barrier(0);
    }
    const bool odd = !Clamp && Entropy && fx != fx;
    if (__any(odd)) clamp = true;
    if (!Clamp && clamp) return false;
    sum += f;
    sum_x += fx;
    return true;
  };
  auto redo = [&](int t, float most) SV_INLINE {
    raise(most, none, none_x);
#pragma unroll 1
    for (int u = 0; u < kVecs; ++u) {
      if (t + u * kThreads + tid >= v1) continue;
      const u32x4 y = load_vec(t, u);
#pragma unroll
      for (int e = 0; e < kPer; ++e) take(R::elem(y, e));
    }
  };
  auto step = [&](int t, u32x4 (&v)[kVecs]) SV_INLINE {
    float vm[kVecs], most;
    if (m0 == -INFINITY) raise(t + tid < v1 ? vec_max(v[0]) : -INFINITY, none, none_x);
    if (t + kTile > v1) {
      // of no weight: -inf, or (no 0 * inf then) about -1e30, 2^22.6 / c below 0 at least, where the
      // shift is less than 2^22 from it
      const uint32_t none = clamp ? BF16 ? 0xFF80FF80u : 0xFF800000u
                                  : BF16 ? 0xF149F149u : 0xF149F2CAu;
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
        if (t + u * kThreads + tid >= v1) v[u] = u32x4{none, none, none, none};
    }
    const bool done = clamp ? pass(std::true_type{}, t, v, vm, most)
                            : pass(std::false_type{}, t, v, vm, most);
    if (!done) redo(t, most);
    top = fmaxf(top, most);
    if constexpr (Top) {
      if (t == v0) {  // n lanes hold as much as `bound`, in different vectors
        const uint32_t one[1] = {key_of(most)};
        const uint32_t bound = nth_key<BF16>(one, a.n);
        kept.tau = bound <= key_of(-INFINITY)
                       ? -INFINITY : of_key(bound - (bound == 0x80000000u ? 2u : 1u));
      }
      if (__any(most > kept.tau)) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
          kept.add(vm[u] > kept.tau, vm[u], (uint32_t)(t + u * kThreads + tid));
        if (kept.count > a.n + kSpare) kept.cut(a.n);
      }
    }
  };

  if (v0 < v1) {
    u32x4 v[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      v[u] = load_vec(v0, u);
      __builtin_amdgcn_sched_barrier(0);  // in this order, in which they are waited for
    }
    for (int t = v0; t < v1; t += kTile) step(t, v);
  }

  // By the first wave: the elements of vectors that are not whole (lanes 0 .. 7 the head's, 8 .. 15
  // the tail's), and those of the token's own vector that are level with it.
  if (tid < 2) s.edge[tid] = 0;
  if (wave == 0 && part == 0) {
    const int64_t i = lane < 8 ? (lane < row.head ? lane : a.V) : row.tail() + lane - 8;
    const bool mine = lane < 16 && i < a.V;
    const float z = mine ? row.load(i) : -INFINITY;
    raise(z, none, none_x);
    take(z);
    top = fmaxf(top, z);
    if constexpr (Rank) {
      above += __popcll(__ballot(mine && (z > level || (z == level && i < token))));
      const int64_t own = (int64_t)token_vec * kPer - row.phase + lane;
      const bool whole = ranked && token_vec >= row.first && token_vec < row.last;
      above += __popcll(__ballot(whole && lane < kPer && own < token && row.load(own) == level));
    }
    if constexpr (Top) {
      float m = z;
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
      if ((lane == 0 || lane == 8) && m > -INFINITY)
        s.edge[lane / 8] = (unsigned long long)key_of(m) << 32 |
                           (lane ? ~(uint32_t)row.last : ~0u);
    }
  }

  // the waves' sums, then the part's
  auto add = [](double x, double y) SV_INLINE { return x + y; };
  const double all = wave_all((double)sum, add), all_x = wave_all((double)sum_x, add);
  top = wave_all(top, [](float x, float y) { return fmaxf(x, y); });
  if (lane == 0) {
    const double shift = m0 == -INFINITY ? -INFINITY : far ? (double)a.c * m0 : (double)k;
    s.stat[wave] = LogprobPart{shift, all, all_x, top, above};
  }
  if constexpr (Top) {
    if (kept.count > a.n) kept.cut(a.n);
    __builtin_amdgcn_wave_barrier();
    if (lane < kept.count)
      s.keys[wave][lane] = (unsigned long long)key_of(kept.val[lane]) << 32 | ~kept.pos[lane];
    if (lane == 0) s.count[wave] = kept.count;
  }
  __syncthreads();
  static_assert(kWaves == 4, "a lane of four a wave");
  const LogprobPart st =
      joined(s.stat[lane & 3], [](auto x, auto op) { return quad_all(x, op); });
  if constexpr (Top) {
    // a vector's rank among the waves' kept ones and the two that are not whole
    auto rank_of = [&](unsigned long long me) SV_INLINE {
      int rank = (s.edge[0] > me) + (s.edge[1] > me);
      for (int i = 0; i < kWaves; ++i)
#pragma unroll 8
        for (int j = 0; j < s.count[i]; ++j) rank += s.keys[i][j] > me;
      return rank;
    };
    const unsigned long long me = lane < kept.count ? s.keys[wave][lane] : 0;
    const int rank = rank_of(me);
    if (me && rank < a.n) s.picked[rank] = me;
    if (tid < 2 && s.edge[tid]) {
      const int at = rank_of(s.edge[tid]);
      if (at < a.n) s.picked[at] = s.edge[tid];
    }
    if (tid == 0) {
      int all = (s.edge[0] != 0) + (s.edge[1] != 0);
      for (int i = 0; i < kWaves; ++i) all += s.count[i];
      s.found = all < a.n ? all : a.n;
    }
  }
  __syncthreads();
  if (a.parts == 1) {
    finish<BF16>(a, s, &row, r, st, token);
  } else {
    if (tid == 0) a.part[unit] = st;
    for (int j = tid; j < a.n; j += kThreads)
      a.part_top[unit * a.n + j] = j < s.found ? s.picked[j] : 0ull;
  }
}

// Joins the parts of a row, whose lists of vectors are in order each.  A vector is among the first n
// only if it comes no later than a bound that n vectors reach: the n-th of the list whose n-th
// comes first, or, for any m, the m-th largest of the parts' (n / m)-th vectors' elements.  The few
// vectors that reach the best of these bounds are ranked against each other.  Latency alone, 7.6 us
// for 16 parts' 20 alternatives each; 15 with the lists merged one vector after the other and the
// parts' sums read likewise, and 2 more with one key of the ranking in flight.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void k_logprob_join(LogprobArgs a) {
  __shared__ Lds s;
  __shared__ unsigned long long lists[kMaxParts * kLogprobMaxTop];
  __shared__ unsigned long long bounds[kWaves];
  constexpr int kMine = kMaxParts * kLogprobMaxTop / kThreads;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
    const int at = row_index(a, r);
    if (at < 0) continue;  // written already
    const Row<BF16> row(a.logits + (int64_t)at * a.V * Row<BF16>::kES, a.V);
    const int all = a.parts * a.n;
    const unsigned long long* given = a.part_top + (int64_t)r * all;
    unsigned long long mine[kMine];
    if (a.n) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int e = tid + i * kThreads;
        mine[i] = e < all ? given[e] : 0ull;
        if (e < all) lists[e] = mine[i];
      }
    }
    LogprobPart mine_st{-INFINITY, 0.0, 0.0, -INFINITY, 0};
    if (lane < a.parts) mine_st = a.part[(int64_t)r * a.parts + lane];
    const LogprobPart st = joined(mine_st, [](auto x, auto op) { return wave_all(x, op); });
    if (a.n) {
      if (tid == 0) s.near = 0;
      __syncthreads();
      unsigned long long bound = 0;
      for (int m = wave; m < 7; m += kWaves) {  // the 2^m-th vectors, in the end the n-th
        const int each = 1 << m < a.n ? 1 << m : a.n, parts = (a.n + each - 1) / each;
        const unsigned long long key = lane < a.parts ? lists[lane * a.n + each - 1] : 0ull;
        if (parts == 1) {
          const unsigned long long b = wave_all(
              key, [](unsigned long long x, unsigned long long y) { return x > y ? x : y; });
          bound = b > bound ? b : bound;
          break;
        }
        const uint32_t one[1] = {(uint32_t)(key >> 32)};
        const unsigned long long b = (unsigned long long)nth_key<BF16>(one, parts) << 32;
        bound = b > bound ? b : bound;
      }
      if (lane == 0) bounds[wave] = bound;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWaves; ++i) bound = bounds[i] > bound ? bounds[i] : bound;
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        if (mine[i] && mine[i] >= bound) lists[atomicAdd(&s.near, 1)] = mine[i];
      __syncthreads();
      const int near = s.near;
      for (int e = tid; e < near; e += kThreads) {  // in no order, as they are all different
        const unsigned long long me = lists[e];
        int rank = 0;
#pragma unroll 8
        for (int k = 0; k < near; ++k) rank += lists[k] > me;
        if (rank < a.n) s.picked[rank] = me;
      }
      if (tid == 0) s.found = near < a.n ? near : a.n;
    }
    __syncthreads();
    finish<BF16>(a, s, &row, r, st, a.tokens ? a.tokens[r] : -1);
    __syncthreads();
  }
}

template <bool BF16, bool Entropy, bool Rank>
void launch_top(const LogprobArgs& a, dim3 blocks, hipStream_t stream) {
  if (a.n)
    hipLaunchKernelGGL((k_logprob<BF16, Entropy, Rank, true>), blocks, dim3(kThreads), 0,
                       stream, a);
  else
    hipLaunchKernelGGL((k_logprob<BF16, Entropy, Rank, false>), blocks, dim3(kThreads), 0,
                       stream, a);
}

template <bool BF16>
hipError_t launch(const LogprobArgs& a, hipStream_t stream) {
  const int64_t units = (int64_t)a.R * a.parts;
  const unsigned wide = (unsigned)(units < kMaxBlocks ? units : kMaxBlocks);
  const dim3 blocks(wide, (unsigned)((units + wide - 1) / wide));
  if (a.entropy && a.rank) launch_top<BF16, true, true>(a, blocks, stream);
  else if (a.entropy) launch_top<BF16, true, false>(a, blocks, stream);
  else if (a.rank) launch_top<BF16, false, true>(a, blocks, stream);
  else launch_top<BF16, false, false>(a, blocks, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.parts == 1) return e;
  hipLaunchKernelGGL(k_logprob_join<BF16>, dim3((unsigned)(a.R < kMaxBlocks ? a.R : kMaxBlocks)),
                     dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

LogprobPlan plan_logprobs(int R, int V, sv_dtype dt, int n) {
  LogprobPlan p{};
  const int per = dt == SV_DTYPE_BF16 ? 8 : 4;
  const int64_t vecs = V / per > 1 ? V / per : 1;  // whole ones of a row, at most
  const int64_t tiles = (vecs + kTile - 1) / kTile;
  // Rows of their own workgroup from one a compute unit on, else parts of them, a tile each at
  // least, for two.  128256 bf16 (32000 fp32) logits a row, both launches in a graph: 64 rows at two
  // workgroups a unit 20.4 (20.6) us, at one 23.1 (20.5), at four 21.5 (20.7); 128 rows 25.0 (21.4),
  // 29.0 (24.2), 24.1 (23.0); 256 rows in one part each 32.5 (21.5), in two 31.4 (25.8), 384 rows
  // 37.9 (23.8), 40.4 (28.9).
  int64_t parts = R >= 256 ? 1 : (512 + (int64_t)R - 1) / R;
  parts = parts < tiles ? parts : tiles;
  parts = parts < kMaxParts ? parts : kMaxParts;
  const int64_t each = (tiles + parts - 1) / parts;
  p.part_vecs = (int)(each * kTile);
  p.parts = (int)((tiles + each - 1) / each);
  if (p.parts > 1) {
    p.o_top = (size_t)R * p.parts * sizeof(LogprobPart);
    p.bytes = p.o_top + (size_t)R * p.parts * n * sizeof(unsigned long long);
  }
  return p;
}

hipError_t launch_logprobs(const LogprobArgs& a, sv_dtype dt, hipStream_t stream) {
  return dt == SV_DTYPE_BF16 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace sv
