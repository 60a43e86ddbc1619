// Log probabilities of given tokens on gfx950, with the entropy of their distributions, the tokens'
// ranks and the most probable alternatives, in one pass over the logits.
//
// With x = z log2(e) / T, a shift k and S = sum 2^(x - k), X = sum 2^(x - k) (x - k):
//   log p(t) = ln2 (x_t - k) - ln S,   H = ln S - ln2 X / S
// k is near the first tile's maximum and follows it when a later one is far above; sums are in
// fp32 a lane, joined in 64 bits.
//
// Alternatives: the top n elements (larger first, ties to the lower index) lie in the n vectors of
// 16 bytes that come first by (their largest element, position): an element of another vector comes
// behind the largest of each of these.  So the pass only keeps vectors whose maximum, which the
// shift needs anyway, beats the wave's n-th so far; a wave meets its vectors in order of position,
// so a tie never does.  The kept vectors' elements are ranked at the end.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "sv_logprob.hpp"

namespace sv {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kVecs = 8;              // vectors a thread and tile
constexpr int kTile = kThreads * kVecs;
constexpr int kList = 128;            // vectors a wave keeps
constexpr int kMaxParts = 64;         // of a row: one a lane of the join
constexpr int64_t kMaxBlocks = 1 << 20;
constexpr double kLn2 = 0.69314718055994530942;

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
  const char* at;   // aligned start: vector 0 may begin before the row
  int phase;        // elements of vector 0 that lie before the row
  int V, vecs;

  __device__ __forceinline__ Row(const char* row, int V_) : V(V_) {
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
    at = row - off;
    phase = (int)off / kES;
    vecs = (int)(((int64_t)phase + V + kPer - 1) / kPer);
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

template <class T, class Op>
__device__ __forceinline__ T wave_all(T x, Op op) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = op(x, __shfl_xor(x, d));
  return x;
}

// The n-th largest of the wave's keys, one or two a lane (largest k with n keys >= k).
template <int Keys>
__device__ __forceinline__ uint32_t nth_key(const uint32_t (&k)[Keys], int n) {
  uint32_t t = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t c = t | 1u << bit;
    int count = 0;
#pragma unroll
    for (int i = 0; i < Keys; ++i) count += __popcll(__ballot(k[i] >= c));
    if (count >= n) t = c;
  }
  return t;
}

struct Lds {
  float val[kWaves][kList];
  uint32_t pos[kWaves][kList];
  unsigned long long keys[kWaves][kLogprobMaxTop];
  unsigned long long picked[kLogprobMaxTop];
  unsigned long long elems[kLogprobMaxTop * 8];
  LogprobPart stat[kWaves];
  int count[kWaves];
  int found;
};

// Kept vectors of a wave, in order of position.
struct Kept {
  float* val;
  uint32_t* pos;
  int count;
  float tau;  // vectors count only above it

  // keeps the n first by (value, position)
  __device__ __forceinline__ void cut(int n) {
    const int lane = threadIdx.x & 63;
    __builtin_amdgcn_wave_barrier();
    uint32_t k[2], p[2];
    float v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = lane + 64 * i;
      v[i] = at < count ? val[at] : 0.0f;
      p[i] = at < count ? pos[at] : 0u;
      k[i] = at < count ? key_of(v[i]) : 0u;
    }
    const uint32_t t = nth_key(k, n);
    const unsigned long long below = (1ull << lane) - 1;
    unsigned long long level[2];
    int quota = n;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      quota -= __popcll(__ballot(k[i] > t));
      level[i] = __ballot(k[i] == t);
    }
    const bool take0 = k[0] > t || (k[0] == t && __popcll(level[0] & below) < quota);
    const bool take1 =
        k[1] > t || (k[1] == t && __popcll(level[0]) + __popcll(level[1] & below) < quota);
    const unsigned long long m0 = __ballot(take0), m1 = __ballot(take1);
    __builtin_amdgcn_wave_barrier();
    if (take0) {
      val[__popcll(m0 & below)] = v[0];
      pos[__popcll(m0 & below)] = p[0];
    }
    if (take1) {
      val[__popcll(m0) + __popcll(m1 & below)] = v[1];
      pos[__popcll(m0) + __popcll(m1 & below)] = p[1];
    }
    __builtin_amdgcn_wave_barrier();
    count = n;
    tau = of_key(t);
  }

  __device__ __forceinline__ void add(bool hit, float v, uint32_t p, int n) {
    const unsigned long long m = __ballot(hit);
    if (!m) return;
    if (count + __popcll(m) > kList) {
      cut(n);
      // some may not count any more
      add_all(hit && v > tau, v, p);
      return;
    }
    add_all(hit, v, p);
  }
  __device__ __forceinline__ void add_all(bool hit, float v, uint32_t p) {
    const unsigned long long m = __ballot(hit);
    const int at = count + __popcll(m & ((1ull << (threadIdx.x & 63)) - 1));
    if (hit) {
      val[at] = v;
      pos[at] = p;
    }
    count += __popcll(m);
  }
};

// Sums of several parts on one shift.
__device__ __forceinline__ LogprobPart joined(const LogprobPart* p, int count) {
  LogprobPart r{-INFINITY, 0.0f, 0.0f, -INFINITY, 0, {0, 0}};
  double sum = 0.0, sum_x = 0.0;
  for (int i = 0; i < count; ++i) r.shift = p[i].shift > r.shift ? p[i].shift : r.shift;
  for (int i = 0; i < count; ++i) {
    r.top = fmaxf(r.top, p[i].top);
    r.above += p[i].above;
    if (p[i].shift == -INFINITY) continue;  // no finite logit
    const double d = p[i].shift - r.shift;
    const double f = (double)exp2f((float)d);
    sum += f * p[i].sum;
    if (f > 0.0) sum_x += f * ((double)p[i].sum_x + d * p[i].sum);
  }
  r.sum = (float)sum;
  r.sum_x = (float)sum_x;
  return r;
}

// A row's results from its statistics and, in s.picked, the keys (largest element, ~position) of
// its first s.found vectors.
template <bool BF16>
__device__ __forceinline__ void finish(const LogprobArgs& a, Lds& s, const Row<BF16>* row, int r,
                       const LogprobPart& st, int token) {
  const int tid = threadIdx.x;
  const bool some = row && st.top > -INFINITY;
  const double ln_s = some ? log((double)st.sum) : 0.0;
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
  for (int e = tid; e < all; e += kThreads) {
    const uint32_t v = ~(uint32_t)s.picked[e / Row<BF16>::kPer];
    const int64_t i = (int64_t)v * Row<BF16>::kPer - row->phase + e % Row<BF16>::kPer;
    const float z = i >= 0 && i < a.V ? row->load(i) : -INFINITY;
    s.elems[e] = z > -INFINITY ? (unsigned long long)key_of(z) << 32 | (uint32_t)~(uint32_t)i : 0;
  }
  __syncthreads();
  int real = 0;
  for (int e0 = 0; e0 < all; e0 += kThreads) {
    const int e = e0 + tid;
    const unsigned long long me = e < all ? s.elems[e] : 0;
    int rank = 0;
    real = 0;
    for (int j = 0; j < all; ++j) {
      const unsigned long long k = s.elems[j];
      rank += k > me;
      real += k != 0;
    }
    if (me && rank < a.n) {
      const uint32_t i = ~(uint32_t)me;
      a.top_tokens[(int64_t)r * a.n + rank] = (int32_t)i;
      a.top_logprobs[(int64_t)r * a.n + rank] = logprob(row->load(i));
    }
  }
  for (int j = real + tid; j < a.n; j += kThreads) {
    a.top_tokens[(int64_t)r * a.n + j] = -1;
    a.top_logprobs[(int64_t)r * a.n + j] = -INFINITY;
  }
}

__device__ __forceinline__ int row_index(const LogprobArgs& a, int r) {
  const int i = a.rows ? a.rows[r] : r;
  return i >= 0 && i < a.num_rows ? i : -1;
}

template <bool BF16, bool Entropy, bool Rank, bool Top>
__global__ __launch_bounds__(kThreads) void k_logprob(LogprobArgs a) {
  using R = Row<BF16>;
  constexpr int kPer = R::kPer;
  __shared__ Lds s;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t units = (int64_t)a.R * a.parts;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int r = (int)(unit / a.parts), part = (int)(unit - (int64_t)r * a.parts);
    const int at = row_index(a, r);
    const int token = a.tokens ? a.tokens[r] : -1;
    if (at < 0) {  // no such row
      if (part == 0) finish<BF16>(a, s, nullptr, r, LogprobPart{}, -1);
      continue;
    }
    const R row(a.logits + (int64_t)at * a.V * R::kES, a.V);
    const int v0 = part * a.part_vecs;
    const int v1 = v0 + a.part_vecs < row.vecs ? v0 + a.part_vecs : row.vecs;
    const bool ranked = Rank && token >= 0 && token < a.V;
    const float zt = ranked ? row.load(token) : 0.0f;

    float sum = 0.0f, sum_x = 0.0f, top = -INFINITY;
    float m0 = -INFINITY, k = 0.0f;  // the shift as a logit (wave-wide), and as c m0
    bool far = false;                // |c m0| is 2^22 or more, and its rounding (then over
                                     // 1/8) shows in x - k: differences of logits first
    int above = 0;
    Kept kept{s.val[wave], s.pos[wave], 0, -INFINITY};
    bool first = true;

    auto load_tile = [&](int t, u32x4 (&v)[kVecs]) {
      if (t >= v1) return;
      const bool whole = (t > 0 || row.phase == 0) && t + kTile <= v1 &&
                         ((int64_t)(t + kTile)) * kPer - row.phase <= a.V;
      if (whole) {
        const u32x4* p = reinterpret_cast<const u32x4*>(row.at) + t + tid;
#pragma unroll
        for (int u = 0; u < kVecs; ++u) v[u] = p[u * kThreads];
        return;
      }
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const int j = t + u * kThreads + tid;
        const int64_t e0 = (int64_t)j * kPer - row.phase;
        const uint32_t fill = BF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
        v[u] = u32x4{fill, fill, fill, fill};
        if (j >= v1) continue;
        if (e0 >= 0 && e0 + kPer <= a.V) {
          v[u] = reinterpret_cast<const u32x4*>(row.at)[j];
        } else {
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            if (e0 + e < 0 || e0 + e >= a.V) continue;
            const uint32_t bits = __float_as_uint(row.load(e0 + e));
            if constexpr (!BF16) v[u][e] = bits;
            else v[u][e >> 1] = e & 1 ? (v[u][e >> 1] & 0xFFFFu) | bits
                                      : (v[u][e >> 1] & 0xFFFF0000u) | bits >> 16;
          }
        }
      }
    };

    auto step = [&](int t, const u32x4 (&v)[kVecs]) {
      float vm[kVecs], most = -INFINITY;
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        vm[u] = R::elem(v[u], 0);
#pragma unroll
        for (int e = 1; e < kPer; ++e) vm[u] = fmaxf(vm[u], R::elem(v[u], e));
        most = fmaxf(most, vm[u]);
      }
      top = fmaxf(top, most);
      // 2^(x - k) of up to 2^24 cost nothing
      if (__any(most > m0 && (m0 == -INFINITY || (most - m0) * a.c > 24.0f))) {
        const float m = wave_all(most, [](float x, float y) { return fmaxf(x, y); });
        const float kn = a.c * m;
        const bool far_n = !(fabsf(kn) < 4194304.0f);
        if (m0 > -INFINITY) {
          const float d = far || far_n ? (m0 - m) * a.c : k - kn;
          const float f = exp2f(d);
          sum_x = f > 0.0f ? f * fmaf(d, sum, sum_x) : 0.0f;
          sum *= f;
        }
        m0 = m;
        far = far_n;
        k = kn;
      }
      // without a finite logit so far (x - k) is -inf, or NaN and put right below
      const float sum_was = sum, sum_x_was = sum_x;
      if (!far) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            const float x = fmaf(R::elem(v[u], e), a.c, -k);
            const float w = __builtin_amdgcn_exp2f(x);
            sum += w;
            if constexpr (Entropy) sum_x = fmaf(w, x, sum_x);
          }
      }
      if (far || (Entropy && __any(sum_x != sum_x))) {
        // -inf, or out of range: a logit of no weight must not count as 0 * inf
        sum = sum_was;
        sum_x = sum_x_was;
        if (m0 > -INFINITY) {
#pragma unroll
          for (int u = 0; u < kVecs; ++u)
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              const float z = R::elem(v[u], e);
              const float x = fmaxf(far ? (z - m0) * a.c : fmaf(z, a.c, -k), -200.0f);
              const float w = __builtin_amdgcn_exp2f(x);
              sum += w;
              if constexpr (Entropy) sum_x = fmaf(w, x, sum_x);
            }
        }
      }
      if (ranked) {
        const int64_t lo = (int64_t)t * kPer - row.phase, hi = lo + (int64_t)kTile * kPer;
        if (hi <= token && zt > -INFINITY) {
#pragma unroll
          for (int u = 0; u < kVecs; ++u)
#pragma unroll
            for (int e = 0; e < kPer; ++e) above += __popcll(__ballot(R::elem(v[u], e) >= zt));
        } else if (lo > token) {
#pragma unroll
          for (int u = 0; u < kVecs; ++u)
#pragma unroll
            for (int e = 0; e < kPer; ++e) above += __popcll(__ballot(R::elem(v[u], e) > zt));
        } else {
#pragma unroll
          for (int u = 0; u < kVecs; ++u)
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              const int64_t j = t + u * kThreads + tid, i = j * kPer - row.phase + e;
              const float z = R::elem(v[u], e);
              above += __popcll(
                  __ballot(z > zt || (z == zt && i >= 0 && i < token && j < v1)));
            }
        }
      }
      if constexpr (Top) {
        if (first) {  // n lanes hold as much as `bound`, in different vectors
          const uint32_t one[1] = {key_of(most)};
          const uint32_t bound = nth_key(one, a.n);
          kept.tau = bound <= key_of(-INFINITY)
                         ? -INFINITY : of_key(bound - (bound == 0x80000000u ? 2u : 1u));
        }
        if (__any(most > kept.tau)) {
#pragma unroll
          for (int u = 0; u < kVecs; ++u)
            kept.add(vm[u] > kept.tau, vm[u], (uint32_t)(t + u * kThreads + tid), a.n);
        }
      }
      first = false;
    };

    u32x4 v[kVecs], w[kVecs];
    load_tile(v0, v);
    for (int t = v0; t < v1; t += 2 * kTile) {
      load_tile(t + kTile, w);
      step(t, v);
      if (t + kTile >= v1) break;
      load_tile(t + 2 * kTile, v);
      step(t + kTile, w);
    }

    // the waves' sums, then the part's
    auto add = [](float x, float y) { return x + y; };
    sum = wave_all(sum, add);
    sum_x = wave_all(sum_x, add);
    top = wave_all(top, [](float x, float y) { return fmaxf(x, y); });
    if (lane == 0) {
      const double shift = m0 == -INFINITY ? -INFINITY : far ? (double)a.c * m0 : (double)k;
      s.stat[wave] = LogprobPart{shift, sum, sum_x, top, above, {0, 0}};
    }
    if constexpr (Top) {
      if (kept.count > a.n) kept.cut(a.n);
      __builtin_amdgcn_wave_barrier();
      if (lane < kept.count)
        s.keys[wave][lane] = (unsigned long long)key_of(kept.val[lane]) << 32 | ~kept.pos[lane];
      if (lane == 0) s.count[wave] = kept.count;
    }
    __syncthreads();
    LogprobPart st = joined(s.stat, kWaves);
    if constexpr (Top) {
      // a vector's rank among the waves' kept ones
      unsigned long long me = lane < kept.count ? s.keys[wave][lane] : 0;
      int rank = 0, all = 0;
      for (int i = 0; i < kWaves; ++i) {
        const int count = s.count[i];
        all += count;
        for (int j = 0; j < count; ++j) rank += s.keys[i][j] > me;
      }
      if (me && rank < a.n) s.picked[rank] = me;
      if (tid == 0) s.found = all < a.n ? all : a.n;
    }
    __syncthreads();
    if (a.parts == 1) {
      finish<BF16>(a, s, &row, r, st, token);
    } else {
      if (tid == 0) a.part[unit] = st;
      for (int j = tid; j < a.n; j += kThreads)
        a.part_top[unit * a.n + j] = j < s.found ? s.picked[j] : 0ull;
    }
    __syncthreads();
  }
}

// Joins the parts of a row: one lane a part holds the first of its vectors that is left.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void k_logprob_join(LogprobArgs a) {
  __shared__ Lds s;
  const int tid = threadIdx.x, lane = tid & 63;
  for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
    const int at = row_index(a, r);
    if (at < 0) continue;  // written already
    const Row<BF16> row(a.logits + (int64_t)at * a.V * Row<BF16>::kES, a.V);
    const LogprobPart st = joined(a.part + (int64_t)r * a.parts, a.parts);
    if (a.n && tid < 64) {
      const unsigned long long* mine = a.part_top + ((int64_t)r * a.parts + lane) * a.n;
      int next = 0, found = 0;
      unsigned long long head = lane < a.parts ? mine[0] : 0ull;
      for (; found < a.n; ++found) {
        const unsigned long long best = wave_all(
            head, [](unsigned long long x, unsigned long long y) { return x > y ? x : y; });
        if (!best) break;
        if (head == best) {
          s.picked[found] = best;
          ++next;
          head = next < a.n ? mine[next] : 0ull;
        }
      }
      if (lane == 0) s.found = found;
    }
    __syncthreads();
    finish<BF16>(a, s, &row, r, st, a.tokens ? a.tokens[r] : -1);
    __syncthreads();
  }
}

template <bool BF16, bool Entropy, bool Rank>
void launch_top(const LogprobArgs& a, unsigned blocks, hipStream_t stream) {
  if (a.n)
    hipLaunchKernelGGL((k_logprob<BF16, Entropy, Rank, true>), dim3(blocks), dim3(kThreads), 0,
                       stream, a);
  else
    hipLaunchKernelGGL((k_logprob<BF16, Entropy, Rank, false>), dim3(blocks), dim3(kThreads), 0,
                       stream, a);
}

template <bool BF16>
hipError_t launch(const LogprobArgs& a, hipStream_t stream) {
  const int64_t units = (int64_t)a.R * a.parts;
  const unsigned blocks = (unsigned)(units < kMaxBlocks ? units : kMaxBlocks);
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
  const int64_t vecs = ((int64_t)V + 2 * (per - 1)) / per + 1;  // of a row at any phase, at most
  const int64_t tiles = (vecs + kTile - 1) / kTile;
  // two workgroups a compute unit, a tile each at least
  int64_t parts = (512 + (int64_t)R - 1) / R;
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
