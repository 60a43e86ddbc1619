// Eviction from a paged cache by accumulated attention weight, on gfx950.  In every layer and kv
// head a sequence of len tokens keeps `want` of them: its first `sinks`, its last `recent`, and of
// those between the ones of largest weight (ties: the earlier token).  Kept tokens stay in order:
// row kept[j] of keys, values and weights moves to j <= kept[j].
//
// k_evict_select finds the tokens: the weight of the last one kept by three histograms of 11, 11
// and 10 bits of an order-preserving key, then the list in order by ballots.  k_evict_move moves the
// rows.  Rows only move down, so rounds of rows in increasing order, all read before any is written,
// overwrite nothing that a later round reads.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "sv_step.hpp"

namespace sv {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr int kBinsEach = kBins / kThreads;
constexpr int kHeld = 8192;   // weights that are kept in LDS, where there are no more
constexpr int kMoveRows = 4;  // rows that a thread has in flight
constexpr int64_t kMaxBlocks = 1 << 20;

// Unsigned order of the weights; NaN below all, the two zeros alike.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Waits until every thread's loads are there: what was read may then be written.
__device__ __forceinline__ void all_read() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

// Workgroups go to the 8 XCDs in turn: gives each of these a stretch of the `count` units.
__device__ __forceinline__ int64_t xcd_order(int64_t unit, int64_t count) {
  const int64_t each = count / 8;
  return unit < 8 * each ? (unit & 7) * each + (unit >> 3) : unit;
}

struct Lds {
  int hist[kBins];
  float held[kHeld];
  int wave[kWaves];
  int2 wave2[kWaves];
  int digit, left, inside;
};

// What is kept of the weights x[0 .. m): those whose key >> shift is above `bound`, and the first
// `quota` of those where it equals it.
struct Cut {
  uint32_t bound;
  int shift, quota;
};

// The weights x[0 .. m) of a workgroup: a wave has a stretch of its own, in order, which it keeps in
// LDS (Held) or reads again every time.
template <bool Held>
struct Weights {
  const float* x;
  float* held;
  int first, end;  // the wave's stretch

  __device__ __forceinline__ Weights(Lds& s, const float* x_, int m) : x(x_), held(s.held) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int stretch = (m + kThreads - 1) / kThreads * 64;
    first = wave * stretch;
    end = first + stretch < m ? first + stretch : m;
    if constexpr (Held)
#pragma unroll 4
      for (int e = first + lane; e < end; e += 64) held[e] = x[e];
  }
  // f(number, weight, whether there is one) for all of the stretch, 64 lanes at a time
  template <class F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll 2
    for (int e0 = first; e0 < end; e0 += 64) {
      const int e = e0 + (int)(threadIdx.x & 63);
      f(e, e < end ? (Held ? held[e] : x[e]) : 0.0f, e < end);
    }
  }
};

// The `count` largest weights (0 < count < m).
template <bool Held>
__device__ __forceinline__ Cut find_cut(Lds& s, const Weights<Held>& w, int count) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Cut cut{0u, 32, count};
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10, shift = cut.shift - bits;
    for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
    __syncthreads();
    w.each([&](int, float weight, bool there) __attribute__((always_inline)) {
      const uint32_t key = order_of(weight);
      const bool in = there && (cut.shift == 32 || key >> cut.shift == cut.bound);
      const int d = (int)(key >> shift & ((1u << bits) - 1));
      // lanes of one bin, as where many weights are alike, add together
      const unsigned long long some = __ballot(in);
      if (!some) return;
      const int lead = __ffsll(some) - 1, d0 = __shfl(d, lead);
      if (__ballot(in && d != d0) == 0) {
        if (lane == lead) atomicAdd(&s.hist[d0], __popcll(some));
      } else if (in) {
        atomicAdd(&s.hist[d], 1);
      }
    });
    __syncthreads();
    // a few bins a thread, largest first
    const int top = kBins - 1 - kBinsEach * tid;
    int n[kBinsEach], mine = 0;
#pragma unroll
    for (int i = 0; i < kBinsEach; ++i) mine += n[i] = s.hist[top - i];
    int incl = mine;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
      const int y = __shfl_up(incl, k);
      incl += lane >= k ? y : 0;
    }
    if (lane == 63) s.wave[wave] = incl;
    __syncthreads();
    int before = incl - mine;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) before += i < wave ? s.wave[i] : 0;
    if (before < cut.quota && cut.quota <= before + mine) {
#pragma unroll
      for (int i = 0; i < kBinsEach; ++i) {
        if (before < cut.quota && cut.quota <= before + n[i]) {
          s.digit = top - i;
          s.left = cut.quota - before;
          s.inside = n[i];
        }
        before += n[i];
      }
    }
    __syncthreads();
    cut.bound = (cut.shift == 32 ? 0u : cut.bound << bits) | (uint32_t)s.digit;
    cut.shift = shift;
    cut.quota = s.left;
    if (s.left == s.inside) break;  // the whole bin is kept
  }
  return cut;
}

// Lists in order, from kept[0] on, the numbers (plus `sinks`) of the count largest of m weights, and
// (Held) the weights themselves from out[0] on.
template <bool Held>
__device__ __forceinline__ void list_largest(Lds& s, const float* x, int m, int count, int sinks,
                                             int32_t* kept, float* out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Weights<Held> w(s, x, m);
  const Cut cut = find_cut(s, w, count);
  // behind those of the waves before it
  int above_n = 0, level_n = 0;
  w.each([&](int, float weight, bool there) __attribute__((always_inline)) {
    const uint32_t k = order_of(weight) >> cut.shift;
    above_n += __popcll(__ballot(there && k > cut.bound));
    level_n += __popcll(__ballot(there && k == cut.bound));
  });
  if (lane == 0) s.wave2[wave] = make_int2(above_n, level_n);
  __syncthreads();
  int above_before = 0, level_before = 0;
  for (int i = 0; i < wave; ++i) {
    above_before += s.wave2[i].x;
    level_before += s.wave2[i].y;
  }
  int at = above_before + (level_before < cut.quota ? level_before : cut.quota);
  const unsigned long long below = (1ull << lane) - 1;
  w.each([&](int e, float weight, bool there) __attribute__((always_inline)) {
    const uint32_t k = order_of(weight) >> cut.shift;
    const bool level = there && k == cut.bound;
    const unsigned long long levels = __ballot(level);
    const bool take = (there && k > cut.bound) ||
                      (level && level_before + __popcll(levels & below) < cut.quota);
    const unsigned long long takes = __ballot(take);
    const int to = at + __popcll(takes & below);
    if (take) kept[to] = sinks + e;
    if (Held && take) out[to] = weight;  // all of them are in LDS: out may be x
    at += __popcll(takes);
    level_before += __popcll(levels);
  });
}

// One workgroup a (layer, sequence, head).  The weights come from memory once, into LDS; what remains
// are the passes over them there: 32 layers, 16 sequences of up to 4096 tokens, 8 heads (4096
// workgroups) take 80 us, 12 of them for the second and third histogram; 12 layers of one sequence of
// 200 tokens 8 us, latency alone.  Weights read from memory in each pass, as where more than kHeld
// are looked at, take 26 us more; 256 threads 53 more; keys in registers instead of weights in LDS
// spill, 1024 threads leave too few waves.  Several histograms, so that fewer lanes meet in a bin, and a
// fourth workgroup a compute unit (fewer weights held) change nothing.
__global__ __launch_bounds__(kThreads, 6) void k_evict_select(EvictArgs a, int64_t groups) {
  __shared__ Lds s;
  const CacheView& c = a.c;
  const int tid = threadIdx.x;
  for (int64_t unit = blockIdx.x; unit < groups; unit += gridDim.x) {
    const int64_t group = xcd_order(unit, groups);  // (layer, sequence, head)
    const int64_t lb = group / c.kv_heads;
    const int b = (int)(lb % c.seqs);
    const float* w = a.w + group * a.length;
    float* out_w = a.out_w + group * a.length;
    int32_t* kept = a.kept + group * a.max_keep;
    const int32_t* table = c.table + (size_t)b * c.width;
    const int len = clamp_len(c, c.lens[b]), want = a.keep[b], held = positions_held(c, b);
    bool ok = want >= 0 && want <= a.max_keep && want - a.sinks >= a.recent && len > want &&
              len <= a.length;
    if (ok) {
      // every page is there, and those written are no other sequence's too
      int bad = 0;
      const int pages = (int)fast_div(c.page_div, (uint32_t)len + c.page_div.d - 1);
      for (int p = tid; p < pages; p += kThreads) {
        const int page = table[p], pos = p * c.page_size;
        if (!names_page(c, held, pos, page)) bad = 1;
        else if (c.refcount && pos < want && pos + c.page_size > a.sinks && c.refcount[page] > 1)
          bad = 1;
      }
      ok = !__syncthreads_or(bad);
    }
    if (group < (int64_t)c.seqs * c.kv_heads && group % c.kv_heads == 0 && tid == 0)
      a.out_lens[b] = ok ? want : len;
    for (int j = (ok ? want : 0) + tid; j < a.max_keep; j += kThreads) kept[j] = -1;
    if (!ok) {
      if (out_w != w)
        for (int j = tid; j < a.length; j += kThreads) out_w[j] = w[j];
      continue;
    }
    for (int j = tid; j < a.sinks; j += kThreads) kept[j] = j;
    for (int j = tid; j < a.recent; j += kThreads) kept[want - a.recent + j] = len - a.recent + j;
    const int m = len - a.sinks - a.recent, count = want - a.sinks - a.recent;
    const bool held_all = m <= kHeld;
    if (count > 0) {
      const float* x = w + a.sinks;
      if (held_all) list_largest<true>(s, x, m, count, a.sinks, kept + a.sinks, out_w + a.sinks);
      else list_largest<false>(s, x, m, count, a.sinks, kept + a.sinks, nullptr);
    }
    __syncthreads();
    // the other weights follow; those of tokens that are gone become 0, those behind len stay
    if (out_w != w)
      for (int j = tid; j < a.sinks; j += kThreads) out_w[j] = w[j];
    for (int j0 = held_all ? want - a.recent : a.sinks; j0 < want; j0 += kThreads) {
      const int j = j0 + tid;
      const float x = j < want ? w[kept[j]] : 0.0f;
      all_read();
      if (j < want) out_w[j] = x;
    }
    for (int j = want + tid; j < len; j += kThreads) out_w[j] = 0.0f;
    if (out_w != w)
      for (int j = len + tid; j < a.length; j += kThreads) out_w[j] = w[j];
  }
}

// One workgroup for the keys or the values of a (layer, sequence, head).  Bound by memory: rows of
// 256 bytes, each read and written once, 3.4 GB in 697 us, 4.9 TB/s (a large copy: 5.2).  Selection
// and move together: loads and stores past the caches, as no row is needed again, 859 -> 817 us, the
// heads of a token on one XCD at about the same time -> 795, rows known a round ahead -> 775.  Four
// rows a thread in flight; two 783, five 779, eight, before that, 1039 against 802 (registers leave
// fewer waves).  Moving in the selection's own launch spills: 769 here, but 113 us against 93 for two
// sequences of 4096 tokens, and 77 against 68 for eight of 400; one of 200 tokens 16 against 17.
//
// One workgroup a head, whatever its length: a few long lists leave the GPU idle.  30000 of 32768 tokens
// in 8 heads take 390 us with the selection (what they move 48), in one 500 (6), in 64 430 (385).
__global__ __launch_bounds__(kThreads) void k_evict_move(EvictArgs a, int64_t groups,
                                                         FastDiv row_div) {
  const CacheView& c = a.c;
  const int tid = threadIdx.x;
  const int vecs = (int)row_div.d, step = kThreads / vecs;  // rows that the threads cover
  const int my = (int)fast_div(row_div, (uint32_t)tid), at = (tid - my * vecs) * 16;
  for (int64_t unit = blockIdx.x; unit < 2 * groups; unit += gridDim.x) {
    const int64_t x = xcd_order(unit, 2 * groups);
    const int64_t group = x >> 1;
    const int32_t* kept = a.kept + group * a.max_keep;
    const int64_t lb = group / c.kv_heads;
    const int b = (int)(lb % c.seqs), want = a.keep[b];
    if (want <= 0 || kept[0] < 0) continue;  // left alone
    const int32_t* table = c.table + (size_t)b * c.width;
    char* base = (x & 1 ? c.v : c.k) + lb / c.seqs * c.layer_stride +
                 (group - lb * c.kv_heads) * c.head_stride + at;
    auto row = [&](int pos) __attribute__((always_inline)) {
      const uint32_t pi = fast_div(c.page_div, (uint32_t)pos);
      return base + (int64_t)table[pi] * c.page_stride +
             (int64_t)(pos - (int)(pi * c.page_div.d)) * c.token_stride;
    };
    // a round's rows are known a round ahead: from[] is nullptr where there is nothing to move
    const char *from[kMoveRows], *next[kMoveRows];
    auto find = [&](int j0, const char* (&at)[kMoveRows]) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kMoveRows; ++i) {
        const int j = j0 + i * step + my, k = my < step && j < want ? kept[j] : j;
        at[i] = k != j ? row(k) : nullptr;
      }
    };
    find(a.sinks, from);
    for (int j0 = a.sinks; j0 < want; j0 += kMoveRows * step) {
      u32x4 r[kMoveRows];
      char* to[kMoveRows];
#pragma unroll
      for (int i = 0; i < kMoveRows; ++i)
        if (from[i]) r[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from[i]));
#pragma unroll
      for (int i = 0; i < kMoveRows; ++i)
        if (from[i]) to[i] = row(j0 + i * step + my);
      find(j0 + kMoveRows * step, next);
      all_read();
#pragma unroll
      for (int i = 0; i < kMoveRows; ++i) {
        if (from[i]) __builtin_nontemporal_store(r[i], reinterpret_cast<u32x4*>(to[i]));
        from[i] = next[i];
      }
    }
  }
}

}  // namespace

hipError_t launch_cache_evict(const EvictArgs& a, hipStream_t stream) {
  const int64_t groups = (int64_t)a.c.layers * a.c.seqs * a.c.kv_heads;
  const unsigned blocks = (unsigned)(groups < kMaxBlocks ? groups : kMaxBlocks);
  hipLaunchKernelGGL(k_evict_select, dim3(blocks), dim3(kThreads), 0, stream, a, groups);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned moves = (unsigned)(2 * groups < kMaxBlocks ? 2 * groups : kMaxBlocks);
  hipLaunchKernelGGL(k_evict_move, dim3(moves), dim3(kThreads), 0, stream, a, groups,
                     make_fast_div((uint32_t)(a.c.head_dim * a.c.esize / 16)));
  return hipGetLastError();
}

}  // namespace sv
