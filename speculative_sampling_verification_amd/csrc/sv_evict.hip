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

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 512;
constexpr int kMoveRows = 4;               // rows that a thread has in flight
constexpr int64_t kEvictMaxBlocks = 1 << 20;

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

struct SelLds {
  int hist[kBins];
  int wave[kSelWaves];
  int2 wave2[kSelWaves];
  int digit, left, inside;
};

// What is kept of the weights x[0 .. m): those whose key >> shift is above `bound`, and the first
// `quota` of those where it equals it.
struct Cut {
  uint32_t bound;
  int shift, quota;
};

// The `count` largest of the m weights (0 < count < m).
__device__ Cut find_cut(SelLds& s, const float* x, int m, int count) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Cut cut{0u, 32, count};
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10, shift = cut.shift - bits;
    for (int i = tid; i < kBins; i += kSelThreads) s.hist[i] = 0;
    __syncthreads();
    for (int e0 = 0; e0 < m; e0 += kSelThreads) {
      const int e = e0 + tid;
      const uint32_t key = e < m ? order_of(x[e]) : 0u;
      const bool in = e < m && (cut.shift == 32 || key >> cut.shift == cut.bound);
      const int d = (int)(key >> shift & ((1u << bits) - 1));
      // lanes of one bin, as where many weights are alike, add together
      const unsigned long long some = __ballot(in);
      if (!some) continue;
      const int first = __ffsll(some) - 1, d0 = __shfl(d, first);
      if (__ballot(in && d != d0) == 0) {
        if (lane == first) atomicAdd(&s.hist[d0], __popcll(some));
      } else if (in) {
        atomicAdd(&s.hist[d], 1);
      }
    }
    __syncthreads();
    // two bins a thread, largest first
    const int top = kBins - 1 - 2 * tid;
    const int n0 = s.hist[top], n1 = s.hist[top - 1];
    int incl = n0 + n1;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
      const int y = __shfl_up(incl, k);
      incl += lane >= k ? y : 0;
    }
    if (lane == 63) s.wave[wave] = incl;
    __syncthreads();
    int before = incl - n0 - n1;
    for (int i = 0; i < wave; ++i) before += s.wave[i];
    if (before < cut.quota && cut.quota <= before + n0 + n1) {
      const bool second = before + n0 < cut.quota;
      s.digit = second ? top - 1 : top;
      s.left = cut.quota - before - (second ? n0 : 0);
      s.inside = second ? n1 : n0;
    }
    __syncthreads();
    cut.bound = (cut.shift == 32 ? 0u : cut.bound << bits) | (uint32_t)s.digit;
    cut.shift = shift;
    cut.quota = s.left;
    const bool all = s.left == s.inside;  // the whole bin is kept
    __syncthreads();
    if (all) break;
  }
  return cut;
}

__global__ __launch_bounds__(kSelThreads) void k_evict_select(EvictArgs a, int64_t groups) {
  __shared__ SelLds s;
  const CacheView& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int64_t group = blockIdx.x; group < groups; group += gridDim.x) {  // (layer, sequence, head)
    const int b = (int)(group / c.kv_heads % c.seqs);
    const float* w = a.w + group * a.length;
    float* out_w = a.out_w + group * a.length;
    int32_t* kept = a.kept + group * a.max_keep;
    const int len = clamp_len(c, c.lens[b]), want = a.keep[b], held = positions_held(c, b);
    bool ok = want >= 0 && want <= a.max_keep && want - a.sinks >= a.recent && len > want &&
              len <= a.length;
    if (ok) {
      // every page is there, and those written are no other sequence's too
      int bad = 0;
      const int pages = (int)fast_div(c.page_div, (uint32_t)len + c.page_div.d - 1);
      for (int p = tid; p < pages; p += kSelThreads) {
        const int page = c.table[(size_t)b * c.width + p], pos = p * c.page_size;
        if (!names_page(c, held, pos, page)) bad = 1;
        else if (c.refcount && pos < want && pos + c.page_size > a.sinks && c.refcount[page] > 1)
          bad = 1;
      }
      ok = !__syncthreads_or(bad);
    }
    if (group < (int64_t)c.seqs * c.kv_heads && group % c.kv_heads == 0 && tid == 0)
      a.out_lens[b] = ok ? want : len;
    for (int j = (ok ? want : 0) + tid; j < a.max_keep; j += kSelThreads) kept[j] = -1;
    if (!ok) {
      if (out_w != w)
        for (int j = tid; j < a.length; j += kSelThreads) out_w[j] = w[j];
      continue;
    }
    for (int j = tid; j < a.sinks; j += kSelThreads) kept[j] = j;
    for (int j = tid; j < a.recent; j += kSelThreads) kept[want - a.recent + j] = len - a.recent + j;
    const int m = len - a.sinks - a.recent, count = want - a.sinks - a.recent;
    if (count > 0) {
      const float* x = w + a.sinks;
      const Cut cut = find_cut(s, x, m, count);
      // a wave lists the tokens of a stretch of its own, behind those of the waves before it
      const int stretch = ((m + kSelThreads - 1) / kSelThreads) * 64;
      const int e0 = wave * stretch, e1 = e0 + stretch < m ? e0 + stretch : m;
      auto above = [&](int e, bool* level) {
        const uint32_t key = order_of(x[e]) >> cut.shift;
        *level = key == cut.bound;
        return key > cut.bound;
      };
      int above_n = 0, level_n = 0;
      for (int e = e0; e < e1; e += 64) {
        bool level = false, over = false;
        if (e + lane < e1) over = above(e + lane, &level);
        above_n += __popcll(__ballot(over));
        level_n += __popcll(__ballot(level));
      }
      if (lane == 0) s.wave2[wave] = make_int2(above_n, level_n);
      __syncthreads();
      int above_before = 0, level_before = 0;
      for (int i = 0; i < wave; ++i) {
        above_before += s.wave2[i].x;
        level_before += s.wave2[i].y;
      }
      int at = a.sinks + above_before + (level_before < cut.quota ? level_before : cut.quota);
      const unsigned long long below = (1ull << lane) - 1;
      for (int e = e0; e < e1; e += 64) {
        bool level = false, over = false;
        if (e + lane < e1) over = above(e + lane, &level);
        const unsigned long long levels = __ballot(level);
        const bool take = over || (level && level_before + __popcll(levels & below) < cut.quota);
        const unsigned long long takes = __ballot(take);
        if (take) kept[at + __popcll(takes & below)] = a.sinks + e + lane;
        at += __popcll(takes);
        level_before += __popcll(levels);
      }
    }
    __syncthreads();
    // the weights follow; those of tokens that are gone become 0, those behind len stay
    for (int j0 = 0; j0 < want; j0 += kSelThreads) {
      const int j = j0 + tid;
      const float x = j < want ? w[kept[j]] : 0.0f;
      all_read();
      if (j < want) out_w[j] = x;
    }
    for (int j = want + tid; j < len; j += kSelThreads) out_w[j] = 0.0f;
    if (out_w != w)
      for (int j = len + tid; j < a.length; j += kSelThreads) out_w[j] = w[j];
  }
}

// One workgroup for the keys or the values of a (layer, sequence, head).
__global__ __launch_bounds__(kMoveThreads) void k_evict_move(EvictArgs a, int64_t groups,
                                                             FastDiv row_div) {
  const CacheView& c = a.c;
  const int tid = threadIdx.x;
  const int vecs = (int)row_div.d, step = kMoveThreads / vecs;  // rows that the threads cover
  const int my = (int)fast_div(row_div, (uint32_t)tid), at = (tid - my * vecs) * 16;
  for (int64_t x = blockIdx.x; x < 2 * groups; x += gridDim.x) {
    const int64_t group = x >> 1;
    const int32_t* kept = a.kept + group * a.max_keep;
    const int64_t lb = group / c.kv_heads;
    const int b = (int)(lb % c.seqs), want = a.keep[b];
    if (want <= 0 || kept[0] < 0) continue;  // refused
    const int32_t* table = c.table + (size_t)b * c.width;
    char* base = (x & 1 ? c.v : c.k) + lb / c.seqs * c.layer_stride +
                 (group - lb * c.kv_heads) * c.head_stride + at;
    auto row = [&](int pos) {
      const uint32_t pi = fast_div(c.page_div, (uint32_t)pos);
      return base + (int64_t)table[pi] * c.page_stride +
             (int64_t)(pos - (int)(pi * c.page_div.d)) * c.token_stride;
    };
    for (int j0 = a.sinks; j0 < want; j0 += kMoveRows * step) {
      u32x4 r[kMoveRows];
      int from[kMoveRows];
#pragma unroll
      for (int i = 0; i < kMoveRows; ++i) {
        const int j = j0 + i * step + my;
        from[i] = my < step && j < want ? kept[j] : j;
        if (from[i] != j) r[i] = *reinterpret_cast<const u32x4*>(row(from[i]));
      }
      all_read();
#pragma unroll
      for (int i = 0; i < kMoveRows; ++i) {
        const int j = j0 + i * step + my;
        if (from[i] != j) *reinterpret_cast<u32x4*>(row(j)) = r[i];
      }
    }
  }
}

}  // namespace

hipError_t launch_cache_evict(const EvictArgs& a, hipStream_t stream) {
  const int64_t groups = (int64_t)a.c.layers * a.c.seqs * a.c.kv_heads;
  const unsigned blocks = (unsigned)(groups < kEvictMaxBlocks ? groups : kEvictMaxBlocks);
  hipLaunchKernelGGL(k_evict_select, dim3(blocks), dim3(kSelThreads), 0, stream, a, groups);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned moves = (unsigned)(2 * groups < kEvictMaxBlocks ? 2 * groups : kEvictMaxBlocks);
  hipLaunchKernelGGL(k_evict_move, dim3(moves), dim3(kMoveThreads), 0, stream, a, groups,
                     make_fast_div((uint32_t)(a.c.head_dim * a.c.esize / 16)));
  return hipGetLastError();
}

}  // namespace sv
