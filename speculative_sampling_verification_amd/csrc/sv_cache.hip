// Rows and pages of a paged key/value cache on gfx950: drafted nodes written behind the
// committed tokens (k_append), an accepted path's rows moved together (k_commit), sequences
// grown, trimmed and freed in a pool of counted pages (k_pool_resize) and forked with shared
// full pages (k_pool_fork, k_fork_copy).  All of it moves or counts; nothing is computed.
//
// The pool's state is one reference count a page: a page is free iff its count is 0, and the
// free pages of lowest index are taken first.  Which page a sequence gets therefore depends on
// the counts alone, not on the order in which earlier pages came back, and the counts are
// changed by integer atomics whose order does not matter.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "sv_cache.hpp"

namespace sv {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMoveThreads = 256;
constexpr int kPoolThreads = 1024;
constexpr int kPoolWaves = kPoolThreads / 64;

// One thread per 16 bytes of a node's keys, and the same of its values: both loads are on their
// way together, and rows of a page are written in full lines.  Bound by the bytes (16 sequences of
// up to 1000 tokens, 8 kv heads of 128 bf16: 124 MB read and written in 20 us, 6.2 TB/s); a few
// nodes take 2 us, the latency of length, table entry and row one after the other.
__global__ __launch_bounds__(kMoveThreads) void k_append(CacheView c, const char* k_new,
                                                         const char* v_new, int64_t new_seq,
                                                         int64_t new_node, int64_t new_head,
                                                         const int32_t* nodes, int N,
                                                         FastDiv row_div, FastDiv head_div) {
  const int b = blockIdx.y;
  const uint32_t x = blockIdx.x * kMoveThreads + threadIdx.x;
  const int i = (int)fast_div(row_div, x);
  const uint32_t y = x - (uint32_t)i * row_div.d;
  const int h = (int)fast_div(head_div, y);
  const int at = (int)(y - (uint32_t)h * head_div.d) * 16;
  const int n = nodes ? nodes[b] : N;
  if (i >= n || i >= N) return;
  const int64_t row = row_offset(c, b, positions_held(c, b), clamp_len(c, c.lens[b]) + i);
  if (row < 0) return;
  const int64_t from = (int64_t)b * new_seq + (int64_t)i * new_node + (int64_t)h * new_head + at;
  const int64_t to = row + (int64_t)h * c.head_stride + at;
  const u32x4 kx = *reinterpret_cast<const u32x4*>(k_new + from);
  const u32x4 vx = *reinterpret_cast<const u32x4*>(v_new + from);
  *reinterpret_cast<u32x4*>(c.k + to) = kx;
  *reinterpret_cast<u32x4*>(c.v + to) = vx;
}

size_t commit_lds_bytes(int N) { return (size_t)N * (2 * sizeof(int64_t) + 4 + 2) + 8; }

// Accepted path of a breadth-first tree: node path[d] at depth d has path[d] >= d, so row
// len + path[d] moves down to len + d and, taken in increasing d, no move overwrites a row that
// a later one reads.  A thread owns 16 bytes of a row in one layer's keys or values and moves
// them for every depth, eight rows in flight; no other thread touches them.  Every workgroup
// finds the path anew in LDS (a few loads of LDS one after the other), which is less than another
// launch.  Bound by latency: 32 trees of 64 nodes, paths of 6, in 32 layers of 8 kv heads of 128
// bf16 (28 MB) take 6.8 us; one tree of 16 nodes in 12 layers 3.6 us.
__global__ __launch_bounds__(kMoveThreads) void k_commit(CacheView c, const int32_t* parent,
                                                         const int32_t* last, int N,
                                                         int32_t* out_lens, FastDiv row_div,
                                                         FastDiv head_div) {
  extern __shared__ int64_t commit_lds[];   // commit_lds_bytes(N)
  int64_t* from = commit_lds;               // row offsets along the path
  int64_t* to = from + N;
  int32_t* up = reinterpret_cast<int32_t*>(to + N);     // parents
  int16_t* walk = reinterpret_cast<int16_t*>(up + N);   // the path from its end
  __shared__ int depth_sh, bad_sh;
  const int b = blockIdx.y, tid = threadIdx.x;
  const int len = clamp_len(c, c.lens[b]), held = positions_held(c, b);
  const int end = last[b];
  bool ok = end >= 0 && end < N;
  if (tid == 0) bad_sh = 0;
  if (parent) {
    for (int i = tid; i < N; i += kMoveThreads) up[i] = parent[(size_t)b * N + i];
    __syncthreads();
    if (tid == 0) {
      int d = -1;
      if (ok) {
        d = 0;
        for (int node = end; node != 0; ++d) {
          walk[d] = (int16_t)node;
          const int p = up[node];
          if (p < 0 || p >= node) {
            d = -1;
            break;
          }
          node = p;
        }
      }
      depth_sh = d;
    }
  } else if (tid == 0) {
    depth_sh = ok ? end : -1;
  }
  __syncthreads();
  const int depth = depth_sh;
  for (int d = tid; d <= depth; d += kMoveThreads) {
    const int node = !parent ? d : d == 0 ? 0 : walk[depth - d];
    const int64_t src = row_offset(c, b, held, len + node), dst = row_offset(c, b, held, len + d);
    if (src < 0 || dst < 0) bad_sh = 1;
    from[d] = src;
    to[d] = dst;
  }
  __syncthreads();
  ok = depth >= 0 && bad_sh == 0;
  if (blockIdx.x == 0 && tid == 0) out_lens[b] = ok ? len + depth + 1 : len;
  if (!ok || !parent) return;
  const uint32_t x = blockIdx.x * kMoveThreads + tid;  // (layer, k or v, head, vector)
  const uint32_t lk = fast_div(row_div, x);
  const uint32_t y = x - lk * row_div.d;
  const uint32_t h = fast_div(head_div, y);
  if ((int)(lk >> 1) >= c.layers) return;
  char* base = (lk & 1 ? c.v : c.k) + (int64_t)(lk >> 1) * c.layer_stride +
               (int64_t)h * c.head_stride + (int64_t)(y - h * head_div.d) * 16;
  int d0 = 1;
  while (d0 <= depth && from[d0] == to[d0]) ++d0;
  for (; d0 <= depth; d0 += 8) {
    u32x4 r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (d0 + i <= depth) r[i] = *reinterpret_cast<const u32x4*>(base + from[d0 + i]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (d0 + i <= depth) *reinterpret_cast<u32x4*>(base + to[d0 + i]) = r[i];
  }
}

// ------------------------------------------------------------------------------- page pool
// One workgroup: the counts of a full pool are at most a few hundred kilobytes, and each step
// depends on the one before (what is given back can be taken, sequences are served in order), so
// several would wait for each other across the GPU twice.  Bound by that chain of loads, prefix
// sums and stores: for 8 sequences over 600 pages 5.4 us taking pages and 4.0 giving them back; for
// 1024 sequences over 131072 pages, four each, 9.8 and 7.6 us (the search passes 16 KB of counts a
// round, and ends where enough are found).

struct PoolScan {
  int2 wave[2][kPoolWaves];
};
static_assert(3 * sizeof(int) * kCacheMaxSeqs + sizeof(PoolScan) <= 160 * 1024,
              "both pool kernels keep three words a sequence in a compute unit's LDS");

// Exclusive prefix of a pair a thread over the workgroup; totals in *all.  `side` alternates
// between calls: one barrier each.
__device__ __forceinline__ int2 block_prefix(PoolScan& s, int side, int2 x, int2* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int2 incl = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(incl.x, d), z = __shfl_up(incl.y, d);
    incl.x += lane >= d ? y : 0;
    incl.y += lane >= d ? z : 0;
  }
  if (lane == 63) s.wave[side][wave] = incl;
  __syncthreads();
  int2 before = make_int2(0, 0), total = make_int2(0, 0);
#pragma unroll
  for (int i = 0; i < kPoolWaves; ++i) {
    const int2 w = s.wave[side][i];
    before.x += i < wave ? w.x : 0;
    before.y += i < wave ? w.y : 0;
    total.x += w.x;
    total.y += w.y;
  }
  *all = total;
  return make_int2(before.x + incl.x - x.x, before.y + incl.y - x.y);
}

// Replaces two rows of counts in LDS (each thread's own entries i = thread mod kPoolThreads) by
// their exclusive prefix sums; returns the totals.
__device__ __forceinline__ int2 prefix_counts(PoolScan& s, int* u, int* v, int n) {
  int2 base = make_int2(0, 0);
  int side = 0;
  for (int i0 = 0; i0 < n; i0 += kPoolThreads, side ^= 1) {
    const int i = i0 + threadIdx.x;
    int2 all;
    const int2 p =
        block_prefix(s, side, i < n ? make_int2(u[i], v[i]) : make_int2(0, 0), &all);
    if (i < n) {
      u[i] = base.x + p.x;
      v[i] = base.y + p.y;
    }
    base.x += all.x;
    base.y += all.y;
  }
  __syncthreads();
  return base;
}

// Largest i with prefix[i] <= r (prefix ascending, prefix[0] = 0): the owner of item r.
__device__ __forceinline__ int owner_of(const int* prefix, int n, int r) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Calls take(owner, rank in owner, page) for the free pages of lowest index, the owners' shares
// given by `prefix` (a thread's ranks follow each other: one search, then steps), until `want`
// are taken; returns how many there were.  Four pages a thread and round (few, so that the pages
// found are spread over many threads), the next round's counts on their way meanwhile.
template <class F>
__device__ __forceinline__ int for_free_pages(PoolScan& s, const CacheView& c, int want,
                                              const int* prefix, int n, F take) {
  constexpr int kPer = 4, kRound = kPoolThreads * kPer;
  const bool vec = (reinterpret_cast<uintptr_t>(c.refcount) & 15u) == 0;
  auto load = [&](int64_t p) {  // a page behind the last counts as held
    int4 x = make_int4(1, 1, 1, 1);
    if (vec && p + kPer <= c.pages) {
      x = *reinterpret_cast<const int4*>(c.refcount + p);
    } else {
      if (p < c.pages) x.x = c.refcount[p];
      if (p + 1 < c.pages) x.y = c.refcount[p + 1];
      if (p + 2 < c.pages) x.z = c.refcount[p + 2];
      if (p + 3 < c.pages) x.w = c.refcount[p + 3];
    }
    return x;
  };
  int base = 0, side = 0;
  int4 next = load((int64_t)threadIdx.x * kPer);
  for (int64_t p0 = 0; p0 < c.pages && base < want; p0 += kRound, side ^= 1) {
    const int64_t p = p0 + (int64_t)threadIdx.x * kPer;
    const int4 x = next;
    next = load(p + kRound);
    uint32_t free = (x.x == 0) | (x.y == 0) << 1 | (x.z == 0) << 2 | (x.w == 0) << 3;
    int2 all;
    int rank = base + block_prefix(s, side, make_int2(__popc(free), 0), &all).x;
    if (free && rank < want) {
      int b = owner_of(prefix, n, rank);
      for (; free && rank < want; ++rank) {
        const int i = __ffs(free) - 1;
        free &= free - 1;
        while (b + 1 < n && prefix[b + 1] <= rank) ++b;
        take(b, rank - prefix[b], (int)p + i);
      }
    }
    base += all.x;
  }
  return base < want ? base : want;
}

__global__ __launch_bounds__(kPoolThreads) void k_pool_resize(CacheView c, const int32_t* want,
                                                              const int32_t* new_lens,
                                                              int32_t* out_ok) {
  // prefix sums of the entries each sequence gives back and takes; kept: the entries that stay
  // (what is dropped or taken follows them), complemented where a value is out of range
  __shared__ int drop[kCacheMaxSeqs], grow[kCacheMaxSeqs], kept[kCacheMaxSeqs];
  __shared__ PoolScan s;
  const int n = c.seqs;
  for (int b = threadIdx.x; b < n; b += kPoolThreads) {
    const int held = c.held[b], w = want[b], nl = new_lens ? new_lens[b] : 0;
    int len = c.lens[b];
    bool ok = held >= 0 && held <= c.width;
    if (ok && new_lens) {
      ok = nl >= 0 && nl <= (int64_t)held * c.page_size;
      const int old = min(max(len, 0), held * (int)c.page_div.d);
      if (ok && nl < old && w != 0) {
        // cut back into committed tokens: their pages are written again, so no other sequence
        // may hold them.  (Counts before this call's changes; loads that leave none behind in
        // the L1, as the changes are made in the L2.)  All pages stay where want is negative, or
        // out of range and about to be refused.
        const int kept_to = w < nl || w > c.cap ? old : min(old, w);
        const int end = (int)fast_div(c.page_div, (uint32_t)kept_to + c.page_div.d - 1);
        for (int j = (int)fast_div(c.page_div, (uint32_t)nl); j < end; ++j) {
          const int page = c.table[(size_t)b * c.width + j];
          if (page >= 0 && page < c.pages &&
              __hip_atomic_load(&c.refcount[page], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 1)
            ok = false;
        }
      }
      if (ok) c.lens[b] = len = nl;
    }
    ok = ok && (w <= 0 || (w >= len && w <= c.cap));
    if (ok && w == 0) c.lens[b] = 0;
    const int need =
        !ok || w < 0 ? held : (int)fast_div(c.page_div, (uint32_t)w + c.page_div.d - 1);
    // a sequence that is refused reaches no page by the entries it asked for (here those whose
    // values are out of range, below those that do not fit), whatever they named before
    if (!ok && held >= 0 && w > 0) {
      const int asked = (int)fast_div(c.page_div, (uint32_t)min(w, c.cap) + c.page_div.d - 1);
      for (int j = held; j < asked; ++j) c.table[(size_t)b * c.width + j] = -1;
    }
    drop[b] = need < held ? held - need : 0;
    grow[b] = need > held ? need - held : 0;
    kept[b] = ok ? min(held, need) : ~0;
  }
  const int2 totals = prefix_counts(s, drop, grow, n);
  const int dropped = totals.x, wanted = totals.y;

  // four dropped pages a thread and round, one after the other
  constexpr int kRun = 4;
  for (uint32_t r0 = threadIdx.x * kRun; r0 < (uint32_t)dropped; r0 += kPoolThreads * kRun) {
    int page[kRun], b = owner_of(drop, n, (int)r0);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int r = (int)r0 + i;
      page[i] = -1;
      if (r < dropped) {
        while (b + 1 < n && drop[b + 1] <= r) ++b;
        page[i] = c.table[(size_t)b * c.width + kept[b] + r - drop[b]];
      }
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i)
      if (page[i] >= 0 && page[i] < c.pages) atomicSub(&c.refcount[page[i]], 1);
  }
  int got = 0;
  if (wanted) {
    // the counts are changed and read by this workgroup alone; the atomics act in the L2, whose
    // lines none of its loads has brought into the L1 yet
    __threadfence_block();
    __syncthreads();
    got = for_free_pages(s, c, wanted, grow, n, [&](int b, int i, int page) {
      c.table[(size_t)b * c.width + kept[b] + i] = page;
      c.refcount[page] = 1;
    });
    __threadfence_block();
    __syncthreads();
  }

  // sequences are served in order until one does not fit; what that one was given goes back
  for (int b = threadIdx.x; b < n; b += kPoolThreads) {
    const int first = grow[b], g = (b + 1 < n ? grow[b + 1] : wanted) - first;
    int ok = kept[b] >= 0;
    if (ok && g > 0 && first + g > got) {
      ok = 0;
      for (int r = first; r < got; ++r)
        c.refcount[c.table[(size_t)b * c.width + kept[b] + r - first]] = 0;
      for (int i = 0; i < g; ++i) c.table[(size_t)b * c.width + kept[b] + i] = -1;
    }
    if (ok) c.held[b] = kept[b] + g;
    out_ok[b] = ok;
  }
}

__global__ __launch_bounds__(kPoolThreads) void k_pool_fork(CacheView c, const int32_t* src,
                                                            const int32_t* dst, int F,
                                                            int32_t* out_ok) {
  // first[s]: the first fork into slot s, F if none; bit 31: s is some fork's source
  __shared__ uint32_t first[kCacheMaxSeqs];
  // prefix sums of the pages each fork needs (0 or 1) and of the full pages it shares
  __shared__ int part[kCacheMaxSeqs], full[kCacheMaxSeqs];
  __shared__ PoolScan s;
  for (int i = threadIdx.x; i < c.seqs; i += kPoolThreads) first[i] = (uint32_t)F;
  __syncthreads();
  for (int f = threadIdx.x; f < F; f += kPoolThreads) {
    const int d = dst[f];
    if (d >= 0 && d < c.seqs) atomicMin(&first[d], (uint32_t)f);
  }
  __syncthreads();
  for (int f = threadIdx.x; f < F; f += kPoolThreads) {
    const int x = src[f];
    if (x >= 0 && x < c.seqs) atomicOr(&first[x], 0x80000000u);
  }
  __syncthreads();
  // a fork needs a page where its source's last page is begun
  for (int f = threadIdx.x; f < F; f += kPoolThreads) {
    const int x = src[f], d = dst[f];
    bool ok = x >= 0 && x < c.seqs && d >= 0 && d < c.seqs;
    const int len = ok ? c.lens[x] : 0, held = ok ? c.held[x] : 0, there = ok ? c.held[d] : 0;
    // into an empty slot that is no fork's source, and by its first fork
    ok = ok && first[d] == (uint32_t)f && there == 0;
    ok = ok && len >= 0 && held >= 0 && held <= c.width && len <= (int64_t)held * c.page_size;
    const int whole = ok ? (int)fast_div(c.page_div, (uint32_t)len) : 0;
    bool begun = ok && len != whole * c.page_size;
    if (begun) {
      const int page = c.table[(size_t)x * c.width + whole];
      ok = begun = page >= 0 && page < c.pages;
    }
    part[f] = begun ? 1 : 0;
    full[f] = ok ? whole : 0;
    out_ok[f] = ok ? 1 : 0;
  }
  const int2 totals = prefix_counts(s, part, full, F);
  const int wanted = totals.x, shared = totals.y;
  auto count = [&](const int* prefix, int f, int all) {
    return (f + 1 < F ? prefix[f + 1] : all) - prefix[f];
  };
  const int got = for_free_pages(s, c, wanted, part, F, [&](int f, int, int page) {
    c.table[(size_t)dst[f] * c.width + count(full, f, shared)] = page;
    c.refcount[page] = 1;
  });
  // a fork without the page it needs fails; the others take their length and the full pages
  auto served = [&](int f) { return count(part, f, wanted) == 0 || part[f] < got; };
  for (int f = threadIdx.x; f < F; f += kPoolThreads) {
    if (out_ok[f] != 1) continue;
    if (served(f)) {
      const int d = dst[f];
      c.held[d] = count(full, f, shared) + count(part, f, wanted);
      c.lens[d] = c.lens[src[f]];
    } else {
      out_ok[f] = 0;
    }
  }
  for (uint32_t r = threadIdx.x; r < (uint32_t)shared; r += kPoolThreads) {
    const int f = owner_of(full, F, (int)r), j = (int)r - full[f];
    if (!served(f)) continue;
    const int page = c.table[(size_t)src[f] * c.width + j];
    c.table[(size_t)dst[f] * c.width + j] = page;
    if (page >= 0 && page < c.pages) atomicAdd(&c.refcount[page], 1);
  }
}

// Copies the begun page of every fork: workgroup (layer and k or v, fork, `rows` of the page).
// Bound by the bytes: 64 forks in 32 layers, up to 15 tokens of 8 kv heads of 128 bf16 each, 135 MB
// read and written in 22 us, 6 TB/s; the pool kernel before it takes 8 us.
__global__ __launch_bounds__(kMoveThreads) void k_fork_copy(CacheView c, const int32_t* src,
                                                            const int32_t* dst,
                                                            const int32_t* ok, int rows,
                                                            FastDiv row_div, FastDiv head_div) {
  const int f = blockIdx.y;
  if (ok[f] != 1) return;
  const int x = src[f], y = dst[f], len = c.lens[x];
  const int full = (int)fast_div(c.page_div, (uint32_t)len);
  const int row0 = blockIdx.z * rows;
  const int rest = min(len - full * c.page_size - row0, rows);
  if (rest <= 0) return;
  const int64_t from = (int64_t)c.table[(size_t)x * c.width + full] * c.page_stride;
  const int64_t to = (int64_t)c.table[(size_t)y * c.width + full] * c.page_stride;
  char* base = (blockIdx.x & 1 ? c.v : c.k) + (int64_t)(blockIdx.x >> 1) * c.layer_stride +
               (int64_t)row0 * c.token_stride;
  const uint32_t all = (uint32_t)rest * row_div.d;
#pragma unroll 4
  for (uint32_t i = threadIdx.x; i < all; i += kMoveThreads) {
    const uint32_t row = fast_div(row_div, i), z = i - row * row_div.d;
    const uint32_t h = fast_div(head_div, z);
    const int64_t at = (int64_t)row * c.token_stride + (int64_t)h * c.head_stride +
                       (int64_t)(z - h * head_div.d) * 16;
    *reinterpret_cast<u32x4*>(base + to + at) = *reinterpret_cast<const u32x4*>(base + from + at);
  }
}

int head_vecs(const CacheView& c) { return c.head_dim * c.esize / 16; }

}  // namespace

hipError_t launch_cache_append(const CacheView& c, const char* k_new, const char* v_new,
                               int64_t new_seq, int64_t new_node, int64_t new_head,
                               const int32_t* nodes, int N, hipStream_t stream) {
  const int hv = head_vecs(c), rv = hv * c.kv_heads;
  const unsigned blocks = (unsigned)(((int64_t)N * rv + kMoveThreads - 1) / kMoveThreads);
  hipLaunchKernelGGL(k_append, dim3(blocks, c.seqs), dim3(kMoveThreads), 0, stream, c, k_new,
                     v_new, new_seq, new_node, new_head, nodes, N, make_fast_div(rv),
                     make_fast_div(hv));
  return hipGetLastError();
}

hipError_t launch_cache_commit(const CacheView& c, const int32_t* parent, const int32_t* last,
                               int N, int32_t* out_lens, hipStream_t stream) {
  const int hv = head_vecs(c), rv = hv * c.kv_heads;
  const int64_t cols = parent ? (int64_t)c.layers * 2 * rv : 1;
  const unsigned blocks = (unsigned)((cols + kMoveThreads - 1) / kMoveThreads);
  hipLaunchKernelGGL(k_commit, dim3(blocks, c.seqs), dim3(kMoveThreads),
                     commit_lds_bytes(N), stream, c, parent, last, N, out_lens, make_fast_div(rv),
                     make_fast_div(hv));
  return hipGetLastError();
}

hipError_t launch_cache_resize(const CacheView& c, const int32_t* want, const int32_t* new_lens,
                               int32_t* out_ok, hipStream_t stream) {
  hipLaunchKernelGGL(k_pool_resize, dim3(1), dim3(kPoolThreads), 0, stream, c, want, new_lens,
                     out_ok);
  return hipGetLastError();
}

hipError_t launch_cache_fork(const CacheView& c, const int32_t* src, const int32_t* dst, int F,
                             int32_t* out_ok, hipStream_t stream) {
  hipLaunchKernelGGL(k_pool_fork, dim3(1), dim3(kPoolThreads), 0, stream, c, src, dst, F, out_ok);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int hv = head_vecs(c), rv = hv * c.kv_heads;
  // 256 KB a workgroup, more where a page has more than 65535 of them (at most 2^30 vectors)
  int rows = (256 * 1024 / 16 + rv - 1) / rv;
  rows = rows > (c.page_size + 65534) / 65535 ? rows : (c.page_size + 65534) / 65535;
  hipLaunchKernelGGL(k_fork_copy, dim3(2 * c.layers, F, (c.page_size + rows - 1) / rows),
                     dim3(kMoveThreads), 0, stream, c, src, dst, out_ok, rows, make_fast_div(rv),
                     make_fast_div(hv));
  return hipGetLastError();
}

}  // namespace sv
