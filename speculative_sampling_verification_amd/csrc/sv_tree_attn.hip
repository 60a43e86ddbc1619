// Attention of drafted token trees over a paged cache, on gfx950.
//
// For sequence b with len committed tokens and n drafted nodes, node i of query head h sees the
// committed keys j < len and the nodes its mask row admits (keys len + j).  With z = scale q.k,
//   m = max z,  l = sum exp(z - m),  out = sum exp(z - m) v / l,  lse = m + ln l
// over the visible keys; a row that sees nothing gives out = 0 and lse = -inf.
//
// The query heads of one kv head and the nodes form the rows r = node * G + g of one product
// with the keys, so each key and value is read once for all of them.  The scores are computed
// transposed, S^T = K Q^T with 32x32 matrix instructions: a lane then holds one row of Q and 16
// of 32 keys, so the running maximum and sum of a row live in a lane and its neighbour 32 lanes
// away, P^T is already the second operand of O^T = V^T P^T, and rescaling O is a product by a
// lane's own factor.  V^T comes out of row-major LDS by the transposing LDS read (bf16) or by
// 4-byte reads (fp32).
//
// All key tiles of all (sequence, kv head, row tile) groups form one line of equal pieces of
// work, cut evenly between the workgroups from the lengths on the device: ragged batches and
// single long sequences load every compute unit alike, and the host needs no lengths.  A group
// that spans several workgroups leaves a part (O, m, l) with each, joined by k_tree_join in
// workgroup order.
//
// What bounds it, by the rows r that share a kv head's keys (8 kv heads of 128 columns, bf16; whole
// calls one behind the other, medians): few rows, the bytes of the keys and values: r = 4, 64
// sequences of 1023 to 8191 tokens, 1.21 GB in 224 us, 5.4 TB/s.  Many rows, the products and the
// exponentials beside them (16 a lane and block of 32 keys take as many cycles as the block's 16
// matrix instructions): r = 512, 131072 tokens, 275 GFLOP in 316 us, 870 TFLOP/s, three quarters of
// what a large library product reaches on the same card, matrix units busy 46% of the cycles of a
// clock that the card lowers to 1.8 GHz; LDS reads have no bank conflicts.  Between them (r = 256,
// 32 sequences of 512 to 4096 tokens, 69 GFLOP in 130 us) the cut itself counts: 256 groups on 256
// workgroups leave 64 MB of parts, written and read again.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "sv_cache.hpp"
#include "sv_lds_load.hpp"

namespace sv {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kLdsBytes = 160 * 1024;  // of a compute unit
constexpr int kKept = 512;
constexpr float kLn2 = 0.69314718055994530942f;

// Every lambda of the kernels is part of its kernel's loop: one that the compiler calls instead, or
// whose captures it keeps in memory, is reached through private memory by flat instructions.
#define SV_INLINE __attribute__((always_inline))
#define SV_LDS(T) __attribute__((address_space(3))) T

// max / sum with the lane 32 away
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Bits of a 32-key mask (shifted down by 4 in the upper half) in a lane's register order.
__device__ __forceinline__ uint32_t of_half(uint32_t x) {
  return (x & 0xFu) | (x >> 4 & 0xF0u) | (x >> 8 & 0xF00u) | (x >> 12 & 0xF000u);
}

// Work of one sequence, in pieces of a key tile's cost: for each live row tile `fixed` pieces
// for what a group costs whatever its length, then its key tiles; one piece (zeros to write)
// for each row tile that holds no node.
struct SeqWork {
  int len, n, keys;  // committed tokens, nodes, keys behind the table
  int tiles, live;   // key tiles (at least one), row tiles with a node
};

template <int MT, int BN>
__device__ __forceinline__ SeqWork seq_work(const AttnArgs& a, int len, int n) {
  SeqWork s;
  len = len < 0 ? 0 : len;
  s.len = len > a.c.cap ? a.c.cap : len;
  n = n < 0 ? 0 : n;
  s.n = n > a.N ? a.N : n;
  const int keys = s.len + s.n;
  s.keys = keys > a.c.cap ? a.c.cap : keys;
  const int tiles = (s.keys + BN - 1) / BN;
  s.tiles = tiles < 1 ? 1 : tiles;
  s.live = (s.n * a.G + MT - 1) / MT;
  return s;
}

__device__ __forceinline__ long long seq_pieces(const AttnArgs& a, const SeqWork& s, int fixed) {
  return (long long)a.c.kv_heads * ((long long)s.live * (s.tiles + fixed) + (a.mts - s.live));
}

// x / d for 0 <= x, 0 < d < 2^31, in 32 bits where x fits (nearly always).
__device__ __forceinline__ long long div_pieces(long long x, long long d) {
  if (x >> 31 == 0) return (uint32_t)x / (uint32_t)d;
  return x / d;
}

__device__ __forceinline__ bool non_finite(uint32_t bits32) {
  return (bits32 & 0x7F800000u) == 0x7F800000u;
}

// Clears the non-finite elements of a 16-byte vector; true if there were any.
template <bool BF16>
__device__ __forceinline__ bool clear_non_finite(u32x4& x) {
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      const bool lo = non_finite(x[i] << 16), hi = non_finite(x[i]);
      any |= lo | hi;
      x[i] &= (lo ? 0xFFFF0000u : 0xFFFFFFFFu) & (hi ? 0x0000FFFFu : 0xFFFFFFFFu);
    } else {
      const bool bad = non_finite(x[i]);
      any |= bad;
      x[i] = bad ? 0u : x[i];
    }
  }
  return any;
}

// WM waves share the rows (32 each), WK the keys of a tile (KS blocks of 32 each); NST tiles are
// kept in LDS, loaded there directly from global memory: no registers hold tiles on their way, so
// the loads of one or two tiles ahead cost none.  32 rows a wave: with 64, its O and scores take
// 256 registers, which leaves one wave a SIMD and scores in the accumulation registers, and took
// 2.5 times as long.
template <bool BF16, int D, int WM, int WK, int KS, int NST>
struct Attn {
  static constexpr int kES = BF16 ? 2 : 4;
  static constexpr int kNW = WM * WK;
  static constexpr int kNT = 64 * kNW;
  static constexpr int kMT = 32 * WM;
  static constexpr int kBN = 32 * WK * KS;
  static constexpr int kRow = D * kES;        // bytes of a row, in memory and in LDS
  static constexpr int kVecs = kRow / 16;     // 16-byte vectors of a row
  static constexpr int kND = D / 32;
  static constexpr int kRing = NST == 4 ? 8 : 4;  // tiles whose rows are known
  static constexpr int kLoads = kBN * kVecs / kNT;  // vectors a thread loads per tensor
  static constexpr int kTileBytes = 2 * kBN * kRow;
  static constexpr int kJoinBytes = WK > 1 ? kNW * kND * 16 * 64 * 4 : 0;
  static constexpr int kPool = NST * kTileBytes > kJoinBytes ? NST * kTileBytes : kJoinBytes;
  static_assert(D % 32 == 0 && (kBN * kVecs) % kNT == 0 && kBN % 64 == 0 && kBN <= kNT, "tile");

  // Direct loads fill LDS in lane order, so rows are not padded; instead vector c of row r lies
  // at place c ^ swz(r) of its row, which a lane gets by loading that vector.
  // K is read 16 bytes a lane down 32 rows: 16 consecutive rows have to cover all 64 banks (16
  // places of 16 bytes).  V (bf16) is read 64 bytes wide from 4 consecutive rows at once: those
  // have to lie in four different quarters of the banks.  V (fp32) is read 128 bytes wide, and
  // the matrix instructions take 16 times as long: no swizzle.
  __device__ static __forceinline__ int swz_k(int r) {
    if constexpr (kRow % 256 == 0) return r & 15;
    else if constexpr (kRow == 128) return (r >> 1) & 7;
    else return (r >> 2) & 3;  // 192, 384: the pitch itself spreads 4 (2) rows
  }
  __device__ static __forceinline__ int swz_v(int r) {
    if constexpr (!BF16) return 0;
    else if constexpr (kRow % 256 == 0) return (r & 3) * 4;
    else if constexpr (kRow == 128) return (r >> 1 & 1) * 4;
    else return 0;             // 192: the pitch itself spreads 4 rows
  }

  struct Lds {
    alignas(1024) char pool[kPool];        // NST times (K tile, V tile); the parts when waves join
    long long rowoff[kRing][kBN];          // byte offset of a key's row (that of page 0: none)
    uint32_t valid[kRing][kBN / 32];       // keys that exist
    uint32_t badv[kRing][kBN / 32];        // drafted nodes with non-finite values
    uint32_t sees[kMT][kBN / 32];          // keys of a rough tile that a node sees
    int32_t entry[NST == 4 ? 4 : 1][kBN];  // table entries of a tile's keys
    float m[kNW][32], l[kNW][32];
    longlong2 scan[kNW];
    int2 seq[kKept];                       // lengths and node counts of the first sequences
    long long start_off;
    int start_b;
  };
};

// A value the compiler takes for a new one: what is computed from it in a loop is computed there
// and does not occupy registers all along.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// A word by each of the active lanes, likewise.
__device__ __forceinline__ void load_word_to_lds(const int32_t* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :
               : "v"(from), "s"(__builtin_amdgcn_readfirstlane(to))
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Waits for this wave's LDS accesses, then for the other waves'; loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <bool BF16, int D, int WM, int WK, int KS, int NST, int OCC>
__global__ __launch_bounds__(64 * WM * WK) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void k_tree_attn(AttnArgs a) {
  using C = Attn<BF16, D, WM, WK, KS, NST>;
  constexpr int MT = C::kMT, BN = C::kBN, NT = C::kNT, ND = C::kND;
  constexpr int QF = BF16 ? D / 16 : D / 8;  // 16-byte pieces of a Q row a lane holds
  __shared__ typename C::Lds S;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wk = wave / WM;
  const int half = lane >> 5, col = lane & 31;
  const float sl2 = a.scale * 1.44269504088896340736f;  // scores to log2 units
  const uint32_t pool_at = (uint32_t)reinterpret_cast<uintptr_t>((SV_LDS(char)*)S.pool);

  // worker number: consecutive workers share keys and should share an XCD's L2 (workgroups are
  // handed to the eight XCDs in turn)
  int w = blockIdx.x;
  if ((a.workers & 7) == 0) w = (w & 7) * (a.workers >> 3) + (w >> 3);

  // where this worker's pieces begin: prefix sums of the sequences' work
  auto work_of = [&](int b) SV_INLINE {
    return b < kKept ? seq_work<MT, BN>(a, S.seq[b].x, S.seq[b].y)
                     : seq_work<MT, BN>(a, a.c.lens[b], a.nodes ? a.nodes[b] : a.N);
  };
  long long total, per, pos, end;
  int fixed;
  {
    const int chunk = (a.c.seqs + NT - 1) / NT;
    const int b0 = tid * chunk, b1 = b0 + chunk < a.c.seqs ? b0 + chunk : a.c.seqs;
    long long mine = 0, live = 0;  // pieces without the fixed ones, live groups
    for (int b = b0; b < b1; ++b) {
      const int len = a.c.lens[b], n = a.nodes ? a.nodes[b] : a.N;
      if (b < kKept) S.seq[b] = make_int2(len, n);
      const SeqWork s = seq_work<MT, BN>(a, len, n);
      mine += seq_pieces(a, s, 0);
      live += (long long)a.c.kv_heads * s.live;
    }
    long long incl = mine, incl_live = live;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const long long y = __shfl_up(incl, d), z = __shfl_up(incl_live, d);
      incl += lane >= d ? y : 0;
      incl_live += lane >= d ? z : 0;
    }
    if (lane == 63) S.scan[wave] = make_longlong2(incl, incl_live);
    __syncthreads();
    long long before = 0, before_live = 0, groups = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < C::kNW; ++i) {
      before += i < wave ? S.scan[i].x : 0;
      before_live += i < wave ? S.scan[i].y : 0;
      total += S.scan[i].x;
      groups += S.scan[i].y;
    }
    // a group's fixed cost is about three tiles; it is counted where a worker has many
    const long long tiles_each = div_pieces(uniform(total), a.workers);
    fixed = tiles_each >= 24 ? 3 : (int)tiles_each / 8;
    total = uniform(total + groups * fixed);
    per = div_pieces(total + a.workers - 1, a.workers);
    pos = w * per;
    end = pos + per < total ? pos + per : total;
    long long p = before + incl - mine + (before_live + incl_live - live) * fixed;
    if (pos >= p && pos < p + mine + live * fixed) {
      int b = b0;
      for (; b < b1; ++b) {
        const long long u = seq_pieces(a, work_of(b), fixed);
        if (pos < p + u) break;
        p += u;
      }
      S.start_b = b;
      S.start_off = pos - p;
    }
    if (tid == 0) a.tail[w] = make_int4(0, 0, 0, 0);
    __syncthreads();
  }
  if (pos >= end) return;
  int b = __builtin_amdgcn_readfirstlane(S.start_b);
  long long off = uniform(S.start_off);
  const long long begin = pos;

  while (pos < end && (uint32_t)b < (uint32_t)a.c.seqs) {
    SeqWork sw = work_of(b);
    sw.len = __builtin_amdgcn_readfirstlane(sw.len);
    sw.n = __builtin_amdgcn_readfirstlane(sw.n);
    sw.keys = __builtin_amdgcn_readfirstlane(sw.keys);
    sw.tiles = __builtin_amdgcn_readfirstlane(sw.tiles);
    sw.live = __builtin_amdgcn_readfirstlane(sw.live);
    if (const long long u = seq_pieces(a, sw, fixed); off >= u) {
      off -= u;
      ++b;
      continue;
    }
    const long long live_units = (long long)a.c.kv_heads * sw.live * (sw.tiles + fixed);
    if (off >= live_units) {  // a row tile without a node: zeros
      const long long u = off - live_units;
      const int dead = a.mts - sw.live;
      const int h = (int)(u / dead), mt = sw.live + (int)(u - (long long)h * dead);
      const int hq = a.c.kv_heads * a.G;
      for (int i = tid; i < MT * C::kVecs; i += NT) {
        const int r = mt * MT + i / C::kVecs, x = i % C::kVecs;
        const int node = r / a.G, g = r - node * a.G;
        if (node < a.N) {
          const size_t row = ((size_t)b * a.N + node) * hq + h * a.G + g;
          *reinterpret_cast<u32x4*>(a.out + row * C::kRow + x * 16) = u32x4{0, 0, 0, 0};
          if (a.lse && x == 0) a.lse[row] = -INFINITY;
        }
      }
      ++pos;
      ++off;
      continue;
    }

    // ------------------------------------------------------------------ one part of a group
    const int group_pieces = sw.tiles + fixed;
    const long long grp = div_pieces(off, group_pieces);
    const int r0 = (int)(off - grp * group_pieces);  // first piece in the group
    const long long left = end - pos;
    const int r1 = (long long)(group_pieces - r0) < left ? group_pieces : r0 + (int)left;
    const int t0 = r0 > fixed ? r0 - fixed : 0, part_end = r1 - fixed;
    if (t0 >= part_end) {  // fixed pieces alone
      pos += r1 - r0;
      off += r1 - r0;
      continue;
    }
    const int h = (int)((uint32_t)grp / (uint32_t)sw.live), mt = (int)grp - h * sw.live;
    const int rows = sw.n * a.G;             // live rows of the (sequence, kv head)
    const int held = positions_held(a.c, b);
    const int32_t* table = a.c.table + (size_t)b * a.c.width;
    const char* kbase = a.c.k + (long long)h * a.c.head_stride;
    const char* vbase = a.c.v + (long long)h * a.c.head_stride;
    // live nodes of the row tile, and the node of this lane's row (a dead row: the last one; what
    // it computes is dropped)
    const int first_node = mt * MT / a.G;
    const int last_node = (rows < (mt + 1) * MT ? sw.n : ((mt + 1) * MT - 1) / a.G + 1) - 1;
    // keys that every row of the tile sees, and the tiles behind those that some row sees (a chain:
    // up to its own node; at least one tile, so that the part has a result).  4 pieces of prompts of
    // 1000 nodes behind up to 1000 tokens take 128 us, 195 without leaving tiles out.  The cut
    // counts all tiles alike, so a worker whose pieces all lie behind has an empty part to show
    const int open = a.mask ? sw.len : sw.len + first_node + 1;
    const int in_sight = a.mask ? part_end : (sw.len + last_node + BN) / BN;
    const int t1 = part_end < in_sight ? part_end : in_sight > t0 ? in_sight : t0 + 1;
    const int my_row = mt * MT + wm * 32 + col;
    const int my_node = my_row < rows ? my_row / a.G : last_node;
    const char* qp = a.q + (long long)b * a.q_seq + (long long)my_node * a.q_node +
                     (long long)(h * a.G + my_row - my_node * a.G) * a.q_head + half * 16;
    u32x4 qf[QF];
#pragma unroll
    for (int s = 0; s < QF; ++s)
      qf[s] = my_row < rows ? *reinterpret_cast<const u32x4*>(qp + s * 32) : u32x4{0, 0, 0, 0};

    // row that this thread's vector of pass i belongs to (a pass covers whole rows, or not)
    auto row_of = [&](int i) SV_INLINE {
      return NT % C::kVecs == 0 ? tid / C::kVecs + i * (NT / C::kVecs)
                                : (tid + i * NT) / C::kVecs;
    };
    auto load_entry = [&](int t) SV_INLINE -> int {  // page of key t * BN + tid, -1: none
      const int key = t * BN + fresh(tid);
      if (tid >= BN || key >= sw.keys) return -1;
      return table[fast_div(a.c.page_div, (uint32_t)key)];
    };
    // by threads first .. first + BN - 1
    auto put_rows = [&](int t, int page, int first = 0) SV_INLINE {
      if (tid >= first && tid < first + BN) {
        const int at = fresh(tid) - first, key = t * BN + at;
        const uint32_t pi = fast_div(a.c.page_div, (uint32_t)key);
        bool ok = page >= 0 && page < a.c.pages;
        if ((t + 1) * BN > held) ok = names_page(a.c, held, key, page);
        const int slot = key - (int)(pi * a.c.page_div.d);
        S.rowoff[t & (C::kRing - 1)][at] =
            ok ? (long long)page * a.c.page_stride + (long long)slot * a.c.token_stride : 0ll;
        const unsigned long long bits = __ballot(ok);
        if (lane == 0) {
          S.valid[t & (C::kRing - 1)][(at >> 5)] = (uint32_t)bits;
          S.valid[t & (C::kRing - 1)][(at >> 5) + 1] = (uint32_t)(bits >> 32);
          S.badv[t & (C::kRing - 1)][(at >> 5)] = 0u;
          S.badv[t & (C::kRing - 1)][(at >> 5) + 1] = 0u;
        }
      }
    };
    // Loads of tile t into LDS, 1 KB per wave, instruction and tensor: the row offsets of its
    // kLoads passes, then pass i.
    long long at_row[C::kLoads];
    auto find_rows = [&](int t) SV_INLINE {
#pragma unroll
      for (int i = 0; i < C::kLoads; ++i) at_row[i] = S.rowoff[t & (C::kRing - 1)][row_of(i)];
    };
    auto issue = [&](int t, int i, auto... lanes) SV_INLINE {
      const uint32_t to =
          pool_at + (t & (NST - 1)) * C::kTileBytes + wave * 1024 + i * (NT * 16);
      const int r = row_of(i);
      const int p = NT % C::kVecs == 0 ? tid % C::kVecs : tid + i * NT - r * C::kVecs;
      load_to_lds(kbase + at_row[i] + (p ^ C::swz_k(r)) * 16, to, lanes...);
      load_to_lds(vbase + at_row[i] + (p ^ C::swz_v(r)) * 16, to + BN * C::kRow, lanes...);
    };
    // A tile that ends behind the committed tokens or holds keys that do not exist: their values
    // are cleared, and non-finite values of drafted nodes, which may be hidden from some rows
    // (0 * inf must not reach them), are set aside.
    auto mend = [&](int t) SV_INLINE {
      char* vt = S.pool + (t & (NST - 1)) * C::kTileBytes + BN * C::kRow;
      const int x0 = fresh(tid);
#pragma unroll 1
      for (int i = 0; i < C::kLoads; ++i) {
        const int x = x0 + i * NT, r = x / C::kVecs;
        u32x4* p = reinterpret_cast<u32x4*>(vt + x * 16);
        if (!(S.valid[t & (C::kRing - 1)][r >> 5] >> (r & 31) & 1u)) {
          *p = u32x4{0, 0, 0, 0};
        } else if (t * BN + r >= sw.len) {
          u32x4 y = *p;
          if (clear_non_finite<BF16>(y)) {
            *p = y;
            atomicOr(&S.badv[t & (C::kRing - 1)][r >> 5], 1u << (r & 31));
          }
        }
      }
      // which keys a node sees: a wave takes a node and 64 keys at a time, eight loads in flight
      // (of a key that is no node or a node past the tile's last, those of its nearest one)
#pragma unroll 1
      for (int k0 = 0; k0 < BN; k0 += 64) {
        const int node = t * BN + k0 + fresh(lane) - sw.len;
        const int near = node < 0 ? 0 : node < a.N ? node : a.N - 1;
        const uint32_t* there32 = &S.valid[t & (C::kRing - 1)][k0 / 32];
        const unsigned long long there = there32[0] | (unsigned long long)there32[1] << 32;
#pragma unroll 1
        for (int r0 = wave; first_node + r0 <= last_node; r0 += 8 * C::kNW) {
          uint8_t shown[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int me = first_node + r0 + i * C::kNW;
            shown[i] = me >= near;
            if (a.mask) {
              const int row = me < last_node ? me : last_node;
              shown[i] = a.mask[((size_t)b * a.N + row) * a.N + near];
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const unsigned long long bits = __ballot(shown[i] != 0 || node < 0) & there;
            const int row = r0 + i * C::kNW;
            if (lane < 2 && first_node + row <= last_node)
              S.sees[row][k0 / 32 + lane] = (uint32_t)(bits >> (32 * lane));
          }
        }
      }
    };

    const int kr = wk * KS * 32 + col;  // this lane's key row in its first block of 32
    const int sw_k = C::swz_k(kr);      // the same for every block of 32 keys
    float m = -INFINITY, l = 0.0f;
    f32x16 acc[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;

    // The shift m of a row's weights 2^(z - m), in units of log2 (so that weights and rescalings
    // use the same rounded number): a key's maximum that was the row's running one, or lies less
    // than kSlack below it.  Weights of up to 2^kSlack cost nothing (fp32 sums, and bf16 rounds
    // relative to size), and O and l are rescaled a few times a row instead of every time some
    // row of the wave meets a new maximum.  Returns what is subtracted (0 while nothing is seen).
    constexpr float kSlack = 8.0f;
    auto raise = [&](float top) SV_INLINE -> float {
      const float m_new = fmaxf(m, half_max(top) * sl2);
      if (__any(m_new > m + kSlack)) {
        const float f = __builtin_amdgcn_exp2f(m - (m_new == -INFINITY ? 0.0f : m_new));
        l *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[d][r] *= f;
        m = m_new;
      }
      return m == -INFINITY ? 0.0f : m;
    };

    // One tile: scores of this wave's keys, softmax, product with the values.  `Rough` tiles hold
    // keys that do not exist or drafted nodes; the others need no masks.
    auto step = [&](int t, auto rough) SV_INLINE {
      constexpr bool Rough = decltype(rough)::value;
      const char* tile = S.pool + (t & (NST - 1)) * C::kTileBytes;
      // scores: lane = row, register r = key 8 (r / 4) + 4 half + r % 4.  LDS reads run kAhead
      // fragments ahead of the matrix instructions (the order is pinned: left alone, the
      // compiler waits for each read)
      constexpr int kAhead = 4, kKeyFrags = KS * QF;
      constexpr int kPace = kKeyFrags / C::kLoads > 0 ? kKeyFrags / C::kLoads : 1;
      static_assert(NST != 2 || kKeyFrags >= C::kLoads, "a pass per fragment at most");
      f32x16 s[KS];
      const char* kp = tile + kr * C::kRow;
      auto key_frag = [&](int n) SV_INLINE {
        return *reinterpret_cast<const u32x4*>(kp + n / QF * (32 * C::kRow) +
                                               (((2 * (n % QF) + half) ^ sw_k) * 16));
      };
      u32x4 kf[kAhead];
#pragma unroll
      for (int n = 0; n < kAhead; ++n) kf[n] = key_frag(n);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int n = 0; n < kKeyFrags; ++n) {
        const int ks = n / QF, q = n % QF;
        if (q == 0)
#pragma unroll
          for (int r = 0; r < 16; ++r) s[ks][r] = 0.0f;
        if constexpr (BF16) {
          s[ks] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(bf16x8, kf[n % kAhead]), __builtin_bit_cast(bf16x8, qf[q]), s[ks],
              0, 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[ks] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(kf[n % kAhead][e]),
                                                         __uint_as_float(qf[q][e]), s[ks], 0, 0, 0);
        }
        if (n + kAhead < kKeyFrags) kf[n % kAhead] = key_frag(n + kAhead);
        // the next tile's loads start in the shadow of these products
        if (NST == 2 && n % kPace == 0 && n / kPace < C::kLoads && t + 1 < t1)
          issue(t + 1, n / kPace);
        __builtin_amdgcn_sched_barrier(0);
      }

      // hide keys that the row does not see
      uint32_t seen[KS];
      if constexpr (Rough) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint32_t bits =
              of_half(S.sees[my_node - first_node][wk * KS + ks] >> (4 * half));
#pragma unroll
          for (int r = 0; r < 16; ++r) s[ks][r] = bits & (1u << r) ? s[ks][r] : -INFINITY;
          seen[ks] = bits;
        }
      }

      float mx = s[0][0];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[ks][r]);
      const float shift = raise(mx);
      // P of registers [8 j + r0, 8 j + r0 + n) of the wave's 16 KS keys a lane
      auto weigh = [&](int j, int r0, int n) SV_INLINE {
#pragma unroll
        for (int r = r0; r < r0 + n; ++r) {
          const int i = 8 * (j & 1) + r;
          s[j >> 1][i] = __builtin_amdgcn_exp2f(s[j >> 1][i] * sl2 - shift);
          l += s[j >> 1][i];
        }
      };

      // O^T += V^T P^T
      const char* vp = tile + BN * C::kRow + wk * KS * 32 * C::kRow;
      if constexpr (BF16) {
        // 16 lanes read 4 keys x 16 columns; lane i supplies row i / 4, 8 bytes i % 4.  The
        // swizzle moves 64-byte pieces and depends on the row's two lowest bits alone
        const int vr = 4 * half + ((lane & 15) >> 2);
        const char* vt = vp + vr * C::kRow + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
        const int sw_v = C::swz_v(vr) * 16;
        typedef short short8v __attribute__((ext_vector_type(8)));
        auto value_frag = [&](int n) SV_INLINE {  // 16 keys n / ND, columns 32 (n % ND) and up
          const char* at = vt + n / ND * (16 * C::kRow) + ((n % ND * 64) ^ sw_v);
          const short4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SV_LDS(short4v)*)at);
          const short4v hi =
              __builtin_amdgcn_ds_read_tr16_b64_v4i16((SV_LDS(short4v)*)(at + 8 * C::kRow));
          return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        };
        constexpr int kChunks = 2 * KS, kFrags = kChunks * ND;
        short8v vf[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) vf[n] = value_frag(n);
        weigh(0, 0, 8);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
          // P rounded to bf16 for the matrix instruction: up to half a step, 2^-8, of a weight, as
          // the inputs carry; the sum l keeps the unrounded weights.  Independent roundings of
          // weights and of the result, each 1.7e-3 of its value in the mean square, make 2.3e-3 of
          // the output's size (measured: 2.3e-3 to 2.4e-3).  Products of both halves of a split
          // weight would take twice the matrix instructions here
          bf16x8 pf;
#pragma unroll
          for (int i = 0; i < 8; ++i) pf[i] = (__bf16)s[j >> 1][8 * (j & 1) + i];
          // the next keys' weights are computed in the shadow of these products
          constexpr int kShare = (8 + ND - 1) / ND;
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            const int n = j * ND + d;
            acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                __builtin_bit_cast(bf16x8, vf[n % kAhead]), pf, acc[d], 0, 0, 0);
            if (n + kAhead < kFrags) vf[n % kAhead] = value_frag(n + kAhead);
            if (j + 1 < kChunks && d * kShare < 8)
              weigh(j + 1, d * kShare, 8 - d * kShare < kShare ? 8 - d * kShare : kShare);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2 * KS; ++j) weigh(j, 0, 8);
        auto value_frag = [&](int n) SV_INLINE {  // key register n / ND, columns 32 (n % ND) and up
          const int r = n / ND;
          return *reinterpret_cast<const float*>(
              vp + (8 * (r >> 2) + 4 * half + (r & 3)) * C::kRow + col * 4 + n % ND * 128);
        };
        constexpr int kFrags = 16 * KS * ND;
        float vf[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) vf[n] = value_frag(n);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kFrags; ++n) {
          const int r = n / ND, d = n % ND;
          acc[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(vf[n % kAhead], s[r >> 4][r & 15], acc[d],
                                                        0, 0, 0);
          if (n + kAhead < kFrags) vf[n % kAhead] = value_frag(n + kAhead);
          __builtin_amdgcn_sched_barrier(0);
        }
      }

#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int blk = wk * KS + ks;
        // non-finite values of drafted nodes, for the rows that see them (rare: a rolled loop
        // over a copy of O in scratch memory keeps it out of the registers of the common path)
        const uint32_t bad = Rough ? S.badv[t & (C::kRing - 1)][blk] : 0u;
        if (Rough && __builtin_expect(bad != 0, 0)) {
          float o[ND * 16];
#pragma unroll
          for (int i = 0; i < ND * 16; ++i) o[i] = acc[i >> 4][i & 15];
          asm volatile("" : : "v"(o) : "memory");  // stays in scratch memory
          for (uint32_t left = bad; left; left &= left - 1) {
            const int kk = __builtin_amdgcn_readfirstlane(__ffs(left) - 1);
            const int hk = (kk >> 2) & 1, rk = ((kk >> 3) << 2) | (kk & 3);
            float p = 0.0f;
#pragma unroll
            for (int r = 0; r < 16; ++r) p = r == rk ? s[ks][r] : p;
            p = __shfl(p, col + 32 * hk);
            const int sees = __shfl((int)(seen[ks] >> rk & 1u), col + 32 * hk);
            const char* row = vbase + S.rowoff[t & (C::kRing - 1)][blk * 32 + kk];
#pragma unroll 1
            for (int i = 0; i < ND * 16; ++i) {
              const int e = (i >> 4) * 32 + 8 * ((i >> 2) & 3) + 4 * half + (i & 3);
              float x;
              if constexpr (BF16)
                x = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[e] << 16);
              else
                x = reinterpret_cast<const float*>(row)[e];
              if (sees && non_finite(__float_as_uint(x))) o[i] += p * x;
            }
          }
#pragma unroll
          for (int i = 0; i < ND * 16; ++i) acc[i >> 4][i & 15] = o[i];
          __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0) here: not in the common path's tiles
        }
      }
    };

    auto issue_all = [&](int t) SV_INLINE {
      find_rows(t);
#pragma unroll
      for (int i = 0; i < C::kLoads; ++i) issue(t, i);
    };
    auto is_rough = [&](int t) SV_INLINE -> bool {
      bool rough = (t + 1) * BN > open;
#pragma unroll
      for (int i = 0; i < BN / 32; ++i) rough |= S.valid[t & (C::kRing - 1)][i] != 0xFFFFFFFFu;
      return __builtin_amdgcn_readfirstlane(rough);
    };
    // plain tiles up to the first rough one (usually where the drafted nodes begin; in a chain,
    // where a node that some row does not see begins), then the rest as rough ones
    if constexpr (NST == 4) {
      // Four tiles in LDS, one workgroup a compute unit.  The products of one block of 32 keys
      // run beside the exponentials of the one before, in one instruction stream:
      //   scores of the next block  |  the first weights of this one
      //   O += first 16 keys        |  the other weights
      //   O += other 16 keys        |  maxima of the next block
      // Tile t + 2 is loaded while t is computed.
      static_assert(NST != 4 || (BF16 && WK == 1 && KS == 2 && BN == 64 && C::kNW == 8), "shape");
      const uint32_t entry_at =
          (uint32_t)reinterpret_cast<uintptr_t>((SV_LDS(char)*)S.entry);
      {  // rows of the first eight tiles, a wave each
        const int t = t0 + wave, key = t * BN + lane;
        const int page =
            t < t1 && key < sw.keys ? table[fast_div(a.c.page_div, (uint32_t)key)] : -1;
        if (t < t1) put_rows(t, page, 64 * wave);
      }
      __syncthreads();
      issue_all(t0);
      if (t0 + 1 < t1) issue_all(t0 + 1);
      // At every fourth tile (its barrier passed), four waves: rows of tile t + 4 + wave from its
      // table entries, entries of tile t + 8 + wave on their way.
      auto keep_books = [&](int t) SV_INLINE {
        if (((t - t0) & 3) != 0 || wave >= 4) return;
        const int e = t + 4 + wave;
        if (t > t0 && e < t1) {
          const int key = e * BN + fresh(lane);
          put_rows(e, key < sw.keys ? S.entry[wave][lane] : -1, 64 * wave);
        }
        if (e + 4 < t1) {
          const int key = (e + 4) * BN + fresh(lane);
          if (key < sw.keys)
            load_word_to_lds(table + fast_div(a.c.page_div, (uint32_t)key),
                             entry_at + wave * (BN * 4));
        }
      };
      // Waits for tile t: only tile t + 1's loads may still be on their way.
      auto arrive = [&](int t) SV_INLINE {
        if (t + 1 < t1)
          asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(2 * C::kLoads)
                       : "memory");
        else
          tile_barrier();
      };

      constexpr int kAhead = 4, kEarly = 6, kFirst = 11;
      f32x16 sa, sb;
      float mx, shift;
      u32x4 kf[kAhead];
      typedef short short8v __attribute__((ext_vector_type(8)));
      short8v vf[kAhead];
      auto key_frag = [&](const char* tile, int sub, int q) SV_INLINE {
        return *reinterpret_cast<const u32x4*>(tile + (sub * 32 + kr) * C::kRow +
                                               (((2 * q + half) ^ sw_k) * 16));
      };
      const int vr = 4 * half + ((lane & 15) >> 2);
      const int sw_v = C::swz_v(vr) * 16;
      auto value_frag = [&](const char* tile, int sub, int n) SV_INLINE {
        const char* at = tile + (BN + sub * 32 + n / ND * 16 + vr) * C::kRow +
                         ((lane >> 4) & 1) * 32 + (lane & 3) * 8 + ((n % ND * 64) ^ sw_v);
        const short4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SV_LDS(short4v)*)at);
        const short4v hi =
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((SV_LDS(short4v)*)(at + 8 * C::kRow));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      };
      // weights of registers u0 .. u1 - 1 of a block
      auto weigh = [&](f32x16& s, int u0, int u1) SV_INLINE {
#pragma unroll
        for (int u = u0; u < u1; ++u) {
          s[u] = __builtin_amdgcn_exp2f(s[u] * sl2 - shift);
          l += s[u];
        }
      };
      auto score = [&](f32x16& s, int q) SV_INLINE {
        if (q == 0)
#pragma unroll
          for (int r = 0; r < 16; ++r) s[r] = 0.0f;
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, kf[q % kAhead]), __builtin_bit_cast(bf16x8, qf[q]),
            s, 0, 0, 0);
      };
      // Scores of block (next tile, next_sub) into nx beside the first weights of cu, whose first
      // values (of cur tile, sub) are fetched at the end; `loads`: tile t + 2's loads start too.
      auto scores_beside = [&](const char* next, int next_sub, f32x16& nx, const char* cur,
                               int sub, f32x16& cu, int load_tile, auto loads) SV_INLINE {
#pragma unroll
        for (int q = 0; q < kAhead; ++q) kf[q] = key_frag(next, next_sub, q);
        weigh(cu, 0, kEarly);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < QF; ++q) {
          score(nx, q);
          weigh(cu, kEarly + (kFirst - kEarly) * q / QF, kEarly + (kFirst - kEarly) * (q + 1) / QF);
          if (q + kAhead < QF) kf[q % kAhead] = key_frag(next, next_sub, q + kAhead);
          else vf[q + kAhead - QF] = value_frag(cur, sub, q + kAhead - QF);
          __builtin_amdgcn_sched_barrier(0);
          if (decltype(loads)::value && q * C::kLoads % QF < C::kLoads)
            issue(load_tile, q * C::kLoads / QF, load_tile < t1 ? ~0ull : 0ull);
        }
      };
      // O += block (cur tile, sub) with weights cu beside the maxima of nx
      auto values_beside = [&](const char* cur, int sub, f32x16& cu, f32x16& nx) SV_INLINE {
        constexpr int kFrags = 2 * ND;
        bf16x8 pf;
#pragma unroll
        for (int n = 0; n < kFrags; ++n) {
          const int c = n / ND, d = n % ND;
          if (d == 0)  // P rounded to bf16: half a step of 2^-8 per weight
#pragma unroll
            for (int i = 0; i < 8; ++i) pf[i] = (__bf16)cu[8 * c + i];
          acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(bf16x8, vf[n % kAhead]), pf, acc[d], 0, 0, 0);
          if (c == 0) {
            weigh(cu, kFirst + (16 - kFirst) * d / ND, kFirst + (16 - kFirst) * (d + 1) / ND);
          } else {
#pragma unroll
            for (int r = 16 * d / ND; r < 16 * (d + 1) / ND; ++r)
              mx = r == 0 ? nx[0] : fmaxf(mx, nx[r]);
          }
          if (n + kAhead < kFrags) vf[n % kAhead] = value_frag(cur, sub, n + kAhead);
          __builtin_amdgcn_sched_barrier(0);
        }
        asm volatile("" : "+v"(mx));  // not moved from here
      };

      int t = t0;
      arrive(t);
      bool plain = !is_rough(t);
      if (plain) {  // the first block's scores and maxima stand alone
        const char* tile = S.pool + (t & 3) * C::kTileBytes;
#pragma unroll
        for (int q = 0; q < kAhead; ++q) kf[q] = key_frag(tile, 0, q);
#pragma unroll
        for (int q = 0; q < QF; ++q) {
          score(sa, q);
          if (q + kAhead < QF) kf[q % kAhead] = key_frag(tile, 0, q + kAhead);
        }
        mx = sa[0];
#pragma unroll
        for (int r = 1; r < 16; ++r) mx = fmaxf(mx, sa[r]);
      }
      while (plain) {
        const char* tile = S.pool + (t & 3) * C::kTileBytes;
        if (t + 2 < t1) find_rows(t + 2);
        keep_books(t);
        shift = raise(mx);
        scores_beside(tile, 1, sb, tile, 0, sa, t + 2, std::true_type{});
        values_beside(tile, 0, sa, sb);
        shift = raise(mx);
        if (++t < t1) arrive(t);
        // the next tile's scores also where it is rough or there is none (LDS holds some tile):
        // they are dropped then, and the stream of instructions stays one
        scores_beside(S.pool + (t & 3) * C::kTileBytes, 0, sa, tile, 1, sb, 0, std::false_type{});
        values_beside(tile, 1, sb, sa);
        plain = t < t1 && !is_rough(t);
      }
      while (t < t1) {
        if (t + 2 < t1) issue_all(t + 2);
        keep_books(t);
        mend(t);
        lds_barrier();
        step(t, std::true_type{});
        if (++t < t1) arrive(t);
      }
    } else {
      const int entry0 = load_entry(t0), entry1 = t0 + 1 < t1 ? load_entry(t0 + 1) : -1;
      int entry = t0 + 2 < t1 ? load_entry(t0 + 2) : -1;
      put_rows(t0, entry0);
      if (t0 + 1 < t1) put_rows(t0 + 1, entry1);
      __syncthreads();
      issue_all(t0);
      auto turn = [&](int t) SV_INLINE {
        tile_barrier();  // tile t is there; the waves are done with the one before
        if (NST > 1 && t + 1 < t1) find_rows(t + 1);
        if (t + 2 < t1) {
          put_rows(t + 2, entry);
          entry = t + 3 < t1 ? load_entry(t + 3) : -1;
        }
      };
      auto leave = [&](int t) SV_INLINE {
        if (NST == 1 && t + 1 < t1) {
          lds_barrier();
          issue_all(t + 1);
        }
      };
      int t = t0;
      turn(t);
      while (!is_rough(t)) {
        step(t, std::false_type{});
        leave(t);
        if (++t == t1) break;
        turn(t);
      }
      while (t < t1) {
        mend(t);
        lds_barrier();
        step(t, std::true_type{});
        leave(t);
        if (++t < t1) turn(t);
      }
    }

    // ------------------------------------------------------------------ the part's result
    l = half_sum(l);
    if constexpr (WK > 1) {  // join the waves that share rows
      if (half == 0) S.m[wave][col] = m;
      if (half == 0) S.l[wave][col] = l;
      __syncthreads();
      float mt_all = -INFINITY;
#pragma unroll
      for (int i = 0; i < WK; ++i) mt_all = fmaxf(mt_all, S.m[i * WM + wm][col]);
      const float mu = mt_all == -INFINITY ? 0.0f : mt_all;
      float lt = 0.0f;
#pragma unroll
      for (int i = 0; i < WK; ++i)
        lt += S.l[i * WM + wm][col] * __builtin_amdgcn_exp2f(S.m[i * WM + wm][col] - mu);
      const float f = __builtin_amdgcn_exp2f(m - mu);
      f32x4* box = reinterpret_cast<f32x4*>(S.pool);
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          box[((wave * ND + d) * 4 + r) * 64 + lane] =
              f32x4{acc[d][4 * r] * f, acc[d][4 * r + 1] * f, acc[d][4 * r + 2] * f,
                    acc[d][4 * r + 3] * f};
      __syncthreads();
      m = mt_all;
      l = lt;
    }

    const long long first = pos - r0;  // the group's first piece
    const bool whole = t0 == 0 && part_end == sw.tiles;
    const int slot = 2 * w + (pos == begin ? 0 : 1);
    const int hq = a.c.kv_heads * a.G;
    const int fcol = fresh(col), fhalf = fresh(half);
    const int row = mt * MT + wm * 32 + fcol;
    const int node = row / a.G, g = row - node * a.G;
    const bool row_live = row < rows;
    const bool row_out = node < a.N;  // padding nodes get zeros
    const size_t orow = ((size_t)b * a.N + node) * hq + h * a.G + g;
    const size_t prow = (size_t)slot * MT + wm * 32 + fcol;
    const float inv = !row_live || l == 0.0f ? 0.0f : 1.0f / l;
    char* op = a.out + orow * C::kRow + 4 * fhalf * C::kES;
    float* pp = a.part + prow * D + 4 * fhalf;
    // columns d * 32 + 8 r4 + 4 half and up of the row; a dead row's O may hold anything
    auto emit_out = [&](int d, int r4, f32x4 x) SV_INLINE {
      if (!row_live) x = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (BF16) {
        bf16x4 y;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = (__bf16)(x[j] * inv);
        *reinterpret_cast<bf16x4*>(op + (d * 32 + 8 * r4) * 2) = y;
      } else {
        *reinterpret_cast<f32x4*>(op + (d * 32 + 8 * r4) * 4) = x * inv;
      }
    };
    auto emit_part = [&](int d, int r4, f32x4 x) SV_INLINE {
      *reinterpret_cast<f32x4*>(pp + d * 32 + 8 * r4) = x;
    };
    auto each = [&](auto emit) SV_INLINE {
      if constexpr (WK > 1) {
        const f32x4* box = reinterpret_cast<const f32x4*>(S.pool);
        for (int d = wk; d < ND; d += WK)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            f32x4 x = box[((wm * ND + d) * 4 + r) * 64 + lane];
#pragma unroll
            for (int i = 1; i < WK; ++i)
              x += box[(((i * WM + wm) * ND + d) * 4 + r) * 64 + lane];
            emit(d, r, x);
          }
      } else {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            emit(d, r, f32x4{acc[d][4 * r], acc[d][4 * r + 1], acc[d][4 * r + 2],
                             acc[d][4 * r + 3]});
      }
    };
    if (whole) {
      if (row_out) each(emit_out);
      if (wk == 0 && fhalf == 0 && a.lse && row_out)
        a.lse[orow] = !row_live || l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
    } else {
      if (row_live) each(emit_part);
      if (wk == 0 && fhalf == 0) a.part_ml[prow] = make_float2(m, l);
    }
    if (tid == 0 && t0 == 0 && !whole)
      a.tail[w] = make_int4(b, h * a.mts + mt, slot,
                            (int)(div_pieces(first + group_pieces - 1, per) - w + 1));
    __syncthreads();
    pos += r1 - r0;
    off += r1 - r0;
  }
}

// Joins the parts of each group that begins as some worker's last part and ends with a later
// worker: every later part is that worker's first.  A workgroup looks after kTails neighbouring
// workers, one after the other, and 256 / W pieces of four columns of a row; W threads share a
// piece's parts, in order, and the first adds up their sums.  Rows that the batch cannot have are
// not launched.  Bound by the parts it reads (64 MB in 14 us, 4.6 TB/s, for 32 ragged trees
// of 256 rows) or, with few rows, by the latency of two dependent loads.  One, two, four and eight
// workers a workgroup: 18.3, 18.1, 18.5 and 20.2 us for attention and join of 4 sequences of up to
// 2000 tokens, 226, 227, 228 and 232 us for 64 of up to 8191; with 256 rows a group they are alike.
constexpr int kTails = 2;

template <bool BF16, int D, int MT, int W>
__device__ __forceinline__ void join_parts(const AttnArgs& a, const int4 g) {
  constexpr int kPieces = 256 / W;
  __shared__ f32x4 box[W > 1 ? 256 : 1];
  __shared__ float2 box_ml[W > 1 ? 256 : 1];
  const int b = g.x, h = g.y / a.mts, mt = g.y - h * a.mts;
  const int share = W > 1 ? threadIdx.x / kPieces : 0;
  const int i = blockIdx.x * kPieces + threadIdx.x % kPieces;
  const int row = i / (D / 4), e = (i - row * (D / 4)) * 4;
  const int r = mt * MT + row;
  const int node = r / a.G, hg = r - node * a.G;
  const bool out = row < MT && node < a.N;
  int n = a.nodes ? a.nodes[b] : a.N;
  n = n > a.N ? a.N : n;
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
  float m = -INFINITY, l = 0.0f;
  // adds kCount parts to (m, l, x), their loads in flight together
  auto add = [&](auto count, auto load) SV_INLINE {
    constexpr int kCount = decltype(count)::value;
    float2 ml[kCount];
    f32x4 y[kCount];
    float top = m;
#pragma unroll
    for (int k = 0; k < kCount; ++k) load(k, ml[k], y[k]);
#pragma unroll
    for (int k = 0; k < kCount; ++k) top = fmaxf(top, ml[k].x);
    const float mu = top == -INFINITY ? 0.0f : top;
    const float f = __builtin_amdgcn_exp2f(m - mu);
    x *= f;
    l *= f;
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      const float p = __builtin_amdgcn_exp2f(ml[k].x - mu);
      l += ml[k].y * p;
      x += y[k] * p;
    }
    m = top;
  };
  if (out && node < n) {
    // parts: slot g.z, then slot 0 of each later worker
    auto take = [&](int s0, auto count) SV_INLINE {
      add(count, [&](int k, float2& ml, f32x4& y) SV_INLINE {
        const int s = s0 + k;
        const size_t slot = s == 0 ? (size_t)g.z : (size_t)2 * (g.z / 2 + s);
        ml = a.part_ml[slot * MT + row];
        y = *reinterpret_cast<const f32x4*>(a.part + (slot * MT + row) * D + e);
      });
    };
    const int each = (g.w + W - 1) / W;
    int s = share * each;
    const int end = s + each < g.w ? s + each : g.w;
    for (; s + 8 <= end; s += 8) take(s, std::integral_constant<int, 8>{});
    for (; s + 2 <= end; s += 2) take(s, std::integral_constant<int, 2>{});
    if (s < end) take(s, std::integral_constant<int, 1>{});
  }
  if constexpr (W > 1) {
    __syncthreads();  // the group before has been read
    box[threadIdx.x] = x;
    box_ml[threadIdx.x] = make_float2(m, l);
    __syncthreads();
    if (share > 0) return;
    add(std::integral_constant<int, W - 1>{}, [&](int k, float2& ml, f32x4& y) SV_INLINE {
      ml = box_ml[threadIdx.x + (k + 1) * kPieces];
      y = box[threadIdx.x + (k + 1) * kPieces];
    });
  }
  if (!out) return;
  const int hq = a.c.kv_heads * a.G;
  const size_t orow = ((size_t)b * a.N + node) * hq + h * a.G + hg;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if constexpr (BF16) {
    bf16x4 y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = (__bf16)(x[j] * inv);
    *reinterpret_cast<bf16x4*>(a.out + (orow * D + e) * 2) = y;
  } else {
    *reinterpret_cast<f32x4*>(a.out + (orow * D + e) * 4) = x * inv;
  }
  if (a.lse && e == 0) a.lse[orow] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
}

template <bool BF16, int D, int MT, int W>
__global__ __launch_bounds__(256) void k_tree_join(AttnArgs a) {
  static_assert(kTails == 2, "two tails in registers");
  int4 g[kTails];
#pragma unroll
  for (int i = 0; i < kTails; ++i) {
    const int w = blockIdx.y * kTails + i;
    g[i] = a.tail[w < a.workers ? w : a.workers - 1];
    if (w >= a.workers) g[i].w = 0;
  }
#pragma unroll 1
  for (int i = 0; i < kTails; ++i) {
    if (g[0].w > 1) join_parts<BF16, D, MT, W>(a, g[0]);
    g[0] = g[1];
  }
}

// Tile shapes: rows of the (sequence, kv head) decide between 32, 64, 128 and 256 (row_tile_for),
// bytes of a row what fits into LDS.  Rows of up to 256 bytes: two tiles of 64 keys, the next one
// loaded while one is computed, beside a second workgroup's two; longer ones: one tile, and the
// other workgroups compute while it is loaded.  bf16 rows of 512 bytes: O and Q of 32 rows take 192
// registers a lane, so four waves and one workgroup a compute unit, with two tiles, for more than
// 64 rows (32 sequences of 512 to 4096 tokens, 8 kv heads, 256 rows: 298 us, 483 with the 64-row
// workgroups); up to 64 two workgroups of two waves with a tile each (64 sequences of 300 tokens,
// 48 rows: 46 us, 50 with the 128-row workgroups; 32 of 512 to 4096, 64 rows: 151 and 150).
struct Shape {
  int wm, wk, ks, nst, occ;
  int per_cu = 0;  // workgroups that a compute unit holds
};

template <bool BF16, int D>
constexpr Shape shape_for(int row_tile) {
  constexpr int row = D * (BF16 ? 2 : 4);
  if (row > 512) return Shape{2, 2, 1, 1, 1};
  if (row > 256) {
    if (row_tile == 32) return Shape{1, 2, 1, 1, 1};
    if (row_tile == 64) return BF16 ? Shape{2, 1, 2, 1, 1} : Shape{2, 2, 1, 1, 2};
    return BF16 ? Shape{4, 1, 2, 2, 1} : Shape{4, 1, 2, 1, 2};
  }
  if (row_tile == 32) return Shape{1, 2, 1, 2, BF16 ? 2 : 1};
  if (row_tile == 64) return Shape{2, 2, 1, 2, 2};
  if (row_tile == 128) return Shape{4, 1, 2, 2, 2};
  return Shape{8, 1, 2, 4, 2};
}

template <bool BF16, int D, int RT>
hipError_t launch_shape(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  constexpr Shape sh = shape_for<BF16, D>(RT);
  using C = Attn<BF16, D, sh.wm, sh.wk, sh.ks, sh.nst>;
  if (p.row_tile != C::kMT || p.key_tile != C::kBN) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_tree_attn<BF16, D, sh.wm, sh.wk, sh.ks, sh.nst, sh.occ>),
                     dim3(p.workers), dim3(C::kNT), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.workers == 1) return hipSuccess;
  const int rows = p.mts == 1 ? a.N * a.G : C::kMT;  // of a tile, at most
  const unsigned pieces = rows * (D / 4), tails = (p.workers + kTails - 1) / kTails;
  // Few threads and many parts each: sixteen threads share them (attention and join of 2 sequences
  // of up to 14304 tokens, one kv head, 5 rows: 15.8 against 31.2 us; of one of 8000, 8 kv heads, 4
  // rows: 16.8 against 20.7).  With 8192 pieces or more the GPU is full either way, and 16 times
  // the workgroups cost (8 such sequences: 35.2 against 34.4; one tree of 256 rows: 62 against 38),
  // and with few parts there is nothing to share (4 each: 14.5 and 14.4).
  const long long groups = (long long)a.c.seqs * a.c.kv_heads * p.mts;
  if (p.workers >= 8 * groups && groups * pieces <= 4096)
    hipLaunchKernelGGL((k_tree_join<BF16, D, C::kMT, 16>), dim3((pieces + 15) / 16, tails),
                       dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((k_tree_join<BF16, D, C::kMT, 1>), dim3((pieces + 255) / 256, tails),
                       dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <bool BF16, int D>
hipError_t launch_dim(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  if constexpr (D * (BF16 ? 2 : 4) > 512) return launch_shape<BF16, D, 64>(a, p, stream);
  else {
    if constexpr (!BF16 || D == 64 || D == 256)
      if (p.row_tile == 32) return launch_shape<BF16, D, 32>(a, p, stream);
    if (p.row_tile == 64) return launch_shape<BF16, D, 64>(a, p, stream);
    if constexpr (BF16 && 256 % (D * 2) == 0)
      if (p.row_tile == 256) return launch_shape<BF16, D, 256>(a, p, stream);
    return launch_shape<BF16, D, 128>(a, p, stream);
  }
}

template <bool BF16>
hipError_t launch_type(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  switch (a.c.head_dim) {
    case 64: return launch_dim<BF16, 64>(a, p, stream);
    case 96: return launch_dim<BF16, 96>(a, p, stream);
    case 128: return launch_dim<BF16, 128>(a, p, stream);
    case 256: return launch_dim<BF16, 256>(a, p, stream);
    default: return hipErrorInvalidValue;
  }
}

// The shape of a row tile, with the workgroups that LDS and the waves' registers leave room for.
template <bool BF16, int D, int RT>
Shape filled_shape() {
  Shape sh = shape_for<BF16, D>(RT);
  constexpr Shape c = shape_for<BF16, D>(RT);
  using C = Attn<BF16, D, c.wm, c.wk, c.ks, c.nst>;
  const int by_lds = kLdsBytes / (int)sizeof(typename C::Lds), by_waves = 4 * c.occ / C::kNW;
  sh.per_cu = by_lds < by_waves ? by_lds : by_waves;
  return sh;
}

template <bool BF16, int D>
Shape shape_of_dim(int row_tile) {
  if constexpr (D * (BF16 ? 2 : 4) > 512) return filled_shape<BF16, D, 64>();
  else {
    if constexpr (!BF16 || D == 64 || D == 256)
      if (row_tile == 32) return filled_shape<BF16, D, 32>();
    if constexpr (BF16 && 256 % (D * 2) == 0)
      if (row_tile == 256) return filled_shape<BF16, D, 256>();
    if (row_tile == 64) return filled_shape<BF16, D, 64>();
    return filled_shape<BF16, D, 128>();
  }
}

template <bool BF16>
Shape shape_of(int D, int row_tile) {
  switch (D) {
    case 64: return shape_of_dim<BF16, 64>(row_tile);
    case 96: return shape_of_dim<BF16, 96>(row_tile);
    case 128: return shape_of_dim<BF16, 128>(row_tile);
    default: return shape_of_dim<BF16, 256>(row_tile);
  }
}

// Rows of a tile.  A tile too small reads the keys again for each further one, a tile too large
// computes rows that do not exist and leaves larger parts; the smallest that holds all rows, but
// (attention and join; 8 kv heads; A: 64 sequences of 1023 to 8191 tokens, 4 rows a kv head; B: 32
// of 512 to 4096, the rows given; C: 32 of 4096, 4 rows):
// - bf16 rows of 192 and 256 bytes take 64 instead of 32: LDS holds two workgroups either way and
//   four waves load better than two (128 columns, tiles of 64 against 32: C 108 and 114 us, B with
//   20 rows 67 and 69, with 32 rows 71 and 74, A 222 and 221; 96 columns: C 86 and 89, B with 32
//   rows 53 and 53, A 205 and 201).  With 128 bytes LDS holds more workgroups of two waves (A: 122
//   us with 32 rows a tile, 142 with 64), with 512 one tile each (A: 422 and 428), and fp32 products
//   of rows that do not exist cost 16 times as much (64 columns, A: 259 and 363).
// - beyond 128 rows bf16 rows of 128 and 256 bytes take 256 rows a workgroup and the kernel's
//   pipelined loop (B with 256 rows, tiles of 256 against 128: 126 and 144 us at 128 columns, 78
//   and 82 at 64; with 128 rows, 128 columns: 106 and 96).  Rows of 192 bytes do not spread evenly
//   over eight waves' loads, those of 512 leave no room for four tiles of the loop's 64 keys; fp32
//   takes 128 (B with 128 rows, tiles of 128 against 64: 366 and 400 us at 128 columns, 187 and 202
//   at 64).
// - rows of 1024 bytes (fp32) stay at 64: O of a row takes 128 registers, Q 128.
int row_tile_for(bool bf16, int row_bytes, long long rows) {
  if (rows <= 32 && !(bf16 && row_bytes > 128 && row_bytes <= 256)) return 32;
  if (rows <= 64) return 64;
  if (rows <= 128 || !bf16 || 256 % row_bytes) return 128;
  return 256;
}

}  // namespace

AttnPlan plan_tree_attention(const CacheView& c, sv_dtype dt, int N, int G) {
  AttnPlan p{};
  const bool bf16 = dt == SV_DTYPE_BF16;
  const long long rows = (long long)N * G;
  const int row_bytes = c.head_dim * c.esize;
  const int want = row_tile_for(bf16, row_bytes, rows);
  const Shape sh = bf16 ? shape_of<true>(c.head_dim, want) : shape_of<false>(c.head_dim, want);
  p.row_tile = 32 * sh.wm;
  p.key_tile = 32 * sh.wk * sh.ks;
  p.mts = (int)((rows + p.row_tile - 1) / p.row_tile);
  // as many workers as the GPU holds at once, and no more than pieces of work the table has room
  // for
  const int per_cu = sh.per_cu;
  const long long most = (long long)c.seqs * c.kv_heads * p.mts *
                         (((long long)c.cap + p.key_tile - 1) / p.key_tile);
  p.workers = (int)(most < (long long)kAttnCus * per_cu ? most : (long long)kAttnCus * per_cu);
  const size_t slots = (size_t)p.workers * 2 * p.row_tile;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  p.o_ml = up(slots * c.head_dim * sizeof(float));
  p.o_tail = p.o_ml + up(slots * sizeof(float2));
  p.bytes = p.o_tail + up((size_t)p.workers * sizeof(int4));
  return p;
}

hipError_t launch_tree_attention(const AttnArgs& a, sv_dtype dt, const AttnPlan& p,
                                 hipStream_t stream) {
  return dt == SV_DTYPE_BF16 ? launch_type<true>(a, p, stream) : launch_type<false>(a, p, stream);
}

}  // namespace sv
