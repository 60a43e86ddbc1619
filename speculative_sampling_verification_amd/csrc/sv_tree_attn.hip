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

#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "sv_cache.hpp"

namespace sv {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLn2 = 0.69314718055994530942f;

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

// Work of one sequence: key tiles of its live row tiles, and one piece (zeros to write) for
// each row tile that holds no node.
struct SeqWork {
  int len, n, keys;  // committed tokens, nodes, keys behind the table
  int tiles, live;   // key tiles (at least one), row tiles with a node
  long long units;
};

template <int MT, int BN>
__device__ __forceinline__ SeqWork seq_work(const AttnArgs& a, int b) {
  SeqWork s;
  int len = a.c.lens[b];
  len = len < 0 ? 0 : len;
  s.len = len > a.c.cap ? a.c.cap : len;
  int n = a.nodes ? a.nodes[b] : a.N;
  n = n < 0 ? 0 : n;
  s.n = n > a.N ? a.N : n;
  const int keys = s.len + s.n;
  s.keys = keys > a.c.cap ? a.c.cap : keys;
  const int tiles = (s.keys + BN - 1) / BN;
  s.tiles = tiles < 1 ? 1 : tiles;
  s.live = (s.n * a.G + MT - 1) / MT;
  s.units = (long long)a.c.kv_heads * ((long long)s.live * s.tiles + (a.mts - s.live));
  return s;
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

// WM waves share the rows (32 each), WK the keys of a tile (KS blocks of 32 each).
template <bool BF16, int D, int WM, int WK, int KS>
struct Attn {
  static constexpr int kES = BF16 ? 2 : 4;
  static constexpr int kNW = WM * WK;
  static constexpr int kNT = 64 * kNW;
  static constexpr int kMT = 32 * WM;
  static constexpr int kBN = 32 * WK * KS;
  static constexpr int kRow = D * kES;        // bytes of a row
  static constexpr int kVecs = kRow / 16;     // 16-byte vectors of a row
  // Row pitches in LDS.  K is read 16 bytes a lane down 32 rows: a pitch of an odd number of
  // 16-byte units spreads 16 rows over all 64 banks.  V (bf16) is read 64 bytes wide over 4
  // rows: a pitch of 64 bytes mod 128 puts those in different banks; V (fp32) is read 128 bytes
  // wide in two rows 4 apart: a pitch of 32 bytes mod 64.
  static constexpr int kPitchK = kRow + 16;
  static constexpr int kPitchV = BF16 ? (kRow % 128 == 0 ? kRow + 64 : kRow) : kRow + 32;
  static constexpr int kND = D / 32;
  static constexpr int kLoads = kBN * kVecs / kNT;  // vectors a thread stages per tensor
  static constexpr int kTileBytes = kBN * (kPitchK + kPitchV);
  static constexpr int kJoinBytes = WK > 1 ? kNW * kND * 16 * 64 * 4 : 0;
  static constexpr int kPool = kTileBytes > kJoinBytes ? kTileBytes : kJoinBytes;
  static_assert(D % 32 == 0 && (kBN * kVecs) % kNT == 0 && kBN % 64 == 0 && kBN <= kNT, "tile");

  struct Lds {
    alignas(16) char pool[kPool];          // K tile, V tile; the parts when waves join
    long long rowoff[2][kBN];              // byte offset of a key's row, -1: no such row
    uint32_t valid[2][kBN / 32];           // keys that exist
    uint32_t badv[2][kBN / 32];            // drafted nodes with non-finite values
    float m[kNW][32], l[kNW][32];
    long long scan[kNW + 1];
    long long start_off;
    int start_b;
  };
};

template <bool BF16, int D, int WM, int WK, int KS, int OCC>
__global__ __launch_bounds__(64 * WM * WK, OCC) void k_tree_attn(AttnArgs a) {
  using C = Attn<BF16, D, WM, WK, KS>;
  constexpr int MT = C::kMT, BN = C::kBN, NT = C::kNT, ND = C::kND;
  constexpr int QF = BF16 ? D / 16 : D / 8;  // 16-byte pieces of a Q row a lane holds
  __shared__ typename C::Lds S;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % WM, wk = wave / WM;
  const int half = lane >> 5, col = lane & 31;
  const float sl2 = a.scale * 1.44269504088896340736f;  // scores to log2 units

  // worker number: consecutive workers share keys and should share an XCD's L2 (workgroups are
  // handed to the eight XCDs in turn)
  int w = blockIdx.x;
  if ((a.workers & 7) == 0) w = (w & 7) * (a.workers >> 3) + (w >> 3);

  // where this worker's pieces begin: prefix sums of the sequences' work
  long long total, per, pos, end;
  {
    const int chunk = (a.c.seqs + NT - 1) / NT;
    const int b0 = tid * chunk, b1 = b0 + chunk < a.c.seqs ? b0 + chunk : a.c.seqs;
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += seq_work<MT, BN>(a, b).units;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const long long y = __shfl_up(incl, d);
      incl += lane >= d ? y : 0;
    }
    if (lane == 63) S.scan[wave] = incl;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < C::kNW; ++i) {
      before += i < wave ? S.scan[i] : 0;
      total += S.scan[i];
    }
    per = (total + a.workers - 1) / a.workers;
    pos = w * per;
    end = pos + per < total ? pos + per : total;
    long long p = before + incl - mine;
    if (pos >= p && pos < p + mine) {
      int b = b0;
      for (; b < b1; ++b) {
        const long long u = seq_work<MT, BN>(a, b).units;
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
  long long off = S.start_off;
  const long long begin = pos;

  while (pos < end) {
    const SeqWork sw = seq_work<MT, BN>(a, b);
    if (off >= sw.units) {
      off -= sw.units;
      ++b;
      continue;
    }
    const long long live_units = (long long)a.c.kv_heads * sw.live * sw.tiles;
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
    const long long grp = off / sw.tiles;
    const int t0 = (int)(off - grp * sw.tiles);
    const int h = (int)(grp / sw.live), mt = (int)(grp - (long long)h * sw.live);
    const long long left = end - pos;
    const int t1 = (long long)(sw.tiles - t0) < left ? sw.tiles : t0 + (int)left;
    const int rows = sw.n * a.G;             // live rows of the (sequence, kv head)
    const int my_row = mt * MT + wm * 32 + col;
    const int my_node = my_row / a.G, my_g = my_row - my_node * a.G;
    const bool row_live = my_row < rows;
    const int32_t* table = a.c.table + (size_t)b * a.c.width;
    const char* kbase = a.c.k + (long long)h * a.c.head_stride;
    const char* vbase = a.c.v + (long long)h * a.c.head_stride;

    u32x4 qf[QF];
    {
      const char* qp = a.q + (long long)b * a.q_seq + (long long)my_node * a.q_node +
                       (long long)(h * a.G + my_g) * a.q_head + half * 16;
#pragma unroll
      for (int s = 0; s < QF; ++s)
        qf[s] = row_live ? *reinterpret_cast<const u32x4*>(qp + s * 32) : u32x4{0, 0, 0, 0};
    }

    auto load_entry = [&](int t) -> int {  // page of key t * BN + tid, -1: none
      const int key = t * BN + tid;
      if (tid >= BN || key >= sw.keys) return -1;
      return table[fast_div(a.c.page_div, (uint32_t)key)];
    };
    auto put_rows = [&](int t, int page) {
      if (tid < BN) {
        const int key = t * BN + tid;
        const bool ok = page >= 0 && page < a.c.pages;
        const uint32_t pi = fast_div(a.c.page_div, (uint32_t)key);
        const int slot = key - (int)(pi * a.c.page_div.d);
        S.rowoff[t & 1][tid] = ok ? (long long)page * a.c.page_stride +
                                        (long long)slot * a.c.token_stride
                                  : -1ll;
        const unsigned long long bits = __ballot(ok);
        if (lane == 0) {
          S.valid[t & 1][(tid >> 5)] = (uint32_t)bits;
          S.valid[t & 1][(tid >> 5) + 1] = (uint32_t)(bits >> 32);
          S.badv[t & 1][(tid >> 5)] = 0u;
          S.badv[t & 1][(tid >> 5) + 1] = 0u;
        }
      }
    };
    u32x4 kr[C::kLoads], vr[C::kLoads];
    uint32_t missing = 0;  // bit i: vector i's row does not exist (its load reads page 0)
    auto issue = [&](int t) {
      missing = 0;
#pragma unroll
      for (int i = 0; i < C::kLoads; ++i) {
        const int x = tid + i * NT, r = x / C::kVecs, cv = x - r * C::kVecs;
        const long long o = S.rowoff[t & 1][r];
        missing |= (o < 0 ? 1u : 0u) << i;
        const long long at = (o < 0 ? 0 : o) + cv * 16;
        kr[i] = *reinterpret_cast<const u32x4*>(kbase + at);
        vr[i] = *reinterpret_cast<const u32x4*>(vbase + at);
      }
    };
    auto stage = [&](int t) {
      if (__any(missing != 0)) {
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) {
          const uint32_t keep = (missing >> i & 1u) - 1u;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            kr[i][j] &= keep;
            vr[i][j] &= keep;
          }
        }
      }
      // a node's values may be hidden from some rows: 0 * inf must not reach them
      if ((t + 1) * BN > sw.len) {
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) {
          const int r = (tid + i * NT) / C::kVecs;
          if (t * BN + r >= sw.len && clear_non_finite<BF16>(vr[i]))
            atomicOr(&S.badv[t & 1][r >> 5], 1u << (r & 31));
        }
      }
#pragma unroll
      for (int i = 0; i < C::kLoads; ++i) {
        const int x = tid + i * NT, r = x / C::kVecs, cv = x - r * C::kVecs;
        *reinterpret_cast<u32x4*>(S.pool + r * C::kPitchK + cv * 16) = kr[i];
        *reinterpret_cast<u32x4*>(S.pool + BN * C::kPitchK + r * C::kPitchV + cv * 16) = vr[i];
      }
    };

    float m = -INFINITY, l = 0.0f;
    f32x16 acc[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;

    put_rows(t0, load_entry(t0));
    int entry = t0 + 1 < t1 ? load_entry(t0 + 1) : -1;
    __syncthreads();
    issue(t0);

    for (int t = t0; t < t1; ++t) {
      __syncthreads();  // the waves are done with the last tile
      stage(t);
      if (t + 1 < t1) put_rows(t + 1, entry);
      __syncthreads();
      if (t + 1 < t1) issue(t + 1);
      entry = t + 2 < t1 ? load_entry(t + 2) : -1;

      __builtin_amdgcn_sched_barrier(0);
      // scores of this wave's keys: lane = row, register r = key 8 (r / 4) + 4 half + r % 4
      f32x16 s[KS];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const char* kp = S.pool + ((wk * KS + ks) * 32 + col) * C::kPitchK + half * 16;
#pragma unroll
        for (int r = 0; r < 16; ++r) s[ks][r] = 0.0f;
#pragma unroll
        for (int q = 0; q < QF; ++q) {
          const u32x4 kf = *reinterpret_cast<const u32x4*>(kp + q * 32);
          if constexpr (BF16) {
            s[ks] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                __builtin_bit_cast(bf16x8, kf), __builtin_bit_cast(bf16x8, qf[q]), s[ks], 0, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[ks] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                  __uint_as_float(kf[e]), __uint_as_float(qf[q][e]), s[ks], 0, 0, 0);
          }
        }
      }

      __builtin_amdgcn_sched_barrier(0);  // keeps the phases' registers apart
      // hide keys that do not exist and nodes that the row does not see
      uint32_t seen[KS];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int blk = wk * KS + ks, key0 = t * BN + blk * 32;
        const uint32_t have = S.valid[t & 1][blk];
        seen[ks] = 0xFFFFu;
        if (have != 0xFFFFFFFFu || key0 + 32 > sw.len) {
          // bit r of `bits`: the row sees register r's key.  Nodes: node0 is that of register 0
          const int node0 = key0 + 4 * half - sw.len;
          const int me = row_live ? my_node : 0;
          uint32_t bits = 0;
          if (a.mask) {
            const uint8_t* mrow = a.mask + ((size_t)b * a.N + me) * a.N;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int node = node0 + 8 * (r >> 2) + (r & 3);
              const int at = node < 0 ? 0 : node < a.N ? node : a.N - 1;
              bits |= (mrow[at] != 0 || node < 0 ? 1u : 0u) << r;
            }
          } else {
            const int lim = me - node0;  // the last key offset that a chain's node sees
            bits = of_half(lim < 0 ? 0u : lim > 30 ? 0xFFFFFFFFu : (2u << lim) - 1u);
          }
          bits &= of_half(have >> (4 * half));
#pragma unroll
          for (int r = 0; r < 16; ++r) s[ks][r] = bits & (1u << r) ? s[ks][r] : -INFINITY;
          seen[ks] = bits;
        }
      }

      // running maximum in units of log2 (z log2 e, so that P and every later rescaling use the
      // same rounded number); P = exp(z - m); O and l rescaled when the maximum grew
      float mx = s[0][0];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[ks][r]);
      const float m_new = fmaxf(m, half_max(mx) * sl2);
      const float m_use = m_new == -INFINITY ? 0.0f : m_new;
      if (__any(m_new > m)) {
        const float f = __builtin_amdgcn_exp2f(m - m_use);
        l *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[d][r] *= f;
        m = m_new;
      }
      float sum = 0.0f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[ks][r] = __builtin_amdgcn_exp2f(s[ks][r] * sl2 - m_use);
          sum += s[ks][r];
        }
      l += sum;

      __builtin_amdgcn_sched_barrier(0);
      // O^T += V^T P^T
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int blk = wk * KS + ks;
        const char* vp = S.pool + BN * C::kPitchK + blk * 32 * C::kPitchV;
        if constexpr (BF16) {
          // P rounded to bf16 for the matrix instruction: half a step of 2^-8 per weight, the
          // rounding the inputs carry; the sum l keeps the unrounded weights
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            bf16x8 pf;
#pragma unroll
            for (int j = 0; j < 8; ++j) pf[j] = (__bf16)s[ks][8 * c + j];
            // 16 lanes read 4 keys x 16 columns; lane i supplies row i / 4, 8 bytes i % 4
            const char* vt = vp + (16 * c + 4 * half + ((lane & 15) >> 2)) * C::kPitchV +
                             ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              const short4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (SV_LDS(short4v)*)(vt + d * 64));
              const short4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (SV_LDS(short4v)*)(vt + 8 * C::kPitchV + d * 64));
              typedef short short8v __attribute__((ext_vector_type(8)));
              const short8v vf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
              acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vf), pf,
                                                               acc[d], 0, 0, 0);
            }
          }
        } else {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const char* vt = vp + (8 * (r >> 2) + 4 * half + (r & 3)) * C::kPitchV + col * 4;
#pragma unroll
            for (int d = 0; d < ND; ++d)
              acc[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                  *reinterpret_cast<const float*>(vt + d * 128), s[ks][r], acc[d], 0, 0, 0);
          }
        }

        // non-finite values of drafted nodes, for the rows that see them (rare: a rolled loop
        // over a copy of O in scratch memory keeps it out of the registers of the common path)
        uint32_t bad = S.badv[t & 1][blk];
        if (__builtin_expect(bad != 0, 0)) {
          float o[ND * 16];
#pragma unroll
          for (int i = 0; i < ND * 16; ++i) o[i] = acc[i >> 4][i & 15];
          while (bad) {
            const int kk = __builtin_amdgcn_readfirstlane(__ffs(bad) - 1);
            bad &= bad - 1;
            const int hk = (kk >> 2) & 1, rk = ((kk >> 3) << 2) | (kk & 3);
            float p = 0.0f;
            int sees = 0;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              p = r == rk ? s[ks][r] : p;
              sees = r == rk ? (int)(seen[ks] >> r & 1u) : sees;
            }
            p = __shfl(p, col + 32 * hk);
            sees = __shfl(sees, col + 32 * hk);
            const char* row = vbase + S.rowoff[t & 1][blk * 32 + kk];
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
        }
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
        lt += S.l[i * WM + wm][col] *
              __builtin_amdgcn_exp2f(S.m[i * WM + wm][col] - mu);
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

    const long long first = pos - t0;  // the group's first piece
    const bool whole = t0 == 0 && t1 == sw.tiles;
    const int slot = 2 * w + (pos == begin ? 0 : 1);
    const int hq = a.c.kv_heads * a.G;
    const size_t orow = ((size_t)b * a.N + my_node) * hq + h * a.G + my_g;
    const bool row_out = my_node < a.N;  // padding nodes get zeros
    const float inv = !row_live || l == 0.0f ? 0.0f : 1.0f / l;
    auto emit = [&](int d, int r4, f32x4 x) {
      const int e = d * 32 + 8 * r4 + 4 * half;
      if (whole) {
        if (!row_out) return;
        if (!row_live) x = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (BF16) {
          bf16x4 y;
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = (__bf16)(x[j] * inv);
          *reinterpret_cast<bf16x4*>(a.out + orow * C::kRow + e * 2) = y;
        } else {
          *reinterpret_cast<f32x4*>(a.out + orow * C::kRow + e * 4) = x * inv;
        }
      } else if (row_live) {
        *reinterpret_cast<f32x4*>(a.part + ((size_t)slot * MT + wm * 32 + col) * D + e) = x;
      }
    };
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
    if (wk == 0 && half == 0) {
      if (whole) {
        if (a.lse && row_out)
          a.lse[orow] = !row_live || l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
      } else {
        a.part_ml[(size_t)slot * MT + wm * 32 + col] = make_float2(m, l);
      }
    }
    if (tid == 0 && t0 == 0 && !whole)
      a.tail[w] = make_int4(b, h * a.mts + mt, slot, (int)((first + sw.tiles - 1) / per - w + 1));
    __syncthreads();
    pos += t1 - t0;
    off += t1 - t0;
  }
}

// Joins the parts of the group that begins with worker blockIdx.x's last part and ends with a
// later worker: every later part is that worker's first.  One thread per four columns of a row.
template <bool BF16, int D, int MT>
__global__ __launch_bounds__(256) void k_tree_join(AttnArgs a) {
  const int4 g = a.tail[blockIdx.x];
  if (g.w < 2) return;
  const int b = g.x, h = g.y / a.mts, mt = g.y - h * a.mts;
  const int i = blockIdx.y * 256 + threadIdx.x;
  const int row = i / (D / 4), e = (i - row * (D / 4)) * 4;
  const int r = mt * MT + row;
  const int node = r / a.G, hg = r - node * a.G;
  if (row >= MT || node >= a.N) return;
  const int hq = a.c.kv_heads * a.G;
  const size_t orow = ((size_t)b * a.N + node) * hq + h * a.G + hg;
  int n = a.nodes ? a.nodes[b] : a.N;
  n = n > a.N ? a.N : n;
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
  float m = -INFINITY, l = 0.0f;
  if (node < n) {
    // parts: slot g.z, then slot 0 of each later worker
    auto slot_of = [&](int s) { return s == 0 ? (size_t)g.z : (size_t)2 * (g.z / 2 + s); };
    for (int s = 0; s < g.w; ++s) m = fmaxf(m, a.part_ml[slot_of(s) * MT + row].x);
    const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll 4
    for (int s = 0; s < g.w; ++s) {
      const float2 ml = a.part_ml[slot_of(s) * MT + row];
      const float f = __builtin_amdgcn_exp2f(ml.x - mu);
      const f32x4 y = *reinterpret_cast<const f32x4*>(a.part + (slot_of(s) * MT + row) * D + e);
      l += ml.y * f;
      x += y * f;
    }
  }
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

// Tile shapes: KS blocks of 32 keys a wave; OCC waves per SIMD that the registers must allow.
struct Shape {
  int wm, wk, ks;
};
constexpr int kRowBytes1 = 256;  // rows up to this many bytes leave room for two workgroups

template <bool BF16, int D>
constexpr Shape shape_for(int row_tile) {
  constexpr int row = D * (BF16 ? 2 : 4);
  if (row > 512) return Shape{2, 2, 1};
  if (row_tile == 32) return Shape{1, 4, 1};
  if (row_tile == 64) return Shape{2, 2, row > kRowBytes1 ? 1 : 2};
  return Shape{4, 1, 2};
}

template <bool BF16, int D, int RT>
hipError_t launch_shape(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  constexpr Shape sh = shape_for<BF16, D>(RT);
  constexpr int occ = D * (BF16 ? 2 : 4) > kRowBytes1 ? 1 : 2;
  using C = Attn<BF16, D, sh.wm, sh.wk, sh.ks>;
  if (p.row_tile != C::kMT || p.key_tile != C::kBN) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_tree_attn<BF16, D, sh.wm, sh.wk, sh.ks, occ>), dim3(p.workers),
                     dim3(C::kNT), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.workers > 1)
    hipLaunchKernelGGL((k_tree_join<BF16, D, C::kMT>), dim3(p.workers, C::kMT * D / 4 / 256),
                       dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <bool BF16, int D>
hipError_t launch_dim(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  if constexpr (D * (BF16 ? 2 : 4) > 512) return launch_shape<BF16, D, 64>(a, p, stream);
  else {
    if (p.row_tile == 32) return launch_shape<BF16, D, 32>(a, p, stream);
    if (p.row_tile == 64) return launch_shape<BF16, D, 64>(a, p, stream);
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

template <bool BF16>
Shape shape_of(int D, int row_tile) {
  switch (D) {
    case 64: return shape_for<BF16, 64>(row_tile);
    case 96: return shape_for<BF16, 96>(row_tile);
    case 128: return shape_for<BF16, 128>(row_tile);
    default: return shape_for<BF16, 256>(row_tile);
  }
}

}  // namespace

AttnPlan plan_tree_attention(const CacheView& c, sv_dtype dt, int N, int G) {
  AttnPlan p{};
  const bool bf16 = dt == SV_DTYPE_BF16;
  const long long rows = (long long)N * G;
  const int want = rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  const Shape sh = bf16 ? shape_of<true>(c.head_dim, want) : shape_of<false>(c.head_dim, want);
  p.row_tile = 32 * sh.wm;
  p.key_tile = 32 * sh.wk * sh.ks;
  p.mts = (int)((rows + p.row_tile - 1) / p.row_tile);
  // two workgroups fit a compute unit where a row has at most 256 bytes; no more workers than
  // pieces of work the table has room for
  const int per_cu = c.head_dim * c.esize > kRowBytes1 ? 1 : 2;
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
