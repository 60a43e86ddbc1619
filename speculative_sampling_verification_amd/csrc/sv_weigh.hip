// Attention weights that a step's nodes spend on the committed tokens, on gfx950.  For every key j of
// a sequence and kv head,
//   w_j <- decay w_j + sum over rows (node i, query head) of exp(scale q.k_j - lse_row),
// a row counting where it sees key j (j below its node's limit).  The logarithm of a row's sum lse
// comes from attention, so one pass over the keys suffices and every key's sum is its own: no parts
// to join, no atomics.
//
// Products Q K^T in 16x16 matrix instructions: a lane then holds one key and four of 16 rows, so a
// key's sum over rows is a lane's own sum and one over the four lanes that share the key.  A wave
// loads the keys of its piece straight into the registers that the matrix instructions read (no LDS:
// no other wave has use for them) and keeps them there for all rows.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "sv_lds_load.hpp"
#include "sv_step.hpp"

namespace sv {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWeighThreads = 256;
constexpr int kWeighWaves = kWeighThreads / 64;
// Rows a kv head up to which k_weigh is taken, the one matrix instruction's: one token of 32 query
// heads to 8 kv heads of 128 in 64 sequences of up to 8191 tokens takes 128 us (k_weigh_rows 155),
// 16 rows in 32 sequences of up to 4096 31 us (38); 20 rows there 35.
constexpr int kFewRows = 16;
// Rows up to which k_weigh_rows has 32 keys of 256 bytes a wave, 64 beyond.  One sequence of 131072
// tokens, 8 kv heads, 32 keys (64): 24 rows 62 us (66), 64 rows 62 (67), 128 rows 76 (79), 160 rows
// 92 (90), 256 rows 114 (109), 512 rows 195 (180).  Shorter keys always go 64 a wave (of 128 bytes:
// 24 rows 34 us, 41 with 32; of 192: 48, 51), longer ones 32 (64 do not fit the registers); fp32 of
// 256 bytes, where products take the time, 32 (64 and 32 alike on long sequences, 70 us against 58 for
// 256 rows in 16 sequences of 2048).
constexpr int kSomeRows = 128;
constexpr float kLog2e = 1.44269504088896340736f;

// Keys of sequence b that are weighed.
__device__ __forceinline__ int keys_of(const WeighArgs& a, int b) {
  const int len = clamp_len(a.c, a.c.lens[b]);
  return len < a.length ? len : a.length;
}

template <int Keys>
__device__ __forceinline__ long long pieces_of(const WeighArgs& a, int b) {
  return (long long)a.c.kv_heads * ((keys_of(a, b) + Keys - 1) / Keys);
}

// This workgroup's share of the pieces: as many as any other's, or one less.  Pieces of a sequence
// are ordered by key tile, then head; *off is the first one's number in sequence *b.
struct Share {
  long long first, end;
};
template <int Keys>
__device__ __forceinline__ Share find_pieces(const WeighArgs& a, int* b_out, long long* off_out) {
  __shared__ long long scan[kWeighWaves];
  __shared__ int start_b;
  __shared__ long long start_off;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunk = (a.c.seqs + kWeighThreads - 1) / kWeighThreads;
  const int b0 = tid * chunk, b1 = b0 + chunk < a.c.seqs ? b0 + chunk : a.c.seqs;
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += pieces_of<Keys>(a, b);
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long long y = __shfl_up(incl, d);
    incl += lane >= d ? y : 0;
  }
  if (lane == 63) scan[wave] = incl;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kWeighWaves; ++i) {
    before += i < wave ? scan[i] : 0;
    all += scan[i];
  }
  const long long each = all / gridDim.x, left = all - each * gridDim.x, w = blockIdx.x;
  const long long pos = each * w + (w < left ? w : left);
  long long p = before + incl - mine;
  if (pos >= p && pos < p + mine) {
    int b = b0;
    for (; b < b1; ++b) {
      const long long n = pieces_of<Keys>(a, b);
      if (pos < p + n) break;
      p += n;
    }
    start_b = b;
    start_off = pos - p;
  }
  __syncthreads();
  *b_out = pos < all ? start_b : a.c.seqs;
  *off_out = pos < all ? start_off : 0;
  return Share{pos, pos + each + (w < left ? 1 : 0)};
}

// Up to 16 rows: a wave takes KT blocks of 16 keys at a time.  The next piece's page numbers are on
// their way while one is computed.  Its keys and queries are not: they take the same registers, so a
// wave loads them behind its products and waits, and the compute unit's other waves fill the time.
//
// Bound by the keys' bytes where rows are long: 620 MB of bf16 keys of 128 columns in 128 us, 4.85 TB/s (a
// large copy runs at 5.2).  Pieces of a page a workgroup took 179 us, three workgroups a compute unit
// and no more than run at once as here 128: a fourth waiting its turn made it 179 again.  Keys loaded
// past the caches: 139.  Shorter pieces wait for their loads more than that hides: 16 sequences of 512 to
// 4096 tokens take 17 us at 64 columns of bf16 (2.35 TB/s), 15 at 96 (3.9), 22 at 64 of fp32 (3.5),
// 35 at 128 (4.35).
template <bool BF16, int D>
struct Few {
  static constexpr int kRow = D * (BF16 ? 2 : 4);
  static constexpr int NF = kRow / 64;  // 16-byte pieces of a row that a lane holds
  static constexpr int KT = kRow <= 256 ? 4 : kRow <= 512 ? 2 : 1;  // 64 registers of keys
  static constexpr int kKeys = 16 * KT;
  static constexpr int kOcc = kRow <= 512 ? 3 : 2;  // workgroups a compute unit
};

template <bool BF16, int D>
__global__ __launch_bounds__(kWeighThreads, (Few<BF16, D>::kOcc)) void k_weigh(WeighArgs a) {
  using C = Few<BF16, D>;
  constexpr int KT = C::KT, NF = C::NF;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const float sl2 = a.scale * kLog2e;
  const int Hkv = a.c.kv_heads;
  struct Piece {
    int b, h, key0, keys, held;
  };
  // the wave's place in the line of pieces
  long long off;
  int b;
  const Share share = find_pieces<C::kKeys>(a, &b, &off);
  b = __builtin_amdgcn_readfirstlane(b);
  long long pos = share.first + wave;
  off += wave;
  auto next_piece = [&](Piece& p) __attribute__((always_inline)) {
    if (pos >= share.end) return false;
    int keys = keys_of(a, b);
    long long n = (long long)Hkv * ((keys + C::kKeys - 1) / C::kKeys);
    while (off >= n) {
      off -= n;
      if (++b >= a.c.seqs) return false;
      keys = keys_of(a, b);
      n = (long long)Hkv * ((keys + C::kKeys - 1) / C::kKeys);
    }
    const int tile = (int)(off >> 31 ? off / Hkv : (uint32_t)off / (uint32_t)Hkv);
    p.b = b;
    p.h = (int)(off - (long long)tile * Hkv);
    p.key0 = tile * C::kKeys;
    p.keys = keys;
    p.held = positions_held(a.c, b);
    pos += kWeighWaves;
    off += kWeighWaves;
    return true;
  };
  auto load_pages = [&](const Piece& p, int (&page)[KT]) __attribute__((always_inline)) {
    const int32_t* table = a.c.table + (size_t)p.b * a.c.width;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int key = p.key0 + t * 16 + col;
      page[t] = table[fast_div(a.c.page_div, (uint32_t)(key < p.keys ? key : p.keys - 1))];
    }
  };
  u32x4 kf[KT][NF], qf[NF];
  int number[KT];  // of this lane's keys; out of every row's sight where one does not exist
  float lse[4], old = 0.0f;
  int see[4];
  auto load_piece = [&](const Piece& p, const int (&page)[KT]) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int key = p.key0 + t * 16 + col;
      int64_t row = 0;
      number[t] = INT32_MAX;
      if (key < p.keys && names_page(a.c, p.held, key, page[t])) {
        const uint32_t pi = fast_div(a.c.page_div, (uint32_t)key);
        row = (int64_t)page[t] * a.c.page_stride +
              (int64_t)(key - (int)(pi * a.c.page_div.d)) * a.c.token_stride;
        number[t] = key;
      }
      const char* at = a.c.k + row + (int64_t)p.h * a.c.head_stride + quad * 16;
#pragma unroll
      for (int s = 0; s < NF; ++s) kf[t][s] = *reinterpret_cast<const u32x4*>(at + s * 64);
    }
    int n = a.nodes ? a.nodes[p.b] : a.N;
    n = n < 0 ? 0 : n < a.N ? n : a.N;
    const int rows = n * a.G;
    {
      const int node = (int)fast_div(a.g_div, (uint32_t)col), g = col - node * a.G;
      const char* at = a.q.at + (int64_t)p.b * a.q.seq + (int64_t)node * a.q.node +
                       (int64_t)(p.h * a.G + g) * a.q.head + quad * 16;
#pragma unroll
      for (int s = 0; s < NF; ++s)
        qf[s] = col < rows ? *reinterpret_cast<const u32x4*>(at + s * 64) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = quad * 4 + e;
      lse[e] = -INFINITY;
      see[e] = 0;
      if (r < rows) {
        const int node = (int)fast_div(a.g_div, (uint32_t)r), g = r - node * a.G;
        const int64_t at = (int64_t)p.b * a.N + node;
        lse[e] = a.lse[at * ((int64_t)Hkv * a.G) + p.h * a.G + g];
        see[e] = a.seen ? a.seen[at] : INT32_MAX - 1;
      }
    }
    if (a.decay != 0.0f && lane < C::kKeys && p.key0 + lane < p.keys)
      old = a.w[((int64_t)p.b * Hkv + p.h) * a.length + p.key0 + lane];
  };

  Piece p, ahead;
  int page[KT], page_ahead[KT];
  bool some = next_piece(p), more = false;
  if (some) {
    load_pages(p, page);
    more = next_piece(ahead);
    if (more) load_pages(ahead, page_ahead);
    load_piece(p, page);
  }
  while (some) {
    float lse2[4];
    int limit[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool live = lse[e] != -INFINITY;
      lse2[e] = live ? lse[e] * kLog2e : 0.0f;
      limit[e] = !live ? 0 : see[e] < p.keys ? see[e] : p.keys;
    }
    float mine = 0.0f;  // the sum of this lane's key: lane 16 t + c has key c of block t
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < NF; ++s) {
        if constexpr (BF16) {
          z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, qf[s]),
                                                      __builtin_bit_cast(bf16x8, kf[t][s]), z, 0, 0,
                                                      0);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            z = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(qf[s][e]),
                                                     __uint_as_float(kf[t][s][e]), z, 0, 0, 0);
        }
      }
      float x = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = __builtin_amdgcn_exp2f(fmaf(z[e], sl2, -lse2[e]));
        x += number[t] < limit[e] ? w : 0.0f;
      }
      x += __shfl_xor(x, 16);  // the four lanes that share a key
      x += __shfl_xor(x, 32);
      mine = quad == t ? x : mine;
    }
    if (lane < C::kKeys && p.key0 + lane < p.keys)
      a.w[((int64_t)p.b * Hkv + p.h) * a.length + p.key0 + lane] =
          a.decay == 0.0f ? mine : fmaf(a.decay, old, mine);
    some = more;
    if (some) {
      p = ahead;
#pragma unroll
      for (int t = 0; t < KT; ++t) page[t] = page_ahead[t];
      more = next_piece(ahead);
      if (more) load_pages(ahead, page_ahead);
      load_piece(p, page);
    }
  }
}

// Many rows: a workgroup takes 128 KB keys, a wave 32 KB of them in registers, and all rows come by
// through LDS, RT at a time, two stages of them.  Products are 32x32 instructions: half the reads
// from LDS that 16x16 ones need for as many products.
//
// Bound by the matrix instructions and, between them, an exponential a product of 2 D operations: 64
// nodes of 64 query heads to 8 kv heads of 128 on 131072 tokens (512 rows) take 180 us, 775 TFLOP/s,
// and 256 nodes 590 us, 945 (a library product of 8192^3 runs at 1350).  Vector instructions fill 85 us
// of the 180, products 61 (at 2.15 GHz), and the two overlap little: waves wait 47% of their time.  The
// compiler waits for the keys, in order of the loads, where the loop of rows first uses them, and in
// every turn: so the first 32 rows of a stage wait for the next stage's, just asked for.
// Rows staged through registers took 209 us, with one workgroup a compute unit less 204; 128 rows a
// stage 272; products of the next 32 rows begun before the last ones' exponentials 217 (registers
// spill); four workgroups a unit 218; pieces that are left over when all workgroups have as many, in
// halves for two, or three stages with loads two ahead: no difference (with that wait in place).
template <bool BF16, int D, int KB, int RT>
struct Rows {
  static constexpr int kES = BF16 ? 2 : 4;
  static constexpr int kRow = D * kES;
  static constexpr int kChunks = kRow / 16;            // 16-byte pieces of a row
  static constexpr int kFrags = kChunks / 2;           // ... that a lane holds
  static constexpr int kKeys = 32 * KB * kWeighWaves;  // of a workgroup
  static constexpr int kLoads = RT * kChunks / kWeighThreads;  // pieces a thread loads a stage
  // workgroups a compute unit: what the registers of the keys and products leave room for, but for a
  // few a piece that are spilled (bf16: 11 of 64 keys of 256 bytes, 4 of 32, 2 of 64 keys of 128)
  static constexpr int kKeyRegs = KB * kRow / 8;
  static constexpr int kOcc = kKeyRegs > 64 ? 1 : kKeyRegs == 64 && KB == 1 ? 2
                              : kKeyRegs > 32 ? 3 : 4;
  // Whether the weights so far come with the keys: 20 rows of 32 sequences of up to 4096 tokens and 8
  // heads of 128 in bf16 37.2 -> 35.2 us, 64 rows 39.1 -> 36.9; with 64 keys of 256 bytes a wave more
  // registers spill (256 rows 72.8 -> 74.6), in fp32 too (64 rows 145 -> 150).
  static constexpr bool kEarly = BF16 && (KB == 1 || kKeyRegs < 64);
  static_assert(RT % 32 == 0 && RT <= kWeighThreads && RT * kChunks % kWeighThreads == 0, "stage");

  // Piece c of row r lies at place c ^ swz(r): rows read together lie in different banks.
  __device__ static __forceinline__ int swz(int r) {
    if constexpr (kRow % 256 == 0) return r & 15;
    else if constexpr (kRow == 128) return (r >> 1) & 7;
    else return (r >> 2) & 3;
  }

  struct Lds {
    alignas(16) char q[2][RT * kRow];
    alignas(16) float lse2[2][RT];
    alignas(16) int see[2][RT];
  };
};

template <bool BF16, int D, int KB, int RT>
__global__ __launch_bounds__(kWeighThreads)
__attribute__((amdgpu_waves_per_eu(Rows<BF16, D, KB, RT>::kOcc, Rows<BF16, D, KB, RT>::kOcc)))
void k_weigh_rows(WeighArgs a) {
  using C = Rows<BF16, D, KB, RT>;
  __shared__ typename C::Lds S;
  const uint32_t q_lds =
      (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)&S.q[0][0]);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const float sl2 = a.scale * kLog2e;
  long long off;
  int b;
  const Share share = find_pieces<C::kKeys>(a, &b, &off);
  constexpr int kAhead = 2;
  const int Hkv = a.c.kv_heads;
  for (long long pos = share.first; pos < share.end; ++pos, ++off) {
    for (; b < a.c.seqs; ++b) {
      const long long n = pieces_of<C::kKeys>(a, b);
      if (off < n) break;
      off -= n;
    }
    if (b >= a.c.seqs) break;
    const int tile = (int)(off >> 31 ? off / Hkv : (uint32_t)off / (uint32_t)Hkv);
    const int h = (int)(off - (long long)tile * Hkv);
    const int keys = keys_of(a, b), held = positions_held(a.c, b);
    const int32_t* table = a.c.table + (size_t)b * a.c.width;
    int n = a.nodes ? a.nodes[b] : a.N;
    n = n < 0 ? 0 : n < a.N ? n : a.N;
    const int rows = n * a.G;

    // A stage of rows on its way to LDS.  Loads fill LDS in lane order, so a lane loads the piece that
    // belongs at its place.  From stage to stage a thread's pieces are a fixed step apart where a
    // node's heads do not straddle stages.  (Behind the last row: the first one's, which no key takes.)
    auto row_at = [&](int r, int c) __attribute__((always_inline)) {
      const int node = (int)fast_div(a.g_div, (uint32_t)r), g = r - node * a.G;
      return a.q.at + (int64_t)b * a.q.seq + (int64_t)node * a.q.node +
             (int64_t)(h * a.G + g) * a.q.head + c * 16;
    };
    const bool even = RT % a.G == 0;
    const int64_t step = (int64_t)(RT / a.G) * a.q.node;
    const char* piece[C::kLoads];
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) {
      const int x = tid + i * kWeighThreads, r = x / C::kChunks;
      piece[i] = row_at(r, (x % C::kChunks) ^ C::swz(r)) - step;
    }
    float next_lse = 0.0f;
    int next_see = 0;
    auto load = [&](int r0, int to) __attribute__((always_inline)) {
      const bool whole = even && r0 + RT <= rows;
#pragma unroll
      for (int i = 0; i < C::kLoads; ++i) {
        const int x = tid + i * kWeighThreads, r = x / C::kChunks;
        piece[i] += step;
        const char* p = piece[i];
        if (!whole) p = row_at(r0 + r < rows ? r0 + r : 0, (x % C::kChunks) ^ C::swz(r));
        load_to_lds(p, q_lds + to * (RT * C::kRow) + wave * 1024 + i * (kWeighThreads * 16));
      }
      if (tid < RT) {
        const int r = r0 + tid;
        next_lse = -INFINITY;
        if (r < rows) {
          const int node = (int)fast_div(a.g_div, (uint32_t)r), g = r - node * a.G;
          next_lse = a.lse[((int64_t)b * a.N + node) * ((int64_t)Hkv * a.G) + h * a.G + g];
          next_see = a.seen ? a.seen[(int64_t)b * a.N + node] : INT32_MAX;
        }
      }
    };
    auto store = [&](int to) __attribute__((always_inline)) {
      if (tid < RT) {
        const bool live = next_lse != -INFINITY;
        S.lse2[to][tid] = live ? next_lse * kLog2e : 0.0f;
        S.see[to][tid] = !live ? 0 : next_see < keys ? next_see : keys;
      }
    };
    if (rows > 0) load(0, 0);

    // this wave's keys
    const int key0 = tile * C::kKeys + wave * (32 * KB);
    u32x4 kf[KB][C::kFrags];
    int number[KB];  // -1: the key does not exist
#pragma unroll
    for (int t = 0; t < KB; ++t) {
      const int key = key0 + t * 32 + col;
      int64_t row = 0;
      number[t] = -1;
      if (key < keys) {
        const uint32_t pi = fast_div(a.c.page_div, (uint32_t)key);
        const int page = table[pi];
        if (names_page(a.c, held, key, page)) {
          row = (int64_t)page * a.c.page_stride +
                (int64_t)(key - (int)(pi * a.c.page_div.d)) * a.c.token_stride;
          number[t] = key;
        }
      }
      const char* p = a.c.k + row + (int64_t)h * a.c.head_stride + half * 16;
#pragma unroll
      for (int s = 0; s < C::kFrags; ++s) kf[t][s] = *reinterpret_cast<const u32x4*>(p + s * 32);
    }
    float* w = a.w + ((int64_t)b * Hkv + h) * a.length + key0 + col;
    float sum[KB], old[KB];
#pragma unroll
    for (int t = 0; t < KB; ++t) {
      sum[t] = old[t] = 0.0f;
      if (C::kEarly && a.decay != 0.0f && half == 0 && key0 + t * 32 + col < keys)
        old[t] = w[t * 32];
    }

    store(0);
    tile_barrier();
    int at = 0;
    for (int r0 = 0; r0 < rows; r0 += RT, at ^= 1) {
      const bool more = r0 + RT < rows;
      if (more) load(r0 + RT, at ^ 1);
      const int see = S.see[at][lane % RT];
      const bool open = __all(see >= key0 + 32 * KB);  // every row sees all of the wave's keys
      if (__any(see > key0)) {
#pragma unroll 1
        for (int m = 0; m < RT; m += 32) {
          if (r0 + m >= rows) break;
          f32x16 z[KB];
          u32x4 qf[kAhead];  // read from LDS that far ahead of the products
          const char* q = &S.q[at][(m + col) * C::kRow];
          auto frag = [&](int s) __attribute__((always_inline)) {
            return *reinterpret_cast<const u32x4*>(q + ((2 * s + half) ^ C::swz(col)) * 16);
          };
#pragma unroll
          for (int s = 0; s < kAhead; ++s) qf[s] = frag(s);
#pragma unroll
          for (int t = 0; t < KB; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) z[t][e] = 0.0f;
#pragma unroll
          for (int s = 0; s < C::kFrags; ++s) {
#pragma unroll
            for (int t = 0; t < KB; ++t) {
              if constexpr (BF16) {
                z[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    __builtin_bit_cast(bf16x8, qf[s % kAhead]),
                    __builtin_bit_cast(bf16x8, kf[t][s]), z[t], 0, 0, 0);
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  z[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(qf[s % kAhead][e]),
                                                              __uint_as_float(kf[t][s][e]), z[t],
                                                              0, 0, 0);
              }
            }
            if (s + kAhead < C::kFrags) qf[s % kAhead] = frag(s + kAhead);
            __builtin_amdgcn_sched_barrier(0);  // the order as it stands
          }
          // register e is row 8 (e / 4) + 4 half + e % 4
          auto add = [&](auto all) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const int r = m + 2 * e + 4 * half;
              const f32x4 l = *reinterpret_cast<const f32x4*>(&S.lse2[at][r]);
              const int4 see = *reinterpret_cast<const int4*>(&S.see[at][r]);
              const int limit[4] = {see.x, see.y, see.z, see.w};
#pragma unroll
              for (int t = 0; t < KB; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float w = __builtin_amdgcn_exp2f(fmaf(z[t][e + i], sl2, -l[i]));
                  sum[t] += decltype(all)::value || key0 + t * 32 + col < limit[i] ? w : 0.0f;
                }
            }
          };
          if (open) add(std::true_type{});
          else add(std::false_type{});
        }
      }
      if (more) store(at ^ 1);
      tile_barrier();
    }
#pragma unroll
    for (int t = 0; t < KB; ++t) {
      const float x = sum[t] + __shfl_xor(sum[t], 32);
      if (half == 0 && key0 + t * 32 + col < keys) {
        const float mine = number[t] >= 0 ? x : 0.0f;
        w[t * 32] = a.decay == 0.0f ? mine : fmaf(a.decay, C::kEarly ? old[t] : w[t * 32], mine);
      }
    }
  }
}

template <int Keys>
unsigned grid_for(const WeighArgs& a, int waves_a_piece, int a_unit) {
  const int most = a_unit * kAttnCus;  // all that run at once
  const int longest = a.c.cap < a.length ? a.c.cap : a.length;
  const int64_t pieces = (int64_t)a.c.seqs * a.c.kv_heads * ((longest + Keys - 1) / Keys);
  const int64_t groups = (pieces * waves_a_piece + kWeighWaves - 1) / kWeighWaves;
  return (unsigned)(groups < most ? groups : most);
}

template <bool BF16, int D, int KB, int RT>
void launch_rows(const WeighArgs& a, hipStream_t stream) {
  using C = Rows<BF16, D, KB, RT>;
  hipLaunchKernelGGL((k_weigh_rows<BF16, D, KB, RT>),
                     dim3(grid_for<C::kKeys>(a, kWeighWaves, C::kOcc)), dim3(kWeighThreads), 0,
                     stream, a);
}

template <bool BF16, int D, int KB, int RT>
void launch(const WeighArgs& a, hipStream_t stream) {
  constexpr bool kWide = KB > 1 && Rows<BF16, D, KB, RT>::kRow >= 256;
  if ((int64_t)a.N * a.G > kFewRows) {
    if constexpr (kWide)
      if ((int64_t)a.N * a.G <= kSomeRows) return launch_rows<BF16, D, 1, RT>(a, stream);
    return launch_rows<BF16, D, KB, RT>(a, stream);
  }
  using C = Few<BF16, D>;
  hipLaunchKernelGGL((k_weigh<BF16, D>), dim3(grid_for<C::kKeys>(a, 1, C::kOcc)),
                     dim3(kWeighThreads), 0, stream, a);
}

}  // namespace

hipError_t launch_cache_weigh(const WeighArgs& a, sv_dtype dt, hipStream_t stream) {
  if (dt == SV_DTYPE_BF16) {
    switch (a.c.head_dim) {
      case 64: launch<true, 64, 2, 64>(a, stream); break;
      case 96: launch<true, 96, 2, 64>(a, stream); break;
      case 128: launch<true, 128, 2, 64>(a, stream); break;
      default: launch<true, 256, 1, 64>(a, stream);
    }
  } else {
    switch (a.c.head_dim) {
      case 64: launch<false, 64, 1, 64>(a, stream); break;
      case 96: launch<false, 96, 1, 64>(a, stream); break;
      case 128: launch<false, 128, 1, 64>(a, stream); break;
      default: launch<false, 256, 1, 32>(a, stream);
    }
  }
  return hipGetLastError();
}

}  // namespace sv
