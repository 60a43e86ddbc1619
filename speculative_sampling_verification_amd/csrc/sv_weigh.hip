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

#include "sv_step.hpp"

namespace sv {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWeighThreads = 256;
constexpr int kWeighWaves = kWeighThreads / 64;
constexpr int kWeighWorkgroups = 4 * kAttnCus;
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

// Where piece `pos` lies: pieces of a sequence are ordered by key tile, then head.  Every thread of
// the workgroup gets the sequence and the piece in it.
template <int Keys>
__device__ __forceinline__ void find_piece(const WeighArgs& a, long long* total, int* b_out,
                                           long long* off_out) {
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
  const long long per = (all + gridDim.x - 1) / gridDim.x, pos = per * blockIdx.x;
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
  *total = all;
  *b_out = pos < all ? start_b : a.c.seqs;
  *off_out = pos < all ? start_off : 0;
}

// KT blocks of 16 keys a piece.
template <bool BF16, int D, int KT>
__global__ __launch_bounds__(kWeighThreads) void k_weigh(WeighArgs a) {
  constexpr int kES = BF16 ? 2 : 4, kRow = D * kES;
  constexpr int NF = kRow / 64;   // 16-byte pieces of a row that a lane holds
  constexpr int kKeys = 16 * KT;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const float sl2 = a.scale * kLog2e;
  long long total, off;
  int b;
  find_piece<kKeys>(a, &total, &b, &off);
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  long long pos = per * blockIdx.x + wave;
  const long long last = per * (blockIdx.x + 1), end = last < total ? last : total;
  off += wave;
  const int Hkv = a.c.kv_heads;
  for (; pos < end; pos += kWeighWaves, off += kWeighWaves) {
    for (; b < a.c.seqs; ++b) {
      const long long n = pieces_of<kKeys>(a, b);
      if (off < n) break;
      off -= n;
    }
    if (b >= a.c.seqs) break;
    const int tile = (int)(off >> 31 ? off / Hkv : (uint32_t)off / (uint32_t)Hkv);
    const int h = (int)(off - (long long)tile * Hkv);
    const int keys = keys_of(a, b), held = positions_held(a.c, b);
    const int32_t* table = a.c.table + (size_t)b * a.c.width;
    // this lane's keys
    u32x4 kf[KT][NF];
    int limit[KT];  // key number, out of every row's sight where it does not exist
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int key = tile * kKeys + t * 16 + col;
      int64_t row = 0;
      limit[t] = INT32_MAX;
      if (key < keys) {
        const uint32_t pi = fast_div(a.c.page_div, (uint32_t)key);
        const int page = table[pi];
        if (names_page(a.c, held, key, page)) {
          row = (int64_t)page * a.c.page_stride +
                (int64_t)(key - (int)(pi * a.c.page_div.d)) * a.c.token_stride;
          limit[t] = key;
        }
      }
      const char* p = a.c.k + row + (int64_t)h * a.c.head_stride + quad * 16;
#pragma unroll
      for (int s = 0; s < NF; ++s) kf[t][s] = *reinterpret_cast<const u32x4*>(p + s * 64);
    }
    float sum[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) sum[t] = 0.0f;
    int n = a.nodes ? a.nodes[b] : a.N;
    n = n < 0 ? 0 : n < a.N ? n : a.N;
    const int rows = n * a.G;
    for (int r0 = 0; r0 < rows; r0 += 16) {
      const int r = r0 + col;
      u32x4 qf[NF];
      {
        const int node = (int)fast_div(a.g_div, (uint32_t)r), g = r - node * a.G;
        const char* p = a.q.at + (int64_t)b * a.q.seq + (int64_t)node * a.q.node +
                        (int64_t)(h * a.G + g) * a.q.head + quad * 16;
#pragma unroll
        for (int s = 0; s < NF; ++s)
          qf[s] = r < rows ? *reinterpret_cast<const u32x4*>(p + s * 64) : u32x4{0, 0, 0, 0};
      }
      float lse2[4];
      int see[4];  // keys that the row sees
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int rr = r0 + quad * 4 + e;
        lse2[e] = 0.0f;
        see[e] = 0;
        if (rr < rows) {
          const int node = (int)fast_div(a.g_div, (uint32_t)rr), g = rr - node * a.G;
          const float x = a.lse[((int64_t)b * a.N + node) * ((int64_t)Hkv * a.G) + h * a.G + g];
          const int s = a.seen ? a.seen[(int64_t)b * a.N + node] : INT32_MAX;
          lse2[e] = x * kLog2e;
          see[e] = x == -INFINITY ? 0 : s < keys ? s : keys;
        }
      }
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < NF; ++s) {
          if constexpr (BF16) {
            z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, qf[s]),
                                                        __builtin_bit_cast(bf16x8, kf[t][s]), z, 0,
                                                        0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              z = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(qf[s][e]),
                                                       __uint_as_float(kf[t][s][e]), z, 0, 0, 0);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = __builtin_amdgcn_exp2f(fmaf(z[e], sl2, -lse2[e]));
          sum[t] += limit[t] < see[e] ? w : 0.0f;
        }
      }
    }
    // the four lanes of a key, then lane 16 t + c has key c of block t
    float mine = 0.0f;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      float x = sum[t];
      x += __shfl_xor(x, 16);
      x += __shfl_xor(x, 32);
      mine = quad == t ? x : mine;
    }
    const int key = tile * kKeys + lane;
    if (lane < kKeys && key < keys) {
      float* w = a.w + ((int64_t)b * Hkv + h) * a.length + key;
      *w = a.decay == 0.0f ? mine : fmaf(a.decay, *w, mine);
    }
  }
}

template <bool BF16, int D, int KT>
void launch(const WeighArgs& a, hipStream_t stream) {
  const int longest = a.c.cap < a.length ? a.c.cap : a.length;
  const int64_t pieces =
      (int64_t)a.c.seqs * a.c.kv_heads * ((longest + 16 * KT - 1) / (16 * KT));
  const int64_t groups = (pieces + kWeighWaves - 1) / kWeighWaves;
  const unsigned grid = (unsigned)(groups < kWeighWorkgroups ? groups : kWeighWorkgroups);
  hipLaunchKernelGGL((k_weigh<BF16, D, KT>), dim3(grid), dim3(kWeighThreads), 0, stream, a);
}

}  // namespace

hipError_t launch_cache_weigh(const WeighArgs& a, sv_dtype dt, hipStream_t stream) {
  // 64 registers of keys a lane
  if (dt == SV_DTYPE_BF16) {
    switch (a.c.head_dim) {
      case 64: launch<true, 64, 4>(a, stream); break;
      case 96: launch<true, 96, 4>(a, stream); break;
      case 128: launch<true, 128, 4>(a, stream); break;
      default: launch<true, 256, 2>(a, stream);
    }
  } else {
    switch (a.c.head_dim) {
      case 64: launch<false, 64, 4>(a, stream); break;
      case 96: launch<false, 96, 2>(a, stream); break;
      case 128: launch<false, 128, 2>(a, stream); break;
      default: launch<false, 256, 1>(a, stream);
    }
  }
  return hipGetLastError();
}

}  // namespace sv
