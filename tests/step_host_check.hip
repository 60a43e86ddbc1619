// Host-side checks of the entry points around tree attention, built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code (tests/test_step_abi_sanitized.py builds and runs it):
// sizes, strides and addresses up to their limits.  Every call here returns before any HIP runtime
// call, so the program needs no GPU; the addresses it passes are never dereferenced.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "spec_verify.h"

static int g_failures = 0;
static int g_checks = 0;

#define EXPECT(cond)                                                   \
  do {                                                                 \
    ++g_checks;                                                        \
    if (!(cond)) {                                                     \
      std::printf("FAILED (line %d): %s\n", __LINE__, #cond);         \
      ++g_failures;                                                    \
    }                                                                  \
  } while (0)

namespace {

template <class T = void>
T* at(int i) {
  return reinterpret_cast<T*>((uintptr_t)i << 32);
}

sv_cache cache() {
  sv_cache c{};
  c.k = at(1);
  c.v = at(2);
  c.dtype = SV_DTYPE_BF16;
  c.layers = 2;
  c.pages = 10;
  c.page_size = 16;
  c.kv_heads = 2;
  c.head_dim = 64;
  c.head_stride = 64;
  c.token_stride = 128;
  c.page_stride = 16 * 128;
  c.layer_stride = 160 * 128;
  c.seqs = 3;
  c.table_width = 5;
  c.page_table = at<int32_t>(3);
  c.seq_lens = at<int32_t>(4);
  c.seq_pages = at<int32_t>(5);
  c.refcount = at<int32_t>(6);
  return c;
}

// A call that is right but for what is asked of it ends with the last check: an odd address of
// inv_freq, lse or the workspace.  So each case has to be refused, without an overflow on the way.
int rotary(const int64_t* qs, const int64_t* ks, int hq, int hk, int seqs, int N, int D, int rot,
           void* oq = at(11), void* ok = at(13)) {
  return spec_rotary(at(10), qs, hq, oq, at(12), ks, hk, ok, SV_DTYPE_BF16, seqs, N, D,
                     reinterpret_cast<double*>((uintptr_t)14 << 32 | 4), rot, 0, 1.0f, nullptr,
                     nullptr, nullptr);
}

int weigh(const sv_cache* c, const int64_t* qs, int N, int heads, float scale, float decay,
          int length) {
  return spec_cache_weigh(at(10), qs, N, heads,
                          reinterpret_cast<float*>((uintptr_t)14 << 32 | 2), c, 1, nullptr, nullptr,
                          scale, decay, at<float>(15), length, nullptr);
}

int evict(const sv_cache* c, int length, int max_keep, int sinks, int recent) {
  return spec_cache_evict(c, at<float>(15), length,
                          reinterpret_cast<int32_t*>((uintptr_t)16 << 32 | 2), max_keep, sinks,
                          recent, at<float>(17), at<int32_t>(18), at<int32_t>(19), nullptr);
}

const int kSizes[] = {INT_MIN, -1, 0, 1, 2, 64, 1 << 20, INT_MAX};
const int64_t kStrides[] = {INT64_MIN, -1,           0,           1, 8, 64, 1 << 20, INT64_MAX / 8,
                            INT64_MAX / 8 - 7, INT64_MAX / 4, INT64_MAX - 7, INT64_MAX};

void rotary_limits() {
  EXPECT(rotary(nullptr, nullptr, 4, 2, 3, 5, 64, 64) == SV_ERR_INVALID_ARG);
  for (int x : kSizes)
    for (int y : kSizes) {
      EXPECT(rotary(nullptr, nullptr, x, y, 3, 5, 64, 64) == SV_ERR_INVALID_ARG);
      EXPECT(rotary(nullptr, nullptr, 4, 2, x, y, 64, 64) == SV_ERR_INVALID_ARG);
      EXPECT(rotary(nullptr, nullptr, 4, 2, 3, 5, x, y) == SV_ERR_INVALID_ARG);
    }
  for (int64_t s : kStrides)
    for (int i = 0; i < 3; ++i) {
      int64_t q[3] = {5 * 512, 512, 64}, k[3] = {5 * 512, 512, 64};
      q[i] = s;
      EXPECT(rotary(q, k, 4, 2, 3, 5, 64, 64) == SV_ERR_INVALID_ARG);
      EXPECT(rotary(k, q, 4, 2, 3, 5, 64, 64) == SV_ERR_INVALID_ARG);
      EXPECT(rotary(q, q, 4, 2, 3, 5, 64, 64, at(10), at(12)) == SV_ERR_INVALID_ARG);
    }
  for (int x : kSizes) {
    const sv_cache c = cache();
    EXPECT(spec_rotary_append(at(10), nullptr, x, at(11), at(12), at(13), nullptr, 4, &c, 1, nullptr,
                              reinterpret_cast<double*>((uintptr_t)14 << 32 | 4), 64, 0, 1.0f,
                              nullptr, nullptr, nullptr) == SV_ERR_INVALID_ARG);
    EXPECT(spec_rotary_append(at(10), nullptr, 4, at(11), at(12), at(13), nullptr, x, &c, 1, nullptr,
                              reinterpret_cast<double*>((uintptr_t)14 << 32 | 4), 64, 0, 1.0f,
                              nullptr, nullptr, nullptr) == SV_ERR_INVALID_ARG);
  }
  double freq[2048];
  float s;
  for (int rot : kSizes)
    for (int how = -1; how < 5; ++how)
      for (double theta : {0.0, 1e-300, 1.0, 1e4, 1e300, (double)INFINITY, (double)NAN})
        for (double factor : {0.0, 1.0, 8.0, 1e300, (double)NAN}) {
          const int st = spec_rotary_frequencies(rot, theta, how, factor, 4096.0, 32.0, 1.0, freq, &s);
          const bool fine = (rot == 2 || rot == 64) && how >= 0 && how <= 3 && theta > 0 &&
                            std::isfinite(theta) && (how == 0 || factor >= 1.0);
          EXPECT(st == (fine ? SV_OK : SV_ERR_INVALID_ARG));
        }
}

void eviction_limits() {
  const sv_cache ok = cache();
  for (int x : kSizes) {
    EXPECT(weigh(&ok, nullptr, x, 4, 0.1f, 1.0f, 70) == SV_ERR_INVALID_ARG);
    EXPECT(weigh(&ok, nullptr, 4, x, 0.1f, 1.0f, 70) == SV_ERR_INVALID_ARG);
    EXPECT(weigh(&ok, nullptr, 4, 4, 0.1f, 1.0f, x) == SV_ERR_INVALID_ARG);
    for (int y : kSizes) {
      EXPECT(evict(&ok, x, y, 1, 1) == SV_ERR_INVALID_ARG);
      EXPECT(evict(&ok, 70, 40, x, y) == SV_ERR_INVALID_ARG);
    }
    for (int field = 0; field < 7; ++field) {
      sv_cache c = ok;
      int32_t* const f[] = {&c.layers, &c.pages, &c.page_size, &c.kv_heads, &c.head_dim, &c.seqs,
                            &c.table_width};
      *f[field] = x;
      EXPECT(weigh(&c, nullptr, 4, 4, 0.1f, 1.0f, 70) == SV_ERR_INVALID_ARG);
      EXPECT(evict(&c, 1 << 30, 1, 0, 0) == SV_ERR_INVALID_ARG);
    }
  }
  for (float f : {0.0f, -1.0f, INFINITY, -INFINITY, NAN, 1e-45f, 3e38f})
    for (float g : {0.0f, -1.0f, 2.0f, INFINITY, NAN, 0.5f})
      EXPECT(weigh(&ok, nullptr, 4, 4, f, g, 70) == SV_ERR_INVALID_ARG);
  for (int64_t s : kStrides)
    for (int i = 0; i < 3; ++i) {
      int64_t q[3] = {4 * 256, 256, 64};
      q[i] = s;
      EXPECT(weigh(&ok, q, 4, 4, 0.1f, 1.0f, 70) == SV_ERR_INVALID_ARG);
    }
}

int logprobs(int num_rows, int V, int R, const int32_t* rows, float T, int n, size_t bytes) {
  return spec_token_logprobs(at(10), SV_DTYPE_F32, num_rows, V, rows, at<int32_t>(12), R, T, n,
                             at<float>(13), nullptr, nullptr, n > 0 ? at<int32_t>(14) : nullptr,
                             n > 0 ? at<float>(15) : nullptr, at(16), bytes, nullptr);
}

void logprob_limits() {
  for (int x : kSizes)
    for (int y : kSizes) {
      for (int n : {INT_MIN, -1, 0, 1, 64, 65, INT_MAX})
        for (sv_dtype dt : {-1, 0, 1, 2}) {
          const size_t need = spec_token_logprobs_workspace_size(x, y, dt, n);
          EXPECT((need != 0) == (x > 0 && y > 0 && n >= 0 && n <= 64 && (dt == 0 || dt == 1)));
        }
      // rows of many parts need a workspace: refused for want of it
      const int st = logprobs(1, 1 << 24, 1, nullptr, 1.0f, 4, 0);
      EXPECT(st == SV_ERR_WORKSPACE_TOO_SMALL);
      if (x <= 0 || y <= 0) EXPECT(logprobs(x, y, x, nullptr, 1.0f, 4, SIZE_MAX) == SV_ERR_INVALID_ARG);
    }
  EXPECT(logprobs(INT_MAX, INT_MAX, 1, at<int32_t>(17), 1.0f, 4, SIZE_MAX) == SV_ERR_INVALID_ARG);
  for (float T : {0.0f, -0.0f, -1.0f, INFINITY, NAN, 1e-45f})
    EXPECT(logprobs(1, 1 << 24, 1, nullptr, T, 4, 0) == SV_ERR_INVALID_ARG);
}

}  // namespace

int main() {
  rotary_limits();
  eviction_limits();
  logprob_limits();
  std::printf("%d checks, %d failures\n", g_checks, g_failures);
  return g_failures != 0;
}
