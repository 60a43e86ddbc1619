// The argument checks of the entry points around tree attention, all the way to the launch, built
// with AddressSanitizer and UndefinedBehaviorSanitizer on the host code (tests/test_step_abi_reach.py
// builds and runs it).  What would launch kernels is replaced here, so that a call that is right returns
// SV_OK after every check and its arithmetic have run, and one that differs from it in a single argument
// shows which check refuses it.  No GPU; the addresses are never dereferenced.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <random>

#include "sv_logprob.hpp"
#include "sv_step.hpp"

namespace {

int failures = 0, checks = 0, launches = 0;
sv::RotaryArgs rotary_seen;

template <class T = void>
T* at(int i) {  // a TB apart
  return reinterpret_cast<T*>((uintptr_t)i << 40);
}

}  // namespace

namespace sv {
hipError_t launch_rotary(const RotaryArgs& a, sv_dtype, bool, bool, hipStream_t) {
  rotary_seen = a;
  ++launches;
  return hipSuccess;
}
hipError_t launch_cache_weigh(const WeighArgs&, sv_dtype, hipStream_t) {
  ++launches;
  return hipSuccess;
}
hipError_t launch_cache_evict(const EvictArgs&, hipStream_t) {
  ++launches;
  return hipSuccess;
}
hipError_t launch_logprobs(const LogprobArgs&, sv_dtype, hipStream_t) {
  ++launches;
  return hipSuccess;
}
LogprobPlan plan_logprobs(int R, int, sv_dtype, int n) {  // two parts a row
  return LogprobPlan{2, 1, (size_t)64 * R, (size_t)64 * R + (size_t)16 * R * n};
}
}  // namespace sv

// A call that has to return `want`, and to launch if that is SV_OK, and only then.
#define CALL(want, call)                                                                     \
  do {                                                                                       \
    const int before = launches, got = (call), wanted = (want);                              \
    ++checks;                                                                                \
    if (got != wanted || (launches > before) != (got == SV_OK)) {                            \
      std::printf("FAILED (line %d): %s returned %d, not %d\n", __LINE__, #call, got, wanted); \
      ++failures;                                                                            \
    }                                                                                        \
  } while (0)

#define EXPECT(cond)                                       \
  do {                                                     \
    ++checks;                                              \
    if (!(cond)) {                                         \
      std::printf("FAILED (line %d): %s\n", __LINE__, #cond); \
      ++failures;                                          \
    }                                                      \
  } while (0)

namespace {

constexpr int kBad = SV_ERR_INVALID_ARG;
const int kSizes[] = {INT_MIN, -1, 0, 1, 2, 3, 64, 2048, 2049, 1 << 20, 1 << 30, (1 << 30) + 1, INT_MAX};
const int64_t kStrides[] = {INT64_MIN, -8, 0, 1, 8, 64, 512, 1 << 20, (int64_t)1 << 59,
                            INT64_MAX / 8 - 7, INT64_MAX / 8, INT64_MAX / 4, INT64_MAX};

// ------------------------------------------------------------------------------------ rotary
struct Rotary {
  const void* q = at(60);  // above all else: how far its strides reach is a matter of overflow alone
  const int64_t* qs = nullptr;
  int hq = 4;
  void* oq = at(11);
  const void* k = at(12);
  const int64_t* ks = nullptr;
  int hk = 2;
  void* ok = at(13);
  int seqs = 3, N = 5, D = 64;
  const int32_t *base = at<int32_t>(15), *positions = at<int32_t>(16);
  const double* freq = at<double>(14);
  int call() const {
    return spec_rotary(q, qs, hq, oq, k, ks, hk, ok, SV_DTYPE_BF16, seqs, N, D, freq, D, 0, 1.0f, base,
                       positions, nullptr);
  }
};

// What rows at these strides (elements of two bytes) span; -1 if 64 bits do not hold it, or a stride
// is none that is taken.
__int128 span(const int64_t (&s)[3], const int (&size)[3], int D) {
  __int128 bytes = 2 * D;
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0 || s[i] > INT64_MAX / 8 || s[i] % 8 != 0) return -1;
    bytes += (__int128)s[i] * 2 * (size[i] - 1);
  }
  return bytes <= INT64_MAX ? bytes : -1;
}

void rotary_strides() {
  const Rotary good;
  CALL(SV_OK, good.call());
  for (int64_t s0 : kStrides)
    for (int64_t s1 : kStrides)
      for (int64_t s2 : kStrides)
        for (int seqs : {1, 2, 1 << 20}) {
          const int64_t s[3] = {s0, s1, s2};
          const int size[3] = {seqs, 5, 4};
          Rotary r;
          r.qs = s;
          r.seqs = seqs;
          CALL(span(s, size, r.D) >= 0 ? SV_OK : kBad, r.call());
          if (span(s, size, r.D) >= 0)
            EXPECT(rotary_seen.q.seq == 2 * s0 && rotary_seen.q.node == 2 * s1 &&
                   rotary_seen.q.head == 2 * s2);
          r.positions = reinterpret_cast<int32_t*>(r.oq);  // the very last check
          CALL(kBad, r.call());
        }
}

void rotary_sizes() {
  for (int x : kSizes)
    for (int y : kSizes) {
      Rotary r;
      r.seqs = x;
      r.N = y;
      CALL(x > 0 && y > 0 && (int64_t)x * y <= INT_MAX ? SV_OK : kBad, r.call());
      Rotary h;
      h.hq = x;
      h.hk = y;
      const bool fine = x > 0 && y > 0 && x <= 65536 && y <= 65536;  // both are given
      CALL(fine ? SV_OK : kBad, h.call());
    }
}

// Arrays of `bytes` each, one written and the others not: refused as soon as any byte is shared.
void rotary_overlaps() {
  const int64_t out = 3 * 5 * 4 * 128, keys = 3 * 5 * 2 * 128;
  for (int64_t d : {-out - 16, -out, -out + 16, (int64_t)-16, (int64_t)0, (int64_t)16, out - 16, out,
                    out + 16}) {
    Rotary r;
    char* const oq = static_cast<char*>(r.oq);
    r.ok = oq + d;  // written both
    CALL(d <= -keys || d >= out ? SV_OK : kBad, r.call());
    r = Rotary();
    r.q = oq + d;  // dense: d = 0 is in place
    CALL(d == 0 || d <= -out || d >= out ? SV_OK : kBad, r.call());
    r = Rotary();
    r.k = oq + d;
    CALL(d <= -keys || d >= out ? SV_OK : kBad, r.call());
    r = Rotary();
    r.freq = reinterpret_cast<const double*>(oq + d);
    CALL(d <= -32 * 8 || d >= out ? SV_OK : kBad, r.call());
    r = Rotary();
    r.base = reinterpret_cast<const int32_t*>(oq + d);
    CALL(d <= -3 * 4 || d >= out ? SV_OK : kBad, r.call());
  }
}

// Queries and keys turned in place, at random strides and offsets in one small buffer: where the call is
// taken, no byte belongs to two rows.
void rotary_in_place() {
  std::mt19937 rng(1);
  auto pick = [&](int n) { return (int)(rng() % n); };
  int taken = 0;
  static int owner[1 << 14];
  for (int round = 0; round < 200000; ++round) {
    Rotary r;
    r.seqs = 1 + pick(3);
    r.N = 1 + pick(3);
    r.hq = 1 + pick(3);
    r.hk = 1 + pick(2);
    r.D = 8 * (1 + pick(2));
    int64_t qs[3], ks[3];
    for (int i = 0; i < 3; ++i) {
      qs[i] = 8 * pick(20);
      ks[i] = pick(4) ? qs[i] : 8 * pick(20);
    }
    r.qs = qs;
    r.ks = ks;
    char* const buffer = at<char>(30);
    const int q0 = 16 * pick(30), k0 = 16 * pick(30);
    r.q = r.oq = buffer + q0;
    r.k = r.ok = buffer + k0;
    const int st = r.call();
    if (st != SV_OK) continue;
    ++taken;
    for (int& o : owner) o = 0;
    int row = 0;
    bool shared = false;
    auto lay = [&](int from, const int64_t* s, int heads) {
      for (int b = 0; b < r.seqs; ++b)
        for (int i = 0; i < r.N; ++i)
          for (int h = 0; h < heads; ++h) {
            const int64_t first = from + 2 * (b * s[0] + i * s[1] + h * s[2]);
            ++row;
            for (int e = 0; e < 2 * r.D; ++e) {
              shared |= owner[first + e] != 0;
              owner[first + e] = row;
            }
          }
    };
    lay(q0, qs, r.hq);
    lay(k0, ks, r.hk);
    EXPECT(!shared);
  }
  EXPECT(taken > 1000);
}

// ------------------------------------------------------------------------------------- caches
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

int append(const sv_cache& c, int N, const void* k_new = at(12), const int32_t* positions = nullptr,
           const int64_t* s = nullptr) {
  return spec_rotary_append(at(10), nullptr, 4, at(11), k_new, at(60), s, N, &c, 1, nullptr,
                            at<double>(14), 64, 0, 1.0f, nullptr, positions, nullptr);
}

int weigh(const sv_cache& c, const int64_t* s, int N, int heads, int length,
          const int32_t* seen = nullptr, float* w = at<float>(20)) {
  return spec_cache_weigh(at(60), s, N, heads, at<float>(14), &c, 1, seen, nullptr, 0.1f, 1.0f, w, length,
                          nullptr);
}

int evict(const sv_cache& c, int length, int max_keep, int sinks, int recent,
          const int32_t* keep = at<int32_t>(16), float* out = at<float>(40),
          int32_t* kept = at<int32_t>(50)) {
  return spec_cache_evict(&c, at<float>(20), length, keep, max_keep, sinks, recent, out, at<int32_t>(18),
                          kept, nullptr);
}

void cache_calls() {
  const sv_cache good = cache();
  CALL(SV_OK, append(good, 5));
  CALL(SV_OK, weigh(good, nullptr, 5, 4, 70));
  CALL(SV_OK, evict(good, 70, 40, 1, 1));
  for (int x : kSizes) {
    CALL(x >= 1 && x <= 2048 ? SV_OK : kBad, append(good, x));
    CALL(x >= 1 && x <= 2048 ? SV_OK : kBad, weigh(good, nullptr, x, 4, 70));
    CALL(x >= 2 && x <= 65536 && x % 2 == 0 ? SV_OK : kBad, weigh(good, nullptr, 5, x, 70));
    CALL(x >= 1 && x <= 1 << 30 ? SV_OK : kBad, weigh(good, nullptr, 5, 4, x));
    for (int y : kSizes) {
      CALL(x >= 1 && x <= 1 << 30 && y >= 1 && y <= x ? SV_OK : kBad, evict(good, x, y, 1, 1));
      CALL(x >= 0 && y >= 0 ? SV_OK : kBad, evict(good, 70, 40, x, y));
    }
    // a field of the cache at its limits: refused or taken, without an overflow on the way
    for (int field = 0; field < 7; ++field)
      for (int64_t stride : {(int64_t)0, (int64_t)1 << 20, INT64_MAX / 8 - 7, INT64_MAX / 4}) {
        sv_cache c = good;
        int32_t* const f[] = {&c.layers, &c.pages, &c.page_size, &c.kv_heads, &c.head_dim, &c.seqs,
                              &c.table_width};
        *f[field] = x;
        if (stride) c.layer_stride = stride;
        const int taken[] = {append(c, 2048), weigh(c, nullptr, 2048, 4, 1 << 30),
                             evict(c, 1 << 30, 1 << 30, 0, 0)};
        for (int st : taken) EXPECT(st == SV_OK || st == kBad);
      }
  }
  for (int64_t s0 : kStrides)
    for (int64_t s1 : kStrides) {
      const int64_t s[3] = {s0, s1, 64};
      const int size[3] = {3, 5, 4};
      CALL(span(s, size, 64) >= 0 ? SV_OK : kBad, weigh(good, s, 5, 4, 70));
    }
  // what is written against what is read, to the byte: the second layer's 6 * 70 weights
  float* const w = at<float>(20);
  const int64_t layer = 3 * 2 * 70, seen = 3 * 5;
  for (int64_t d : {layer - seen, layer - seen + 1, layer, 2 * layer - 1, 2 * layer})
    CALL(d <= layer - seen || d >= 2 * layer ? SV_OK : kBad,
         weigh(good, nullptr, 5, 4, 70, reinterpret_cast<int32_t*>(w + d)));
  char* const page = static_cast<char*>(good.k) + 160 * 256;  // of the calls' layer
  float* const end = reinterpret_cast<float*>(page + 160 * 256);
  CALL(kBad, weigh(good, nullptr, 5, 4, 70, nullptr, end - layer - 1));
  CALL(SV_OK, weigh(good, nullptr, 5, 4, 70, nullptr, end - layer));
  const int64_t kept = 2 * 3 * 2 * 40, all = 2 * 3 * 2 * 70;
  for (int64_t d : {(int64_t)-3, (int64_t)-2, (int64_t)0, kept - 1, kept})
    CALL(d <= -3 || d >= kept ? SV_OK : kBad, evict(good, 70, 40, 1, 1, at<int32_t>(50) + d));
  for (int64_t d : {-all, -all + 1, (int64_t)0, all - 1, all})
    CALL(d == 0 || d <= -all || d >= all ? SV_OK : kBad,
         evict(good, 70, 40, 1, 1, at<int32_t>(16), w + d));
  // 2^36 heads in all
  sv_cache most = good;
  most.layers = most.seqs = 8192;
  most.kv_heads = 1024;
  most.token_stride = 64 * 1024;
  most.page_stride = 16 * most.token_stride;
  most.layer_stride = 10 * most.page_stride;
  CALL(SV_OK, evict(most, 2, 2, 0, 0));
  CALL(kBad, evict(most, 2, 2, 0, 0, at<int32_t>(50) + ((int64_t)1 << 37) - 1));
  // keys that end where the values begin, and one row further
  const int64_t rows = (int64_t)2 * 160 * 2;
  for (int64_t d : {rows - 1, rows}) {
    sv_cache c = good;
    c.v = static_cast<char*>(c.k) + d * 128;
    CALL(d == rows ? SV_OK : kBad, append(c, 5));
    CALL(d == rows ? SV_OK : kBad, evict(c, 70, 40, 1, 1));
  }
  // new keys in the cache's pages of the call's layer, and behind them
  CALL(kBad, append(good, 5, page + 160 * 256 - 16));
  CALL(SV_OK, append(good, 5, page + 160 * 256));
  CALL(kBad, append(good, 5, at(12), at<int32_t>(11)));
}

// ------------------------------------------------------------------------ log probabilities
int logprobs(int num_rows, int V, int R, const int32_t* rows, int n, const int32_t* tokens = at<int32_t>(12),
             int32_t* top = at<int32_t>(40)) {
  return spec_token_logprobs(at(60), SV_DTYPE_F32, num_rows, V, rows, tokens, R, 1.0f, n, at<float>(13),
                             at<int32_t>(14), at<float>(15), n > 0 ? top : nullptr,
                             n > 0 ? at<float>(16) : nullptr, at(50), SIZE_MAX, nullptr);
}

void logprob_calls() {
  for (int x : kSizes)
    for (int y : kSizes)
      for (int n : {-1, 0, 1, 64, 65}) {
        const bool fine = x > 0 && y > 0 && n >= 0 && n <= 64;
        CALL(fine && (__int128)x * y <= (__int128)1 << 60 ? SV_OK : kBad, logprobs(x, y, x, nullptr, n));
        CALL(fine ? SV_OK : kBad, logprobs(1, x, y, at<int32_t>(17), n));
      }
  const int64_t top = 7 * 5;
  for (int64_t d : {(int64_t)-7, (int64_t)-6, (int64_t)0, top - 1, top})
    CALL(d <= -7 || d >= top ? SV_OK : kBad, logprobs(7, 100, 7, nullptr, 5, at<int32_t>(40) + d));
}

}  // namespace

int main() {
  rotary_strides();
  rotary_sizes();
  rotary_overlaps();
  rotary_in_place();
  cache_calls();
  logprob_calls();
  std::printf("%d checks, %d failures\n", checks, failures);
  return failures != 0;
}
