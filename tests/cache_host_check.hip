// Host-side checks of the paged-cache entry points, built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code (tests/test_cache_abi_sanitized.py builds and runs
// it): cache descriptions, strides and sizes up to their limits, attention workspaces over every
// shape class, and the refusals that come before any launch.  Every call here returns before any
// HIP runtime call, so the program needs no GPU; the addresses it passes are never dereferenced.
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

void* const kDev = reinterpret_cast<void*>(uintptr_t{1} << 20);
void* const kDev2 = reinterpret_cast<void*>(uintptr_t{1} << 30);
int32_t* const kInt = static_cast<int32_t*>(kDev);
int32_t* const kInt2 = static_cast<int32_t*>(kDev2);

sv_cache cache(sv_dtype dt, int layers, int pages, int page, int heads, int dim, int seqs,
               int width) {
  sv_cache c{};
  c.k = kDev;
  c.v = kDev2;
  c.dtype = dt;
  c.layers = layers;
  c.pages = pages;
  c.page_size = page;
  c.kv_heads = heads;
  c.head_dim = dim;
  c.head_stride = dim;
  c.token_stride = (int64_t)heads * dim;
  c.page_stride = c.token_stride * page;
  c.layer_stride = c.page_stride * pages;
  c.seqs = seqs;
  c.table_width = width;
  c.page_table = c.seq_lens = c.seq_pages = c.refcount = kInt;
  return c;
}

int attend(const sv_cache* c, int N, int heads, size_t bytes, const int64_t* strides = nullptr,
           float scale = 1.0f) {
  return spec_tree_attention(kDev, strides, N, heads, c, 0, nullptr, nullptr, scale, kDev, nullptr,
                             kDev, bytes, nullptr);
}

// Workspace sizes over shapes: given for each that is taken, and one byte less is refused.
void workspaces() {
  for (sv_dtype dt : {SV_DTYPE_F32, SV_DTYPE_BF16})
    for (int dim : {64, 96, 128, 256})
      for (int seqs : {1, 3, 256, 8192})
        for (int heads : {1, 8, 1024})
          for (int group : {1, 5, 64})
            for (int N : {1, 2, 17, 512, 2048}) {
              const sv_cache c = cache(dt, 2, 1 << 20, 16, heads, dim, seqs, 1 << 12);
              const size_t n = spec_tree_attention_workspace_size(&c, N, heads * group);
              EXPECT(n > 0);
              EXPECT(attend(&c, N, heads * group, n - 1) == SV_ERR_WORKSPACE_TOO_SMALL);
              if (heads > 1) EXPECT(attend(&c, N, heads * group + 1, n) == SV_ERR_INVALID_ARG);
            }
}

// Sizes and strides at and beyond their limits, each of which must be refused or taken without
// an overflow on the way.
void extents() {
  const int sizes[] = {INT_MIN, -1, 0, 1, 2, 1 << 20, INT_MAX};
  const int64_t strides[] = {INT64_MIN, -1, 0, 1, 8, 64, 1 << 20, INT64_MAX / 8, INT64_MAX / 4,
                             INT64_MAX - 7, INT64_MAX};
  const sv_cache ok = cache(SV_DTYPE_BF16, 2, 10, 16, 2, 64, 3, 5);
  EXPECT(attend(&ok, 4, 4, 0) == SV_ERR_WORKSPACE_TOO_SMALL);
  for (int s : sizes) {
    for (int field = 0; field < 7; ++field) {
      sv_cache c = ok;
      int32_t* const f[] = {&c.layers, &c.pages, &c.page_size, &c.kv_heads, &c.head_dim, &c.seqs,
                            &c.table_width};
      *f[field] = s;
      const int st = attend(&c, 4, 4, 0);
      EXPECT(st == SV_ERR_INVALID_ARG || st == SV_ERR_WORKSPACE_TOO_SMALL);
      if (s <= 0) EXPECT(st == SV_ERR_INVALID_ARG);
    }
    EXPECT(attend(&ok, s, 4, 0) == (s == 1 || s == 2 ? SV_ERR_WORKSPACE_TOO_SMALL : SV_ERR_INVALID_ARG));
    const int heads = attend(&ok, 4, s, 0);
    EXPECT(s > 0 || heads == SV_ERR_INVALID_ARG);
  }
  for (int64_t s : strides) {
    for (int field = 0; field < 4; ++field) {
      sv_cache c = ok;
      int64_t* const f[] = {&c.layer_stride, &c.page_stride, &c.token_stride, &c.head_stride};
      *f[field] = s;
      const int st = attend(&c, 4, 4, 0);
      EXPECT(st == SV_ERR_INVALID_ARG || st == SV_ERR_WORKSPACE_TOO_SMALL);
      if (s <= 1) EXPECT(st == SV_ERR_INVALID_ARG);
    }
    for (int i = 0; i < 3; ++i) {
      int64_t q[3] = {4 * 256, 256, 64};
      q[i] = s;
      const int st = attend(&ok, 4, 4, 0, q);
      const bool fine = s >= 0 && s <= INT64_MAX / 8 && s % 8 == 0;
      EXPECT(st == (fine ? SV_ERR_WORKSPACE_TOO_SMALL : SV_ERR_INVALID_ARG));
    }
  }
}

void refusals() {
  const sv_cache ok = cache(SV_DTYPE_F32, 2, 10, 16, 2, 64, 3, 5);
  for (float scale : {0.0f, -1.0f, INFINITY, -INFINITY, NAN})
    EXPECT(attend(&ok, 4, 4, SIZE_MAX, nullptr, scale) == SV_ERR_INVALID_ARG);
  EXPECT(attend(nullptr, 4, 4, SIZE_MAX) == SV_ERR_INVALID_ARG);
  EXPECT(spec_tree_attention_workspace_size(nullptr, 4, 4) == 0);
  EXPECT(spec_cache_append(nullptr, kDev, nullptr, 4, &ok, 0, nullptr, nullptr) == SV_ERR_INVALID_ARG);
  for (int N : {INT_MIN, 0, 2049, INT_MAX}) {
    EXPECT(spec_cache_append(kDev, kDev, nullptr, N, &ok, 0, nullptr, nullptr) == SV_ERR_INVALID_ARG);
    EXPECT(spec_cache_commit(&ok, kInt, kInt, N, kInt2, nullptr) == SV_ERR_INVALID_ARG);
  }
  for (int layer : {INT_MIN, -1, 2, INT_MAX})
    EXPECT(spec_cache_append(kDev, kDev, nullptr, 4, &ok, layer, nullptr, nullptr) == SV_ERR_INVALID_ARG);
  for (int off : {-2, -1, 0, 1, 2})
    EXPECT(spec_cache_commit(&ok, kInt, kInt, 4, kInt + off, nullptr) == SV_ERR_INVALID_ARG);
  EXPECT(spec_cache_resize(&ok, nullptr, nullptr, kInt2, nullptr) == SV_ERR_INVALID_ARG);
  EXPECT(spec_cache_resize(nullptr, kInt2, nullptr, kInt2, nullptr) == SV_ERR_INVALID_ARG);
  for (int F : {INT_MIN, -1, 4, INT_MAX})
    EXPECT(spec_cache_fork(&ok, kInt, kInt, F, kInt2, nullptr) == SV_ERR_INVALID_ARG);
  EXPECT(spec_cache_fork(&ok, nullptr, nullptr, 0, nullptr, nullptr) == SV_OK);
}

}  // namespace

int main() {
  workspaces();
  extents();
  refusals();
  std::printf("%d checks, %d failures\n", g_checks, g_failures);
  return g_failures != 0;
}
