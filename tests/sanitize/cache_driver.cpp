// cache_driver.cpp -- drives the argument checks of rotary positions and the
// 4-bit cache (cache_api.hip) in a host build under AddressSanitizer and
// UndefinedBehaviorSanitizer.  The launches are stand-ins that only count, so
// calls that pass their checks can be made too: none may launch before an
// argument error, and the pointers, fake device addresses, may not be touched.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>
#include <vector>

#include "../../w8a8_rotated_int8_convrot_amd/csrc/api_checks.hpp"
#include "../../w8a8_rotated_int8_convrot_amd/csrc/convrot_internal.hpp"

static int g_launches = 0;
static int64_t g_tokens = 0;     // tokens a cache of the last launch may hold

extern "C" const char* convrot_last_error(void) { return convrot::g_last_error; }

namespace convrot {
int num_cus() { return 256; }
hipError_t launch_rope(const Rope& p, bool, hipStream_t) {
  ++g_launches;
  return p.M > 100 ? hipErrorInvalidConfiguration : hipSuccess;
}
hipError_t launch_cache_append(const Cache& c, const void*, int64_t, const void*, int64_t, bool, int64_t, const int32_t*,
                               const int32_t*, hipStream_t) {
  ++g_launches;
  g_tokens = c.max_tokens;
  return hipSuccess;
}
hipError_t launch_cache_read(const Cache& c, void*, int64_t, void*, int64_t, bool, int64_t, const int32_t*, const int32_t*,
                             hipStream_t) {
  ++g_launches;
  g_tokens = c.max_tokens;
  return hipSuccess;
}
hipError_t launch_cache_copy(uint8_t*, int64_t, int64_t, int64_t, const int32_t* src, const int32_t* dst, int64_t n, hipStream_t) {
  ++g_launches;
  g_tokens = 0;
  for (int64_t i = 0; i < n; ++i) g_tokens += src[i] + dst[i];
  return hipSuccess;
}
AttentionPlan plan_cache_attention(int64_t M, int64_t, int64_t, int, int64_t, int64_t, int64_t, bool) {
  AttentionPlan p{};
  p.splits = 1;
  p.workspace = static_cast<size_t>(M) * 16;
  return p;
}
hipError_t launch_cache_attention(const Attention& a, bool, hipStream_t) {
  ++g_launches;
  g_tokens = a.cache.max_tokens;
  return hipSuccess;
}
}  // namespace convrot

static int g_checks = 0, g_failed = 0;

static void expect(int got, int want, int launches, const char* what) {
  ++g_checks;
  if (got != want || g_launches != launches || (got != CONVROT_OK) != (std::strlen(convrot_last_error()) != 0)) {
    ++g_failed;
    std::printf("FAIL %s: status %d, expected %d, %d launches (%s)\n", what, got, want, g_launches,
                convrot_last_error());
  }
  g_launches = 0;
}

int main() {
  char* A = reinterpret_cast<char*>(uintptr_t(1) << 40);
  auto* i32 = reinterpret_cast<const int32_t*>(A);
  auto* f64 = reinterpret_cast<const double*>(A);
  constexpr int64_t kMin = std::numeric_limits<int64_t>::min(), kMax = std::numeric_limits<int64_t>::max();

  // frequencies: host memory of exactly the size they need
  for (int rot : {2, 64, 1024}) {
    std::vector<double> f(rot / 2);
    float s = 0.0f;
    for (int kind = CONVROT_ROPE_NONE; kind <= CONVROT_ROPE_BANDS; ++kind)
      expect(convrot_rope_frequencies(rot, 10000.0, kind, 8.0, 4096.0, 1.0, 32.0, f.data(), &s),
             rot == 2 && kind == CONVROT_ROPE_NTK ? CONVROT_EINVAL : CONVROT_OK, 0, "frequencies");
    expect(convrot_rope_frequencies(rot, 1.0000001, CONVROT_ROPE_YARN, 1e30, 1e-300, 1e-300, 1e300, f.data(), &s), CONVROT_OK, 0,
           "frequencies: extremes");
    expect(convrot_rope_frequencies(rot, 10000.0, -1, 8.0, 4096.0, 1.0, 32.0, f.data(), &s), CONVROT_EUNSUPPORTED, 0,
           "frequencies: kind");
  }

  auto rope = [&](int64_t hq, int64_t qs, int64_t hk, int64_t ks, int64_t M, int D, int rot, int layout) {
    return convrot_rope(A, hq, qs, A, qs, hk ? A + 4096 : nullptr, hk, ks, hk ? A + 4096 : nullptr, ks, CONVROT_BF16, M, D, rot,
                        layout, i32, f64, 1.0f, 0, nullptr);
  };
  expect(rope(8, 1024, 2, 256, 3, 128, 128, CONVROT_ROPE_HALF), CONVROT_OK, 1, "rope");
  expect(rope(8, 1024, 0, 0, 3, 128, 64, CONVROT_ROPE_INTERLEAVED), CONVROT_OK, 1, "rope: queries alone");
  expect(rope(8, 1024, 2, 256, 0, 128, 128, CONVROT_ROPE_HALF), CONVROT_OK, 0, "rope: no rows");
  expect(rope(8, 1024, 2, 256, 101, 128, 128, CONVROT_ROPE_HALF), CONVROT_EHIP, 1, "rope: failed launch");
  for (int64_t bad : {kMin, int64_t{-1}, kMax}) {
    expect(rope(bad, 1024, 2, 256, 3, 128, 128, CONVROT_ROPE_HALF), CONVROT_EINVAL, 0, "rope: heads");
    expect(rope(8, 1024, bad, 256, 3, 128, 128, CONVROT_ROPE_HALF), CONVROT_EINVAL, 0, "rope: key heads");
    expect(rope(8, bad, 2, 256, 3, 128, 128, CONVROT_ROPE_HALF), CONVROT_EINVAL, 0, "rope: stride");
    expect(rope(8, 1024, 2, 256, bad, 128, 128, CONVROT_ROPE_HALF), CONVROT_EINVAL, 0, "rope: M");
  }

  convrot_cache c{A, 5, 64, 128, 2, i32, 3, 2, 3, i32, i32};
  auto append = [&](int64_t ks, int64_t M) { return convrot_cache_append(&c, A, ks, A, 256, CONVROT_F16, M, nullptr); };
  auto read = [&](int64_t ks, int64_t M) { return convrot_cache_read(&c, A, ks, nullptr, 0, CONVROT_F16, M, nullptr); };
  auto attention = [&](int64_t hq, int64_t qs, int64_t M, int64_t window, size_t ws) {
    return convrot_cache_attention(&c, A, hq, qs, CONVROT_BF16, M, 0.1f, 1, window, A, A, ws, nullptr);
  };
  expect(append(256, 3), CONVROT_OK, 1, "append");
  expect(read(256, 3), CONVROT_OK, 1, "read");
  expect(attention(8, 1024, 3, 5, 48), CONVROT_OK, 1, "attention");
  expect(attention(8, 1024, 3, 5, 47), CONVROT_EWORKSPACE, 0, "attention: workspace");
  for (int64_t bad : {kMin, int64_t{-1}, kMax}) {
    expect(append(bad, 3), CONVROT_EINVAL, 0, "append: stride");
    expect(append(256, bad), CONVROT_EINVAL, 0, "append: M");
    expect(read(bad, 3), CONVROT_EINVAL, 0, "read: stride");
    expect(read(256, bad), CONVROT_EINVAL, 0, "read: M");
    expect(attention(bad, 1024, 3, 0, 48), CONVROT_EINVAL, 0, "attention: heads");
    expect(attention(8, bad, 3, 0, 48), CONVROT_EINVAL, 0, "attention: stride");
    expect(attention(8, 1024, bad, 0, 48), CONVROT_EINVAL, 0, "attention: M");
    expect(attention(8, 1024, 3, bad, 48), CONVROT_EINVAL, 0, "attention: window");
    for (int64_t* field : {&c.n_pages, &c.kv_heads, &c.table_stride, &c.n_seqs, &c.max_pages}) {
      const int64_t was = *field;
      *field = bad;
      expect(append(256, 3), CONVROT_EINVAL, 0, "append: a size of the cache");
      expect(attention(8, 1024, 3, 0, 48), CONVROT_EINVAL, 0, "attention: a size of the cache");
      *field = was;
    }
  }
  c.max_pages = c.table_stride = (int64_t{1} << 30) / 64;
  expect(append(256, 3), CONVROT_OK, 1, "append: the longest table");
  if (g_tokens != int64_t{1} << 30) ++g_failed;
  ++c.max_pages, ++c.table_stride;
  expect(append(256, 3), CONVROT_EINVAL, 0, "append: a longer one");
  for (int64_t bad : {kMin, int64_t{-1}, kMax}) {
    if (convrot_cache_attention_workspace(bad, 8, 2, 128, 2, 64) || convrot_cache_attention_workspace(1, bad, 2, 128, 2, 64) ||
        convrot_cache_attention_workspace(1, 8, bad, 128, 2, 64) || convrot_cache_attention_workspace(1, 8, 2, 128, bad, 64) ||
        convrot_cache_attention_workspace(1, 8, 2, 128, 2, bad) || convrot_cache_page_bytes(64, bad, 128))
      ++g_failed;
  }

  // the lists are host memory, of exactly their size
  std::vector<int32_t> src{0, 1, 2, 0}, dst{3, 4, 5, 6};
  auto copy = [&](int64_t layers, int64_t layer_bytes, int64_t n_pages, int64_t page_bytes, int64_t n) {
    return convrot_cache_copy(A, layers, layer_bytes, n_pages, page_bytes, src.data(), dst.data(), n, nullptr);
  };
  expect(copy(2, 7 * 64, 7, 64, 4), CONVROT_OK, 1, "copy");
  if (g_tokens != 21) ++g_failed;
  expect(copy(2, 7 * 64, 6, 64, 4), CONVROT_EINVAL, 0, "copy: a page past the last");
  expect(copy(2, 6 * 64, 7, 64, 4), CONVROT_EINVAL, 0, "copy: layers that overlap");
  expect(copy(1, 0, 7, 64, 0), CONVROT_OK, 0, "copy: none");
  for (int64_t bad : {kMin, int64_t{-1}, kMax}) {
    expect(copy(bad, 7 * 64, 7, 64, 4), CONVROT_EINVAL, 0, "copy: layers");
    expect(copy(2, bad, 7, 64, 4), CONVROT_EINVAL, 0, "copy: layer_bytes");
    expect(copy(2, 7 * 64, bad, 64, 4), CONVROT_EINVAL, 0, "copy: n_pages");
    expect(copy(2, 7 * 64, 7, bad, 4), CONVROT_EINVAL, 0, "copy: page_bytes");
    expect(copy(2, 7 * 64, 7, 64, bad), CONVROT_EINVAL, 0, "copy: n");
  }
  dst[3] = 3;
  expect(copy(1, 0, 7, 64, 4), CONVROT_EINVAL, 0, "copy: named twice");
  dst[3] = 1;
  expect(copy(1, 0, 7, 64, 4), CONVROT_EINVAL, 0, "copy: onto a source");

  std::printf("cache_driver: %d checks %s\n", g_checks, g_failed ? "FAILED" : "passed");
  return g_failed ? 1 : 0;
}
