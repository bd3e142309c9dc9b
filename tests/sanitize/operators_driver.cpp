// operators_driver.cpp -- drives the argument checks of the operators around
// the layer (operators_api.hip) in a host build under AddressSanitizer and
// UndefinedBehaviorSanitizer.  The launches are stand-ins that only count, so
// calls that pass their checks can be made too: none may launch before an
// argument error, and the pointers, fake device addresses, may not be touched.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>

#include "../../w8a8_rotated_int8_convrot_amd/csrc/api_checks.hpp"
#include "../../w8a8_rotated_int8_convrot_amd/csrc/convrot_internal.hpp"

static int g_launches = 0;
static int64_t g_rows = 0;       // tokens the launches were asked for

extern "C" const char* convrot_last_error(void) { return convrot::g_last_error; }

namespace convrot {
int num_cus() { return 256; }
hipError_t launch_block_norm(const BlockNorm& p, int, bool, hipStream_t) {
  g_rows += p.M;
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_rotate_quant(const uint16_t*, int64_t, int64_t, int, int8_t*, float*, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_rotate_quant_f16(const uint16_t*, int64_t, int64_t, int, int8_t*, float*, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_gemm_grouped(const int8_t*, const float*, int64_t, const int8_t*, const float*, bool, const uint16_t*,
                               uint16_t*, bool, const int32_t*, const int32_t*, int64_t, int64_t, int64_t, int64_t,
                               hipStream_t) {
  ++g_launches;
  return hipErrorInvalidConfiguration;      // a failed launch
}
bool grouped_is_few(int64_t M, int64_t) { return M <= 2; }
hipError_t launch_grouped_few(const void*, int64_t, int64_t, int, bool, const int8_t*, const float*, bool,
                              const uint16_t*, uint16_t*, const int32_t*, const int32_t*, int64_t, int64_t, int64_t,
                              hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_lora_down(const uint16_t*, int64_t M, int64_t, int, bool, int8_t*, float*, const uint16_t*, int64_t,
                            const float*, const int32_t*, int64_t, const int32_t*, int64_t, uint16_t*, int64_t, float*,
                            hipStream_t) {
  g_rows += M;
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_gemm_lora(const int8_t*, const float*, const int8_t*, const float*, bool, const uint16_t*, uint16_t*,
                            bool, int64_t, int64_t, int64_t, const uint16_t*, int64_t, const uint16_t*, int64_t,
                            const int32_t*, int64_t, const int32_t*, int64_t, hipStream_t) {
  ++g_launches;
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
  auto* f32 = reinterpret_cast<const float*>(A);
  auto* i8 = reinterpret_cast<const int8_t*>(A);

  convrot_block b{};
  expect(convrot_block_norm(nullptr, nullptr), CONVROT_EINVAL, 0, "block: NULL");
  expect(convrot_block_norm(&b, nullptr), CONVROT_EUNSUPPORTED, 0, "block: all zero");
  b.io_dtype = CONVROT_F16;
  b.residual_scale = 1.0f;
  b.K = 512;
  expect(convrot_block_norm(&b, nullptr), CONVROT_OK, 0, "block: no tokens");
  b.M = 5;
  expect(convrot_block_norm(&b, nullptr), CONVROT_EINVAL, 0, "block: no stream");
  b.h = A;
  expect(convrot_block_norm(&b, nullptr), CONVROT_EINVAL, 0, "block: nothing to do");
  b.out = A + 4096;
  expect(convrot_block_norm(&b, nullptr), CONVROT_OK, 1, "block: norm alone");
  b.group = 256;
  expect(convrot_block_norm(&b, nullptr), CONVROT_EINVAL, 0, "block: codes without scales");
  b.group = 0;
  b.u = A + 8192;
  expect(convrot_block_norm(&b, nullptr), CONVROT_EINVAL, 0, "block: no h_out");
  b.h_out = A;
  b.n_routes = 3;
  expect(convrot_block_norm(&b, nullptr), CONVROT_EINVAL, 0, "block: routes without rows");
  b.route_row = i32;
  b.route_weight = f32;
  expect(convrot_block_norm(&b, nullptr), CONVROT_OK, 1, "block: no rows at all to route");
  b.gate = A;
  b.n_mod = 2;
  b.mod_stride = std::numeric_limits<int64_t>::max();
  expect(convrot_block_norm(&b, nullptr), CONVROT_EINVAL, 0, "block: odd stride");
  b.mod_stride = 1024;
  expect(convrot_block_norm(&b, nullptr), CONVROT_OK, 1, "block: modulated");
  for (int64_t K : {std::numeric_limits<int64_t>::min(), int64_t{-8}, int64_t{0}, std::numeric_limits<int64_t>::max()}) {
    b.K = K;
    expect(convrot_block_norm(&b, nullptr), CONVROT_EINVAL, 0, "block: K");
  }
  b.K = int64_t{1} << 40;
  expect(convrot_block_norm(&b, nullptr), CONVROT_EUNSUPPORTED, 0, "block: K past the registers");
  b.K = 512;
  b.M = std::numeric_limits<int64_t>::max();
  expect(convrot_block_norm(&b, nullptr), CONVROT_EINVAL, 0, "block: M");

  auto grouped = [&](int64_t M, int64_t K, int64_t E, int64_t N, int64_t P, const int32_t* rows, size_t ws) {
    return convrot_grouped_linear(A, CONVROT_BF16, M, K, i8, f32, CONVROT_SCALE_ROW, E, N, 128, nullptr, i32, rows, P, A, A,
                                  ws, nullptr);
  };
  const size_t big = std::numeric_limits<size_t>::max();
  expect(grouped(4, 128, 2, 16, 8, i32, big), CONVROT_EHIP, 2, "grouped: failed launch");
  expect(grouped(2, 128, 2, 16, 8, i32, big), CONVROT_OK, 1, "grouped: few tokens");
  expect(grouped(4, 128, 2, 16, 8, i32, convrot_grouped_workspace(4, 128) - 1), CONVROT_EWORKSPACE, 0, "grouped: workspace");
  expect(grouped(4, 128, 2, 16, 8, nullptr, big), CONVROT_EINVAL, 0, "grouped: rows missing");
  expect(grouped(4, 128, 65536, int64_t{1} << 30, int64_t{1} << 30, i32, big), CONVROT_EINVAL, 0, "grouped: tiles");
  expect(grouped(int64_t{1} << 30, 131072, 1, 1, 1, i32, 1), CONVROT_EWORKSPACE, 0, "grouped: large workspace");
  expect(grouped(std::numeric_limits<int64_t>::min(), 128, 1, 1, 1, i32, big), CONVROT_EINVAL, 0, "grouped: M");
  expect(grouped(1, 128, std::numeric_limits<int64_t>::max(), 1, 1, i32, big), CONVROT_EINVAL, 0, "grouped: E");
  expect(grouped(1, 128, 1, std::numeric_limits<int64_t>::max(), 1, i32, big), CONVROT_EINVAL, 0, "grouped: N");

  auto lora = [&](int64_t M, int64_t N, int64_t R, int64_t n, int64_t rank, size_t ws) {
    return convrot_linear_lora(A, CONVROT_F16, M, 256, i8, f32, CONVROT_SCALE_TENSOR, N, 256, A, A, A, R, f32, i32, n, rank,
                               i32, A, A, ws, nullptr);
  };
  g_rows = 0;
  expect(lora(100, 8, 32, 2, 16, convrot_lora_workspace(100, 256, 8, 16)), CONVROT_OK, 14, "lora: seven slices");
  if (g_rows != 100) ++g_failed;
  expect(lora(100, 8, 32, 2, 16, convrot_lora_workspace(100, 256, 8, 16) - 1), CONVROT_EWORKSPACE, 0, "lora: workspace");
  expect(lora(100, 8, 32, 2, std::numeric_limits<int64_t>::max(), big), CONVROT_EINVAL, 0, "lora: rank");
  expect(lora(100, 8, std::numeric_limits<int64_t>::max(), 2, 16, big), CONVROT_EINVAL, 0, "lora: R");
  expect(lora(int64_t{1} << 30, int64_t{1} << 29, 32, 2, 512, 1), CONVROT_EWORKSPACE, 0, "lora: large workspace");
  expect(lora(0, 8, 32, 2, 16, 0), CONVROT_OK, 0, "lora: no tokens");

  std::printf("operators_driver: %d checks %s\n", g_checks, g_failed ? "FAILED" : "passed");
  return g_failed ? 1 : 0;
}
