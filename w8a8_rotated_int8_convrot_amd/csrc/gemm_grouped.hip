// gemm_grouped.hip -- the int8 product grouped by expert: launches of
// gemm_i8_kernel over a Grouped (gemm_core.hpp) and the choice of its tile.
#include "gemm_core.hpp"

namespace convrot {
namespace {

// The most token tiles of bm rows that P rows of `experts` experts can make:
// every expert with rows may end in one partial tile.
int64_t most_tiles(int64_t P, int64_t experts, int64_t bm) {
  const int64_t t = P / bm + (experts < P ? experts : P);
  return t < P ? t : P;
}

template <class T, int EPI>
hipError_t launch_tile(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                       const uint16_t* bias, uint16_t* y, const Grouped& g, int64_t N, int64_t K,
                       hipStream_t stream) {
  const int64_t tiles_n = (N + T::BN - 1) / T::BN;
  const int64_t blocks = tiles_n * most_tiles(g.P, g.experts, T::BM);
  if (blocks > kMaxGroupedTiles) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((gemm_i8_kernel<T, EPI, Grouped>), dim3(static_cast<uint32_t>(blocks)), dim3(T::kThreads), 0,
                     stream, wq, xq, 0, static_cast<int>(N), static_cast<int>(K), static_cast<int>(tiles_n), 0, x_scale,
                     w_scale, bias, y, g);
  return hipGetLastError();
}

// The tile goes by the mean rows of an expert, which is all the host knows.
template <int EPI>
hipError_t launch_epi(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                      const uint16_t* bias, uint16_t* y, const Grouped& g, int64_t N, int64_t K, hipStream_t stream) {
  const int64_t mean = (static_cast<int64_t>(g.P) + g.experts - 1) / g.experts;
  if (mean <= 16) return launch_tile<TileSkinny16, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
  if (mean <= 64) return launch_tile<TileM64, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
  if (mean <= 256) return launch_tile<TileMid, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
  return launch_tile<TileTall, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
}

}  // namespace

hipError_t launch_gemm_grouped(const int8_t* xq, const float* x_scale, int64_t x_rows, const int8_t* wq,
                               const float* w_scale, bool row_scale, const uint16_t* bias, uint16_t* y, bool f16,
                               const int32_t* offsets, const int32_t* rows, int64_t experts, int64_t P, int64_t N,
                               int64_t K, hipStream_t stream) {
  if (P == 0) return hipSuccess;
  const Grouped g{offsets, rows, static_cast<int>(experts), static_cast<int>(P), static_cast<int>(x_rows)};
  if (f16)
    return row_scale ? launch_epi<kEpiF16Row>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream)
                     : launch_epi<kEpiF16>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
  return row_scale ? launch_epi<kEpiBf16Row>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream)
                   : launch_epi<kEpiBf16>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
}

}  // namespace convrot
