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

// The tile goes by the mean rows of an expert, which is all the host knows
// (weights from HBM, 64 experts of 1536 x 2048, us):
//   rows      4     8    16    32    64
//   16 x 16  40.3  43.8  56.5  80.8   130
//   64 x 64  37.4  37.4  42.8  53.1  68.5
//   128x128  39.0  40.2  47.7  53.0  57.9
//   192x288  45.0  46.6  49.4  54.0  57.4
// and 32 of 2048 x 4096:  96   128   192   256
//   128x128              88.3  87.6   108   134
//   192x288              96.4   102   105   109
// 64 x 64 up to 24 rows, 128 x 128 up to 160, then 192 x 288; 16 x 16 where
// 64-channel tiles would not give every CU one.
template <int EPI>
hipError_t launch_epi(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                      const uint16_t* bias, uint16_t* y, const Grouped& g, int64_t N, int64_t K, hipStream_t stream) {
  const int64_t mean = (static_cast<int64_t>(g.P) + g.experts - 1) / g.experts;
  const int64_t met = g.experts < g.P ? g.experts : g.P;
  if (mean <= 16 && met * ((N + 63) / 64) < num_cus())
    return launch_tile<TileSkinny16, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
  if (mean <= 24) return launch_tile<TileM64, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
  if (mean <= 160) return launch_tile<TileMid, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
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
