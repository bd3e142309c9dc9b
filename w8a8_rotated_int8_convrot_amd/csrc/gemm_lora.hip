// gemm_lora.hip -- the int8 product with the low-rank adapters' second product
// in its epilogue: launches of gemm_i8_kernel over a Lora (gemm_core.hpp).
#include "gemm_core.hpp"

namespace convrot {
namespace {

template <class T, int EPI>
hipError_t launch_tile(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                       const uint16_t* bias, uint16_t* y, const Lora& l, int64_t M, int64_t N, int64_t K,
                       hipStream_t stream) {
  const int tiles_n = static_cast<int>((N + T::BN - 1) / T::BN);
  const int tiles_m = static_cast<int>((M + T::BM - 1) / T::BM);
  const int64_t blocks = static_cast<int64_t>(tiles_n) * tiles_m;
  hipLaunchKernelGGL((gemm_i8_kernel<T, EPI, Lora>), dim3(static_cast<uint32_t>(blocks)), dim3(T::kThreads), 0, stream,
                     wq, xq, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), tiles_n, tiles_m, x_scale,
                     w_scale, bias, y, l);
  return hipGetLastError();
}

template <int EPI>
hipError_t launch_epi(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                      const uint16_t* bias, uint16_t* y, const Lora& l, int64_t M, int64_t N, int64_t K,
                      hipStream_t stream) {
  if (M <= 16) return launch_tile<TileSkinny16, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
  if (M <= 64) return launch_tile<TileM64, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
  if (M <= 1024) return launch_tile<TileMid, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
  return launch_tile<TileTall, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
}

}  // namespace

hipError_t launch_gemm_lora(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                            bool row_scale, const uint16_t* bias, uint16_t* y, bool f16, int64_t M, int64_t N, int64_t K,
                            const uint16_t* t, int64_t t_stride, const uint16_t* b, int64_t ranks,
                            const int32_t* offsets, int64_t adapters, const int32_t* index, int64_t max_rank,
                            hipStream_t stream) {
  if (M == 0) return hipSuccess;
  const Lora l{t, b, offsets, index, static_cast<int>(adapters), static_cast<int>(ranks), static_cast<int>(max_rank),
               static_cast<int>(t_stride)};
  if (f16)
    return row_scale ? launch_epi<kEpiF16Row>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream)
                     : launch_epi<kEpiF16>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
  return row_scale ? launch_epi<kEpiBf16Row>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream)
                   : launch_epi<kEpiBf16>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
}

}  // namespace convrot
