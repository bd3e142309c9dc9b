// gemm_lora.hip -- the int8 product with the low-rank adapters' second product
// in its epilogue: launches of gemm_i8_kernel over a Lora (gemm_core.hpp).
#include "gemm_core.hpp"

namespace convrot {
namespace {

template <class T, int EPI, class X>
hipError_t launch_tile(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                       const uint16_t* bias, uint16_t* y, const X& l, int64_t M, int64_t N, int64_t K,
                       hipStream_t stream) {
  const int tiles_n = static_cast<int>((N + T::BN - 1) / T::BN);
  const int tiles_m = static_cast<int>((M + T::BM - 1) / T::BM);
  const int64_t blocks = static_cast<int64_t>(tiles_n) * tiles_m;
  hipLaunchKernelGGL((gemm_i8_kernel<T, EPI, X>), dim3(static_cast<uint32_t>(blocks)), dim3(T::kThreads), 0, stream,
                     wq, xq, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), tiles_n, tiles_m, x_scale,
                     w_scale, bias, y, l);
  return hipGetLastError();
}

template <class T, int EPI>
hipError_t launch_persist(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                          const uint16_t* bias, uint16_t* y, const LoraList& l, int64_t M, int64_t N, int64_t K,
                          hipStream_t stream) {
  if (K < 3 * T::BK) return launch_tile<T, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
  const int tiles_n = static_cast<int>((N + T::BN - 1) / T::BN);
  const int tiles_m = static_cast<int>((M + T::BM - 1) / T::BM);
  const int64_t tiles = static_cast<int64_t>(tiles_n) * tiles_m;
  const int64_t grid = tiles < num_cus() ? tiles : num_cus();
  hipLaunchKernelGGL((gemm_persist_kernel<T, EPI, LoraList>), dim3(static_cast<uint32_t>(grid)), dim3(T::kThreads), 0,
                     stream, wq, xq, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), tiles_n, tiles_m,
                     x_scale, w_scale, bias, y, l);
  return hipGetLastError();
}

// Whether these tiles make one round that gives more than 5/8 of the CUs a
// tile: 256 x 128, else 256 x 192.  Such a round is as long as one tile, and
// nothing runs beside a tile's prologue and the adapters' panels, so the smallest
// tile that still makes one round wins; the layer's own choice (two 128 x 128
// tiles a CU, half-empty rounds of 384 x 96 or 192 x 288) gives each CU more.  us
// a call with six adapters of rank 32 in bf16, weight from HBM, the layer's
// choice -> this (M x K x N, tiles):
//   2000 x 12288 x 4096 (256)  180 -> 137     1024 x 8192 x 8192 (256)  113 -> 87
//   1500 x 4096 x 4096 (192)    52 -> 49      512 x 4096 x 12288 (192)  59 -> 50
//   1300 x 4096 x 4096 (176)    53 -> 47      777 x 2048 x 6144 (168)   33 -> 32
// with 256 x 192:
//   1500 x 2048 x 8192 (256)    74 -> 47      1500 x 4096 x 8192 (256)  109 -> 72
//   3000 x 4096 x 4096 (256)    78 -> 77      2300 x 4096 x 4096 (192)   69 -> 65
//   2816 x 12288 x 4096 (240)  182 -> 175     769 x 4096 x 12288 (240)   72 -> 68
// and past those bounds, 256 x 128: 1024 x 4096 x 4096 (128 tiles)  37 -> 45,
// 4608 x 4096 x 12288 (1728)  247 -> 284.
template <class T>
bool one_round(int64_t M, int64_t N) {
  const int64_t tiles = ((M + T::BM - 1) / T::BM) * ((N + T::BN - 1) / T::BN);
  return M > 256 && tiles <= num_cus() && 8 * tiles > 5 * num_cus();
}

// The tiles are the layer's own (pick_gemm_tile) otherwise, with the persistent
// 192 x 288 kernel for its largest ones and the one-wave 16 x 16 tile for few
// tokens.
// Where lora_by_token says so each lane adds its own token's ranks; other batches
// go through the list of the tile's adapters.
template <int EPI>
hipError_t launch_epi(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                      const uint16_t* bias, uint16_t* y, const Lora& lora, int64_t M, int64_t N, int64_t K,
                      hipStream_t stream) {
  const int tile = pick_gemm_tile(M, N);
  if (lora_by_token(M, lora.adapters, lora.max_rank)) {
    const LoraGather l{lora};
    if (M <= 16) return launch_tile<TileSkinny16, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
    if (tile == 10) return launch_tile<TileM32, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
    if (tile == 11) return launch_tile<TileM64, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
    if (tile == 12) return launch_tile<TileM128, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
    return launch_tile<TileSkinny, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
  }
  const LoraList l{lora};
  if (one_round<TileDeep>(M, N))
    return launch_tile<TileDeep, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
  if (one_round<TileDeep192>(M, N))
    return launch_tile<TileDeep192, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
  switch (tile) {
    case 7: return launch_tile<TileSkinny16, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
    case 5: return launch_tile<TileSkinny, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
    case 10: return launch_tile<TileM32, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
    case 11: return launch_tile<TileM64, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
    case 12: return launch_tile<TileM128, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
    case 3: return launch_tile<TileMid, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
    case 8: return launch_tile<TileWideHalf, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
    default: return launch_persist<TileTall, EPI>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
  }
}

}  // namespace

hipError_t launch_gemm_lora(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                            bool row_scale, const uint16_t* bias, uint16_t* y, bool f16, int64_t M, int64_t N, int64_t K,
                            const uint16_t* t, int64_t t_stride, const uint16_t* b, int64_t ranks,
                            const int32_t* offsets, int64_t adapters, const int32_t* index, int64_t max_rank,
                            hipStream_t stream) {
  if (M == 0) return hipSuccess;
  const Lora l{lora_behind_t(t, M, t_stride), reinterpret_cast<const float*>(t), b, offsets, index, static_cast<int>(adapters), static_cast<int>(ranks), static_cast<int>(max_rank),
               static_cast<int>(t_stride)};
  if (f16)
    return row_scale ? launch_epi<kEpiF16Row>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream)
                     : launch_epi<kEpiF16>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
  return row_scale ? launch_epi<kEpiBf16Row>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream)
                   : launch_epi<kEpiBf16>(xq, x_scale, wq, w_scale, bias, y, l, M, N, K, stream);
}

}  // namespace convrot
