// gemm_i8.hip -- the ConvRot linear layer's int8 product and the default
// path's bf16 / fp16 product: launches of the kernels in gemm_core.hpp and the
// choice of tile.
#include "gemm_core.hpp"

namespace convrot {
namespace {

template <class T, int EPI>
hipError_t launch_tile(const int8_t* xq, const float* x_scale, const int8_t* wq,
                       const float* w_scale, const uint16_t* bias, void* out, int64_t M,
                       int64_t N, int64_t K, hipStream_t stream) {
  const int tiles_n = static_cast<int>((N + T::BN - 1) / T::BN);
  const int tiles_m = static_cast<int>((M + T::BM - 1) / T::BM);
  const int64_t blocks = static_cast<int64_t>(tiles_n) * tiles_m;
  hipLaunchKernelGGL((gemm_i8_kernel<T, EPI>), dim3(static_cast<uint32_t>(blocks)),
                     dim3(T::kThreads), 0, stream, wq, xq, static_cast<int>(M), static_cast<int>(N),
                     static_cast<int>(K), tiles_n, tiles_m, x_scale, w_scale, bias, out,
                     NoExtra{});
  return hipGetLastError();
}

// Few-token launch: 16 output channels per workgroup, K split over its four
// waves (M <= 16); the register-streamed kernel where K = 3072 or 4096.
template <int EPI, int S>
hipError_t launch_ksplit(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                         const uint16_t* bias, void* out, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>((N + 15) / 16));
  const int m = static_cast<int>(M), n = static_cast<int>(N), k = static_cast<int>(K);
  if (K == 512 * 8)
    hipLaunchKernelGGL((gemm_ksplit_reg_kernel<EPI, 8>), grid, dim3(256), 0, stream, wq, xq, m, n, k, x_scale,
                       w_scale, bias, out);
  else if (K == 512 * 6)
    hipLaunchKernelGGL((gemm_ksplit_reg_kernel<EPI, 6>), grid, dim3(256), 0, stream, wq, xq, m, n, k, x_scale,
                       w_scale, bias, out);
  else
    hipLaunchKernelGGL((gemm_ksplit_kernel<EPI, S>), grid, dim3(256), 0, stream, wq, xq, m, n, k, x_scale, w_scale,
                       bias, out);
  return hipGetLastError();
}

// Persistent launch: one workgroup per CU (at most one per tile).
template <class T, int EPI>
hipError_t launch_persist(const int8_t* xq, const float* x_scale, const int8_t* wq,
                          const float* w_scale, const uint16_t* bias, void* out, int64_t M,
                          int64_t N, int64_t K, hipStream_t stream) {
  const int tiles_n = static_cast<int>((N + T::BN - 1) / T::BN);
  const int tiles_m = static_cast<int>((M + T::BM - 1) / T::BM);
  const int64_t tiles = static_cast<int64_t>(tiles_n) * tiles_m;
  const int64_t grid = tiles < num_cus() ? tiles : num_cus();
  if (K < 3 * T::BK) return launch_tile<T, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  hipLaunchKernelGGL((gemm_persist_kernel<T, EPI>), dim3(static_cast<uint32_t>(grid)), dim3(T::kThreads), 0,
                     stream, wq, xq, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), tiles_n,
                     tiles_m, x_scale, w_scale, bias, out, NoExtra{});
  return hipGetLastError();
}

// Tile choice: CONVROT_GEMM_TILE=big|big8|wide|wide128|mid|skinny|skinny16|half|m32|m64|m128|p128|phalf|tall|ptall|ksplit
// forces one (the result does not depend on it; p128, phalf and ptall are the
// persistent 384 x 192, 384 x 96 and 192 x 288 kernels, which take the
// one-tile kernel below three slabs of K; ksplit holds at most 16 tokens).
// Otherwise: M <= 16 streams the weight with the K-split 16 x 16 tile where
// N / 16 is at least twice the CU count, else with the one-wave 16 x 16
// tile, and M <= 256 with the small tile whose
// slowest CU moves the fewest operand bytes; larger layers with fewer
// 384 x 192 tiles than half the CUs use 384 x 96, 128 x 128 or 64 x 128
// tiles.  Else the cost of a large tile is the number of rounds its tiles
// take over the CUs times the work of one tile: 192 x 288 wherever 384 x 192
// would need its half-height tail or costs no less, then the cheaper of
// 384 x 192 and 256 x 256 (the latter only by a clear margin).
int forced_tile() {
  const char* e = getenv("CONVROT_GEMM_TILE");
  if (e == nullptr) return 0;
  if (strcmp(e, "big") == 0) return 1;
  if (strcmp(e, "big8") == 0) return 2;
  if (strcmp(e, "mid") == 0) return 3;
  if (strcmp(e, "wide") == 0) return 4;
  if (strcmp(e, "skinny") == 0) return 5;
  if (strcmp(e, "wide128") == 0) return 6;
  if (strcmp(e, "skinny16") == 0) return 7;
  if (strcmp(e, "half") == 0) return 8;
  if (strcmp(e, "m32") == 0) return 10;
  if (strcmp(e, "m64") == 0) return 11;
  if (strcmp(e, "m128") == 0) return 12;
  if (strcmp(e, "p128") == 0) return 13;
  if (strcmp(e, "phalf") == 0) return 14;
  if (strcmp(e, "tall") == 0) return 15;
  if (strcmp(e, "ptall") == 0) return 16;
  if (strcmp(e, "ksplit") == 0) return 19;
  return 0;
}

int64_t tile_cost(int64_t M, int64_t N, int64_t bn, int64_t bm) {
  const int64_t kCUs = num_cus();
  const int64_t tiles = ((N + bn - 1) / bn) * ((M + bm - 1) / bm);
  return (tiles + kCUs - 1) / kCUs * bn * bm;
}

// Token tiles of 384 x 192 that run in whole rounds.  When their last round
// would be at most half full and the remaining token rows fit one round of
// 384 x 96 tiles, only the whole rounds use 384 x 192 and the rest of M runs
// as half-height tiles; otherwise every token tile is 384 x 192.
int64_t wide_main_m(int64_t M, int64_t N) {
  const int64_t kCUs = num_cus();
  const int64_t tn = (N + 383) / 384, tm = (M + 191) / 192;
  const int64_t tiles = tn * tm, rounds = (tiles + kCUs - 1) / kCUs;
  const int64_t last = tiles - (rounds - 1) * kCUs;
  if (rounds < 2 || 2 * last > kCUs) return tm;
  const int64_t main_m = (rounds - 1) * kCUs / tn;
  const int64_t tail = (M - main_m * 192 + 95) / 96 * tn;
  return main_m > 0 && tail <= kCUs ? main_m : tm;
}

// Cost of 384 x 192 tiles, counting the half-height tail as half a round.
int64_t wide_cost(int64_t M, int64_t N) {
  const int64_t kCUs = num_cus();
  const int64_t tn = (N + 383) / 384, tm = (M + 191) / 192, main_m = wide_main_m(M, N);
  if (main_m == tm) return tile_cost(M, N, 384, 192);
  return ((main_m * tn + kCUs - 1) / kCUs * 2 + 1) * 384 * 96;
}

}  // namespace

int pick_gemm_tile(int64_t M, int64_t N) {
  const int64_t kCUs = num_cus();
  if (M <= 16) return (N + 15) / 16 >= 2 * kCUs ? 19 : 7;
  if (M <= 256) {
    // Weight-streaming layers.  The slowest CU runs ceil(tiles / CUs) tiles,
    // each moving its BN weight rows and BM token rows per K byte; weight rows
    // count twice (they come from HBM, token rows mostly from L2).  The
    // candidate with the least such traffic wins, ties to the narrower tile.
    // Against the best forced tile on 28 shapes (M = 16..256, N = 3072..12288,
    // K = 3072, weight from HBM): 1.3 % slower on average and 9 % at worst,
    // where a rule by channel count alone was 4 % and 34 %.
    struct Cand { int t, bn, bm; };
    constexpr Cand kCands[] = {{7, 16, 16}, {5, 32, 32}, {10, 64, 32}, {11, 64, 64}, {12, 64, 128}, {3, 128, 128}};
    int best = 7;
    int64_t best_cost = -1;
    for (const Cand& c : kCands) {
      const int64_t tiles = ((N + c.bn - 1) / c.bn) * ((M + c.bm - 1) / c.bm);
      const int64_t cost = (tiles + kCUs - 1) / kCUs * (2 * c.bn + c.bm);
      if (best_cost < 0 || cost < best_cost) best = c.t, best_cost = cost;
    }
    return best;
  }
  // Fewer 384 x 192 tiles than half the CUs: smaller tiles give more
  // workgroups: 384 x 96 when they make one full round (more than 3/8 of the
  // CUs' worth of large tiles: 3072 x 3072 x 3072 in 34.5 us instead of 40.4),
  // else 128 x 128 (two per CU), or 64 x 128 where even those would fill less
  // than half the CUs (weight from HBM: 512 x 12288 x 4096 in 51 us instead of
  // 59, 512 x 3072 x 12288 in 52 instead of 73; from 128 large tiles on,
  // 384 x 192 is faster again: 768 x 12288 x 4096 in 64 us against 76 with
  // 128 x 128)
  const int64_t wide = ((M + 191) / 192) * ((N + 383) / 384);
  if (2 * wide <= kCUs && 8 * wide > 3 * kCUs) return 8;
  if (2 * wide < kCUs)
    return 2 * ((M + 127) / 128) * ((N + 127) / 128) < kCUs ? 12 : 3;
  // 192 x 288 tiles where their rounds cost no more than those of 384 x 192
  // with its tail: with the epilogue run beside the next tile's first MFMAs
  // they are the faster of the two at equal cost (M = 4608, N = 12288,
  // K = 3072: 140.4 us against 145.7; N = 3072 and 9216 take fewer rounds).
  // Where 384 x 192 would need its half-height tail, 192 x 288 tiles are
  // taken at any cost: the tail is a launch of its own whose 384 x 96 tiles
  // run one per workgroup with nothing beside their prologue and epilogue,
  // and it lost on every shape measured (4700 x 12290 x 640: 67 us with
  // 192 x 288 against 80; 16896 x 9216 x 3072: 404 against 427;
  // 19894 x 4096 x 384: 55 against 68).
  if (wide_main_m(M, N) < (M + 191) / 192) return 16;
  if (tile_cost(M, N, 192, 288) <= wide_cost(M, N)) return 16;
  // the 256 x 256 tile (one wave per SIMD) wins only by a clear margin: it
  // was as fast or slower on every shape measured, also where its cost is
  // lower (M = 4608, N = 3072: 184 us for 216 tiles against 180 us for 192 at
  // K = 12288, 57-59 against 52-53 us at K = 3072; 3072 x 9216 x 4096: 142.5
  // against 138.5 us)
  return wide_cost(M, N) * 100 < tile_cost(M, N, 256, 256) * 115 ? 6 : 1;
}

namespace {

template <int EPI>
hipError_t launch_gemm(const int8_t* xq, const float* x_scale, const int8_t* wq,
                       const float* w_scale, const uint16_t* bias, void* out, int64_t M,
                       int64_t N, int64_t K, hipStream_t stream) {
  int t = forced_tile();
  const bool automatic = t == 0;
  if (automatic) t = pick_gemm_tile(M, N);
  if (t == 1) return launch_tile<TileBig, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  if (t == 2) return launch_tile<TileBig8, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  if (t == 4) return launch_tile<TileWide, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  if (t == 5) return launch_tile<TileSkinny, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  if (automatic && t == 6) {
    // persistent 384 x 192 tiles where a workgroup gets several (more tiles
    // than CUs) and K has three or more slabs, one-tile workgroups
    // otherwise; both with the half-height tail below
    const int64_t tiles = ((N + 383) / 384) * wide_main_m(M, N);
    if (tiles > num_cus() && K >= 3 * 128) t = 13;
  }
  if (t == 6) {
    // whole rounds of 384 x 192, then (if any) the rest of M as 384 x 96;
    // K counts bytes, and the output rows are 2 (dequant) or 4 (int32) bytes
    const int64_t split = wide_main_m(M, N) * 192;
    if (split >= M) return launch_tile<TileWide128, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
    hipError_t e = launch_tile<TileWide128, EPI>(xq, x_scale, wq, w_scale, bias, out, split, N, K, stream);
    if (e != hipSuccess) return e;
    const int64_t out_elem = EPI == kEpiI32 ? 4 : 2;
    return launch_tile<TileWideHalf, EPI>(xq + split * K, x_scale ? x_scale + split : nullptr, wq, w_scale,
                                          bias, static_cast<char*>(out) + split * N * out_elem, M - split, N,
                                          K, stream);
  }
  if (t == 8) return launch_tile<TileWideHalf, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  if (t == 13) {
    const int64_t split = wide_main_m(M, N) * 192;
    if (split >= M) return launch_persist<TileWide128, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
    hipError_t e = launch_persist<TileWide128, EPI>(xq, x_scale, wq, w_scale, bias, out, split, N, K, stream);
    if (e != hipSuccess) return e;
    // the tail is at most one round: one tile per workgroup
    const int64_t out_elem = EPI == kEpiI32 ? 4 : 2;
    return launch_tile<TileWideHalf, EPI>(xq + split * K, x_scale ? x_scale + split : nullptr, wq, w_scale, bias,
                                          static_cast<char*>(out) + split * N * out_elem, M - split, N, K, stream);
  }
  if (t == 14) return launch_persist<TileWideHalf, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  if (t == 15) return launch_tile<TileTall, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  if (t == 16) return launch_persist<TileTall, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  if (t == 19 && M > 16) t = 7;   // the K-split tile holds 16 tokens
  if (t == 19) return launch_ksplit<EPI, 2>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  if (t == 7) return launch_tile<TileSkinny16, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  if (t == 10) return launch_tile<TileM32, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  if (t == 11) return launch_tile<TileM64, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  if (t == 12) return launch_tile<TileM128, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
  return launch_tile<TileMid, EPI>(xq, x_scale, wq, w_scale, bias, out, M, N, K, stream);
}

}  // namespace

hipError_t launch_gemm_dequant(const int8_t* xq, const float* x_scale, const int8_t* wq,
                               const float* w_scale, const uint16_t* bias, uint16_t* y,
                               int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  return launch_gemm_dequant_ex(xq, x_scale, wq, w_scale, false, bias, y, false, M, N, K, stream);
}

hipError_t launch_gemm_dequant_ex(const int8_t* xq, const float* x_scale, const int8_t* wq,
                                  const float* w_scale, bool row_scale, const uint16_t* bias,
                                  uint16_t* y, bool out_f16, int64_t M, int64_t N, int64_t K,
                                  hipStream_t stream) {
  if (M == 0) return hipSuccess;
  if (out_f16)
    return row_scale ? launch_gemm<kEpiF16Row>(xq, x_scale, wq, w_scale, bias, y, M, N, K, stream)
                     : launch_gemm<kEpiF16>(xq, x_scale, wq, w_scale, bias, y, M, N, K, stream);
  return row_scale ? launch_gemm<kEpiBf16Row>(xq, x_scale, wq, w_scale, bias, y, M, N, K, stream)
                   : launch_gemm<kEpiBf16>(xq, x_scale, wq, w_scale, bias, y, M, N, K, stream);
}

hipError_t launch_gemm_i32(const int8_t* xq, const int8_t* wq, int32_t* acc, int64_t M,
                           int64_t N, int64_t K, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  return launch_gemm<kEpiI32>(xq, nullptr, wq, nullptr, nullptr, acc, M, N, K, stream);
}

hipError_t launch_gemm_default(const uint16_t* x, const uint16_t* wu, const uint16_t* bias, uint16_t* y,
                               bool f16, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  // operands travel as bytes: a row of K 16-bit values is 2K bytes
  const auto* a = reinterpret_cast<const int8_t*>(x);
  const auto* b = reinterpret_cast<const int8_t*>(wu);
  return f16 ? launch_gemm<kEpiDefF16>(a, nullptr, b, nullptr, bias, y, M, N, 2 * K, stream)
             : launch_gemm<kEpiDefBf16>(a, nullptr, b, nullptr, bias, y, M, N, 2 * K, stream);
}

}  // namespace convrot
