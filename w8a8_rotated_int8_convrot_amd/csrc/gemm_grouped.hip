// gemm_grouped.hip -- the int8 product grouped by expert: launches of
// gemm_i8_kernel over a Grouped (gemm_core.hpp) and the choice of its tile.
// For one to four tokens grouped_few_kernel does the whole call in one launch.
#include "gemm_core.hpp"
#include "rotate_device.hpp"

namespace convrot {
namespace {

// HIP counts a grid's threads along x in 32 bits.
constexpr int64_t kMaxGridThreads = (int64_t{1} << 32) - 1;

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
  if (blocks * T::kThreads > kMaxGridThreads) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((gemm_i8_kernel<T, EPI, Grouped>), dim3(static_cast<uint32_t>(blocks)), dim3(T::kThreads), 0,
                     stream, wq, xq, 0, static_cast<int>(N), static_cast<int>(K), static_cast<int>(tiles_n), 0, x_scale,
                     w_scale, bias, y, g);
  return hipGetLastError();
}

// The tile goes by the mean rows of an expert, which is all the host knows.  Up
// to 24 rows 64 x 64, or 16 x 16 where 64-channel tiles would not give every CU
// one (weights from HBM, 64 experts of 1536 x 2048, us):
//   rows      4     8    16    32
//   16 x 16  40.3  43.8  56.5  80.8
//   64 x 64  37.4  37.4  42.8  53.1
//   128x128  39.0  40.2  47.7  53.0
// Beyond, the larger tiles read less a product but come in fewer, coarser
// rounds.  A tile costs a round of its own weight: the time of a round of
// 256 x 128 is 1, and 128 x 128 0.7, 256 x 192 1.2, 192 x 288 1.25, 384 x 192
// 1.75 (the larger the tile, the less its prologue weighs and the better its
// loads are used); an expert has half a tile more than its rows fill, and more
// than one round end 0.4 of one late.  Over 11 layers and 32 to 1500 rows an
// expert this choice is 2.4 % behind the best of the five on the mean, called
// back to back, and 2.5 % with everything from HBM; thresholds on the mean rows
// 3.5 %, any one tile 6 to 16 %:
//   us                  128x128  256x128  256x192  192x288  384x192
//   16 x 1408 x 2048, 64   23.3    25.7     30.8     29.1
//   64 x 1536 x 2048, 64   66.6    58.0     64.5     65.1
//   8 x 7168 x 4096, 128   93.1    92.2     68.2     111
//   16 x 1408 x 2048, 512  58.8    52.6     64.4     65.7     46.1
//   8 x 14336 x 4096, 384                   249      259      234
//   8 x 14336 x 4096, 512   422     359      322      298      303
double round_cost(double mean, int64_t experts, int64_t N, int bn, int bm, double weight) {
  const double filled = mean / bm + 0.5;
  const double rounds =
      static_cast<double>(experts) * static_cast<double>((N + bn - 1) / bn) * (filled < 1.0 ? 1.0 : filled) / num_cus();
  return weight * (rounds > 1.0 ? rounds + 0.4 : 1.0);
}

template <int EPI>
hipError_t launch_epi(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                      const uint16_t* bias, uint16_t* y, const Grouped& g, int64_t N, int64_t K, hipStream_t stream) {
  const int64_t met = g.experts < g.P ? g.experts : g.P;
  const double mean = static_cast<double>(g.P) / static_cast<double>(met);
  if (mean <= 16 && met * ((N + 63) / 64) < num_cus())
    return launch_tile<TileSkinny16, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
  if (mean <= 24) return launch_tile<TileM64, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
  const double cost[5] = {round_cost(mean, met, N, 128, 128, 0.7), round_cost(mean, met, N, 256, 128, 1.0),
                          round_cost(mean, met, N, 256, 192, 1.2), round_cost(mean, met, N, 192, 288, 1.25),
                          round_cost(mean, met, N, 384, 192, 1.75)};
  int best = 0;
  for (int i = 1; i < 5; ++i)
    if (cost[i] < cost[best]) best = i;
  switch (best) {
    case 0: return launch_tile<TileMid, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
    case 1: return launch_tile<TileDeep, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
    case 2: return launch_tile<TileDeep192, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
    case 3: return launch_tile<TileTall, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
    default: return launch_tile<TileWide128, EPI>(xq, x_scale, wq, w_scale, bias, y, g, N, K, stream);
  }
}

// At most kFewTokens tokens of at most kFewK values: a launch costs the host as
// much as this product's weight takes to read, so one kernel does it all.  A
// workgroup has 16 channels of one expert and 16 of its rows, its four waves
// share K.  Each wave first sends for all of its weight (STEPS pieces of 16 rows
// x 64 bytes in the registers of v_mfma_i32_16x16x64_i8's operand), then the
// workgroup rotates and codes all the tokens into LDS, every workgroup the same,
// and the products take them from there.  Loads return in order, so a token's
// values arrive behind the weight: one latency covers both, and the coding of a
// few hundred instructions a wave and token comes after it, as does each further
// token's own latency.  The waves' sums are joined in LDS.
// One token, 4 of 16 experts of 1408 x 2048: 7.7 us in the trace, 9.8 a call,
// 7.9 captured; in two launches rotate + quant took 2.4 us, the product 6.2 and
// the call 13.6.
constexpr int kFewTokens = 4;
constexpr int kFewK = 8192;
struct FewTile { static constexpr int BN = 16, BM = 16, kGroupM = 1; };

template <typename In, int G, int STEPS>
__global__ __launch_bounds__(kThreads) void grouped_few_kernel(
    const In* __restrict__ x, int K, const int8_t* __restrict__ wq, int N, int tiles_n,
    const float* __restrict__ w_scale, int row_scale, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y,
    Grouped g) {
  constexpr bool F16 = !std::is_same_v<In, uint16_t>;
  constexpr int kCpt = (STEPS * 256 + kThreads * 8 - 1) / (kThreads * 8);   // K <= 256 STEPS
  extern __shared__ __attribute__((aligned(16))) char codes[];   // [x_rows][K]
  __shared__ float amax[kFewTokens][4];
  __shared__ __attribute__((aligned(16))) v4i red[3][64];
  int e, n0, m0, m_end;
  if (!grouped_tile<FewTile>(g, tiles_n, e, n0, m0, m_end)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, c16 = (lane >> 4) * 16;

  // this wave's pieces of K: wave, wave + 4, ... of 64 bytes
  const int pieces = K / 64;
  v4i w[STEPS];
  const int8_t* w_row = wq + (static_cast<int64_t>(e) * N + min(n0 + r, N - 1)) * K + c16;
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
    w[i] = *reinterpret_cast<const v4i*>(w_row + min(4 * i + wave, pieces - 1) * 64);

  // every token's codes, and its absolute maximum per wave
  for (int t = 0; t < g.x_rows; ++t) {
    const In* xr = x + static_cast<int64_t>(t) * K;
    float v[kCpt][8];
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < kCpt; ++j) {
      const int k = (j * kThreads + tid) * 8;
      if (k < K) load8(xr + k, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kCpt; ++j) {
      if ((j * kThreads + tid) * 8 < K) {
        rotate_chunk_fast<G>(v[j], tid % (G / 8));
#pragma unroll
        for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[j][i]));
      }
    }
    a = wave_max(a);
    if (lane == 0) amax[t][wave] = a;
    __syncthreads();
    const float s = fmaxf(fmaxf(amax[t][0], amax[t][1]), fmaxf(amax[t][2], amax[t][3])) / 127.0f;
#pragma unroll
    for (int j = 0; j < kCpt; ++j) {
      const int k = (j * kThreads + tid) * 8;
      if (k < K) *reinterpret_cast<uint2*>(codes + t * K + k) = pack8_fast(v[j], s);
    }
  }
  __syncthreads();

  // rows past the expert's end are its last one (not stored)
  const int p = m0 + r;
  const int src = g.source(min(p, m_end - 1));
  v4i acc = {};
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    if (4 * i + wave < pieces) {
      const v4i b = *reinterpret_cast<const v4i*>(codes + src * K + (4 * i + wave) * 64 + c16);
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[i], b, acc, 0, 0, 0);
    }
  }
  if (wave > 0) red[wave - 1][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int q = 0; q < 3; ++q) acc += red[q][lane];

  // lane l: channels n0 + 4 (l >> 4) + (0..3) of row m0 + (l & 15); the layer's
  // own epilogue, operation by operation
  if (p >= m_end || !g.has_source(p)) return;
  const float xs = fmaxf(fmaxf(amax[src][0], amax[src][1]), fmaxf(amax[src][2], amax[src][3])) / 127.0f;
  const int n = n0 + 4 * (lane >> 4);
  const float* ws = w_scale + (row_scale ? static_cast<int64_t>(e) * N : e);
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ne = min(n + i, N - 1);
    float b = 0.0f;
    if (bias != nullptr) {
      const uint16_t h = bias[static_cast<int64_t>(e) * N + ne];
      b = F16 ? static_cast<float>(__builtin_bit_cast(_Float16, h)) : __uint_as_float(static_cast<uint32_t>(h) << 16);
    }
    v[i] = __builtin_fmaf(static_cast<float>(acc[i]), xs * ws[row_scale ? ne : 0], b);
    if constexpr (F16) asm volatile("" : "+v"(v[i]));      // no fused multiply-add and conversion
  }
  const uint32_t lo = F16 ? pack_f16x2(v[0], v[1]) : pack_bf16x2(v[0], v[1]);
  const uint32_t hi = F16 ? pack_f16x2(v[2], v[3]) : pack_bf16x2(v[2], v[3]);
  uint16_t* out = y + static_cast<int64_t>(p) * N + n;
  if ((N & 3) == 0 && n + 3 < N) {
    *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) out[i] = static_cast<uint16_t>((i < 2 ? lo : hi) >> (16 * (i & 1)));
  }
}

template <typename In>
hipError_t launch_few(const void* x, const int8_t* wq, const float* w_scale, bool row_scale, const uint16_t* bias,
                      uint16_t* y, const Grouped& g, int64_t N, int64_t K, int group, hipStream_t stream) {
  const int64_t tiles_n = (N + 15) / 16;
  const int64_t blocks = tiles_n * most_tiles(g.P, g.experts, 16);
  if (blocks * kThreads > kMaxGridThreads) return hipErrorInvalidConfiguration;
  auto go = [&](auto g_c, auto steps_c) {
    hipLaunchKernelGGL((grouped_few_kernel<In, decltype(g_c)::value, decltype(steps_c)::value>),
                       dim3(static_cast<uint32_t>(blocks)), dim3(kThreads), static_cast<size_t>(g.x_rows) * K, stream,
                       static_cast<const In*>(x), static_cast<int>(K), wq, static_cast<int>(N),
                       static_cast<int>(tiles_n), w_scale, row_scale ? 1 : 0, bias, y, g);
    return hipGetLastError();
  };
  auto go_group = [&](auto g_c) {
    if (K <= 2048) return go(g_c, std::integral_constant<int, 8>{});
    if (K <= 4096) return go(g_c, std::integral_constant<int, 16>{});
    return go(g_c, std::integral_constant<int, 32>{});
  };
  return group == 128 ? go_group(std::integral_constant<int, 128>{}) : go_group(std::integral_constant<int, 256>{});
}

}  // namespace

bool grouped_is_few(int64_t M, int64_t K) { return M <= kFewTokens && K <= kFewK; }

hipError_t launch_grouped_few(const void* x, int64_t M, int64_t K, int group, bool f16, const int8_t* wq,
                              const float* w_scale, bool row_scale, const uint16_t* bias, uint16_t* y,
                              const int32_t* offsets, const int32_t* rows, int64_t experts, int64_t P, int64_t N,
                              hipStream_t stream) {
  if (P == 0) return hipSuccess;
  const Grouped g{offsets, rows, static_cast<int>(experts), static_cast<int>(P), static_cast<int>(M)};
  return f16 ? launch_few<_Float16>(x, wq, w_scale, row_scale, bias, y, g, N, K, group, stream)
             : launch_few<uint16_t>(x, wq, w_scale, row_scale, bias, y, g, N, K, group, stream);
}

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
