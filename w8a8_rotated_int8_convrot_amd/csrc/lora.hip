// lora.hip -- the first product of the low-rank adapters beside the layer:
//   t[m][r] = rnd(scale[a] * sum_k A[offsets[a] + r][k] * x[m][k]),  a = index[m]
// for r below the rank of a, 0 up to the row's stride; tokens without an
// adapter are skipped (nobody reads their rows).  x is the layer's own input,
// neither rotated nor coded.  The sum is held in fp32 and rounded to the io
// type once, as the second product's matrix operand (an adapter run as two
// layers rounds there too); it moves the result by at most half a step of the
// adapter's part.
//
// A workgroup takes 16 tokens: its eight waves split K (64 elements at a time,
// so a row piece is a whole 128-byte line), each keeps the sums of up to four
// blocks of 16 ranks in registers (v_mfma_*_16x16x32, ranks x tokens) and the
// waves' sums are joined through LDS in a fixed order.  The tokens' adapters
// are taken one after another, or, where few token tiles would leave the chip
// idle, dealt out over gridDim.y workgroups; gridDim.z deals out the ranks in
// blocks of 64.
#include <type_traits>

#include "convrot_internal.hpp"

namespace convrot {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kWaves = 8;
constexpr int kBlocks = 4;      // 16-rank blocks of one pass

template <bool F16>
__device__ inline v4f mfma(v4i a, v4i b, v4f c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

template <bool F16>
__device__ inline uint16_t round16(float v) {
  if constexpr (F16) return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  else return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

template <bool F16>
__global__ __launch_bounds__(kWaves * 64) void lora_down_kernel(
    const uint16_t* __restrict__ x, int M, int K, const uint16_t* __restrict__ a_rows, int ranks,
    const float* __restrict__ scale, const int32_t* __restrict__ offsets, int adapters,
    const int32_t* __restrict__ index, int max_rank, uint16_t* __restrict__ t, int t_stride) {
  __shared__ __attribute__((aligned(16))) v4f part[kWaves][kBlocks][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, k8 = lane >> 4 << 3;
  const int m = blockIdx.x * 16 + r;
  int own = m < M ? index[m] : -1;
  if (own >= adapters) own = -1;
  const uint16_t* x_row = x + static_cast<int64_t>(min(m, M - 1)) * K + k8;

  // the tile's distinct adapters, every gridDim.y-th one here
  uint64_t left = __ballot(lane < 16 && own >= 0);
  for (int turn = 0; left != 0; ++turn) {
    const int a = __builtin_amdgcn_readlane(own, __builtin_ctzll(left));
    left &= ~__ballot(own == a);
    if (turn % gridDim.y != blockIdx.y) continue;
    const int row0 = min(max(offsets[a], 0), ranks);
    const int rank = min(min(max(offsets[a + 1], row0), ranks) - row0, max_rank);
    const float s = scale[a];
    for (int base = blockIdx.z * 16 * kBlocks; base < t_stride; base += gridDim.z * 16 * kBlocks) {
      const int blocks = min(kBlocks, (t_stride - base) / 16);       // t_stride is a multiple of 32
      const int full = min(kBlocks, max(0, (rank - base + 15) / 16));   // blocks that hold ranks
      v4f acc[kBlocks] = {};
      if (full > 0) {
        const uint16_t* w_row[kBlocks];
#pragma unroll
        for (int q = 0; q < kBlocks; ++q)
          w_row[q] = a_rows + static_cast<int64_t>(row0 + min(base + 16 * q + r, rank - 1)) * K + k8;
        for (int k = wave * 64; k < K; k += kWaves * 64) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v4i xf = *reinterpret_cast<const v4i*>(x_row + k + 32 * h);
#pragma unroll
            for (int q = 0; q < kBlocks; ++q)
              if (q < full) acc[q] = mfma<F16>(*reinterpret_cast<const v4i*>(w_row[q] + k + 32 * h), xf, acc[q]);
          }
        }
      }
#pragma unroll
      for (int q = 0; q < kBlocks; ++q) part[wave][q][lane] = acc[q];
      __syncthreads();
      // wave q adds block q: lane l holds ranks 4 (l >> 4) + e of token l & 15
      if (wave < blocks) {
        v4f sum = part[0][wave][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum += part[w][wave][lane];
        if (own == a) {
          const int rank0 = base + 16 * wave + (lane >> 4) * 4;
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = rank0 + e < rank ? round16<F16>(s * sum[e]) : 0;
          *reinterpret_cast<uint2*>(t + static_cast<int64_t>(m) * t_stride + rank0) =
              make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
        }
      }
      __syncthreads();
    }
  }
}

}  // namespace

hipError_t launch_lora_down(const uint16_t* x, int64_t M, int64_t K, bool f16, const uint16_t* a, int64_t ranks,
                            const float* scale, const int32_t* offsets, int64_t adapters, const int32_t* index,
                            int64_t max_rank, uint16_t* t, int64_t t_stride, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  const int64_t tiles = (M + 15) / 16;
  const int64_t most = adapters < 16 ? adapters : 16;         // adapters a tile can hold
  const int64_t want = (2 * num_cus() + tiles - 1) / tiles;
  const int64_t turns = want < most ? want : most;
  const int64_t rank_blocks = (t_stride + 16 * kBlocks - 1) / (16 * kBlocks);
  const dim3 grid(static_cast<uint32_t>(tiles), static_cast<uint32_t>(turns), static_cast<uint32_t>(rank_blocks));
  const int m = static_cast<int>(M), k = static_cast<int>(K);
  if (f16)
    hipLaunchKernelGGL(lora_down_kernel<true>, grid, dim3(kWaves * 64), 0, stream, x, m, k, a, static_cast<int>(ranks),
                       scale, offsets, static_cast<int>(adapters), index, static_cast<int>(max_rank), t,
                       static_cast<int>(t_stride));
  else
    hipLaunchKernelGGL(lora_down_kernel<false>, grid, dim3(kWaves * 64), 0, stream, x, m, k, a, static_cast<int>(ranks),
                       scale, offsets, static_cast<int>(adapters), index, static_cast<int>(max_rank), t,
                       static_cast<int>(t_stride));
  return hipGetLastError();
}

}  // namespace convrot
