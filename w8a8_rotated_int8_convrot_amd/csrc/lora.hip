// lora.hip -- the first product of the low-rank adapters beside the layer:
//   t[m][r] = rnd(scale[a] * sum_k A[offsets[a] + r][k] * x[m][k]),  a = index[m]
// for r below the rank of a, 0 up to the row's stride; tokens without an
// adapter are skipped (nobody reads their rows).  x is the layer's own input,
// neither rotated nor coded.  The sum is held in fp32 and rounded to the io
// type once, as the second product's matrix operand (an adapter run as two
// layers rounds there too); it moves the result by at most half a step of the
// adapter's part.
//
// lora_down_kernel: a workgroup takes 64 tokens and a part of K, which its four
// waves split again; each wave keeps the sums of 4 x NB blocks (16 tokens x 16
// ranks, v_mfma_*_16x16x32) in registers, so a loaded piece of x serves 16 NB
// ranks and a piece of the adapter 64 tokens.  What bounds it is what a CU can
// draw from its L2 (about 27 bytes a cycle here), and 64 tokens a workgroup
// with K split over gridDim.y move half of what 16 tokens with all of K do
// while filling the chip.  A wave that has several pieces of K loads two before it
// multiplies.  The waves' sums are joined through LDS, the parts
// of K by lora_sum, both in a fixed order.  The adapters met among the
// tokens are taken one after another, or, where the tiles would leave the chip
// idle, dealt out over gridDim.z workgroups.
//
// lora_dot, for few tokens with adapters of their own: a wave per token and two
// of its ranks, each lane a plain dot product over its part of K.
#include <type_traits>

#include "convrot_internal.hpp"
#include "rotate_device.hpp"

namespace convrot {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kTile = 64;       // tokens of a workgroup
constexpr int kWaves = 4;

struct Down {
  const uint16_t *x, *a_rows;
  const float* scale;
  const int32_t *offsets, *index;
  uint16_t* t;
  int M, K, ranks, adapters, max_rank, t_stride;
  // rows [row0, row0 + rank) of adapter a, inside [0, ranks)
  __device__ void range(int a, int& row0, int& rank) const {
    row0 = min(max(offsets[a], 0), ranks);
    rank = min(min(max(offsets[a + 1], row0), ranks) - row0, max_rank);
  }
};

template <bool F16>
__device__ inline v4f mfma(v4i a, v4i b, v4f c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

template <bool F16>
__device__ inline uint32_t round16(float v) {
  if constexpr (F16) return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  else return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// sums [gridDim.y][M][t_stride] fp32
template <bool F16, int NB, int DEPTH>
__global__ __launch_bounds__(kWaves * 64) void lora_down_kernel(Down p, float* __restrict__ sums) {
  __shared__ __attribute__((aligned(16))) v4f part[kWaves][4][NB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, k8 = lane >> 4 << 3;
  const int m0 = blockIdx.x * kTile;
  const int M = p.M, K = p.K;
  const int mine = p.index[min(m0 + lane, M - 1)];
  // this part's pieces of 64 elements are neighbours, dealt out to the waves
  constexpr int step = kWaves * 64;
  const int part_k = (K / 64 + gridDim.y - 1) / gridDim.y * 64;
  const int k0 = blockIdx.y * part_k + wave * 64, k_end = min(K, static_cast<int>(blockIdx.y + 1) * part_k);
  // after the sum this wave stores token block `wave`
  const int m_out = m0 + 16 * wave + r;
  const int own = m_out < M ? p.index[m_out] : -1;

  uint64_t left = __ballot(m0 + lane < M && mine >= 0 && mine < p.adapters);
  for (int turn = 0; left != 0; ++turn) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    const uint64_t same = __ballot(m0 + lane < M && mine == a);
    left &= ~same;
    if (turn % gridDim.z != blockIdx.z) continue;
    int row0, rank;
    p.range(a, row0, rank);
    // a block of 16 tokens without this adapter reads the rows of one with it
    // (its sums are not used), so that it draws nothing more from L2
    const uint16_t* x_row[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int from = (same >> (16 * j) & 0xffff) != 0 ? j : __builtin_ctzll(same) / 16;
      x_row[j] = p.x + static_cast<int64_t>(min(m0 + 16 * from + r, M - 1)) * K + k8;
    }
    for (int base = 0; base < rank; base += 16 * NB) {
      v4f acc[4][NB] = {};
      // rows past the rank: the last one (its sums are not used)
      const uint16_t* w_row[NB];
#pragma unroll
      for (int q = 0; q < NB; ++q)
        w_row[q] = p.a_rows + static_cast<int64_t>(row0 + min(base + 16 * q + r, rank - 1)) * K + k8;
      for (int k = k0; k < k_end; k += DEPTH * step) {
        v4i xf[DEPTH][2][4], wf[DEPTH][2][NB];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
          const int kd = k + d * step < k_end ? k + d * step : k;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 4; ++j) xf[d][h][j] = *reinterpret_cast<const v4i*>(x_row[j] + kd + 32 * h);
#pragma unroll
            for (int q = 0; q < NB; ++q) wf[d][h][q] = *reinterpret_cast<const v4i*>(w_row[q] + kd + 32 * h);
          }
        }
        __builtin_amdgcn_sched_barrier(0);      // every load before the first product
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
          if (d > 0 && k + d * step >= k_end) break;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int q = 0; q < NB; ++q) acc[j][q] = mfma<F16>(wf[d][h][q], xf[d][h][j], acc[j][q]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < NB; ++q) part[wave][j][q][lane] = acc[j][q];
      __syncthreads();
      // lane l holds ranks 4 (l >> 4) + e of token l & 15
#pragma unroll
      for (int q = 0; q < NB; ++q) {
        v4f sum = part[0][wave][q][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum += part[w][wave][q][lane];
        const int rank0 = base + 16 * q + (lane >> 4) * 4;
        if (own == a && rank0 < p.t_stride)
          *reinterpret_cast<v4f*>(sums + (static_cast<int64_t>(blockIdx.y) * M + m_out) * p.t_stride + rank0) = sum;
      }
      __syncthreads();
    }
  }
}

// t from the parts of K: thread i of a thread per four ranks of a token.
template <bool F16>
__device__ inline void lora_sum(const Down& p, const float* __restrict__ sums, int parts, int64_t i) {
  const int quads = p.t_stride / 4;
  const int64_t m = i / quads;
  if (m >= p.M) return;
  const int rank0 = static_cast<int>(i - m * quads) * 4;
  // every part is read before the token's adapter is known (what an unwritten
  // one holds is not used), so that one latency covers them all
  v4f v[kMaxLoraParts];
#pragma unroll
  for (int z = 0; z < kMaxLoraParts; ++z)
    v[z] = *reinterpret_cast<const v4f*>(sums + (min(z, parts - 1) * static_cast<int64_t>(p.M) + m) * p.t_stride + rank0);
  const int a = p.index[m];
  if (a < 0 || a >= p.adapters) return;
  int row0, rank;
  p.range(a, row0, rank);
  v4f sum = v[0];
#pragma unroll
  for (int z = 1; z < kMaxLoraParts; ++z)
    if (z < parts) sum += v[z];
  const float s = p.scale[a];
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = rank0 + e < rank ? round16<F16>(s * sum[e]) : 0u;
  *reinterpret_cast<uint2*>(p.t + m * p.t_stride + rank0) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Ranks 8 * part + 2 * wave + (0, 1) of token m.
template <typename In>
__device__ inline void lora_dot(const Down& p, int64_t m, int part) {
  constexpr bool F16 = !std::is_same_v<In, uint16_t>;
  const int lane = threadIdx.x & 63;
  const int rank0 = part * 8 + (threadIdx.x >> 6) * 2;
  const int a = p.index[m];
  if (a < 0 || a >= p.adapters) return;
  int row0, rank;
  p.range(a, row0, rank);
  float sum[2] = {0.0f, 0.0f};
  if (rank0 < rank) {
    const In* x = reinterpret_cast<const In*>(p.x) + m * p.K;
    const In* w = reinterpret_cast<const In*>(p.a_rows) + static_cast<int64_t>(row0 + rank0) * p.K;
    const In* w2 = rank0 + 1 < rank ? w + p.K : w;
#pragma unroll 4
    for (int k = lane * 8; k < p.K; k += 512) {
      float xv[8], wv[8], w2v[8];
      load8(x + k, xv);
      load8(w + k, wv);
      load8(w2 + k, w2v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[0] = __builtin_fmaf(xv[i], wv[i], sum[0]);
        sum[1] = __builtin_fmaf(xv[i], w2v[i], sum[1]);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = sum[e];
      v += lane_xor<1>(v);
      v += lane_xor<2>(v);
      v += lane_xor<4>(v);
      v += lane_xor<8>(v);
      v += __shfl_xor(v, 16);
      v += __shfl_xor(v, 32);
      sum[e] = v;
    }
  }
  if (lane == 0) {
    const float s = p.scale[a];
    const uint32_t lo = rank0 < rank ? round16<F16>(s * sum[0]) : 0u;
    const uint32_t hi = rank0 + 1 < rank ? round16<F16>(s * sum[1]) : 0u;
    *reinterpret_cast<uint32_t*>(p.t + m * p.t_stride + rank0) = lo | (hi << 16);
  }
}

// The rest of the first product (DOTS: token by token, else the sum of the
// parts of K), and beside it, in the first `rows` workgroups, the rotation and
// the codes of the tokens: two kernels of a few microseconds in the time of
// one.  G = 0: the tokens are coded elsewhere.
template <typename In, bool DOTS, int G, int CPT>
__global__ __launch_bounds__(kThreads) void lora_rows_kernel(Down p, int rows, int8_t* __restrict__ xq,
                                                             float* __restrict__ xs,
                                                             const float* __restrict__ sums, int parts) {
  const int block = static_cast<int>(blockIdx.x) - rows;
  if constexpr (G != 0) {
    if (block < 0) {
      const int64_t m = blockIdx.x;
      rotate_quant_row<G, CPT>(reinterpret_cast<const In*>(p.x) + m * p.K, p.K, xq + m * p.K, xs + m);
      return;
    }
  }
  if constexpr (DOTS) {
    const int per_token = p.t_stride / 8;
    lora_dot<In>(p, block / per_token, block % per_token);
  } else {
    lora_sum<!std::is_same_v<In, uint16_t>>(p, sums, parts, static_cast<int64_t>(block) * kThreads + threadIdx.x);
  }
}

template <bool F16, int NB>
hipError_t launch_down(const Down& p, float* sums, int parts, hipStream_t stream) {
  const int tiles = (p.M + kTile - 1) / kTile;
  // Workgroups that share a tile's adapters: one, and three times as many as
  // the runs of a batch of this many adapters put into a tile on the mean; the
  // workgroups without an adapter end at once and come last in the grid.  (Each
  // adapter more in a tile costs its pass: 2000 tokens, K = 12288, rank 32, one
  // adapter a tile 13.5 us, two 19.6, four 34.5.)
  const int64_t cuts = (int64_t{3} * p.adapters * kTile + p.M - 1) / p.M;
  const int64_t most = p.adapters < kTile ? p.adapters : kTile;         // adapters a tile can hold
  const dim3 grid(static_cast<uint32_t>(tiles), static_cast<uint32_t>(parts),
                  static_cast<uint32_t>(1 + cuts < most ? 1 + cuts : most));
  if (p.K / 64 > parts * kWaves)
    hipLaunchKernelGGL((lora_down_kernel<F16, NB, 2>), grid, dim3(kWaves * 64), 0, stream, p, sums);
  else
    hipLaunchKernelGGL((lora_down_kernel<F16, NB, 1>), grid, dim3(kWaves * 64), 0, stream, p, sums);
  return hipGetLastError();
}

template <typename In, bool DOTS>
hipError_t launch_rows(const Down& p, int group, int8_t* xq, float* xs, const float* sums, int parts,
                       hipStream_t stream) {
  // group 0: coded elsewhere
  const int rows = group != 0 ? p.M : 0;
  const int64_t work = DOTS ? static_cast<int64_t>(p.M) * (p.t_stride / 8)
                            : (static_cast<int64_t>(p.M) * (p.t_stride / 4) + kThreads - 1) / kThreads;
  const dim3 grid(static_cast<uint32_t>(rows + work));
  const int slots = (p.K + kThreads * 8 - 1) / (kThreads * 8);
  auto go = [&](auto g_c, auto cpt_c) {
    hipLaunchKernelGGL((lora_rows_kernel<In, DOTS, decltype(g_c)::value, decltype(cpt_c)::value>), grid,
                       dim3(kThreads), 0, stream, p, rows, xq, xs, sums, parts);
    return hipGetLastError();
  };
  auto go_group = [&](auto g_c) {
    if (slots <= 1) return go(g_c, std::integral_constant<int, 1>{});
    if (slots <= 2) return go(g_c, std::integral_constant<int, 2>{});
    return go(g_c, std::integral_constant<int, 4>{});
  };
  if (group == 0) return go(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{});
  if (group == 128) return go_group(std::integral_constant<int, 128>{});
  return go_group(std::integral_constant<int, 256>{});
}

// Parts of K: up to two and a half workgroups a CU, and the fewest with which
// a wave has as few pieces of K as with that many.
int parts_of(int64_t M, int64_t K) {
  const int64_t tiles = (M + kTile - 1) / kTile, pieces = K / 64;
  int64_t parts = 5 * num_cus() / (2 * tiles);
  if (parts * M > kLoraSumRows) parts = kLoraSumRows / M;
  parts = parts < 1 ? 1 : parts > kMaxLoraParts ? kMaxLoraParts : parts;
  auto turns = [&](int64_t n) { return ((pieces + n - 1) / n + kWaves - 1) / kWaves; };
  while (parts > 1 && turns(parts - 1) == turns(parts)) --parts;
  return static_cast<int>(parts);
}

template <bool F16>
hipError_t launch(const Down& p, int group, int8_t* xq, float* xs, float* sums, bool dots, hipStream_t stream) {
  using In = std::conditional_t<F16, _Float16, uint16_t>;
  if (!rotate_by_row(p.M, p.K)) {
    const hipError_t e = F16 ? launch_rotate_quant_f16(p.x, p.M, p.K, group, xq, xs, stream)
                             : launch_rotate_quant(p.x, p.M, p.K, group, xq, xs, stream);
    if (e != hipSuccess) return e;
    group = 0;
  }
  if (dots) return launch_rows<In, true>(p, group, xq, xs, nullptr, 0, stream);
  const int parts = parts_of(p.M, p.K);
  const hipError_t e = p.max_rank <= 16   ? launch_down<F16, 1>(p, sums, parts, stream)
                       : p.max_rank <= 32 ? launch_down<F16, 2>(p, sums, parts, stream)
                                          : launch_down<F16, 4>(p, sums, parts, stream);
  if (e != hipSuccess) return e;
  return launch_rows<In, false>(p, group, xq, xs, sums, parts, stream);
}

}  // namespace

hipError_t launch_lora_down(const uint16_t* x, int64_t M, int64_t K, int group, bool f16, int8_t* xq, float* xs,
                            const uint16_t* a, int64_t ranks, const float* scale, const int32_t* offsets,
                            int64_t adapters, const int32_t* index, int64_t max_rank, uint16_t* t, int64_t t_stride,
                            float* sums, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  const Down p{x, a, scale, offsets, index, t, static_cast<int>(M), static_cast<int>(K), static_cast<int>(ranks),
               static_cast<int>(adapters), static_cast<int>(max_rank), static_cast<int>(t_stride)};
  const bool dots = lora_by_token(M, adapters);
  return f16 ? launch<true>(p, group, xq, xs, sums, dots, stream) : launch<false>(p, group, xq, xs, sums, dots, stream);
}

}  // namespace convrot
