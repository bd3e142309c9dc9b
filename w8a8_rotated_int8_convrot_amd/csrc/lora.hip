// lora.hip -- the first product of the low-rank adapters beside the layer:
//   t[m][r] = scale[a] * sum_k A[offsets[a] + r][k] * x[m][k],  a = index[m]
// for r below the rank of a, 0 up to the row's stride; tokens without an
// adapter are skipped (nobody reads their rows).  x is the layer's own input,
// neither rotated nor coded.  The sum is held in fp32.  The second product
// takes it as it is where it runs on the vector unit (token by token); on the
// matrix units, whose operands have 16 bits, as two parts, the nearest value of
// the io type and the nearest to what that leaves: one part alone would move
// the result by up to half a step of sum_r |t_r b_r|, however much of that
// cancels.  Two are off by 2^-16 of each t_r in bf16 and 2^-22 in fp16 (there
// also by 2^-39 of the largest of its 32 ranks).  fp16 parts are those of t scaled by a
// power of two that takes the largest of 32 ranks to [2^14, 2^15), so that
// neither its range nor its smallest step meets a t of fp32.
//
// lora_down_kernel: a workgroup takes 64 tokens, 16 a wave, and a part of K
// (gridDim.y of them fill the chip).  Pieces of 64 elements of K, 64 token rows
// and 16 NB rows of the adapter, stream through a ring of LDS stages by
// direct-to-LDS loads of whole 128-byte lines, several pieces ahead, and each
// wave multiplies its tokens with the shared adapter rows from there
// (v_mfma_*_16x16x32, ranks x tokens).  A wave's token rows are its own, so a
// wave without the adapter loads and multiplies none.  What bounds it is what a
// CU can draw from L2 and the latency of the draw.  The parts of K are summed by
// lora_sum in a fixed order.  The adapters met among the tokens are taken one
// after another, or, where the tiles would leave the chip idle, dealt out over
// gridDim.z workgroups.
//
// lora_dot, for few tokens with adapters of their own: a wave per token and two
// of its ranks, each lane a plain dot product over its part of K.
#include <type_traits>

#include "convrot_internal.hpp"
#include "rotate_block.hpp"
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
  float* factor;
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

// v as the nearest value of the io type and the nearest to the rest (none of an
// infinity)
template <bool F16>
__device__ inline void split16(float v, uint32_t& first, uint32_t& second) {
  using H = std::conditional_t<F16, _Float16, __bf16>;
  const H h = static_cast<H>(v);
  const float rest = v - static_cast<float>(h);
  first = __builtin_bit_cast(uint16_t, h);
  second = __builtin_bit_cast(uint16_t, static_cast<H>(fabsf(rest) <= 0x1.fffffep127f ? rest : 0.0f));
}

typedef __attribute__((address_space(3))) void lds_void_t;
typedef const __attribute__((address_space(1))) void glb_void_t;

// 16-byte chunk `chunk` of LDS row `row` (128 bytes), swizzled so that the rows
// and chunks one fragment read takes fall into distinct banks
__device__ inline int chunk_at(int row, int chunk) { return row * 128 + ((chunk ^ ((row >> 1) & 7)) << 4); }

// sums [gridDim.y][M][t_stride] fp32
template <bool F16, int NB, int STAGES>
__global__ __launch_bounds__(kWaves * 64) void lora_down_kernel(Down p, float* __restrict__ sums) {
  constexpr int kXBytes = kTile * 128, kStage = kXBytes + NB * 16 * 128;
  constexpr int kALoads = NB > 2 ? NB / 2 : 1;      // of a wave (with one block two waves load each row twice)
  __shared__ __attribute__((aligned(16))) char lds[STAGES * kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15;
  const int m0 = blockIdx.x * kTile;
  const int M = p.M, K = p.K;
  const int mine = p.index[min(m0 + lane, M - 1)];
  // this part's pieces
  const int pieces = K / 64, per_part = (pieces + gridDim.y - 1) / gridDim.y;
  const int first = blockIdx.y * per_part, n = min(pieces - first, per_part);
  // a load fills eight LDS rows: lane -> row 8 i + (lane >> 3), stored chunk
  // lane & 7
  const char* x_base = reinterpret_cast<const char*>(p.x + static_cast<int64_t>(m0) * K) + static_cast<int64_t>(first) * 128;
  uint32_t x_off[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int row = 16 * wave + 8 * j + (lane >> 3);
    x_off[j] = static_cast<uint32_t>(min(m0 + row, M - 1) - m0) * (2u * static_cast<uint32_t>(K)) +
               (((lane & 7) ^ ((row >> 1) & 7)) << 4);
  }
  const int m_out = m0 + 16 * wave + r;
  const int own = m_out < M ? p.index[m_out] : -1;

  uint64_t left = __ballot(m0 + lane < M && mine >= 0 && mine < p.adapters);
  for (int turn = 0; left != 0; ++turn) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    const uint64_t same = __ballot(m0 + lane < M && mine == a);
    left &= ~same;
    if (turn % gridDim.z != blockIdx.z) continue;
    const bool here = (same >> (16 * wave) & 0xffff) != 0;
    int row0, rank;
    p.range(a, row0, rank);
    for (int base = 0; base < rank; base += 16 * NB) {
      const char* w_base = reinterpret_cast<const char*>(p.a_rows + static_cast<int64_t>(row0 + base) * K) +
                           static_cast<int64_t>(first) * 128;
      // rows past the rank: the last one (its sums are not used)
      uint32_t w_off[kALoads];
      int w_dst[kALoads];
#pragma unroll
      for (int j = 0; j < kALoads; ++j) {
        const int i = NB == 1 ? (wave & 1) : wave * kALoads + j;
        const int row = 8 * i + (lane >> 3);
        w_off[j] = static_cast<uint32_t>(min(row, rank - 1 - base)) * (2u * static_cast<uint32_t>(K)) +
                   (((lane & 7) ^ ((row >> 1) & 7)) << 4);
        w_dst[j] = kXBytes + i * 1024;
      }
      auto issue = [&](int piece, int stage, auto with_x_c) {
        const int64_t k0 = static_cast<int64_t>(min(piece, n - 1)) * 128;
        char* st = lds + stage * kStage;
        if constexpr (decltype(with_x_c)::value) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            __builtin_amdgcn_global_load_lds((glb_void_t*)(x_base + k0 + x_off[j]),
                                             (lds_void_t*)(st + (2 * wave + j) * 1024), 16, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < kALoads; ++j)
          __builtin_amdgcn_global_load_lds((glb_void_t*)(w_base + k0 + w_off[j]), (lds_void_t*)(st + w_dst[j]), 16, 0, 0);
      };
      v4f acc[NB] = {};
      // one barrier a piece: it has landed everywhere, and everyone is done with
      // the stage that is filled next; pieces past the end fill stages that are
      // not read
      auto stream = [&](auto with_x_c) {
        constexpr int kLoads = kALoads + (decltype(with_x_c)::value ? 2 : 0);
#pragma unroll
        for (int d = 0; d < STAGES - 1; ++d) issue(d, d, with_x_c);
        for (int i = 0; i < n; ++i) {
          asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STAGES - 2) * kLoads) : "memory");
          issue(i + STAGES - 1, (i + STAGES - 1) % STAGES, with_x_c);
          if constexpr (decltype(with_x_c)::value) {
            const char* st = lds + (i % STAGES) * kStage;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const v4i xf = *reinterpret_cast<const v4i*>(st + chunk_at(16 * wave + r, 4 * h + (lane >> 4)));
#pragma unroll
              for (int q = 0; q < NB; ++q) {
                const v4i wf = *reinterpret_cast<const v4i*>(st + kXBytes + chunk_at(16 * q + r, 4 * h + (lane >> 4)));
                acc[q] = mfma<F16>(wf, xf, acc[q]);
              }
            }
          }
        }
      };
      if (here) stream(std::true_type{});
      else stream(std::false_type{});
      // lane l holds ranks 4 (l >> 4) + e of token l & 15
      if (own == a) {
#pragma unroll
        for (int q = 0; q < NB; ++q) {
          const int rank0 = base + 16 * q + (lane >> 4) * 4;
          if (rank0 < p.t_stride)
            *reinterpret_cast<v4f*>(sums + (static_cast<int64_t>(blockIdx.y) * M + m_out) * p.t_stride + rank0) = acc[q];
        }
      }
      // the ring is quiet before it starts again
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
  }
}

// t from the parts of K: thread i of a thread per four ranks of a token.  The
// eight threads of 32 ranks are neighbours in a wave (t_stride is a multiple of
// 32), which has read all it needs of their words before it writes there.
template <bool F16>
__device__ inline void lora_sum(const Down& p, float* sums, int parts, int64_t i) {
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
  float t[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) t[e] = rank0 + e < rank ? s * sum[e] : 0.0f;
  float* words = sums + m * p.t_stride + rank0 / 32 * 32 + (rank0 & 31) / 2;
  if constexpr (F16) {
    float most = 0.0f;            // of the finite ones
#pragma unroll
    for (int e = 0; e < 4; ++e) most = fabsf(t[e]) <= 0x1.fffffep127f ? fmaxf(most, fabsf(t[e])) : most;
    most = fmaxf(most, lane_xor<1>(most));
    most = fmaxf(most, lane_xor<2>(most));
    most = fmaxf(most, lane_xor<4>(most));
    // 2^(14 - e) for most in [2^e, 2^(e+1)); below 2^-100 nothing is left that fp16 could show
    const int e = max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -100);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
#pragma unroll
    for (int q = 0; q < 4; ++q) t[q] *= up;
    if ((rank0 & 31) == 0)
      p.factor[static_cast<int64_t>(rank0 / 32) * p.M + m] = __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
  }
  uint32_t first[4], second[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) split16<F16>(t[e], first[e], second[e]);
  *reinterpret_cast<uint2*>(words) = make_uint2(first[0] | (first[1] << 16), first[2] | (first[3] << 16));
  *reinterpret_cast<uint2*>(words + 16) = make_uint2(second[0] | (second[1] << 16), second[2] | (second[3] << 16));
}

// Ranks 8 * part + 2 * wave + (0, 1) of token m, into t [M, t_stride].
template <typename In>
__device__ inline void lora_dot(const Down& p, float* t, int64_t m, int part) {
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
    *reinterpret_cast<float2*>(t + m * p.t_stride + rank0) =
        make_float2(rank0 < rank ? s * sum[0] : 0.0f, rank0 + 1 < rank ? s * sum[1] : 0.0f);
  }
}

// The rest of the first product (DOTS: token by token, else the sum of the
// parts of K), and beside it, in the first `rows` workgroups, the rotation and
// the codes of the tokens: two kernels of a few microseconds in the time of
// one.  G = 0: the tokens are coded elsewhere.
template <typename In, bool DOTS, int G, int CPT>
__global__ __launch_bounds__(kThreads) void lora_rows_kernel(Down p, int rows, int8_t* __restrict__ xq,
                                                             float* __restrict__ xs, float* sums, int parts) {
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
    lora_dot<In>(p, sums, block / per_token, block % per_token);
  } else {
    lora_sum<!std::is_same_v<In, uint16_t>>(p, sums, parts, static_cast<int64_t>(block) * kThreads + threadIdx.x);
  }
}

// The same for larger batches: behind the wgs workgroups that rotate and code
// by token blocks, others sum, their latency under the coding (a call of 1000 x
// 4096 x 4096, rank 16: 41.4 -> 38.9 us; 2000 x 12288 x 4096, rank 32: 160 -> 158).
template <bool F16>
struct SumsBeside {
  Down p;
  float* sums;
  int parts;
  uint32_t wgs;
  __device__ bool operator()(uint32_t wg) const {
    if (wg < wgs) return false;
    lora_sum<F16>(p, sums, parts, static_cast<int64_t>(wg - wgs) * blockDim.x + threadIdx.x);
    return true;
  }
};

template <bool F16, int NB>
hipError_t launch_down(const Down& p, float* sums, int parts, hipStream_t stream) {
  const int tiles = (p.M + kTile - 1) / kTile;
  // Workgroups that share a tile's adapters: one, and three times as many as
  // the runs of a batch of this many adapters put into a tile on the mean; the
  // workgroups without an adapter end at once and come last in the grid.  (Each
  // adapter more in a tile costs its pass: 2000 tokens, K = 12288, rank 32, one
  // adapter a tile 11.3 us, two 16.7, runs of 48 adapters 23.)
  const int64_t cuts = (int64_t{3} * p.adapters * kTile + p.M - 1) / p.M;
  const int64_t most = p.adapters < kTile ? p.adapters : kTile;         // adapters a tile can hold
  const dim3 grid(static_cast<uint32_t>(tiles), static_cast<uint32_t>(parts),
                  static_cast<uint32_t>(1 + cuts < most ? 1 + cuts : most));
  // two workgroups a CU
  constexpr int kStages = NB == 4 ? 4 : NB == 2 ? 6 : 7;
  hipLaunchKernelGGL((lora_down_kernel<F16, NB, kStages>), grid, dim3(kWaves * 64), 0, stream, p, sums);
  return hipGetLastError();
}

template <typename In, bool DOTS>
hipError_t launch_rows(const Down& p, int group, int8_t* xq, float* xs, float* sums, int parts,
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
// a workgroup has as few pieces of K as with that many (every part has some).
int parts_of(int64_t M, int64_t K) {
  const int64_t tiles = (M + kTile - 1) / kTile, pieces = K / 64;
  int64_t parts = 5 * num_cus() / (2 * tiles);
  if (parts * M > kLoraSumRows) parts = kLoraSumRows / M;
  parts = parts < 1 ? 1 : parts > kMaxLoraParts ? kMaxLoraParts : parts;
  const int64_t per_part = (pieces + parts - 1) / parts;
  return static_cast<int>((pieces + per_part - 1) / per_part);
}

template <typename In, bool F16>
hipError_t launch_codes(const Down& p, int group, int8_t* xq, float* xs, float* sums, int parts,
                        hipStream_t stream) {
  const BlockGrid g = block_grid(p.M, p.K);
  const int64_t work = static_cast<int64_t>(p.M) * (p.t_stride / 4);
  const uint32_t sum_wgs = static_cast<uint32_t>((work + g.threads - 1) / g.threads);
  auto go = [&](auto g_c) {
    hipLaunchKernelGGL((rotq_block_kernel<decltype(g_c)::value, In, SumsBeside<F16>>), dim3(g.wgs + sum_wgs),
                       dim3(g.threads), g.lds, stream, reinterpret_cast<const In*>(p.x), static_cast<int64_t>(p.M), p.K,
                       g.rows_per_wg, g.bpr_inv, xq, xs, SumsBeside<F16>{p, sums, parts, g.wgs});
    return hipGetLastError();
  };
  return group == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 256>{});
}

template <bool F16>
hipError_t launch(const Down& p, int group, int8_t* xq, float* xs, float* sums, bool dots, hipStream_t stream) {
  using In = std::conditional_t<F16, _Float16, uint16_t>;
  // larger batches are coded by token blocks, beside the sums where there are
  // any and rows fit
  const bool blocks = !rotate_by_row(p.M, p.K) && !dots && p.K <= kMaxBlockK;
  if (!rotate_by_row(p.M, p.K) && !blocks) {
    const hipError_t e = F16 ? launch_rotate_quant_f16(p.x, p.M, p.K, group, xq, xs, stream)
                             : launch_rotate_quant(p.x, p.M, p.K, group, xq, xs, stream);
    if (e != hipSuccess) return e;
    group = 0;
  }
  if (dots) return launch_rows<In, true>(p, group, xq, xs, sums, 0, stream);
  const int parts = parts_of(p.M, p.K);
  const hipError_t e = p.max_rank <= 16   ? launch_down<F16, 1>(p, sums, parts, stream)
                       : p.max_rank <= 32 ? launch_down<F16, 2>(p, sums, parts, stream)
                                          : launch_down<F16, 4>(p, sums, parts, stream);
  if (e != hipSuccess) return e;
  if (blocks) return launch_codes<In, F16>(p, group, xq, xs, sums, parts, stream);
  return launch_rows<In, false>(p, group, xq, xs, sums, parts, stream);
}

}  // namespace

hipError_t launch_lora_down(const uint16_t* x, int64_t M, int64_t K, int group, bool f16, int8_t* xq, float* xs,
                            const uint16_t* a, int64_t ranks, const float* scale, const int32_t* offsets,
                            int64_t adapters, const int32_t* index, int64_t max_rank, uint16_t* t, int64_t t_stride,
                            float* sums, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  const Down p{x, a, scale, offsets, index, reinterpret_cast<float*>(t), static_cast<int>(M), static_cast<int>(K), static_cast<int>(ranks),
               static_cast<int>(adapters), static_cast<int>(max_rank), static_cast<int>(t_stride)};
  const bool dots = lora_by_token(M, adapters, max_rank);
  return f16 ? launch<true>(p, group, xq, xs, sums, dots, stream) : launch<false>(p, group, xq, xs, sums, dots, stream);
}

}  // namespace convrot
