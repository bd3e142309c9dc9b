// rotate_block.hpp -- the token-block form of rotate + quantize, for the
// kernels that run it: rotate_quant.hip, and lora.hip beside the adapters' sums.
#pragma once

#include "convrot_internal.hpp"
#include "rotate_device.hpp"

namespace convrot {
namespace {

// ---------------------------------------------------------------- token blocks
// Activation path for K <= 32768.  The workgroup's rows are staged through
// LDS by direct-to-LDS loads (each wave moves its own 32 blocks, 1 KB of
// consecutive input per instruction), and two lanes hold one 128-element
// block in registers: lane 2b + h takes elements [64h, 64h + 64) of block b.
// Stages h' = 1..32 stay in the lane; stage 64 pairs the two lanes (one DPP
// exchange); for g = 256 stage 128 pairs the same half of blocks b and b ^ 1
// (lanes two apart).  A lane that must keep a - b while it holds b computes
// RN(b - a) = -RN(a - b) with the same fma its partner uses for RN(a + b) and
// carries the sign into the final multiply (rounding to nearest is
// symmetric), so every add is the one the sequential butterfly does and the
// values match it up to the sign of an exact zero (a = b gives +0 where the
// butterfly has +0 too, turned into -0 by the negated constant), which neither
// the row maximum nor the code can see.  (The weight unpacking of rotate_quant.hip,
// whose output is the values themselves, uses RN(own * sgn + partner) instead.)
// With
// 64 values per lane a wave needs about 94 registers, so twice as many waves
// share a SIMD as with a whole block per lane (4608 x 3072: 13.2 -> 11.7 us;
// 4608 x 12288: 43.5 -> 36.8 us; identical codes and scales).  The codes go
// back through LDS so that every wave stores its own blocks as 16-byte
// chunks of consecutive codes; the only workgroup barrier completes the
// per-row maxima (rows cross wave boundaries).
//
// Codes: rne(v / s) with the quotient correctly rounded, computed with a
// reciprocal and two fused multiply-adds instead of a full division per
// element (rows whose scale is too small for a normal reciprocal divide).
constexpr int kBlockElems = 128;
constexpr int kMaxBlocksPerWg = 256;                 // two lanes per block: 512 lanes
constexpr int kMaxBlockK = kMaxBlocksPerWg * kBlockElems;

// v[i] <- RN(v[i] + sgn * v[i] of the partner lane) for all 64 values, one
// v_fmac_f32 with a DPP source per value (the partner is the neighbour lane,
// P = 0, or the lane two away, P = 1, inside each quad).  Eight values per
// asm block; each block opens with the two wait states a DPP read needs after
// a VALU write of its source (inside a block no instruction reads what another
// of the block wrote).
template <int P>
__device__ inline void dpp_fmac8(float (&v)[64], float sgn) {
#define CONVROT_DPP8(i0, PERM)                                                                          \
  asm volatile("s_nop 1\n\t"                                                                            \
               "v_fmac_f32_dpp %0, %0, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                      \
               "v_fmac_f32_dpp %1, %1, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                      \
               "v_fmac_f32_dpp %2, %2, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                      \
               "v_fmac_f32_dpp %3, %3, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                      \
               "v_fmac_f32_dpp %4, %4, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                      \
               "v_fmac_f32_dpp %5, %5, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                      \
               "v_fmac_f32_dpp %6, %6, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                      \
               "v_fmac_f32_dpp %7, %7, %8 " PERM " row_mask:0xf bank_mask:0xf"                            \
               : "+v"(v[i0]), "+v"(v[i0 + 1]), "+v"(v[i0 + 2]), "+v"(v[i0 + 3]), "+v"(v[i0 + 4]),         \
                 "+v"(v[i0 + 5]), "+v"(v[i0 + 6]), "+v"(v[i0 + 7])                                         \
               : "v"(sgn))
#pragma unroll
  for (int i = 0; i < 64; i += 8) {
    if constexpr (P == 0) CONVROT_DPP8(i, "quad_perm:[1,0,3,2]");
    else CONVROT_DPP8(i, "quad_perm:[2,3,0,1]");
  }
#undef CONVROT_DPP8
}

// What rotq_block_kernel is launched with for K <= kMaxBlockK.
struct BlockGrid {
  int rows_per_wg, threads;
  uint32_t wgs, bpr_inv;
  size_t lds;
};
inline BlockGrid block_grid(int64_t M, int64_t K) {
  // Rows per workgroup: as many as fit (256 blocks, 512 lanes), but no more
  // than an even share of two workgroups per CU, so that every CU gets the
  // same work when the batch is small (M = 4608, K = 3072: 512 workgroups of
  // 9 rows instead of 461 of 10, of which 205 CUs would run two).  Where
  // that share is two rows, one row per workgroup is taken when it puts
  // fewer rows on the busiest CU (M = 701, K = 3072: 701 workgroups, at
  // most 3 rows per CU instead of 4; 5.7 us instead of 6.7).  Two lanes
  // per block, threads rounded up to whole waves; LDS holds 256 bytes per
  // block, sized at launch (K = 12288: 48 KB, three workgroups per CU).
  const int fit = kMaxBlocksPerWg / static_cast<int>(K / kBlockElems);
  const int64_t cus = num_cus();
  int64_t share = (M + 2 * cus - 1) / (2 * cus);
  if (share == 2 && (M + cus - 1) / cus < 2 * (((M + 1) / 2 + cus - 1) / cus)) share = 1;
  BlockGrid g;
  g.rows_per_wg = static_cast<int>(share < fit ? share : fit);
  g.wgs = static_cast<uint32_t>((M + g.rows_per_wg - 1) / g.rows_per_wg);
  const int blocks = g.rows_per_wg * static_cast<int>(K / kBlockElems);
  g.threads = (2 * blocks + 63) / 64 * 64;
  g.lds = static_cast<size_t>(blocks) * 256;
  const uint32_t bpr = static_cast<uint32_t>(K / kBlockElems);
  g.bpr_inv = (65536u + bpr - 1u) / bpr;
  return g;
}

// Beside: nothing, or the work of the workgroups behind the BlockGrid's, whose
// call operator takes a workgroup's index and says whether it was its own.
template <int G, typename In16, class... Beside>
__global__ __launch_bounds__(512) void rotq_block_kernel(
    const In16* __restrict__ x, int64_t M, int K, int rows_per_wg, uint32_t bpr_inv,
    int8_t* __restrict__ q, float* __restrict__ scale, Beside... beside) {
  if constexpr (sizeof...(Beside) != 0)
    if ((beside(blockIdx.x) || ...)) return;
  // the input tile, 256 bytes per block of the workgroup (sized at launch)
  extern __shared__ __attribute__((aligned(16))) uint4 tile[];
  __shared__ uint32_t row_amax[kMaxBlocksPerWg];
  const int tid = threadIdx.x;
  const int bpr = K / kBlockElems;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_per_wg;
  const int rows = static_cast<int>(min(static_cast<int64_t>(rows_per_wg), M - row0));
  const int nblk = rows * bpr;

  if (tid < rows_per_wg) row_amax[tid] = 0u;
  __syncthreads();
  // wave w loads its own 32 blocks: instruction u fills LDS slots
  // p = 512 w + 64 u + lane, slot p holding chunk (p & 15) ^ (b & 15) of
  // block b = p >> 4
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wchunks = max(0, min(32, nblk - 32 * wave)) * 16;
  const char* wbase = reinterpret_cast<const char*>(x + row0 * K) + static_cast<int64_t>(wave) * 32 * 256;
  uint32_t loff[4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    loff[r] = static_cast<uint32_t>(((lane >> 4) * 16 + ((lane & 15) ^ ((4 * r + (lane >> 4)) & 15))) * 16);
  if (wchunks == 512) {
    // a whole wave: eight unconditional loads, each a scalar base (kept
    // opaque, so that it stays in scalar registers) plus the lane's offset
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      asm volatile("" : "+v"(loff[u & 3]));
      const char* base = wbase + u * 1024;
      asm volatile("" : "+s"(base));
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(base + loff[u & 3]),
                                       (__attribute__((address_space(3))) void*)(tile + 512 * wave + 64 * u), 16, 0, 0);
    }
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (u * 64 >= wchunks) break;
      if (64 * u + lane < wchunks) {
        asm volatile("" : "+v"(loff[u & 3]));
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(wbase + u * 1024 + loff[u & 3]),
                                         (__attribute__((address_space(3))) void*)(tile + 512 * wave + 64 * u), 16, 0, 0);
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  const int b = tid >> 1, half = tid & 1;
  const bool active = b < nblk;
  // b / bpr as (b * bpr_inv) >> 16 with bpr_inv = ceil(2^16 / bpr), exact
  // for b < 256 and bpr <= 256 (checked for every pair), instead of an
  // integer division
  const int lrow = active ? static_cast<int>(__umul24(static_cast<uint32_t>(b), bpr_inv) >> 16) : 0;
  const bool row_first = b == lrow * bpr;
  float v[64];
  float amax = 0.0f;
  // the normalisation constant times the sign this lane's values carry
  float c = RotScale<G>::value;
  if (active) {
#pragma unroll
    for (int jj = 0; jj < 8; ++jj) {
      const uint4 w = tile[b * 16 + ((8 * half + jj) ^ (b & 15))];
      v[8 * jj + 0] = in_lo<In16>(w.x); v[8 * jj + 1] = in_hi<In16>(w.x);
      v[8 * jj + 2] = in_lo<In16>(w.y); v[8 * jj + 3] = in_hi<In16>(w.y);
      v[8 * jj + 4] = in_lo<In16>(w.z); v[8 * jj + 5] = in_hi<In16>(w.z);
      v[8 * jj + 6] = in_lo<In16>(w.w); v[8 * jj + 7] = in_hi<In16>(w.w);
    }
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) {
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        if ((i & h) == 0) {
          const float a = v[i], d = v[i + h];
          v[i] = a + d;
          v[i + h] = a - d;
        }
      }
    }
    {  // stage 64: the lower half keeps RN(a + b), the upper RN(b - a)
      const float sgn = half ? -1.0f : 1.0f;
      c = half ? -c : c;
      dpp_fmac8<0>(v, sgn);
    }
    if constexpr (G == 256) {
      // stage 128: the same half of blocks b (even) and b ^ 1, two lanes
      // apart; both carry the same sign, so the odd block's RN(v - p)
      // flips it
      const bool odd = (b & 1) != 0;
      const float sgn = odd ? -1.0f : 1.0f;
      c = odd ? -c : c;
      dpp_fmac8<1>(v, sgn);
    }
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      v[i] = v[i] * c;
      amax = fmaxf(amax, fabsf(v[i]));
    }
    // one LDS atomic per block, or per two blocks when rows hold an even
    // number of blocks (a block pair then never straddles two rows): the
    // atomics of one row all hit one LDS word and are served one at a time
    amax = fmaxf(amax, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(amax), 0xB1, 0xF, 0xF, false)));
    const bool pairs = (bpr & 1) == 0;
    if (pairs)
      amax = fmaxf(amax, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(amax), 0x4E, 0xF, 0xF, false)));
    if ((tid & (pairs ? 3 : 1)) == 0)
      atomicMax(&row_amax[lrow], __float_as_uint(amax));   // amax >= 0: bit order = value order
  }
  __syncthreads();

  // codes -> LDS (block b's 8 code chunks at j ^ ((b >> 1) & 7); this lane
  // writes chunks 4 * half .. 4 * half + 3), then out
  uint4* codes = tile;
  if (active) {
    const float s = __uint_as_float(row_amax[lrow]) / 127.0f;
    if (row_first && half == 0) scale[row0 + lrow] = s;
    const float r = 1.0f / s;
    char* out = reinterpret_cast<char*>(codes) + b * 128;
    if (r < 1e30f) {
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        uint32_t wd[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t t[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float val = v[16 * jj + 4 * d + e];
            const float q0 = val * r;
            const float rem = __builtin_fmaf(-q0, s, val);
            const float q1 = __builtin_fmaf(rem, r, q0);
            t[e] = __float_as_uint(q1 + 12582912.0f);
          }
          const uint32_t lo = __builtin_amdgcn_perm(t[1], t[0], 0x0c0c0400u);
          const uint32_t hi = __builtin_amdgcn_perm(t[3], t[2], 0x0c0c0400u);
          wd[d] = lo | (hi << 16);
        }
        reinterpret_cast<uint4*>(out)[(4 * half + jj) ^ ((b >> 1) & 7)] = make_uint4(wd[0], wd[1], wd[2], wd[3]);
      }
    } else {
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        uint32_t wd[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t packed = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            packed |= (static_cast<uint32_t>(quant_code(v[16 * jj + 4 * d + e], s)) & 0xffu) << (8 * e);
          wd[d] = s != 0.0f ? packed : 0u;
        }
        reinterpret_cast<uint4*>(out)[(4 * half + jj) ^ ((b >> 1) & 7)] = make_uint4(wd[0], wd[1], wd[2], wd[3]);
      }
    }
  }
  // this wave stores its own 32 blocks' codes
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  uint4* dstq = reinterpret_cast<uint4*>(q + row0 * K);
  const int wcodes = wchunks / 2;
  if (wcodes == 256) {
    // a whole wave: piece i of lane l is chunk l & 7 of block
    // 32 wave + (l >> 3) + 8 i, stored at chunk (l & 7) ^ (l >> 4) for even
    // i and ^ (l >> 4) ^ 4 for odd i: two lane offsets and immediates
    const char* cb = reinterpret_cast<const char*>(codes);
    const int o = (32 * wave + (lane >> 3)) * 128 + (((lane & 7) ^ (lane >> 4)) << 4);
    uint4* d = dstq + 256 * wave + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) d[64 * i] = *reinterpret_cast<const uint4*>(cb + (o ^ (64 * (i & 1))) + 1024 * i);
  } else {
    for (int cc = 256 * wave + lane; cc < 256 * wave + wcodes; cc += 64) {
      const int bb = cc >> 3, j = cc & 7;
      dstq[cc] = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(codes) + bb * 128)[j ^ ((bb >> 1) & 7)];
    }
  }
}

}  // namespace
}  // namespace convrot
