// rotate_quant.hip -- group-wise Walsh-Hadamard rotation + int8 quantization
// for gfx950.
//
// What is computed (page "int8 Compute", InvokeAI docs, opening section: a
// layer's activation is rotated, then given int8 codes with one scale per
// token; its weight holds int8 codes with a single tensor scale; the rotation
// works in groups, "What stays on the default path"):
//   v      = x_row rotated block by block by H_g / sqrt(g)
//   scale  = max |v| / 127  (per token for activations, one for a weight)
//   code   = clamp(rne(v / scale), -127, 127), 0 where scale == 0
// The rotation is the fp32 radix-2 butterfly with half-span h = 1, 2, ...,
// g/2 ((a, b) -> (a + b, a - b)) followed by one multiply by the float nearest
// to 1/sqrt(g).  Every add happens in that order on the GPU too, so the codes
// are bit-identical to a sequential evaluation of the same butterfly.
//
// Row kernel (small batches, weights, rows past 32768 elements; the
// token-block kernel below has its own layout): one workgroup of 256 threads
// per row.  A thread owns
// up to CPT chunks of 8 consecutive elements (16-byte bf16 loads, 8-byte code
// stores, both coalesced across the wave); chunk c of a segment of
// 256 * 8 * CPT elements sits in thread c % 256.  Stages h = 1, 2, 4 stay inside a thread; stage h = 8 * 2^t pairs
// thread lanes whose index differs in bit t, so a g-group spans g/8
// consecutive lanes of one wavefront and the exchange is a lane shuffle.
// Rows of up to 256 * 8 * kMaxChunksPerThread elements are rotated once and
// held in registers; longer rows are rotated twice (absmax pass, then code pass),
// which gives the same values because the arithmetic is deterministic.
#include "convrot_internal.hpp"
#include "rotate_block.hpp"
#include "rotate_device.hpp"

namespace convrot {
namespace {

constexpr int kMaxChunksPerThread = 6;   // rows up to 12288 elements are rotated once

enum Mode { kActQuant = 0, kWeightAbsmax = 1, kWeightQuant = 2 };

template <int G, int CPT, typename In, int MODE>
__global__ __launch_bounds__(kThreads) void rotate_rows_kernel(
    const In* __restrict__ x, int64_t K, int8_t* __restrict__ q, float* __restrict__ scale,
    uint32_t* __restrict__ amax_cell) {
  constexpr int kSegment = kThreads * 8 * CPT;
  const int64_t row = blockIdx.x;
  const In* xr = x + row * K;
  const int tid = threadIdx.x;
  const int lane_in_group = tid % (G / 8);
  const int nseg = static_cast<int>((K + kSegment - 1) / kSegment);

  // Chunk slots past the row end are skipped lane by lane.  K is a multiple
  // of G, so a g-group is either wholly inside the row or wholly outside,
  // and the lane exchange of a valid group only reads valid lanes.
  float v[CPT][8];
  float amax = 0.0f;

  // absmax pass (for one-segment rows the rotated values stay in registers)
  for (int seg = 0; seg < nseg; ++seg) {
    const int64_t base = static_cast<int64_t>(seg) * kSegment;
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int64_t e = base + (static_cast<int64_t>(j) * kThreads + tid) * 8;
      if (e < K) load8(xr + e, v[j]);
    }
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int64_t e = base + (static_cast<int64_t>(j) * kThreads + tid) * 8;
      if (e < K) {
        rotate_chunk<G>(v[j], lane_in_group);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[j][i]));
      }
    }
  }

  if (MODE == kWeightAbsmax) {
    const float m = block_max(amax);
    if (tid == 0) atomicMax(amax_cell, __float_as_uint(m));  // m >= 0: bit order = value order
    return;
  }

  float s;
  if (MODE == kActQuant) {
    s = block_max(amax) / 127.0f;
    if (tid == 0) scale[row] = s;
  } else {
    s = __uint_as_float(*amax_cell) / 127.0f;
    if (row == 0 && tid == 0) scale[0] = s;
  }

  int8_t* qr = q + row * K;
  for (int seg = 0; seg < nseg; ++seg) {
    const int64_t base = static_cast<int64_t>(seg) * kSegment;
    if (nseg > 1) {
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        const int64_t e = base + (static_cast<int64_t>(j) * kThreads + tid) * 8;
        if (e < K) load8(xr + e, v[j]);
      }
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        const int64_t e = base + (static_cast<int64_t>(j) * kThreads + tid) * 8;
        if (e < K) rotate_chunk<G>(v[j], lane_in_group);
      }
    }
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int64_t e = base + (static_cast<int64_t>(j) * kThreads + tid) * 8;
      if (e < K) *reinterpret_cast<uint2*>(qr + e) = pack8(v[j], s);
    }
  }
}

// ---------------------------------------------------------------- token blocks
// (rotate_block.hpp)
constexpr int64_t kSmallBatchElems = int64_t{1} << 21;

__global__ void zero_word_kernel(uint32_t* p) { *p = 0u; }

// ---------------------------------------------------------------- default path
// Unpacking of a rotated int8 weight for the default (dequantizing) path
// (page "int8 Compute", "What stays on the default path": such layers keep
// unpacking their weights): every row is dequantized (s * q in fp32) and
// rotated back by R, which is its own inverse (symmetric and orthogonal), so
// the same butterfly in the same order applies; the result is rounded to
// bf16 or fp16.  Two lanes per 128-element block, as in the token-block
// kernel: lane 2b + h dequantizes and rotates elements [64h, 64h + 64) of
// block b (blocks counted over the whole row-major weight), stages 1..32 in
// the lane, stage 64 by one DPP exchange, stage 128 (g = 256) with the same
// half of block b ^ 1.  Both lanes of an exchange run RN(own * sgn + partner),
// sgn = +1 where a + b is kept and -1 where the lane holds b and keeps a - b,
// so every value, zeros' signs included, is the sequential butterfly's.  No
// LDS and no barrier: every lane reads 64 contiguous codes and writes 128
// contiguous bytes (12288 x 3072: 30-33 us like the one-row-per-workgroup
// kernel it replaced at g = 128, 30 instead of 35 us at g = 256).
template <int G, bool OutF16>
__global__ __launch_bounds__(256) void unpack_block_kernel(
    const int8_t* __restrict__ wq, int64_t nblk, int bpr, const float* __restrict__ w_scale, int row_scale,
    uint16_t* __restrict__ out) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t b = t >> 1;
  const int half = static_cast<int>(t & 1);
  // whole blocks (and, for g = 256, whole block pairs: rows hold an even
  // number of blocks) leave together, so every exchange partner is active
  if (b >= nblk) return;
  const float s = w_scale[row_scale ? b / bpr : 0];
  const uint4* src = reinterpret_cast<const uint4*>(wq + b * 128 + 64 * half);
  float v[64];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint4 w = src[c];
    const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[16 * c + 4 * k + i] = s * static_cast<float>(static_cast<int8_t>(wd[k] >> (8 * i)));
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
  {  // stage 64: the lower lane keeps RN(a + b), the upper RN(a - b)
    const float sgn = half ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      const float p = __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v[i]), 0xB1, 0xF, 0xF, false));
      v[i] = __builtin_fmaf(v[i], sgn, p);
    }
  }
  if constexpr (G == 256) {  // stage 128: block b (even) keeps RN(a + b), b ^ 1 RN(a - b)
    const float sgn = (b & 1) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      const float p = __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v[i]), 0x4E, 0xF, 0xF, false));
      v[i] = __builtin_fmaf(v[i], sgn, p);
    }
  }
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    v[i] = v[i] * RotScale<G>::value;
    // fp16 output: keep the product in fp32 (no fused multiply + conversion)
    if constexpr (OutF16) asm volatile("" : "+v"(v[i]));
  }
  uint4* dst = reinterpret_cast<uint4*>(out + b * 128 + 64 * half);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t lo, hi;
      if constexpr (OutF16) {
        lo = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[8 * j + 2 * i]));
        hi = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[8 * j + 2 * i + 1]));
      } else {
        lo = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[8 * j + 2 * i]));
        hi = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[8 * j + 2 * i + 1]));
      }
      p[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    }
    dst[j] = make_uint4(p[0], p[1], p[2], p[3]);
  }
}

template <int G, bool OutF16>
hipError_t launch_unpack_g(const int8_t* wq, const float* w_scale, bool row_scale, int64_t N, int64_t K,
                           uint16_t* out, hipStream_t stream) {
  const int64_t nblk = N * (K / 128);
  const int64_t wgs = (2 * nblk + 255) / 256;
  hipLaunchKernelGGL((unpack_block_kernel<G, OutF16>), dim3(static_cast<uint32_t>(wgs)), dim3(256), 0, stream, wq,
                     nblk, static_cast<int>(K / 128), w_scale, row_scale ? 1 : 0, out);
  return hipGetLastError();
}

template <int G, int CPT, typename In, int MODE>
hipError_t launch_rows(const In* x, int64_t rows, int64_t K, int8_t* q, float* scale,
                       uint32_t* cell, hipStream_t stream) {
  hipLaunchKernelGGL((rotate_rows_kernel<G, CPT, In, MODE>), dim3(static_cast<uint32_t>(rows)),
                     dim3(kThreads), 0, stream, x, K, q, scale, cell);
  return hipGetLastError();
}

// Chunks per thread: the fewest that hold the row (2048 elements per chunk
// slot), else the maximum with a two-pass row.
template <int G, typename In, int MODE>
hipError_t launch_rows_k(const In* x, int64_t rows, int64_t K, int8_t* q, float* scale,
                         uint32_t* cell, hipStream_t stream) {
  const int64_t slots = (K + kThreads * 8 - 1) / (kThreads * 8);
  if (slots <= 1) return launch_rows<G, 1, In, MODE>(x, rows, K, q, scale, cell, stream);
  if (slots <= 2) return launch_rows<G, 2, In, MODE>(x, rows, K, q, scale, cell, stream);
  if (slots <= 4) return launch_rows<G, 4, In, MODE>(x, rows, K, q, scale, cell, stream);
  return launch_rows<G, kMaxChunksPerThread, In, MODE>(x, rows, K, q, scale, cell, stream);
}

template <typename In, int MODE>
hipError_t dispatch_group(int group, const In* x, int64_t rows, int64_t K, int8_t* q,
                          float* scale, uint32_t* cell, hipStream_t stream) {
  if (group == 128) return launch_rows_k<128, In, MODE>(x, rows, K, q, scale, cell, stream);
  return launch_rows_k<256, In, MODE>(x, rows, K, q, scale, cell, stream);
}

}  // namespace

namespace {

template <typename In16>
hipError_t rotate_quant_16(const In16* x, int64_t M, int64_t K, int group, int8_t* q,
                           float* scale, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  // Small batches (up to 2^21 elements, e.g. 512 x 4096) with rows shorter
  // than 8192: the token-block kernel has only a handful of waves there, and
  // the row kernel, which spreads a row over 256 lanes, is faster (16 x 4096:
  // 3.2 us instead of 5.4; 256 x 3072: 3.4 instead of 5.4).  From K = 8192 on
  // a row kernel lane holds four or more chunks in a serial chain, and the
  // block kernel wins at any batch (16 x 12288: 5.7 us instead of 8.1;
  // 16 x 16384, rotated twice by the row kernel: 5.8 instead of 16.1).
  if (K <= kMaxBlockK && !rotate_by_row(M, K)) {
    const BlockGrid g = block_grid(M, K);
    if (group == 128)
      hipLaunchKernelGGL((rotq_block_kernel<128, In16>), dim3(g.wgs), dim3(g.threads), g.lds, stream, x, M,
                         static_cast<int>(K), g.rows_per_wg, g.bpr_inv, q, scale);
    else
      hipLaunchKernelGGL((rotq_block_kernel<256, In16>), dim3(g.wgs), dim3(g.threads), g.lds, stream, x, M,
                         static_cast<int>(K), g.rows_per_wg, g.bpr_inv, q, scale);
    return hipGetLastError();
  }
  return dispatch_group<In16, kActQuant>(group, x, M, K, q, scale, nullptr, stream);
}

}  // namespace

bool rotate_by_row(int64_t M, int64_t K) { return M * K <= kSmallBatchElems && K < 8192; }

int num_cus() {
  // read once (thread-safe static initialisation), from the device current
  // at the first call
  static const int n = [] {
    int dev = 0, v = 0;
    if (hipGetDevice(&dev) == hipSuccess &&
        hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && v > 0)
      return v;
    return 256;
  }();
  return n;
}

hipError_t launch_unpack_weight(const int8_t* wq, const float* w_scale, bool row_scale, int64_t N,
                                int64_t K, int group, bool out_f16, uint16_t* out, hipStream_t stream) {
  if (group == 128)
    return out_f16 ? launch_unpack_g<128, true>(wq, w_scale, row_scale, N, K, out, stream)
                   : launch_unpack_g<128, false>(wq, w_scale, row_scale, N, K, out, stream);
  return out_f16 ? launch_unpack_g<256, true>(wq, w_scale, row_scale, N, K, out, stream)
                 : launch_unpack_g<256, false>(wq, w_scale, row_scale, N, K, out, stream);
}

hipError_t launch_rotate_quant(const uint16_t* x, int64_t M, int64_t K, int group, int8_t* q,
                               float* scale, hipStream_t stream) {
  return rotate_quant_16(x, M, K, group, q, scale, stream);
}

hipError_t launch_rotate_quant_f16(const uint16_t* x, int64_t M, int64_t K, int group, int8_t* q,
                                   float* scale, hipStream_t stream) {
  return rotate_quant_16(reinterpret_cast<const _Float16*>(x), M, K, group, q, scale, stream);
}

hipError_t launch_prepare_weight(const void* w, int in_dtype, bool row_scale, int64_t N, int64_t K,
                                 int group, int8_t* wq, float* w_scale, uint32_t* amax_cell,
                                 hipStream_t stream) {
  // One scale per output channel: every weight row is quantized exactly like
  // a token (the same rotation, absmax, scale and codes).
  if (row_scale) {
    if (in_dtype == kInBf16)
      return rotate_quant_16(static_cast<const uint16_t*>(w), N, K, group, wq, w_scale, stream);
    if (in_dtype == kInF16)
      return rotate_quant_16(static_cast<const _Float16*>(w), N, K, group, wq, w_scale, stream);
    return dispatch_group<float, kActQuant>(group, static_cast<const float*>(w), N, K, wq, w_scale,
                                            nullptr, stream);
  }
  hipLaunchKernelGGL(zero_word_kernel, dim3(1), dim3(1), 0, stream, amax_cell);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (in_dtype == kInBf16) {
    const auto* x = static_cast<const uint16_t*>(w);
    e = dispatch_group<uint16_t, kWeightAbsmax>(group, x, N, K, nullptr, nullptr, amax_cell, stream);
    if (e != hipSuccess) return e;
    return dispatch_group<uint16_t, kWeightQuant>(group, x, N, K, wq, w_scale, amax_cell, stream);
  }
  if (in_dtype == kInF16) {
    const auto* x = static_cast<const _Float16*>(w);
    e = dispatch_group<_Float16, kWeightAbsmax>(group, x, N, K, nullptr, nullptr, amax_cell, stream);
    if (e != hipSuccess) return e;
    return dispatch_group<_Float16, kWeightQuant>(group, x, N, K, wq, w_scale, amax_cell, stream);
  }
  const auto* x = static_cast<const float*>(w);
  e = dispatch_group<float, kWeightAbsmax>(group, x, N, K, nullptr, nullptr, amax_cell, stream);
  if (e != hipSuccess) return e;
  return dispatch_group<float, kWeightQuant>(group, x, N, K, wq, w_scale, amax_cell, stream);
}

}  // namespace convrot
