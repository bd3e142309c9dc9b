// block_norm.hip -- the step between two blocks of a transformer in one
// kernel: norm of a block's output, gate, residual scale and residual sum,
// then the next block's norm with its scale and shift, as 16-bit values or as
// the rotated int8 codes the next layer's product reads.
//
// Per token m (all in fp32):
//   u  = U[m], or the sum over j of w[m][j] * U[route[m][j]]
//   p  = post(u)          none | u * rsqrt(mean u^2 + eps) * weight
//                              | (u - mean) * rsqrt(mean (u - mean)^2 + eps) * weight
//   h' = rnd(residual_scale * h + gate * p)
//   z  = pre(h') * (1 + scale) + shift
//   out: rnd(z), or codes and scale of the rotated z
// h' is rounded to the io type once, because it is stored, and its norm is
// taken from the rounded values: the norm is then that of the stream the next
// block adds to, and the same whether it comes from this call or from a later
// one that reads the stored h'.  z is not rounded before it is rotated.
//
// One workgroup per token; the row stays in registers from the loads to the
// stores (chunk c of 8 elements in thread c % THREADS, the layout of the row
// kernel in rotate_quant.hip, so the butterfly and the codes are the same), so
// every byte of h, U, h' and the result crosses memory once: 6 bytes an
// element and 2 (or 1, coded) for the result.  The layer norm's variance is
// the mean square of the centred values, a second sum over the registers, so
// a mean far above the spread costs no digits.  Sums: eight values a chunk in
// a lane, then across lanes and waves in a fixed order, so a row repeats its
// bytes.
#include "convrot_internal.hpp"
#include "rotate_device.hpp"

namespace convrot {
namespace {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// two fp32 values rounded to nearest even and packed
template <typename In> __device__ inline uint32_t pack2(float a, float b);
template <> __device__ inline uint32_t pack2<uint16_t>(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2bf));
}
template <> __device__ inline uint32_t pack2<_Float16>(float a, float b) {
  // keep the fp32 results: a multiply-add fused with its conversion would
  // round the exact value to fp16 once
  asm volatile("" : "+v"(a), "+v"(b));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2h));
}

template <typename In>
__device__ inline void widen8(const uint4& w, float (&v)[8]) {
  v[0] = in_lo<In>(w.x); v[1] = in_hi<In>(w.x);
  v[2] = in_lo<In>(w.y); v[3] = in_hi<In>(w.y);
  v[4] = in_lo<In>(w.z); v[5] = in_hi<In>(w.z);
  v[6] = in_lo<In>(w.w); v[7] = in_hi<In>(w.w);
}

template <typename In>
__device__ inline uint4 narrow8(const float (&v)[8]) {
  return make_uint4(pack2<In>(v[0], v[1]), pack2<In>(v[2], v[3]), pack2<In>(v[4], v[5]), pack2<In>(v[6], v[7]));
}

template <bool MAX>
__device__ inline float join(float a, float b) { return MAX ? fmaxf(a, b) : a + b; }

// Sum (or maximum) over the workgroup, the same value in every thread: inside
// each 16-lane row by DPP moves, over the four rows by lane reads, over the
// waves through `part` (one word per wave, not used by an earlier reduction,
// so one barrier is enough).
template <int THREADS, bool MAX>
__device__ inline float reduce(float a, float* part) {
  a = join<MAX>(a, lane_xor<1>(a));
  a = join<MAX>(a, lane_xor<2>(a));
  a = join<MAX>(a, lane_xor<4>(a));
  a = join<MAX>(a, lane_xor<8>(a));
  auto row = [&](int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(a), l)); };
  a = join<MAX>(join<MAX>(row(0), row(16)), join<MAX>(row(32), row(48)));
  if constexpr (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64] = a;
    __syncthreads();
    a = part[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) a = join<MAX>(a, part[w]);
  }
  return a;
}

// G: rotation group of a coded result, 0 for 16-bit values.
template <int G, int THREADS, int CPT, typename In>
__global__ __launch_bounds__(THREADS) void block_norm_kernel(BlockNorm p) {
  constexpr int kWaves = THREADS / 64;
  __shared__ float part[5][kWaves];
  const int tid = threadIdx.x;
  const int64_t row = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
  if (row >= p.M) return;
  const int K = p.K;
  const float inv_k = 1.0f / static_cast<float>(K);
  const In* hr = static_cast<const In*>(p.h) + row * K;
  int elem[CPT];
  bool live[CPT];
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    elem[j] = (j * THREADS + tid) * 8;
    live[j] = elem[j] < K;
  }
  auto load = [&](const void* base, int64_t off, int j) {
    return *reinterpret_cast<const uint4*>(static_cast<const In*>(base) + off + elem[j]);
  };

  // this token's row of gate, scale and shift; a token without one has none
  const int64_t mod = p.mod_index != nullptr ? p.mod_index[row] : 0;
  const bool has_mod = mod >= 0 && mod < p.n_mod;
  const int64_t mod_off = has_mod ? mod * p.mod_stride : 0;

  uint4 hw[CPT];
#pragma unroll
  for (int j = 0; j < CPT; ++j) hw[j] = live[j] ? load(hr, 0, j) : make_uint4(0, 0, 0, 0);

  // y = v normalised (kind: kNormRms, kNormLayer), times the weight
  float v[CPT][8];
  auto norm = [&](int kind, const void* weight, float* sum_part, float* sq_part) {
    if (kind == kNormNone) return;
    if (kind == kNormLayer) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < CPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[j][i];
      const float mean = reduce<THREADS, false>(s, sum_part) * inv_k;
#pragma unroll
      for (int j = 0; j < CPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = live[j] ? v[j][i] - mean : 0.0f;
    }
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < CPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s = __builtin_fmaf(v[j][i], v[j][i], s);
    const float r = 1.0f / sqrtf(reduce<THREADS, false>(s, sq_part) * inv_k + p.eps);
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      float w[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
      if (weight != nullptr && live[j]) widen8<In>(load(weight, 0, j), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * r * w[i];
    }
  };

  if (p.u != nullptr) {
    if (p.n_routes == 0) {
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        const uint4 w = live[j] ? load(p.u, row * K, j) : make_uint4(0, 0, 0, 0);
        widen8<In>(w, v[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < CPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
      for (int t = 0; t < p.n_routes; ++t) {
        const int64_t at = p.route_row[row * p.n_routes + t];
        const float rw = p.route_weight[row * p.n_routes + t];
        if (at < 0 || at >= p.u_rows) continue;
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
          if (!live[j]) continue;
          float w[8];
          widen8<In>(load(p.u, at * K, j), w);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] = __builtin_fmaf(rw, w[i], v[j][i]);
        }
      }
    }
    norm(p.post_norm, p.post_weight, part[0], part[1]);
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      float h[8], gate[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
      widen8<In>(hw[j], h);
      if (p.gate != nullptr && has_mod && live[j]) widen8<In>(load(p.gate, mod_off, j), gate);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = __builtin_fmaf(gate[i], v[j][i], p.residual_scale * h[i]);
      hw[j] = narrow8<In>(h);
      if (live[j]) *reinterpret_cast<uint4*>(static_cast<In*>(p.h_out) + row * K + elem[j]) = hw[j];
    }
  }
  if (p.out == nullptr) return;

#pragma unroll
  for (int j = 0; j < CPT; ++j) widen8<In>(hw[j], v[j]);
  norm(p.pre_norm, p.pre_weight, part[2], part[3]);
  if (has_mod && (p.scale != nullptr || p.shift != nullptr)) {
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      float sc[8] = {}, sh[8] = {};
      if (p.scale != nullptr && live[j]) widen8<In>(load(p.scale, mod_off, j), sc);
      if (p.shift != nullptr && live[j]) widen8<In>(load(p.shift, mod_off, j), sh);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = __builtin_fmaf(v[j][i], 1.0f + sc[i], sh[i]);
    }
  }

  if constexpr (G == 0) {
#pragma unroll
    for (int j = 0; j < CPT; ++j)
      if (live[j]) *reinterpret_cast<uint4*>(static_cast<In*>(p.out) + row * K + elem[j]) = narrow8<In>(v[j]);
  } else {
    // K is a multiple of G, so a g-group lies wholly inside the row or
    // wholly past it, and a live lane exchanges with live lanes only
    const int lane_in_group = tid % (G / 8);
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      if (live[j]) {
        rotate_chunk_fast<G>(v[j], lane_in_group);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[j][i]));
      }
    }
    const float s = reduce<THREADS, true>(amax, part[4]) / 127.0f;
    if (tid == 0) p.out_scale[row] = s;
#pragma unroll
    for (int j = 0; j < CPT; ++j)
      if (live[j]) *reinterpret_cast<uint2*>(static_cast<int8_t*>(p.out) + row * K + elem[j]) = pack8_fast(v[j], s);
  }
}

template <int G, int THREADS, int CPT, typename In>
hipError_t launch(const BlockNorm& p, hipStream_t stream) {
  // HIP counts the threads along x in 32 bits: very many rows wrap into y
  constexpr int64_t kMostX = int64_t{1} << 20;
  const int64_t x = p.M < kMostX ? p.M : kMostX;
  hipLaunchKernelGGL((block_norm_kernel<G, THREADS, CPT, In>),
                     dim3(static_cast<uint32_t>(x), static_cast<uint32_t>((p.M + x - 1) / x)), dim3(THREADS), 0, stream,
                     p);
  return hipGetLastError();
}

// Threads and chunks per thread: the fewest that hold the row, with two or
// three chunks a thread where that leaves few lanes idle (4608 x 4096: 36.7 us
// with 256 threads of two chunks, 35.6 with 512 of one, 45.1 with 128 of four;
// 16896 x 6144: 177 us with 256 threads of three, 193 with 512 of two, 204 with
// 768 of one, 16-bit; now 168, and 167 coded).
template <int G, typename In>
hipError_t launch_k(const BlockNorm& p, hipStream_t stream) {
  const int chunks = (p.K + 7) / 8;
  if (chunks <= 64) return launch<G, 64, 1, In>(p, stream);
  if (chunks <= 128) return launch<G, 128, 1, In>(p, stream);
  if (chunks <= 256) return launch<G, 256, 1, In>(p, stream);
  if (chunks <= 512) return launch<G, 256, 2, In>(p, stream);
  if (chunks <= 768) return launch<G, 256, 3, In>(p, stream);
  if (chunks <= 1024) return launch<G, 512, 2, In>(p, stream);
  if (chunks <= 2048) return launch<G, 1024, 2, In>(p, stream);
  return launch<G, 1024, 4, In>(p, stream);
}

template <typename In>
hipError_t launch_g(const BlockNorm& p, int group, hipStream_t stream) {
  if (group == 128) return launch_k<128, In>(p, stream);
  if (group == 256) return launch_k<256, In>(p, stream);
  return launch_k<0, In>(p, stream);
}

}  // namespace

hipError_t launch_block_norm(const BlockNorm& p, int group, bool f16, hipStream_t stream) {
  if (p.M == 0) return hipSuccess;
  return f16 ? launch_g<_Float16>(p, group, stream) : launch_g<uint16_t>(p, group, stream);
}

}  // namespace convrot
