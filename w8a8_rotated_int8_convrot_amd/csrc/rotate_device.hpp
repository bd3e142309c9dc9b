// rotate_device.hpp -- device code shared by the kernels that rotate rows held
// in registers (rotate_quant.hip, block_norm.hip, and those of the cache of
// heads): 16-bit loads widened to fp32, two fp32 values rounded to 16 bits, the
// butterfly of one 8-element chunk of a g-group spread over g/8 lanes, and the
// int8 code of a value.
#pragma once

#include "convrot_internal.hpp"

namespace convrot {
namespace {

constexpr int kThreads = 256;          // of a workgroup that holds one row

// The float nearest to 1/sqrt(g): 2^-3.5 rounds to 0x3db504f3 for g = 128;
// 2^-4 is exact for g = 256.
template <int G> struct RotScale;
template <> struct RotScale<128> { static constexpr float value = 0x1.6a09e6p-4f; };
template <> struct RotScale<256> { static constexpr float value = 0x1p-4f; };

__device__ inline float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// IEEE binary16 -> fp32 is exact (v_cvt_f32_f16)
__device__ inline float f16_lo(uint32_t w) {
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w)));
}
__device__ inline float f16_hi(uint32_t w) {
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w >> 16)));
}
// the two 16-bit input formats: bf16 bits (uint16_t) and IEEE binary16 (_Float16)
template <typename In> __device__ inline float in_lo(uint32_t w);
template <typename In> __device__ inline float in_hi(uint32_t w);
template <> __device__ inline float in_lo<uint16_t>(uint32_t w) { return bf16_lo(w); }
template <> __device__ inline float in_hi<uint16_t>(uint32_t w) { return bf16_hi(w); }
template <> __device__ inline float in_lo<_Float16>(uint32_t w) { return f16_lo(w); }
template <> __device__ inline float in_hi<_Float16>(uint32_t w) { return f16_hi(w); }

// Load 8 consecutive inputs as fp32.
template <typename In16>
__device__ inline void load8_16(const In16* p, float (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  v[0] = in_lo<In16>(w.x); v[1] = in_hi<In16>(w.x);
  v[2] = in_lo<In16>(w.y); v[3] = in_hi<In16>(w.y);
  v[4] = in_lo<In16>(w.z); v[5] = in_hi<In16>(w.z);
  v[6] = in_lo<In16>(w.w); v[7] = in_hi<In16>(w.w);
}
__device__ inline void load8(const uint16_t* p, float (&v)[8]) { load8_16(p, v); }
__device__ inline void load8(const _Float16* p, float (&v)[8]) { load8_16(p, v); }
__device__ inline void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

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

// v of lane (this lane ^ T).  Inside a 16-lane row DPP moves do it: xor 1
// and xor 2 are quad permutations, xor 4 is the quad reversal (xor 3)
// followed by the half-row mirror (xor 7), xor 8 is a rotation of the row by
// 8; wider distances go through ds_bpermute.
template <int T>
__device__ inline float lane_xor(float v) {
  const int b = __float_as_int(v);
  if constexpr (T == 1) return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0xB1, 0xF, 0xF, true));
  else if constexpr (T == 2) return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0x4E, 0xF, 0xF, true));
  else if constexpr (T == 4)
    return __int_as_float(__builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(b, 0x1B, 0xF, 0xF, true), 0x141, 0xF, 0xF, true));
  else if constexpr (T == 8) return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0x128, 0xF, 0xF, true));
  else return __shfl_xor(v, T);
}

// One butterfly stage between lanes T apart: the lower element keeps
// RN(a + b), the upper RN(a - b) (a = lower), each as RN(own * sgn + partner)
// with sgn = -1 on the upper lane.
template <int T>
__device__ inline void lane_stage(float (&v)[8], int lane_in_group) {
  const float sgn = (lane_in_group & T) != 0 ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(v[i], sgn, lane_xor<T>(v[i]));
}

// Butterfly of one 8-element chunk that is part of a g-group spread over g/8
// lanes; `lane_in_group` is this lane's index inside the group.
template <int G>
__device__ inline void rotate_chunk(float (&v)[8], int lane_in_group) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((i & h) == 0) {
        const float a = v[i], b = v[i + h];
        v[i] = a + b;
        v[i + h] = a - b;
      }
    }
  }
  lane_stage<1>(v, lane_in_group);
  lane_stage<2>(v, lane_in_group);
  lane_stage<4>(v, lane_in_group);
  lane_stage<8>(v, lane_in_group);
  if constexpr (G == 256) lane_stage<16>(v, lane_in_group);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * RotScale<G>::value;
}

// Butterfly stages between lanes 1, 2 and 8 apart as one v_fmac_f32 with a DPP
// source per value, v <- RN(v + sgn * partner).  With sgn = -1 the upper lane
// holds b and gets b - a, the negative of what it keeps (rounding to nearest is
// symmetric): its sign is put right by the constant of the last multiply.  The
// block opens with the two wait states a DPP read needs after a VALU write of
// its source; inside it no instruction reads what another one wrote.
template <int T>
__device__ inline void lane_stage_dpp(float (&v)[8], float sgn) {
#define CONVROT_DPP8(PERM)                                                                               \
  asm volatile("s_nop 1\n\t"                                                                             \
               "v_fmac_f32_dpp %0, %0, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                       \
               "v_fmac_f32_dpp %1, %1, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                       \
               "v_fmac_f32_dpp %2, %2, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                       \
               "v_fmac_f32_dpp %3, %3, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                       \
               "v_fmac_f32_dpp %4, %4, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                       \
               "v_fmac_f32_dpp %5, %5, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                       \
               "v_fmac_f32_dpp %6, %6, %8 " PERM " row_mask:0xf bank_mask:0xf\n\t"                       \
               "v_fmac_f32_dpp %7, %7, %8 " PERM " row_mask:0xf bank_mask:0xf"                             \
               : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]),      \
                 "+v"(v[7])                                                                               \
               : "v"(sgn))
  if constexpr (T == 1) CONVROT_DPP8("quad_perm:[1,0,3,2]");
  else if constexpr (T == 2) CONVROT_DPP8("quad_perm:[2,3,0,1]");
  else CONVROT_DPP8("row_ror:8");
#undef CONVROT_DPP8
}

// rotate_chunk with those stages: the same values, up to the sign of a zero.
template <int G>
__device__ inline void rotate_chunk_fast(float (&v)[8], int lane_in_group) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((i & h) == 0) {
        const float a = v[i], b = v[i + h];
        v[i] = a + b;
        v[i + h] = a - b;
      }
    }
  }
  const float s1 = (lane_in_group & 1) != 0 ? -1.0f : 1.0f, s2 = (lane_in_group & 2) != 0 ? -1.0f : 1.0f;
  const float s8 = (lane_in_group & 8) != 0 ? -1.0f : 1.0f;
  lane_stage_dpp<1>(v, s1);
  lane_stage_dpp<2>(v, s2);
  lane_stage<4>(v, lane_in_group);
  lane_stage_dpp<8>(v, s8);
  if constexpr (G == 256) lane_stage<16>(v, lane_in_group);
  const float c = RotScale<G>::value * (s1 * s2 * s8);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * c;
}

__device__ inline int quant_code(float v, float s) {
  float r = __builtin_rintf(v / s);
  r = fminf(fmaxf(r, -127.0f), 127.0f);
  return static_cast<int>(r);
}

__device__ inline uint2 pack8(const float (&v)[8], float s) {
  uint32_t lo = 0, hi = 0;
  if (s != 0.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) lo |= (static_cast<uint32_t>(quant_code(v[i], s)) & 0xffu) << (8 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i) hi |= (static_cast<uint32_t>(quant_code(v[4 + i], s)) & 0xffu) << (8 * i);
  }
  return make_uint2(lo, hi);
}

// The same codes with a reciprocal and two fused multiply-adds a value instead
// of a division (the quotient comes out correctly rounded), the nearest integer
// by adding 1.5 * 2^23; rows whose scale is too small for a normal reciprocal
// divide.
__device__ inline uint2 pack8_fast(const float (&v)[8], float s) {
  const float r = 1.0f / s;
  if (!(r < 1e30f)) return pack8(v, s);
  uint32_t w[2];
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    uint32_t t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = v[4 * d + e];
      const float q0 = x * r;
      const float rem = __builtin_fmaf(-q0, s, x);
      t[e] = __float_as_uint(__builtin_fmaf(rem, r, q0) + 12582912.0f);
    }
    w[d] = __builtin_amdgcn_perm(t[1], t[0], 0x0c0c0400u) | (__builtin_amdgcn_perm(t[3], t[2], 0x0c0c0400u) << 16);
  }
  return make_uint2(w[0], w[1]);
}

// Maximum over the wave (max is exact and order-free): inside each 16-lane row
// by DPP moves, over the four rows by lane reads.
__device__ inline float wave_max(float a) {
  a = fmaxf(a, lane_xor<1>(a));
  a = fmaxf(a, lane_xor<2>(a));
  a = fmaxf(a, lane_xor<4>(a));
  a = fmaxf(a, lane_xor<8>(a));
  return fmaxf(fmaxf(__int_as_float(__builtin_amdgcn_readlane(__float_as_int(a), 0)),
                     __int_as_float(__builtin_amdgcn_readlane(__float_as_int(a), 16))),
               fmaxf(__int_as_float(__builtin_amdgcn_readlane(__float_as_int(a), 32)),
                     __int_as_float(__builtin_amdgcn_readlane(__float_as_int(a), 48))));
}

// Maximum over the workgroup: the waves' through LDS.
__device__ inline float block_max(float a) {
  __shared__ float part[kThreads / 64];
  a = wave_max(a);
  const int wave = threadIdx.x / 64;
  if ((threadIdx.x & 63) == 0) part[wave] = a;
  __syncthreads();
  float r = part[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) r = fmaxf(r, part[w]);
  return r;
}

// Rotate + quantize one row of at most kThreads * 8 * CPT values by a workgroup
// of kThreads: the row kernel of rotate_quant.hip for a row that fits its
// registers, for kernels that do other work beside it.
template <int G, int CPT, typename In>
__device__ inline void rotate_quant_row(const In* __restrict__ x, int K, int8_t* __restrict__ q,
                                        float* __restrict__ scale) {
  const int tid = threadIdx.x;
  float v[CPT][8];
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const int e = (j * kThreads + tid) * 8;
    if (e < K) load8(x + e, v[j]);
  }
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    if ((j * kThreads + tid) * 8 < K) {
      rotate_chunk_fast<G>(v[j], tid % (G / 8));
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[j][i]));
    }
  }
  const float s = block_max(amax) / 127.0f;
  if (tid == 0) *scale = s;
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const int e = (j * kThreads + tid) * 8;
    if (e < K) *reinterpret_cast<uint2*>(q + e) = pack8_fast(v[j], s);
  }
}

}  // namespace
}  // namespace convrot
