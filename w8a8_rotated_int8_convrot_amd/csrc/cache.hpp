// cache.hpp -- the paged 4-bit cache of keys and values: its layout, and device
// code shared by the kernels that write it (kv_cache.hip) and read it
// (kv_cache.hip, cache_attention.hip).
//
// A page holds `page` tokens (a power of two from 32 to 256) of every key head
// as units of 32 tokens, page = [heads][page / 32] units; a unit of head size D
// is 32 D + 128 bytes (whole 128-byte lines):
//   key codes     [32][D / 2] bytes: dim 2 i in the low half of byte i
//   value codes   [4][D] words: token 8 o + i of dim d in bits 4 i of word [o][d]
//   key scales    [32] bf16
//   value scales  [32] bf16
// A code c in [-7, 7] is held as c + 8.  One unit is what one step of the
// attention reads, in one piece, and both code arrays are in the order of the
// matrix instructions' operands: a lane's key words hold dims of one token, its
// value words hold eight tokens of one dim, so that neither is ever transposed.
#pragma once

#include "convrot_internal.hpp"
#include "rotate_device.hpp"

namespace convrot {
namespace {

constexpr int kUnit = 32;               // tokens
__host__ __device__ constexpr int unit_bytes(int d) { return kUnit * d + 128; }
__host__ __device__ constexpr int value_codes_at(int d) { return 16 * d; }
__host__ __device__ constexpr int key_scales_at(int d) { return 32 * d; }
__host__ __device__ constexpr int value_scales_at(int d) { return 32 * d + 64; }

// Rows [off, end) of sequence b, both inside [0, M] whatever the offsets hold.
struct Span {
  int off, end;
};
__device__ inline Span span_of(const int32_t* offsets, int b, int M) {
  Span s;
  s.off = max(0, min(offsets[b], M));
  s.end = max(s.off, min(offsets[b + 1], M));
  return s;
}

// The sequence of row i: the first b whose rows end behind i.  The caller checks
// that its rows begin at or before i (offsets need not be ascending).
__device__ inline int sequence_of(const int32_t* offsets, int n_seqs, int i) {
  int lo = 0, hi = n_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid + 1] > i) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// The same for one row of the whole wave: 64 sequences' ends looked at in one
// latency, so three of them find one of 2^18 sequences.
__device__ inline int sequence_of_wave(const int32_t* offsets, int n_seqs, int i) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = n_seqs;
  while (lo < hi) {
    const int step = (hi - lo + 63) >> 6;
    const int at = lo + (lane + 1) * step - 1;
    const uint64_t behind = __ballot(at >= hi || offsets[at + 1] > i);
    if (behind == 0) return hi;
    const int l = __builtin_ctzll(behind);
    hi = min(hi, lo + (l + 1) * step - 1);
    lo += l * step;
  }
  return lo;
}

}  // namespace
}  // namespace convrot
