// convrot_internal.hpp -- shared declarations of the HIP library (not part of
// the C ABI).  Kernels live in rotate_quant.hip (rotation + quantization, and
// the default path's weight unpacking), gemm_core.hpp (the int8 GEMM with its
// epilogues, and the default path's bf16/fp16 product on the same tiles),
// launched by gemm_i8.hip, per expert by gemm_grouped.hip and with low-rank
// adapters by gemm_lora.hip, lora.hip (the adapters' first product),
// default_path.hip (the guarded layer's check), block_norm.hip (the step
// between two blocks), rope.hip, kv_cache.hip and cache_attention.hip (rotary
// positions, the 4-bit cache and the attention over it) and mfma_probe.hip (two
// measurement aids); argument checking, dispatch and the guard state live in
// convrot_api.hip, the entry points of the operators around the layer in
// operators_api.hip and those between two layers in cache_api.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <type_traits>

namespace convrot {

// Largest K the library accepts: 127 * 127 * K must stay below 2^31 so that
// an int32 accumulator cannot overflow.
constexpr int64_t kMaxK = 131072;

// Compute units of the current device (read once; 256 on MI355X), which the
// launch shapes are balanced over.
int num_cus();

// ---------------------------------------------------------------- rotate + quant

// Per-token rotate + quantize of a bf16 [M, K] activation into int8 codes and
// fp32 scales.  group is 128 or 256; K % group == 0.
hipError_t launch_rotate_quant(const uint16_t* x, int64_t M, int64_t K, int group,
                               int8_t* q, float* scale, hipStream_t stream);
// The same for an IEEE binary16 activation (bits passed as uint16_t).
hipError_t launch_rotate_quant_f16(const uint16_t* x, int64_t M, int64_t K, int group,
                                   int8_t* q, float* scale, hipStream_t stream);

// Whether an activation of this size takes the row kernel (a workgroup per
// token, the row in registers) rather than the token-block kernel.
bool rotate_by_row(int64_t M, int64_t K);

// Weight preparation.  in_dtype: kInF32, kInBf16 or kInF16.  Tensorwise (one
// scale; `amax_cell` is one 4-byte device word of scratch) or, with
// row_scale, one scale per output channel (w_scale [N]; no scratch).
constexpr int kInF32 = 0, kInBf16 = 1, kInF16 = 2;
hipError_t launch_prepare_weight(const void* w, int in_dtype, bool row_scale, int64_t N, int64_t K,
                                 int group, int8_t* wq, float* w_scale, uint32_t* amax_cell,
                                 hipStream_t stream);

// Default path: unpack a rotated int8 weight, out[n] = rnd(rotate(s * wq[n]))
// (s = w_scale[row_scale ? n : 0]), rnd = bf16 or fp16 (out_f16) RNE.
hipError_t launch_unpack_weight(const int8_t* wq, const float* w_scale, bool row_scale, int64_t N,
                                int64_t K, int group, bool out_f16, uint16_t* out, hipStream_t stream);

// ---------------------------------------------------------------- GEMM

// GEMM + fused dequant/bias epilogue: y[m][n] (bf16) from xq [M, K] and
// wq [N, K].  K % 128 == 0.
hipError_t launch_gemm_dequant(const int8_t* xq, const float* x_scale, const int8_t* wq,
                               const float* w_scale, const uint16_t* bias, uint16_t* y,
                               int64_t M, int64_t N, int64_t K, hipStream_t stream);

// The tile the layer's product picks for a shape, by the numbers of
// gemm_i8.hip's choices.
int pick_gemm_tile(int64_t M, int64_t N);

// Variants: one weight scale per output channel (row_scale: w_scale [N]) and
// fp16 in place of bf16 for the bias and the output (out_f16).
hipError_t launch_gemm_dequant_ex(const int8_t* xq, const float* x_scale, const int8_t* wq,
                                  const float* w_scale, bool row_scale, const uint16_t* bias,
                                  uint16_t* y, bool out_f16, int64_t M, int64_t N, int64_t K,
                                  hipStream_t stream);

// Same main loop with the raw int32 products stored.
hipError_t launch_gemm_i32(const int8_t* xq, const int8_t* wq, int32_t* acc,
                           int64_t M, int64_t N, int64_t K, hipStream_t stream);

// Default path product: y = rnd(x . wu^T + bias) on bf16 (or fp16, f16)
// operands x [M, K] and wu [N, K] with an fp32 accumulator.  K % 64 == 0.
hipError_t launch_gemm_default(const uint16_t* x, const uint16_t* wu, const uint16_t* bias, uint16_t* y,
                               bool f16, int64_t M, int64_t N, int64_t K, hipStream_t stream);

// The product per expert (gemm_grouped.hip): rows [offsets[e], offsets[e+1])
// of y [P, N] are those of expert e (wq [experts, N, K], w_scale [experts] or
// with row_scale [experts, N], bias [experts, N] or null), row p made from row
// rows[p] of xq [x_rows, K] (null: p).  offsets and rows are device memory.
// hipErrorInvalidConfiguration where the grid would be larger than HIP takes.
hipError_t launch_gemm_grouped(const int8_t* xq, const float* x_scale, int64_t x_rows, const int8_t* wq,
                               const float* w_scale, bool row_scale, const uint16_t* bias, uint16_t* y, bool f16,
                               const int32_t* offsets, const int32_t* rows, int64_t experts, int64_t P, int64_t N,
                               int64_t K, hipStream_t stream);

// The whole call for few tokens (M, K that grouped_is_few takes): x [M, K] in
// the io type, rotated and coded by the kernel itself.  The same bytes.
bool grouped_is_few(int64_t M, int64_t K);
hipError_t launch_grouped_few(const void* x, int64_t M, int64_t K, int group, bool f16, const int8_t* wq,
                              const float* w_scale, bool row_scale, const uint16_t* bias, uint16_t* y,
                              const int32_t* offsets, const int32_t* rows, int64_t experts, int64_t P, int64_t N,
                              hipStream_t stream);

// Whether a batch's adapters are taken token by token or as a list per tile.  By
// sizes alone, so that a token's result does not depend on the other tokens'
// adapters.  A token's own ranks run on the vector unit, each token reading its
// adapter, so the time goes with the rank; a list costs a latency and a matrix
// product for each adapter and 32 ranks, whoever shares them.  us a call, weight
// from HBM, 128 tokens in equal runs of each adapter, list / token by token:
//                      4096 x 4096               2048 x 8192
//   rank            16      64     128        16      64     128
//    5 adapters   23/22   26/35   31/52     19/17   21/31   28/48
//   12            24/22   27/34   34/52     21/18   26/32   36/51
//   48            33/24   43/37   62/56     37/20   55/38   90/65
// Over these, 17, 32 and 64 tokens, two adapters, and the tokens shuffled, the
// rule is 1.6 % behind the better of the two on the mean and 22 % at worst; more
// than four adapters at any rank would be 10 % and 114 %, the list alone 19 %,
// token by token alone 22 %.
inline bool lora_by_token(int64_t M, int64_t adapters, int64_t max_rank) {
  const int64_t shared = (max_rank < 64 ? max_rank : 64) * 3 / 16;
  return M <= 16 || (M <= 128 && adapters > (shared > 4 ? shared : 4));
}

// The first product of low-rank adapters (lora.hip):
//   t[m][r] = scale[a] * (row offsets[a] + r of a_rows [ranks, K]) . x[m]
// with a = index[m]; zero from the adapter's rank on, unset for a token whose
// index is outside [0, adapters).  t_stride: max_rank rounded up to 32.  sums:
// lora_sum_rows(M) * t_stride floats, lora_behind_t of t.  Token by token t is
// left there in fp32, [M, t_stride].  Else the first [M, t_stride] words hold it
// as two parts in the io type, t = (first + second) * factor, each 32 ranks as
// 32 values of the first part and then 32 of the second; the factors of each 32
// ranks are [t_stride / 32, M] floats in t's [M, t_stride] 16-bit words (1, and
// not written, in bf16).  Rotates and quantizes x too (xq, xs as
// launch_rotate_quant), in the same launch where the row kernel would do it.
constexpr int kMaxLoraParts = 8;
// Rows of the partial sums: parts of K times tokens, K being split only while
// they stay within kLoraSumRows.
constexpr int64_t kLoraSumRows = 40960;
inline int64_t lora_sum_rows(int64_t M) {
  if (kMaxLoraParts * M <= kLoraSumRows) return kMaxLoraParts * M;
  return M > kLoraSumRows ? M : kLoraSumRows;
}
// The first 256-byte boundary behind t [M, t_stride].
template <class U16>
inline auto lora_behind_t(U16* t, int64_t M, int64_t t_stride) {
  constexpr bool kConst = std::is_const_v<U16>;
  return reinterpret_cast<std::conditional_t<kConst, const float, float>*>(t + (M * t_stride + 127) / 128 * 128);
}
hipError_t launch_lora_down(const uint16_t* x, int64_t M, int64_t K, int group, bool f16, int8_t* xq, float* xs,
                            const uint16_t* a, int64_t ranks, const float* scale, const int32_t* offsets,
                            int64_t adapters, const int32_t* index, int64_t max_rank, uint16_t* t, int64_t t_stride,
                            float* sums, hipStream_t stream);

// The layer's product with the adapters' second one, t . b (b [ranks, N], t as
// launch_lora_down leaves it in t and in the sums behind it), added before the
// output is rounded (gemm_lora.hip).
hipError_t launch_gemm_lora(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                            bool row_scale, const uint16_t* bias, uint16_t* y, bool f16, int64_t M, int64_t N, int64_t K,
                            const uint16_t* t, int64_t t_stride, const uint16_t* b, int64_t ranks,
                            const int32_t* offsets, int64_t adapters, const int32_t* index, int64_t max_rank,
                            hipStream_t stream);

// ---------------------------------------------------------------- guard check
// (default_path.hip)

// xs[i] = x[row_i] for the R sampled rows row_i = i * (M - 1) / (R - 1).
hipError_t launch_gather_rows(const uint16_t* x, int64_t M, int64_t K, int R, uint16_t* xs,
                              hipStream_t stream);
// Per sampled row i: partial[3i..3i+2] = {sum_n (a - b)^2, sum_n b^2, count of
// mismatched non-finite values}, a = y[row_i][n] (negated when flip),
// b = ydef[i][n], in fp64; where a and b are the same infinity the position
// is left out of the sums, and where either is otherwise not finite it counts.
hipError_t launch_compare_rows(const uint16_t* y, const uint16_t* ydef, bool f16, int64_t M, int64_t N,
                               int R, bool flip, double* partial, hipStream_t stream);
// The sampled row i of R over M rows.
__host__ __device__ inline int64_t sample_row(int i, int R, int64_t M) {
  return R > 1 ? static_cast<int64_t>(i) * (M - 1) / (R - 1) : 0;
}

// ---------------------------------------------------------------- between two blocks
// (block_norm.hip)

constexpr int kNormNone = 0, kNormRms = 1, kNormLayer = 2;
// The longest row the kernel holds in its registers (1024 threads of four
// 8-element chunks).
constexpr int64_t kMaxNormK = 32768;

// Arguments as in convrot_block_norm (16-bit values behind void pointers); a
// null u leaves the stream as it is, a null out ends after h_out.
struct BlockNorm {
  int64_t M;
  int K, n_routes, post_norm, pre_norm;
  const void *h, *u;
  const int32_t* route_row;
  const float* route_weight;
  int64_t u_rows;
  const void *post_weight, *pre_weight, *gate, *scale, *shift;
  const int32_t* mod_index;
  int64_t n_mod, mod_stride;
  float residual_scale, eps;
  void *h_out, *out;
  float* out_scale;
};
// group: 128 or 256 for codes, 0 for 16-bit values.
hipError_t launch_block_norm(const BlockNorm& p, int group, bool f16, hipStream_t stream);

// ---------------------------------------------------------------- between two layers
// (rope.hip, kv_cache.hip, cache_attention.hip)

// One tensor of heads: rows of `heads` vectors, `stride` elements apart.
struct RopePart {
  const void* in;
  void* out;
  int64_t heads, in_stride, out_stride;
};
// Arguments as in convrot_rope; a part without heads is left out.
struct Rope {
  RopePart part[2];
  int64_t M;
  int head_dim, rot_dim;
  bool interleaved, inverse;
  const int32_t* positions;
  const double* freqs;
  float scale;
};
hipError_t launch_rope(const Rope& p, bool f16, hipStream_t stream);

// convrot_cache by value, with the sizes the kernels need.
struct Cache {
  uint8_t* pages;
  int64_t n_pages, page_bytes;
  int page_shift, kv_heads, head_dim;
  const int32_t* table;
  int64_t table_stride;
  int n_seqs;
  int max_tokens;                       // columns of the table times the page
};
// Rows of keys and values to or from the cache, [M, kv_heads, head_dim], rows
// k_stride and v_stride elements apart; starts [n_seqs], offsets [n_seqs + 1].
hipError_t launch_cache_append(const Cache& c, const void* k, int64_t k_stride, const void* v, int64_t v_stride, bool f16,
                               int64_t M, const int32_t* starts, const int32_t* offsets, hipStream_t stream);
hipError_t launch_cache_read(const Cache& c, void* k, int64_t k_stride, void* v, int64_t v_stride, bool f16, int64_t M,
                             const int32_t* starts, const int32_t* offsets, hipStream_t stream);

// Pages src[i] -> dst[i] in each of `layers` caches, layer_bytes apart (host lists).
hipError_t launch_cache_copy(uint8_t* pages, int64_t layers, int64_t layer_bytes, int64_t page_bytes, const int32_t* src,
                             const int32_t* dst, int64_t n, hipStream_t stream);

// How convrot_cache_attention cuts its work, from sizes the host knows: the keys
// that a tile of rows sees in `splits` parts of `chunk` (the last takes the rest).
struct AttentionPlan {
  int splits, chunk;
  int64_t slots, slot_units;            // long prompts whose keys and values are made operands, units of each
  int limit;                            // rows a key head that a sequence of them has more than
  size_t parts, workspace;              // bytes, of the parts' sums and of all
};
AttentionPlan plan_cache_attention(int64_t M, int64_t q_heads, int64_t kv_heads, int head_dim, int64_t n_seqs,
                                   int64_t max_tokens, int64_t window, bool f16);
struct Attention {
  Cache cache;
  const void* q;
  int64_t q_stride;
  int M, q_heads;
  const int32_t *starts, *offsets;
  float scale;
  bool causal;
  int window;                           // 0: none
  void* out;                            // [M, q_heads, head_dim]
  int splits, chunk;
  float* part;                          // workspace: [splits][M * q_heads][head_dim], then [splits][M * q_heads][2]
  uint8_t* operands;                    // behind it, for `slots` prompts
  int64_t slots, slot_units;
  int limit;
};
hipError_t launch_cache_attention(const Attention& a, bool f16, hipStream_t stream);

// ---------------------------------------------------------------- measurement aid

// Register-only MFMA loop (mfma_probe.hip): `blocks` workgroups of 256
// threads, `iters` x 16 v_mfma_i32_32x32x32_i8 per wave on 16-byte fragments
// taken from a and b; one int32 per thread written to out.
hipError_t launch_mfma_probe(const int8_t* a, int64_t a_bytes, const int8_t* b, int64_t b_bytes,
                             int blocks, int iters, int32_t* out, hipStream_t stream);
// Plain stream (mfma_probe.hip): q[i] = high byte of x[i] for n 16-bit
// values (n % 8 == 0, 16-byte aligned buffers).
hipError_t launch_stream_probe(const uint16_t* x, int64_t n, int8_t* q, hipStream_t stream);

}  // namespace convrot
