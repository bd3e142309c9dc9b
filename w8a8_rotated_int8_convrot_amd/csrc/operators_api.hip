// operators_api.hip -- the C ABI of the operators around the layer (declared
// in include/convrot.h): argument checks and dispatch, by the rules of
// convrot_api.hip.
#include "../../include/convrot.h"

#include <algorithm>
#include <cmath>

#include "api_checks.hpp"
#include "convrot_internal.hpp"

namespace {

using namespace convrot;

constexpr int64_t kMaxTokens = int64_t{1} << 30;       // and channels, as check_mn
constexpr int kMaxRoutes = 64;
constexpr int64_t kMaxExperts = 65536;
constexpr int64_t kMaxAdapters = 65536;
constexpr int64_t kMaxRank = 512;

int check_norm(int kind, const char* what, const char* who) {
  if (kind != CONVROT_NORM_NONE && kind != CONVROT_NORM_RMS && kind != CONVROT_NORM_LAYER)
    return fail(CONVROT_EUNSUPPORTED, "%s: %s %d (CONVROT_NORM_NONE, CONVROT_NORM_RMS or CONVROT_NORM_LAYER)", who,
                what, kind);
  return CONVROT_OK;
}

hipError_t rotate_quant(const void* x, bool f16, int64_t M, int64_t K, int group, int8_t* xq, float* xs,
                        hipStream_t stream) {
  const auto* xb = static_cast<const uint16_t*>(x);
  return f16 ? launch_rotate_quant_f16(xb, M, K, group, xq, xs, stream)
             : launch_rotate_quant(xb, M, K, group, xq, xs, stream);
}

// The parts of convrot_linear_lora's workspace for slices of S tokens.
struct LoraLayout {
  int64_t S, t_stride;
  size_t scales, t, total;
};
LoraLayout lora_layout(int64_t M, int64_t K, int64_t N, int64_t max_rank) {
  LoraLayout l;
  l.S = M < 2 * N ? M : 2 * N;
  l.t_stride = (max_rank + 31) / 32 * 32;
  l.scales = round_up(static_cast<size_t>(l.S) * K, 256);
  l.t = l.scales + round_up(static_cast<size_t>(l.S) * 4, 256);
  const size_t t_bytes = round_up(static_cast<size_t>(l.S) * l.t_stride * 2, 256);
  l.total = l.t + t_bytes + static_cast<size_t>(lora_sum_rows(l.S)) * l.t_stride * 4;
  return l;
}

}  // namespace

extern "C" {

int convrot_block_norm(const convrot_block* b, void* stream) {
  const char* who = "convrot_block_norm";
  if (!b) return fail(CONVROT_EINVAL, "%s: NULL pointer", who);
  if (int rc = check_io(b->io_dtype, who)) return rc;
  if (b->group != 0)
    if (int rc = check_group(b->group, b->K, who)) return rc;
  if (b->K < 8 || b->K % 8 != 0)
    return fail(CONVROT_EINVAL, "%s: K=%lld must be a positive multiple of 8", who, static_cast<long long>(b->K));
  if (b->K > kMaxNormK)
    return fail(CONVROT_EUNSUPPORTED, "%s: K=%lld is over %lld", who, static_cast<long long>(b->K),
                static_cast<long long>(kMaxNormK));
  if (b->M < 0 || b->M > (int64_t(1) << 31) - 1)
    return fail(CONVROT_EINVAL, "%s: M=%lld must be in [0, 2^31)", who, static_cast<long long>(b->M));
  if (int rc = check_norm(b->post_norm, "post_norm", who)) return rc;
  if (int rc = check_norm(b->pre_norm, "pre_norm", who)) return rc;
  if (!std::isfinite(b->eps) || b->eps < 0.0f)
    return fail(CONVROT_EINVAL, "%s: eps %g must be finite and not negative", who, b->eps);
  if (!std::isfinite(b->residual_scale))
    return fail(CONVROT_EINVAL, "%s: residual_scale %g must be finite", who, b->residual_scale);
  if (b->n_routes < 0 || b->n_routes > kMaxRoutes)
    return fail(CONVROT_EINVAL, "%s: n_routes %d must be in [0, %d]", who, b->n_routes, kMaxRoutes);
  if (b->u_rows < 0) return fail(CONVROT_EINVAL, "%s: u_rows must not be negative", who);
  const bool mods = b->gate || b->scale || b->shift;
  if (mods ? b->n_mod < 1 : b->n_mod != 0)
    return fail(CONVROT_EINVAL, "%s: n_mod=%lld for %s of gate, scale and shift", who,
                static_cast<long long>(b->n_mod), mods ? "some" : "none");
  if (mods && (b->mod_stride < b->K || b->mod_stride % 8 != 0))
    return fail(CONVROT_EINVAL, "%s: mod_stride=%lld must be a multiple of 8, at least K", who,
                static_cast<long long>(b->mod_stride));
  if (b->M == 0) return ok();
  if (!b->h) return fail(CONVROT_EINVAL, "%s: NULL pointer (h)", who);
  if (!b->u && !b->out) return fail(CONVROT_EINVAL, "%s: nothing to do (u and out are NULL)", who);
  if (b->u && !b->h_out) return fail(CONVROT_EINVAL, "%s: NULL pointer (h_out)", who);
  if (!b->u && (b->post_norm != CONVROT_NORM_NONE || b->gate || b->n_routes != 0 || b->residual_scale != 1.0f))
    return fail(CONVROT_EINVAL, "%s: post_norm, gate, n_routes or residual_scale given without u", who);
  if (b->n_routes > 0 && (!b->route_row || !b->route_weight))
    return fail(CONVROT_EINVAL, "%s: NULL pointer (route_row, route_weight)", who);
  if (b->group != 0 && b->out && !b->out_scale) return fail(CONVROT_EINVAL, "%s: NULL pointer (out_scale)", who);
  const void* aligned[] = {b->h, b->u, b->post_weight, b->pre_weight, b->gate, b->scale, b->shift, b->h_out, b->out};
  for (const void* q : aligned)
    if (!aligned16(q))
      return fail(CONVROT_EALIGN, "%s: h, u, the weights, gate, scale, shift, h_out and out must be 16-byte aligned",
                  who);
  const BlockNorm p{b->M, static_cast<int>(b->K), b->n_routes, b->post_norm, b->pre_norm, b->h, b->u, b->route_row,
                    b->route_weight, b->u_rows, b->post_weight, b->pre_weight, b->gate, b->scale, b->shift,
                    mods ? b->mod_index : nullptr, b->n_mod, b->mod_stride, b->residual_scale, b->eps, b->h_out, b->out,
                    b->out_scale};
  return hip_status(launch_block_norm(p, b->group, b->io_dtype == CONVROT_F16, static_cast<hipStream_t>(stream)), who);
}

size_t convrot_grouped_workspace(int64_t M, int64_t K) {
  if (M < 0 || M > kMaxTokens || K < 1 || K > kMaxK) return 0;
  return round_up(static_cast<size_t>(M) * static_cast<size_t>(K), 256) + static_cast<size_t>(M) * 4;
}

int convrot_grouped_linear(const void* x, int io_dtype, int64_t M, int64_t K, const int8_t* wq, const float* w_scale,
                           int scale_mode, int64_t n_experts, int64_t N, int group, const void* bias,
                           const int32_t* offsets, const int32_t* rows, int64_t P, void* y, void* workspace,
                           size_t ws_bytes, void* stream) {
  const char* who = "convrot_grouped_linear";
  if (int rc = check_group(group, K, who)) return rc;
  if (int rc = check_mn(M, N, who)) return rc;
  if (int rc = check_io(io_dtype, who)) return rc;
  if (int rc = check_scale_mode(scale_mode, who)) return rc;
  if (n_experts < 1 || n_experts > kMaxExperts)
    return fail(CONVROT_EINVAL, "%s: n_experts=%lld must be in [1, %lld]", who, static_cast<long long>(n_experts),
                static_cast<long long>(kMaxExperts));
  if (P < 0 || P > (int64_t(1) << 30))
    return fail(CONVROT_EINVAL, "%s: P=%lld must be in [0, 2^30]", who, static_cast<long long>(P));
  if (P == 0) return ok();
  if (!rows && P != M)
    return fail(CONVROT_EINVAL, "%s: without rows P=%lld has to be M=%lld", who, static_cast<long long>(P),
                static_cast<long long>(M));
  if (M == 0) return fail(CONVROT_EINVAL, "%s: P=%lld rows of no tokens", who, static_cast<long long>(P));
  if ((P / 16 + n_experts) * ((N + 15) / 16) >= (int64_t(1) << 31))
    return fail(CONVROT_EINVAL, "%s: P=%lld, n_experts=%lld and N=%lld make too many tiles", who,
                static_cast<long long>(P), static_cast<long long>(n_experts), static_cast<long long>(N));
  if (!x || !wq || !w_scale || !offsets || !y) return fail(CONVROT_EINVAL, "%s: NULL pointer", who);
  if (!aligned16(x) || !aligned16(wq) || !aligned16(y) || (workspace && !aligned16(workspace)))
    return fail(CONVROT_EALIGN, "%s: x, wq, y and workspace must be 16-byte aligned", who);
  if (!workspace || ws_bytes < convrot_grouped_workspace(M, K))
    return fail(CONVROT_EWORKSPACE, "%s: workspace of %zu bytes needed (convrot_grouped_workspace)", who,
                convrot_grouped_workspace(M, K));
  auto* xq = static_cast<int8_t*>(workspace);
  auto* xs = reinterpret_cast<float*>(static_cast<char*>(workspace) + round_up(static_cast<size_t>(M) * K, 256));
  const bool f16 = io_dtype == CONVROT_F16;
  auto s = static_cast<hipStream_t>(stream);
  if (grouped_is_few(M, K))
    return hip_status(launch_grouped_few(x, M, K, group, f16, wq, w_scale, scale_mode == CONVROT_SCALE_ROW,
                                         static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y), offsets, rows,
                                         n_experts, P, N, s),
                      who);
  if (hipError_t e = rotate_quant(x, f16, M, K, group, xq, xs, s); e != hipSuccess) return hip_status(e, who);
  return hip_status(launch_gemm_grouped(xq, xs, M, wq, w_scale, scale_mode == CONVROT_SCALE_ROW,
                                        static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y), f16, offsets,
                                        rows, n_experts, P, N, K, s),
                    who);
}

size_t convrot_lora_workspace(int64_t M, int64_t K, int64_t N, int64_t max_rank) {
  if (M < 0 || M > kMaxTokens || K < 1 || K > kMaxK || N < 1 || N > kMaxTokens || max_rank < 1 || max_rank > kMaxRank)
    return 0;
  return lora_layout(M, K, N, max_rank).total;
}

int convrot_linear_lora(const void* x, int io_dtype, int64_t M, int64_t K, const int8_t* wq, const float* w_scale,
                        int scale_mode, int64_t N, int group, const void* bias, const void* lora_a,
                        const void* lora_b, int64_t R, const float* lora_scale, const int32_t* offsets,
                        int64_t n_adapters, int64_t max_rank, const int32_t* index, void* y, void* workspace,
                        size_t ws_bytes, void* stream) {
  const char* who = "convrot_linear_lora";
  if (int rc = check_group(group, K, who)) return rc;
  if (int rc = check_mn(M, N, who)) return rc;
  if (int rc = check_io(io_dtype, who)) return rc;
  if (int rc = check_scale_mode(scale_mode, who)) return rc;
  if (n_adapters < 1 || n_adapters > kMaxAdapters)
    return fail(CONVROT_EINVAL, "%s: n_adapters=%lld must be in [1, %lld]", who, static_cast<long long>(n_adapters),
                static_cast<long long>(kMaxAdapters));
  if (max_rank < 1 || max_rank > kMaxRank)
    return fail(CONVROT_EINVAL, "%s: max_rank=%lld must be in [1, %lld]", who, static_cast<long long>(max_rank),
                static_cast<long long>(kMaxRank));
  if (R < 0 || R > (int64_t(1) << 30))
    return fail(CONVROT_EINVAL, "%s: R=%lld must be in [0, 2^30]", who, static_cast<long long>(R));
  if (M == 0) return ok();
  if (!x || !wq || !w_scale || !y || !lora_scale || !offsets || !index || (R > 0 && (!lora_a || !lora_b)))
    return fail(CONVROT_EINVAL, "%s: NULL pointer", who);
  if (!aligned16(x) || !aligned16(wq) || !aligned16(y) || !aligned16(lora_a) || (workspace && !aligned16(workspace)))
    return fail(CONVROT_EALIGN, "%s: x, wq, y, lora_a and workspace must be 16-byte aligned", who);
  const LoraLayout l = lora_layout(M, K, N, max_rank);
  if (!workspace || ws_bytes < l.total)
    return fail(CONVROT_EWORKSPACE, "%s: workspace of %zu bytes needed (convrot_lora_workspace)", who, l.total);
  auto* ws = static_cast<char*>(workspace);
  auto* xq = reinterpret_cast<int8_t*>(ws);
  auto* xs = reinterpret_cast<float*>(ws + l.scales);
  auto* t = reinterpret_cast<uint16_t*>(ws + l.t);
  const bool f16 = io_dtype == CONVROT_F16;
  auto s = static_cast<hipStream_t>(stream);
  for (int64_t r0 = 0; r0 < M; r0 += l.S) {
    const int64_t rows = std::min(M - r0, l.S);
    const auto* xr = static_cast<const uint16_t*>(x) + r0 * K;
    if (hipError_t e = launch_lora_down(xr, rows, K, group, f16, xq, xs, static_cast<const uint16_t*>(lora_a), R,
                                        lora_scale, offsets, n_adapters, index + r0, max_rank, t, l.t_stride,
                                        lora_behind_t(t, rows, l.t_stride), s);
        e != hipSuccess)
      return hip_status(e, who);
    if (hipError_t e = launch_gemm_lora(xq, xs, wq, w_scale, scale_mode == CONVROT_SCALE_ROW,
                                        static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y) + r0 * N, f16,
                                        rows, N, K, t, l.t_stride, static_cast<const uint16_t*>(lora_b), R, offsets,
                                        n_adapters, index + r0, max_rank, s);
        e != hipSuccess)
      return hip_status(e, who);
  }
  return ok();
}

}  // extern "C"
