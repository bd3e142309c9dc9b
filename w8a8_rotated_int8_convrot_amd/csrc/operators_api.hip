// operators_api.hip -- the C ABI of the operators around the layer (declared
// in include/convrot.h): argument checks and dispatch, by the rules of
// convrot_api.hip.
#include "../../include/convrot.h"

#include <cmath>

#include "api_checks.hpp"
#include "convrot_internal.hpp"

namespace {

using namespace convrot;

constexpr int kMaxRoutes = 64;

int check_norm(int kind, const char* what, const char* who) {
  if (kind != CONVROT_NORM_NONE && kind != CONVROT_NORM_RMS && kind != CONVROT_NORM_LAYER)
    return fail(CONVROT_EUNSUPPORTED, "%s: %s %d (CONVROT_NORM_NONE, CONVROT_NORM_RMS or CONVROT_NORM_LAYER)", who,
                what, kind);
  return CONVROT_OK;
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
  const BlockNorm p{static_cast<int>(b->K), b->n_routes, b->post_norm, b->pre_norm, b->h, b->u, b->route_row,
                    b->route_weight, b->u_rows, b->post_weight, b->pre_weight, b->gate, b->scale, b->shift,
                    mods ? b->mod_index : nullptr, b->n_mod, b->mod_stride, b->residual_scale, b->eps, b->h_out, b->out,
                    b->out_scale};
  return hip_status(launch_block_norm(p, b->M, b->group, b->io_dtype == CONVROT_F16, static_cast<hipStream_t>(stream)),
                    who);
}

}  // extern "C"
