// api_checks.hpp -- error messages and argument checks shared by the files
// that define entry points of the C ABI.
#pragma once

#include "../../include/convrot.h"

#include <cstdarg>
#include <cstdio>

#include "convrot_internal.hpp"

namespace convrot {

// The message convrot_last_error returns (one per thread, shared by every
// file that defines entry points).
inline thread_local char g_last_error[512] = "";

inline int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
  va_end(ap);
  return status;
}

inline int ok() {
  g_last_error[0] = '\0';
  return CONVROT_OK;
}

inline int hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(CONVROT_EHIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Checks shared by the entry points that take a K dimension of codes.
inline int check_k(int64_t K, const char* who) {
  if (K < 128 || K > convrot::kMaxK || K % 128 != 0)
    return fail(CONVROT_EINVAL, "%s: K=%lld must be a multiple of 128 in [128, %lld]", who,
                static_cast<long long>(K), static_cast<long long>(convrot::kMaxK));
  return CONVROT_OK;
}

inline int check_group(int group, int64_t K, const char* who) {
  if (group != 128 && group != 256)
    return fail(CONVROT_EUNSUPPORTED, "%s: group %d is not supported (128 or 256)", who, group);
  if (K < group || K % group != 0 || K > convrot::kMaxK)
    return fail(CONVROT_EINVAL, "%s: K=%lld must be a positive multiple of the group %d, at most %lld",
                who, static_cast<long long>(K), group, static_cast<long long>(convrot::kMaxK));
  return CONVROT_OK;
}

// Rows and columns are passed to kernels as int; keep every product in range.
inline int check_mn(int64_t M, int64_t N, const char* who) {
  if (M < 0 || N < 1 || M > (int64_t(1) << 30) || N > (int64_t(1) << 30))
    return fail(CONVROT_EINVAL, "%s: M=%lld N=%lld out of range (0 <= M, 1 <= N, both <= 2^30)", who,
                static_cast<long long>(M), static_cast<long long>(N));
  return CONVROT_OK;
}

inline int check_io(int io_dtype, const char* who) {
  if (io_dtype != CONVROT_BF16 && io_dtype != CONVROT_F16)
    return fail(CONVROT_EUNSUPPORTED, "%s: activation/bias/output dtype %d (CONVROT_BF16 or CONVROT_F16)",
                who, io_dtype);
  return CONVROT_OK;
}

inline int check_scale_mode(int scale_mode, const char* who) {
  if (scale_mode != CONVROT_SCALE_TENSOR && scale_mode != CONVROT_SCALE_ROW)
    return fail(CONVROT_EUNSUPPORTED, "%s: weight scale mode %d (CONVROT_SCALE_TENSOR or CONVROT_SCALE_ROW)",
                who, scale_mode);
  return CONVROT_OK;
}

}  // namespace convrot
