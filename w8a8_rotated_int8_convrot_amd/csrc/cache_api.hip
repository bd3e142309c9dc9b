// cache_api.hip -- the C ABI of what stands between two layers (declared in
// include/convrot.h): rotary positions, the 4-bit cache, the attention over it.
// Argument checks and dispatch, by the rules of convrot_api.hip.
#include "../../include/convrot.h"

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "api_checks.hpp"
#include "convrot_internal.hpp"

namespace {

using namespace convrot;

constexpr int64_t kMaxRows = int64_t{1} << 30;
constexpr int64_t kMaxCacheTokens = int64_t{1} << 30;
constexpr int64_t kMaxKvHeads = 1024;
constexpr int64_t kMaxSeqs = int64_t{1} << 20;
constexpr int64_t kMaxPairs = int64_t{1} << 20;
constexpr int64_t kMaxStride = int64_t{1} << 40;

bool page_known(int page) { return page == 32 || page == 64 || page == 128 || page == 256; }
bool head_known(int head_dim) { return head_dim == 64 || head_dim == 128 || head_dim == 256; }
int page_shift(int page) { return page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : 8; }

// Rows of heads: their stride and their pointer.
int check_heads(const void* p, int64_t heads, int64_t stride, int64_t head_dim, const char* what, const char* who) {
  if (stride < heads * head_dim || stride % 8 != 0 || stride > kMaxStride)
    return fail(CONVROT_EINVAL, "%s: %s stride %lld must be a multiple of 8, at least %lld", who, what,
                static_cast<long long>(stride), static_cast<long long>(heads * head_dim));
  if (!p) return fail(CONVROT_EINVAL, "%s: NULL pointer (%s)", who, what);
  if (!aligned16(p)) return fail(CONVROT_EALIGN, "%s: %s must be 16-byte aligned", who, what);
  return CONVROT_OK;
}

int check_rows(int64_t M, const char* who) {
  if (M < 0 || M > kMaxRows)
    return fail(CONVROT_EINVAL, "%s: M=%lld must be in [0, 2^30]", who, static_cast<long long>(M));
  return CONVROT_OK;
}

// The sizes of a cache; its pointers, and that it holds pages, columns and sequences, only where
// there are rows.
int check_cache(const convrot_cache* c, int64_t M, const char* who) {
  if (!c) return fail(CONVROT_EINVAL, "%s: NULL pointer (cache)", who);
  if (!page_known(c->page))
    return fail(CONVROT_EUNSUPPORTED, "%s: page %d is not supported (32, 64, 128 or 256 tokens)", who, c->page);
  if (!head_known(c->head_dim))
    return fail(CONVROT_EUNSUPPORTED, "%s: head_dim %d is not supported (64, 128 or 256)", who, c->head_dim);
  if (c->kv_heads < 1 || c->kv_heads > kMaxKvHeads)
    return fail(CONVROT_EINVAL, "%s: kv_heads=%lld must be in [1, %lld]", who, static_cast<long long>(c->kv_heads),
                static_cast<long long>(kMaxKvHeads));
  const int64_t least = M == 0 ? 0 : 1;
  if (c->n_pages < least || c->n_pages > 0x7fffffff)
    return fail(CONVROT_EINVAL, "%s: n_pages=%lld must be in [1, 2^31)", who, static_cast<long long>(c->n_pages));
  if (c->n_seqs < least || c->n_seqs > kMaxSeqs)
    return fail(CONVROT_EINVAL, "%s: n_seqs=%lld must be in [1, 2^20]", who, static_cast<long long>(c->n_seqs));
  if (c->max_pages < least || c->max_pages > kMaxCacheTokens / c->page)
    return fail(CONVROT_EINVAL, "%s: max_pages=%lld must be in [1, %lld]", who, static_cast<long long>(c->max_pages),
                static_cast<long long>(kMaxCacheTokens / c->page));
  if (c->table_stride < c->max_pages || c->table_stride > kMaxStride)
    return fail(CONVROT_EINVAL, "%s: table_stride=%lld must be at least max_pages", who,
                static_cast<long long>(c->table_stride));
  if (M == 0) return CONVROT_OK;
  if (!c->pages || !c->table || !c->starts || !c->offsets)
    return fail(CONVROT_EINVAL, "%s: NULL pointer (pages, table, starts, offsets)", who);
  if (!aligned16(c->pages)) return fail(CONVROT_EALIGN, "%s: pages must be 16-byte aligned", who);
  return CONVROT_OK;
}

Cache cache_of(const convrot_cache& c) {
  return Cache{static_cast<uint8_t*>(c.pages), c.n_pages,
               static_cast<int64_t>(convrot_cache_page_bytes(c.page, c.kv_heads, c.head_dim)), page_shift(c.page),
               static_cast<int>(c.kv_heads), c.head_dim, c.table, c.table_stride, static_cast<int>(c.n_seqs),
               static_cast<int>(c.max_pages * c.page)};
}

}  // namespace

extern "C" {

int convrot_rope_frequencies(int rot_dim, double base, int scaling, double factor, double original_length, double low,
                             double high, double* freqs, float* scale) {
  const char* who = "convrot_rope_frequencies";
  if (scaling < CONVROT_ROPE_NONE || scaling > CONVROT_ROPE_BANDS)
    return fail(CONVROT_EUNSUPPORTED, "%s: unknown scaling %d", who, scaling);
  if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2 != 0)
    return fail(CONVROT_EINVAL, "%s: rot_dim %d must be even, in [2, 1024]", who, rot_dim);
  if (!std::isfinite(base) || !(base > 1.0)) return fail(CONVROT_EINVAL, "%s: base %g must be finite and over 1", who, base);
  if (scaling != CONVROT_ROPE_NONE && (!std::isfinite(factor) || !(factor >= 1.0)))
    return fail(CONVROT_EINVAL, "%s: factor %g must be finite and at least 1", who, factor);
  if (scaling == CONVROT_ROPE_NTK && rot_dim == 2)
    return fail(CONVROT_EINVAL, "%s: NTK scaling of a single pair", who);
  const bool bands = scaling == CONVROT_ROPE_YARN || scaling == CONVROT_ROPE_BANDS;
  if (bands && (!std::isfinite(original_length) || !(original_length > 0.0)))
    return fail(CONVROT_EINVAL, "%s: original_length %g must be finite and positive", who, original_length);
  if (bands && !(0.0 < low && low < high && std::isfinite(high)))
    return fail(CONVROT_EINVAL, "%s: low %g and high %g must be 0 < low < high", who, low, high);
  if (!freqs || !scale) return fail(CONVROT_EINVAL, "%s: NULL pointer", who);
  constexpr double kTwoPi = 6.283185307179586477;
  if (scaling == CONVROT_ROPE_NTK) base *= std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
  if (!std::isfinite(base)) return fail(CONVROT_EINVAL, "%s: base and factor are too large", who);
  const auto dim_of = [&](double turns) {
    return rot_dim * std::log(original_length / (turns * kTwoPi)) / (2.0 * std::log(base));
  };
  double lo = 0.0, hi = 0.0;
  *scale = 1.0f;
  if (scaling == CONVROT_ROPE_YARN) {
    lo = std::max(std::floor(dim_of(high)), 0.0);
    hi = std::min(std::ceil(dim_of(low)), rot_dim - 1.0);
    *scale = static_cast<float>(0.1 * std::log(factor) + 1.0);
  }
  const auto unit = [](double v) { return std::min(std::max(v, 0.0), 1.0); };
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot_dim);
    double keep = 1.0;                  // of f; the rest is f / factor
    if (scaling == CONVROT_ROPE_LINEAR) keep = 0.0;
    if (scaling == CONVROT_ROPE_YARN) keep = 1.0 - unit((i - lo) / std::max(hi - lo, 0.001));
    if (scaling == CONVROT_ROPE_BANDS) keep = unit((original_length * f / kTwoPi - low) / (high - low));
    freqs[i] = keep == 1.0 ? f : f * keep + f / factor * (1.0 - keep);
  }
  return ok();
}

int convrot_rope(const void* q, int64_t q_heads, int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k,
                 int64_t k_heads, int64_t k_stride, void* k_out, int64_t k_out_stride, int io_dtype, int64_t M,
                 int head_dim, int rot_dim, int layout, const int32_t* positions, const double* freqs, float scale,
                 int inverse, void* stream) {
  const char* who = "convrot_rope";
  if (int rc = check_io(io_dtype, who)) return rc;
  if (layout != CONVROT_ROPE_HALF && layout != CONVROT_ROPE_INTERLEAVED)
    return fail(CONVROT_EUNSUPPORTED, "%s: layout %d (CONVROT_ROPE_HALF or CONVROT_ROPE_INTERLEAVED)", who, layout);
  if (int rc = check_rows(M, who)) return rc;
  if (head_dim < 8 || head_dim > 1024 || head_dim % 8 != 0)
    return fail(CONVROT_EINVAL, "%s: head_dim %d must be a multiple of 8 in [8, 1024]", who, head_dim);
  if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2 != 0)
    return fail(CONVROT_EINVAL, "%s: rot_dim %d must be even, in [2, head_dim]", who, rot_dim);
  if (q_heads < 0 || k_heads < 0 || q_heads > 16384 || k_heads > 16384 || q_heads + k_heads < 1 ||
      q_heads + k_heads > 16384)
    return fail(CONVROT_EINVAL, "%s: q_heads=%lld and k_heads=%lld must be 1 to 16384 together", who,
                static_cast<long long>(q_heads), static_cast<long long>(k_heads));
  if (!std::isfinite(scale)) return fail(CONVROT_EINVAL, "%s: scale %g must be finite", who, scale);
  if (M == 0) return ok();
  if (q_heads > 0) {
    if (int rc = check_heads(q, q_heads, q_stride, head_dim, "q", who)) return rc;
    if (int rc = check_heads(q_out, q_heads, q_out_stride, head_dim, "q_out", who)) return rc;
    if (q == q_out && q_stride != q_out_stride)
      return fail(CONVROT_EINVAL, "%s: q_out is q with another stride", who);
  }
  if (k_heads > 0) {
    if (int rc = check_heads(k, k_heads, k_stride, head_dim, "k", who)) return rc;
    if (int rc = check_heads(k_out, k_heads, k_out_stride, head_dim, "k_out", who)) return rc;
    if (k == k_out && k_stride != k_out_stride)
      return fail(CONVROT_EINVAL, "%s: k_out is k with another stride", who);
  }
  if (!positions || !freqs) return fail(CONVROT_EINVAL, "%s: NULL pointer (positions, freqs)", who);
  const Rope p{{{q, q_out, q_heads, q_stride, q_out_stride}, {k, k_out, k_heads, k_stride, k_out_stride}},
               M, head_dim, rot_dim, layout == CONVROT_ROPE_INTERLEAVED, inverse != 0, positions, freqs, scale};
  return hip_status(launch_rope(p, io_dtype == CONVROT_F16, static_cast<hipStream_t>(stream)), who);
}

size_t convrot_cache_page_bytes(int page, int64_t kv_heads, int head_dim) {
  if (!page_known(page) || !head_known(head_dim) || kv_heads < 1 || kv_heads > kMaxKvHeads) return 0;
  return static_cast<size_t>(kv_heads) * (page / 32) * (32 * head_dim + 128);
}

int convrot_cache_append(const convrot_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                         int io_dtype, int64_t M, void* stream) {
  const char* who = "convrot_cache_append";
  if (int rc = check_io(io_dtype, who)) return rc;
  if (int rc = check_rows(M, who)) return rc;
  if (int rc = check_cache(cache, M, who)) return rc;
  if (M == 0) return ok();
  if (int rc = check_heads(k, cache->kv_heads, k_stride, cache->head_dim, "k", who)) return rc;
  if (int rc = check_heads(v, cache->kv_heads, v_stride, cache->head_dim, "v", who)) return rc;
  return hip_status(launch_cache_append(cache_of(*cache), k, k_stride, v, v_stride, io_dtype == CONVROT_F16, M,
                                        cache->starts, cache->offsets, static_cast<hipStream_t>(stream)),
                    who);
}

int convrot_cache_read(const convrot_cache* cache, void* k, int64_t k_stride, void* v, int64_t v_stride, int io_dtype,
                       int64_t M, void* stream) {
  const char* who = "convrot_cache_read";
  if (int rc = check_io(io_dtype, who)) return rc;
  if (int rc = check_rows(M, who)) return rc;
  if (int rc = check_cache(cache, M, who)) return rc;
  if (M == 0) return ok();
  if (!k && !v) return fail(CONVROT_EINVAL, "%s: nothing to do (k and v are NULL)", who);
  if (k)
    if (int rc = check_heads(k, cache->kv_heads, k_stride, cache->head_dim, "k", who)) return rc;
  if (v)
    if (int rc = check_heads(v, cache->kv_heads, v_stride, cache->head_dim, "v", who)) return rc;
  return hip_status(launch_cache_read(cache_of(*cache), k, k_stride, v, v_stride, io_dtype == CONVROT_F16, M,
                                      cache->starts, cache->offsets, static_cast<hipStream_t>(stream)),
                    who);
}

size_t convrot_cache_attention_workspace(int64_t M, int64_t q_heads, int64_t kv_heads, int head_dim, int64_t n_seqs,
                                         int64_t max_tokens) {
  if (M < 1 || q_heads < 1 || M > kMaxRows / q_heads || kv_heads < 1 || kv_heads > kMaxKvHeads ||
      q_heads % kv_heads != 0 || !head_known(head_dim) || n_seqs < 1 || n_seqs > kMaxSeqs || max_tokens < 1 ||
      max_tokens > kMaxCacheTokens)
    return 0;
  return std::max(plan_cache_attention(M, q_heads, kv_heads, head_dim, n_seqs, max_tokens, 0, false).workspace,
                  plan_cache_attention(M, q_heads, kv_heads, head_dim, n_seqs, max_tokens, 0, true).workspace);
}

int convrot_cache_attention(const convrot_cache* cache, const void* q, int64_t q_heads, int64_t q_stride, int io_dtype,
                            int64_t M, float scale, int causal, int64_t window, void* out, void* workspace,
                            size_t ws_bytes, void* stream) {
  const char* who = "convrot_cache_attention";
  if (int rc = check_io(io_dtype, who)) return rc;
  if (int rc = check_rows(M, who)) return rc;
  if (int rc = check_cache(cache, M, who)) return rc;
  if (q_heads < 1 || q_heads % cache->kv_heads != 0)
    return fail(CONVROT_EINVAL, "%s: q_heads=%lld must be a positive multiple of kv_heads=%lld", who,
                static_cast<long long>(q_heads), static_cast<long long>(cache->kv_heads));
  if (M > kMaxRows / q_heads)
    return fail(CONVROT_EINVAL, "%s: M=%lld times q_heads=%lld is over 2^30", who, static_cast<long long>(M),
                static_cast<long long>(q_heads));
  if (!std::isfinite(scale)) return fail(CONVROT_EINVAL, "%s: scale %g must be finite", who, scale);
  if (window < 0 || window > 0x7fffffff || (window != 0 && !causal))
    return fail(CONVROT_EINVAL, "%s: window=%lld must be in [0, 2^31), and 0 unless causal", who,
                static_cast<long long>(window));
  if (M == 0) return ok();
  if (int rc = check_heads(q, q_heads, q_stride, cache->head_dim, "q", who)) return rc;
  if (!out) return fail(CONVROT_EINVAL, "%s: NULL pointer (out)", who);
  if (!aligned16(out) || (workspace && !aligned16(workspace)))
    return fail(CONVROT_EALIGN, "%s: out and workspace must be 16-byte aligned", who);
  const AttentionPlan plan = plan_cache_attention(M, q_heads, cache->kv_heads, cache->head_dim, cache->n_seqs,
                                                  cache->max_pages * cache->page, window, io_dtype == CONVROT_F16);
  if (plan.workspace != 0 && (!workspace || ws_bytes < plan.workspace))
    return fail(CONVROT_EWORKSPACE, "%s: workspace of %zu bytes needed (convrot_cache_attention_workspace)", who,
                plan.workspace);
  const Attention a{cache_of(*cache), q, q_stride, static_cast<int>(M), static_cast<int>(q_heads), cache->starts,
                    cache->offsets, scale, causal != 0, static_cast<int>(window), out, plan.splits, plan.chunk,
                    static_cast<float*>(workspace), static_cast<uint8_t*>(workspace) + plan.parts, plan.slots,
                    plan.slot_units, plan.limit};
  return hip_status(launch_cache_attention(a, io_dtype == CONVROT_F16, static_cast<hipStream_t>(stream)), who);
}

int convrot_cache_copy(void* pages, int64_t layers, int64_t layer_bytes, int64_t n_pages, int64_t page_bytes,
                       const int32_t* src, const int32_t* dst, int64_t n, void* stream) {
  const char* who = "convrot_cache_copy";
  if (n < 0 || n > kMaxPairs)
    return fail(CONVROT_EINVAL, "%s: n=%lld must be in [0, 2^20]", who, static_cast<long long>(n));
  if (layers < 1 || layers > 65535)
    return fail(CONVROT_EINVAL, "%s: layers=%lld must be in [1, 65535]", who, static_cast<long long>(layers));
  if (n_pages < 1 || n_pages > 0x7fffffff)
    return fail(CONVROT_EINVAL, "%s: n_pages=%lld must be in [1, 2^31)", who, static_cast<long long>(n_pages));
  if (page_bytes < 16 || page_bytes % 16 != 0 || page_bytes > (int64_t{1} << 31))
    return fail(CONVROT_EINVAL, "%s: page_bytes=%lld must be a multiple of 16, at most 2^31", who,
                static_cast<long long>(page_bytes));
  if (layers > 1 && (layer_bytes < n_pages * page_bytes || layer_bytes % 16 != 0 || layer_bytes > kMaxStride))
    return fail(CONVROT_EINVAL, "%s: layer_bytes=%lld must be a multiple of 16, at least n_pages * page_bytes", who,
                static_cast<long long>(layer_bytes));
  if (n == 0) return ok();
  if (!pages || !src || !dst) return fail(CONVROT_EINVAL, "%s: NULL pointer", who);
  if (!aligned16(pages)) return fail(CONVROT_EALIGN, "%s: pages must be 16-byte aligned", who);
  for (int64_t i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= n_pages || dst[i] < 0 || dst[i] >= n_pages)
      return fail(CONVROT_EINVAL, "%s: pair %lld, page %d to %d, is outside [0, %lld)", who, static_cast<long long>(i),
                  src[i], dst[i], static_cast<long long>(n_pages));
  try {
    std::vector<int32_t> to(dst, dst + n);
    std::sort(to.begin(), to.end());
    if (const auto twice = std::adjacent_find(to.begin(), to.end()); twice != to.end())
      return fail(CONVROT_EINVAL, "%s: page %d is a destination twice", who, *twice);
    for (int64_t i = 0; i < n; ++i)
      if (std::binary_search(to.begin(), to.end(), src[i]))
        return fail(CONVROT_EINVAL, "%s: page %d is both a source and a destination", who, src[i]);
  } catch (const std::bad_alloc&) {
    return fail(CONVROT_EHIP, "%s: no host memory", who);
  }
  return hip_status(launch_cache_copy(static_cast<uint8_t*>(pages), layers, layers > 1 ? layer_bytes : 0, page_bytes, src,
                                      dst, n, static_cast<hipStream_t>(stream)),
                    who);
}

}  // extern "C"
