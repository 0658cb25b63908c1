// moe_kv.h — what the paged-cache operators share on the host: checks of a
// cache description.
#pragma once

#include "moe_internal.h"

namespace moe {

// n / d for 0 <= n < 2^31 by a multiplication: m = ceil(2^(31 + s) / d) with
// s = ceil(log2 d) is below 2^32 and exact there.
struct FastDiv {
  uint32_t mul = 0;  // 0: d = 1
  int32_t shift = 0;
  FastDiv() = default;
  explicit FastDiv(int32_t d) {
    int s = 0;
    while ((1ll << s) < d) ++s;
    mul = s ? static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d) : 0u;
    shift = s - 1;
  }
  __device__ __forceinline__ int operator()(int n) const {
    return mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(n), mul) >> shift) : n;
  }
};

inline bool ptr16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks a cache description against the new tensors' dtype.
inline moe_status_t check_cache(const moe_kv_cache_t* c, int32_t dtype) {
  if (!c) return set_error(MOE_ERR_INVALID_ARG, "cache is NULL");
  if (dtype != MOE_F16 && dtype != MOE_BF16)
    return set_error(MOE_ERR_UNSUPPORTED, "dtype must be MOE_F16 or MOE_BF16");
  if (c->dtype != dtype && c->dtype != MOE_E4M3)
    return set_error(MOE_ERR_UNSUPPORTED, "cache: dtype must be the new tensors' or MOE_E4M3");
  if (c->n_pages < 1 || c->page_size < 1 || c->n_kv_heads < 1 || c->head_dim < 1)
    return set_error(MOE_ERR_INVALID_ARG, "cache: sizes must be positive");
  const int lane = c->dtype == MOE_E4M3 ? 16 : 8;  // elements of 16 bytes
  if (c->head_dim % lane || c->head_dim > 256)
    return set_error(MOE_ERR_UNSUPPORTED, "cache: head_dim must be a multiple of %d up to 256", lane);
  const int64_t s = c->k_page_stride | c->k_token_stride | c->k_head_stride | c->v_page_stride | c->v_token_stride |
                    c->v_head_stride;
  const int64_t most = INT32_MAX / 2 + 1;  // 2^30 elements, below 2^32 bytes
  for (int64_t v : {c->k_page_stride, c->k_token_stride, c->k_head_stride, c->v_page_stride, c->v_token_stride,
                    c->v_head_stride})
    if (v < 0 || v > most) return set_error(MOE_ERR_UNSUPPORTED, "cache: strides must be from 0 to 2^30 elements");
  if (s % lane) return set_error(MOE_ERR_UNSUPPORTED, "cache: strides must be multiples of 16 bytes");
  if (!c->k || !c->v) return set_error(MOE_ERR_INVALID_ARG, "cache: k / v is NULL");
  if (!ptr16(c->k) || !ptr16(c->v)) return set_error(MOE_ERR_INVALID_ARG, "cache: k / v is not 16-byte aligned");
  if (c->dtype != MOE_E4M3 && (c->k_scale || c->v_scale))
    return set_error(MOE_ERR_INVALID_ARG, "cache: scales go with MOE_E4M3 only");
  if ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) & 3u)
    return set_error(MOE_ERR_INVALID_ARG, "cache: scales are not 4-byte aligned");
  return MOE_OK;
}

}  // namespace moe
