// Host-side checks shared by the C entries (serving_abi.cu, step_abi.cu).
#pragma once

#include "qsa_internal.h"

namespace qsa {
namespace abi {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline qsa_status bad(const char* what) { return set_error(QSA_ERR_INVALID_ARG, "%s", what); }

inline qsa_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return QSA_OK;
  return set_error(QSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool stride_ok(int64_t s) { return s > 0 && s % 16 == 0; }

inline qsa_status validate_kv(const qsa_kv_desc& d) {
  if (d.dtype != QSA_HALF_BF16 && d.dtype != QSA_HALF_F16)
    return set_error(QSA_ERR_INVALID_ARG, "unknown cache dtype %d", d.dtype);
  if (d.num_pages < 1) return bad("num_pages < 1");
  if (d.page_tokens < 1) return bad("page_tokens < 1");
  if (d.num_kv_heads < 1) return bad("num_kv_heads < 1");
  if (d.head_dim < 8 || d.head_dim > 1024 || d.head_dim % 8 != 0)
    return set_error(QSA_ERR_INVALID_ARG, "head_dim must be a multiple of 8 in 8..1024 (got %d)", d.head_dim);
  if (d.reserved != 0) return bad("kv.reserved must be 0");
  if (!stride_ok(d.k_page_stride) || !stride_ok(d.k_token_stride) || !stride_ok(d.k_head_stride) ||
      !stride_ok(d.v_page_stride) || !stride_ok(d.v_token_stride) || !stride_ok(d.v_head_stride))
    return bad("cache strides must be positive multiples of 16 bytes");
  return QSA_OK;
}

}  // namespace abi
}  // namespace qsa
