"""GB300 (sm_103a) QSA-indexer hot path: paged MQA-logits scoring and per-row top-k,
and the serving operators around it (page maps, head rotation, paged stores, paged
attention, draft verification).

The compute lives in libqsa.so (CUDA kernels behind the C ABI in include/qsa.h).
This package is its thin binding: :mod:`._abi` marshals pointers and sizes
through ctypes, :mod:`.torch_api` takes torch tensors and passes their device
pointers and the current stream, and :mod:`.build` compiles the library.
"""
from ._abi import (ATTN_AUTO, ATTN_COUNTER_BYTES, ATTN_GATHER, ATTN_TILE, AttnDesc, EXPORTED, HALF_BF16, HALF_F16,
                   HeadRows, NORM_LAYER, NORM_NONE, NORM_RMS, PROBS_BF16, PROBS_F16, PROBS_F32, ROTARY_HALF,
                   ROTARY_PAIRS, RotaryDesc, VerifyDesc,
                   IndexCacheDesc, KvDesc, PageMapsDesc, KV_BF16, KV_FP8_E4M3, LIB_PATH, Q_BF16, Q_FP8_E4M3, QSA_ERR_CUDA, QSA_ERR_INVALID_ARG,
                   QSA_ERR_UNSUPPORTED, QSA_OK, VARIANT_AUTO, VARIANT_NAMES, VARIANT_ROWCORE,
                   VARIANT_UMMA, VARIANT_UMMA_LEAN, VARIANT_UMMA_TOPK, PagedDesc, QSAError, abi_version, device_status,
                   force_variant, last_error, last_variant, load_library, make_desc, page_stream,
                   paged_attention_workspace_bytes, paged_mqa_logits, paged_mqa_topk, plan_attention, plan_variant, select_topk, select_topk_bounded, status_string,
                   topk_workspace_bytes)

__all__ = [
    "EXPORTED", "KV_BF16", "KV_FP8_E4M3", "LIB_PATH", "Q_BF16", "Q_FP8_E4M3", "QSA_OK", "QSA_ERR_INVALID_ARG", "QSA_ERR_UNSUPPORTED",
    "QSA_ERR_CUDA", "VARIANT_AUTO", "VARIANT_ROWCORE", "VARIANT_UMMA", "VARIANT_UMMA_LEAN", "VARIANT_UMMA_TOPK", "VARIANT_NAMES",
    "PagedDesc", "QSAError", "abi_version", "device_status", "force_variant", "last_error", "last_variant",
    "load_library", "make_desc", "page_stream", "paged_mqa_logits", "paged_mqa_topk", "plan_variant", "select_topk",
    "select_topk_bounded", "status_string", "topk_workspace_bytes", "ATTN_AUTO", "ATTN_COUNTER_BYTES", "ATTN_GATHER",
    "ATTN_TILE", "AttnDesc", "HALF_BF16", "HALF_F16", "IndexCacheDesc", "KvDesc", "PageMapsDesc",
    "paged_attention_workspace_bytes", "plan_attention", "HeadRows", "NORM_LAYER", "NORM_NONE", "NORM_RMS", "PROBS_BF16",
    "PROBS_F16", "PROBS_F32", "ROTARY_HALF", "ROTARY_PAIRS", "RotaryDesc", "VerifyDesc",
]
