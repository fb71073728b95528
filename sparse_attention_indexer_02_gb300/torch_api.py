"""torch-tensor form of the C-ABI calls (argument marshalling only).

The descriptor is read off the tensors' shapes and strides; every byte of the
result is computed by libqsa.so.  All tensors must be on the current CUDA
device; work is enqueued on the current torch stream unless one is given.
"""
from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional

import torch

from . import _abi


def _desc_from(q, kv_cache, block_table, page_cols, out_cols, kv_dtype, scale_offset):
    R, H, D = q.shape
    B, max_pages = block_table.shape
    if B == 0 or R % B:
        raise ValueError("rows must be a whole number of rows per request")
    page_stride = kv_cache.stride(0) * kv_cache.element_size()
    scales = None
    scale_stride = 0
    if kv_dtype == _abi.KV_FP8_E4M3:
        if scale_offset < 0:
            raise ValueError("fp8 keys need the scale offset inside a block")
        scales = kv_cache.data_ptr() + scale_offset
        scale_stride = page_stride
    desc = _abi.make_desc(B, R // B, H, page_cols, max_pages, kv_cache.shape[0], out_cols, page_stride,
                          kv_dtype=kv_dtype, scale_page_stride=scale_stride, head_dim=D)
    q_dtype = _abi.Q_FP8_E4M3 if q.dtype in (torch.float8_e4m3fn, torch.uint8) else _abi.Q_BF16
    return desc, scales, q_dtype


def paged_mqa_logits(q: torch.Tensor, weights: torch.Tensor, kv_cache: torch.Tensor,
                     block_table: torch.Tensor, visible_cols: torch.Tensor, *, page_cols: int,
                     out_cols: int, kv_dtype: int = _abi.KV_BF16, scale_offset: int = -1,
                     out: Optional[torch.Tensor] = None, stream=None,
                     next_n_lens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Index logits fp32 [R, out_cols] (include/qsa.h, qsa_paged_mqa_logits).

    q: bf16 [R, H, 128], or float8_e4m3fn (fp8 keys only: qsa_paged_mqa_logits_ex
    with fp8 q); weights: fp32 [R, H]; kv_cache: [num_pages, ...] paged
    keys whose dim-0 stride is the page stride; block_table: int32
    [num_requests, max_pages]; visible_cols: int32 [R].  For fp8 keys in the
    block-flat layout pass kv_dtype=KV_FP8_E4M3 and the byte offset of the
    scales inside a block (page_cols * 128).  next_n_lens (int32
    [num_requests]) selects qsa_paged_mqa_logits_ragged: a request's rows past
    its count are -inf."""
    desc, scales, q_dtype = _desc_from(q, kv_cache, block_table, page_cols, out_cols, kv_dtype, scale_offset)
    if out is None:
        out = torch.empty((q.shape[0], out_cols), dtype=torch.float32, device=q.device)
    _abi.paged_mqa_logits(desc, q, weights, kv_cache, scales, block_table, visible_cols, out, stream,
                          next_n_lens=next_n_lens, q_dtype=q_dtype)
    return out


def select_topk(logits: torch.Tensor, visible_cols: torch.Tensor, k: int,
                out: Optional[torch.Tensor] = None, stream=None, max_visible: int = 0) -> torch.Tensor:
    """Top-k column indices int32 [rows, k] (include/qsa.h, qsa_select_topk;
    with max_visible > 0, qsa_select_topk_bounded: the visible counts are
    clamped to that host bound)."""
    rows = logits.shape[0]
    if out is None:
        out = torch.empty((rows, k), dtype=torch.int32, device=logits.device)
    if max_visible > 0:
        _abi.select_topk_bounded(logits, rows, logits.stride(0), visible_cols, max_visible, k, out, stream)
    else:
        _abi.select_topk(logits, rows, logits.stride(0), visible_cols, k, out, stream)
    return out


def page_stream(pool: torch.Tensor, page_stride: int, page_bytes: int, pages: torch.Tensor,
                checksum: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Stream the listed pages of `pool` (a device buffer of whole pages) and
    XOR their 32-bit words into `checksum` (include/qsa.h, qsa_page_stream)."""
    if checksum is None:
        checksum = torch.zeros(1, dtype=torch.int32, device=pool.device)
    pool_pages = pool.numel() * pool.element_size() // page_stride
    _abi.page_stream(pool, page_stride, page_bytes, pages, pages.numel(), pool_pages, checksum, stream)
    return checksum


_workspaces: dict = {}


def topk_workspace(nbytes: int, device: torch.device) -> torch.Tensor:
    """A zeroed workspace of at least nbytes on `device`, kept for later calls
    (every completed qsa_paged_mqa_topk call leaves it zero again).  One per
    device: calls that may overlap on other streams need their own."""
    key = torch.device(device).index if torch.device(device).index is not None else torch.cuda.current_device()
    ws = _workspaces.get(key)
    if ws is None or ws.numel() * 4 < nbytes:
        ws = torch.zeros(max(64, (nbytes + 3) // 4), dtype=torch.int32, device=device)
        _workspaces[key] = ws
    return ws


def paged_mqa_topk(q: torch.Tensor, weights: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                   visible_cols: torch.Tensor, k: int, *, page_cols: int, out_cols: int,
                   kv_dtype: int = _abi.KV_BF16, scale_offset: int = -1, max_visible: int = 0,
                   out_logits: Optional[torch.Tensor] = None, out_idx: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None,
                   next_n_lens: Optional[torch.Tensor] = None):
    """(logits fp32 [R, out_cols], top-k int32 [R, k]) in one call
    (include/qsa.h, qsa_paged_mqa_topk); arguments as paged_mqa_logits, plus k
    and the host bound max_visible of the visible counts (0: unknown)."""
    desc, scales, q_dtype = _desc_from(q, kv_cache, block_table, page_cols, out_cols, kv_dtype, scale_offset)
    R = q.shape[0]
    if out_logits is None:
        out_logits = torch.empty((R, out_cols), dtype=torch.float32, device=q.device)
    if out_idx is None:
        out_idx = torch.empty((R, k), dtype=torch.int32, device=q.device)
    nbytes = _abi.topk_workspace_bytes(desc)
    if workspace is None and nbytes:
        workspace = topk_workspace(nbytes, q.device)
    _abi.paged_mqa_topk(desc, q, weights, kv_cache, scales, block_table, visible_cols, k, out_logits, out_idx,
                        workspace, 0 if workspace is None else workspace.numel() * workspace.element_size(),
                        stream, next_n_lens=next_n_lens, q_dtype=q_dtype, max_visible=max_visible)
    return out_logits, out_idx


# ---- serving operators: page maps, paged stores, paged attention -------------

_HALF = {torch.bfloat16: _abi.HALF_BF16, torch.float16: _abi.HALF_F16}


def _on(stream):
    """Context in which tensors a call allocates belong to the stream it runs on."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _vec(t: torch.Tensor, name: str, dtype: torch.dtype, *shape: int) -> None:
    _need(t.dtype == dtype and t.dim() == len(shape) and t.is_contiguous() and
          all(n < 0 or t.shape[i] == n for i, n in enumerate(shape)),
          f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} (-1: any), "
          f"got {t.dtype} {list(t.shape)} strides {list(t.stride())}")


def _table(t: torch.Tensor) -> None:
    _need(t.dtype == torch.int32 and t.dim() == 2 and (t.shape[1] <= 1 or t.stride(1) == 1),
          "block_table must be an int32 [num_requests, max_pages] tensor with contiguous rows")


def _strides(t: torch.Tensor) -> list:
    """Element strides with those of dimensions of one entry, which may be
    anything, set to what a contiguous tensor has."""
    out, inner = [], 1
    for n, st in zip(reversed(t.shape), reversed(t.stride())):
        out.append(st if n > 1 else inner)
        inner *= max(n, 1)
    return out[::-1]


class PageMaps(NamedTuple):
    """What build_page_maps writes beside the block table (include/qsa.h)."""
    query_start: torch.Tensor    # int32 [B + 1]
    seq_lens: torch.Tensor       # int32 [B]
    slots: torch.Tensor          # int64 [max_tokens]
    positions: torch.Tensor      # int32 [max_tokens]
    token_request: torch.Tensor  # int32 [max_tokens]
    visible_cols: torch.Tensor   # int32 [max_tokens]
    column_slots: torch.Tensor   # int64 [max_tokens]
    pages_used: torch.Tensor     # int32 [1]


def build_page_maps(context_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                    block_table: torch.Tensor, *, page_tokens: int, max_tokens: int, ratio: int = 1,
                    partial_cols: bool = False, out: Optional[PageMaps] = None, stream=None) -> PageMaps:
    """Page bookkeeping of one step on the device (include/qsa.h,
    qsa_build_page_maps): block_table is extended in place with pages of
    free_pages, the rest is returned (or written into `out`, a PageMaps whose
    tensors a captured graph keeps).  context_lens, new_lens: int32 [B];
    free_pages: int32; block_table: int32 [B, max_pages]; max_tokens: rows of
    the per-token outputs (padding past the step's tokens)."""
    B = context_lens.numel()
    _vec(context_lens, "context_lens", torch.int32, -1)
    _vec(new_lens, "new_lens", torch.int32, B)
    _vec(free_pages, "free_pages", torch.int32, -1)
    _table(block_table)
    _need(block_table.shape[0] == B, "block_table must have a row a request")
    _need(max_tokens >= 0, "max_tokens < 0")
    if out is None:
        dev = context_lens.device
        with _on(stream):
            i32 = lambda n: torch.empty(n, dtype=torch.int32, device=dev)  # noqa: E731
            i64 = lambda n: torch.empty(n, dtype=torch.int64, device=dev)  # noqa: E731
            out = PageMaps(i32(B + 1), i32(B), i64(max_tokens), i32(max_tokens), i32(max_tokens), i32(max_tokens),
                           i64(max_tokens), i32(1))
    else:
        for t, name, dt, n in ((out.query_start, "query_start", torch.int32, B + 1),
                               (out.seq_lens, "seq_lens", torch.int32, B),
                               (out.slots, "slots", torch.int64, max_tokens),
                               (out.positions, "positions", torch.int32, max_tokens),
                               (out.token_request, "token_request", torch.int32, max_tokens),
                               (out.visible_cols, "visible_cols", torch.int32, max_tokens),
                               (out.column_slots, "column_slots", torch.int64, max_tokens),
                               (out.pages_used, "pages_used", torch.int32, 1)):
            _vec(t, name, dt, n)
    desc = _abi.PageMapsDesc(B, int(page_tokens), block_table.shape[1], int(ratio), 1 if partial_cols else 0, 0,
                             _strides(block_table)[0], free_pages.numel(), int(max_tokens))
    _abi.build_page_maps(desc, context_lens, new_lens, free_pages, block_table, *out, stream=stream)
    return out


def _kv_desc(k_cache: torch.Tensor, v_cache: torch.Tensor) -> _abi.KvDesc:
    _need(k_cache.dtype in _HALF and v_cache.dtype == k_cache.dtype, "the caches must both be bf16 or both fp16")
    _need(k_cache.dim() == 4 and v_cache.shape == k_cache.shape,
          "the caches must be [num_pages, page_tokens, num_kv_heads, head_dim], values like keys")
    _need(k_cache.stride(3) == 1 and v_cache.stride(3) == 1, "the caches' last dimension must be contiguous")
    e = 2
    pages, pt, h, d = k_cache.shape
    return _abi.KvDesc(_HALF[k_cache.dtype], pages, pt, h, d, 0, *(s * e for s in _strides(k_cache)[:3]),
                       *(s * e for s in _strides(v_cache)[:3]))


def store_paged_kv(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, *, stream=None) -> None:
    """Write key and value rows into their cache slots (include/qsa.h,
    qsa_store_paged_kv).  k, v: [T, num_kv_heads, head_dim] in the caches' type,
    any token and head strides (multiples of 8 elements), so views of a fused
    projection go as they are; slots: int64 [T], rows with a slot outside the
    cache are skipped; caches: [num_pages, page_tokens, num_kv_heads, head_dim]
    of any strides (permute a head-major cache into this order)."""
    desc = _kv_desc(k_cache, v_cache)
    T = slots.numel()
    _vec(slots, "slots", torch.int64, -1)
    for t, name in ((k, "k"), (v, "v")):
        _need(t.dtype == k_cache.dtype and t.dim() == 3 and tuple(t.shape) == (T, *k_cache.shape[2:]) and
              t.stride(2) == 1, f"{name} must be [T, num_kv_heads, head_dim] in the cache's type, last dimension "
              f"contiguous")
    ks, vs = _strides(k), _strides(v)
    _abi.store_paged_kv(desc, k, ks[0] * 2, ks[1] * 2, v, vs[0] * 2, vs[1] * 2, slots, T, k_cache, v_cache, stream)


def store_index_keys(keys: torch.Tensor, slots: torch.Tensor, kv_cache: torch.Tensor, *, page_cols: int,
                     kv_dtype: int = _abi.KV_BF16, scale_offset: int = -1, stream=None) -> None:
    """Write compressed index keys into the paged index cache paged_mqa_logits
    reads (include/qsa.h, qsa_store_index_keys).  keys: bf16 [T, 128]; slots:
    int64 [T] column slots (build_page_maps' column_slots), rows outside the
    cache skipped; kv_cache, page_cols, kv_dtype and scale_offset as in
    paged_mqa_logits (fp8: keys are quantised with one scale each)."""
    T = slots.numel()
    _vec(slots, "slots", torch.int64, -1)
    _need(keys.dtype == torch.bfloat16 and keys.dim() == 2 and keys.shape[0] == T and keys.stride(1) == 1,
          "keys must be bf16 [T, head_dim] with contiguous rows")
    stride = kv_cache.stride(0) * kv_cache.element_size()
    fp8 = kv_dtype == _abi.KV_FP8_E4M3
    _need(not fp8 or scale_offset >= 0, "fp8 keys need the scale offset inside a block")
    _need(fp8 or kv_cache.dtype == torch.bfloat16, "a bf16 index cache must be a bf16 tensor")
    used = scale_offset + 4 * page_cols if fp8 else page_cols * 256
    _need(kv_cache[0].is_contiguous() and kv_cache[0].numel() * kv_cache.element_size() >= used if len(kv_cache)
          else False, "a page of kv_cache must be contiguous and hold page_cols keys (and scales)")
    desc = _abi.IndexCacheDesc(kv_dtype, kv_cache.shape[0], int(page_cols), keys.shape[1], stride, stride if fp8 else 0)
    _abi.store_index_keys(desc, keys, _strides(keys)[0] * 2, slots, T, kv_cache,
                          kv_cache.data_ptr() + scale_offset if fp8 else None, stream)


_attn_workspaces: dict = {}


def _attention_workspace(nbytes: int, device: torch.device, stream) -> torch.Tensor:
    with _on(stream):
        def fresh():
            ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
            ws[:_abi.ATTN_COUNTER_BYTES].zero_()
            return ws

        if torch.cuda.is_current_stream_capturing():
            return fresh()  # belongs to the graph: replays must not meet eager calls in it
        key = (torch.cuda.current_device(), torch.cuda.current_stream().cuda_stream)
        ws = _attn_workspaces.get(key)
        if ws is None or ws.numel() < nbytes:
            ws = _attn_workspaces[key] = fresh()
        return ws


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    query_start: torch.Tensor, seq_lens: torch.Tensor, *, scale: Optional[float] = None,
                    max_new: int = 0, selected: Optional[torch.Tensor] = None, ratio: int = 1, local_tokens: int = 0,
                    form: int = _abi.ATTN_AUTO, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of the requests' new tokens over their paged cache
    (include/qsa.h, qsa_paged_attention): out [T, num_q_heads, head_dim], and
    with return_lse (or a given lse tensor) also lse fp32 [T, num_q_heads].

    q: [T, num_q_heads, head_dim] in the caches' type, any token and head
    strides; caches as in store_paged_kv; block_table: int32 [B, max_pages];
    query_start: int32 [B + 1]; seq_lens: int32 [B].  scale: 1/sqrt(head_dim)
    unless given.  max_new: the host's bound on a request's new tokens (0:
    unknown), which only chooses the kernel form.  selected: int32 [T, k]
    columns of `ratio` tokens (select_topk's output): a row then sees these and
    its last `local_tokens` tokens only.

    Without a workspace, one is kept for each stream that calls; a call under
    graph capture gets its own, cleared again by every replay (a given
    workspace, zeroed once, spares that)."""
    _need(q.dim() == 3 and q.dtype == k_cache.dtype and q.stride(2) == 1,
          "q must be [T, num_q_heads, head_dim] in the caches' type, last dimension contiguous")
    kv = _kv_desc(k_cache, v_cache)
    T, H, D = q.shape
    _need(D == kv.head_dim, "q and the caches differ in head_dim")
    _table(block_table)
    B = block_table.shape[0]
    _vec(query_start, "query_start", torch.int32, B + 1)
    _vec(seq_lens, "seq_lens", torch.int32, B)
    k = 0
    if selected is not None:
        _vec(selected, "selected", torch.int32, T, -1)
        k = selected.shape[1]
        _need(k > 0, "selected lists no columns")
    with _on(stream):
        if out is None:
            out = torch.empty((T, H, D), dtype=q.dtype, device=q.device)
        if lse is None and return_lse:
            lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    _need(out.shape == q.shape and out.dtype == q.dtype and out.stride(2) == 1,
          "out must have q's shape and type, last dimension contiguous")
    if lse is not None:
        _vec(lse, "lse", torch.float32, T, H)
    e, qs, os = 2, _strides(q), _strides(out)
    desc = _abi.AttnDesc(kv, B, H, block_table.shape[1], int(max_new), k, int(ratio), int(local_tokens), int(form), T,
                         _strides(block_table)[0], qs[0] * e, qs[1] * e, os[0] * e, os[1] * e,
                         D ** -0.5 if scale is None else float(scale), 0)
    nbytes = _abi.paged_attention_workspace_bytes(desc)
    if workspace is None:
        workspace = _attention_workspace(nbytes, q.device, stream)
    _abi.paged_attention(desc, q, k_cache, v_cache, block_table, query_start, seq_lens, selected, out, lse, workspace,
                         workspace.numel() * workspace.element_size(), stream)
    return out if lse is None else (out, lse)
