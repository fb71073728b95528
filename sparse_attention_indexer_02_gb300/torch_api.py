"""torch-tensor form of the C-ABI calls (argument marshalling only).

The descriptor is read off the tensors' shapes and strides; every byte of the
result is computed by libqsa.so.  All tensors must be on the current CUDA
device; work is enqueued on the current torch stream unless one is given.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _abi


class _Binding:
    """The module _qsa_torch, loaded by its first use; loud when it is missing."""

    def __getattr__(self, name):
        _abi.load_library()  # _qsa_torch links against libqsa.so
        try:
            from . import _qsa_torch as mod
        except ImportError as e:
            raise RuntimeError("_qsa_torch is not built for this torch: run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`") from e
        for n in ("build_page_maps", "store_paged_kv", "store_index_keys", "paged_attention", "drop_workspaces"):
            setattr(self, n, getattr(mod, n))
        return getattr(mod, name)


_qsa_torch = _Binding()


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _dense(t, dtype, n):
    return t.dtype is dtype and t.is_contiguous() and t.numel() >= n


def _check_scored(q, weights, block_table):
    """The scorers take these by address and shape alone."""
    _need(q.dim() == 3 and q.is_contiguous() and q.element_size() <= 2 and q.dtype is not torch.float16,
          "q must be a contiguous bf16 (or e4m3) [R, H, 128] tensor")
    _need(_dense(weights, torch.float32, q.shape[0] * q.shape[1]), "weights must be a contiguous fp32 [R, H] tensor")
    _need(block_table.dim() == 2 and block_table.dtype is torch.int32,
          "block_table must be an int32 [num_requests, max_pages] tensor")


def _refuse(q, weights, kv_cache, block_table, visible_cols, next_n_lens, out, out_cols):
    """Says what of a scoring call's tensors does not fit."""
    _check_scored(q, weights, block_table)
    R, B = q.shape[0], block_table.shape[0]
    _need(block_table.is_contiguous(), "block_table must be contiguous (a slice of a wider table's columns is not)")
    _need(_dense(visible_cols, torch.int32, R), "visible_cols must be a contiguous int32 [R] tensor")
    _need(next_n_lens is None or _dense(next_n_lens, torch.int32, B),
          "next_n_lens must be a contiguous int32 [num_requests] tensor")
    _need(out is None or _dense(out, torch.float32, R * out_cols), "out must be a contiguous fp32 [R, out_cols] tensor")
    inner = 1
    for n, step in zip(reversed(kv_cache.shape[1:]), reversed(kv_cache.stride()[1:])):
        _need(n == 1 or step == inner, "a page of kv_cache must be contiguous")
        inner *= n


def _desc_from(q, weights, kv_cache, block_table, visible_cols, next_n_lens, out, page_cols, out_cols, kv_dtype,
               scale_offset):
    try:
        R, H, D = q.shape
        B, max_pages = block_table.shape
    except ValueError:
        R = H = D = B = max_pages = 0
    # the usual call in one expression (through the helpers alone: a microsecond more a call)
    if not (q.is_contiguous() and weights.is_contiguous() and block_table.is_contiguous() and
            visible_cols.is_contiguous() and kv_cache.is_contiguous() and next_n_lens is None and
            q.dtype is _BF16 and weights.dtype is _F32 and block_table.dtype is _I32 and visible_cols.dtype is _I32 and
            weights.numel() == R * H > 0 and visible_cols.numel() == R and
            (out is None or out.dtype is _F32 and out.is_contiguous() and out.numel() == R * out_cols)):
        _refuse(q, weights, kv_cache, block_table, visible_cols, next_n_lens, out, out_cols)
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
    its count are -inf.  All but kv_cache's pages are contiguous (ValueError
    otherwise)."""
    desc, scales, q_dtype = _desc_from(q, weights, kv_cache, block_table, visible_cols, next_n_lens, out, page_cols,
                                       out_cols, kv_dtype, scale_offset)
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
    desc, scales, q_dtype = _desc_from(q, weights, kv_cache, block_table, visible_cols, next_n_lens, out_logits,
                                       page_cols, out_cols, kv_dtype, scale_offset)
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
# Checked and called from _qsa_torch (csrc/torch_binding.cpp): tensors that do
# not fit a call raise ValueError, a status of the C ABI other than OK QSAError.

def _on(stream):
    """Context in which a call's launches and allocations belong to `stream`
    (a stream, or a handle; ExternalStream takes handle 0, the default stream's,
    for "none given" and makes another stream)."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


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
    tensors a captured graph keeps; new ones share one allocation).
    context_lens, new_lens: int32 [B]; free_pages: int32; block_table: int32
    [B, max_pages]; max_tokens: rows of the per-token outputs (padding past the
    step's tokens)."""
    if stream is not None:
        with _on(stream):
            return build_page_maps(context_lens, new_lens, free_pages, block_table, page_tokens=page_tokens,
                                   max_tokens=max_tokens, ratio=ratio, partial_cols=partial_cols, out=out)
    st, maps = _qsa_torch.build_page_maps(context_lens, new_lens, free_pages, block_table, page_tokens, max_tokens,
                                          ratio, partial_cols, out, PageMaps)
    if st:
        _abi._check(st)
    return maps


def store_paged_kv(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, *, stream=None) -> None:
    """Write key and value rows into their cache slots (include/qsa.h,
    qsa_store_paged_kv).  k, v: [T, num_kv_heads, head_dim] in the caches' type,
    any token and head strides (multiples of 8 elements), so views of a fused
    projection go as they are; slots: int64 [T], rows with a slot outside the
    cache are skipped; caches: [num_pages, page_tokens, num_kv_heads, head_dim]
    of any strides (permute a head-major cache into this order)."""
    if stream is not None:
        with _on(stream):
            return store_paged_kv(k, v, slots, k_cache, v_cache)
    st = _qsa_torch.store_paged_kv(k, v, slots, k_cache, v_cache)
    if st:
        _abi._check(st)


def store_index_keys(keys: torch.Tensor, slots: torch.Tensor, kv_cache: torch.Tensor, *, page_cols: int,
                     kv_dtype: int = _abi.KV_BF16, scale_offset: int = -1, stream=None) -> None:
    """Write compressed index keys into the paged index cache paged_mqa_logits
    reads (include/qsa.h, qsa_store_index_keys).  keys: bf16 [T, 128]; slots:
    int64 [T] column slots (build_page_maps' column_slots), rows outside the
    cache skipped; kv_cache, page_cols, kv_dtype and scale_offset as in
    paged_mqa_logits (fp8: keys are quantised with one scale each)."""
    if stream is not None:
        with _on(stream):
            return store_index_keys(keys, slots, kv_cache, page_cols=page_cols, kv_dtype=kv_dtype,
                                    scale_offset=scale_offset)
    st = _qsa_torch.store_index_keys(keys, slots, kv_cache, page_cols, kv_dtype, scale_offset)
    if st:
        _abi._check(st)


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
    strides; caches as in store_paged_kv; block_table: int32 [B, max_pages]
    (tokens of an entry of -1, a page build_page_maps could not get, are not
    seen); query_start: int32 [B + 1]; seq_lens: int32 [B].  scale:
    1/sqrt(head_dim) unless given.  max_new: the host's bound on a request's new tokens (0:
    unknown), which only chooses the kernel form.  selected: int32 [T, k]
    columns of `ratio` tokens (select_topk's output): a row then sees these and
    its last `local_tokens` tokens only.

    Without a workspace, one is kept for each stream that calls (the 32 streams
    that called last); a call under
    graph capture gets its own, cleared again by every replay (a given
    workspace, zeroed once, spares that)."""
    if stream is not None:
        with _on(stream):
            return paged_attention(q, k_cache, v_cache, block_table, query_start, seq_lens, scale=scale,
                                   max_new=max_new, selected=selected, ratio=ratio, local_tokens=local_tokens,
                                   form=form, out=out, lse=lse, return_lse=return_lse, workspace=workspace)
    st, out, lse = _qsa_torch.paged_attention(q, k_cache, v_cache, block_table, query_start, seq_lens, scale, max_new,
                                              selected, ratio, local_tokens, form, out, lse, return_lse, workspace)
    if st:
        _abi._check(st)
    return out if lse is None else (out, lse)


def drop_attention_workspaces() -> None:
    """Forget the workspaces paged_attention keeps (the next call on each stream
    makes a new one).  device_status does so itself when it clears bit 3, a call
    that gave up on a wait: that may leave their counters uncleared."""
    _qsa_torch.drop_workspaces()
