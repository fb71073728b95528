"""One serving step of sparse attention over paged caches, from the requests'
lengths to the attention output: page maps, stores, index scoring, top-k and
attention to the selected columns, all on the device.

    pool = PagedPool(num_pages=4096, page_tokens=64, num_kv_heads=8, head_dim=128)
    res = step(pool, block_table, context_lens, new_lens, free_pages, q=q, k=k, v=v, index_q=iq,
               index_keys=ik, index_weights=iw, top_k=2048, local_tokens=64, max_context=131072)

Every call goes to the current stream, nothing waits for the device, and the
shapes depend on host values only, so a step can be captured in a CUDA graph.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _abi, torch_api


class PagedPool:
    """Key, value and index-key caches that share one pool of pages.

    A page holds page_tokens tokens, and page_tokens / ratio compressed index
    columns of them.  index_fp8 keeps the index keys as e4m3 with a scale each
    (132 bytes a column in place of 256, a page rounded up to 16 bytes, as the
    scoring takes them)."""

    def __init__(self, num_pages: int, page_tokens: int, num_kv_heads: int, head_dim: int, ratio: int = 4,
                 dtype: torch.dtype = torch.bfloat16, index_fp8: bool = False, device="cuda"):
        if page_tokens % ratio:
            raise ValueError("ratio must divide page_tokens")
        self.page_tokens, self.ratio, self.page_cols = page_tokens, ratio, page_tokens // ratio
        kv = torch.zeros((2, num_pages, page_tokens, num_kv_heads, head_dim), dtype=dtype, device=device)
        self.k_cache, self.v_cache = kv[0], kv[1]
        if index_fp8:
            self.index = torch.zeros((num_pages, -(-self.page_cols * 132 // 16) * 16), dtype=torch.uint8, device=device)
            self.index_args = dict(page_cols=self.page_cols, kv_dtype=_abi.KV_FP8_E4M3, scale_offset=self.page_cols * 128)
        else:
            self.index = torch.zeros((num_pages, self.page_cols, 128), dtype=torch.bfloat16, device=device)
            self.index_args = dict(page_cols=self.page_cols)


class StepResult(NamedTuple):
    out: torch.Tensor          # [T, num_q_heads, head_dim]
    lse: torch.Tensor          # fp32 [T, num_q_heads]
    selected: torch.Tensor     # int32 [T, top_k]
    maps: torch_api.PageMaps

    def valid(self) -> torch.Tensor:
        """A bool on the device, for a caller whose lengths or free pages live there
        alone: every request brought the same number of new tokens, and every
        token got a cache slot.  Where it is false, rows were scored for another
        request than their own, or tokens (theirs or later ones') are not in the
        caches and not seen; the step's results are not to be used."""
        T, B = self.out.shape[0], self.maps.seq_lens.shape[0]
        rows = torch.arange(B + 1, device=self.out.device) * (T // B)
        return (self.maps.query_start == rows).all() & (self.maps.slots >= 0).all()


def step(pool: PagedPool, block_table: torch.Tensor, context_lens: torch.Tensor, new_lens: torch.Tensor,
         free_pages: torch.Tensor, *, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, index_q: torch.Tensor,
         index_keys: torch.Tensor, index_weights: torch.Tensor, top_k: int, max_context: int, local_tokens: int = 0,
         scale: Optional[float] = None) -> StepResult:
    """The step for B requests of T / B new tokens each (decode rows, rows to
    verify, or prompt chunks of one length; new_lens holds that count).

    block_table int32 [B, max_pages] is extended in place from free_pages;
    q, k, v, index_q [T, index heads, 128], index_keys [T, 128] (the compressed
    key of the column a token completes; other rows are ignored) and
    index_weights [T, index heads] are request-major.  max_context bounds the
    requests' tokens.  A token attends to the top_k complete columns its index
    scores select and to its last local_tokens tokens.

    Nothing of the device is read, so neither a new_lens that holds other counts
    nor a free list with too few pages raises: StepResult.valid() tells.

    Views are taken as they are; of block_table (columns of a wider table),
    index_q and index_weights the scoring gets a contiguous copy."""
    T, B = q.shape[0], block_table.shape[0]
    if B == 0 or T == 0 or T % B:
        raise ValueError("rows must be a whole number of rows per request")
    index_q, index_weights = index_q.contiguous(), index_weights.contiguous()
    torch_api._check_scored(index_q, index_weights, block_table)  # before anything is launched
    if index_q.shape[0] != T:
        raise ValueError("index_q must have a row a token")
    maps = torch_api.build_page_maps(context_lens, new_lens, free_pages, block_table, page_tokens=pool.page_tokens,
                                     max_tokens=T, ratio=pool.ratio)
    scored_table = block_table.contiguous()
    torch_api.store_paged_kv(k, v, maps.slots, pool.k_cache, pool.v_cache)
    torch_api.store_index_keys(index_keys, maps.column_slots, pool.index, **pool.index_args)
    cols = max(1, max_context // pool.ratio)
    logits = torch_api.paged_mqa_logits(index_q, index_weights, pool.index, scored_table, maps.visible_cols,
                                        out_cols=cols, **pool.index_args)
    selected = torch_api.select_topk(logits, maps.visible_cols, top_k, max_visible=cols)
    out, lse = torch_api.paged_attention(q, pool.k_cache, pool.v_cache, block_table, maps.query_start, maps.seq_lens,
                                         scale=scale, max_new=T // B, selected=selected, ratio=pool.ratio,
                                         local_tokens=local_tokens, return_lse=True)
    return StepResult(out, lse, selected, maps)
