// C ABI of the serving operators: host-side validation, dispatch and launches.
// Declarations, argument meaning and error behaviour are in include/qsa.h.
#include <math.h>

#include "abi_checks.h"
#include "qsa_internal.h"

namespace {

using namespace qsa::abi;
using qsa::set_error;

qsa_status validate_attn(const qsa_attn_desc* d) {
  if (!d) return bad("desc is NULL");
  qsa_status st = validate_kv(d->kv);
  if (st != QSA_OK) return st;
  if (d->kv.head_dim != 64 && d->kv.head_dim != 128)
    return set_error(QSA_ERR_UNSUPPORTED, "attention serves head_dim 64 and 128 (got %d)", d->kv.head_dim);
  if (d->num_requests < 0) return bad("num_requests < 0");
  if (d->num_q_heads < 1 || d->num_q_heads % d->kv.num_kv_heads != 0)
    return bad("num_q_heads must be a positive multiple of num_kv_heads");
  if (d->num_q_heads / d->kv.num_kv_heads > 256) return bad("more than 256 query heads a key/value head");
  if (d->max_pages < 1) return bad("max_pages < 1");
  if (d->max_new < 0) return bad("max_new < 0");
  if (d->num_selected < 0) return bad("num_selected < 0");
  if (d->ratio < 1) return bad("ratio < 1");
  if (d->local_tokens < 0) return bad("local_tokens < 0");
  if (d->num_selected > 0 && (int64_t)d->num_selected * d->ratio + d->local_tokens > 0x3FFFFFFFLL)
    return bad("num_selected * ratio + local_tokens is too large");
  if (d->form != QSA_ATTN_AUTO && d->form != QSA_ATTN_GATHER && d->form != QSA_ATTN_TILE)
    return set_error(QSA_ERR_INVALID_ARG, "unknown attention form %d", d->form);
  if (d->num_tokens < 0 || d->num_tokens > 0x7FFFFFFFLL) return bad("num_tokens out of range");
  if (d->table_stride < 0) return bad("table_stride < 0");
  if (!stride_ok(d->q_token_stride) || !stride_ok(d->q_head_stride) || !stride_ok(d->out_token_stride) ||
      !stride_ok(d->out_head_stride))
    return bad("q and out strides must be positive multiples of 16 bytes");
  if (!(d->scale > 0.0f) || isinf(d->scale)) return bad("scale must be finite and positive");
  if (d->reserved != 0) return bad("reserved must be 0");
  return QSA_OK;
}

// Query rows a key/value head has of a request, as far as the host knows.
int64_t query_rows(const qsa_attn_desc* d) {
  int64_t toks = d->max_new;
  if (toks == 0 && d->num_requests > 0) toks = (d->num_tokens + d->num_requests - 1) / d->num_requests;
  return toks * (d->num_q_heads / d->kv.num_kv_heads);
}

qsa_status plan_form(const qsa_attn_desc* d, int32_t* form) {
  qsa_status st = validate_attn(d);
  if (st != QSA_OK) return st;
  const char* why = "";
  const bool tile = qsa::attn_tile_supports(*d, &why);
  if (d->form == QSA_ATTN_TILE && !tile)
    return set_error(QSA_ERR_UNSUPPORTED, "the tile form cannot serve this shape: %s", why);
  if (d->form != QSA_ATTN_AUTO) {
    *form = d->form;
    return QSA_OK;
  }
  *form = tile && query_rows(d) > qsa::kTileAbove ? QSA_ATTN_TILE : QSA_ATTN_GATHER;
  return QSA_OK;
}

// window 0: every key up to a row's own is seen (or the selected ones).
qsa_status attention(const qsa_attn_desc* d, int32_t window, int32_t sinks, const void* q, const void* k_cache,
                     const void* v_cache, const int32_t* block_table, const int32_t* query_start,
                     const int32_t* seq_lens, const int32_t* selected, void* out, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int32_t form = 0;
  qsa_status st = plan_form(d, &form);
  if (st != QSA_OK) return st;
  // Short windows of rows that fit the gathered form's tiles (us, gathered / tiles: 16
  // requests of 32 rows and 128 keys 11.2 / 14.3, 9 of 24 and 300 11.5 / 16.1; of 1024
  // keys tiles win, 22.6 / 18.2).  Tiles' workspace is the larger one.
  if (window > 0 && d->form == QSA_ATTN_AUTO && query_rows(d) <= qsa::kGatherRows &&
      (int64_t)window + sinks <= qsa::kGatherWindow)
    form = QSA_ATTN_GATHER;
  if (d->num_selected > 0 && !selected && d->num_tokens > 0) return bad("num_selected > 0 needs the selected columns");
  if (d->num_selected == 0 && selected) return bad("selected given with num_selected 0");
  if (d->num_requests == 0 || d->num_tokens == 0) return QSA_OK;
  if (!q || !k_cache || !v_cache || !block_table || !query_start || !seq_lens || !out)
    return bad("a required pointer is NULL");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
    return bad("q, the caches and out must be 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(query_start, 4) || !aligned(seq_lens, 4) || !aligned(selected, 4) ||
      !aligned(lse, 4))
    return bad("a 4-byte pointer is misaligned");
  const size_t need = form == QSA_ATTN_TILE ? qsa::attn_tile_workspace(d->kv.head_dim)
                                            : qsa::attn_gather_workspace(d->kv.head_dim);
  if (!workspace || workspace_bytes < need) return set_error(QSA_ERR_INVALID_ARG, "workspace below %zu bytes", need);
  if (!aligned(workspace, 16)) return bad("workspace is not 16-byte aligned");
  qsa::AttnParams p = {};
  p.q = (const uint8_t*)q;
  p.k = (const uint8_t*)k_cache;
  p.v = (const uint8_t*)v_cache;
  p.out = (uint8_t*)out;
  p.lse = lse;
  p.block_table = block_table;
  p.query_start = query_start;
  p.seq_lens = seq_lens;
  p.selected = selected;
  cudaError_t e = qsa::fault_word_address(&p.fault);
  if (e != cudaSuccess) return launched(e, "fault word");
  p.q_token_stride = d->q_token_stride;
  p.q_head_stride = d->q_head_stride;
  p.out_token_stride = d->out_token_stride;
  p.out_head_stride = d->out_head_stride;
  p.k_page_stride = d->kv.k_page_stride;
  p.k_token_stride = d->kv.k_token_stride;
  p.k_head_stride = d->kv.k_head_stride;
  p.v_page_stride = d->kv.v_page_stride;
  p.v_token_stride = d->kv.v_token_stride;
  p.v_head_stride = d->kv.v_head_stride;
  p.table_stride = d->table_stride;
  p.num_requests = d->num_requests;
  p.num_tokens = (int32_t)d->num_tokens;
  p.num_q_heads = d->num_q_heads;
  p.max_pages = d->max_pages;
  p.num_pages = d->kv.num_pages;
  p.page_tokens = d->kv.page_tokens;
  p.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if ((1 << s) == d->kv.page_tokens) p.page_shift = s;
  const int64_t cap = (int64_t)d->max_pages * d->kv.page_tokens;
  p.capacity = (int32_t)(cap < qsa::kMaxKeys ? cap : qsa::kMaxKeys);
  p.group = d->num_q_heads / d->kv.num_kv_heads;
  p.num_selected = d->num_selected;
  p.ratio = d->ratio;
  p.local_tokens = d->local_tokens;
  p.window = window;
  p.sinks = sinks < p.capacity ? sinks : p.capacity;
  p.scale_log2 = d->scale * 1.4426950408889634f;
  if (form == QSA_ATTN_TILE) {
    const char* msg = nullptr;
    e = qsa::launch_attn_tile(p, *d, (uint8_t*)workspace, (cudaStream_t)stream, &msg);
    if (msg) return set_error(QSA_ERR_UNSUPPORTED, "%s", msg);
    return launched(e, "attention (tile) launch");
  }
  return launched(qsa::launch_attn_gather(p, *d, (uint8_t*)workspace, (cudaStream_t)stream), "attention launch");
}

}  // namespace

extern "C" {

qsa_status qsa_build_page_maps(const qsa_page_maps_desc* d, const int32_t* context_lens, const int32_t* new_lens,
                               const int32_t* free_pages, int32_t* block_table, int32_t* query_start,
                               int32_t* seq_lens, int64_t* slots, int32_t* positions, int32_t* token_request,
                               int32_t* visible_cols, int64_t* column_slots, int32_t* pages_used, void* stream) {
  if (!d) return bad("desc is NULL");
  if (d->num_requests < 0) return bad("num_requests < 0");
  if (d->num_requests > qsa::kMaxMapRequests)
    return set_error(QSA_ERR_UNSUPPORTED, "num_requests > %d", qsa::kMaxMapRequests);
  if (d->page_tokens < 1) return bad("page_tokens < 1");
  if (d->max_pages < 1) return bad("max_pages < 1");
  if ((int64_t)d->max_pages * d->page_tokens > 0x7FFFFFFFLL) return bad("max_pages * page_tokens exceeds 2^31 - 1");
  if (d->ratio < 1 || d->page_tokens % d->ratio != 0) return bad("ratio must be at least 1 and divide page_tokens");
  if (d->partial_cols != 0 && d->partial_cols != 1) return bad("partial_cols must be 0 or 1");
  if (d->reserved != 0) return bad("reserved must be 0");
  if (d->table_stride < d->max_pages) return bad("table_stride < max_pages");
  if (d->num_free < 0) return bad("num_free < 0");
  if (d->max_tokens < 0 || d->max_tokens > 0x7FFFFFFFLL) return bad("max_tokens out of range");
  if (!query_start || (d->num_requests > 0 && (!context_lens || !new_lens || !block_table || !seq_lens)) ||
      (d->num_free > 0 && !free_pages) || (d->max_tokens > 0 && !slots))
    return bad("a required pointer is NULL");
  if (!aligned(context_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) || !aligned(block_table, 4) ||
      !aligned(query_start, 4) || !aligned(seq_lens, 4) || !aligned(positions, 4) || !aligned(token_request, 4) ||
      !aligned(visible_cols, 4) || !aligned(pages_used, 4))
    return bad("an int32 pointer is not 4-byte aligned");
  if (!aligned(slots, 8) || !aligned(column_slots, 8)) return bad("an int64 pointer is not 8-byte aligned");
  qsa::PageMapsParams p;
  p.context_lens = context_lens;
  p.new_lens = new_lens;
  p.free_pages = free_pages;
  p.block_table = block_table;
  p.query_start = query_start;
  p.seq_lens = seq_lens;
  p.slots = slots;
  p.positions = positions;
  p.token_request = token_request;
  p.visible_cols = visible_cols;
  p.column_slots = column_slots;
  p.pages_used = pages_used;
  p.table_stride = d->table_stride;
  p.num_free = d->num_free;
  p.max_tokens = d->max_tokens;
  p.num_requests = d->num_requests;
  p.page_tokens = d->page_tokens;
  p.max_pages = d->max_pages;
  p.ratio = d->ratio;
  p.partial_cols = d->partial_cols;
  return launched(qsa::launch_page_maps(p, (cudaStream_t)stream), "page maps launch");
}

qsa_status qsa_store_paged_kv(const qsa_kv_desc* d, const void* k, int64_t k_row_stride, int64_t k_row_head_stride,
                              const void* v, int64_t v_row_stride, int64_t v_row_head_stride, const int64_t* slots,
                              int64_t num_tokens, void* k_cache, void* v_cache, void* stream) {
  if (!d) return bad("desc is NULL");
  qsa_status st = validate_kv(*d);
  if (st != QSA_OK) return st;
  if (num_tokens < 0 || num_tokens > 0x7FFFFFFFLL) return bad("num_tokens out of range");
  const int64_t per_tok = (int64_t)d->num_kv_heads * (d->head_dim / 8);
  if (per_tok > (1 << 24) || num_tokens * per_tok > (1LL << 40)) return bad("too many elements for one call");
  if (!stride_ok(k_row_stride) || !stride_ok(k_row_head_stride) || !stride_ok(v_row_stride) ||
      !stride_ok(v_row_head_stride))
    return bad("row strides must be positive multiples of 16 bytes");
  if (num_tokens == 0) return QSA_OK;
  if (!k || !v || !slots || !k_cache || !v_cache) return bad("a required pointer is NULL");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return bad("k, v and the caches must be 16-byte aligned");
  if (!aligned(slots, 8)) return bad("slots is not 8-byte aligned");
  qsa::StoreKvParams p;
  p.k = (const uint8_t*)k;
  p.v = (const uint8_t*)v;
  p.slots = slots;
  p.k_cache = (uint8_t*)k_cache;
  p.v_cache = (uint8_t*)v_cache;
  p.k_row_stride = k_row_stride;
  p.k_row_head_stride = k_row_head_stride;
  p.v_row_stride = v_row_stride;
  p.v_row_head_stride = v_row_head_stride;
  p.k_page_stride = d->k_page_stride;
  p.k_token_stride = d->k_token_stride;
  p.k_head_stride = d->k_head_stride;
  p.v_page_stride = d->v_page_stride;
  p.v_token_stride = d->v_token_stride;
  p.v_head_stride = d->v_head_stride;
  p.num_tokens = num_tokens;
  p.num_slots = (int64_t)d->num_pages * d->page_tokens;
  p.page_tokens = d->page_tokens;
  p.num_kv_heads = d->num_kv_heads;
  p.head_chunks = d->head_dim / 8;
  return launched(qsa::launch_store_kv(p, (cudaStream_t)stream), "key/value store launch");
}

qsa_status qsa_store_index_keys(const qsa_index_cache_desc* d, const void* keys, int64_t row_stride,
                                const int64_t* slots, int64_t num_tokens, void* kv_cache, float* scales,
                                void* stream) {
  if (!d) return bad("desc is NULL");
  if (d->kv_dtype != QSA_KV_BF16 && d->kv_dtype != QSA_KV_FP8_E4M3)
    return set_error(QSA_ERR_INVALID_ARG, "unknown kv_dtype %d", d->kv_dtype);
  const bool fp8 = d->kv_dtype == QSA_KV_FP8_E4M3;
  if (d->num_pages < 1) return bad("num_pages < 1");
  if (d->page_cols < 1) return bad("page_cols < 1");
  if (d->head_dim != 128) return set_error(QSA_ERR_UNSUPPORTED, "head_dim must be 128 (got %d)", d->head_dim);
  if (d->key_page_stride < (int64_t)d->page_cols * 128 * (fp8 ? 1 : 2) || d->key_page_stride % (fp8 ? 4 : 16) != 0)
    return bad("key_page_stride must cover a page's keys and be a multiple of 16 (fp8: of 4) bytes");
  if (fp8 && (d->scale_page_stride < 4LL * d->page_cols || d->scale_page_stride % 4 != 0))
    return bad("scale_page_stride must be a multiple of 4 and >= 4 * page_cols");
  if (!stride_ok(row_stride)) return bad("row_stride must be a positive multiple of 16 bytes");
  if (num_tokens < 0 || num_tokens > 0x7FFFFFFFLL) return bad("num_tokens out of range");
  if (fp8 && !scales && num_tokens > 0) return bad("fp8 keys need a scales pointer");
  if (!fp8 && scales) return bad("bf16 keys take no scales (mixed operand types)");
  if (num_tokens == 0) return QSA_OK;
  if (!keys || !slots || !kv_cache) return bad("a required pointer is NULL");
  if (!aligned(keys, 16) || !aligned(slots, 8) || !aligned(kv_cache, fp8 ? 4 : 16) || !aligned(scales, 4))
    return bad("misaligned pointer (keys 16 bytes, slots 8, bf16 cache 16, fp8 cache and scales 4)");
  qsa::StoreIndexParams p;
  p.keys = (const uint8_t*)keys;
  p.slots = slots;
  p.cache = (uint8_t*)kv_cache;
  p.scales = (uint8_t*)scales;
  p.row_stride = row_stride;
  p.key_page_stride = d->key_page_stride;
  p.scale_page_stride = d->scale_page_stride;
  p.num_tokens = num_tokens;
  p.num_slots = (int64_t)d->num_pages * d->page_cols;
  p.page_cols = d->page_cols;
  p.fp8 = fp8 ? 1 : 0;
  p.wide = aligned(kv_cache, 8) && d->key_page_stride % 8 == 0 ? 1 : 0;
  return launched(qsa::launch_store_index(p, (cudaStream_t)stream), "index key store launch");
}

qsa_status qsa_plan_attention(const qsa_attn_desc* d, int32_t* form) {
  if (!form) return bad("form is NULL");
  return plan_form(d, form);
}

qsa_status qsa_paged_attention_workspace(const qsa_attn_desc* d, size_t* bytes) {
  if (!bytes) return bad("bytes is NULL");
  int32_t form = 0;
  qsa_status st = plan_form(d, &form);
  if (st != QSA_OK) return st;
  *bytes = form == QSA_ATTN_TILE ? qsa::attn_tile_workspace(d->kv.head_dim)
                                 : qsa::attn_gather_workspace(d->kv.head_dim);
  return QSA_OK;
}

qsa_status qsa_paged_attention(const qsa_attn_desc* d, const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_table, const int32_t* query_start, const int32_t* seq_lens,
                               const int32_t* selected, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return attention(d, 0, 0, q, k_cache, v_cache, block_table, query_start, seq_lens, selected, out, lse, workspace,
                   workspace_bytes, stream);
}

qsa_status qsa_paged_attention_window(const qsa_attn_desc* d, int32_t window, int32_t sink_tokens, const void* q,
                                      const void* k_cache, const void* v_cache, const int32_t* block_table,
                                      const int32_t* query_start, const int32_t* seq_lens, void* out, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!d) return bad("desc is NULL");
  if (window < 1) return bad("window < 1");
  if (sink_tokens < 0) return bad("sink_tokens < 0");
  if (d->num_selected != 0 || d->local_tokens != 0) return bad("a window takes no selected columns (num_selected and local_tokens 0)");
  return attention(d, window, sink_tokens, q, k_cache, v_cache, block_table, query_start, seq_lens, nullptr, out, lse,
                   workspace, workspace_bytes, stream);
}

}  // extern "C"
