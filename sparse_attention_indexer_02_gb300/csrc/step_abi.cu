// C ABI of the head rotation and of draft verification: host-side validation
// and launches.  Declarations, argument meaning and error behaviour are in
// include/qsa.h.
#include <math.h>

#include "abi_checks.h"
#include "qsa_internal.h"

namespace {

using namespace qsa::abi;
using qsa::set_error;

qsa_status validate_rotary(const qsa_rotary_desc* d) {
  if (!d) return bad("desc is NULL");
  if (d->dtype != QSA_HALF_BF16 && d->dtype != QSA_HALF_F16)
    return set_error(QSA_ERR_INVALID_ARG, "unknown row dtype %d", d->dtype);
  if (d->head_dim < 8 || d->head_dim % 8 != 0)
    return set_error(QSA_ERR_INVALID_ARG, "head_dim must be a positive multiple of 8 (got %d)", d->head_dim);
  if (d->head_dim > 256) return set_error(QSA_ERR_UNSUPPORTED, "head_dim above 256 (got %d)", d->head_dim);
  if (d->rot_dim < 2 || d->rot_dim % 2 != 0 || d->rot_dim > d->head_dim)
    return bad("rot_dim must be even, at least 2 and at most head_dim");
  if (d->rot_offset < 0 || d->rot_offset > d->head_dim - d->rot_dim)
    return bad("rot_offset + rot_dim must lie within the head");
  if (d->layout != QSA_ROTARY_HALF && d->layout != QSA_ROTARY_PAIRS)
    return set_error(QSA_ERR_INVALID_ARG, "unknown rotary layout %d", d->layout);
  if (d->layout == QSA_ROTARY_PAIRS && d->rot_offset % 2 != 0) return bad("pairs begin at an even rot_offset");
  if (d->norm != QSA_NORM_NONE && d->norm != QSA_NORM_RMS && d->norm != QSA_NORM_LAYER)
    return set_error(QSA_ERR_INVALID_ARG, "unknown norm %d", d->norm);
  if (d->weight_f32 != 0 && d->weight_f32 != 1) return bad("weight_f32 must be 0 or 1");
  if (d->reserved != 0) return bad("reserved must be 0");
  if (d->norm != QSA_NORM_NONE && !(d->eps >= 0.0f && !isinf(d->eps))) return bad("eps must be finite and >= 0");
  if (isnan(d->magnitude) || isinf(d->magnitude)) return bad("magnitude must be finite");
  if (d->num_tokens < 0 || d->num_tokens > 0x7FFFFFFFLL) return bad("num_tokens out of range");
  return QSA_OK;
}

// `stored`: the output is the cache.
qsa_status validate_rows(const qsa_rotary_desc& d, const qsa_head_rows& h, bool stored) {
  if (h.num_heads < 1 || h.num_heads > 65536) return bad("num_heads must be 1..65536");
  if (h.reserved != 0) return bad("rows.reserved must be 0");
  if (!stride_ok(h.x_row_stride) || !stride_ok(h.x_head_stride) ||
      (!stored && (!stride_ok(h.out_row_stride) || !stride_ok(h.out_head_stride))))
    return bad("row and head strides must be positive multiples of 16 bytes");
  if (d.norm == QSA_NORM_NONE && h.weight) return bad("a weight needs a norm");
  if (d.norm != QSA_NORM_LAYER && h.bias) return bad("a bias needs the layer norm");
  const uintptr_t a = d.weight_f32 ? 4 : 2;
  if (!aligned(h.weight, a) || !aligned(h.bias, a)) return bad("weight or bias is misaligned");
  if (stored && h.out) return bad("k goes to the cache: its out must be NULL");
  if (d.num_tokens == 0) return QSA_OK;
  if (!h.x || (!stored && !h.out)) return bad("a required pointer is NULL");
  if (!aligned(h.x, 16) || !aligned(h.out, 16)) return bad("rows must be 16-byte aligned");
  return QSA_OK;
}

void fill(qsa::HeadRows& o, const qsa_head_rows& h) {
  o.x = (const uint8_t*)h.x;
  o.out = (uint8_t*)h.out;
  o.weight = h.weight;
  o.bias = h.bias;
  o.x_row = h.x_row_stride;
  o.x_head = h.x_head_stride;
  o.out_row = h.out_row_stride;
  o.out_head = h.out_head_stride;
  o.heads = h.num_heads;
}

qsa::RotateParams rotate_params(const qsa_rotary_desc& d, const qsa_head_rows& q, const qsa_head_rows* k,
                                const int32_t* positions, const uint64_t* freqs) {
  qsa::RotateParams p = {};
  fill(p.rows[0], q);
  if (k) fill(p.rows[1], *k);
  p.positions = positions;
  p.freqs = freqs;
  p.num_tokens = d.num_tokens;
  p.head_dim = d.head_dim;
  p.rot_dim = d.rot_dim;
  p.rot_offset = d.rot_offset;
  p.layout = d.layout;
  p.norm = d.norm;
  p.weight32 = d.weight_f32;
  p.eps = d.eps;
  p.inv_dim = 1.0f / (float)d.head_dim;
  p.magnitude = d.magnitude;
  p.page_tokens = 1;
  return p;
}

qsa_status rotate(const qsa::RotateParams& p, int32_t dtype, void* stream) {
  return launched(dtype == QSA_HALF_F16 ? qsa::launch_rotate_fp16(p, (cudaStream_t)stream)
                                        : qsa::launch_rotate_bf16(p, (cudaStream_t)stream),
                  "head rotation launch");
}

}  // namespace

extern "C" {

qsa_status qsa_rotate_heads(const qsa_rotary_desc* d, const qsa_head_rows* q, const qsa_head_rows* k,
                            const int32_t* positions, const uint64_t* freqs, void* stream) {
  qsa_status st = validate_rotary(d);
  if (st != QSA_OK) return st;
  if (!q) return bad("q is NULL");
  st = validate_rows(*d, *q, false);
  if (st == QSA_OK && k) st = validate_rows(*d, *k, false);
  if (st != QSA_OK) return st;
  if (d->num_tokens == 0) return QSA_OK;
  if (!positions || !freqs) return bad("a required pointer is NULL");
  if (!aligned(positions, 4) || !aligned(freqs, 8)) return bad("positions (4 bytes) or freqs (8 bytes) is misaligned");
  return rotate(rotate_params(*d, *q, k, positions, freqs), d->dtype, stream);
}

qsa_status qsa_rotate_store_kv(const qsa_rotary_desc* d, const qsa_head_rows* q, const qsa_head_rows* k,
                               const int32_t* positions, const uint64_t* freqs, const qsa_kv_desc* kv, const void* v,
                               int64_t v_row_stride, int64_t v_head_stride, const int64_t* slots, void* k_cache,
                               void* v_cache, void* stream) {
  qsa_status st = validate_rotary(d);
  if (st != QSA_OK) return st;
  if (!q || !k || !kv) return bad("q, k or kv is NULL");
  st = validate_rows(*d, *q, false);
  if (st == QSA_OK) st = validate_rows(*d, *k, true);
  if (st == QSA_OK) st = validate_kv(*kv);
  if (st != QSA_OK) return st;
  if (kv->dtype != d->dtype || kv->head_dim != d->head_dim || kv->num_kv_heads != k->num_heads)
    return bad("the caches' dtype, head_dim and heads must be the rows'");
  if (!stride_ok(v_row_stride) || !stride_ok(v_head_stride)) return bad("v strides must be positive multiples of 16 bytes");
  if (d->num_tokens == 0) return QSA_OK;
  if (!positions || !freqs || !v || !slots || !k_cache || !v_cache) return bad("a required pointer is NULL");
  if (!aligned(positions, 4) || !aligned(freqs, 8) || !aligned(slots, 8))
    return bad("positions (4 bytes), freqs or slots (8 bytes) is misaligned");
  if (!aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return bad("v and the caches must be 16-byte aligned");
  qsa::RotateParams p = rotate_params(*d, *q, k, positions, freqs);
  qsa::HeadRows& r = p.rows[2];
  r.x = (const uint8_t*)v;
  r.x_row = v_row_stride;
  r.x_head = v_head_stride;
  r.heads = k->num_heads;
  p.slots = slots;
  p.k_cache = (uint8_t*)k_cache;
  p.v_cache = (uint8_t*)v_cache;
  p.k_page_stride = kv->k_page_stride;
  p.k_token_stride = kv->k_token_stride;
  p.k_head_stride = kv->k_head_stride;
  p.v_page_stride = kv->v_page_stride;
  p.v_token_stride = kv->v_token_stride;
  p.v_head_stride = kv->v_head_stride;
  p.num_slots = (int64_t)kv->num_pages * kv->page_tokens;
  p.page_tokens = kv->page_tokens;
  return rotate(p, d->dtype, stream);
}

qsa_status qsa_verify_drafts(const qsa_verify_desc* d, const int32_t* draft_tokens, const int32_t* num_drafts,
                             const void* target_probs, const void* draft_probs, const float* uniforms,
                             const int32_t* context_lens, int32_t* out_tokens, int32_t* num_accepted,
                             int32_t* next_lens, void* stream) {
  if (!d) return bad("desc is NULL");
  if (d->num_requests < 0 || d->num_requests > 65536) return bad("num_requests must be 0..65536");
  if (d->max_drafts < 0 || d->max_drafts > 1024) return bad("max_drafts must be 0..1024");
  if (d->vocab < 1 || d->vocab > (1 << 30)) return bad("vocab must be 1..2^30");
  if (d->dtype != QSA_PROBS_F32 && d->dtype != QSA_PROBS_BF16 && d->dtype != QSA_PROBS_F16)
    return set_error(QSA_ERR_INVALID_ARG, "unknown probability dtype %d", d->dtype);
  if (d->target_request_stride < 0 || d->target_row_stride < 0 || d->draft_request_stride < 0 || d->draft_row_stride < 0)
    return bad("a stride is negative");
  if (!context_lens != !next_lens) return bad("context_lens and next_lens are given together");
  if (d->num_requests == 0) return QSA_OK;
  if (!target_probs || !uniforms || !out_tokens || !num_accepted || (d->max_drafts > 0 && !draft_tokens))
    return bad("a required pointer is NULL");
  const uintptr_t size = d->dtype == QSA_PROBS_F32 ? 4 : 2;
  if (!aligned(target_probs, size) || !aligned(draft_probs, size)) return bad("probabilities are misaligned");
  if (!aligned(draft_tokens, 4) || !aligned(num_drafts, 4) || !aligned(uniforms, 4) || !aligned(context_lens, 4) ||
      !aligned(out_tokens, 4) || !aligned(num_accepted, 4) || !aligned(next_lens, 4))
    return bad("a 4-byte pointer is misaligned");
  qsa::VerifyParams p;
  p.target = target_probs;
  p.draft = d->max_drafts > 0 ? draft_probs : nullptr;
  p.tokens = draft_tokens;
  p.num_drafts = num_drafts;
  p.context_lens = context_lens;
  p.uniforms = uniforms;
  p.out_tokens = out_tokens;
  p.num_accepted = num_accepted;
  p.next_lens = next_lens;
  p.target_request = d->target_request_stride;
  p.target_row = d->target_row_stride;
  p.draft_request = d->draft_request_stride;
  p.draft_row = d->draft_row_stride;
  p.num_requests = d->num_requests;
  p.max_drafts = d->max_drafts;
  p.vocab = d->vocab;
  p.dtype = d->dtype;
  return launched(qsa::launch_verify(p, (cudaStream_t)stream), "draft verification launch");
}

}  // extern "C"
