// Internal declarations shared by the library's translation units (host side).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/qsa.h"

namespace qsa {

// Parameters of one scoring launch, resolved on the host from qsa_paged_desc.
struct ScoreParams {
  const uint16_t* q;        // bf16 bits [R][H][128], or e4m3 codes when q8
  const float* weights;     // [R][H]
  const uint8_t* kv;        // paged keys
  const uint8_t* scales;    // fp8 scales base (NULL for bf16)
  const int32_t* block_table;
  const int32_t* visible;
  const int32_t* next_n_lens;  // [num_requests] live rows of each request, or null (all live)
  float* out;
  int64_t out_cols;
  int64_t key_page_stride;
  int64_t scale_page_stride;
  int64_t capacity;         // min(out_cols, max_pages * page_cols): largest legal visible count
  int32_t num_requests, rows_per_req, num_rows, num_heads, page_cols, max_pages, num_pages;
  int32_t fp8;
  int32_t q8;               // q as e4m3 codes [R][H][128] (fp8 keys only)
};

// Selection fused into a tcgen05 scoring launch (qsa_paged_mqa_topk).
constexpr int kFuseMaxGroups = 256;  // row groups a fused launch takes at most
struct FuseArgs {
  int32_t* topk_out;  // [num_rows][k]
  uint32_t* sync;     // 2 * groups + 1 words, zero (and zero again once the launch completes)
  int32_t k;
};

// Each launcher returns cudaSuccess or the launch error; `msg` gets a reason
// when a shape is rejected (then the return is cudaErrorInvalidValue).
cudaError_t launch_rowcore(const ScoreParams& p, cudaStream_t stream, const char** msg);
bool umma_supports(const qsa_paged_desc& d, const char** why);
// The lean form of the tcgen05 scorer serves `d` (with fp8 q when q8).
bool umma_lean_supports(const qsa_paged_desc& d, bool q8, const char** why);
// Row groups the tcgen05 scorer splits `d` into (rows x heads of a group <= 256).
int64_t umma_num_groups(const qsa_paged_desc& d);
cudaError_t launch_umma(const ScoreParams& p, cudaStream_t stream, const char** msg,
                        const FuseArgs* fuse = nullptr, bool lean = false);
// Device address of the fault word on the current device (bit 0: a scoring
// kernel's bounded wait gave up; bit 1: a top-k kernel's).
cudaError_t fault_word_address(unsigned int** out);
// Reads (and optionally clears) the device fault word the kernels set when a
// bounded wait gives up.  Synchronises the device.
cudaError_t read_fault_word(uint32_t* flags, bool clear);
// Top-k of every row over [0, n_r): n_r = visible[r] clamped to [0, min(capacity,
// row_stride)], and 0 for a dead row (next_n_lens non-null: row r is dead when
// r % rows_per_req >= next_n_lens[r / rows_per_req]).  max_visible > 0 is the
// caller's bound on the n_r, a dispatch hint only: a row above it is still
// selected exactly, more slowly.
cudaError_t launch_topk(const float* logits, int64_t num_rows, int64_t row_stride, const int32_t* visible,
                        const int32_t* next_n_lens, int32_t rows_per_req, int64_t capacity, int64_t max_visible,
                        int32_t k, int32_t* out, cudaStream_t stream);

// Cached per-device properties (queried once per device).
struct DeviceInfo {
  int device;
  int num_sms;
  int max_smem_optin;
};
cudaError_t device_info(DeviceInfo* info);

// Raises a kernel's dynamic shared memory limit to `bytes`, on the first call
// for a device (`done`: one bit a device, one word a kernel).  A call every
// launch costs about a microsecond of host time.
template <typename K>
cudaError_t allow_smem(K kern, int bytes, int device, std::atomic<uint64_t>& done) {
  const bool known = device >= 0 && device < 64;
  if (known && (done.load(std::memory_order_acquire) >> device & 1)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && known) done.fetch_or(1ull << device, std::memory_order_release);
  return e;
}

// Records this thread's last error and returns `st` (qsa_abi.cu).
qsa_status set_error(qsa_status st, const char* fmt, ...);

// page_maps.cu
constexpr int kMaxMapRequests = 16384;  // their two sums fit a CTA's shared memory
struct PageMapsParams {
  const int32_t *context_lens, *new_lens, *free_pages;
  int32_t *block_table, *query_start, *seq_lens;
  int64_t* slots;
  int32_t *positions, *token_request, *visible_cols;  // may be null
  int64_t* column_slots;                              // may be null
  int32_t* pages_used;                                // may be null
  int64_t table_stride, num_free, max_tokens;
  int32_t num_requests, page_tokens, max_pages, ratio, partial_cols;
};
cudaError_t launch_page_maps(const PageMapsParams& p, cudaStream_t stream);

// kv_store.cu
struct StoreKvParams {
  const uint8_t *k, *v;
  const int64_t* slots;
  uint8_t *k_cache, *v_cache;
  int64_t k_row_stride, k_row_head_stride, v_row_stride, v_row_head_stride;
  int64_t k_page_stride, k_token_stride, k_head_stride, v_page_stride, v_token_stride, v_head_stride;
  int64_t num_tokens, num_slots;
  int32_t page_tokens, num_kv_heads, head_chunks;  // head_chunks: 16-byte chunks of a head's row
};
cudaError_t launch_store_kv(const StoreKvParams& p, cudaStream_t stream);
struct StoreIndexParams {
  const uint8_t* keys;
  const int64_t* slots;
  uint8_t *cache, *scales;
  int64_t row_stride, key_page_stride, scale_page_stride, num_tokens, num_slots;
  int32_t page_cols, fp8, wide;  // wide: every key of the cache is 8-byte aligned
};
cudaError_t launch_store_index(const StoreIndexParams& p, cudaStream_t stream);

// attn_gather.cu, attn_tile.cu: qsa_paged_attention.
struct AttnParams {
  const uint8_t *q, *k, *v;
  uint8_t* out;
  float* lse;                 // may be null
  const int32_t *block_table, *query_start, *seq_lens, *selected;
  float* parts;               // unfinished parts of split items
  uint32_t* counters;         // arrivals at split items (zero between calls)
  int32_t* meta;              // tile form: the split items, for the joining launch
  unsigned int* fault;
  int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride;
  int64_t k_page_stride, k_token_stride, k_head_stride, v_page_stride, v_token_stride, v_head_stride;
  int64_t table_stride;
  int32_t num_requests, num_tokens, num_q_heads, max_pages, num_pages, page_tokens, page_shift;
  int32_t capacity;           // max_pages * page_tokens, at most kMaxKeys
  int32_t group;              // query heads of a key/value head
  int32_t hv, splits, sub;    // virtual heads = kv heads * splits, of `sub` query heads each
  int32_t tpi;                // tokens an item
  int32_t item_cost;          // units an item costs behind those of its keys
  int32_t out32;              // tile form: rows of out are 32-byte aligned
  int32_t min_shift;          // a CTA takes at least 2^min_shift units (fewer CTAs take part then)
  int32_t num_selected, ratio, ratio_shift, local_tokens;  // ratio_shift: log2, or -1
  int32_t near_rows;          // keys and values: equal strides, offsets below 2^36 bytes
  float scale_log2;           // scale * log2(e)
};
constexpr int64_t kMaxKeys = 0x7FFFFC00;  // keys of a request (room for rounding up in 32 bits)
constexpr int kGatherRows = 32;  // rows of the gathered form's largest tile
// Query rows of a key/value head above which a call takes tiles.  At 16 rows
// the gathered form wins (us, gathered / tiles: 16 requests of 8000 keys 85 /
// 92, 64 of 1000 51 / 59, one of 1000 9.9 / 11.8, one of 30000 with two heads
// 21.8 / 25.7), at 20, where it needs a second row tile, it does not (90 / 92,
// 60 / 59, 13.2 / 12.0; 32 rows: 91 / 93, 63 / 60, 14.2 / 12.4, 35.0 / 29.0).
constexpr int kTileAbove = 16;
size_t attn_gather_workspace(int head_dim);
size_t attn_tile_workspace(int head_dim);
bool attn_tile_supports(const qsa_attn_desc& d, const char** why);
cudaError_t launch_attn_gather(AttnParams p, const qsa_attn_desc& d, uint8_t* workspace, cudaStream_t stream);
cudaError_t launch_attn_tile(AttnParams p, const qsa_attn_desc& d, uint8_t* workspace, cudaStream_t stream,
                             const char** msg);

// page_stream.cu: qsa_page_stream's launch (arguments already validated).
cudaError_t launch_page_stream(const uint8_t* base, int64_t page_stride, int32_t page_bytes, const int32_t* pages,
                               int64_t num_listed, int64_t pool_pages, uint32_t* checksum, cudaStream_t stream);

}  // namespace qsa
