// qsa_store_paged_kv and qsa_store_index_keys: rows into the slots of a paged
// cache.  Both move each byte once and are bound by HBM for prefill chunks and
// by launch latency for decode rows.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"
#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace {

// 16 bytes past L1.  Not through the read-only path: a launch may begin while
// the kernel that writes the rows still runs.
__device__ __forceinline__ uint4 ld_rows_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// ---- keys and values --------------------------------------------------------
// A row of a token is num_kv_heads * head_dim / 8 chunks of 16 bytes, for the
// key and for the value.  The chunks of all tokens are numbered through, and a
// thread moves kU of them, kNT apart (neighbouring threads move neighbouring
// chunks), with all its loads in flight before its first store.
constexpr int kNT = 256;
constexpr int kU = 2;  // (four: 19.8 us for 16 K tokens of 8 heads x 128, two: 17.3)

__global__ void __launch_bounds__(kNT) store_kv_kernel(const StoreKvParams p) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const uint32_t per_tok = (uint32_t)(p.num_kv_heads * p.head_chunks);
  const int64_t base = (int64_t)blockIdx.x * (kNT * kU) + threadIdx.x;
  const int64_t total = p.num_tokens * per_tok;
  uint4 kv[kU], vv[kU];
  int64_t slot[kU];
  uint32_t head[kU], chunk[kU];
  // the block's first chunk by a 64-bit division, the rest from 32-bit offsets
  const int64_t tok0 = (int64_t)blockIdx.x * (kNT * kU) / per_tok;
  const uint32_t off0 = (uint32_t)((int64_t)blockIdx.x * (kNT * kU) - tok0 * per_tok);
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    slot[u] = -1;
    if (base + u * kNT >= total) continue;
    const uint32_t o = off0 + threadIdx.x + u * kNT;
    const uint32_t dt = o / per_tok, c = o - dt * per_tok;
    const int64_t t = tok0 + dt;
    head[u] = c / (uint32_t)p.head_chunks;
    chunk[u] = c - head[u] * (uint32_t)p.head_chunks;
    const int64_t s = p.slots[t];
    if (s < 0 || s >= p.num_slots) continue;
    slot[u] = s;
    kv[u] = ld_rows_v4(p.k + t * p.k_row_stride + head[u] * p.k_row_head_stride + chunk[u] * 16);
    vv[u] = ld_rows_v4(p.v + t * p.v_row_stride + head[u] * p.v_row_head_stride + chunk[u] * 16);
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    if (slot[u] < 0) continue;
    const int64_t pg = slot[u] / p.page_tokens, j = slot[u] - pg * p.page_tokens;
    *reinterpret_cast<uint4*>(p.k_cache + pg * p.k_page_stride + j * p.k_token_stride + head[u] * p.k_head_stride +
                              chunk[u] * 16) = kv[u];
    *reinterpret_cast<uint4*>(p.v_cache + pg * p.v_page_stride + j * p.v_token_stride + head[u] * p.v_head_stride +
                              chunk[u] * 16) = vv[u];
  }
}

// ---- index keys -------------------------------------------------------------
// 16 lanes a key, 8 elements each.  fp8: the largest magnitude over the lanes
// by shuffles, one fp32 division for the scale, and the codes of the quotients.
// A code is the definition's, e4m3(fp32(x / scale)), bit for bit, almost always
// without the division: t = x * (1 / scale) is within 3 * 2^-24 of the quotient
// (two roundings and its own), so where t (1 - 2^-20) and t (1 + 2^-20) round to
// one code, so does the quotient between them.  Where they do not (about one
// element in 2^16), and for scales whose reciprocal is not ordinary, the eight
// divisions are made.  (Divisions throughout: 11.2 us for 64 K rows, a quarter of
// them live; so: 6.7 us.)
constexpr int kIdxNT = 256;
constexpr float kBelow = 1.0f - 0x1p-20f, kAbove = 1.0f + 0x1p-20f;

// Two e4m3 codes, nearest with ties to even, beyond +-448 the largest.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__global__ void __launch_bounds__(kIdxNT) store_index_kernel(const StoreIndexParams p) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int64_t t = ((int64_t)blockIdx.x * kIdxNT + threadIdx.x) >> 4;
  const int l = (int)threadIdx.x & 15;
  const int64_t s = t < p.num_tokens ? p.slots[t] : -1;
  const bool live = s >= 0 && s < p.num_slots;
  if (__ballot_sync(0xffffffffu, live) == 0) return;
  uint4 w = make_uint4(0, 0, 0, 0);
  if (live) w = ld_rows_v4(p.keys + t * p.row_stride + l * 16);
  const int64_t pg = live ? s / p.page_cols : 0, j = live ? s - pg * p.page_cols : 0;
  if (!p.fp8) {
    if (live) *reinterpret_cast<uint4*>(p.cache + pg * p.key_page_stride + j * 256 + l * 16) = w;
    return;
  }
  float x[8] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y),
                bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = __fdiv_rn(amax, 448.0f);
  const float d = scale > 0.0f ? scale : 1.0f;
  uint32_t c[2] = {0, 0}, hi[2] = {0, 0};
  const float rd = __frcp_rn(d);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = make_float2(x[2 * i] * rd, x[2 * i + 1] * rd);
    c[i >> 1] |= e4m3x2(t.x * kBelow, t.y * kBelow) << (16 * (i & 1));
    hi[i >> 1] |= e4m3x2(t.x * kAbove, t.y * kAbove) << (16 * (i & 1));
  }
  if (c[0] != hi[0] || c[1] != hi[1] || !(d >= 1e-30f)) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      c[h] = e4m3x2(__fdiv_rn(x[4 * h], d), __fdiv_rn(x[4 * h + 1], d)) |
             e4m3x2(__fdiv_rn(x[4 * h + 2], d), __fdiv_rn(x[4 * h + 3], d)) << 16;
  }
  if (!(scale > 0.0f)) c[0] = c[1] = 0;
  if (!live) return;
  uint8_t* dst = p.cache + pg * p.key_page_stride + j * 128 + l * 8;
  if (p.wide) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
  } else {
    reinterpret_cast<uint32_t*>(dst)[0] = c[0];
    reinterpret_cast<uint32_t*>(dst)[1] = c[1];
  }
  if (l == 0) *reinterpret_cast<float*>(p.scales + pg * p.scale_page_stride + 4 * j) = scale;
}

template <typename P>
cudaError_t launch(void (*kern)(const P), const P& p, int64_t blocks, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_store_kv(const StoreKvParams& p, cudaStream_t stream) {
  const int64_t chunks = p.num_tokens * (int64_t)p.num_kv_heads * p.head_chunks;
  return launch(store_kv_kernel, p, (chunks + kNT * kU - 1) / (kNT * kU), kNT, stream);
}

cudaError_t launch_store_index(const StoreIndexParams& p, cudaStream_t stream) {
  return launch(store_index_kernel, p, (p.num_tokens * 16 + kIdxNT - 1) / kIdxNT, kIdxNT, stream);
}

}  // namespace qsa
