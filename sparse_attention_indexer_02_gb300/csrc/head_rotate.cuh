// qsa_rotate_heads and qsa_rotate_store_kv: rows of heads normalised, rotated by
// their position's angles and written out, or into the slots of a paged cache.
//
// A head x of D elements becomes
//   n = x                                      (no norm)
//   n = x w / sqrt(mean(x^2) + eps)            (RMS)
//   n = (x - mean) w / sqrt(var + eps) + b     (layer)
// and the pairs (lo, hi) of its rotated part are turned by a_i = position * f_i:
//   lo' = lo cos a_i - hi sin a_i,   hi' = hi cos a_i + lo sin a_i.
// A frequency is a 64-bit fixed-point number of turns a position, so position *
// f_i modulo 2^64 is the angle modulo a turn exactly, whatever the position: the
// fp32 rounding that follows is that of an angle below half a turn.
//
// LP lanes hold a head, two chunks of 8 elements (16 bytes) each, so 32 / LP
// heads are a warp's pass.  In the half layout a lane's two chunks are partners
// (when half the rotated part is a multiple of 8; else the partners come through
// shared memory), in the pairs layout an element's partner is its neighbour, so
// a head needs no exchange but the norm's sums.  The passes of all tokens (of a
// token: q's, k's, then v's, which are copied) are numbered through; a CTA takes
// kWarps or 2 kWarps neighbouring ones, so that it reads and writes one stretch
// of memory, loads them all, and computes the cosines and sines of its tokens
// into shared memory meanwhile, each once.
// (A warp a token, a pass of it at a time, reached 4.6 of the 6.8 TB/s whatever
// the loads in flight: 73 us for 16 K tokens of 40 heads x 128, and 93 with the
// norm and the store.)
//
// What bounds it: HBM for chunks, which every byte crosses once each way, and
// for a decode step the launch and the loads (position and heads together,
// frequencies), the angles and the output one after the other.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "device_common.cuh"
#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace rot {

constexpr int kNT = 256;
constexpr int kWarps = kNT / 32;
constexpr int kU = 2;          // passes a warp takes, at most
constexpr int kTokens = kWarps * kU;  // tokens a CTA's passes can belong to

enum { kHalf = 0, kPairs = 1, kAnyHalf = 2 };

// 16 bytes past L1 (not through the read-only path: rows may be rotated in place).
__device__ __forceinline__ uint4 ld_row(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (F16) {
    float2 r;
    asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "r"(w));
    return r;
  }
  return make_float2(bf16_lo(w), bf16_hi(w));
}

// Two fp32 values in a register pair.
using f2 = uint64_t;
__device__ __forceinline__ f2 pair(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 both(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Element e of a weight or bias vector, `none` without one.
template <bool F16>
__device__ __forceinline__ float weight_at(const void* w, int32_t is32, int e, float none) {
  if (w == nullptr) return none;
  if (is32) return static_cast<const float*>(w)[e];
  return unpack2<F16>(static_cast<const uint16_t*>(w)[e]).x;
}

template <int LP>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LP / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <bool F16, int LP, int NORM, int LAYOUT>
__global__ void __launch_bounds__(kNT, 3) rotate_kernel(const RotateParams p) {
  constexpr int kHeads = 32 / LP;    // heads a pass
  constexpr int kMaxPairs = LP * 8;  // pairs of a head's rotated part, at most
  __shared__ __align__(16) float cosines[kTokens][kMaxPairs], sines[kTokens][kMaxPairs];
  __shared__ __align__(16) float stage[LAYOUT == kAnyHalf ? kWarps : 1][LAYOUT == kAnyHalf ? 32 * 16 : 1];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  // weights and biases of q and k
  __shared__ __align__(16) float weights[NORM ? 2 : 1][NORM ? LP * 16 : 1], biases[NORM == 2 ? 2 : 1][NORM == 2 ? LP * 16 : 1];
  const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
  const int32_t passes = p.part_end[2];  // of a token
  const int mine = kWarps * p.per_warp;  // passes of the CTA
  const int64_t first = (int64_t)blockIdx.x * mine;
  const int64_t tok0 = first / passes;
  const int32_t off0 = (int32_t)(first - tok0 * passes);

  // the lane's chunks: elements e[0] .. e[0] + 7 and e[1] .. e[1] + 7 of its head
  const int sub = lane / LP, i = lane % LP, half = p.rot_dim >> 1;
  int e[2];
  bool turned_lane = false;  // kHalf: both chunks are rotated
  if (LAYOUT == kHalf) {
    const int pairs = p.rot_dim >> 4, m = 2 * (i - pairs);
    turned_lane = i < pairs;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      e[c] = turned_lane ? p.rot_offset + 8 * i + c * half
                         : 8 * (m + c) + (8 * (m + c) < p.rot_offset ? 0 : p.rot_dim);
  } else {
    e[0] = 16 * i;
    e[1] = 16 * i + 8;
  }
  const bool in[2] = {e[0] < p.head_dim, e[1] < p.head_dim};

  // the warp's passes, and their loads
  int32_t dt[kU], head[kU], part[kU];
  uint32_t raw[kU][8];
  int32_t pos[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int32_t at = off0 + warp + u * kWarps;
    dt[u] = at / passes;
    const int32_t pass = at - dt[u] * passes;
    part[u] = pass < p.part_end[0] ? 0 : (pass < p.part_end[1] ? 1 : 2);
    head[u] = (pass - (part[u] == 0 ? 0 : p.part_end[part[u] - 1])) * kHeads + sub;
    const bool there = u < p.per_warp && tok0 + dt[u] < p.num_tokens;
    pos[u] = there ? p.positions[tok0 + dt[u]] : -1;
    const HeadRows& h = p.rows[part[u]];
    if (!there || head[u] >= h.heads) head[u] = -1;
    const uint8_t* row = h.x + (tok0 + dt[u]) * h.x_row + head[u] * h.x_head;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (head[u] >= 0 && in[c]) v = ld_row(row + 2 * e[c]);
      raw[u][4 * c] = v.x;
      raw[u][4 * c + 1] = v.y;
      raw[u][4 * c + 2] = v.z;
      raw[u][4 * c + 3] = v.w;
    }
  }
  if (NORM) {
    for (int k = (int)threadIdx.x; k < 2 * p.head_dim; k += kNT) {
      const int r = k < p.head_dim ? 0 : 1, el = k - r * p.head_dim;
      weights[r][el] = weight_at<F16>(p.rows[r].weight, p.weight32, el, 1.0f);
      if (NORM == 2) biases[r][el] = weight_at<F16>(p.rows[r].bias, p.weight32, el, 0.0f);
    }
  }
  // the angles of the CTA's tokens
  const int tokens = (off0 + mine - 1) / passes + 1;
  for (int k = (int)threadIdx.x; k < tokens * half; k += kNT) {
    const int d = k / half, r = k - d * half;
    if (tok0 + d >= p.num_tokens) break;
    const uint64_t turns = (uint64_t)(uint32_t)p.positions[tok0 + d] * p.freqs[r];
    float s, c;
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
    cosines[d][r] = c * p.magnitude;
    sines[d][r] = s * p.magnitude;
  }
  __syncthreads();

#pragma unroll
  for (int u = 0; u < kU; ++u) {
    if (pos[u] < 0) continue;  // no pass, or a padding row (the whole warp's)
    const HeadRows& h = p.rows[part[u]];
    uint8_t* dst;
    if (h.out == nullptr) {
      const int64_t slot = p.slots[tok0 + dt[u]];
      if (slot < 0 || slot >= p.num_slots) continue;
      const int64_t page = slot / p.page_tokens, off = slot - page * p.page_tokens;
      dst = part[u] == 1 ? p.k_cache + page * p.k_page_stride + off * p.k_token_stride + head[u] * p.k_head_stride
                         : p.v_cache + page * p.v_page_stride + off * p.v_token_stride + head[u] * p.v_head_stride;
    } else {
      dst = h.out + (tok0 + dt[u]) * h.out_row + head[u] * h.out_head;
    }
    if (part[u] < 2) {
      f2 x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // element e[j / 4] + 2 (j % 4), and the next
        const float2 v = unpack2<F16>(raw[u][j]);
        x[j] = pair(v.x, v.y);
      }
      if (NORM == 2) {
        f2 s = add2(x[0], x[1]);
#pragma unroll
        for (int j = 2; j < 8; ++j) s = add2(s, x[j]);
        const float2 b = both(s);
        const float mean = head_sum<LP>(b.x + b.y) * p.inv_dim;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float m = in[j >> 2] ? -mean : 0.0f;
          x[j] = add2(x[j], pair(m, m));
        }
      }
      if (NORM) {
        f2 s = mul2(x[0], x[0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) s = fma2(x[j], x[j], s);
        const float2 b = both(s);
        const float f = rsqrtf(fmaf(head_sum<LP>(b.x + b.y), p.inv_dim, p.eps));
        const f2 ff = pair(f, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = mul2(x[j], ff);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int el = in[j >> 2] ? e[j >> 2] + 2 * (j & 3) : 0;
          x[j] = mul2(x[j], *reinterpret_cast<const f2*>(&weights[part[u]][el]));
          if (NORM == 2) x[j] = add2(x[j], *reinterpret_cast<const f2*>(&biases[part[u]][el]));
        }
      }
      // the rotation; elements beside the rotated part stay (without a norm: their bits)
      f2 y[8];
      uint32_t keep[8];  // bits of the packed pair that stay
      if (LAYOUT == kHalf) {
        const f2* c = reinterpret_cast<const f2*>(&cosines[dt[u]][turned_lane ? 8 * i : 0]);
        const f2* s = reinterpret_cast<const f2*>(&sines[dt[u]][turned_lane ? 8 * i : 0]);
        const f2 minus = pair(-1.0f, -1.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[j] = fma2(mul2(x[j + 4], minus), s[j], mul2(x[j], c[j]));
          y[j + 4] = fma2(x[j], s[j], mul2(x[j + 4], c[j]));
          keep[j] = keep[j + 4] = turned_lane ? 0u : ~0u;
        }
      } else if (LAYOUT == kPairs) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = (j < 4 ? e[0] : e[1] - 8) + 2 * j - p.rot_offset;  // of the pair's first element
          const bool turned = in[j >> 2] && r >= 0 && r < p.rot_dim;
          const float c = cosines[dt[u]][turned ? r >> 1 : 0], s = sines[dt[u]][turned ? r >> 1 : 0];
          const float2 v = both(x[j]);
          y[j] = pair(fmaf(-v.y, s, v.x * c), fmaf(v.x, s, v.y * c));
          keep[j] = turned ? 0u : ~0u;
        }
      } else {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) *reinterpret_cast<f2*>(&stage[warp][lane * 16 + 2 * j]) = x[j];
        __syncwarp();
        const float* row = &stage[warp][sub * LP * 16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 v = both(x[j]);
          float o[2] = {v.x, v.y};
          keep[j] = ~0u;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int el = 16 * i + 2 * j + k, r = el - p.rot_offset;
            if (r >= 0 && r < p.rot_dim && el < p.head_dim) {
              const int q = r < half ? r : r - half;
              const float s = sines[dt[u]][q], xp = row[r < half ? el + half : el - half];
              o[k] = fmaf(xp, r < half ? -s : s, o[k] * cosines[dt[u]][q]);
              keep[j] &= k ? 0xFFFFu : 0xFFFF0000u;
            }
          }
          y[j] = pair(o[0], o[1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 v = both(y[j]);
        uint32_t o = attn::pack2<F16>(v.x, v.y);
        if (NORM && LAYOUT != kAnyHalf) {
          const float2 n = both(x[j]);
          o = keep[j] ? attn::pack2<F16>(n.x, n.y) : o;
        } else if (!NORM) {
          o = (raw[u][j] & keep[j]) | (o & ~keep[j]);
        }
        raw[u][j] = o;
      }
    }
    if (head[u] < 0) continue;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (in[c])
        *reinterpret_cast<uint4*>(dst + 2 * e[c]) =
            make_uint4(raw[u][4 * c], raw[u][4 * c + 1], raw[u][4 * c + 2], raw[u][4 * c + 3]);
  }
}

template <bool F16, int LP, int NORM, int LAYOUT>
cudaError_t launch(const RotateParams& p, dim3 grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kNT, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotate_kernel<F16, LP, NORM, LAYOUT>, p);
}

template <bool F16, int LP, int NORM>
cudaError_t launch_layout(const RotateParams& p, dim3 grid, cudaStream_t stream) {
  if (p.layout == QSA_ROTARY_PAIRS) return launch<F16, LP, NORM, kPairs>(p, grid, stream);
  if (p.rot_dim % 16 == 0 && p.rot_offset % 8 == 0) return launch<F16, LP, NORM, kHalf>(p, grid, stream);
  return launch<F16, LP, NORM, kAnyHalf>(p, grid, stream);
}

template <bool F16, int LP>
cudaError_t launch_norm(const RotateParams& p, dim3 grid, cudaStream_t stream) {
  if (p.norm == QSA_NORM_RMS) return launch_layout<F16, LP, 1>(p, grid, stream);
  if (p.norm == QSA_NORM_LAYER) return launch_layout<F16, LP, 2>(p, grid, stream);
  return launch_layout<F16, LP, 0>(p, grid, stream);
}

// Two passes a warp when one each already fills every SM with four CTAs.
template <bool F16>
cudaError_t launch_rotate_t(RotateParams p, cudaStream_t stream) {
  DeviceInfo info;
  cudaError_t e = device_info(&info);
  if (e != cudaSuccess) return e;
  const int lp = p.head_dim <= 64 ? 4 : (p.head_dim <= 128 ? 8 : 16), heads = 32 / lp;
  int32_t end = 0;
  for (int i = 0; i < 3; ++i) p.part_end[i] = end += (p.rows[i].heads + heads - 1) / heads;
  const int64_t passes = p.num_tokens * end;
  p.per_warp = passes > (int64_t)info.num_sms * kWarps * 4 ? kU : 1;
  const int64_t blocks = (passes + kWarps * p.per_warp - 1) / (kWarps * p.per_warp);
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, 1, 1);
  if (lp == 4) return launch_norm<F16, 4>(p, grid, stream);
  if (lp == 8) return launch_norm<F16, 8>(p, grid, stream);
  return launch_norm<F16, 16>(p, grid, stream);
}

}  // namespace rot
}  // namespace qsa
