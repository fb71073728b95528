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
// A warp works on one token; LP lanes hold a head, 8 elements (16 bytes) each, so
// 32 / LP heads are a pass.  A lane has the same elements of every head: sines
// and cosines are computed once a token, and with a norm they are folded with
// the weights,
//   y_e = s (x_e A_e + x_p B_e) (+ C_e),  A_e = w_e cos, B_e = -+ w_p sin,
// s the head's factor and p the partner of e, so that a head costs two sums and
// two products an element.  In the half layout a lane's partners are the 8
// elements of one other lane (shuffles of the packed input) when half the
// rotated part is a multiple of 8, else any (through shared memory).
//
// What bounds it: HBM for chunks, which every byte crosses once each way, and
// for a decode step the launch and three loads one after the other (position,
// frequencies and heads together, output).
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
constexpr int kU = 4;  // passes whose loads are in flight together

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

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<F16>(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <bool F16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(attn::pack2<F16>(x[0], x[1]), attn::pack2<F16>(x[2], x[3]), attn::pack2<F16>(x[4], x[5]),
                    attn::pack2<F16>(x[6], x[7]));
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
__global__ void __launch_bounds__(kNT) rotate_kernel(const RotateParams p) {
  constexpr int kHeads = 32 / LP;  // heads a pass
  __shared__ float stage[LAYOUT == kAnyHalf ? kNT / 32 : 1][LAYOUT == kAnyHalf ? 32 * 8 : 1];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
  const int64_t item = (int64_t)blockIdx.x * (kNT / 32) + warp;  // (token, block of passes)
  const int64_t t = item / p.blocks;
  if (t >= p.num_tokens) return;
  const int32_t pos = p.positions[t];
  if (pos < 0) return;  // a padding row
  const int sub = lane / LP, chunk = lane % LP, e0 = chunk * 8;
  const bool in_head = e0 < p.head_dim;
  const int32_t pass0 = (int32_t)(item - t * p.blocks) * p.per_block, pass1 = pass0 + p.per_block;
  int64_t slot = -1;
  if (p.slots != nullptr) {
    slot = p.slots[t];
    if (slot >= p.num_slots) slot = -1;
  }
  const int64_t page = slot >= 0 ? slot / p.page_tokens : 0, off = slot >= 0 ? slot - page * p.page_tokens : 0;

  // angles of the lane's elements: turned[j], partner, cos and signed sin
  float cs[8], sn[8];
  uint32_t turned = 0;
  const int half = p.rot_dim >> 1;
  int partner = lane;
  bool ready = false;
  auto angles = [&]() {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = e0 + j - p.rot_offset;
      const bool in = in_head && r >= 0 && r < p.rot_dim;
      if (in) turned |= 1u << j;
      if (LAYOUT == kPairs && (j & 1)) {  // the pair's second element: the first one's angle
        cs[j] = cs[j - 1];
        sn[j] = -sn[j - 1];
        continue;
      }
      const int i = LAYOUT == kPairs ? r >> 1 : (r < half ? r : r - half);
      const uint64_t turns = in ? (uint64_t)(uint32_t)pos * p.freqs[i] : 0;
      float s, c;
      sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
      cs[j] = c * p.magnitude;
      s *= p.magnitude;
      sn[j] = LAYOUT == kPairs || r < half ? -s : s;
    }
    if (LAYOUT == kHalf && turned) partner = lane + ((e0 - p.rot_offset < half ? half : -half) >> 3);
  };

  // The q heads' passes come first, then k's, then v's, which are copied.
  int32_t first = 0;
#pragma unroll 1
  for (int part = 0; part < 3; ++part) {
    const HeadRows& h = p.rows[part];
    const int32_t n = (h.heads + kHeads - 1) / kHeads;
    const int32_t lo = max(pass0, first), hi = min(pass1, first + n);
    const int32_t base = first;
    first += n;
    if (lo >= hi) continue;
    const bool to_cache = h.out == nullptr;
    if (to_cache && slot < 0) continue;
    const uint8_t* src = h.x + t * h.x_row + e0 * 2;
    uint8_t* dst = to_cache ? (part == 1 ? p.k_cache + page * p.k_page_stride + off * p.k_token_stride
                                         : p.v_cache + page * p.v_page_stride + off * p.v_token_stride)
                            : h.out + t * h.out_row;
    dst += e0 * 2;
    const int64_t dst_head = to_cache ? (part == 1 ? p.k_head_stride : p.v_head_stride) : h.out_head;
    float A[8], B[8], C[8];
    bool folded = false;
    for (int32_t q0 = lo; q0 < hi; q0 += kU) {
      uint4 w[kU];
      bool live[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int head = (q0 + u - base) * kHeads + sub;
        live[u] = q0 + u < hi && head < h.heads && in_head;
        w[u] = make_uint4(0, 0, 0, 0);
        if (live[u]) w[u] = ld_row(src + head * h.x_head);
      }
      if (part < 2) {
        if (!ready) {
          angles();
          ready = true;
        }
        if (!folded) {
          folded = true;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            A[j] = cs[j];
            B[j] = sn[j];
            C[j] = 0.0f;
            if (NORM) {
              const bool in = (turned >> j) & 1u;
              const int e = in_head ? e0 + j : 0, r = e - p.rot_offset;
              const int pe = !in ? e : (LAYOUT == kPairs ? e ^ 1 : (r < half ? e + half : e - half));
              const float we = weight_at<F16>(h.weight, p.weight32, e, 1.0f);
              const float wp = weight_at<F16>(h.weight, p.weight32, pe, 1.0f);
              A[j] = in ? we * cs[j] : we;
              B[j] = in ? wp * sn[j] : 0.0f;
              if (NORM == 2) {
                const float be = weight_at<F16>(h.bias, p.weight32, e, 0.0f);
                const float bp = weight_at<F16>(h.bias, p.weight32, pe, 0.0f);
                C[j] = in ? fmaf(be, cs[j], bp * sn[j]) : be;
              }
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          float x[8], xp[8];
          unpack8<F16>(w[u], x);
          if (LAYOUT == kHalf) {
            const uint4 o = make_uint4(__shfl_sync(0xffffffffu, w[u].x, partner), __shfl_sync(0xffffffffu, w[u].y, partner),
                                       __shfl_sync(0xffffffffu, w[u].z, partner), __shfl_sync(0xffffffffu, w[u].w, partner));
            unpack8<F16>(o, xp);
          } else if (LAYOUT == kPairs) {
#pragma unroll
            for (int j = 0; j < 8; ++j) xp[j] = x[j ^ 1];
          } else {
            float* row = stage[warp] + sub * LP * 8;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) row[e0 + j] = x[j];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int e = e0 + j, r = e - p.rot_offset;
              xp[j] = (turned >> j) & 1u ? row[r < half ? e + half : e - half] : x[j];
            }
          }
          float y[8];
          if (NORM == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = fmaf(x[j], A[j], xp[j] * B[j]);
            uint4 o = pack8<F16>(y);
            if (LAYOUT == kHalf) {
              if (!turned) o = w[u];
            } else if (turned != 0xFFu) {  // elements beside the rotated part keep their bits
              uint32_t* ow = &o.x;
              const uint32_t* iw = &w[u].x;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (!((turned >> j) & 1u)) {
                  const uint32_t mask = 0xFFFFu << (16 * (j & 1));
                  ow[j >> 1] = (ow[j >> 1] & ~mask) | (iw[j >> 1] & mask);
                }
            }
            w[u] = o;
          } else {
            float mean = 0.0f;
            if (NORM == 2) {
              float s = 0.0f;
#pragma unroll
              for (int j = 0; j < 8; ++j) s += x[j];
              mean = head_sum<LP>(s) * p.inv_dim;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                x[j] = in_head ? x[j] - mean : 0.0f;
                xp[j] -= mean;
              }
            }
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(x[j], x[j], s);
            const float f = rsqrtf(fmaf(head_sum<LP>(s), p.inv_dim, p.eps));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float v = (turned >> j) & 1u ? fmaf(x[j], A[j], xp[j] * B[j]) : x[j] * A[j];
              y[j] = NORM == 2 ? fmaf(v, f, C[j]) : v * f;
            }
            w[u] = pack8<F16>(y);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int head = (q0 + u - base) * kHeads + sub;
        if (live[u]) *reinterpret_cast<uint4*>(dst + head * dst_head) = w[u];
      }
    }
  }
}

template <bool F16, int LP, int NORM, int LAYOUT>
cudaError_t launch(const RotateParams& p, int64_t blocks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
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
cudaError_t launch_layout(const RotateParams& p, int64_t blocks, cudaStream_t stream) {
  if (p.layout == QSA_ROTARY_PAIRS) return launch<F16, LP, NORM, kPairs>(p, blocks, stream);
  if (p.rot_dim % 16 == 0 && p.rot_offset % 8 == 0) return launch<F16, LP, NORM, kHalf>(p, blocks, stream);
  return launch<F16, LP, NORM, kAnyHalf>(p, blocks, stream);
}

template <bool F16, int LP>
cudaError_t launch_norm(const RotateParams& p, int64_t blocks, cudaStream_t stream) {
  if (p.norm == QSA_NORM_RMS) return launch_layout<F16, LP, 1>(p, blocks, stream);
  if (p.norm == QSA_NORM_LAYER) return launch_layout<F16, LP, 2>(p, blocks, stream);
  return launch_layout<F16, LP, 0>(p, blocks, stream);
}

// p.per_block and p.blocks are set here: a warp takes all passes of a token when
// the tokens alone make enough warps, else as few as spread the work over the GPU.
template <bool F16>
cudaError_t launch_rotate_t(RotateParams p, cudaStream_t stream) {
  DeviceInfo info;
  cudaError_t e = device_info(&info);
  if (e != cudaSuccess) return e;
  const int lp = p.head_dim <= 64 ? 8 : (p.head_dim <= 128 ? 16 : 32), heads = 32 / lp;
  int32_t passes = 0;
  for (const HeadRows& h : p.rows) passes += (h.heads + heads - 1) / heads;
  const int64_t warps = (int64_t)info.num_sms * 32;
  const int64_t per = (p.num_tokens * passes + warps - 1) / warps;
  p.per_block = (int32_t)(per < 1 ? 1 : (per < passes ? per : passes));
  p.blocks = (passes + p.per_block - 1) / p.per_block;
  const int64_t blocks = (p.num_tokens * p.blocks + kNT / 32 - 1) / (kNT / 32);
  if (lp == 8) return launch_norm<F16, 8>(p, blocks, stream);
  if (lp == 16) return launch_norm<F16, 16>(p, blocks, stream);
  return launch_norm<F16, 32>(p, blocks, stream);
}

}  // namespace rot
}  // namespace qsa
