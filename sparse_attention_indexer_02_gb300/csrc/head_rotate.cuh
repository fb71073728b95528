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
// (four pieces of 4 elements, two and two, when half the rotated part is a
// multiple of 4 only), in the pairs layout an element's partner is its neighbour
// (places that are no such multiples: partners through shared memory), so
// a head needs no exchange but the norm's sums.  A token's passes (q's, k's, then
// v's, which are copied) are the warps of a CTA, each with one pass of a few
// neighbouring tokens: where its heads lie and what weighs them stays the same,
// the CTA reads and writes a token's row at a time, the next one's heads on their
// way, and each token's cosines and sines are worked out once, into shared memory.
//
// What bounds it: HBM for chunks, which every byte crosses once each way (16 K
// tokens of 32 + 8 heads x 128: 53 us, 6.3 TB/s; with norm and store 64 us, 6.3), and
// for a decode step the launch and the loads (position and heads together,
// frequencies), the angles and the output one after the other (16 tokens 2.1 us).
// Instructions come next, integer ones at half the rate: 73 us (93) with a warp a
// token, 63 (81) with the passes of a few tokens numbered through, at 230 and 250
// instructions a pass, most of them index arithmetic; 60 (78) with the heads of one
// token ahead in registers in place of kDepth in shared memory.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "device_common.cuh"
#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace rot {

constexpr int kWarps = 12;   // passes of a token a CTA takes, at most
constexpr int kTokens = 8;   // tokens a CTA takes, at most
constexpr int kDepth = 4;    // tokens whose heads are on their way
constexpr int kSlot = 1024;  // bytes of a warp's pass

// The half layout with half the rotated part a multiple of 8 or of 4, the pairs
// layout at multiples of 8, and either one anywhere.
enum { kHalf = 0, kPairs = 1, kAny = 2, kHalf4 = 3 };

// 16 bytes past L1, or 8 bytes, into shared memory, asynchronously.
template <int kBytes>
__device__ __forceinline__ void copy_row(void* dst, const void* src) {
  if (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
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

// Where the tables keep pair r of a token: neighbouring lanes read neighbouring 16
// bytes, though in the half layout they need every second four pairs.
template <int LAYOUT, int kMaxPairs>
__device__ __forceinline__ int place_of(int r) {
  return LAYOUT == kHalf ? ((r >> 2) & 1) * (kMaxPairs / 2) + (r >> 3) * 4 + (r & 3) : r;
}

template <int LP>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LP / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Registers: 64 without a norm (three CTAs of ten warps an SM), 80 with one (two of
// twelve; at 64 its spills and recomputed addresses cost more than a third CTA gives).
template <bool F16, int LP, int NORM, int LAYOUT>
__global__ void __launch_bounds__(NORM || LAYOUT == kAny ? 32 * kWarps : 512, 2) rotate_kernel(const RotateParams p) {
  constexpr int kHeads = 32 / LP;    // heads a pass
  constexpr int kMaxPairs = LP * 8;  // pairs of a head's rotated part, at most
  constexpr int kStageRow = LP * 16 + 2;  // floats from head to head: apart in their banks
  __shared__ __align__(16) float cosines[kTokens][kMaxPairs], sines[kTokens][kMaxPairs];
  __shared__ __align__(16) float weights[NORM ? 2 : 1][NORM ? LP * 16 : 1];  // of q and k
  __shared__ __align__(16) float biases[NORM == 2 ? 2 : 1][NORM == 2 ? LP * 16 : 1];
  __shared__ __align__(16) float stage[LAYOUT == kAny ? kWarps : 1][LAYOUT == kAny ? kHeads * kStageRow : 1];
  // where a token's heads go: -1 nowhere (padding); q's, k's and v's byte offset else
  __shared__ int64_t places[kTokens][3];
  extern __shared__ __align__(16) uint8_t ring[];  // [warps][kDepth][kSlot]: of a lane two times 16 bytes
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5, warps = (int)blockDim.x >> 5;
  const int64_t tok0 = (int64_t)blockIdx.x * p.tokens;
  const int tokens = (int)min((int64_t)p.tokens, p.num_tokens - tok0);

  // the lane's pieces: elements e[c] .. e[c] + kPiece - 1 of its head
  const int sub = lane / LP, i = lane % LP, half = p.rot_dim >> 1;
  // In fours of elements, g = 0..3; a chunk is two of them, but in kHalf4, where a
  // lane has two pairs of fours that are partners.
  constexpr bool kByHalf = LAYOUT == kHalf || LAYOUT == kHalf4;
  constexpr int kPiece = LAYOUT == kHalf4 ? 4 : 8;  // elements that lie together
  constexpr int kPieces = 16 / kPiece;
  // Element a lane's piece begins at, head_dim or more: none.  By halves: lower and upper piece of
  // a pair, the rotated ones first, then the others two by two.
  auto piece_of = [&](int of_lane, int c) {
    if (!kByHalf) return 8 * (of_lane + c * LP);
    const int q = LAYOUT == kHalf4 ? of_lane + (c >> 1) * LP : of_lane, upper = c & 1;
    const int pairs = p.rot_dim / (2 * kPiece);
    if (q < pairs) return p.rot_offset + kPiece * q + upper * half;
    const int others = (p.head_dim - p.rot_dim) / kPiece, lower = (others + 1) >> 1;
    const int m = q - pairs < lower ? q - pairs + upper * lower : others;
    return m < others ? kPiece * m + (kPiece * m < p.rot_offset ? 0 : p.rot_dim) : p.head_dim;
  };
  int e[kPieces];
#pragma unroll
  for (int c = 0; c < kPieces; ++c) e[c] = piece_of(i, c);
  // Not kAny: the fours that are rotated together, their cosines' place in the tables.
  bool turned[2];
  int pairs_at[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int el = LAYOUT == kHalf ? e[0] : e[(LAYOUT == kHalf4 ? 2 : 1) * t], r = el - p.rot_offset;
    turned[t] = el < p.head_dim && r >= 0 && r < p.rot_dim;
    const int q = LAYOUT == kHalf ? 8 * i + 4 * t : (LAYOUT == kHalf4 ? 4 * (i + t * LP) : r >> 1);
    pairs_at[t] = turned[t] ? place_of<LAYOUT, kMaxPairs>(q) : 0;
  }
  const bool whole = p.rot_dim == p.head_dim;
  // the warp's pass: q's, k's or v's, and the lane's head of it
  const int pass = (int)blockIdx.y * warps + warp;
  const int part = pass < p.part_end[0] ? 0 : (pass < p.part_end[1] ? 1 : 2);
  const HeadRows& h = p.rows[part];
  const int head = (pass - (part == 0 ? 0 : p.part_end[part - 1])) * kHeads + sub;
  bool in[kPieces];
#pragma unroll
  for (int c = 0; c < kPieces; ++c) in[c] = head < h.heads && e[c] < p.head_dim;
  const uint8_t* src = h.x + tok0 * h.x_row + head * h.x_head;
  // The lane's pieces of the next token, into its own places of a slot.
  constexpr int kPieceBytes = 2 * kPiece;
  uint8_t* slots = ring + warp * (kDepth * kSlot) + lane * kPieceBytes;
  auto fetch = [&](int d) {
    if (d < tokens) {
#pragma unroll
      for (int c = 0; c < kPieces; ++c)
        if (in[c]) copy_row<kPieceBytes>(slots + (d % kDepth) * kSlot + c * (32 * kPieceBytes), src + 2 * e[c]);
      src += h.x_row;
    }
    copies_commit();
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d) fetch(d);

  // ---- of the CTA's tokens: their places, the angles; of the heads: the weights
  if ((int)threadIdx.x < tokens) {
    const int64_t t = tok0 + threadIdx.x;
    int64_t at[3] = {t * p.rows[0].out_row, t * p.rows[1].out_row, 0};
    if (p.slots != nullptr) {
      const int64_t slot = p.slots[t];
      at[1] = at[2] = -1;
      if (slot >= 0 && slot < p.num_slots) {
        const int64_t page = attn::div_nn(slot, p.page_tokens), off = slot - page * p.page_tokens;
        at[1] = page * p.k_page_stride + off * p.k_token_stride;
        at[2] = page * p.v_page_stride + off * p.v_token_stride;
      }
    }
    const bool padding = p.positions[t] < 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) places[threadIdx.x][k] = padding ? -1 : at[k];
  }
  if (NORM) {
    // four by four: the first four of every lane's 16, then the next
    for (int k = (int)threadIdx.x; k < 2 * LP * 16; k += (int)blockDim.x) {
      const int r = k / (LP * 16), at = k % (LP * 16), four = at / (LP * 4);
      const int el = piece_of((at >> 2) % LP, four * 4 / kPiece) + (four * 4) % kPiece + (at & 3);
      if (el >= p.head_dim) continue;
      weights[r][at] = weight_at<F16>(p.rows[r].weight, p.weight32, el, 1.0f);
      if (NORM == 2) biases[r][at] = weight_at<F16>(p.rows[r].bias, p.weight32, el, 0.0f);
    }
  }
  for (int k = (int)threadIdx.x; k < tokens * half; k += (int)blockDim.x) {
    const int d = k / half, r = k - d * half;
    const uint64_t turns = (uint32_t)p.positions[tok0 + d] * p.freqs[r];
    float s, c;
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
    cosines[d][place_of<LAYOUT, kMaxPairs>(r)] = c * p.magnitude;
    sines[d][place_of<LAYOUT, kMaxPairs>(r)] = s * p.magnitude;
  }
  __syncthreads();
  if (pass >= p.part_end[2]) return;

  uint8_t* base = h.out;
  int64_t step = h.out_head;
  if (base == nullptr) {
    base = part == 1 ? p.k_cache : p.v_cache;
    step = part == 1 ? p.k_head_stride : p.v_head_stride;
  }
  base += head * step;
#pragma unroll 1
  for (int d = 0; d < tokens; ++d) {
    copies_wait<kDepth - 1>();
    uint32_t raw[8];
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      const uint8_t* from = slots + (d % kDepth) * kSlot + c * (32 * kPieceBytes);
      if constexpr (kPiece == 8) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in[c]) v = *reinterpret_cast<const uint4*>(from);
        raw[4 * c] = v.x;
        raw[4 * c + 1] = v.y;
        raw[4 * c + 2] = v.z;
        raw[4 * c + 3] = v.w;
      } else {
        uint2 v = make_uint2(0, 0);
        if (in[c]) v = *reinterpret_cast<const uint2*>(from);
        raw[2 * c] = v.x;
        raw[2 * c + 1] = v.y;
      }
    }
    const int64_t place = places[d][part];
    if (place >= 0) {
      if (part < 2) {
        f2 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // elements 2 j and 2 j + 1 of the lane's 16
          const float2 v = unpack2<F16>(raw[j]);
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
            const float m = in[2 * j / kPiece] ? -mean : 0.0f;
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
          for (int j = 0; j < 8; j += 2) {
            const int at = (j / 2) * (LP * 4) + i * 4;  // (beside the head: whatever is there, not stored)
            const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(&weights[part][at]);
            x[j] = mul2(mul2(x[j], ff), w.x);
            x[j + 1] = mul2(mul2(x[j + 1], ff), w.y);
            if (NORM == 2) {
              const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&biases[part][at]);
              x[j] = add2(x[j], v.x);
              x[j + 1] = add2(x[j + 1], v.y);
            }
          }
        }
        // the rotation; elements beside the rotated part stay (without a norm: their bits)
        f2 y[8];
        uint32_t keep[8];  // bits of the packed pair that stay
        if (kByHalf) {
          const f2 minus = pair(-1.0f, -1.0f);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int lo = LAYOUT == kHalf ? 2 * t : 4 * t, hi = LAYOUT == kHalf ? 4 + 2 * t : 4 * t + 2;
            const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&cosines[d][pairs_at[t]]);
            const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(&sines[d][pairs_at[t]]);
            y[lo] = fma2(mul2(x[hi], minus), s.x, mul2(x[lo], c.x));
            y[lo + 1] = fma2(mul2(x[hi + 1], minus), s.y, mul2(x[lo + 1], c.y));
            y[hi] = fma2(x[lo], s.x, mul2(x[hi], c.x));
            y[hi + 1] = fma2(x[lo + 1], s.y, mul2(x[hi + 1], c.y));
            keep[lo] = keep[lo + 1] = keep[hi] = keep[hi + 1] = turned[t] ? 0u : ~0u;
          }
        } else if (LAYOUT == kPairs) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float4 c = *reinterpret_cast<const float4*>(&cosines[d][pairs_at[q]]);
            const float4 s = *reinterpret_cast<const float4*>(&sines[d][pairs_at[q]]);
            const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 v = both(x[4 * q + k]);
              y[4 * q + k] = pair(fmaf(-v.y, sn[k], v.x * cs[k]), fmaf(v.x, sn[k], v.y * cs[k]));
              keep[4 * q + k] = turned[q] ? 0u : ~0u;
            }
          }
        } else {
          float* row = &stage[warp][sub * kStageRow];
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) *reinterpret_cast<f2*>(&row[piece_of(i, j >> 2) + 2 * (j & 3)]) = x[j];
          __syncwarp();
          const bool pairs = p.layout == QSA_ROTARY_PAIRS;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 v = both(x[j]);
            float o[2] = {v.x, v.y};
            keep[j] = ~0u;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int el = piece_of(i, j >> 2) + 2 * (j & 3) + k, r = el - p.rot_offset;
              if (r >= 0 && r < p.rot_dim) {
                const bool first = pairs ? k == 0 : r < half;
                const int q = pairs ? r >> 1 : (first ? r : r - half);
                const float s = sines[d][q], xp = row[first ? el + (pairs ? 1 : half) : el - (pairs ? 1 : half)];
                o[k] = fmaf(xp, first ? -s : s, o[k] * cosines[d][q]);
                keep[j] &= k ? 0xFFFFu : 0xFFFF0000u;
              }
            }
            y[j] = pair(o[0], o[1]);
          }
        }
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 v = both(y[j]);
          o[j] = attn::pack2<F16>(v.x, v.y);
        }
        if (!whole) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (NORM) {
              const float2 n = both(x[j]);
              raw[j] = attn::pack2<F16>(n.x, n.y);
            }
            o[j] = (raw[j] & keep[j]) | (o[j] & ~keep[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) raw[j] = o[j];
      }
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        if (!in[c]) continue;
        if constexpr (kPiece == 8)
          *reinterpret_cast<uint4*>(base + place + 2 * e[c]) =
              make_uint4(raw[4 * c], raw[4 * c + 1], raw[4 * c + 2], raw[4 * c + 3]);
        else
          *reinterpret_cast<uint2*>(base + place + 2 * e[c]) = make_uint2(raw[2 * c], raw[2 * c + 1]);
      }
    }
    fetch(d + kDepth);  // into the slot just read and worked on
  }
}

template <bool F16, int LP, int NORM, int LAYOUT>
cudaError_t launch(const RotateParams& p, int device, dim3 grid, int threads, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(rotate_kernel<F16, LP, NORM, LAYOUT>, kWarps * kDepth * kSlot, device, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)(threads / 32) * kDepth * kSlot;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotate_kernel<F16, LP, NORM, LAYOUT>, p);
}

template <bool F16, int LP, int NORM>
cudaError_t launch_layout(const RotateParams& p, int device, dim3 grid, int threads, cudaStream_t stream) {
  if (p.layout == QSA_ROTARY_PAIRS && p.rot_dim % 8 == 0 && p.rot_offset % 8 == 0)
    return launch<F16, LP, NORM, kPairs>(p, device, grid, threads, stream);
  if (p.layout == QSA_ROTARY_HALF && p.rot_dim % 8 == 0 && p.rot_offset % 4 == 0 &&
      (p.rot_dim % 16 != 0 || p.rot_offset % 8 != 0))
    return launch<F16, LP, NORM, kHalf4>(p, device, grid, threads, stream);
  if (p.layout == QSA_ROTARY_HALF && p.rot_dim % 16 == 0 && p.rot_offset % 8 == 0) return launch<F16, LP, NORM, kHalf>(p, device, grid, threads, stream);
  return launch<F16, LP, NORM, kAny>(p, device, grid, threads, stream);
}

template <bool F16, int LP>
cudaError_t launch_norm(const RotateParams& p, int device, dim3 grid, int threads, cudaStream_t stream) {
  if (p.norm == QSA_NORM_RMS) return launch_layout<F16, LP, 1>(p, device, grid, threads, stream);
  if (p.norm == QSA_NORM_LAYER) return launch_layout<F16, LP, 2>(p, device, grid, threads, stream);
  return launch_layout<F16, LP, 0>(p, device, grid, threads, stream);
}

// A CTA takes the number of tokens that ends soonest: rounds of the CTAs that the
// GPU holds at once, each as long as its tokens and a start that costs three
// (at most three tokens instead: 4000 tokens with norm and store 23.2 us for 19.4,
// 2051 of 64 heads 13.0 for 12.4).
template <bool F16>
cudaError_t launch_rotate_t(RotateParams p, cudaStream_t stream) {
  DeviceInfo info;
  cudaError_t e = device_info(&info);
  if (e != cudaSuccess) return e;
  const int lp = p.head_dim <= 64 ? 4 : (p.head_dim <= 128 ? 8 : 16), heads = 32 / lp;
  int32_t end = 0;
  for (int i = 0; i < 3; ++i) p.part_end[i] = end += (p.rows[i].heads + heads - 1) / heads;
  const int groups = (end + kWarps - 1) / kWarps, warps = (end + groups - 1) / groups;
  const int resident = (p.norm == QSA_NORM_NONE ? 32 : 25) / warps;  // CTAs an SM, by their registers
  const int64_t held = (int64_t)info.num_sms * (resident > 0 ? resident : 1);
  int64_t best = INT64_MAX;
  for (int n = 1; n <= kTokens; ++n) {
    const int64_t ctas = (p.num_tokens + n - 1) / n * groups, cost = (ctas + held - 1) / held * (n + 3);
    if (cost < best) best = cost, p.tokens = n;
  }
  const dim3 grid((unsigned)((p.num_tokens + p.tokens - 1) / p.tokens), (unsigned)groups, 1);
  if (lp == 4) return launch_norm<F16, 4>(p, info.device, grid, 32 * warps, stream);
  if (lp == 8) return launch_norm<F16, 8>(p, info.device, grid, 32 * warps, stream);
  return launch_norm<F16, 16>(p, info.device, grid, 32 * warps, stream);
}

}  // namespace rot
}  // namespace qsa
