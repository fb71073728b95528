// Parameters and the work schedule shared by the two forms of
// qsa_paged_attention (attn_gather.cu, attn_tile.cu).
//
// Work is counted in units of `unit` keys (128, or 192) of one item; an item is a group of
// query rows that share their keys: `tpi` consecutive new tokens of a request
// times the query heads of a (virtual) key/value head.  The items of a call,
// request by request, then head by head, then along the tokens, form one list
// of units, and CTA c of `ge` takes the units [total * c / ge, total * (c+1) /
// ge): every CTA has the same work to within a unit whatever the lengths are,
// one long request among short ones included, and an item whose units lie in
// several CTAs is joined from their parts (partial sums with their running
// maximum and sum).  A CTA has at most two unfinished parts, the one it begins
// with and the one it ends with, so the workspace is two parts a CTA.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"
#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace attn {

constexpr int kMaxGrid = 160;   // CTAs a launch, at most (GB300 has 152 SMs)
static_assert(kMaxGrid * 4 == QSA_ATTN_COUNTER_BYTES, "one counter a CTA");
constexpr float kLn2 = 0.6931471805599453f;
constexpr long long kSpin = 2000000000LL;  // about one second of SM clocks

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 values rounded to the 16-bit type, `lo` in the low half.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

struct Request {
  int32_t first, n;   // first row of q, new tokens
  int32_t pos0;       // position of its first new token (negative: inconsistent lengths, sees nothing)
};

__device__ __forceinline__ Request request_of(const AttnParams& p, int b) {
  const int32_t a = min(max(p.query_start[b], 0), p.num_tokens);
  const int32_t z = min(max(p.query_start[b + 1], a), p.num_tokens);
  return {a, z - a, (int32_t)min(max((int64_t)p.seq_lens[b], (int64_t)0), kMaxKeys) - (z - a)};
}

// Keys that the last of the tokens [0, i1) of a request sees, at most the table's capacity.
__device__ __forceinline__ int32_t keys_of(const AttnParams& p, const Request& r, int i1) {
  return min(max(r.pos0 + i1, 0), p.capacity);
}

__device__ __forceinline__ int32_t units_of(const AttnParams& p, int32_t keys) {
  return max(1, (keys + p.unit - 1) / p.unit);
}

// Units of one head of a request: the sum over its items.
__device__ __forceinline__ int64_t head_units(const AttnParams& p, const Request& r) {
  int64_t u = 0;
  for (int i = 0; i < r.n; i += p.tpi) u += units_of(p, keys_of(p, r, min(i + p.tpi, r.n)));
  return u;
}

struct Item {
  int32_t b, hv;     // request, virtual head
  int32_t i0, n;     // first token within the request, tokens
  int32_t row0;      // row of q of the first token
  int32_t pos0;      // position of the first token
  int32_t keys;      // keys the last token sees
  int64_t s0, s1;    // the item's units in the call's list
};

// The schedule of a launch; made by every thread of a CTA together.
struct Schedule {
  int64_t total;
  int32_t ge;        // CTAs that take part
  int64_t u0, u1;    // this CTA's units

  __device__ __forceinline__ int64_t share(int c) const { return total * c / ge; }
  // The CTA whose share holds unit u.
  __device__ __forceinline__ int owner(int64_t u) const {
    int c = (int)min((int64_t)(ge - 1), u * ge / total);
    while (c + 1 < ge && share(c + 1) <= u) ++c;
    while (c > 0 && share(c) > u) --c;
    return c;
  }
};

struct SchedShared {
  int64_t warp_sum[32];
  int64_t base;   // units before the first request of this CTA's share
  int32_t b;      // that request
};

// Builds the schedule over the requests' lengths: each thread sums a
// contiguous run of requests, a block scan orders the runs, and the thread
// whose run holds the CTA's first unit finds its request.
template <int NT>
__device__ __forceinline__ Schedule make_schedule(const AttnParams& p, SchedShared& sh) {
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.num_requests;
  const int per = (B + NT - 1) / NT;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += head_units(p, request_of(p, b)) * p.hv;
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += a;
  }
  if (lane == 31) sh.warp_sum[warp] = incl;
  if (tid == 0) sh.b = B, sh.base = 0;
  __syncthreads();
  int64_t before = incl - sum, total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += sh.warp_sum[w];
    total += sh.warp_sum[w];
  }
  Schedule s;
  s.total = total;
  const int64_t want = (total + p.min_units - 1) / p.min_units;
  s.ge = (int)min((int64_t)gridDim.x, max((int64_t)1, want));
  const int c = (int)blockIdx.x;
  s.u0 = c < s.ge ? s.share(c) : total;
  s.u1 = c < s.ge ? s.share(c + 1) : total;
  if (s.u0 < s.u1 && before <= s.u0 && s.u0 < before + sum) {
    int64_t base = before;
    for (int b = b0; b < b1; ++b) {
      const int64_t u = head_units(p, request_of(p, b)) * p.hv;
      if (s.u0 < base + u) {
        sh.b = b;
        sh.base = base;
        break;
      }
      base += u;
    }
  }
  __syncthreads();
  return s;
}

// Walks the items of the list from the one that holds unit u0.
struct Walker {
  const AttnParams& p;
  Item it;
  Request r;

  __device__ __forceinline__ Walker(const AttnParams& p_, const SchedShared& sh, int64_t u0) : p(p_) {
    it.b = sh.b;
    r = request_of(p, it.b);
    const int64_t per_head = head_units(p, r);
    int64_t rem = u0 - sh.base;
    it.hv = (int32_t)(rem / per_head);
    rem -= it.hv * per_head;
    int64_t s = u0 - rem;
    it.i0 = 0;
    for (;;) {
      set();
      const int32_t u = units_of(p, it.keys);
      if (rem < u) {
        it.s0 = s;
        it.s1 = s + u;
        return;
      }
      rem -= u;
      s += u;
      it.i0 += p.tpi;
    }
  }
  __device__ __forceinline__ Walker(const AttnParams& p_, const Item& at) : p(p_), it(at), r(request_of(p_, at.b)) {}
  __device__ __forceinline__ void set() {
    it.n = min(p.tpi, r.n - it.i0);
    it.row0 = r.first + it.i0;
    it.pos0 = r.pos0 + it.i0;
    it.keys = keys_of(p, r, it.i0 + it.n);
  }
  // To the next item; there is one (its first unit is it.s1).
  __device__ __forceinline__ void next() {
    it.i0 += p.tpi;
    if (it.i0 >= r.n) {
      it.i0 = 0;
      if (++it.hv == p.hv) {
        it.hv = 0;
        do r = request_of(p, ++it.b);
        while (r.n == 0);
      }
    }
    set();
    it.s0 = it.s1;
    it.s1 += units_of(p, it.keys);
  }
};

// Bounded wait on an mbarrier phase; false on a time-out (fault bit 3).
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                           unsigned int* fault) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kSpin) {
      *abort_flag = 1;
      atomicOr(fault, 8u);
      return false;
    }
  }
}

}  // namespace attn
}  // namespace qsa
