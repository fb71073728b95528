// Parameters and the work schedule shared by the two forms of
// qsa_paged_attention (attn_gather.cu, attn_tile.cu).
//
// Work is counted in units of 128 keys of one item; an item is a group of
// query rows that share their keys: `tpi` consecutive new tokens of a request
// times the query heads of a (virtual) key/value head.  The items of a call,
// request by request, then head by head, then along the tokens, form one list
// of units, of which each of the launch's CTAs takes an equal, contiguous
// share: every CTA has the same work to within a unit whatever the lengths are,
// one long request among short ones included.  An item counts item_cost units
// behind those of its keys, for its start and its end: without them the CTAs
// that get many short items finish last.  An item whose units lie in several
// CTAs is joined from their parts (partial sums with their running maximum and
// sum).  A CTA has at most two unfinished parts, the one it begins with and the
// one it ends with, so the workspace is two parts a CTA.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"
#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace attn {

constexpr int kUnit = 128;      // keys a unit
constexpr int kMaxGrid = 160;   // CTAs a launch, at most (GB300 has 152 SMs)
static_assert(kMaxGrid * 4 == QSA_ATTN_COUNTER_BYTES, "one counter a CTA");
constexpr int32_t kNoPage = -1; // block-table entry: the page is missing (free list exhausted), its tokens are not seen
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

__device__ __forceinline__ int32_t units_of(int32_t keys) { return max(1, (keys + kUnit - 1) / kUnit); }
__device__ __forceinline__ int32_t item_units(const AttnParams& p, int32_t keys) { return units_of(keys) + p.item_cost; }

// a / b of non-negative values; in 32 bits when they allow it (a 64-bit
// division is some hundred instructions).
__device__ __forceinline__ int64_t div_nn(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

__device__ __forceinline__ int32_t tiles_of(const AttnParams& p, int32_t n) { return (n + p.tpi - 1) / p.tpi; }

// Units of tile t of a request: of the tokens [t * tpi, (t + 1) * tpi).
__device__ __forceinline__ int32_t tile_units(const AttnParams& p, const Request& r, int32_t t) {
  return item_units(p, keys_of(p, r, min((t + 1) * p.tpi, r.n)));
}

// Units of one head of each lane's request (n = 0: none), by the whole warp: a
// lane adds up a few tiles itself, many are shared out over the lanes.
__device__ __forceinline__ int64_t head_units(const AttnParams& p, const Request& r) {
  constexpr int32_t kAlone = 4;
  const int lane = (int)threadIdx.x & 31;
  const int32_t tiles = tiles_of(p, r.n);
  int64_t u = 0;
  if (tiles <= kAlone)
    for (int32_t t = 0; t < tiles; ++t) u += tile_units(p, r, t);
  uint32_t many = __ballot_sync(0xffffffffu, tiles > kAlone);
  while (many) {
    const int src = __ffs(many) - 1;
    many &= many - 1;
    Request q;
    q.n = __shfl_sync(0xffffffffu, r.n, src);
    q.pos0 = __shfl_sync(0xffffffffu, r.pos0, src);
    int64_t part = 0;
    for (int32_t t = lane; t < tiles_of(p, q.n); t += 32) part += tile_units(p, q, t);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == src) u = part;
  }
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

// How the list is shared out: the first `more` CTAs take each + 1 units, the others `each`.
struct Schedule {
  int64_t total, each;
  int32_t ge, more;  // CTAs that take part
  int64_t u0, u1;    // this CTA's units

  __device__ __forceinline__ void share_out(int64_t units, int32_t min_shift) {
    total = units;
    ge = (int32_t)min((int64_t)gridDim.x, max((int64_t)1, total >> min_shift));
    each = div_nn(total, ge);
    more = (int32_t)(total - each * ge);
    const int c = (int)blockIdx.x;
    u0 = c < ge ? share(c) : total;
    u1 = c < ge ? share(c + 1) : total;
  }
  __device__ __forceinline__ int64_t share(int c) const { return c * each + min(c, more); }
  // The CTA whose share holds unit u.
  __device__ __forceinline__ int owner(int64_t u) const {
    const int64_t cut = more * (each + 1);
    return u < cut ? (int)div_nn(u, each + 1) : more + (int)div_nn(u - cut, each);
  }
};

// A CTA's part of an item: its units [a, z) of the item's keys.  An item's keys
// come before its item_cost, so only the first item of a share can be one the
// CTA has no part in (a >= z).
struct Part {
  int32_t a, z;
  __device__ __forceinline__ Part(const AttnParams& p, const Schedule& s, const Item& it) {
    a = (int32_t)(max(s.u0, it.s0) - it.s0);
    z = (int32_t)(min(s.u1, it.s1 - p.item_cost) - it.s0);
  }
};
// The first and the last CTA that have a part of the item, given that this one has.
__device__ __forceinline__ int first_cta(const Schedule& s, const Item& it) {
  return it.s0 >= s.u0 ? (int)blockIdx.x : s.owner(it.s0);
}
__device__ __forceinline__ int last_cta(const AttnParams& p, const Schedule& s, const Item& it) {
  const int64_t end = it.s1 - p.item_cost;
  return end <= s.u1 ? (int)blockIdx.x : s.owner(end - 1);
}

// What the warps that work on an item need of it, from the one that walks the list.
struct ItemInfo {
  int32_t a, z;        // the CTA's units of it
  int32_t row0, n;     // rows of q
  int32_t pos0, keys;
  int32_t gs, head0;   // query heads of its virtual head
  int32_t c0, c1;      // the CTAs that have a part of it
  int32_t last;        // of this CTA
};

struct SchedShared {
  int64_t warp_sum[32];
  int64_t base;      // as in Start
  int64_t per_head;
  int32_t b;
};

// Where a CTA's share begins: the request its first unit belongs to.
struct Start {
  int64_t base;      // units before that request
  int64_t per_head;  // units of one head of it
  int32_t b;
  Request r;
};

// Builds the schedule over the requests' lengths; called by all NT threads, it
// contains a CTA barrier.  Up to 32 requests every warp does it by itself, a
// lane a request.  More: NT requests a round, a thread a request, ordered by a
// block scan, and the thread whose request holds the CTA's first unit says so.
// Up to NT requests the second pass works on what the first has in registers.
template <int NT>
__device__ __forceinline__ Schedule make_schedule(const AttnParams& p, SchedShared& sh, Start& at) {
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.num_requests;
  Schedule s;
  auto scan = [&](int64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += a;
    }
    return v;
  };
  if (B <= 32) {
    Request r = {0, 0, 0};
    if (lane < B) r = request_of(p, lane);
    const int64_t head = head_units(p, r), mine = head * p.hv, incl = scan(mine);
    s.share_out(__shfl_sync(0xffffffffu, incl, 31), p.min_shift);
    const uint32_t here = __ballot_sync(0xffffffffu, incl - mine <= s.u0 && s.u0 < incl);
    const int src = here ? __ffs(here) - 1 : 0;
    at.b = src;
    at.base = __shfl_sync(0xffffffffu, incl - mine, src);
    at.per_head = __shfl_sync(0xffffffffu, head, src);
    at.r.first = __shfl_sync(0xffffffffu, r.first, src);
    at.r.n = __shfl_sync(0xffffffffu, r.n, src);
    at.r.pos0 = __shfl_sync(0xffffffffu, r.pos0, src);
    __syncthreads();
    return s;
  }
  int64_t head = 0, before = 0, sum = 0;  // of this thread's request; of the rounds so far
  auto round = [&](int b0) {
    Request r = {0, 0, 0};
    if (b0 + tid < B) r = request_of(p, b0 + tid);
    head = head_units(p, r);
    const int64_t mine = head * p.hv, incl = scan(mine);
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    before = sum + incl - mine;
    for (int w = 0; w < NT / 32; ++w) {
      const int64_t v = sh.warp_sum[w];
      if (w < warp) before += v;
      sum += v;
    }
  };
  round(0);
  for (int b0 = NT; b0 < B; b0 += NT) {
    __syncthreads();
    round(b0);
  }
  s.share_out(sum, p.min_shift);
  auto look = [&](int b0) {
    const int64_t mine = head * p.hv;
    if (s.u0 < s.u1 && before <= s.u0 && s.u0 < before + mine) {
      sh.b = b0 + tid;
      sh.base = before;
      sh.per_head = head;
    }
  };
  if (B <= NT) {
    look(0);
  } else {
    sum = 0;
    for (int b0 = 0; b0 < B; b0 += NT) {
      __syncthreads();
      round(b0);
      look(b0);
    }
  }
  __syncthreads();
  if (s.u0 < s.u1) at = {sh.base, sh.per_head, sh.b, request_of(p, sh.b)};
  return s;
}

// Walks the items of the list from the one that holds unit u0; made and moved
// by whole warps.
struct Walker {
  const AttnParams& p;
  Item it;
  Request r;

  __device__ __forceinline__ Walker(const AttnParams& p_, const Item& at) : p(p_), it(at), r(request_of(p_, at.b)) {}
  __device__ __forceinline__ Walker(const AttnParams& p_, const Item& at, const Request& r_) : p(p_), it(at), r(r_) {}
  __device__ __forceinline__ Walker(const AttnParams& p_, const Start& at, int64_t u0) : p(p_), r(at.r) {
    const int lane = (int)threadIdx.x & 31;
    it.b = at.b;
    int64_t rem = u0 - at.base;
    it.hv = (int32_t)div_nn(rem, at.per_head);
    rem -= it.hv * at.per_head;
    int64_t s = u0 - rem;  // the head's first unit
    const int32_t tiles = tiles_of(p, r.n);
    for (int32_t t0 = 0;; t0 += 32) {  // 32 tiles at a time: the one that holds the unit
      const int32_t u = t0 + lane < tiles ? tile_units(p, r, t0 + lane) : 0;
      int32_t incl = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t a = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += a;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, rem < incl);
      if (past) {
        const int src = __ffs(past) - 1;
        const int32_t n = __shfl_sync(0xffffffffu, u, src), z = __shfl_sync(0xffffffffu, incl, src);
        it.i0 = (t0 + src) * p.tpi;
        it.s1 = s + z;
        it.s0 = it.s1 - n;
        break;
      }
      const int32_t all = __shfl_sync(0xffffffffu, incl, 31);
      rem -= all;
      s += all;
      if (t0 + 32 >= tiles) {  // not reached: the head holds the unit
        it.i0 = 0;
        it.s0 = it.s1 = s;
        break;
      }
    }
    set();
  }
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
    it.s1 += item_units(p, it.keys);
  }
};

// Whether the CTA has work at all, and `it` moved to its first item.
// (Its callers have units, s.u0 < s.u1.)
template <typename Next>
__device__ __forceinline__ bool first_part(const AttnParams& p, const Schedule& s, Item& it, const Next& next) {
  if (s.u0 < it.s1 - p.item_cost) return true;
  if (it.s1 >= s.u1) return false;
  next(it);
  return true;
}

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
