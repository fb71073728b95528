// qsa_verify_drafts: which drafted tokens the target accepts, and the token that
// follows them, from given random numbers.
//
// Draft i of a request is accepted while u_i q_i(x_i) < p_i(x_i), p the target's
// probabilities and q the draft's (1 for a certain draft).  At the first refusal
// a the next token is drawn from max(p_a - q_a, 0), after the last acceptance
// from p_n: the smallest j whose cumulative weight exceeds u times the total.
// Accepted so, the tokens are distributed as the target's own samples.
//
// Weights count in units of 2^-45 (exactly, from 2^-22 up in fp32), so totals and
// cumulative sums do not depend on the order in which the parts are added, and the
// comparison u * total < cumulative is exact too.  A row's weights are summed
// once, by a cluster of CTAs that each take a contiguous share and each warp a
// contiguous part of it; the totals cross the cluster through shared memory, and
// the CTA whose share holds the drawn point reads the one part that does again, a
// group of tokens a warp.
//
// What bounds it: the row of p (and of q) of each request, from HBM, once; for
// few requests the chain of loads ahead of the row (the drafts, their
// probabilities), the row, and the cluster's exchange; between the two the sums'
// instructions.  Units comes to six a value: integer significands shifted into 64
// bits took 54 (those instructions run at half rate or less), 32 us for 64 requests
// x 131072 tokens, three exact fp32 accumulators nine, 20 us.
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"
#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace {

constexpr int kNT = 512;
constexpr int kWarps = kNT / 32;
constexpr int kMaxCluster = 16;  // above 8: where the device takes such clusters
constexpr uint32_t kAll = 0xffffffffu;

template <typename T>
__device__ __forceinline__ float as_float(T v);
template <>
__device__ __forceinline__ float as_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float as_float<__half>(__half v) { return __half2float(v); }

// The units of a probability in [0, 1]: the significand times a power of two.
// Below 2^-22, where that would be a fraction, the sum with 2^-22 rounds to whole
// units (ties to even), which the difference of the bit patterns counts.
__device__ __forceinline__ uint64_t units_of(float p) {
  const uint32_t bits = __float_as_uint(p);
  if (p < 0x1p-22f) return __float_as_uint(p + 0x1p-22f) - __float_as_uint(0x1p-22f);
  return (uint64_t)((bits & 0x7FFFFFu) | 0x800000u) << ((bits >> 23) - 105);
}

using f2 = uint64_t;  // two fp32 values in a register pair
__device__ __forceinline__ f2 pair(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 sub2(f2 a, f2 b, f2 minus) {  // minus: (-1, -1)
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(b), "l"(minus), "l"(a));
  return r;
}

// A sum of values in [-1, 1], two a call, in units of 2^-45.  Added to 3 a value is
// rounded to a multiple of 2^-22, which the bit pattern counts from that of 3; the
// rest, found without error, added to 1.5 * 2^-22 likewise to one of 2^-45 (ties to
// even).  Both counts stay within 22 bits and their sign, so kValues of them, and
// the patterns they are counted from, add up in 32 bits.
struct Units {
  static constexpr int kValues = 128;
  static constexpr float kFirst = 3.0f, kSecond = 0x1.8p-22f;
  uint32_t high = 0, low = 0;
  uint64_t sum = 0;
  __device__ __forceinline__ void add(f2 v, f2 minus) {
    const f2 first = pair(kFirst, kFirst);
    const f2 t = add2(v, first);
    const f2 r = sub2(v, sub2(t, first, minus), minus);
    const f2 s = add2(r, pair(kSecond, kSecond));
    uint32_t x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(t));
    high += x + y;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(s));
    low += x + y;
  }
  // To whole units, after n values.
  __device__ __forceinline__ void total(uint32_t n) {
    const int32_t h = (int32_t)(high - n * __float_as_uint(kFirst)), l = (int32_t)(low - n * __float_as_uint(kSecond));
    sum += (uint64_t)((int64_t)h * (1LL << 23) + l);
    high = low = 0;
  }
};

// Which of the kWarps sums in shared memory `want` falls into, counted from the
// first: the lowest k with sums[0] + .. + sums[k] >= want (kWarps: none, `want`
// is left less all of them).  By a whole warp; want less the sums before.
__device__ __forceinline__ int find(const uint64_t* sums, uint64_t& want) {
  const int lane = (int)threadIdx.x & 31;
  const uint64_t mine = lane < kWarps ? sums[lane] : 0;
  uint64_t incl = mine;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const uint64_t v = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += v;
  }
  const uint32_t hit = __ballot_sync(kAll, lane < kWarps && incl >= want);
  const int k = hit ? __ffs(hit) - 1 : kWarps;
  want -= __shfl_sync(kAll, hit ? incl - mine : incl, hit ? k : kWarps - 1);
  return k;
}

// The probability of a drafted token as a double, clamped the same way.
template <typename T>
__device__ __forceinline__ double prob_at(const T* row, int64_t x) {
  return (double)__saturatef(as_float(row[x]));
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// kV probabilities from 16 bytes of them, in [0, 1].
template <typename T, int kV>
__device__ __forceinline__ void unpack(const uint4& w, float (&v)[kV]) {
  const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
  for (int i = 0; i < kV; ++i) v[i] = __saturatef(as_float(e[i]));
}

// A request's two rows, read in 16-byte pieces of kV tokens that lie on 16 bytes
// of p's row.  ALIGNED: every row of the call begins on 16 bytes and has a whole
// number of pieces.  Otherwise p's row begins `off` tokens into its first piece,
// and q's tokens of a piece begin `turn` tokens into one of its own, so that they
// are put together from two.  Pieces that do not lie within the row (its first
// and last) are read token by token, those past it as zeros.
template <typename T, bool ALIGNED>
struct Rows {
  static constexpr int kV = 16 / (int)sizeof(T);
  const T *p, *q;  // q null: p alone
  int32_t vocab, off, turn;

  __device__ __forceinline__ void place() {
    off = ALIGNED ? 0 : (int32_t)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    turn = ALIGNED || !q ? 0 : (int32_t)(((reinterpret_cast<uintptr_t>(q) - off * sizeof(T)) & 15) / sizeof(T));
  }
  // Piece n holds the tokens first(n) .. first(n) + kV - 1.
  __device__ __forceinline__ int32_t first(int32_t n) const { return n * kV - off; }
  __device__ __forceinline__ uint4 one_by_one(const T* row, int32_t j) const {
    alignas(16) T e[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) e[i] = j + i >= 0 && j + i < vocab ? row[j + i] : T(0.0f);
    return *reinterpret_cast<const uint4*>(e);
  }
  __device__ __forceinline__ uint4 load_p(int32_t j) const {
    if (ALIGNED) return j < vocab ? *reinterpret_cast<const uint4*>(p + j) : make_uint4(0, 0, 0, 0);
    if (j >= 0 && j + kV <= vocab) return *reinterpret_cast<const uint4*>(p + j);
    return one_by_one(p, j);
  }
  // v and (not ALIGNED) the piece behind it; `whole` false: v are the tokens already.
  __device__ __forceinline__ bool whole_q(int32_t j) const { return j - turn >= 0 && j - turn + 2 * kV <= vocab; }
  __device__ __forceinline__ void load_q(int32_t j, uint4& v, uint4& behind) const {
    if (ALIGNED) {
      v = j < vocab ? *reinterpret_cast<const uint4*>(q + j) : make_uint4(0, 0, 0, 0);
    } else if (whole_q(j)) {
      v = *reinterpret_cast<const uint4*>(q + j - turn);
      behind = *reinterpret_cast<const uint4*>(q + j - turn + kV);
    } else {
      v = one_by_one(q, j);
    }
  }
  __device__ __forceinline__ uint4 tokens_of_q(int32_t j, const uint4& v, const uint4& behind) const {
    if (ALIGNED || turn == 0) return v;  // (turn 0: whole or one by one, v are the tokens)
    uint32_t w[8] = {v.x, v.y, v.z, v.w, behind.x, behind.y, behind.z, behind.w};
    const int bytes = turn * (int)sizeof(T);
    if (bytes & 8) {
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (bytes & 4) {
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (sizeof(T) == 2) {
      const int bits = 8 * (bytes & 3);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
    }
    return whole_q(j) ? make_uint4(w[0], w[1], w[2], w[3]) : v;
  }
};

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kNT, 2) verify_kernel(const VerifyParams p, int cluster) {
  constexpr int kV = 16 / (int)sizeof(T);
  __shared__ uint64_t cta_sum[2][kMaxCluster];  // of every CTA of the cluster; a second try's apart
  __shared__ uint64_t part_sum[kWarps], group_sum[2][kWarps];
  const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
  const int b = (int)blockIdx.x / cluster, rank = (int)blockIdx.x - b * cluster;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  // Every CTA of the cluster runs before one writes into its shared memory; the wait is below.
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  const T* target = static_cast<const T*>(p.target) + (int64_t)b * p.target_request;
  const T* draft = p.draft ? static_cast<const T*>(p.draft) + (int64_t)b * p.draft_request : nullptr;
  const float* u = p.uniforms + (int64_t)b * (p.max_drafts + 1);
  const int32_t* tokens = p.tokens + (int64_t)b * p.max_drafts;
  const float uf = u[p.max_drafts];
  const int32_t n = p.num_drafts ? min(max(p.num_drafts[b], 0), p.max_drafts) : p.max_drafts;

  // ---- accepted drafts, by every warp for itself
  int32_t a = n;
  for (int32_t i0 = 0; i0 < p.max_drafts; i0 += 32) {
    const int32_t i = i0 + lane;
    bool ok = false;
    if (i < p.max_drafts) {  // read beside num_drafts, used where i < n
      const int32_t x = tokens[i];
      if (x >= 0 && x < p.vocab) {
        const double pt = prob_at(target + (int64_t)i * p.target_row, x);
        const double qd = draft ? prob_at(draft + (int64_t)i * p.draft_row, x) : 1.0;
        ok = (double)__saturatef(u[i]) * qd < pt;  // (saturated, NaN is 0)
      }
    }
    const uint32_t refused = __ballot_sync(kAll, i < n && !ok);
    if (refused) {
      a = i0 + __ffs(refused) - 1;
      break;
    }
    if (i0 + 32 >= n) break;
  }

  // The row's weights: max(p - q, 0) of a refused draft's, or p but for the certain
  // draft (all its distribution's weight: never below p's); p alone otherwise.
  bool refused = a < n;
  Rows<T, ALIGNED> rows;
  rows.p = target + (int64_t)a * p.target_row;
  rows.q = refused && draft ? draft + (int64_t)a * p.draft_row : nullptr;
  rows.vocab = p.vocab;
  rows.place();
  int32_t without = refused && !draft ? tokens[a] : -1;

  // ---- the parts of the row: groups of 32 pieces, of which a lane has one
  constexpr int kGroup = 32 * kV;
  const int32_t groups = (p.vocab + rows.off + kGroup - 1) / kGroup;
  const int32_t parts = cluster * kWarps;
  const int32_t each = groups / parts, more = groups - each * parts;
  auto part_begin = [&](int32_t k) { return k * each + min(k, more); };
  uint64_t all = 0;
  int attempt = 0;
#pragma unroll 1
  for (;; ++attempt) {
    // max(p - q, 0) = p - min(p, q).  kAhead groups' loads are in flight.
    constexpr int kAhead = ALIGNED ? 4 : 2;
    uint32_t count = 0;  // values added since the last total
    const f2 minus = pair(-1.0f, -1.0f);
    Units units;
    const int32_t g0 = part_begin(rank * kWarps + warp), g1 = part_begin(rank * kWarps + warp + 1);
#pragma unroll 1
    for (int32_t g = g0; g < g1; g += kAhead) {
      uint4 w[kAhead], v[kAhead], x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int32_t j = g + k < g1 ? rows.first((g + k) * 32 + lane) : p.vocab;
        w[k] = rows.load_p(j);
        if (rows.q) rows.load_q(j, v[k], x[k]);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (g + k >= g1) break;
        float pv[kV], qv[kV];
        unpack<T, kV>(w[k], pv);
#pragma unroll
        for (int i = 0; i < kV; i += 2) units.add(pair(pv[i], pv[i + 1]), minus);
        if (rows.q) {
          unpack<T, kV>(rows.tokens_of_q(rows.first((g + k) * 32 + lane), v[k], x[k]), qv);
#pragma unroll
          for (int i = 0; i < kV; i += 2)
            units.add(pair(fmaxf(-pv[i], -qv[i]), fmaxf(-pv[i + 1], -qv[i + 1])), minus);
        }
      }
      count += min(kAhead, g1 - g) * (rows.q ? 2 * kV : kV);
      if (count > Units::kValues - 2 * kAhead * kV || g + kAhead >= g1) {
        units.total(count);
        count = 0;
      }
    }
    uint64_t sum = warp_sum(units.sum);
    if (without >= max(rows.first(g0 * 32), 0) && without < min(rows.first(g1 * 32), p.vocab))
      sum -= units_of(__saturatef(as_float(rows.p[without])));
    if (lane == 0) part_sum[warp] = sum;
    __syncthreads();
    // ---- totals to every CTA of the cluster
    if (attempt == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if ((int)threadIdx.x < cluster) {
      uint64_t mine = 0;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) mine += part_sum[k];
      uint32_t remote;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                   : "=r"(remote)
                   : "r"(ptx::smem_u32(&cta_sum[attempt][rank])), "r"((int)threadIdx.x));
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote), "l"(mine) : "memory");
    }
    __syncwarp();  // the barrier takes whole warps
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
    all = 0;
    for (int c = 0; c < cluster; ++c) all += cta_sum[attempt][c];
    if (all > 0 || !refused) break;
    refused = false;  // nothing left of the refused row: p itself
    rows.q = nullptr;
    without = -1;
  }

  // ---- the drawn point: this CTA's, one of its parts', a token of one group
  int32_t next = -1;
  if (all == 0) {  // no weight at all: no token
    if (rank != 0 || warp != 0) return;
  } else {
    // u in units of 2^-64, in [0, 1); point = floor(all * u), and a cumulative sum
    // exceeds all * u exactly when it exceeds that
    const uint64_t u64 = uf > 0.0f ? (uf < 1.0f ? (uint64_t)(uf * 0x1p64f) : ~0ull) : 0ull;
    const uint64_t point = __umul64hi(all, u64);
    uint64_t before = 0;
    for (int c = 0; c < rank; ++c) before += cta_sum[attempt][c];
    if (point < before || point - before >= cta_sum[attempt][rank]) return;
    uint64_t want = point - before + 1;  // the first token with which the sum reaches this
    const int part = min(find(part_sum, want), kWarps - 1);
    const int32_t g1 = part_begin(rank * kWarps + part + 1);
    int turn = 0;
#pragma unroll 1
    for (int32_t g = part_begin(rank * kWarps + part) + warp; next < 0; g += kWarps, turn ^= 1) {
      if (g - warp >= g1) {  // (not reached: the part's sum is that of its groups)
        if (warp != 0) return;
        next = p.vocab - 1;
        break;
      }
      const int32_t j0 = g < g1 ? rows.first(g * 32 + lane) : p.vocab;
      uint64_t wt[kV], own = 0;
      float pv[kV], qv[kV];
      unpack<T, kV>(rows.load_p(j0), pv);
      uint4 v = make_uint4(0, 0, 0, 0), x = v;
      if (rows.q) {
        rows.load_q(j0, v, x);
        v = rows.tokens_of_q(j0, v, x);
      }
      unpack<T, kV>(v, qv);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        wt[i] = pv[i] > qv[i] && j0 + i != without ? units_of(pv[i]) - units_of(qv[i]) : 0;
        own += wt[i];
      }
      uint64_t incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t c = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += c;
      }
      if (lane == 31) group_sum[turn][warp] = incl;
      __syncthreads();
      const int at = find(group_sum[turn], want);
      if (at == kWarps) continue;
      if (at != warp) return;
      uint64_t upto = incl - own;
      int k = 0;  // the lane's tokens that do not reach it
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        upto += wt[i];
        k += upto < want ? 1 : 0;
      }
      next = __shfl_sync(kAll, j0 + k, __ffs(__ballot_sync(kAll, incl >= want)) - 1);
    }
  }
  // ---- outputs
  int32_t* out = p.out_tokens + (int64_t)b * (p.max_drafts + 1);
  for (int32_t i = lane; i <= p.max_drafts; i += 32) out[i] = i < a ? tokens[i] : (i == a ? next : -1);
  if (lane == 0) {
    p.num_accepted[b] = a;
    if (p.next_lens) {
      const int64_t c = (int64_t)max(p.context_lens[b], 0) + 1 + a;
      p.next_lens[b] = (int32_t)min(c, (int64_t)0x7FFFFFFF);
    }
  }
}

template <typename T, bool ALIGNED>
cudaError_t launch_a(const VerifyParams& p, cudaStream_t stream) {
  DeviceInfo info;
  cudaError_t e = device_info(&info);
  if (e != cudaSuccess) return e;
  // As many CTAs a request as the GPU holds at once (two an SM), while each warp has
  // a group of tokens or more (one of 131072 tokens alone: 8 CTAs 7.8 us, 16 5.0).
  static std::atomic<uint64_t> known{0};  // devices asked
  static std::atomic<int> at_once[64];    // clusters of 16 each of them holds
  const uint64_t bit = info.device < 64 ? 1ull << info.device : 0;
  if (!(known.load(std::memory_order_acquire) & bit)) {
    int n = 0;
    bool ok = bit != 0;
    if (ok) ok = cudaFuncSetAttribute(verify_kernel<T, ALIGNED>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    if (ok) {
      cudaLaunchConfig_t c = {};
      c.gridDim = dim3(kMaxCluster, 1, 1);
      c.blockDim = dim3(kNT, 1, 1);
      cudaLaunchAttribute a[1];
      a[0].id = cudaLaunchAttributeClusterDimension;
      a[0].val.clusterDim.x = kMaxCluster;
      a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
      c.attrs = a;
      c.numAttrs = 1;
      ok = cudaOccupancyMaxActiveClusters(&n, verify_kernel<T, ALIGNED>, &c) == cudaSuccess;
    }
    if (!ok) {
      n = 0;
      if (bit) cudaGetLastError();  // not the launch's
    }
    if (bit) at_once[info.device].store(n, std::memory_order_relaxed);
    known.fetch_or(bit, std::memory_order_release);
  }
  // Clusters of 16 only where all of them run at once (16 requests, more than did: the last
  // cluster began 5 to 8 us behind the others).
  const int most = bit && p.num_requests <= at_once[info.device].load(std::memory_order_relaxed) ? kMaxCluster : 8;
  int cluster = 1;
  while (cluster < most && (int64_t)p.num_requests * cluster <= info.num_sms &&
         (int64_t)p.vocab * (int)sizeof(T) >= (int64_t)cluster * 2 * kWarps * 512)
    cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.num_requests * cluster), 1, 1);
  cfg.blockDim = dim3(kNT, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T, ALIGNED>, p, cluster);
}

// Aligned rows: all of them, so by addresses and strides alone.  (64 requests x 131071
// tokens, fp32 / bf16: read token by token 23 / 46 us, by pieces put together 22 / 18;
// x 131072 16 / 15.)
template <typename T>
cudaError_t launch_t(const VerifyParams& p, cudaStream_t stream) {
  constexpr int kV = 16 / (int)sizeof(T);
  const uintptr_t bases = reinterpret_cast<uintptr_t>(p.target) | reinterpret_cast<uintptr_t>(p.draft);
  const int64_t strides = p.target_request | p.target_row | p.draft_request | p.draft_row;
  return bases % 16 == 0 && strides % kV == 0 && p.vocab % kV == 0 ? launch_a<T, true>(p, stream)
                                                                   : launch_a<T, false>(p, stream);
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
  if (p.dtype == QSA_PROBS_F32) return launch_t<float>(p, stream);
  return p.dtype == QSA_PROBS_BF16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<__half>(p, stream);
}

}  // namespace qsa
