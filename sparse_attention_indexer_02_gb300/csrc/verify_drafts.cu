// qsa_verify_drafts: which drafted tokens the target accepts, and the token that
// follows them, from given random numbers.
//
// Draft i of a request is accepted while u_i q_i(x_i) < p_i(x_i), p the target's
// probabilities and q the draft's (1 for a certain draft).  At the first refusal
// a the next token is drawn from max(p_a - q_a, 0), after the last acceptance
// from p_n: the smallest j whose cumulative weight exceeds u times the total.
// Accepted so, the tokens are distributed as the target's own samples.
//
// The sums are integers: a probability counts in units of 2^-60 (exactly, from
// 2^-36 up in fp32), so totals and cumulative sums do not depend on the order in
// which the parts are added, and the comparison u * total < cumulative is exact
// too.  A row's weights are summed once, by a cluster of CTAs that each take a
// contiguous share and each warp a contiguous part of it; the totals cross the
// cluster through shared memory, and the one warp whose part holds the drawn
// point reads that part again.
//
// What bounds it: the row of p (and of q) of each request, from HBM, once; for
// few requests the chain of loads ahead of the row (the drafts, their
// probabilities) and the cluster's exchange.
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"
#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace {

constexpr int kNT = 256;
constexpr int kWarps = kNT / 32;
constexpr int kMaxCluster = 8;
constexpr uint32_t kAll = 0xffffffffu;

template <typename T>
__device__ __forceinline__ float as_float(T v);
template <>
__device__ __forceinline__ float as_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float as_float<__half>(__half v) { return __half2float(v); }

// A probability in units of 2^-60, clamped to [0, 1]; NaN counts as 0.
__device__ __forceinline__ uint64_t units_of(float p) { return __float2ull_rn(__saturatef(p) * 0x1p60f); }

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

// kV consecutive probabilities, 16 bytes of them.
template <typename T, int kV>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[kV]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
  for (int i = 0; i < kV; ++i) v[i] = as_float(e[i]);
}

// What a row's tokens weigh: max(p - q, 0), p where nothing was refused.
template <typename T>
struct Row {
  const T* p;
  const T* q;      // null: no draft distribution
  int64_t certain; // the refused certain draft, -1 none

  __device__ __forceinline__ uint64_t weight(float pv, float qv, int64_t j, uint64_t& full) const {
    const uint64_t a = units_of(pv);
    full = a;
    if (q != nullptr) {
      const uint64_t b = units_of(qv);
      return a > b ? a - b : 0;
    }
    // a certain draft has all its distribution's weight: 2^60 units, never below p's
    return j == certain ? 0 : a;
  }
};

template <typename T>
__global__ void __launch_bounds__(kNT) verify_kernel(const VerifyParams p, int cluster) {
  constexpr int kV = 16 / (int)sizeof(T);
  __shared__ uint64_t cta_sum[kMaxCluster][2];  // of every CTA of the cluster: refused weights, p
  __shared__ uint64_t part_sum[kWarps][2];
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
        ok = (double)u[i] * qd < pt;
      }
    }
    const uint32_t refused = __ballot_sync(kAll, i < n && !ok);
    if (refused) {
      a = i0 + __ffs(refused) - 1;
      break;
    }
    if (i0 + 32 >= n) break;
  }

  Row<T> row;
  row.p = target + (int64_t)a * p.target_row;
  row.q = a < n && draft ? draft + (int64_t)a * p.draft_row : nullptr;
  row.certain = a < n && !draft ? tokens[a] : -1;

  // ---- this warp's part of the row: [v0, v1), whole groups of 32 * kV but for the row's end
  constexpr int kGroup = 32 * kV;
  const int64_t groups = (p.vocab + kGroup - 1) / kGroup;
  const int64_t parts = (int64_t)cluster * kWarps, me = (int64_t)rank * kWarps + warp;
  const int64_t each = groups / parts, more = groups - each * parts;
  const int64_t g0 = me * each + min(me, more), g1 = g0 + each + (me < more ? 1 : 0);
  const bool vec = ((reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q)) & 15) == 0;
  // A group's weights: lane l has elements l * kV .. l * kV + kV - 1 of it, in both ways of loading.
  auto group_at = [&](int64_t g, float (&pv)[kV], float (&qv)[kV]) {
    const int64_t j0 = g * kGroup + lane * kV;
    if (vec && j0 + kV <= p.vocab) {
      load_vec(row.p + j0, pv);
      if (row.q) load_vec(row.q + j0, qv);
    } else {
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const bool in = j0 + i < p.vocab;
        pv[i] = in ? as_float(row.p[j0 + i]) : 0.0f;
        qv[i] = in && row.q ? as_float(row.q[j0 + i]) : 0.0f;
      }
    }
  };
  uint64_t left = 0, full = 0;
  constexpr int kAhead = 4;
  for (int64_t g = g0; g < g1; g += kAhead) {
    float pv[kAhead][kV], qv[kAhead][kV];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (g + k < g1) group_at(g + k, pv[k], qv[k]);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (g + k < g1) {
        const int64_t j0 = (g + k) * kGroup + lane * kV;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          uint64_t f;
          left += row.weight(pv[k][i], row.q ? qv[k][i] : 0.0f, j0 + i, f);
          full += f;
        }
      }
  }
  left = warp_sum(left);
  full = warp_sum(full);
  if (lane == 0) {
    part_sum[warp][0] = left;
    part_sum[warp][1] = full;
  }
  __syncthreads();
  // ---- totals to every CTA of the cluster
  uint64_t mine[2] = {0, 0};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    mine[0] += part_sum[w][0];
    mine[1] += part_sum[w][1];
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if ((int)threadIdx.x < 2 * cluster) {
    const int to = (int)threadIdx.x >> 1, which = (int)threadIdx.x & 1;
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(remote)
                 : "r"(ptx::smem_u32(&cta_sum[rank][which])), "r"(to));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote), "l"(mine[which]) : "memory");
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");

  // ---- the drawn point, and the warp whose part holds it
  uint64_t total[2] = {0, 0};
  for (int c = 0; c < cluster; ++c) {
    total[0] += cta_sum[c][0];
    total[1] += cta_sum[c][1];
  }
  const int which = total[0] > 0 ? 0 : 1;  // nothing left of a refused row: p itself
  const uint64_t all = total[which];
  const float uf = u[p.max_drafts];
  // u in units of 2^-64, in [0, 1); point = floor(all * u), and a cumulative sum
  // exceeds all * u exactly when it exceeds that
  const uint64_t u64 = uf > 0.0f ? (uf < 1.0f ? (uint64_t)(uf * 0x1p64f) : ~0ull) : 0ull;
  const uint64_t point = __umul64hi(all, u64);
  uint64_t before = 0;
  for (int c = 0; c < rank; ++c) before += cta_sum[c][which];
  for (int w = 0; w < warp; ++w) before += part_sum[w][which];
  int64_t next = -1;
  if (all == 0) {
    if (me != 0) return;  // no weight at all: no token
  } else {
    if (point < before || point - before >= part_sum[warp][which]) return;
    const uint64_t want = point - before;  // the first j whose sum within this part exceeds it
    uint64_t sum = 0;
    for (int64_t g = g0; g < g1 && next < 0; ++g) {
      float pv[kV], qv[kV];
      group_at(g, pv, qv);
      const int64_t j0 = g * kGroup + lane * kV;
      uint64_t w[kV], own = 0;
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        uint64_t f;
        const uint64_t l = row.weight(pv[i], row.q ? qv[i] : 0.0f, j0 + i, f);
        w[i] = which == 0 ? l : f;
        own += w[i];
      }
      uint64_t incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += v;
      }
      const uint32_t past = __ballot_sync(kAll, sum + incl > want);
      if (past) {
        const int src = __ffs(past) - 1;
        uint64_t s = sum + incl - own;
        int at = kV - 1;
#pragma unroll
        for (int i = kV - 1; i >= 0; --i) {  // from behind: the first that exceeds
          uint64_t upto = s;
#pragma unroll
          for (int k = 0; k <= i; ++k) upto += w[k];
          if (upto > want) at = i;
        }
        next = __shfl_sync(kAll, j0 + at, src);
      }
      sum += __shfl_sync(kAll, incl, 31);
    }
  }
  // ---- outputs
  int32_t* out = p.out_tokens + (int64_t)b * (p.max_drafts + 1);
  for (int32_t i = lane; i <= p.max_drafts; i += 32) out[i] = i < a ? tokens[i] : (i == a ? (int32_t)next : -1);
  if (lane == 0) {
    p.num_accepted[b] = a;
    if (p.next_lens) {
      const int64_t c = (int64_t)max(p.context_lens[b], 0) + 1 + a;
      p.next_lens[b] = (int32_t)min(c, (int64_t)0x7FFFFFFF);
    }
  }
}

template <typename T>
cudaError_t launch_t(const VerifyParams& p, cudaStream_t stream) {
  DeviceInfo info;
  cudaError_t e = device_info(&info);
  if (e != cudaSuccess) return e;
  // As many CTAs a request as fill the GPU twice over, while each has 2048 tokens or more.
  int cluster = 1;
  while (cluster < kMaxCluster && (int64_t)p.num_requests * cluster < 2 * info.num_sms &&
         p.vocab >= (int64_t)cluster * 2 * 2048)
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
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, p, cluster);
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
  if (p.dtype == QSA_PROBS_F32) return launch_t<float>(p, stream);
  return p.dtype == QSA_PROBS_BF16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<__half>(p, stream);
}

}  // namespace qsa
