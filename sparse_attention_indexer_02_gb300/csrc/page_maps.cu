// qsa_build_page_maps: a step's block table, slots, positions and visible
// counts from the requests' lengths, in one launch.
//
// Two exclusive sums over the requests (new tokens, new pages) decide where
// everything goes.  Every CTA computes both sums for all requests itself, in
// shared memory, instead of one CTA computing them for the others: the
// lengths are a few KB that sit in L2, and a second launch or a grid-wide
// hand-over would cost more than the scan.  The CTAs then share out the tokens
// and the new pages; a token finds its request by binary search in the sums.
// The tokens' own page lookups never meet a write of the launch: pages a
// request had before come from the table, new ones straight from the free list.
//
// The launch does not let the next kernel in the stream start early: it writes
// the block table and the visible counts, which the scorers load before they
// wait for the kernel ahead of them.  A grid that never releases its dependents
// has completed, its writes visible, when they start.
//
// Bound by latency at every size that occurs (28 bytes a token): the launch, the
// lengths' load, the scan, a search and a page lookup one after the other; 3.8 us
// for 16 requests of a token, 5.3 for 512 requests and 33 K tokens.
#include <cuda_runtime.h>
#include <stdint.h>

#include "qsa_internal.h"
#include "sm100_ptx.cuh"

namespace qsa {
namespace {

constexpr int kNT = 512;

__device__ __forceinline__ int32_t sat31(int64_t v) { return (int32_t)(v < 0x7FFFFFFFLL ? v : 0x7FFFFFFFLL); }

struct Lens {
  int32_t ctx, n;      // tokens held, tokens to come
  int32_t have, need;  // pages before and after, at most max_pages
};

__device__ __forceinline__ Lens lens_of(const PageMapsParams& p, int b) {
  Lens l;
  l.ctx = max(p.context_lens[b], 0);
  l.n = max(p.new_lens[b], 0);
  const int64_t pt = p.page_tokens;
  l.have = (int32_t)min(((int64_t)l.ctx + pt - 1) / pt, (int64_t)p.max_pages);
  l.need = (int32_t)min(((int64_t)sat31((int64_t)l.ctx + l.n) + pt - 1) / pt, (int64_t)p.max_pages);
  return l;
}

// Largest i in [0, n) with a[i] <= v (a non-decreasing, a[0] = 0 <= v).
__device__ __forceinline__ int last_le(const int32_t* a, int n, int32_t v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kNT) page_maps_kernel(const PageMapsParams p) {
  extern __shared__ int32_t sums[];
  __shared__ int64_t warp_n[kNT / 32], warp_pg[kNT / 32];
  const int B = p.num_requests;
  int32_t* start = sums;          // [B + 1] new tokens before request b
  int32_t* first = sums + B + 1;  // [B + 1] new pages before request b
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;

  ptx::grid_dep_wait();  // (and no grid_dep_launch: see above)

  // each thread sums a contiguous run of requests; the runs are then scanned
  const int per = (B + kNT - 1) / kNT;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  int64_t sn = 0, sp = 0;
  for (int b = b0; b < b1; ++b) {
    const Lens l = lens_of(p, b);
    sn += l.n;
    sp += l.need - l.have;
  }
  int64_t in = sn, ip = sp;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, in, o), c = __shfl_up_sync(0xffffffffu, ip, o);
    if (lane >= o) in += a, ip += c;
  }
  if (lane == 31) warp_n[warp] = in, warp_pg[warp] = ip;
  __syncthreads();
  int64_t rn = in - sn, rp = ip - sp;
  for (int w = 0; w < warp; ++w) rn += warp_n[w], rp += warp_pg[w];
  for (int b = b0; b < b1; ++b) {
    const Lens l = lens_of(p, b);
    start[b] = sat31(rn);
    first[b] = sat31(rp);
    rn += l.n;
    rp += l.need - l.have;
  }
  if (tid == kNT - 1) start[B] = sat31(rn), first[B] = sat31(rp);
  __syncthreads();

  const int64_t gtid = (int64_t)blockIdx.x * kNT + tid, gsize = (int64_t)gridDim.x * kNT;
  for (int64_t b = gtid; b <= B; b += gsize) {
    p.query_start[b] = start[b];
    if (b < B) p.seq_lens[b] = sat31((int64_t)max(p.context_lens[b], 0) + max(p.new_lens[b], 0));
  }
  if (gtid == 0 && p.pages_used) *p.pages_used = first[B];

  const int32_t new_pages = first[B];
  for (int64_t i = gtid; i < new_pages; i += gsize) {
    const int b = last_le(first, B, (int32_t)i);
    const Lens l = lens_of(p, b);
    p.block_table[(int64_t)b * p.table_stride + l.have + (i - first[b])] = i < p.num_free ? p.free_pages[i] : -1;
  }

  const int32_t total = start[B];
  for (int64_t t = gtid; t < p.max_tokens; t += gsize) {
    int64_t slot = -1, col = -1;
    int32_t pos = -1, req = -1, vis = 0;
    if (t < total) {
      req = last_le(start, B, (int32_t)t);
      const Lens l = lens_of(p, req);
      const int64_t ps = (int64_t)l.ctx + (t - start[req]);
      pos = sat31(ps);
      const int64_t pg = ps / p.page_tokens;
      const int32_t off = (int32_t)(ps - pg * p.page_tokens);
      int32_t page = -1;
      if (pg < l.have) {
        page = p.block_table[(int64_t)req * p.table_stride + pg];
      } else if (pg < l.need) {
        const int64_t i = first[req] + (pg - l.have);
        if (i < p.num_free) page = p.free_pages[i];
      }
      if (page >= 0) slot = (int64_t)page * p.page_tokens + off;
      const int64_t q = ps / p.ratio;
      const int32_t r = (int32_t)(ps - q * p.ratio);
      vis = sat31(q + ((p.partial_cols || r == p.ratio - 1) ? 1 : 0));
      if (slot >= 0 && r == p.ratio - 1) col = slot / p.ratio;
    }
    p.slots[t] = slot;
    if (p.positions) p.positions[t] = pos;
    if (p.token_request) p.token_request[t] = req;
    if (p.visible_cols) p.visible_cols[t] = vis;
    if (p.column_slots) p.column_slots[t] = col;
  }
}

}  // namespace

cudaError_t launch_page_maps(const PageMapsParams& p, cudaStream_t stream) {
  DeviceInfo info;
  cudaError_t e = device_info(&info);
  if (e != cudaSuccess) return e;
  const size_t smem = (size_t)(p.num_requests + 1) * 8;
  static std::atomic<uint64_t> allowed{0};
  e = allow_smem(page_maps_kernel, (kMaxMapRequests + 1) * 8, info.device, allowed);
  if (e != cudaSuccess) return e;
  const int64_t work = p.max_tokens > p.num_requests + 1 ? p.max_tokens : p.num_requests + 1;
  const int64_t want = (work + kNT - 1) / kNT;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(want < info.num_sms ? want : info.num_sms), 1, 1);
  cfg.blockDim = dim3(kNT, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_maps_kernel, p);
}

}  // namespace qsa
