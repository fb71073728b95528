// qsa_paged_attention, gathered form: few query rows a request, or rows that
// each see their own selected columns.
//
// One pass over the keys with a running maximum and sum.  For row i with
// scores x_j = scale * q_i . k_j (kept in units of log2): m = max x_j,
// l = sum 2^(x_j - m), o = sum 2^(x_j - m) v_j; when m grows, l and o are
// multiplied by 2^(m_old - m_new).  Two such triples (m, l, o) over disjoint
// keys join the same way, so keys can be split freely: over the warps of a CTA
// and over CTAs.
//
// What bounds it is the key/value bytes: HBM for a decode step, whose 16 or 32
// query rows do at most 32 flop a byte, L2 for chunks of selected rows.  So
// the kernel is a stream first: every warp works alone on 16 keys at a time
// (warp w of the CTA's 8 on keys 16 w .. 16 w + 15 of each 128-key unit) with
// a ring of kStages 16-key stages of its own, and no barrier stands between
// the warps until an item ends; even then the next item's first stages are on
// their way.  A stage is filled by 16-byte asynchronous copies, half a warp a
// row, from row addresses that each lane works out for one row and the warp
// passes round by shuffles.  Rows may lie anywhere, so pages of any size, any
// cache strides and selected columns are one path; rows that are not seen are
// filled with zeros by the same instruction (source size 0), so that nothing a
// cache holds elsewhere can enter a product.  Rows are 16 bytes apart more than
// their length, which keeps the matrix loads free of bank conflicts.  192 KB
// of copies in flight on each SM cover the latency.
//
// The products are mma.sync (m16n8k16): with at most 32 query rows a tcgen05
// tile of 128 rows would be three quarters padding, and the stream leaves the
// tensor cores idle most of the time either way.  The probabilities go from
// the accumulator layout of the first product straight into the operand layout
// of the second, in registers, rounded to the 16-bit type there (relative
// 2^-9 or 2^-12 a term; their sum is taken from the fp32 values).
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_common.cuh"

namespace qsa {
namespace attn {
namespace {

constexpr int kSlice = 16;       // keys a stage: one k-step of the second product
constexpr float kRaise = 8.0f;

// One 16-row tile: 12 warps with two stages each (168 registers a thread).  A
// slice is a chain of dependent steps that a warp takes 2000 cycles and more
// for, whatever the memory does, so three warps a scheduler pay more than a
// third stage (MEASURED).  Two tiles hold
// twice the accumulators, 8 warps' worth, and take three stages.
template <int MT>
struct Conf {
  static constexpr int kWarps = MT == 1 ? 12 : 8;
  static constexpr int kStages = MT == 1 ? 2 : 3;
  static constexpr int kNT = 32 * kWarps;
  static constexpr int kUnit = kWarps * kSlice;  // keys a unit of the schedule
};

template <int D, int MT>
struct Geo {
  static constexpr int kRow = 2 * D + 16;                  // bytes from row to row
  static constexpr int kStage = 2 * kSlice * kRow;         // key rows, then value rows
  static constexpr int kWarpBytes = Conf<MT>::kStages * kStage;
  static constexpr int kMergeRow = D + 4;                  // floats from row to row of a warp's o
};

template <int D, int MT>
struct Layout {
  using G = Geo<D, MT>;
  static constexpr int kRows = 16 * MT;
  static constexpr int q = Conf<MT>::kWarps * G::kWarpBytes;
  static constexpr int ml = q + kRows * G::kRow;               // [warp][row] of (m, l)
  static constexpr int total = ml + Conf<MT>::kWarps * kRows * 8;
  static_assert(16 * G::kMergeRow * 4 <= G::kStage, "16 rows of a warp's o fit a stage");
  static_assert(MT < Conf<MT>::kStages, "a stage for the next item while the warps join");
  static_assert(total <= 225 * 1024, "shared memory");
};

// What the warps need of an item, in shared memory.
struct ItemSh {
  int32_t ua, uz;          // its units in this CTA's share
  int32_t row0, n, pos0, keys;
  int32_t gs, head0;       // query heads of the virtual head, the first of them
  int32_t local0;          // SEL: first of the last tokens
  int32_t c0, c1;          // the CTAs it lies in
  int32_t live;            // it exists
  int64_t k_off, v_off;    // of its key/value head in the caches
  const int32_t* table;
  const int32_t* sel;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes to shared memory; zeros, nothing read, when `bytes` is 0.
__device__ __forceinline__ void copy16(uint32_t dst, uint64_t src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until all but the `ahead` youngest groups have landed (0, 1 or 2).
__device__ __forceinline__ void copies_wait(uint32_t ahead) {
  if (ahead >= 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (ahead == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// An unfinished part: o [kRows][D] floats, then (m, l) of each row.
template <int D, int MT>
constexpr int64_t part_floats() {
  return 16 * MT * (D + 2);
}

// The item of unit u of a selected call: one token row of one virtual head.
__device__ __forceinline__ Item selected_item(const AttnParams& p, int64_t u, int32_t units, int32_t from_b) {
  Item it;
  const int64_t i = u / units;
  const int32_t t = (int32_t)(i / p.hv);
  it.hv = (int32_t)(i - (int64_t)t * p.hv);
  it.s0 = i * units;
  it.s1 = it.s0 + units;
  it.row0 = t;
  it.n = 1;
  it.i0 = 0;
  int lo = from_b, hi = p.num_requests;  // the last request that starts at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.query_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  it.b = lo;
  const Request r = request_of(p, lo);
  it.pos0 = t < r.first + r.n ? r.pos0 + (t - r.first) : -1;
  it.keys = min(max(it.pos0 + 1, 0), p.capacity);
  return it;
}

template <bool SEL>
__device__ __forceinline__ void publish(const AttnParams& p, const Schedule& s, const Item& it, ItemSh* o) {
  const int kvh = it.hv / p.splits;
  const int sub0 = (it.hv - kvh * p.splits) * p.sub;
  o->ua = (int)(max(s.u0, it.s0) - it.s0);
  o->uz = (int)(min(s.u1, it.s1) - it.s0);
  o->row0 = it.row0;
  o->n = it.n;
  o->pos0 = it.pos0;
  o->keys = it.keys;
  o->gs = min(p.sub, p.group - sub0);
  o->head0 = kvh * p.group + sub0;
  o->local0 = it.pos0 + 1 - p.local_tokens;
  const int c = (int)blockIdx.x;
  o->c0 = it.s0 >= s.u0 ? c : s.owner(it.s0);
  o->c1 = it.s1 <= s.u1 ? c : s.owner(it.s1 - 1);
  o->live = 1;
  o->k_off = (int64_t)kvh * p.k_head_stride;
  o->v_off = (int64_t)kvh * p.v_head_stride;
  o->table = p.block_table + (int64_t)it.b * p.table_stride;
  o->sel = SEL ? p.selected + (int64_t)it.row0 * p.num_selected : nullptr;
}

template <bool F16, int D, int MT, bool SEL>
__global__ void __launch_bounds__(Conf<MT>::kNT, 1) attn_gather_kernel(const AttnParams p) {
  using G = Geo<D, MT>;
  using L = Layout<D, MT>;
  constexpr int kWarps = Conf<MT>::kWarps, kStages = Conf<MT>::kStages, kNT = Conf<MT>::kNT, kUnit = Conf<MT>::kUnit;
  constexpr int kRows = 16 * MT;
  constexpr int kChunks = D / 8;            // 16-byte chunks of a row
  constexpr int kRpi = 32 / kChunks;        // rows a copy instruction of the warp
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ SchedShared sched_sh;
  __shared__ Item walk_item;                // thread 0's place in the list
  __shared__ ItemSh items[2];               // this item and the next, by turns
  __shared__ uint32_t masks_sh[kWarps][kStages];  // SEL: the rows of a stage that are seen
  __shared__ int last_sh;
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float2* ml = reinterpret_cast<float2*>(smem + L::ml);
  uint8_t* ring = smem + warp * G::kWarpBytes;
  const uint32_t ring_u32 = ptx::smem_u32(ring);

  ptx::grid_dep_wait();
  ptx::grid_dep_launch();

  // ---- the CTA's share of the units
  const int32_t list_len = SEL ? p.num_selected * p.ratio + p.local_tokens : 0;
  const int32_t sel_end = SEL ? p.num_selected * p.ratio : 0;
  const int32_t sel_units = SEL ? units_of(p, list_len) : 0;
  Schedule s;
  if (SEL) {
    const int64_t rows = min(max(p.query_start[p.num_requests], 0), p.num_tokens);
    s.total = rows * p.hv * sel_units;
    const int64_t want = (s.total + p.min_units - 1) / p.min_units;
    s.ge = (int)min((int64_t)gridDim.x, max((int64_t)1, want));
    const int c = (int)blockIdx.x;
    s.u0 = c < s.ge ? s.share(c) : s.total;
    s.u1 = c < s.ge ? s.share(c + 1) : s.total;
  } else {
    s = make_schedule<kNT>(p, sched_sh);
  }
  if (s.u0 >= s.u1) return;
  if (tid == 0) {
    walk_item = SEL ? selected_item(p, s.u0, sel_units, 0) : Walker(p, sched_sh, s.u0).it;
    publish<SEL>(p, s, walk_item, &items[0]);
  }
  __syncthreads();

  // ---- the copy side: (slot, j) is the next slice to copy, slice j of items[slot]
  uint32_t issued = 0, used = 0;  // stages filled and consumed by this warp
  const int r16 = lane & 15;
  int slot = 0, ij = items[0].ua;
  int32_t tok1, page1, col2 = 0;  // its token and page, loaded ahead; SEL: the column after it
  auto col_of = [&](int32_t at) -> int32_t { return p.ratio_shift >= 0 ? at >> p.ratio_shift : at / p.ratio; };
  auto sel_entry = [&](int j) -> int32_t {  // SEL: the column listed for the lane's place, -1 none
    const int32_t at = j * kUnit + warp * kSlice + r16;
    return j < items[slot].uz && at < sel_end ? __ldg(items[slot].sel + col_of(at)) : -1;
  };
  auto token_of = [&](int j, int32_t col) -> int32_t {  // the lane's token, -1 none
    const int32_t at = j * kUnit + warp * kSlice + r16;
    const ItemSh& it = items[slot];
    if (j >= it.uz) return -1;
    if (!SEL) return at < it.keys ? at : -1;
    int64_t t;
    if (at < sel_end) {
      t = (int64_t)col * p.ratio + (at - col_of(at) * p.ratio);
      if (col < 0 || t >= it.local0) return -1;
    } else {
      t = (int64_t)it.local0 + (at - sel_end);
      if (t < 0 || at >= list_len) return -1;
    }
    return t < it.keys ? (int32_t)t : -1;
  };
  auto page_of = [&](int32_t tok) -> int32_t {
    if (tok < 0) return 0;
    return __ldg(items[slot].table + (p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_tokens));
  };
  auto enter = [&]() {  // at the first slice of items[slot]
    ij = items[slot].ua;
    tok1 = token_of(ij, SEL ? sel_entry(ij) : 0);
    page1 = page_of(tok1);
    if (SEL) col2 = sel_entry(ij + 1);
  };
  enter();
  auto issue = [&]() {  // copies the next slice into the next stage
    const uint32_t st = ring_u32 + (issued % kStages) * G::kStage;
    const uint32_t vm = __ballot_sync(0xffffffffu, tok1 >= 0) & 0xFFFFu;
    const int32_t pg = min(max(page1, 0), p.num_pages - 1);
    const int32_t tk = max(tok1, 0);
    const int32_t off = p.page_shift >= 0 ? tk & (p.page_tokens - 1) : tk % p.page_tokens;
    const ItemSh& it = items[slot];
    const int chunk = lane % kChunks;
    const int64_t ko = it.k_off + (int64_t)pg * p.k_page_stride + (int64_t)off * p.k_token_stride;
    if (p.near_rows) {  // one 32-bit offset a row, in units of 16 bytes, for key and value
      const uint32_t o16 = (uint32_t)(ko >> 4);
      const uint8_t *kb = p.k + chunk * 16, *vb = p.v + chunk * 16;
#pragma unroll
      for (int i = 0; i < kSlice / kRpi; ++i) {
        const int row = i * kRpi + lane / kChunks;
        const uint64_t o = (uint64_t)__shfl_sync(0xffffffffu, o16, row) << 4;
        const uint32_t bytes = (vm >> row) & 1u ? 16u : 0u;
        const uint32_t dst = st + row * G::kRow + chunk * 16;
        copy16(dst, reinterpret_cast<uint64_t>(kb) + o, bytes);
        copy16(dst + kSlice * G::kRow, reinterpret_cast<uint64_t>(vb) + o, bytes);
      }
    } else {
      const uint64_t ka = reinterpret_cast<uint64_t>(p.k) + (uint64_t)ko;
      const uint64_t va = reinterpret_cast<uint64_t>(p.v) + (uint64_t)(it.v_off + (int64_t)pg * p.v_page_stride +
                                                                       (int64_t)off * p.v_token_stride);
#pragma unroll 1
      for (int i = 0; i < kSlice / kRpi; ++i) {
        const int row = i * kRpi + lane / kChunks;
        const uint64_t ks = __shfl_sync(0xffffffffu, ka, row), vs = __shfl_sync(0xffffffffu, va, row);
        const uint32_t bytes = (vm >> row) & 1u ? 16u : 0u;
        const uint32_t dst = st + row * G::kRow + chunk * 16;
        copy16(dst, ks + chunk * 16, bytes);
        copy16(dst + kSlice * G::kRow, vs + chunk * 16, bytes);
      }
    }
    copies_commit();
    if (SEL && lane == 0) masks_sh[warp][issued % kStages] = vm;
    ++issued;
    ++ij;
    tok1 = token_of(ij, col2);
    page1 = page_of(tok1);
    if (SEL) col2 = sel_entry(ij + 1);
  };

  // `rem` slices of the current item (slot cur) are not consumed yet.  The next
  // item's may take kStages - MT stages: the warps join in the others.
  auto try_issue = [&](int cur, int rem) -> bool {
    if (issued - used >= kStages) return false;
    if (slot == cur) {
      if (ij < items[cur].uz) {
        issue();
        return true;
      }
      if (!items[cur ^ 1].live) return false;
      slot = cur ^ 1;
      enter();
    }
    if (ij >= items[slot].uz || (int)(issued - used) - rem >= kStages - MT) return false;
    issue();
    return true;
  };

  for (int k = 0;; ++k) {
    const int cur = k & 1;
    const ItemSh& it = items[cur];
    const int ua = it.ua, uz = it.uz, gs = it.gs, head0 = it.head0, row0 = it.row0;
    const int live = it.n * gs;

    // ---- the next item; q: rows (token, head) into shared memory, the padding rows zero
    if (tid == 0) {
      if (walk_item.s1 < s.u1) {
        if (SEL) {
          walk_item = selected_item(p, walk_item.s1, sel_units, walk_item.b);
        } else {
          Walker w(p, walk_item);
          w.next();
          walk_item = w.it;
        }
        publish<SEL>(p, s, walk_item, &items[cur ^ 1]);
      } else {
        items[cur ^ 1].live = 0;
      }
    }
    for (int i = tid; i < kRows * kChunks; i += kNT) {
      const int r = i / kChunks, c = i - r * kChunks;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (r < live) {
        const int tk = r / gs, g = r - tk * gs;
        w = *reinterpret_cast<const uint4*>(p.q + (int64_t)(row0 + tk) * p.q_token_stride +
                                            (int64_t)(head0 + g) * p.q_head_stride + c * 16);
      }
      *reinterpret_cast<uint4*>(smem + L::q + r * G::kRow + c * 16) = w;
    }
    __syncthreads();
    while (try_issue(cur, uz - ua)) {
    }

    uint32_t qf[MT == 1 ? D / 16 : 1][4];
    const uint32_t q_addr =
        ptx::smem_u32(smem + L::q) + (lane & 15) * G::kRow + (lane >> 4) * 16;  // row, 8-element half
    if (MT == 1) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) ldsm4(qf[MT == 1 ? ks : 0], q_addr + ks * 32);
    }
    int32_t lim[MT][2];  // keys [0, lim) are seen by the thread's rows
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        lim[mt][h] = min(max(it.pos0 + 1 + (mt * 16 + h * 8 + (lane >> 2)) / gs, 0), it.keys);
    const int32_t all_see = min(max(it.pos0 + 1, 0), it.keys);

    float o[MT][D / 8][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.0f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.0f;
    }

    for (int j = ua; j < uz; ++j) {
      copies_wait(issued - used - 1);
      __syncwarp();
      const int32_t key0 = j * kUnit + warp * kSlice;
      const uint32_t vm = SEL ? masks_sh[warp][used % kStages] : 0u;
      if (SEL ? vm != 0 : key0 < it.keys) {
        const uint32_t kb = ring_u32 + (used % kStages) * G::kStage;
        float x[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[mt][e >> 2][e & 3] = 0.0f;
        // keys: lanes 0-7 rows 0-7 and 16-23 rows 8-15 of 8-element half 0, the others of half 1
        const uint32_t k_addr = kb + ((lane & 7) + ((lane >> 4) << 3)) * G::kRow + ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t bk[4];
          ldsm4(bk, k_addr + ks * 32);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t aq[4];
            if (MT == 1) {
#pragma unroll
              for (int e = 0; e < 4; ++e) aq[e] = qf[MT == 1 ? ks : 0][e];
            } else {
              ldsm4(aq, q_addr + mt * 16 * G::kRow + ks * 32);
            }
            mma16816<F16>(x[mt][0], aq, bk[0], bk[1]);
            mma16816<F16>(x[mt][1], aq, bk[2], bk[3]);
          }
        }
        if (SEL ? vm != 0xFFFFu : key0 + kSlice > all_see) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int c = n * 8 + (lane & 3) * 2 + (e & 1);
                const bool seen = SEL ? (vm >> c) & 1u : key0 + c < lim[mt][e >> 1];
                if (!seen) x[mt][n][e] = -INFINITY;
              }
        }
        uint32_t pa[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mx = fmaxf(fmaxf(x[mt][0][2 * h], x[mt][0][2 * h + 1]), fmaxf(x[mt][1][2 * h], x[mt][1][2 * h + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx *= p.scale_log2;
            // m is raised when a maximum passes it by more than 8 only: any m that keeps
            // the exponentials in range gives the same quotient, and raising costs a pass over o
            if (__any_sync(0xffffffffu, mx > m[mt][h] + kRaise || (m[mt][h] == -INFINITY && mx > m[mt][h]))) {
              const float mn = fmaxf(m[mt][h], mx);
              const float f = mn == -INFINITY ? 1.0f : ex2(m[mt][h] - mn);
              m[mt][h] = mn;
              l[mt][h] *= f;
#pragma unroll
              for (int i = 0; i < D / 8; ++i) {
                o[mt][i][2 * h] *= f;
                o[mt][i][2 * h + 1] *= f;
              }
            }
            const float sub = m[mt][h] == -INFINITY ? 0.0f : -m[mt][h];
            float pr[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) pr[e] = ex2(fmaf(x[mt][e >> 1][2 * h + (e & 1)], p.scale_log2, sub));
            l[mt][h] += (pr[0] + pr[1]) + (pr[2] + pr[3]);
            pa[mt][h] = pack2<F16>(pr[0], pr[1]);
            pa[mt][2 + h] = pack2<F16>(pr[2], pr[3]);
          }
        }
        // values: transposed loads, lanes 0-15 rows 0-15 of columns 0-7, lanes 16-31 of columns 8-15
        const uint32_t v_addr = kb + kSlice * G::kRow + (lane & 15) * G::kRow + (lane >> 4) * 16;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t bv[4];
          ldsm4t(bv, v_addr + i * 32);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816<F16>(o[mt][2 * i], pa[mt], bv[0], bv[1]);
            mma16816<F16>(o[mt][2 * i + 1], pa[mt], bv[2], bv[3]);
          }
        }
      }
      __syncwarp();
      ++used;
      try_issue(cur, uz - 1 - j);
    }

    // ---- join the warps, in the stages that hold nothing for the next item
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint8_t* stage = ring + ((used + kStages - 1 - mt) % kStages) * G::kStage;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float t = l[mt][h];
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        const int r = h * 8 + (lane >> 2);
        if ((lane & 3) == 0) ml[warp * kRows + mt * 16 + r] = make_float2(m[mt][h], t);
        float* dst = reinterpret_cast<float*>(stage) + r * G::kMergeRow + (lane & 3) * 2;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(dst + i * 8) = make_float2(o[mt][i][2 * h], o[mt][i][2 * h + 1]);
      }
    }
    __syncthreads();

    const int c = (int)blockIdx.x, c0 = it.c0, c1 = it.c1;
    const bool split = c0 != c1;
    float* part = p.parts + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * part_floats<D, MT>();
    auto write_out = [&](int r, int d, float M, float Lsum, const float (&acc)[4]) {
      const int tk = r / gs, g = r - tk * gs;
      const int64_t row = row0 + tk;
      const float inv = Lsum > 0.0f ? 1.0f / Lsum : (Lsum == 0.0f ? 0.0f : Lsum);
      uint2 w = make_uint2(pack2<F16>(acc[0] * inv, acc[1] * inv), pack2<F16>(acc[2] * inv, acc[3] * inv));
      *reinterpret_cast<uint2*>(p.out + row * p.out_token_stride + (int64_t)(head0 + g) * p.out_head_stride + d * 2) = w;
      if (d == 0 && p.lse) p.lse[row * p.num_q_heads + head0 + g] = (M + log2f(Lsum)) * kLn2;
    };
    for (int i = tid; i < kRows * (D / 4); i += kNT) {
      const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
      if (r >= live) continue;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * kRows + r].x);
      float Ls = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 e = ml[w * kRows + r];
        const float f = e.x == -INFINITY ? 0.0f : ex2(e.x - M);
        const float4 v = *reinterpret_cast<const float4*>(
            reinterpret_cast<const float*>(smem + w * G::kWarpBytes +
                                           ((used + kStages - 1 - (r >> 4)) % kStages) * G::kStage) +
            (r & 15) * G::kMergeRow + d);
        Ls += e.y * f;
        acc[0] = fmaf(v.x, f, acc[0]);
        acc[1] = fmaf(v.y, f, acc[1]);
        acc[2] = fmaf(v.z, f, acc[2]);
        acc[3] = fmaf(v.w, f, acc[3]);
      }
      if (!split) {
        write_out(r, d, M, Ls, acc);
      } else {
        __stcg(reinterpret_cast<float4*>(part + r * D + d), make_float4(acc[0], acc[1], acc[2], acc[3]));
        if (d == 0) __stcg(reinterpret_cast<float2*>(part + kRows * D + 2 * r), make_float2(M, Ls));
      }
    }
    if (split) {
      // ---- join the CTAs: the last one to arrive adds up the parts, in the CTAs' order
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const uint32_t n = (uint32_t)(c1 - c0 + 1);
        const uint32_t old = atomicAdd(p.counters + c0, 1u);
        last_sh = old + 1 == n;
        if (old + 1 == n) p.counters[c0] = 0;  // every arrival is in: zero for the next call
        __threadfence();
      }
      __syncthreads();
      if (last_sh) {
        auto part_of = [&](int f) { return p.parts + ((int64_t)f * 2 + (f == c0 ? 1 : 0)) * part_floats<D, MT>(); };
        for (int i = tid; i < live * (D / 4); i += kNT) {
          const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
          float M = -INFINITY;
          for (int f = c0; f <= c1; ++f)
            M = fmaxf(M, __ldcg(reinterpret_cast<const float2*>(part_of(f) + kRows * D + 2 * r)).x);
          float Ls = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
          for (int f = c0; f <= c1; ++f) {
            const float* pf = part_of(f);
            const float2 e = __ldcg(reinterpret_cast<const float2*>(pf + kRows * D + 2 * r));
            const float4 v = __ldcg(reinterpret_cast<const float4*>(pf + r * D + d));
            const float w = e.x == -INFINITY ? 0.0f : ex2(e.x - M);
            Ls += e.y * w;
            acc[0] = fmaf(v.x, w, acc[0]);
            acc[1] = fmaf(v.y, w, acc[1]);
            acc[2] = fmaf(v.z, w, acc[2]);
            acc[3] = fmaf(v.w, w, acc[3]);
          }
          write_out(r, d, M, Ls, acc);
        }
      }
    }
    if (!items[cur ^ 1].live) break;
    __syncthreads();
  }
}

template <bool F16, int D, int MT, bool SEL>
cudaError_t launch_t(const AttnParams& p, int device, int grid, cudaStream_t stream) {
  auto kern = attn_gather_kernel<F16, D, MT, SEL>;
  constexpr int smem = Layout<D, MT>::total;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(kern, smem, device, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(Conf<MT>::kNT, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool F16, int D>
cudaError_t launch_d(const AttnParams& p, int mt, int device, int grid, cudaStream_t stream) {
  if (p.num_selected > 0)
    return mt == 1 ? launch_t<F16, D, 1, true>(p, device, grid, stream) : launch_t<F16, D, 2, true>(p, device, grid, stream);
  return mt == 1 ? launch_t<F16, D, 1, false>(p, device, grid, stream) : launch_t<F16, D, 2, false>(p, device, grid, stream);
}

}  // namespace
}  // namespace attn

using namespace attn;

// Counters first (one a CTA), then two parts a CTA of the larger row count.
size_t attn_gather_workspace(int head_dim) {
  return (size_t)kMaxGrid * 4 + (size_t)kMaxGrid * 2 * kGatherRows * (head_dim + 2) * 4;
}

cudaError_t launch_attn_gather(AttnParams p, const qsa_attn_desc& d, uint8_t* workspace, cudaStream_t stream) {
  DeviceInfo info;
  cudaError_t e = device_info(&info);
  if (e != cudaSuccess) return e;
  p.counters = reinterpret_cast<uint32_t*>(workspace);
  p.parts = reinterpret_cast<float*>(workspace + (size_t)kMaxGrid * 4);
  // query heads beyond what an item's rows hold become further virtual heads
  p.splits = (p.group + kGatherRows - 1) / kGatherRows;
  p.sub = (p.group + p.splits - 1) / p.splits;
  p.hv = d.kv.num_kv_heads * p.splits;
  // One 16-row tile when the expected rows fit it (the bound, else the mean),
  // two otherwise; an item takes as many whole tokens as its rows hold.
  int64_t toks = 1;
  if (p.num_selected == 0)
    toks = d.max_new > 0 ? d.max_new : (d.num_tokens + d.num_requests - 1) / d.num_requests;
  const int mt = toks * p.sub <= 16 ? 1 : 2;
  p.tpi = p.num_selected > 0 ? 1 : 16 * mt / p.sub;
  p.unit = mt == 1 ? Conf<1>::kUnit : Conf<2>::kUnit;
  p.min_units = 1;
  p.ratio_shift = -1;
  for (int sh = 0; sh < 31; ++sh)
    if ((1 << sh) == p.ratio) p.ratio_shift = sh;
  const int64_t span = (int64_t)(d.kv.num_pages - 1) * p.k_page_stride +
                       (int64_t)(d.kv.page_tokens - 1) * p.k_token_stride +
                       (int64_t)(d.kv.num_kv_heads - 1) * p.k_head_stride;
  p.near_rows = p.k_page_stride == p.v_page_stride && p.k_token_stride == p.v_token_stride &&
                p.k_head_stride == p.v_head_stride && span < (1LL << 36);
  const int grid = info.num_sms < kMaxGrid ? info.num_sms : kMaxGrid;
  const bool f16 = d.kv.dtype == QSA_HALF_F16;
  if (d.kv.head_dim == 128) return f16 ? launch_d<true, 128>(p, mt, info.device, grid, stream) : launch_d<false, 128>(p, mt, info.device, grid, stream);
  return f16 ? launch_d<true, 64>(p, mt, info.device, grid, stream) : launch_d<false, 64>(p, mt, info.device, grid, stream);
}

}  // namespace qsa
