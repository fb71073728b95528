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
// query rows do at most 32 flop a byte (9 requests x 4 rows at 64-128K tokens:
// 485 to 501 us, 6.9 to 7.1 TB/s), random 256-byte rows of HBM for selected decode (16 x 8256
// keys: 50 us, of which copies alone are 49), the consumers' chain of steps for
// selected chunks, whose rows come from L2 (512 rows x 2148 keys: 115 us; copies
// alone 81).  So the kernel is a stream first.  Eight consumer warps work on 16
// keys each of a 128-key unit, every one alone, with a ring of kStages 16-key
// stages of its own; producer warps fill the rings, 32 rows at a time: a lane
// works out where its row lies (list entry, token, page: loaded ahead) and the
// warp copies the rows with 16-byte asynchronous copies, half a warp a row, the
// row offsets passed round by shuffles.  Producers run ahead into the next
// items, their q included; consumers meet only to join their parts at the end
// of an item.  (With the copies issued by the consuming warps themselves a slice
// was one chain of copies, products and softmax steps, 2000 cycles and more
// whatever the memory did: 178 us for those 512 selected rows.)
//
// Rows may lie anywhere, so pages of any size, any cache strides and selected
// columns are one path; rows that are not seen are filled with zeros by the
// same instruction (source size 0), so that nothing a cache holds elsewhere can
// enter a product.  Rows are 16 bytes apart more than their length, which keeps
// the matrix loads free of bank conflicts.
//
// The products are mma.sync (m16n8k16): with at most 32 query rows a tcgen05
// tile of 128 rows would be three quarters padding, and the stream leaves the
// tensor cores idle most of the time either way.  The probabilities go from
// the accumulator layout of the first product straight into the operand layout
// of the second, in registers, rounded to the 16-bit type there (by at most
// 2^-8 or 2^-11 of a term; their sum is taken from the fp32 values).
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attn_common.cuh"

namespace qsa {
namespace attn {
namespace {

constexpr int kSlice = 16;       // keys a stage: one k-step of the second product
constexpr float kRaise = 8.0f;
constexpr int kItemCost = 2;     // units an item costs behind those of its keys

constexpr int kConsumers = kUnit / kSlice;  // warps; a slice of each unit each
constexpr int kNC = 32 * kConsumers;
// Two stages, 136 KB of copies in flight on an SM, leave L1 92 KB to land them
// through; three leave it 28 KB (the 9 x 4 rows: 503 us against 620).
constexpr int kStages = 2;

// Producer warps and the register split.  A warp issues one copy instruction
// in about 70 cycles, so four producers move 28 bytes a cycle, below what L2
// delivers: one row tile, whose consumers leave the registers, takes a producer
// for each consumer.  With two tiles a producer serves two consumers.
template <int MT>
struct Conf {
  static constexpr bool kOwn = MT == 1;  // a producer for each consumer
  static constexpr int kProducers = kOwn ? kConsumers : kConsumers / 2;
  static constexpr int kNT = kNC + 32 * kProducers;
};

template <int D, int MT>
struct Layout {
  static constexpr int kRows = 16 * MT;
  static constexpr int kRow = 2 * D + 16;                  // bytes from row to row
  static constexpr int kStage = 2 * kSlice * kRow;         // key rows, then value rows
  static constexpr int kRing = kStages * kStage;           // of a consumer
  static constexpr int kMergeRow = D + 8;                  // floats from row to row of a warp's o (8 rows: all banks)
  static constexpr int kQ = kRows * kRow;
  static constexpr int q = kConsumers * kRing;             // two, by turns
  static constexpr int ml = q + 2 * kQ;                    // [warp][row] of (m, l)
  static constexpr int items = ml + kConsumers * kRows * 8;  // two ItemInfo, by turns
  static constexpr int bars = items + 2 * 48;              // full, empty [warp][stage], q full, q empty [2]
  static constexpr int masks = bars + (2 * kConsumers * kStages + 4) * 8;  // [warp][stage]
  static constexpr int total = masks + kConsumers * kStages * 4;
  static_assert(16 * kMergeRow * 4 <= kStage, "16 rows of a warp's o fit a stage");
  static_assert(total <= 226 * 1024, "shared memory");
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

// 16 bytes to shared memory; zeros, nothing read, when `bytes` is 0.  Through
// L1: past it (.cg) the same copies of random 256-byte rows moved half as much
// again from L2 (5.98 GB for 3.98) and ran at 11.2 TB/s of rows against 15.7.
__device__ __forceinline__ void copy16(uint32_t dst, uint64_t src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrives on `bar` when this thread's copies so far have landed (one of the barrier's expected arrivals).
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copies_drain() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ bool consumers_any(bool mine) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)mine), "n"(kNC)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kNC) : "memory"); }

// An unfinished part: o [kRows][D] floats, then (m, l) of each row.
template <int D, int MT>
constexpr int64_t part_floats() {
  return 16 * MT * (D + 2);
}

// The item of unit u of a selected call: one token row of one virtual head.  A
// row before the first request's, or of none, has no tokens: nothing is written.
__device__ __forceinline__ Item selected_item(const AttnParams& p, int64_t u, int32_t units, int32_t from_b) {
  Item it;
  const int64_t i = u / units;
  const int32_t t = (int32_t)(i / p.hv);
  it.hv = (int32_t)(i - (int64_t)t * p.hv);
  it.s0 = i * units;
  it.s1 = it.s0 + units;
  it.row0 = t;
  it.i0 = 0;
  int lo = from_b, hi = p.num_requests;  // the last request that starts at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.query_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  it.b = lo;
  const Request r = request_of(p, lo);
  it.n = t >= r.first && t < r.first + r.n ? 1 : 0;
  it.pos0 = it.n > 0 ? r.pos0 + (t - r.first) : -1;
  it.keys = min(max(it.pos0 + 1, 0), p.capacity);
  it.skip = 0;
  return it;
}

template <bool F16, int D, int MT, bool SEL, bool WIN>
__global__ void __launch_bounds__(Conf<MT>::kNT, 1) attn_gather_kernel(const AttnParams p) {
  using L = Layout<D, MT>;
  constexpr int kProducers = Conf<MT>::kProducers, kNT = Conf<MT>::kNT;
  constexpr bool kOwn = Conf<MT>::kOwn;
  constexpr int kRows = L::kRows;
  constexpr int kChunks = D / 8;       // 16-byte chunks of a row
  constexpr int kRpi = 32 / kChunks;   // rows a copy instruction of the warp
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ SchedShared sched_sh;
  __shared__ int abort_sh;
  __shared__ int last_sh;
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bars);
  uint64_t* empty = full + kConsumers * kStages;
  uint64_t* q_full = empty + kConsumers * kStages;
  uint64_t* q_empty = q_full + 2;
  volatile uint32_t* masks = reinterpret_cast<uint32_t*>(smem + L::masks);
  float2* ml = reinterpret_cast<float2*>(smem + L::ml);
  static_assert(sizeof(ItemInfo) <= 48, "item slots");
  volatile int* abort_flag = &abort_sh;

  if (tid < kConsumers * kStages) {
    ptx::mbar_init(&full[tid], 33);  // the producer warp's copies, and its lane 0 for the mask
    ptx::mbar_init(&empty[tid], 1);
  } else if (tid >= 32 && tid < 34) {
    ptx::mbar_init(&q_full[tid - 32], 32 * kProducers + 1);
    ptx::mbar_init(&q_empty[tid - 32], kConsumers);
  }
  if (tid == 0) abort_sh = 0;
  ptx::fence_mbar_init();
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();

  // ---- the CTA's share of the units
  const int32_t list_len = SEL ? p.num_selected * p.ratio + p.local_tokens : 0;
  const int32_t sel_end = SEL ? p.num_selected * p.ratio : 0;
  const int32_t sel_units = SEL ? item_units(p, list_len) : 0;
  Schedule s;
  Start at;
  if (SEL) {
    const int64_t rows = min(max(p.query_start[p.num_requests], 0), p.num_tokens);
    s.share_out(rows * p.hv * sel_units, p.min_shift);
    __syncthreads();
  } else {
    s = make_schedule<kNT, WIN>(p, sched_sh, at);
  }
  if (s.u0 >= s.u1) return;
  auto next = [&](Item& it) {
    if (SEL) {
      it = selected_item(p, it.s1, sel_units, it.b);
    } else {
      Walker<WIN> w(p, it);
      w.next();
      it = w.it;
    }
  };
  Item it;
  if (SEL) it = selected_item(p, s.u0, sel_units, 0);
  else it = Walker<WIN>(p, at, s.u0).it;
  if (!first_part<WIN>(p, s, it, next)) return;
  // Registers: 512 threads of 128 at launch, 256 * 72 + 256 * 176 are less; or
  // 384 of 168, of which 128 * 88 + 256 * 208 is the same sum.
  if (warp >= kConsumers) {
    // ------------------------------------------------------------ producers
    if (kOwn) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const int pw = warp - kConsumers;
    const int chunk = lane % kChunks, sub_row = lane / kChunks;
    const int half = lane >> 4;
    constexpr int kStep = kOwn ? 2 : 1;  // units an iteration
    uint32_t n = 0;                      // slices filled, of any of its consumers
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      const Part<WIN> part(p, s, it);
      const int ua = part.a, uz = part.z;
      const int kvh = p.splits == 1 ? it.hv : it.hv / p.splits;
      const int sub0 = (it.hv - kvh * p.splits) * p.sub;
      const int gs = min(p.sub, p.group - sub0), head0 = kvh * p.group + sub0;
      // An iteration copies 32 rows: two units' slices of the warp's consumer, or a
      // unit's slices of its two; a lane stands for place_of(j) in the list of keys.
      auto place_of = [&](int j) -> int32_t {
        return kOwn ? (j + half) * kUnit + pw * kSlice + (lane & 15) : j * kUnit + pw * 32 + lane;
      };
      auto in_share = [&](int j) -> bool { return (kOwn ? j + half : j) < uz; };
      const int32_t* table = p.block_table + (int64_t)it.b * p.table_stride;
      const int32_t* sel = SEL ? p.selected + (int64_t)it.row0 * p.num_selected : nullptr;
      const int32_t local0 = SEL ? it.pos0 + 1 - p.local_tokens : 0;  // first of the last tokens
      const int32_t keys = it.keys, skip = it.skip, low0 = WIN ? window_from(p, it.pos0) : 0;
      auto col_of = [&](int32_t at) -> int32_t { return p.ratio_shift >= 0 ? at >> p.ratio_shift : at / p.ratio; };
      auto entry_of = [&](int j) -> int32_t {  // SEL: the column listed for the place, -1 none
        const int32_t at = place_of(j);
        return in_share(j) && at < sel_end ? sel[col_of(at)] : -1;
      };
      auto token_of = [&](int j, int32_t col) -> int32_t {  // the token of the place, -1 none
        const int32_t at = place_of(j);
        if (!in_share(j)) return -1;
        if (!SEL) {
          const int32_t key = key_at<WIN>(p, at, skip);
          return key < keys && (!WIN || key < p.sinks || key >= low0) ? key : -1;
        }
        int64_t t;
        if (at < sel_end) {
          t = (int64_t)col * p.ratio + (at - col_of(at) * p.ratio);
          if (col < 0 || t >= local0) return -1;
        } else {
          t = (int64_t)local0 + (at - sel_end);
          if (t < 0 || at >= list_len) return -1;
        }
        return t < keys ? (int32_t)t : -1;
      };
      auto page_of = [&](int32_t tok) -> int32_t {
        return tok < 0 ? 0 : table[p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_tokens];
      };
      int32_t tok = token_of(ua, SEL ? entry_of(ua) : 0), page = page_of(tok);
      int32_t col2 = SEL ? entry_of(ua + kStep) : 0;
      // q: rows (token, head) into shared memory, the padding rows zero
      if (k >= 2) ok = __all_sync(0xffffffffu, wait_phase(&q_empty[k & 1], ((k >> 1) & 1u) ^ 1u, abort_flag, p.fault));
      if (!ok) break;
      const int live = it.n * gs;
      for (int i = pw * 32 + lane; i < kRows * kChunks; i += 32 * kProducers) {
        const int r = i / kChunks, c = i - r * kChunks;
        const int tk = r < live ? r / gs : 0, g = r < live ? r - tk * gs : 0;
        copy16(ptx::smem_u32(smem + L::q) + (k & 1) * L::kQ + r * L::kRow + c * 16,
               reinterpret_cast<uint64_t>(p.q) + (uint64_t)((int64_t)(it.row0 + tk) * p.q_token_stride +
                                                            (int64_t)(head0 + g) * p.q_head_stride + c * 16),
               r < live ? 16u : 0u);
      }
      copies_arrive(&q_full[k & 1]);
      if (pw == 0 && lane == 0) {
        ItemInfo* o = reinterpret_cast<ItemInfo*>(smem + L::items + (k & 1) * 48);
        o->a = ua;
        o->z = uz;
        o->gs = gs;
        o->head0 = head0;
        o->row0 = it.row0;
        o->n = it.n;
        o->pos0 = it.pos0;
        o->keys = it.keys;
        o->c0 = first_cta<WIN>(p, s, it);
        o->c1 = last_cta<WIN>(p, s, it);
        o->last = it.s1 >= s.u1;
        o->skip = it.skip;
        ptx::mbar_arrive(&q_full[k & 1]);
      }

      for (int j = ua; j < uz && ok; j += kStep) {
        const uint32_t vm = __ballot_sync(0xffffffffu, tok >= 0 && page != kNoPage);
        const int32_t pg = min(max(page, 0), p.num_pages - 1), tk = max(tok, 0);
        const int32_t off = p.page_shift >= 0 ? tk & (p.page_tokens - 1) : tk % p.page_tokens;
        const int64_t ko = (int64_t)kvh * p.k_head_stride + (int64_t)pg * p.k_page_stride + (int64_t)off * p.k_token_stride;
        const int64_t vo = p.near_rows ? 0 : (int64_t)kvh * p.v_head_stride + (int64_t)pg * p.v_page_stride +
                                                 (int64_t)off * p.v_token_stride;
        tok = token_of(j + kStep, col2);
        page = page_of(tok);
        if (SEL) col2 = entry_of(j + 2 * kStep);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (kOwn && j + h >= uz) break;
          const int cw = kOwn ? pw : 2 * pw + h;
          const uint32_t st = n % kStages;
          if (n >= kStages)
            ok = __all_sync(0xffffffffu, wait_phase(&empty[cw * kStages + st], ((n / kStages) & 1u) ^ 1u, abort_flag,
                                                    p.fault));
          if (!ok) break;
          const uint32_t dst0 = ptx::smem_u32(smem) + cw * L::kRing + st * L::kStage + sub_row * L::kRow + chunk * 16;
          if (p.near_rows) {  // one 32-bit offset a row, in units of 16 bytes, for key and value
            const uint64_t kb = reinterpret_cast<uint64_t>(p.k) + chunk * 16, vb = reinterpret_cast<uint64_t>(p.v) + chunk * 16;
#pragma unroll
            for (int i = 0; i < kSlice / kRpi; ++i) {
              const int row = h * kSlice + i * kRpi + sub_row;
              const uint64_t o = (uint64_t)__shfl_sync(0xffffffffu, (uint32_t)(ko >> 4), row) << 4;
              const uint32_t bytes = (vm >> row) & 1u ? 16u : 0u;
              copy16(dst0 + i * kRpi * L::kRow, kb + o, bytes);
              copy16(dst0 + (kSlice + i * kRpi) * L::kRow, vb + o, bytes);
            }
          } else {
#pragma unroll 1
            for (int i = 0; i < kSlice / kRpi; ++i) {
              const int row = h * kSlice + i * kRpi + sub_row;
              const int64_t k1 = __shfl_sync(0xffffffffu, ko, row), v1 = __shfl_sync(0xffffffffu, vo, row);
              const uint32_t bytes = (vm >> row) & 1u ? 16u : 0u;
              copy16(dst0 + i * kRpi * L::kRow, reinterpret_cast<uint64_t>(p.k) + (uint64_t)(k1 + chunk * 16), bytes);
              copy16(dst0 + (kSlice + i * kRpi) * L::kRow, reinterpret_cast<uint64_t>(p.v) + (uint64_t)(v1 + chunk * 16),
                     bytes);
            }
          }
          copies_arrive(&full[cw * kStages + st]);
          if (lane == 0) {
            masks[cw * kStages + st] = (vm >> (h * kSlice)) & 0xFFFFu;
            ptx::mbar_arrive(&full[cw * kStages + st]);
          }
          if (kOwn || h == 1) ++n;
        }
      }
      if (!ok || it.s1 >= s.u1) break;
      next(it);
    }
    copies_drain();
  } else {
    // ------------------------------------------------------------ consumers
    if (kOwn) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    uint64_t* my_full = full + warp * kStages;
    uint64_t* my_empty = empty + warp * kStages;
    uint8_t* ring = smem + warp * L::kRing;
    uint32_t used = 0;
    bool ok = true;
    for (uint32_t k = 0;; ++k) {
      if (ok) ok = __all_sync(0xffffffffu, wait_phase(&q_full[k & 1], (k >> 1) & 1u, abort_flag, p.fault));
      if (consumers_any(!ok)) break;  // together: the item will not come
      const ItemInfo info = *reinterpret_cast<const ItemInfo*>(smem + L::items + (k & 1) * 48);
      const int gs = info.gs, head0 = info.head0, live = info.n * info.gs;
      const int64_t row0 = info.row0;
      const uint32_t q_addr = ptx::smem_u32(smem + L::q) + (k & 1) * L::kQ + (lane & 15) * L::kRow +
                              (lane >> 4) * 16;  // row, 8-element half
      uint32_t qf[MT == 1 ? D / 16 : 1][4];
      if (MT == 1) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) ldsm4(qf[MT == 1 ? ks : 0], q_addr + ks * 32);
      }
      int32_t lim[MT][2], low[MT][2];  // keys [0, lim) are seen by the thread's rows (windowed: [low, lim) and the sinks)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
        {
          const int32_t pos = info.pos0 + (mt * 16 + h * 8 + (lane >> 2)) / gs;
          lim[mt][h] = min(max(pos + 1, 0), info.keys);
          low[mt][h] = WIN ? window_from(p, pos) : 0;
        }
      const int32_t all_see = min(max(info.pos0 + 1, 0), info.keys);
      const int32_t low_all = WIN ? window_from(p, info.pos0 + info.n - 1) : 0;  // every row's window holds the keys from here

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

      for (int j = info.a; j < info.z; ++j, ++used) {
        const uint32_t st = used % kStages;
        if (ok) ok = __all_sync(0xffffffffu, wait_phase(&my_full[st], (used / kStages) & 1u, abort_flag, p.fault));
        const uint32_t vm = masks[warp * kStages + st];
        if (ok && vm != 0) {
          const uint32_t kb = ptx::smem_u32(ring) + st * L::kStage;
          // two accumulators a key half (even and odd k-steps), for shorter chains
          float x[MT][2][4], y[MT][2][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[mt][e >> 2][e & 3] = y[mt][e >> 2][e & 3] = 0.0f;
          // keys: lanes 0-7 rows 0-7 and 16-23 rows 8-15 of 8-element half 0, the others of half 1
          const uint32_t k_addr = kb + ((lane & 7) + ((lane >> 4) << 3)) * L::kRow + ((lane >> 3) & 1) * 16;
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
                ldsm4(aq, q_addr + mt * 16 * L::kRow + ks * 32);
              }
              mma16816<F16>(MT == 1 && (ks & 1) ? y[mt][0] : x[mt][0], aq, bk[0], bk[1]);
              mma16816<F16>(MT == 1 && (ks & 1) ? y[mt][1] : x[mt][1], aq, bk[2], bk[3]);
            }
          }
          if (MT == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[0][e >> 2][e & 3] += y[0][e >> 2][e & 3];
          }
          const int32_t at0 = j * kUnit + warp * kSlice, key0 = key_at<WIN>(p, at0, info.skip);
          if (vm != 0xFFFFu || (!SEL && key_at<WIN>(p, at0 + kSlice - 1, info.skip) + 1 > all_see) ||
              (WIN && key0 < low_all)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int c = n * 8 + (lane & 3) * 2 + (e & 1);
                  const int32_t key = key_at<WIN>(p, at0 + c, info.skip);
                  const bool seen = ((vm >> c) & 1u) && (SEL || key < lim[mt][e >> 1]) &&
                                    (!WIN || key < p.sinks || key >= low[mt][e >> 1]);
                  if (!seen) x[mt][n][e] = -INFINITY;
                }
          }
          // m is raised when a maximum passes it by more than 8 only: any m that keeps the
          // exponentials in range gives the same quotient, and raising costs a pass over o.
          // So a row's lanes look at their own scores, and find the row's maximum only then.
          float mx[MT][2];
          bool raise = false;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              mx[mt][h] = p.scale_log2 * fmaxf(fmaxf(x[mt][0][2 * h], x[mt][0][2 * h + 1]),
                                               fmaxf(x[mt][1][2 * h], x[mt][1][2 * h + 1]));
              raise = raise || mx[mt][h] > m[mt][h] + kRaise || (m[mt][h] == -INFINITY && mx[mt][h] > -INFINITY);
            }
          if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float t = fmaxf(mx[mt][h], __shfl_xor_sync(0xffffffffu, mx[mt][h], 1));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                const float mn = fmaxf(m[mt][h], t);
                const float f = mn == -INFINITY ? 1.0f : ex2(m[mt][h] - mn);
                m[mt][h] = mn;
                l[mt][h] *= f;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                  o[mt][i][2 * h] *= f;
                  o[mt][i][2 * h + 1] *= f;
                }
              }
          }
          uint32_t pa[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float sub = m[mt][h] == -INFINITY ? 0.0f : -m[mt][h];
              float pr[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) pr[e] = ex2(fmaf(x[mt][e >> 1][2 * h + (e & 1)], p.scale_log2, sub));
              l[mt][h] += (pr[0] + pr[1]) + (pr[2] + pr[3]);
              pa[mt][h] = pack2<F16>(pr[0], pr[1]);
              pa[mt][2 + h] = pack2<F16>(pr[2], pr[3]);
            }
          // values: transposed loads, lanes 0-15 rows 0-15 of columns 0-7, lanes 16-31 of columns
          // 8-15 (all before the softmax, to overlap it: 2 us slower on the selected chunk)
          const uint32_t v_addr = kb + kSlice * L::kRow + (lane & 15) * L::kRow + (lane >> 4) * 16;
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
        // the last slice's stage stays: the warps join in it
        if (j + 1 < info.z && lane == 0) ptx::mbar_arrive(&my_empty[st]);
      }
      if (lane == 0) ptx::mbar_arrive(&q_empty[k & 1]);

      // ---- join the warps: their maxima first, then o, each warp's on the common one, 16 rows at a time
      const uint32_t held = (used + kStages - 1) % kStages;
      const int c = (int)blockIdx.x, c0 = info.c0, c1 = info.c1;
      const bool split = c0 != c1;
      float* part = p.parts + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * part_floats<D, MT>();
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float t = l[mt][h];
          t += __shfl_xor_sync(0xffffffffu, t, 1);
          t += __shfl_xor_sync(0xffffffffu, t, 2);
          if ((lane & 3) == 0) ml[warp * kRows + mt * 16 + h * 8 + (lane >> 2)] = make_float2(m[mt][h], t);
        }
      consumers_sync();
      auto write_out = [&](int r, int d, float M, float Lsum, const auto& acc) {
        const int tk = r / gs, g = r - tk * gs;
        const int64_t row = row0 + tk;
        const float inv = Lsum > 0.0f ? 1.0f / Lsum : (Lsum == 0.0f ? 0.0f : Lsum);
        uint8_t* dst = p.out + row * p.out_token_stride + (int64_t)(head0 + g) * p.out_head_stride + d * 2;
        if constexpr (sizeof(acc) == 16)
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(pack2<F16>(acc[0] * inv, acc[1] * inv), pack2<F16>(acc[2] * inv, acc[3] * inv));
        else
          *reinterpret_cast<uint32_t*>(dst) = pack2<F16>(acc[0] * inv, acc[1] * inv);
        if (d == 0 && p.lse) p.lse[row * p.num_q_heads + head0 + g] = (M + log2f(Lsum)) * kLn2;
      };
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (mt > 0) consumers_sync();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = h * 8 + (lane >> 2);
          float M = m[mt][h];
#pragma unroll
          for (int x = 0; x < kConsumers; ++x) M = fmaxf(M, ml[x * kRows + mt * 16 + r].x);
          const float f = M == -INFINITY ? 0.0f : ex2(m[mt][h] - M);
          float* dst = reinterpret_cast<float*>(ring + held * L::kStage) + r * L::kMergeRow + (lane & 3) * 2;
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2*>(dst + i * 8) = make_float2(o[mt][i][2 * h] * f, o[mt][i][2 * h + 1] * f);
        }
        consumers_sync();
        for (int i = tid; i < 16 * (D / 4); i += kNC) {
          const int rr = i / (D / 4), d = (i - rr * (D / 4)) * 4, r = mt * 16 + rr;
          if (r >= live) continue;
          float M = -INFINITY, Ls = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          float2 e[kConsumers];
#pragma unroll
          for (int x = 0; x < kConsumers; ++x) e[x] = ml[x * kRows + r];
#pragma unroll
          for (int x = 0; x < kConsumers; ++x) M = fmaxf(M, e[x].x);
#pragma unroll
          for (int x = 0; x < kConsumers; ++x) {
            const float4 v = *reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(smem + x * L::kRing + held * L::kStage) + rr * L::kMergeRow + d);
            Ls += e[x].x == -INFINITY ? 0.0f : e[x].y * ex2(e[x].x - M);
            acc[0] += v.x;
            acc[1] += v.y;
            acc[2] += v.z;
            acc[3] += v.w;
          }
          if (!split) {
            write_out(r, d, M, Ls, acc);
          } else {
            __stcg(reinterpret_cast<float4*>(part + r * D + d), make_float4(acc[0], acc[1], acc[2], acc[3]));
            if (d == 0) __stcg(reinterpret_cast<float2*>(part + kRows * D + 2 * r), make_float2(M, Ls));
          }
        }
      }
      if (split) __threadfence();
      consumers_sync();
      if (lane == 0) ptx::mbar_arrive(&my_empty[held]);
      if (split) {
        // ---- join the CTAs: the last one to arrive adds up the parts, in the CTAs' order
        if (tid == 0) {
          const uint32_t n = (uint32_t)(c1 - c0 + 1);
          const uint32_t old = atomicAdd(p.counters + c0, 1u);
          last_sh = old + 1 == n;
          if (old + 1 == n) p.counters[c0] = 0;  // every arrival is in: zero for the next call
          __threadfence();
        }
        consumers_sync();
        if (last_sh) {
          // A warp takes two rows at a time, a lane kPer columns of each; the lanes hold
          // the parts' weights.  Eight parts of both rows are in flight together: the
          // parts of a long request with one key/value head are 600 KB, read by this CTA
          // alone (a thread a column, four parts at a time: 115 us at 30000 keys of one
          // head and 32 rows; so: 50).
          constexpr int kPer = D / 32, kHold = (kMaxGrid + 31) / 32;
          const int n = c1 - c0 + 1;
          auto part_of = [&](int f) {
            return p.parts + ((int64_t)(c0 + f) * 2 + (f == 0 ? 1 : 0)) * part_floats<D, MT>();
          };
          for (int r0 = warp; r0 < live; r0 += 2 * kConsumers) {
            float2 e[2][kHold];
            float M[2] = {-INFINITY, -INFINITY}, Ls[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < kHold; ++k)
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const int f = k * 32 + lane, r = r0 + t * kConsumers;
                e[t][k] = make_float2(-INFINITY, 0.0f);
                if (f < n && r < live)
                  e[t][k] = __ldcg(reinterpret_cast<const float2*>(part_of(f) + kRows * D + 2 * r));
              }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
              for (int k = 0; k < kHold; ++k) M[t] = fmaxf(M[t], e[t][k].x);
#pragma unroll
              for (int o = 16; o >= 1; o >>= 1) M[t] = fmaxf(M[t], __shfl_xor_sync(0xffffffffu, M[t], o));
#pragma unroll
              for (int k = 0; k < kHold; ++k) {
                e[t][k].x = e[t][k].x == -INFINITY ? 0.0f : ex2(e[t][k].x - M[t]);  // the weight now
                Ls[t] += e[t][k].y * e[t][k].x;
              }
#pragma unroll
              for (int o = 16; o >= 1; o >>= 1) Ls[t] += __shfl_xor_sync(0xffffffffu, Ls[t], o);
            }
            float acc[2][kPer] = {};
            const bool two = r0 + kConsumers < live;
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
              for (int f0 = k * 32; f0 < min(n, (k + 1) * 32); f0 += 8) {
                float v[2][8][kPer];
#pragma unroll
                for (int b = 0; b < 8; ++b)
#pragma unroll
                  for (int t = 0; t < 2; ++t) {
                    const bool there = f0 + b < n && (t == 0 || two);
                    const float* src = part_of(there ? f0 + b : 0) + (r0 + (there ? t : 0) * kConsumers) * D + lane * kPer;
                    if constexpr (kPer == 4) {
                      const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
                      v[t][b][0] = x.x, v[t][b][1] = x.y, v[t][b][2] = x.z, v[t][b][3] = x.w;
                    } else {
                      const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
                      v[t][b][0] = x.x, v[t][b][1] = x.y;
                    }
                  }
#pragma unroll
                for (int b = 0; b < 8; ++b)
#pragma unroll
                  for (int t = 0; t < 2; ++t) {
                    const float w = __shfl_sync(0xffffffffu, e[t][k].x, (f0 + b) & 31);
#pragma unroll
                    for (int c2 = 0; c2 < kPer; ++c2)
                      acc[t][c2] = f0 + b < n ? fmaf(v[t][b][c2], w, acc[t][c2]) : acc[t][c2];
                  }
              }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
              if (t == 0 || two) write_out(r0 + t * kConsumers, lane * kPer, M[t], Ls[t], acc[t]);
          }
        }
      }
      if (info.last) break;
    }
  }
}

template <bool F16, int D, int MT, bool SEL, bool WIN>
cudaError_t launch_t(const AttnParams& p, int device, int grid, cudaStream_t stream) {
  auto kern = attn_gather_kernel<F16, D, MT, SEL, WIN>;
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
  auto by_tiles = [&](auto sel, auto win) {
    return mt == 1 ? launch_t<F16, D, 1, sel.value, win.value>(p, device, grid, stream)
                   : launch_t<F16, D, 2, sel.value, win.value>(p, device, grid, stream);
  };
  if (p.num_selected > 0) return by_tiles(std::true_type{}, std::false_type{});
  return p.window > 0 ? by_tiles(std::false_type{}, std::true_type{}) : by_tiles(std::false_type{}, std::false_type{});
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
  p.min_shift = 0;
  p.item_cost = kItemCost;
  p.whole_units = 5;
  p.win_align = 1;
  p.sink_span = p.sinks;
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
