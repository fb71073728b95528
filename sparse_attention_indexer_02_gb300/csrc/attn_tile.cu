// qsa_paged_attention, tile form: chunks of new tokens, on tcgen05.
//
// The mathematics is the gathered form's (attn_gather.cu): one pass over the
// keys with a running maximum m, sum l and output o per row.  Here 128 query
// rows are one MMA tile - as many whole tokens as fit, each with all query
// heads of the key/value head, so that grouped heads share the key tile and the
// causal edge is as wide as a few tokens only - and a CTA works on two such
// tiles, its streams 0 and 1, against the same key and value tiles of 128 keys:
//
//   S = Q K^T   (128 x 128, fp32 in TMEM; Q and K from shared memory)
//   P = 2^(S * scale * log2 e - m)   in registers, one thread a row
//   O = O + P V (128 x D, fp32 in TMEM; P as 16-bit in TMEM over S, V from
//                shared memory, where its rows are keys: the MN-major operand)
//
// P is rounded to the type the second product takes, by at most 2^-8 or 2^-11 of a
// term; l is the sum of the fp32 values.
//
// TMEM is full: S/P and O of both streams are 2 * 128 + 2 * D columns.
// What bounds a chunk is the tensor core (4 * D flop a row and key): 8192 new
// tokens at 32768, 32 heads of 128, take 2050 to 2120 us alone, 1815 to 1880
// TFLOP/s, 0.95 to 0.99 of the measured bf16 rate, and 2360 to 2520 back to back,
// 1530 to 1630 TFLOP/s, under the power limit (a library product keeps 1733
// there).  The exponentials are half its time.  The two streams exist to keep it busy: the
// softmax of one runs while the MMAs of the other do.  Two tiles on one key
// tile also halve what L2 has to deliver, 64 KB for 2048 cycles of MMA.
//
// m is not the exact running maximum: it is raised only when a row's maximum
// passes it by more than 8 (in units of log2), since any m that keeps the
// exponentials in range gives the same quotient o / l.  P then reaches 2^8 at
// most, and the pass over O that raising m costs (TMEM to registers and back)
// happens a few times a row in all, instead of a few times a tile.
//
// Roles: warp 0 copies (TMA: the pages of a key tile are one box each a 64-element half),
// warp 1 issues the MMAs, warps 4-7 and 8-11 are the softmax and the epilogue
// of stream 0 and 1.  Key and value tiles share one ring of stages.  Keys past
// the last one a tile sees are masked in S; the values there are zeroed in
// shared memory by the MMA warp before it uses them (up to the next multiple of
// 16 keys, the product stops there), so nothing that a page holds past a
// request's end enters a product.  A missing page is loaded from past the pool's
// last page, which the copies fill with zeros, and its keys are masked in S,
// from a word a key tile that the copying warp leaves.
//
// Schedule: equal shares of the (item, 128-key) units (attn_common.cuh).  Items
// that lie in several CTAs leave unnormalised parts; a second, small launch
// joins them, in the CTAs' order and with as many CTAs as there are parts (one
// CTA joining the parts of a long item alone would take longer than the item's
// share).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "attn_common.cuh"
#include "attn_ptx.cuh"

namespace qsa {
namespace attn {
namespace {

// The driver's tensor-map encoder (looked up once), or null.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

constexpr int kNT = 384;
constexpr int kRows = 128;     // query rows a stream
constexpr int kMetaWords = 8;  // of a split item: parts, first row, tokens, first query head
constexpr float kRaise = 8.0f;
constexpr int kItemCost = 1;   // units an item costs beside its tiles (start, epilogue)

template <int D>
struct Geo {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kRows * 2 * D;          // bytes of a 128-row tile
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int q = 0;                          // two tiles
  static constexpr int ring = 2 * kTile;
  static constexpr int bars = ring + kStages * kTile;
  static constexpr int kBars = 2 * kStages + 2 + 2 + 2 + 2 + 1;
  static constexpr int misc = bars + kBars * 8;
  static constexpr int total = 1024 + misc + 16;
  static_assert(total <= 227 * 1024 - 1024, "shared memory (static part aside)");
};

template <int D>
constexpr int64_t part_floats() {  // o as [D / 4][128 rows][4], then (m, l) of each row
  return kRows * (D + 2);
}

__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 64 bytes of an output row, in 32-byte stores when rows are aligned to them
// (a thread writes a row of its own, so a store instruction touches 32 rows,
// and half as many instructions take half the time).
__device__ __forceinline__ void store64(uint8_t* dst, const uint32_t (&e)[16], bool by32) {
  if (by32) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 32 * i), "r"(e[8 * i]),
                   "r"(e[8 * i + 1]), "r"(e[8 * i + 2]), "r"(e[8 * i + 3]), "r"(e[8 * i + 4]), "r"(e[8 * i + 5]),
                   "r"(e[8 * i + 6]), "r"(e[8 * i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(dst + 16 * i) = make_uint4(e[4 * i], e[4 * i + 1], e[4 * i + 2], e[4 * i + 3]);
  }
}

// The products of a tile, issued together by one elected lane of the warp.  The
// MMA warp shares its scheduler with two softmax warps and gets an instruction
// in some ten cycles, so its loop has few: with an election, 64-bit descriptor
// sums and a modulo for each MMA the tensor core idled between them (2048 new
// tokens at 8K: 237 us against 218).
// S = Q K^T: D / 16 k-steps of 32 bytes, four to a 64-element half; then an
// arrival on `s_full`, and on `empty` when `last`.  Descriptors: low words of Q
// and K, and the high word they share.
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                         uint64_t* s_full, uint64_t* empty, bool last) {
  static_assert(kRows * 128 / 16 == 1024, "descriptor offset of a half");
  if constexpr (D == 128)
    asm volatile(
        "{\n .reg .pred e, t, f, q;\n .reg .b64 a, b;\n .reg .b32 la, lb;\n elect.sync _|e, 0xffffffff;\n"
        " setp.eq.u32 t, 0, 0;\n setp.ne.u32 f, 0, 0;\n setp.ne.and.u32 q, %7, 0, e;\n"
        " mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %2};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, f;\n"
        " add.u32 la, %1, 2;\n add.u32 lb, %3, 2;\n mov.b64 a, {la, %2};\n mov.b64 b, {lb, %2};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.u32 la, %1, 4;\n add.u32 lb, %3, 4;\n mov.b64 a, {la, %2};\n mov.b64 b, {lb, %2};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.u32 la, %1, 6;\n add.u32 lb, %3, 6;\n mov.b64 a, {la, %2};\n mov.b64 b, {lb, %2};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.u32 la, %1, 1024;\n add.u32 lb, %3, 1024;\n mov.b64 a, {la, %2};\n mov.b64 b, {lb, %2};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.u32 la, %1, 1026;\n add.u32 lb, %3, 1026;\n mov.b64 a, {la, %2};\n mov.b64 b, {lb, %2};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.u32 la, %1, 1028;\n add.u32 lb, %3, 1028;\n mov.b64 a, {la, %2};\n mov.b64 b, {lb, %2};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.u32 la, %1, 1030;\n add.u32 lb, %3, 1030;\n mov.b64 a, {la, %2};\n mov.b64 b, {lb, %2};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n}\n" ::"r"(d), "r"(a), "r"(hi), "r"(b), "r"(idesc), "r"(ptx::smem_u32(s_full)), "r"(ptx::smem_u32(empty)),
        "r"((uint32_t)last)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred e, t, f, q;\n .reg .b64 a, b;\n .reg .b32 la, lb;\n elect.sync _|e, 0xffffffff;\n"
        " setp.eq.u32 t, 0, 0;\n setp.ne.u32 f, 0, 0;\n setp.ne.and.u32 q, %7, 0, e;\n"
        " mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %2};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, f;\n"
        " add.u32 la, %1, 2;\n add.u32 lb, %3, 2;\n mov.b64 a, {la, %2};\n mov.b64 b, {lb, %2};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.u32 la, %1, 4;\n add.u32 lb, %3, 4;\n mov.b64 a, {la, %2};\n mov.b64 b, {lb, %2};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.u32 la, %1, 6;\n add.u32 lb, %3, 6;\n mov.b64 a, {la, %2};\n mov.b64 b, {lb, %2};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n}\n" ::"r"(d), "r"(a), "r"(hi), "r"(b), "r"(idesc), "r"(ptx::smem_u32(s_full)), "r"(ptx::smem_u32(empty)),
        "r"((uint32_t)last)
        : "memory");
}
// O (+)= P V over 128 keys: 8 k-steps of 8 TMEM columns of P and 16 value rows.
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred e, p, t;\n .reg .b64 b;\n .reg .b32 la, lb;\n elect.sync _|e, 0xffffffff;\n"
      " setp.ne.b32 p, %5, 0;\n setp.eq.u32 t, 0, 0;\n"
      " mov.b32 la, %1;\n mov.b64 b, {%2, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [la], b, %4, p;\n"
      " add.u32 la, %1, 8;\n add.u32 lb, %2, 128;\n mov.b64 b, {lb, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [la], b, %4, t;\n"
      " add.u32 la, %1, 16;\n add.u32 lb, %2, 256;\n mov.b64 b, {lb, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [la], b, %4, t;\n"
      " add.u32 la, %1, 24;\n add.u32 lb, %2, 384;\n mov.b64 b, {lb, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [la], b, %4, t;\n"
      " add.u32 la, %1, 32;\n add.u32 lb, %2, 512;\n mov.b64 b, {lb, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [la], b, %4, t;\n"
      " add.u32 la, %1, 40;\n add.u32 lb, %2, 640;\n mov.b64 b, {lb, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [la], b, %4, t;\n"
      " add.u32 la, %1, 48;\n add.u32 lb, %2, 768;\n mov.b64 b, {lb, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [la], b, %4, t;\n"
      " add.u32 la, %1, 56;\n add.u32 lb, %2, 896;\n mov.b64 b, {lb, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [la], b, %4, t;\n"
      "}\n" ::"r"(d), "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <bool F16, int D, bool WIN>
__global__ void __launch_bounds__(kNT, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const AttnParams p) {
  using G = Geo<D>;
  constexpr int kStages = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ SchedShared sched_sh;
  __shared__ ItemInfo item_sh[2];  // by turns, from the copying warp
  // Missing keys of a key tile, a bit for each 8, from the copying warp, by turns.  Tile T's is
  // written when its key stage is free.  Of five stages that is when the product with tile
  // T - 3's values is done, of eight when the scores of tile T - 4 are, which come after the
  // probabilities of T - 5: the softmax warps have at most five tiles' words to read yet.
  __shared__ volatile uint32_t missing_sh[8];
  uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::bars);
  uint64_t* empty = full + kStages;
  uint64_t* s_full = empty + kStages;   // [2] scores of a stream ready
  uint64_t* p_ready = s_full + 2;       // [2] probabilities stored (and O raised)
  uint64_t* o_done = p_ready + 2;       // [2] an item's last product done
  uint64_t* q_bar = o_done + 2;         // [2] q (and the item's slot) loaded, free
  uint64_t* done = q_bar + 2;           // abort: the MMAs in flight are done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + G::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + G::misc + 4);
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&s_full[i], 1);
      ptx::mbar_init(&p_ready[i], kRows);
      ptx::mbar_init(&o_done[i], 1);
      ptx::mbar_init(&q_bar[i], i == 0 ? 1 : 1 + 2 * kRows / 32);  // free: the MMAs, the softmax warps
    }
    ptx::mbar_init(done, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&q_map);
    ptx::prefetch_tmap(&k_map);
    ptx::prefetch_tmap(&v_map);
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  ptx::tc_fence_before();
  Start at;
  const Schedule s = make_schedule<kNT, WIN>(p, sched_sh, at);  // with a CTA barrier
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tpt = p.tpi / 2;  // tokens a stream
  const int c = (int)blockIdx.x;
  if (threadIdx.x == 0) p.meta[c * kMetaWords] = 0;

  // Registers: 384 threads of 168 at launch, of which the first four warps
  // leave some to the softmax warps (128 * 72 + 256 * 216 is the same sum).
  if (s.u0 < s.u1) {
    if (warp == 0) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      // ------------------------------------------------------------ copies
      const int box = min(p.page_tokens, kUnit);
      uint32_t r = 0, items = 0;
      bool ok = true;
      Walker<WIN> w(p, at, s.u0);
      const Item& it = w.it;
      const bool any = first_part<WIN>(p, s, w.it, [&](Item&) { w.next(); });
      if (!any && lane == 0) {
        item_sh[0].a = -1;
        ptx::mbar_arrive(&q_bar[0]);
      }
      if (any) for (;;) {
        const Part<WIN> part(p, s, it);
        const int ua = part.a, uz = part.z;
        const int nst = it.n > tpt ? 2 : 1;
        if (items > 0) ok = __all_sync(0xffffffffu, wait_phase(&q_bar[1], (items - 1) & 1u, abort_flag, p.fault));
        if (!ok) break;
        if (lane == 0) {
          ItemInfo& o = item_sh[items & 1];
          o.a = ua;
          o.z = uz;
          o.row0 = it.row0;
          o.n = it.n;
          o.pos0 = it.pos0;
          o.keys = it.keys;
          o.head0 = it.hv * p.group;
          o.c0 = first_cta<WIN>(p, s, it);
          o.c1 = last_cta<WIN>(p, s, it);
          o.last = it.s1 >= s.u1;
          o.skip = it.skip;
        }
        ++items;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&q_bar[0], (uint32_t)(nst * G::kHalves * tpt * p.group * 128));
          for (int st = 0; st < nst; ++st)
            for (int h = 0; h < G::kHalves; ++h)
              ptx::tma_load_3d_plain(smem + G::q + st * G::kTile + h * (kRows * 128), &q_map, h * 64,
                                     it.hv * p.group, it.row0 + st * tpt, &q_bar[0]);
        }
        const int32_t* table = p.block_table + (int64_t)it.b * p.table_stride;
        const int32_t low0 = WIN ? window_from(p, it.pos0) : 0;
        // A box between the sinks and the window of every row: zeros are loaded in its place.
        auto unseen = [&](int32_t t) { return WIN && t >= p.sinks && t + box <= low0; };
        auto page_at = [&](int j) -> int32_t {  // the page of the lane's box of key tile j
          const int32_t t = key_at<WIN>(p, j * kUnit + lane * box, it.skip);
          return j < uz && lane * box < kUnit && t < it.keys && !unseen(t) ? table[t / p.page_tokens] : 0;
        };
        int32_t page = page_at(ua);
        for (int j = ua; j < uz && ok; ++j) {
          const int32_t key = key_at<WIN>(p, j * kUnit + lane * box, it.skip);  // the lane's box's first
          const int valid = min(kUnit, it.keys - (WIN ? it.skip : 0) - j * kUnit);
          const int nb = valid > 0 ? (valid + box - 1) / box : 0;
          // past the pool's end the copies write zeros
          const int32_t pg = page == kNoPage || unseen(key) ? p.num_pages
                                                                          : min(max(page, 0), p.num_pages - 1);
          const uint32_t missing = __reduce_or_sync(
              0xffffffffu, page == kNoPage ? ((1u << (box >> 3)) - 1u) << (lane * (box >> 3)) : 0u);
          page = page_at(j + 1);
          const int off = key % p.page_tokens;
          for (int kv = 0; kv < 2 && ok; ++kv, ++r) {
            const int st = r % kStages;
            ok = __all_sync(0xffffffffu, wait_phase(&empty[st], ((r / kStages) & 1u) ^ 1u, abort_flag, p.fault));
            if (!ok) break;
            if (lane == 0) {
              if (kv == 0) missing_sh[(r >> 1) & 7u] = missing;  // r: two stages a tile
              ptx::mbar_arrive_expect_tx(&full[st], (uint32_t)(nb * box * 128 * G::kHalves));
            }
            __syncwarp();
            if (lane < nb)
              for (int h = 0; h < G::kHalves; ++h)
                ptx::tma_load_4d(smem + G::ring + st * G::kTile + h * (kRows * 128) + lane * box * 128,
                                 kv ? &v_map : &k_map, h * 64, off, it.hv, pg, &full[st]);
          }
        }
        if (!ok || it.s1 >= s.u1) break;
        w.next();
      }
      if (*abort_flag) {  // copies in flight land before the CTA ends
        for (uint32_t i = r > kStages ? r - kStages : 0; i < r; ++i) {
          const long long t0 = clock64();
          while (!ptx::mbar_try_wait(&full[i % kStages], (i / kStages) & 1u) && clock64() - t0 < kSpin) {
          }
        }
        if (items > 0) {
          const long long t0 = clock64();
          while (!ptx::mbar_try_wait(&q_bar[0], (items - 1) & 1u) && clock64() - t0 < kSpin) {
          }
        }
      }
    } else if (warp == 1) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      // ------------------------------------------------------------ products
      constexpr uint32_t id_qk = F16 ? ptx::idesc_f16_f32(128, 128) : ptx::idesc_bf16_f32(128, 128);
      constexpr uint32_t id_pv = (F16 ? ptx::idesc_f16_f32(128, D) : ptx::idesc_bf16_f32(128, D)) | ptx::kIdescBMnMajor;
      const uint64_t q_desc = ptx::sw128_desc(ptx::smem_u32(smem + G::q));
      const uint64_t k_desc = ptx::sw128_desc(ptx::smem_u32(smem + G::ring));
      const uint64_t v_desc = ptx::sw128_mn_desc(ptx::smem_u32(smem + G::ring), kRows * 128);
      const uint32_t q_lo = (uint32_t)q_desc, k_lo = (uint32_t)k_desc, qk_hi = (uint32_t)(k_desc >> 32);
      const uint32_t v_lo = (uint32_t)v_desc, v_hi = (uint32_t)(v_desc >> 32);
      constexpr uint32_t kTile16 = G::kTile / 16;  // from tile to tile in a descriptor
      uint32_t stage = 0, phase = 0;               // of the next tile of the ring
      uint32_t items = 0, turn[2] = {0, 0};
      bool ok = true;
      auto wwait = [&](uint64_t* bar, uint32_t parity) {
        const bool there = ptx::mbar_try_wait(bar, parity);
        return __all_sync(0xffffffffu, there) ||
               __all_sync(0xffffffffu, wait_phase(bar, parity, abort_flag, p.fault));
      };
      auto advance = [&]() {
        if (++stage == kStages) stage = 0, phase ^= 1u;
      };
      for (;;) {
        ok = wwait(&q_bar[0], items & 1u);
        const ItemInfo& it = item_sh[items & 1u];
        if (!ok || it.a < 0) break;
        const int ua = it.a, uz = it.z, keys = it.keys, last_item = it.last;
        const int skip = WIN ? it.skip : 0, low0 = WIN ? window_from(p, it.pos0) : 0;
        const int nst = it.n > tpt ? 2 : 1;
        ok = wwait(&full[stage], phase);
        if (!ok) break;
        ++items;
        ptx::tc_fence_after();
        for (int st = 0; st < nst; ++st)
          issue_qk<D>(tmem + st * 128, q_lo + st * kTile16, k_lo + stage * kTile16, qk_hi, id_qk, &s_full[st],
                      &empty[stage], st == nst - 1);
        // After the item's last scores q's place is free: the next item's q, and its first keys
        // and values behind it, are on their way during the last softmax and product (1024 items
        // of one key tile 58 -> 45 us, 8 x 1000 new tokens 100 -> 93; the 8 K chunk at 32 K 2105 ->
        // 2053, 2137 with the release looked for beside the scores of each stream).
        if (ua + 1 >= uz) ptx::mma_commit_elect(&q_bar[1]);
        advance();
        const int release = uz - 2;
#pragma unroll 1
        for (int j = ua; j < uz; ++j) {
          const uint32_t vst = stage;
          ok = wwait(&full[vst], phase);
          if (!ok) break;
          advance();  // to the key tile of j + 1, if there is one
          const bool more = j + 1 < uz;
          const int valid = max(0, min(kUnit, keys - skip - j * kUnit));
          const int steps = (valid + 15) / 16;
          auto zero_rows = [&](int r0, int rows) {
            uint8_t* v = smem + G::ring + vst * G::kTile + r0 * 128;
            for (int i = lane * 16; i < rows * 128; i += 512)
#pragma unroll
              for (int h = 0; h < G::kHalves; ++h)
                *reinterpret_cast<uint4*>(v + h * (kRows * 128) + i) = make_uint4(0, 0, 0, 0);
          };
          bool zeroed = false;
          if (valid & 15) {  // the value rows between the last key and the product's end
            zero_rows(valid, steps * 16 - valid);
            zeroed = true;
          }
          const int dead0 = p.sinks - j * kUnit, dead1 = low0 - skip - j * kUnit;  // windowed: rows no token sees
          if (WIN && max(dead0, 0) < min(dead1, valid)) {
            // those between the sinks and the first row's window, but for the boxes loaded as
            // zeros: from the sinks' end to its box's, and from the window's box to its start
            const int box = min(p.page_tokens, kUnit), end = min(dead1, valid);
            const int s0 = max(dead0, 0), s1 = min((s0 + box - 1) / box * box, end);
            const int w0 = max(end / box * box, s1);
            if (s0 < s1) zero_rows(s0, s1 - s0);
            if (w0 < end) zero_rows(w0, end - w0);
            zeroed = true;
          }
          if (zeroed) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
          }
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            if (st >= nst) break;
            const bool last = st == nst - 1;
            ok = wwait(&p_ready[st], turn[st]);
            if (!ok) break;
            turn[st] ^= 1u;
            ptx::tc_fence_after();
            const uint32_t d_o = tmem + 256 + st * D, a_p = tmem + st * 128, b_v = v_lo + vst * kTile16;
            if (valid == kUnit) {
              issue_pv(d_o, a_p, b_v, v_hi, id_pv, (uint32_t)(j > ua));
            } else {
              for (int ks = 0; ks < steps; ++ks)
                ptx::mma_bf16_ts_elect(d_o, a_p + ks * 8, ((uint64_t)v_hi << 32) | (b_v + ks * (2048 >> 4)), id_pv,
                                       j > ua || ks > 0);
            }
            if (!more) ptx::mma_commit_elect(&o_done[st]);
            if (last) ptx::mma_commit_elect(&empty[vst]);
            if (more) {
              if (st == 0) {
                ok = wwait(&full[stage], phase);
                if (!ok) break;
                ptx::tc_fence_after();
              }
              issue_qk<D>(tmem + st * 128, q_lo + st * kTile16, k_lo + stage * kTile16, qk_hi, id_qk, &s_full[st],
                          &empty[stage], last);
            }
          }
          if (!ok) break;
          if (more) {
            advance();
            if (__builtin_expect(j == release, 0)) ptx::mma_commit_elect(&q_bar[1]);
          }
        }
        if (!ok || last_item) break;
      }
      if (!ok) {
        ptx::mma_commit_elect(done);
        const long long t0 = clock64();
        while (!ptx::mbar_try_wait(done, 0) && clock64() - t0 < kSpin) {
        }
      }
    } else if (warp < 4) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      // ------------------------------------------------------------ softmax and epilogue
      const int st = (warp - 4) >> 2;
      const int row = ((warp & 3) << 5) + lane;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t t_s = tmem + lanes + st * 128, t_o = tmem + lanes + 256 + st * D;
      const float sc = p.scale_log2;
      const uint64_t sc2 = pack_f32x2(sc, sc);
      const float raise = kRaise / sc;  // in units of S
      uint32_t tiles = 0, items = 0;
      uint32_t before = 0;  // key tiles of the CTA's items before this one
      bool ok = true;
      for (uint32_t k = 0;; ++k) {
        ok = __all_sync(0xffffffffu, wait_phase(&q_bar[0], k & 1u, abort_flag, p.fault));
        const ItemInfo& it = item_sh[k & 1u];
        if (!ok || it.a < 0) break;
        // Here now: the last item's slot is free, the next item may be loaded into it.
        if (lane == 0) ptx::mbar_arrive(&q_bar[1]);
        const int ua = it.a, uz = it.z;
        const int n = min(it.n - st * tpt, tpt);  // tokens of this stream
        if (n > 0) {
          const int tk = row / p.group;
          const int32_t lim = min(max(it.pos0 + st * tpt + tk + 1, 0), it.keys);  // keys [0, lim) are seen
          const int32_t low = WIN ? window_from(p, it.pos0 + st * tpt + tk) : 0;  // windowed: [low, lim) and the sinks
          const int32_t skip = WIN ? it.skip : 0;
          // m in units of S.  Rows of no token (the tile's rows past its tokens, whose q is
          // whatever shared memory held) ask for no raise: it would move the warp's other rows.
          const bool live = tk < n && row < tpt * p.group;
          const float above = live ? raise : INFINITY;
          float m = live ? -INFINITY : 0.0f, l = 0.0f;
          for (int j = ua; j < uz; ++j, ++tiles) {
            ok = __all_sync(0xffffffffu, wait_phase(&s_full[st], tiles & 1u, abort_flag, p.fault));
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t missing = missing_sh[(before + (uint32_t)(j - ua)) & 7u];
            uint32_t x[4][32];
            ptx::tmem_ld32(t_s, x[0]);
            ptx::tmem_ld32(t_s + 32, x[1]);
            // Missing pages: masked in TMEM, out of the loop's registers.  (In x, in the block of
            // the edge below: the loop's code grows, 8K new tokens at 32K 5 % slower; here 0 to 2 %.)
            if (__builtin_expect(__any_sync(0xffffffffu, missing != 0), 0)) {
              ptx::tmem_ld_wait();
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                uint32_t y[32];
                ptx::tmem_ld32(t_s + q * 32, y);
                ptx::tmem_ld_wait();
                ptx::tmem_ld_done32(y);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if ((missing >> (q * 4 + i / 8)) & 1u) y[i] = 0xFF800000u;
                ptx::tmem_st32(t_s + q * 32, y);
              }
              ptx::tmem_st_wait();
              ptx::tmem_ld32(t_s, x[0]);
              ptx::tmem_ld32(t_s + 32, x[1]);
            }
            ptx::tmem_ld_wait();
            ptx::tmem_ld_done32(x[0]);
            ptx::tmem_ld_done32(x[1]);
            ptx::tmem_ld32(t_s + 64, x[2]);  // on their way while the first half is worked on
            ptx::tmem_ld32(t_s + 96, x[3]);
            const int seen = lim - skip - j * kUnit;
            // columns [sink, from) are masked
            const int from = WIN ? low - skip - j * kUnit : 0, sink = WIN ? max(p.sinks - j * kUnit, 0) : 0;
            const bool edge = __any_sync(0xffffffffu, seen < kUnit || (WIN && from > sink && sink < kUnit));
            float top[4];
            uint64_t sum[2];
            // The causal edge and the end of the keys: one block, out of the way of the loop,
            // whose instructions then follow one another (masks between its steps cost the
            // whole loop a tenth: 8K new tokens at 32K 2265 us against 2080).
            if (__builtin_expect(edge, 0)) {
              ptx::tmem_ld_wait();
              ptx::tmem_ld_done32(x[2]);
              ptx::tmem_ld_done32(x[3]);
              if constexpr (WIN) {
                // By words of 32 columns, those without an edge left alone (a window's start and
                // the sinks' end or the causal edge seldom meet in one; compared one by one: 1500
                // cycles a tile more than without an edge).
                auto below = [](int n) { return n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1u); };
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const uint32_t vis = below(seen - q * 32) & ~(below(from - q * 32) & ~below(sink - q * 32));
                  if (__any_sync(0xffffffffu, vis != ~0u)) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                      if (!((vis >> i) & 1u)) x[q][i] = 0xFF800000u;
                  }
                }
              } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    if (q * 32 + i >= seen) x[q][i] = 0xFF800000u;
              }
            }
            auto max_of = [&](int q) {
              float t[2] = {__uint_as_float(x[q][0]), __uint_as_float(x[q][1])};
#pragma unroll
              for (int i = 2; i < 30; i += 4) {
                t[0] = max3(t[0], __uint_as_float(x[q][i]), __uint_as_float(x[q][i + 1]));
                t[1] = max3(t[1], __uint_as_float(x[q][i + 2]), __uint_as_float(x[q][i + 3]));
              }
              top[q] = fmaxf(max3(t[0], __uint_as_float(x[q][30]), __uint_as_float(x[q][31])), t[1]);
            };
            // columns 64 h .. 64 h + 63: 2^(x * sc - m * sc), their sum, and as 16-bit pairs into TMEM
            auto probabilities = [&](int h, float neg) {
              const uint64_t neg2 = pack_f32x2(neg, neg);
              uint32_t pk[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const uint32_t* xs = &x[2 * h + (i >> 4)][(2 * i) & 31];
                float a, b;
                unpack_f32x2(fma2(pack_f32x2(__uint_as_float(xs[0]), __uint_as_float(xs[1])), sc2, neg2), a, b);
                a = ex2(a);
                b = ex2(b);
                sum[i & 1] = add2(sum[i & 1], pack_f32x2(a, b));
                pk[i] = pack2<F16>(a, b);
              }
              ptx::tmem_st32(t_s + h * 32, pk);
            };
            // With the m there is, while the maxima are taken along: that m stands unless a
            // row's maximum passes it by more than 8, seldom after an item's first tiles.
            // Then the same code runs once more (not a copy of it: the loop shares the
            // instruction cache with the copy and MMA warps').
            // Windowed, 64-wide heads: an item's first tile has no m yet, so its maxima come first
            // (8 x 1000 tokens, window 128: 106 -> 92 us; of 128-wide heads the code spills, 8 K
            // tokens, window 4096: 359 -> 385).
            const bool probe = WIN && D == 64 && j == ua;
            if (probe) {
              ptx::tmem_ld_wait();
              ptx::tmem_ld_done32(x[2]);
              ptx::tmem_ld_done32(x[3]);
#pragma unroll
              for (int q = 0; q < 4; ++q) max_of(q);
              m = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
            }
            for (bool again = probe;; again = true) {
              const float neg = m == -INFINITY ? 0.0f : -m * sc;
              sum[0] = sum[1] = 0;
              probabilities(0, neg);
              max_of(0);
              max_of(1);
              ptx::tmem_ld_wait();
              ptx::tmem_ld_done32(x[2]);
              ptx::tmem_ld_done32(x[3]);
              probabilities(1, neg);
              max_of(2);
              max_of(3);
              const float tile_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
              if (again ||
                  !__any_sync(0xffffffffu, tile_top > m + above || (m == -INFINITY && tile_top > m)))
                break;
              const float mn = fmaxf(m, tile_top);
              const float f = mn == -INFINITY ? 1.0f : ex2((m - mn) * sc);
              m = mn;
              l *= f;
              if (j > ua) {  // the stream's product before this S is done: O holds it
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                  uint32_t o[32];
                  ptx::tmem_ld32(t_o + q * 32, o);
                  ptx::tmem_ld_wait();
                  ptx::tmem_ld_done32(o);
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  ptx::tmem_st32(t_o + q * 32, o);
                }
              }
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            ptx::mbar_arrive(&p_ready[st]);
            float a, b;
            unpack_f32x2(add2(sum[0], sum[1]), a, b);
            l += a + b;
          }
          if (ok) ok = __all_sync(0xffffffffu, wait_phase(&o_done[st], items & 1u, abort_flag, p.fault));
          ++items;
          if (ok) {
            ptx::tc_fence_after();
            const int c0 = it.c0, c1 = it.c1;
            const int64_t qrow = it.row0 + st * tpt + tk;
            const int head = it.head0 + (row - tk * p.group);
            if (c0 == c1) {
              const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
              uint8_t* dst = p.out + qrow * p.out_token_stride + (int64_t)head * p.out_head_stride;
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                ptx::tmem_ld32(t_o + q * 32, o);
                ptx::tmem_ld_wait();
                ptx::tmem_ld_done32(o);
                uint32_t e[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)  // a row that sees nothing: O is 0 * V, or was never written
                  e[i] = l == 0.0f ? 0u : pack2<F16>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                if (live) store64(dst + q * 64, e, p.out32);
              }
              if (live && p.lse) p.lse[qrow * p.num_q_heads + head] = (m * sc + log2f(l)) * kLn2;
            } else {
              float* dst = p.parts + (((int64_t)c * 2 + (c == c0 ? 1 : 0)) * 2 + st) * part_floats<D>();
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                ptx::tmem_ld32(t_o + q * 32, o);
                ptx::tmem_ld_wait();
                ptx::tmem_ld_done32(o);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  *reinterpret_cast<uint4*>(dst + ((q * 8 + i) * kRows + row) * 4) =
                      l == 0.0f ? make_uint4(0, 0, 0, 0) : make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
              }
              *reinterpret_cast<float2*>(dst + kRows * D + 2 * row) = make_float2(m * sc, l);
              if (c == c0 && st == 0 && row == 0) {
                int32_t* meta = p.meta + c * kMetaWords;
                meta[1] = it.row0;
                meta[2] = it.n;
                meta[3] = it.head0;
                meta[0] = c1 - c0 + 1;
              }
            }
            ptx::tc_fence_before();  // O read before the next item's products (through p_ready)
          }
        }
        before += (uint32_t)(uz - ua);
        if (!ok || it.last) break;
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

// Joins the parts of the items that lie in several CTAs: block (c0, stream, 32
// rows) for the item that begins in CTA c0's share and ends in a later one.  A
// lane is a row and a warp takes every eighth float4 column, so parts are read
// 512 contiguous bytes a warp; four parts' loads are in flight together, joined
// with a running maximum.
template <bool F16, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnParams p) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int c0 = (int)blockIdx.x, st = (int)blockIdx.y;
  const int4 meta = *reinterpret_cast<const int4*>(p.meta + c0 * kMetaWords);
  const int nf = meta.x;
  if (nf == 0) return;
  const int tpt = p.tpi / 2;
  const int n = min(meta.z - st * tpt, tpt);
  const int row = (int)blockIdx.z * 32 + ((int)threadIdx.x & 31), warp = (int)threadIdx.x >> 5;
  const int tk = row / p.group;
  if (tk >= n) return;
  auto part_of = [&](int f) {
    return p.parts + (((int64_t)(c0 + f) * 2 + (f == 0 ? 1 : 0)) * 2 + st) * part_floats<D>();
  };
  constexpr int kPer = D / 32;  // float4 columns a thread
  constexpr int kBatch = 4;
  float M = -INFINITY, L = 0.0f;
  float4 acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = make_float4(0, 0, 0, 0);
  for (int f0 = 0; f0 < nf; f0 += kBatch) {
    float2 e[kBatch];
    float4 v[kBatch][kPer];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      e[b] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[b][i] = make_float4(0, 0, 0, 0);
      if (f0 + b < nf) {
        const float* pf = part_of(f0 + b);
        e[b] = reinterpret_cast<const float2*>(pf + kRows * D)[row];
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[b][i] = reinterpret_cast<const float4*>(pf)[(warp + 8 * i) * kRows + row];
      }
    }
    float m = M;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) m = fmaxf(m, e[b].x);
    const float keep = M == -INFINITY ? 0.0f : ex2(M - m);
    M = m;
    L *= keep;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = make_float4(acc[i].x * keep, acc[i].y * keep, acc[i].z * keep, acc[i].w * keep);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const float w = e[b].x == -INFINITY ? 0.0f : ex2(e[b].x - M);
      L += e[b].y * w;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        acc[i].x = fmaf(v[b][i].x, w, acc[i].x);
        acc[i].y = fmaf(v[b][i].y, w, acc[i].y);
        acc[i].z = fmaf(v[b][i].z, w, acc[i].z);
        acc[i].w = fmaf(v[b][i].w, w, acc[i].w);
      }
    }
  }
  const int64_t qrow = meta.y + st * tpt + tk;
  const int head = meta.w + (row - tk * p.group);
  const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);
  uint8_t* dst = p.out + qrow * p.out_token_stride + (int64_t)head * p.out_head_stride;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    *reinterpret_cast<uint2*>(dst + (warp + 8 * i) * 8) =
        make_uint2(pack2<F16>(acc[i].x * inv, acc[i].y * inv), pack2<F16>(acc[i].z * inv, acc[i].w * inv));
  if (warp == 0 && p.lse) p.lse[qrow * p.num_q_heads + head] = (M + log2f(L)) * kLn2;
}

template <bool F16, int D, bool WIN>
cudaError_t launch_w(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const AttnParams& p, int device,
                     int grid, cudaStream_t stream) {
  auto kern = attn_tile_kernel<F16, D, WIN>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(kern, Geo<D>::total, device, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kNT, 1, 1);
  cfg.dynamicSmemBytes = Geo<D>::total;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, qm, km, vm, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)grid, 2, kRows / 32);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attn_join_kernel<F16, D>, p);
}

template <bool F16, int D>
cudaError_t launch_t(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const AttnParams& p, int device,
                     int grid, cudaStream_t stream) {
  return p.window > 0 ? launch_w<F16, D, true>(qm, km, vm, p, device, grid, stream)
                      : launch_w<F16, D, false>(qm, km, vm, p, device, grid, stream);
}

}  // namespace
}  // namespace attn

using namespace attn;

bool attn_tile_supports(const qsa_attn_desc& d, const char** why) {
  const int pt = d.kv.page_tokens;
  if (d.num_selected > 0) {
    *why = "selected columns take the gathered form";
    return false;
  }
  if (pt % 8 != 0 || !(kUnit % pt == 0 || pt % kUnit == 0)) {
    *why = "page_tokens must be 8, 16, 32, 64 or a multiple of 128";
    return false;
  }
  if (d.num_q_heads / d.kv.num_kv_heads > kRows) {
    *why = "more than 128 query heads a key/value head";
    return false;
  }
  const int64_t s[] = {d.kv.k_page_stride, d.kv.k_token_stride, d.kv.k_head_stride, d.kv.v_page_stride,
                       d.kv.v_token_stride, d.kv.v_head_stride, d.q_token_stride, d.q_head_stride};
  for (int64_t v : s)
    if (v >= (1LL << 40)) {
      *why = "a stride of 2^40 bytes or more";
      return false;
    }
  return true;
}

// The gathered form's counters (not touched here: one workspace serves both
// forms in turn), two parts a CTA of both streams, the joining launch's list.
size_t attn_tile_workspace(int head_dim) {
  return (size_t)kMaxGrid * 4 + (size_t)kMaxGrid * 4 * kRows * (head_dim + 2) * 4 + (size_t)kMaxGrid * kMetaWords * 4;
}

cudaError_t launch_attn_tile(AttnParams p, const qsa_attn_desc& d, uint8_t* workspace, cudaStream_t stream,
                             const char** msg) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) {
    *msg = "cuTensorMapEncodeTiled is unavailable from the driver";
    return cudaErrorInvalidValue;
  }
  DeviceInfo info;
  cudaError_t e = device_info(&info);
  if (e != cudaSuccess) return e;
  const int D = d.kv.head_dim;
  const bool f16 = d.kv.dtype == QSA_HALF_F16;
  p.parts = reinterpret_cast<float*>(workspace + (size_t)kMaxGrid * 4);
  p.meta = reinterpret_cast<int32_t*>(workspace + (size_t)kMaxGrid * 4 + (size_t)kMaxGrid * 4 * kRows * (D + 2) * 4);
  p.splits = 1;
  p.sub = p.group;
  p.hv = d.kv.num_kv_heads;
  const int tpt = kRows / p.group;
  p.tpi = 2 * tpt;
  p.min_shift = 1;
  p.item_cost = kItemCost;
  p.whole_units = 0;
  // sinks and window both begin at a box of the copies (a multiple of its keys)
  p.win_align = p.page_tokens < kUnit ? p.page_tokens : kUnit;
  p.sink_span = (p.sinks + p.win_align - 1) / p.win_align * p.win_align;
  p.out32 = reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && p.out_token_stride % 32 == 0 && p.out_head_stride % 32 == 0;
  const CUtensorMapDataType ty = f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap qm, km, vm;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)d.num_q_heads, (cuuint64_t)d.num_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)d.q_head_stride, (cuuint64_t)d.q_token_stride};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)tpt};
    if (enc(&qm, ty, 3, const_cast<uint8_t*>(p.q), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
      *msg = "q tensor map rejected by the driver";
      return cudaErrorInvalidValue;
    }
  }
  const int box_rows = p.page_tokens < kUnit ? p.page_tokens : kUnit;
  for (int kv = 0; kv < 2; ++kv) {
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)p.page_tokens, (cuuint64_t)d.kv.num_kv_heads,
                                (cuuint64_t)p.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)(kv ? p.v_token_stride : p.k_token_stride),
                                   (cuuint64_t)(kv ? p.v_head_stride : p.k_head_stride),
                                   (cuuint64_t)(kv ? p.v_page_stride : p.k_page_stride)};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1};
    if (enc(kv ? &vm : &km, ty, 4, const_cast<uint8_t*>(kv ? p.v : p.k), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
      *msg = "key/value tensor map rejected by the driver";
      return cudaErrorInvalidValue;
    }
  }
  const int grid = info.num_sms < kMaxGrid ? info.num_sms : kMaxGrid;
  if (D == 128) return f16 ? launch_t<true, 128>(qm, km, vm, p, info.device, grid, stream) : launch_t<false, 128>(qm, km, vm, p, info.device, grid, stream);
  return f16 ? launch_t<true, 64>(qm, km, vm, p, info.device, grid, stream) : launch_t<false, 64>(qm, km, vm, p, info.device, grid, stream);
}

}  // namespace qsa
