// pa_prefill_q8: causal attention of each sequence's new tokens over the
// 8-bit cache (e4m3 codes, one fp32 scale for each block and KV head of K and
// of V), on the 5th-generation tensor cores.
//
// What is computed: pa_prefill's attention with K = kcode ks[block, head] and
// V = vcode vs[block, head].
//
// What bounds it: long chunks by the tensor cores and the exponentials (4 D
// operations and one exponential for each query and key), a few rows per
// sequence by HBM (one byte per cached element).  Both products are 16-bit:
// 8-bit weights would lose keys whose weight is below 2^-17 of the largest,
// which over a long context add up, and an 8-bit query would cost far more
// than the cache's own rounding.  So the codes become fp16 (exact: every
// e4m3 value is one), and everything else follows from there:
//  * Four converter warps turn 64-key code tiles into fp16 tiles in the tensor
//    core's swizzled layout, in shared memory.  Codes are converted without
//    their scales; the tile each query tile works on is converted once per
//    128 query rows, next to 128 x 64 exponentials.
//  * q is put into fp16 times the power of two that takes its row's largest
//    element to [2^14, 2^15): exact for elements above 2^-28 of the largest,
//    and to 2^-39 of it for smaller ones.
//  * ks is one factor per block of keys in the exponent's argument (a max per
//    block, then one product).  vs joins the argument as log2(vs) - E: the
//    exponential gives p vs / 2^E directly, and the row's sum of p is
//    gathered from block sums times 2^E / vs.  So neither scale costs work
//    per element.  E is the exponent of the largest vs so far, to within 2;
//    O is rescaled when it grows, by the same path as for a grown maximum.
//  * Weights are the fp16 values of 2^8 p vs / 2^E, p up to 2^4 (the maximum
//    is followed lazily): below 2^15, normal down to 2^-22 of the largest vs
//    and kept to 2^-33 of it.  Their rounding, 2^-11 of a weight, is what an fp16
//    output's own rounding is and an eighth of a bf16 output's, so no
//    residual is added.
//
// The longest-first work items, the persistent grid, the query tiles of 128
// rows and the barriers' discipline (each counted over the CTA's tiles,
// waited on in order, never two phases ahead) are pa_prefill's (prefill.cu).
// Here one CTA has an SM to itself and an item is a pair of query tiles, which
// share the converted keys and take turns on the tensor cores.  Warps 0..3 and
// 4..7, one query row per thread, load and convert q and run the softmax of
// one tile each; 8..11 convert K and V; 12 takes the items, copies pages
// (contiguous in this layout: one bulk copy each) and stages their scales; 13
// and 14 issue the MMAs, whole warps with an elected thread (a lone thread
// spends about 90 cycles on each).  Half of q's dims sit in tensor memory: at
// 64 keys a tile, reading both operands of S from shared memory bounds it.
// 8 chunks of 512 rows over 26k tokens with 64 query heads: 627 us, against
// 767 with one query tile per CTA and two CTAs per SM, 721 with 128-key tiles.
// A tile pair takes about 2600 cycles of an SM; its MMAs need 1450 and its
// exponentials 1024, the rest is the latency between the steps.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "device_utils.cuh"
#include "e4m3.cuh"
#include "pagedkv.h"
#include "prefill_plan.cuh"
#include "status.h"
#include "tcgen05_ts.cuh"

namespace pagedkv {
namespace {

constexpr int kKeys = 64;        // keys per K/V tile
constexpr int kPair = 2;         // query tiles (128 rows each) per work item
constexpr int kStages = 4;       // fp16 K tiles, and V tiles
constexpr int kRaw = 3;          // tiles of codes in flight, of K and of V
constexpr int kScaleSlots = 16;  // tiles whose scales are staged
// Warps 0..3 and 4..7: softmax of query tile 0 and 1; 8..11 converters; 12
// pages and scales; 13 and 14 MMAs of query tile 0 and 1.
constexpr int kConvWarp = 8, kPageWarp = 12, kMmaWarp = 13;
constexpr int kThreads = 16 * 32;  // whole warpgroups; warp 15 has no work
// Registers: 128 a thread at launch, shared out anew between the warpgroups
// (a softmax thread holds 64 scores; converters that had 48 spilled, 645 us
// instead of 627 for the chunks above).  The sum must not exceed the launch's:
// an increase waits for registers that the others gave up.
constexpr int kLaunchRegs = 128;
constexpr int kSoftmaxRegs = 192, kConvRegs = 56, kIssueRegs = 72;
static_assert(2 * kSoftmaxRegs + kConvRegs + kIssueRegs == 4 * kLaunchRegs,
              "more registers than the block was launched with");
// What the page warp stages for a tile: for each of its blocks ks, the
// exponent log2(vs) - E + kShift and 2^-that; and E, last.
constexpr int kSlotFloats = 16;
// For each of eight items in turn, where NaN codes of V were taken out (see the
// converters).
constexpr int kNanSlots = 8, kNanInts = 8;
// Tensor memory columns, for each query tile: S 64, P 32, the last 64 dims of
// q 32, O head_dim (up to 128).
constexpr int kTmemCols = 512;
constexpr int kColS = 0, kColP = 128, kColQ = 192, kColO = 256;
// fp16 weights stay below 2^15: a maximum may grow by 2^kRescaleLog2 and a
// block's vs exceed 2^E by less than 2^(kVsSlack + 1) before O is rescaled.
constexpr float kRescaleLog2 = 4.f;
constexpr int kVsSlack = 2;
constexpr float kShift = 8.f;    // weights are 2^kShift p vs / 2^E
constexpr int kTileHalf = kKeys * 128;  // 64 keys x 64 dims of fp16

struct PrefillQ8Args {
  void* out;
  const void* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scales;
  const float* v_scales;
  const int2* tiles;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  int32_t* dev_err;
  float scale_log2;
  int num_q_heads;
  int num_kv_heads;
  int max_blocks_per_seq;
  int num_blocks;
  int max_context_len;
  int total_q;
  int out_f32;
  int* counter;
  int num_items;
};

// raw_full[], raw_empty[] (of K, then of V), k_full[], k_empty[], v_full[],
// v_empty[]; for each of the pair q_full, q_empty, s_full, s_free, p_full,
// o_done; half_done, half_read; done; item_full[2], item_empty[2].
constexpr int kNumBars = 4 * kRaw + 4 * kStages + 6 * kPair + 2 + 1 + 4;
constexpr int kItemWords = 8;

template <int D>
struct LayoutQ8 {
  static constexpr int kHalves = D / 64;
  // q's last 64 dims are in tensor memory, those before in shared memory.
  static constexpr int kQTile = (kHalves - 1) * kRows * 128;
  static constexpr int kTile = kHalves * kTileHalf;  // fp16 K or V tile
  static constexpr int kRawTile = kKeys * D;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kPair * kQTile;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffRaw = kOffV + kStages * kTile;
  static constexpr int kOffScales = kOffRaw + 2 * kRaw * kRawTile;
  // maximum, sum and E of each row of query tile 1, for its merge with tile 0
  static constexpr int kOffMerge = kOffScales + kScaleSlots * kSlotFloats * 4;
  // of kNanSlots items in turn: kNanInts ints (see the converters)
  static constexpr int kOffNan = kOffMerge + 3 * kRows * 4;
  static constexpr int kOffBars = kOffNan + kNanSlots * kNanInts * 4;
  static constexpr size_t kSmemBytes =
      1024 + kOffBars + kNumBars * 8 + 16 + 2 * kItemWords * 4;
};
static_assert(LayoutQ8<128>::kSmemBytes <= 232448, "shared memory of an SM");

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

constexpr uint32_t kSuspendNs = 20000;

// A try_wait with a suspend-time hint: a waiting thread sleeps in the barrier
// instead of polling it, which leaves the issue slots to the others.
__device__ __forceinline__ bool try_wait_hint(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kSuspendNs)
      : "memory");
  return ok != 0;
}
// By a whole warp, converged: every branch is uniform (a wait each lane loops
// on by itself costs about 250 cycles even when there is nothing to wait
// for), and so is the result, which collectives follow.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, try_wait_hint(bar, parity))) return true;
  const uint64_t t0 = dev::globaltimer();
  for (;;) {
    if (__all_sync(0xffffffffu, try_wait_hint(bar, parity))) return true;
    if (__any_sync(0xffffffffu,
                   dev::globaltimer() - t0 > dev::kWaitLimitNs))
      return false;
  }
}
constexpr float kTiny = 1.1754944e-38f;  // the smallest normal float

// The larger of the two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 0xff for each byte of w that is a NaN code (0x7f, 0xff), 0 for the others.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  const uint32_t n = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return 2u * n - (n >> 7);
}

// One arrival for a converged warp, without a branch.  (What it publishes is
// ordered by the caller: a warp-wide tcgen05 wait, or __syncwarp.)
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// `bytes` contiguous bytes global -> shared, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src,
                                          uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// kShareKeys: for calls whose items all have at most 128 rows (host rule in
// dispatch_share): the pair of query tiles shares an item's keys (see Span).
template <typename T, int BS, int G, int D, bool kShareKeys>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_q8_kernel(const PrefillQ8Args a) {
  using Lay = LayoutQ8<D>;
  using M = dev::Mma<__half>;
  constexpr int kHalves = Lay::kHalves;
  constexpr int kTok = kRows / G;           // new tokens per query tile
  constexpr int kItemTok = kPair * kTok;    // and per work item
  constexpr int kNB = kKeys / BS;           // blocks (pages) per K/V tile
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem =
      smem_dyn + ((1024u - (dev::smem_u32(smem_dyn) & 1023u)) & 1023u);
  const uint32_t base = dev::smem_u32(smem);
  float* scale_s = reinterpret_cast<float*>(smem + Lay::kOffScales);
  const uint32_t bars = base + Lay::kOffBars;
  const uint32_t raw_full0 = bars;
  const uint32_t raw_empty0 = raw_full0 + 16 * kRaw;
  const uint32_t k_full0 = raw_empty0 + 16 * kRaw;
  const uint32_t k_empty0 = k_full0 + 8 * kStages;
  const uint32_t v_full0 = k_empty0 + 8 * kStages;
  const uint32_t v_empty0 = v_full0 + 8 * kStages;
  // For query tile x of the pair: its q is in place / the item's S MMAs are
  // done with it; S(t) is in tensor memory / in the softmax warps' registers;
  // P(t) is in tensor memory; P(t).V is done (O is current, P's buffer free).
  const uint32_t q_full0 = v_empty0 + 8 * kStages;
  const uint32_t q_empty0 = q_full0 + 8 * kPair;
  const uint32_t s_full0 = q_empty0 + 8 * kPair;
  const uint32_t s_free0 = s_full0 + 8 * kPair;
  const uint32_t p_full0 = s_free0 + 8 * kPair;
  const uint32_t o_done0 = p_full0 + 8 * kPair;
  // An item whose keys the pair shares (below): tile 1's part is complete /
  // has been read.
  const uint32_t half_done = o_done0 + 8 * kPair;
  const uint32_t half_read = half_done + 8;
  const uint32_t done = half_read + 8;
  const uint32_t item_full0 = done + 8;
  const uint32_t item_empty0 = item_full0 + 16;
  uint32_t* tmem_slot =
      reinterpret_cast<uint32_t*>(smem + Lay::kOffBars + kNumBars * 8);
  volatile int* item_s = reinterpret_cast<volatile int*>(tmem_slot + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  dev::pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < 2 * kRaw; ++s) {
      dev::mbar_init(raw_full0 + 8 * s, 1);
      dev::mbar_init(raw_empty0 + 8 * s, 4);
    }
    for (int s = 0; s < kStages; ++s) {
      dev::mbar_init(k_full0 + 8 * s, 4);
      dev::mbar_init(k_empty0 + 8 * s, 2);
      dev::mbar_init(v_full0 + 8 * s, 4);
      dev::mbar_init(v_empty0 + 8 * s, 2);
    }
    for (int x = 0; x < kPair; ++x) {
      dev::mbar_init(q_full0 + 8 * x, 4);
      dev::mbar_init(q_empty0 + 8 * x, 1);
      dev::mbar_init(s_full0 + 8 * x, 1);
      dev::mbar_init(s_free0 + 8 * x, 4);
      dev::mbar_init(p_full0 + 8 * x, 4);
      dev::mbar_init(o_done0 + 8 * x, 1);
    }
    dev::mbar_init(half_done, 4);
    dev::mbar_init(half_read, 4);
    dev::mbar_init(done, 8);
    for (int s = 0; s < 2; ++s) {
      dev::mbar_init(item_full0 + 8 * s, 1);
      dev::mbar_init(item_empty0 + 8 * s, 14);
    }
    dev::fence_mbar_init();
  }
  int* nan_s = reinterpret_cast<int*>(smem + Lay::kOffNan);
  if (tid < kNanSlots) nan_s[kNanInts * tid] = 0;
  if (warp == kMmaWarp) {
    dev::tmem_alloc(dev::smem_u32(tmem_slot), kTmemCols);
    dev::tmem_relinquish();
  }
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  dev::pdl_wait();

  struct Item {
    int state;  // kWork, kSkip (invalid input, flagged) or kEnd
    int b, kvh, qt, L, q0, q_len;
  };
  constexpr int kWork = 0, kSkip = 1, kEnd = 2;
  // What an item computes: for query tile x new tokens tok0[x] .. + n_q[x] - 1
  // over n_tiles[x] tiles of keys; tile 1 has the later tokens, so it sees at
  // least as many.  kv_end: the keys the item sees, in `tiles` tiles.  With
  // kShareKeys (a few draft tokens: no tile 1) an item that sees two key tiles
  // or more has its rows in both query tiles: tile x takes key tiles x, x + 2,
  // ... (stride 2), and tile 0 merges the two.
  struct Span {
    int tok0[kPair], n_q[kPair], n_tiles[kPair], kv_end, tiles, stride;
  };
  auto span_of = [](const Item& it) {
    Span sp;
    sp.kv_end = 0;
#pragma unroll
    for (int x = 0; x < kPair; ++x) {
      sp.tok0[x] = it.qt * kItemTok + x * kTok;
      sp.n_q[x] = max(0, min(kTok, it.q_len - sp.tok0[x]));
      const int end = it.L - it.q_len + sp.tok0[x] + sp.n_q[x];
      sp.n_tiles[x] = sp.n_q[x] > 0 ? (end + kKeys - 1) / kKeys : 0;
      if (sp.n_q[x] > 0) sp.kv_end = end;
    }
    sp.tiles = max(sp.n_tiles[0], sp.n_tiles[1]);
    sp.stride = kShareKeys && sp.tiles >= 2 ? 2 : 1;
    if (sp.stride == 2) {
      sp.tok0[1] = sp.tok0[0];
      sp.n_q[1] = sp.n_q[0];
      sp.n_tiles[0] = (sp.tiles + 1) / 2;
      sp.n_tiles[1] = sp.tiles / 2;
    }
    return sp;
  };
  auto read_item = [&](int n, Item& it) -> bool {
    const int slot = n & 1;
    if (!warp_wait(item_full0 + 8 * slot, (n >> 1) & 1)) return false;
    const volatile int* d = item_s + kItemWords * slot;
    it.state = d[0];
    it.b = d[1];
    it.kvh = d[2];
    it.qt = d[3];
    it.L = d[4];
    it.q0 = d[5];
    it.q_len = d[6];
    return true;
  };
  auto next_item = [&](int n, Item& it) -> bool {
    if (!read_item(n, it)) return false;
    __syncwarp();
    warp_arrive(item_empty0 + 8 * (n & 1));
    return true;
  };

  if (warp >= kPageWarp) regs_dec<kIssueRegs>();
  if (warp == kPageWarp) {
    // ---------------- work items, pages and scales ----------------
    // Lane k looks after page k of a group of 32 / kNB tiles: ids and scales
    // of a group are read a group ahead (read a tile ahead, their latency
    // was every tile's period).
    constexpr int kGroup = 32 / kNB;  // tiles
    uint32_t g = 0;  // K/V tiles of this CTA's earlier items
    bool ok = true;
    // Tile t (counted over the CTA's items) of K (w = 0) or V (w = 1): its
    // pages, lane p's own being `id`.
    auto copy = [&](int w, uint32_t t, const uint8_t* cache, int kvh,
                    int32_t id) -> bool {
      const uint32_t slot = w * kRaw + t % kRaw;
      if (t >= kRaw &&
          !warp_wait(raw_empty0 + 8 * slot, ((t / kRaw) - 1) & 1))
        return false;
      const uint32_t full = raw_full0 + 8 * slot;
      if (lane == 0) dev::mbar_arrive_expect_tx(full, Lay::kRawTile);
      __syncwarp();
      if (lane < kNB)
        bulk_load(base + Lay::kOffRaw + slot * Lay::kRawTile + lane * BS * D,
                  cache + (static_cast<int64_t>(id) * a.num_kv_heads + kvh) *
                              (BS * D),
                  BS * D, full);
      return true;
    };
    for (int n = 0; ok; ++n) {
      int i = 0;
      if (lane == 0) i = atomicAdd(a.counter, 1);
      i = __shfl_sync(0xffffffffu, i, 0);
      Item it{kEnd, 0, 0, 0, 0, 0, 0};
      // Unsigned: each CTA draws once past the last item.
      const int2 e = static_cast<unsigned>(i) <
                             static_cast<unsigned>(a.num_items)
                         ? a.tiles[i / a.num_kv_heads]
                         : make_int2(-1, 0);
      if (e.x >= 0) {
        it.b = e.x;
        it.qt = e.y;
        it.kvh = i % a.num_kv_heads;
        it.L = a.context_lens[it.b];
        it.q0 = a.query_start[it.b];
        it.q_len = a.query_start[it.b + 1] - it.q0;
        const bool bad =
            it.L < 0 || it.L > a.max_blocks_per_seq * BS ||
            it.L > a.max_context_len || it.q_len < 0 || it.q_len > it.L ||
            it.q0 < 0 || it.q0 > a.total_q - it.q_len ||
            it.qt * kItemTok >= it.q_len;
        if (bad && lane == 0) dev::set_error(a.dev_err, PA_ERR_DEVICE_OOB);
        it.state = bad ? kSkip : kWork;
      }
      const int slot = n & 1;
      if (n >= 2 && !warp_wait(item_empty0 + 8 * slot, ((n >> 1) - 1) & 1)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        volatile int* d = item_s + kItemWords * slot;
        d[0] = it.state;
        d[1] = it.b;
        d[2] = it.kvh;
        d[3] = it.qt;
        d[4] = it.L;
        d[5] = it.q0;
        d[6] = it.q_len;
        dev::mbar_arrive(item_full0 + 8 * slot);
      }
      __syncwarp();
      if (it.state == kEnd) break;
      if (it.state == kSkip) continue;
      const Span sp = span_of(it);
      const int kvh = it.kvh;
      const int32_t* row =
          a.block_tables + static_cast<int64_t>(it.b) * a.max_blocks_per_seq;
      const int n_pages = (sp.kv_end + BS - 1) / BS;
      bool bad_id = false;
      // Pages past the sequence are masked; they read its first page (an
      // invalid id page 0) and take scales that change nothing.
      struct Page {
        int32_t id;
        float ks, vs;
      };
      auto fetch_id = [&](int group) -> int32_t {
        const int page = group * 32 + lane;
        const int32_t id = __ldg(row + (page < n_pages ? page : 0));
        const bool bad = id < 0 || id >= a.num_blocks;
        bad_id |= bad;
        return bad ? 0 : id;
      };
      auto fetch = [&](int group, int32_t id) -> Page {
        if (group * 32 + lane >= n_pages) return Page{id, 1.f, 0.f};
        const int64_t at = static_cast<int64_t>(id) * a.num_kv_heads + kvh;
        return Page{id, a.k_scales[at], a.v_scales[at]};
      };
      const int groups = (sp.tiles + kGroup - 1) / kGroup;
      int32_t id2 = fetch_id(0);  // ids of group next + 1
      Page next = fetch(0, id2);
      if (groups > 1) id2 = fetch_id(1);
      Page cur = next;
      float lv = 0.f, top = 0.f;
      int e_ref = 0;       // E
      int32_t v_id = 0;    // the page of the V tile that is next
      for (int t = 0; ok && t <= sp.tiles; ++t) {
        if (t < sp.tiles) {
          const int in = t % kGroup;
          if (in == 0) {
            cur = next;
            const int group = t / kGroup;
            if (group + 1 < groups) next = fetch(group + 1, id2);
            if (group + 2 < groups) id2 = fetch_id(group + 2);
            // -100 keeps E - kShift in exp2_int's range (at the top it is: a
            // float's log2 ends at 128).  A scale of 0: no weight at all.
            lv = cur.vs > 0.f ? fmaxf(log2f(cur.vs), -100.f) : -1000.f;
            top = lv;  // the largest of each tile's pages
#pragma unroll
            for (int m = 1; m < kNB; m <<= 1)
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
          }
          const int from = in * kNB + (lane < kNB ? lane : 0);
          const int32_t id = __shfl_sync(0xffffffffu, cur.id, from);
          // (a NaN scale, of K or of V, makes its block's scores NaN)
          const float ks =
              __shfl_sync(0xffffffffu, cur.ks + 0.f * cur.vs, from);
          const float my_lv = __shfl_sync(0xffffffffu, lv, from);
          const int e_top = static_cast<int>(fmaxf(
              floorf(__shfl_sync(0xffffffffu, top, in * kNB)), -100.f));
          if (t == 0 || e_top > e_ref + kVsSlack) e_ref = e_top;
          // A slot is written again kScaleSlots tiles on.  K tile t is copied
          // at most kRaw tiles ahead of the one being converted, which is at
          // most kStages ahead of the one whose S is next, at most two of a
          // query tile's own ahead of the one in its softmax (four where the
          // pair shares the keys): kRaw + kStages + 4 < kScaleSlots, so the
          // slot's old readers are past it once the copy may start.
          if (g + t >= kRaw &&
              !warp_wait(raw_empty0 + 8 * ((g + t) % kRaw),
                         (((g + t) / kRaw) - 1) & 1)) {
            ok = false;
            break;
          }
          float* to = scale_s + ((g + t) % kScaleSlots) * kSlotFloats;
          if (lane < kNB) {
            const float lvn =
                fmaxf(my_lv - static_cast<float>(e_ref), -96.f) + kShift;
            to[lane] = ks;
            to[kNB + lane] = lvn;
            to[2 * kNB + lane] = exp2f(-lvn);
          }
          if (lane == 0) to[kSlotFloats - 1] = static_cast<float>(e_ref);
          __syncwarp();  // before lane 0's arrival publishes them
          ok = copy(0, g + t, a.k_cache, kvh, id);
          if (ok && t >= 1) ok = copy(1, g + t - 1, a.v_cache, kvh, v_id);
          v_id = id;
        } else {
          ok = copy(1, g + t - 1, a.v_cache, kvh, v_id);
        }
      }
      if (bad_id) dev::set_error(a.dev_err, PA_ERR_DEVICE_OOB);
      g += sp.tiles;
    }
    if (!ok && lane == 0) dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
    return;
  }

  if (warp >= kMmaWarp + kPair) return;
  if (warp >= kMmaWarp) {
    // ---------------- MMA issuers, one per query tile ----------------
    // The whole warp runs this, with uniform values; one thread issues.
    {
      const int x = __shfl_sync(0xffffffffu, warp - kMmaWarp, 0);
      const uint32_t tbase = __shfl_sync(0xffffffffu, *tmem_slot, 0);
      bool ok = true;
      constexpr uint32_t idesc_qk =
          dev::umma_idesc_f16(false, kRows, kKeys, false, false);
      constexpr uint32_t idesc_pv =
          dev::umma_idesc_f16(false, kRows, D, false, true);
      const uint32_t s_tmem = tbase + kColS + x * 64;
      const uint32_t p_tmem = tbase + kColP + x * 32;
      const uint32_t qt_tmem = tbase + kColQ + x * 32;
      const uint32_t o_tmem = tbase + kColO + x * 128;
      const uint32_t s_full = s_full0 + 8 * x, s_free = s_free0 + 8 * x;
      const uint32_t p_full = p_full0 + 8 * x, o_done = o_done0 + 8 * x;
      // Descriptors differ from these by an offset in their address field
      // (16-byte units): one addition each.
      const uint64_t qd =
          dev::sw128_desc(base + Lay::kOffQ + x * Lay::kQTile, 16, 1024);
      const uint64_t kd = dev::sw128_desc(base + Lay::kOffK, 16, 1024);
      const uint64_t vd = dev::sw128_desc(base + Lay::kOffV, kTileHalf, 1024);
      uint32_t g = 0;   // K/V tiles of this CTA's earlier items
      uint32_t ts = 0;  // S tiles issued (query tile x)
      uint32_t ps = 0;  // and P.V
      int v = 0;        // items
      // S(t) = Q K(t)^T: the dims whose q is in tensor memory need no read of
      // the A operand from shared memory, which at 64 keys a tile is what
      // bounds the other form.
      auto issue_s = [&](uint32_t t, bool last) -> bool {
        const uint32_t s = t % kStages;
        if (!warp_wait(k_full0 + 8 * s, (t / kStages) & 1) ||
            (ts >= 1 && !warp_wait(s_free, (ts - 1) & 1)))
          return false;
        dev::tc_fence_after();
        const uint64_t k = kd + s * (Lay::kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int h = kk >> 2, k4 = kk & 3;
          const uint64_t kb = k + ((h * kTileHalf + k4 * 32) >> 4);
          if (h + 1 < kHalves)
            dev::umma_f16_warp(s_tmem, qd + ((h * kRows * 128 + k4 * 32) >> 4), kb,
                          idesc_qk, kk > 0 ? 1u : 0u);
          else
            dev::umma_f16_ts_warp(s_tmem, qt_tmem + k4 * 8, kb, idesc_qk,
                             kk > 0 ? 1u : 0u);
        }
        dev::umma_commit_warp(s_full);
        dev::umma_commit_warp(k_empty0 + 8 * s);
        if (last) dev::umma_commit_warp(q_empty0 + 8 * x);
        ++ts;
        return true;
      };
      // O (+)= P(t) V(t); p: P's phase.
      auto issue_pv = [&](uint32_t t, uint32_t p, bool first) -> bool {
        const uint32_t s = t % kStages;
        if (!warp_wait(v_full0 + 8 * s, (t / kStages) & 1) ||
            !warp_wait(p_full, p & 1))
          return false;
        dev::tc_fence_after();
        const uint64_t vb = vd + s * (Lay::kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          dev::umma_f16_ts_warp(o_tmem, p_tmem + kk * 8, vb + kk * (2048 >> 4),
                           idesc_pv, (!first || kk > 0) ? 1u : 0u);
        dev::umma_commit_warp(o_done);
        dev::umma_commit_warp(v_empty0 + 8 * s);
        return true;
      };
      // A tile this query tile does not see (the other one does): only its
      // share of the release, once the tile's phase has begun.
      auto skip = [&](uint32_t t, uint32_t full0, uint32_t empty0) -> bool {
        const uint32_t s = t % kStages;
        if (!warp_wait(full0 + 8 * s, (t / kStages) & 1)) return false;
        warp_arrive(empty0 + 8 * s);
        return true;
      };
      for (int n = 0; ok; ++n) {
        Item it;
        ok = next_item(n, it);
        if (!ok || it.state == kEnd) break;
        if (it.state == kSkip) continue;
        const Span sp = span_of(it);
        const int nt =
            __shfl_sync(0xffffffffu, x ? sp.n_tiles[1] : sp.n_tiles[0], 0);
        const int tiles = __shfl_sync(0xffffffffu, sp.tiles, 0);
        const int stride = __shfl_sync(0xffffffffu, sp.stride, 0);
        const int first = stride == 2 ? x : 0;
        int kt = 0, vt = 0;  // K and V tiles of the item released so far
        // S of this query tile's j-th key tile, past the tiles between.
        auto s_of = [&](int j) -> bool {
          for (const int t = first + j * stride; kt < t; ++kt)
            if (!skip(g + kt, k_full0, k_empty0)) return false;
          return issue_s(g + kt++, j + 1 == nt);
        };
        auto pv_of = [&](int j) -> bool {
          for (const int t = first + j * stride; vt < t; ++vt)
            if (!skip(g + vt, v_full0, v_empty0)) return false;
          return issue_pv(g + vt++, ps++, j == 0);
        };
        if (nt > 0) {
          ok = warp_wait(q_full0 + 8 * x, v & 1) && s_of(0);
          ++v;
        }
        // S(j+1) goes ahead of P(j).V, which waits for the softmax.
        for (int j = 0; ok && j < nt; ++j)
          ok = (j + 1 >= nt || s_of(j + 1)) && pv_of(j);
        // Tiles past its last one, K a tile ahead of V as they are converted.
        while (ok && vt < tiles) {
          if (kt < tiles && kt <= vt + 1)
            ok = skip(g + kt++, k_full0, k_empty0);
          else
            ok = skip(g + vt++, v_full0, v_empty0);
        }
        g += tiles;
      }
      // Tensor memory is released once the softmax warps are done with it;
      // they have then seen their last P.V complete.
      if (!warp_wait(done, 0)) ok = false;
      if (!ok && lane == 0)
        dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
    }
    __syncwarp();
    dev::tc_fence_after();
    if (warp == kMmaWarp) dev::tmem_dealloc(tbase, kTmemCols);
    return;
  }

  if (warp >= kConvWarp) {
    // ---------------- converters: codes -> fp16 tiles ----------------
    regs_dec<kConvRegs>();
    const int ctid = tid - kConvWarp * 32;
    // This thread's 16-code chunks: chunk cc of a 64-dim half, in rows row0,
    // row0 + 32, ...; each becomes two 16-byte chunks of fp16.  Odd rows take
    // the halves in the opposite order: the eight lanes of a load phase then
    // read all 32 banks, and those of a store phase (four even, four odd
    // rows' chunks) hit eight different swizzled places.
    const int cc = ctid & 3, row0 = ctid >> 2;
    const int flip = kHalves == 2 ? row0 & 1 : 0;
    const int e0 = row0 * 128 + (((2 * cc) ^ (row0 & 7)) << 4);
    const int e1 = row0 * 128 + (((2 * cc + 1) ^ (row0 & 7)) << 4);
    constexpr int kPer = kKeys / 32 * kHalves;  // chunks per thread and tile
    uint32_t g = 0;
    bool ok = true;
    // Tile t of K (w = 0) or V (w = 1) into its stage, once the one before
    // there was read.  Of a V tile that some row of the item sees in part, what
    // would reach that row with its weight of 0 becomes zero, as 0 * NaN is NaN
    // in the MMA: rows from `limit` on, the context's end, and NaN codes; if
    // there were any of these, *nan_flag is set.
    auto convert = [&](int w, uint32_t t, bool partly, int limit,
                       int* nan_flag) -> bool {
      const uint32_t slot = w * kRaw + t % kRaw, s = t % kStages;
      if (!warp_wait(raw_full0 + 8 * slot, (t / kRaw) & 1) ||
          (t >= kStages && !warp_wait((w ? v_empty0 : k_empty0) + 8 * s,
                                      ((t / kStages) - 1) & 1)))
        return false;
      const uint8_t* raw = smem + Lay::kOffRaw + slot * Lay::kRawTile +
                           row0 * D + cc * 16;
      uint8_t* d = smem + (w ? Lay::kOffV : Lay::kOffK) + s * Lay::kTile;
      auto load = [&](int i) {
        return *reinterpret_cast<const uint4*>(
            raw + 32 * (i / kHalves) * D + ((i % kHalves) ^ flip) * 64);
      };
      auto store = [&](int i, const uint4& w) {
        uint8_t* to = d + ((i % kHalves) ^ flip) * kTileHalf +
                      32 * (i / kHalves) * 128;
        *reinterpret_cast<uint4*>(to + e0) = make_uint4(
            dev::e4m3x2_to_f16x2(w.x), dev::e4m3x2_to_f16x2_hi(w.x),
            dev::e4m3x2_to_f16x2(w.y), dev::e4m3x2_to_f16x2_hi(w.y));
        *reinterpret_cast<uint4*>(to + e1) = make_uint4(
            dev::e4m3x2_to_f16x2(w.z), dev::e4m3x2_to_f16x2_hi(w.z),
            dev::e4m3x2_to_f16x2(w.w), dev::e4m3x2_to_f16x2_hi(w.w));
      };
      if (!partly) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) store(i, load(i));
      } else {
        uint32_t nans = 0u;
#pragma unroll 1
        for (int i = 0; i < kPer; ++i) {
          uint4 w = load(i);
          if (row0 + 32 * (i / kHalves) >= limit)
            w = make_uint4(0u, 0u, 0u, 0u);
          const uint4 n = make_uint4(nan_bytes(w.x), nan_bytes(w.y),
                                     nan_bytes(w.z), nan_bytes(w.w));
          nans |= n.x | n.y | n.z | n.w;
          store(i, make_uint4(w.x & ~n.x, w.y & ~n.y, w.z & ~n.z,
                              w.w & ~n.w));
        }
        if (nans) *nan_flag = 1;
      }
      dev::fence_proxy_async_smem();  // visible to the tensor cores
      __syncwarp();
      warp_arrive((w ? v_full0 : k_full0) + 8 * s);
      warp_arrive(raw_empty0 + 8 * slot);
      return true;
    };
    for (int n = 0; ok; ++n) {
      Item it;
      ok = next_item(n, it);
      if (!ok || it.state == kEnd) break;
      // NaN codes that are taken out belong to the rows that see them: the
      // item's slot (flag, sequence, KV head, first key, row of position 0)
      // tells the epilogue to look for them.  Its flag is cleared four items
      // ahead: an item is published once every warp has taken up the one two
      // before, so the slot's last readers (of eight items back) are done when
      // it is cleared, and it is clear when its first writer comes.
      int* nan_at = nan_s + kNanInts * (n % kNanSlots);
      if (ctid == 0) nan_s[kNanInts * ((n + 4) % kNanSlots)] = 0;
      if (it.state == kSkip) continue;
      const Span sp = span_of(it);
      const int seen = it.L - it.q_len + sp.tok0[0] + 1;  // by every row
      if (ctid == 0) {
        nan_at[1] = it.b;
        nan_at[2] = it.kvh;
        nan_at[3] = seen / kKeys * kKeys;
        nan_at[4] = it.q0 + it.q_len - it.L;
      }
      for (int t = 0; ok && t <= sp.tiles; ++t) {
        if (t < sp.tiles) ok = convert(0, g + t, false, 0, nullptr);
        if (ok && t >= 1)
          ok = convert(1, g + t - 1, t * kKeys > seen,
                       it.L - (t - 1) * kKeys, nan_at);
      }
      g += sp.tiles;
    }
    if (!ok) dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
    return;
  }

  // ---------------- softmax warps (thread = query row) ----------------
  regs_inc<kSoftmaxRegs>();
  const int x = warp >> 2;        // query tile of the pair
  const int quarter = warp & 3;   // tensor-memory lane quarter of this warp
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t s_tmem = tbase + kColS + x * 64 + lane_off;
  const uint32_t p_tmem = tbase + kColP + x * 32 + lane_off;
  const uint32_t qt_tmem = tbase + kColQ + x * 32 + lane_off;
  const uint32_t o_tmem = tbase + kColO + x * 128 + lane_off;
  const uint32_t q_full = q_full0 + 8 * x, q_empty = q_empty0 + 8 * x;
  const uint32_t s_full = s_full0 + 8 * x, s_free = s_free0 + 8 * x;
  const uint32_t p_full = p_full0 + 8 * x, o_done = o_done0 + 8 * x;
  const int r = quarter * 32 + lane;
  const int t_loc = r / G;
  const int hg = r - t_loc * G;
  bool ok = true;
  uint32_t g = 0;   // K/V tiles of this CTA's earlier items (scale slots)
  uint32_t ts = 0;  // S tiles of this query tile so far
  int v = 0;        // items so far
  int halves = 0;   // of which the pair shared the keys
  float* merge = reinterpret_cast<float*>(smem + Lay::kOffMerge) + r;
  for (int n = 0; ok; ++n) {
    Item it;
    ok = next_item(n, it);
    if (!ok || it.state == kEnd) break;
    if (it.state == kSkip) continue;
    const Span sp = span_of(it);
    const int n_q = x ? sp.n_q[1] : sp.n_q[0];
    const int n_tiles = x ? sp.n_tiles[1] : sp.n_tiles[0];
    const int tok0 = x ? sp.tok0[1] : sp.tok0[0];
    if (n_tiles == 0) {  // no rows for the second tile
      g += sp.tiles;
      continue;
    }
    const int tok = tok0 + t_loc;
    const bool valid = t_loc < n_q;
    // Padding rows see what the tile's last row sees; never stored.
    const int qpos = it.L - it.q_len + (valid ? tok : tok0 + n_q - 1);
    // A warp whose rows are all padding only keeps the barriers' protocol.
    const bool idle = quarter * 32 >= n_q * G;
    const int64_t row_at =
        (static_cast<int64_t>(it.q0 + tok) * a.num_q_heads + it.kvh * G + hg) *
        D;
    float c_row = 0.f;
    // This row of Q: to fp16 times a power of two, into the swizzled operand
    // once the previous item's S MMAs are done with it.
    {
      uint4 w[D / 8];
      if (!idle) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          w[i] = valid ? reinterpret_cast<const uint4*>(
                             static_cast<const T*>(a.q) + row_at)[i]
                       : make_uint4(0u, 0u, 0u, 0u);
      }
      if (v >= 1 && !warp_wait(q_empty, (v - 1) & 1)) {
        ok = false;
        break;
      }
      if (!idle) {
        // The largest magnitude, on the packed bits (ordered like the
        // values; unpacked here, 128 floats would stay in registers until
        // they are converted).
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t y[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top = __vmaxu2(top, y[e] & 0x7fff7fffu);
        }
        const float2 top2 = dev::Mma<T>::unpack(top);
        const float amax = fmaxf(top2.x, top2.y);
        const int k = min(14 - dev::floor_log2(amax), 100);
        // a negative scale turns the sign of q, so that scores can be
        // compared before they are scaled
        const float up =
            a.scale_log2 < 0.f ? -dev::exp2_int(k) : dev::exp2_int(k);
        c_row = fabsf(a.scale_log2) * dev::exp2_int(-k);
        auto convert8 = [&](const uint4& in, uint32_t* z) {
          const uint32_t y[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = dev::Mma<T>::unpack(y[e]);
            z[e] = M::pack(f.x * up, f.y * up);
          }
        };
        constexpr int kInSmem = (kHalves - 1) * 8;  // 16-byte chunks
#pragma unroll
        for (int i = 0; i < kInSmem; ++i) {
          uint32_t z[4];
          convert8(w[i], z);
          *reinterpret_cast<uint4*>(smem + Lay::kOffQ + x * Lay::kQTile +
                                    r * 128 + ((i ^ (r & 7)) << 4)) =
              make_uint4(z[0], z[1], z[2], z[3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t z[16];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            convert8(w[kInSmem + 4 * h + i], z + 4 * i);
          dev::tmem_st16u(qt_tmem + 16 * h, z);
        }
        dev::tmem_st_wait();
        dev::tc_fence_before();
        dev::fence_proxy_async_smem();
      }
      __syncwarp();
      warp_arrive(q_full);
      ++v;
    }
    float m_ref = 0.f, l = 0.f, e_ref = 0.f;  // e_ref: E
    const int first = sp.stride == 2 ? x : 0;
    for (int j = 0; j < n_tiles && ok; ++j, ++ts) {
      ok = warp_wait(s_full, ts & 1);
      if (!ok) break;
      float sv[kKeys];
      if (!idle) {
        dev::tc_fence_after();
        float (&lo)[32] = *reinterpret_cast<float(*)[32]>(sv);
        float (&hi)[32] = *reinterpret_cast<float(*)[32]>(sv + 32);
        dev::tmem_ld32(s_tmem, lo);
        dev::tmem_ld32(s_tmem + 32, hi);
        dev::tmem_ld_wait();
        dev::tc_fence_before();
      }
      warp_arrive(s_free);
      if (idle) {
        // Arrives for tile ts only once P(ts-1).V is done: an arrival a tile
        // ahead would count toward tile ts-1 on the single p_full barrier.
        if (ts >= 1 && !warp_wait(o_done, (ts - 1) & 1)) {
          ok = false;
          break;
        }
        warp_arrive(p_full);
        continue;
      }
      const int tile = first + j * sp.stride;
      const int lim = qpos - tile * kKeys;  // the last key this row sees
      // A factor c_row ks_b for each block (never 0: -inf * 0 is NaN).
      const float* sc = scale_s + ((g + tile) % kScaleSlots) * kSlotFloats;
      float cb[kNB];
#pragma unroll
      for (int b = 0; b < kNB; ++b) cb[b] = max_nan(c_row * sc[b], kTiny);
      if (lim < kKeys - 1) {
#pragma unroll
        for (int k = 0; k < kKeys; ++k)
          if (k > lim) sv[k] = -INFINITY;
        // nor does a NaN scale reach a row that sees nothing of its block
#pragma unroll
        for (int b = 0; b < kNB; ++b)
          if (b * BS > lim) cb[b] = kTiny;
      }
      // The row's maximum, by blocks.
      float mx = -INFINITY;
#pragma unroll
      for (int b = 0; b < kNB; ++b) {
        float m4[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          m4[u] = dev::fmax3(sv[b * BS + u], sv[b * BS + 4 + u],
                             sv[b * BS + 8 + u]);
          m4[u] = fmaxf(m4[u], sv[b * BS + 12 + u]);
        }
        if constexpr (BS == 32) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            m4[u] = dev::fmax3(m4[u], sv[b * BS + 16 + u],
                               sv[b * BS + 20 + u]);
            m4[u] = dev::fmax3(m4[u], sv[b * BS + 24 + u],
                               sv[b * BS + 28 + u]);
          }
        }
        mx = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) *
                           cb[b]);
      }
      // O's factor for what E grew by since this row's last tile (1: not)
      const float e_now = sc[kSlotFloats - 1];
      float factor = 1.f;
      if (j == 0) {
        // O is still empty: the first P.V overwrites it.  (A row may see no
        // key of tile 1's first tile: finite, so that its weights are 0.)
        m_ref = fmaxf(mx, -3e38f);
      } else {
        factor = dev::fast_exp2(e_ref - e_now);
        if (mx > m_ref + kRescaleLog2) {
          const float f = dev::fast_exp2(m_ref - mx);
          m_ref = mx;
          l *= f;
          factor *= f;
        }
      }
      e_ref = e_now;
      if (__any_sync(0xffffffffu, factor != 1.f)) {
        // Rare (the maxima settle): a rolled loop over 16 columns, which
        // leaves the scores in their registers.
        ok = warp_wait(o_done, (ts - 1) & 1);
        if (!ok) break;
        dev::tc_fence_after();
#pragma unroll 1
        for (int col = 0; col < D; col += 16) {
          uint32_t ov[16];
          dev::tmem_ld16u(o_tmem + col, ov);
          dev::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            ov[e] = __float_as_uint(__uint_as_float(ov[e]) * factor);
          dev::tmem_st16u(o_tmem + col, ov);
        }
      }
      // w = 2^(s c_b + log2(vs_b) - E + shift - m), two keys per
      // instruction; the sum of p from the block sums of w.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t hw[16];
#pragma unroll
        for (int b = h * kNB / 2; b < (h + 1) * kNB / 2; ++b) {
          const float off = sc[kNB + b] - m_ref;
          const float2 c2 = make_float2(cb[b], cb[b]);
          const float2 o2 = make_float2(off, off);
          float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int e = b * BS / 2; e < (b + 1) * BS / 2; ++e) {
            const float2 y =
                dev::ffma2(make_float2(sv[2 * e], sv[2 * e + 1]), c2, o2);
            const float w0 = dev::fast_exp2(y.x), w1 = dev::fast_exp2(y.y);
            l2[e & 1] = dev::fadd2(l2[e & 1], make_float2(w0, w1));
            hw[e - 16 * h] = M::pack(w0, w1);
          }
          const float2 lb = dev::fadd2(l2[0], l2[1]);
          l = fmaf(lb.x + lb.y, sc[2 * kNB + b], l);
        }
        if (h == 0) {
          // P(ts-1).V must have read the P buffer before it is overwritten.
          if (ts >= 1 && !warp_wait(o_done, (ts - 1) & 1)) ok = false;
          if (!ok) break;
          dev::tc_fence_after();
        }
        dev::tmem_st16u(p_tmem + 16 * h, hw);
      }
      if (!ok) break;
      dev::tmem_st_wait();
      dev::tc_fence_before();
      warp_arrive(p_full);
    }
    // The item's output: O 2^(E - shift) / l -> out[token, query head].
    // (The phase before it was waited for with the last tile's P.)
    if (ok) ok = warp_wait(o_done, (ts - 1) & 1);
    // Factors of O and, where the pair shared the keys, of tile 1's O.
    float f0 = dev::exp2_int(static_cast<int>(e_ref - kShift)), f1 = 0.f;
    if (ok && sp.stride == 2) {
      if (x == 1) {
        merge[0] = m_ref;
        merge[kRows] = l;
        merge[2 * kRows] = e_ref;
        dev::tc_fence_before();
        __syncwarp();
        warp_arrive(half_done);
        // the next item's P.V may overwrite O once tile 0 has read it
        ok = warp_wait(half_read, halves & 1);
      } else {
        ok = warp_wait(half_done, halves & 1);
        if (ok) {
          const float m1 = merge[0], l1 = merge[kRows];
          const float top = fmaxf(m_ref, m1);
          const float w0 = dev::fast_exp2(m_ref - top);
          const float w1 = dev::fast_exp2(m1 - top);
          l = l * w0 + l1 * w1;
          f0 *= w0;
          f1 = w1 *
               dev::exp2_int(static_cast<int>(merge[2 * kRows] - kShift));
        }
      }
      ++halves;
    }
    if (ok && !idle && (x == 0 || sp.stride == 1)) {
      dev::tc_fence_after();
      // l is above 0 (each row sees a key) or NaN, which is passed on
      const float inv = 1.f / l;
      f0 *= inv;
      f1 *= inv;
      T* dst = static_cast<T*>(a.out) + row_at;
      float* dst32 = static_cast<float*>(a.out) + row_at;  // out_f32 only
#pragma unroll 1
      for (int col = 0; col < D; col += 32) {
        float ov[32];
        dev::tmem_ld32(o_tmem + col, ov);
        dev::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) ov[e] *= f0;
        if (sp.stride == 2) {
          float o1[32];
          dev::tmem_ld32(o_tmem + 128 + col, o1);
          dev::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = fmaf(o1[e], f1, ov[e]);
        }
        if (valid && a.out_f32) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(dst32 + col + e) =
                make_float4(ov[e], ov[e + 1], ov[e + 2],
                            ov[e + 3]);
        } else if (valid) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 w;
            w.x = dev::Mma<T>::pack(ov[e], ov[e + 1]);
            w.y = dev::Mma<T>::pack(ov[e + 2], ov[e + 3]);
            w.z = dev::Mma<T>::pack(ov[e + 4], ov[e + 5]);
            w.w = dev::Mma<T>::pack(ov[e + 6], ov[e + 7]);
            *reinterpret_cast<uint4*>(dst + col + e) = w;
          }
        }
      }
      dev::tc_fence_before();
      // Rare: the NaN codes that the converters took out, back into the
      // outputs of the row that sees them.
      const volatile int* nan_at = nan_s + kNanInts * (n % kNanSlots);
      if (nan_at[0] != 0 && valid) {
        const int64_t row =
            (static_cast<int64_t>(nan_at[4] + qpos) * a.num_q_heads +
             nan_at[2] * G + hg) * D;
#pragma unroll 1
        for (int key = nan_at[3]; key <= qpos; ++key) {
          const int32_t id =
              a.block_tables[static_cast<int64_t>(nan_at[1]) *
                                 a.max_blocks_per_seq + key / BS];
          if (id < 0 || id >= a.num_blocks) continue;  // flagged already
          const uint8_t* codes =
              a.v_cache + ((static_cast<int64_t>(id) * a.num_kv_heads +
                            nan_at[2]) * BS + key % BS) * D;
#pragma unroll 1
          for (int i = 0; i < D; ++i) {
            if ((codes[i] & 0x7f) != 0x7f) continue;
            if (a.out_f32)
              static_cast<float*>(a.out)[row + i] = NAN;
            else
              static_cast<uint16_t*>(a.out)[row + i] =
                  static_cast<uint16_t>(dev::Mma<T>::pack(NAN, NAN));
          }
        }
      }
    }
    if (ok && sp.stride == 2 && x == 0) {
      __syncwarp();
      warp_arrive(half_read);
    }
    g += sp.tiles;
  }
  if (!ok) dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
  dev::tc_fence_before();
  __syncwarp();
  if (lane == 0) dev::mbar_arrive(done);
}

// ---------------------------------------------------------------------------
// Host side.

template <typename T, int BS, int G, int D, bool kShareKeys>
pa_status launch(const PrefillQ8Args& a, cudaStream_t st) {
  auto kern = prefill_q8_kernel<T, BS, G, D, kShareKeys>;
  const size_t smem = LayoutQ8<D>::kSmemBytes;
  static OncePerDevice configured;
  cudaError_t e = cudaSuccess;
  if (configured.needed()) {
    // The warpgroups' shares of the registers assume kLaunchRegs a thread.
    cudaFuncAttributes attrs;
    e = cudaFuncGetAttributes(&attrs, kern);
    if (e != cudaSuccess || attrs.numRegs != kLaunchRegs)
      return fail(PA_ERR_CUDA,
                  "pa_prefill_q8: built with %d registers, not %d",
                  e == cudaSuccess ? attrs.numRegs : -1, kLaunchRegs);
    e = cudaFuncSetAttribute(
        kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
        static_cast<int>(smem));
    if (e != cudaSuccess)
      return fail(PA_ERR_CUDA, "pa_prefill_q8: cudaFuncSetAttribute(%zu): %s",
                  smem, cudaGetErrorString(e));
    configured.mark();
  }
  cudaLaunchConfig_t cfg = {};
  const int64_t slots = std::max(device_sm_count(), 1);  // one CTA per SM
  cfg.gridDim =
      dim3(static_cast<unsigned>(std::min<int64_t>(a.num_items, slots)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  count_launch();
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(PA_ERR_CUDA, "pa_prefill_q8: launch failed: %s",
                cudaGetErrorString(e));
  return PA_OK;
}

// A call whose sequences have at most one query tile of new tokens, and
// contexts that may exceed four key tiles, runs with kShareKeys.  4 new tokens
// of 256 sequences, 64 query heads: contexts of 1500 tokens 377 us instead of
// 442, of 300 137 instead of 145, but of 128 100 instead of 96 and of 64 88
// instead of 81; 218 draft rows over 72k cached tokens 89 instead of 110.  As a
// branch of the one kernel it cost the others 3 to 5 % (registers).
template <typename T, int BS, int G, int D>
pa_status dispatch_share(const pa_prefill_desc* d, const PrefillQ8Args& a,
                         cudaStream_t st) {
  return static_cast<int64_t>(d->max_q_len) * G <= kRows &&
                 a.max_context_len > 4 * kKeys
             ? launch<T, BS, G, D, true>(a, st)
             : launch<T, BS, G, D, false>(a, st);
}

template <typename T, int BS, int D>
pa_status dispatch_group(const pa_prefill_desc* d, const PrefillQ8Args& a,
                         cudaStream_t st) {
  switch (d->num_q_heads / d->num_kv_heads) {
    case 1: return dispatch_share<T, BS, 1, D>(d, a, st);
    case 2: return dispatch_share<T, BS, 2, D>(d, a, st);
    case 4: return dispatch_share<T, BS, 4, D>(d, a, st);
    default: return dispatch_share<T, BS, 8, D>(d, a, st);
  }
}

template <typename T>
pa_status dispatch_shape(const pa_prefill_desc* d, const PrefillQ8Args& a,
                         cudaStream_t st) {
  if (d->head_dim == 128)
    return d->block_size == 16 ? dispatch_group<T, 16, 128>(d, a, st)
                               : dispatch_group<T, 32, 128>(d, a, st);
  return d->block_size == 16 ? dispatch_group<T, 16, 64>(d, a, st)
                             : dispatch_group<T, 32, 64>(d, a, st);
}

}  // namespace
}  // namespace pagedkv

using pagedkv::fail;

extern "C" pa_status pa_prefill_q8(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const float* k_scales, const float* v_scales, const int32_t* block_tables,
    const int32_t* context_lens, const int32_t* query_start, float scale,
    const pa_prefill_desc* d, void* workspace, size_t workspace_bytes,
    int32_t* dev_err, void* stream) {
  pagedkv::clear_error();
  const pa_status ok = pagedkv::check_prefill(
      "pa_prefill_q8", out, q, k_cache, v_cache, block_tables, context_lens,
      query_start, scale, d, workspace, workspace_bytes);
  if (ok != PA_OK || pagedkv::nothing_to_do(d)) return ok;
  if (!k_scales || !v_scales)
    return fail(PA_ERR_INVALID_ARG, "pa_prefill_q8: NULL scales");
  const int max_ctx = d->max_context_len > 0
                          ? d->max_context_len
                          : d->max_blocks_per_seq * d->block_size;
  pagedkv::PrefillQ8Args a;
  a.out = out;
  a.q = q;
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.tiles = pagedkv::tile_map(d, workspace);
  a.counter = pagedkv::work_counter(d, workspace);
  // Items of kPair query tiles: the tile map holds at most as many entries
  // as with tiles of one, for which the workspace is sized.
  const int item_tok = pagedkv::kPair * pagedkv::tile_tokens(d);
  const int64_t cap = pagedkv::tile_cap(d, item_tok);
  a.num_items = static_cast<int>(cap * d->num_kv_heads);
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.query_start = query_start;
  a.dev_err = dev_err;
  a.scale_log2 = scale * pagedkv::kLog2e;
  a.num_q_heads = d->num_q_heads;
  a.num_kv_heads = d->num_kv_heads;
  a.max_blocks_per_seq = d->max_blocks_per_seq;
  a.num_blocks = d->num_blocks;
  a.max_context_len = max_ctx;
  a.total_q = d->total_q;
  a.out_f32 = d->out_fp32;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const pa_status planned =
      pagedkv::launch_plan("pa_prefill_q8", d, context_lens, query_start,
                           max_ctx, item_tok, workspace, dev_err, s);
  if (planned != PA_OK) return planned;
  return d->dtype == PA_BF16
             ? pagedkv::dispatch_shape<__nv_bfloat16>(d, a, s)
             : pagedkv::dispatch_shape<__half>(d, a, s);
}
