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
//    element to [2^14, 2^15): exact for fp16, and for bf16 down to 2^-39 of
//    the largest element.
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
// Work items, the persistent grid (two CTAs per SM), the query tiles of 128
// rows and the barriers' discipline (each counted over the CTA's tiles,
// waited on in order, never two phases ahead) are pa_prefill's
// (prefill.cu).  Warps: 0..3 hold one query row per thread: they load and
// convert its q, and run the softmax; 4..7 convert K and V; 8 takes the
// items, copies pages (contiguous in this layout: one bulk copy each) and
// stages their scales; 9 issues the MMAs.
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
constexpr int kRaw = 4;          // tiles of codes in flight (K and V in turn)
constexpr int kScaleSlots = 8;   // tiles whose scales are staged
// Warps 0..3 softmax, 4..7 converters, 8 pages and scales, 9 MMA (10 and 11
// only complete its warpgroup).  Registers: 80 a thread at launch, shared out
// anew between the warpgroups; kept at 80 x 3 in sum (an increase waits for
// registers that the others gave up).
constexpr int kThreads = 384;
constexpr int kConvThreads = 128;
constexpr int kLaunchRegs = 80;
constexpr int kSoftmaxRegs = 176, kConvRegs = 24, kIssueRegs = 40;
static_assert(kSoftmaxRegs + kConvRegs + kIssueRegs == 3 * kLaunchRegs,
              "more registers than the block was launched with");
constexpr int kTmemCols = 256;   // S [0, 64), P [64, 96), O [128, 128 + D)
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

// q_full, raw_full[], raw_empty[], k_full, k_empty, v_full, v_empty, s_full,
// s_free, p_full, o_ready, done, q_empty, item_full[2], item_empty[2].
constexpr int kNumBars = 1 + 2 * kRaw + 4 + 4 + 2 + 4;
constexpr int kItemWords = 8;

template <int D>
struct LayoutQ8 {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalfQ = kRows * 128;
  static constexpr int kTile = kHalves * kTileHalf;  // fp16 K or V tile
  static constexpr int kRawTile = kKeys * D;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kHalves * kHalfQ;
  static constexpr int kOffV = kOffK + kTile;
  static constexpr int kOffRaw = kOffV + kTile;
  static constexpr int kOffScales = kOffRaw + kRaw * kRawTile;
  static constexpr int kOffBars = kOffScales + kScaleSlots * 32;
  static constexpr size_t kSmemBytes =
      1024 + kOffBars + kNumBars * 8 + 16 + 2 * kItemWords * 4;
};

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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

template <typename T, int BS, int G, int D>
__global__ void __launch_bounds__(kThreads, 2)
    prefill_q8_kernel(const PrefillQ8Args a) {
  using Lay = LayoutQ8<D>;
  using M = dev::Mma<__half>;
  constexpr int kTok = kRows / G;   // new tokens per tile
  constexpr int kNB = kKeys / BS;   // blocks (pages) per tile
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem =
      smem_dyn + ((1024u - (dev::smem_u32(smem_dyn) & 1023u)) & 1023u);
  const uint32_t base = dev::smem_u32(smem);
  const uint32_t q_s = base + Lay::kOffQ;
  const uint32_t k_s = base + Lay::kOffK;
  const uint32_t v_s = base + Lay::kOffV;
  float* scale_s = reinterpret_cast<float*>(smem + Lay::kOffScales);
  const uint32_t bars = base + Lay::kOffBars;
  const uint32_t q_full = bars;
  const uint32_t raw_full0 = q_full + 8;
  const uint32_t raw_empty0 = raw_full0 + 8 * kRaw;
  const uint32_t k_full = raw_empty0 + 8 * kRaw;
  const uint32_t k_empty = k_full + 8;
  const uint32_t v_full = k_empty + 8;
  const uint32_t v_empty = v_full + 8;
  const uint32_t s_full = v_empty + 8;
  const uint32_t s_free = s_full + 8;
  const uint32_t p_full = s_free + 8;
  const uint32_t o_ready = p_full + 8;
  const uint32_t done = o_ready + 8;
  const uint32_t q_empty = done + 8;
  const uint32_t item_full0 = q_empty + 8;
  const uint32_t item_empty0 = item_full0 + 16;
  uint32_t* tmem_slot =
      reinterpret_cast<uint32_t*>(smem + Lay::kOffBars + kNumBars * 8);
  volatile int* item_s = reinterpret_cast<volatile int*>(tmem_slot + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  dev::pdl_trigger();
  if (tid == 0) {
    dev::mbar_init(q_full, 4);
    for (int s = 0; s < kRaw; ++s) {
      dev::mbar_init(raw_full0 + 8 * s, 1);
      dev::mbar_init(raw_empty0 + 8 * s, 4);
    }
    dev::mbar_init(k_full, 4);
    dev::mbar_init(k_empty, 1);
    dev::mbar_init(v_full, 4);
    dev::mbar_init(v_empty, 1);
    dev::mbar_init(s_full, 1);
    dev::mbar_init(s_free, 4);
    dev::mbar_init(p_full, 4);
    dev::mbar_init(o_ready, 1);
    dev::mbar_init(done, 4);
    dev::mbar_init(q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      dev::mbar_init(item_full0 + 8 * s, 1);
      dev::mbar_init(item_empty0 + 8 * s, 9);
    }
    dev::fence_mbar_init();
  }
  if (warp == 9) {
    dev::tmem_alloc(dev::smem_u32(tmem_slot), kTmemCols);
    dev::tmem_relinquish();
  }
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const uint32_t s_tmem = tbase;
  const uint32_t p_tmem = tbase + kKeys;
  const uint32_t o_tmem = tbase + 128;
  dev::pdl_wait();

  struct Item {
    int state;  // kWork, kSkip (invalid input, flagged) or kEnd
    int b, kvh, qt, L, q0, q_len;
  };
  constexpr int kWork = 0, kSkip = 1, kEnd = 2;
  struct Span {
    int tok0, n_q, kv_end, n_tiles;
  };
  auto span_of = [](const Item& it) {
    Span sp;
    sp.tok0 = it.qt * kTok;
    sp.n_q = min(kTok, it.q_len - sp.tok0);
    sp.kv_end = it.L - it.q_len + sp.tok0 + sp.n_q;
    sp.n_tiles = (sp.kv_end + kKeys - 1) / kKeys;
    return sp;
  };
  auto read_item = [&](int n, Item& it) -> bool {
    const int slot = n & 1;
    if (!dev::mbar_wait(item_full0 + 8 * slot, (n >> 1) & 1)) return false;
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
  // The same for a whole warp (the waits of collectives are warp-uniform).
  auto next_item = [&](int n, Item& it) -> bool {
    if (!__all_sync(0xffffffffu, read_item(n, it))) return false;
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(item_empty0 + 8 * (n & 1));
    return true;
  };

  if (warp >= 8) regs_dec<kIssueRegs>();
  if (warp == 8) {
    // ---------------- work items, pages and scales ----------------
    // Lane p looks after page p of each tile.
    const int p = lane;
    const bool mine = p < kNB;
    uint32_t u = 0;  // raw tiles of this CTA so far
    uint32_t g = 0;  // tiles of this CTA's earlier items
    bool ok = true;
    auto warp_wait = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, dev::mbar_wait(bar, parity));
    };
    auto acquire = [&]() -> bool {
      return u < kRaw ||
             warp_wait(raw_empty0 + 8 * (u % kRaw), ((u / kRaw) - 1) & 1);
    };
    auto copy = [&](const uint8_t* cache, int kvh, int32_t id) {
      const uint32_t full = raw_full0 + 8 * (u % kRaw);
      __syncwarp();  // the tile's scales, if any, are stored
      if (lane == 0) dev::mbar_arrive_expect_tx(full, Lay::kRawTile);
      __syncwarp();
      if (mine)
        bulk_load(base + Lay::kOffRaw + (u % kRaw) * Lay::kRawTile +
                      p * BS * D,
                  cache + (static_cast<int64_t>(id) * a.num_kv_heads + kvh) *
                              (BS * D),
                  BS * D, full);
      ++u;
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
            it.qt * kTok >= it.q_len;
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
      auto fetch = [&](int j) -> int32_t {
        const int page = j * kNB + p;
        const int32_t id = __ldg(row + (page < n_pages ? page : 0));
        const bool bad = id < 0 || id >= a.num_blocks;
        bad_id |= bad;
        return bad ? 0 : id;
      };
      auto fetch_scales = [&](int j, int32_t id) -> float2 {
        if (j * kNB + p >= n_pages) return make_float2(1.f, 0.f);
        const int64_t at = static_cast<int64_t>(id) * a.num_kv_heads + kvh;
        return make_float2(a.k_scales[at], a.v_scales[at]);
      };
      // Ids are read two tiles and scales one tile ahead of their use.
      int32_t cur = 0, nxt = 0, nn = 0, prv = 0;
      float2 sc = make_float2(1.f, 0.f), nsc = sc;
      if (mine) {
        nxt = fetch(0);
        if (sp.n_tiles > 1) nn = fetch(1);
        nsc = fetch_scales(0, nxt);
      }
      for (int t = 0; t <= sp.n_tiles; ++t) {
        if (t < sp.n_tiles) {
          cur = nxt;
          nxt = nn;
          sc = nsc;
          if (mine && t + 2 < sp.n_tiles) nn = fetch(t + 2);
          if (mine && t + 1 < sp.n_tiles) nsc = fetch_scales(t + 1, nxt);
          if (!acquire()) {
            ok = false;
            break;
          }
          // A slot is written again kScaleSlots tiles on.  With kRaw tiles
          // in flight the K tile it comes with is at most three ahead of the
          // one whose S is next, so its old reader is long past.
          if (mine) {
            float* to = scale_s + ((g + t) % kScaleSlots) * 8;
            to[p] = sc.x;
            to[kNB + p] = fminf(fmaxf(log2f(sc.y), -100.f), 100.f);
          }
          copy(a.k_cache, kvh, cur);
        }
        if (t >= 1) {
          if (!acquire()) {
            ok = false;
            break;
          }
          copy(a.v_cache, kvh, prv);
        }
        prv = cur;
      }
      if (bad_id) dev::set_error(a.dev_err, PA_ERR_DEVICE_OOB);
      g += sp.n_tiles;
    }
    if (!ok && lane == 0) dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
    return;
  }

  if (warp >= 10) return;
  if (warp == 9) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      bool ok = true;
      constexpr uint32_t idesc_qk =
          dev::umma_idesc_f16(false, kRows, kKeys, false, false);
      constexpr uint32_t idesc_pv =
          dev::umma_idesc_f16(false, kRows, D, false, true);
      auto issue_pv = [&](uint32_t t, bool first) -> bool {
        if (!dev::mbar_wait(v_full, t & 1) || !dev::mbar_wait(p_full, t & 1))
          return false;
        dev::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk) {
          const uint64_t bd =
              dev::sw128_desc(v_s + kk * 2048, kTileHalf, 1024);
          dev::umma_f16_ts(o_tmem, p_tmem + kk * 8, bd, idesc_pv,
                           (!first || kk > 0) ? 1u : 0u);
        }
        dev::umma_commit(o_ready);
        dev::umma_commit(v_empty);
        return true;
      };
      auto issue_s = [&](uint32_t t, bool last) -> bool {
        if (!dev::mbar_wait(k_full, t & 1) ||
            (t >= 1 && !dev::mbar_wait(s_free, (t - 1) & 1)))
          return false;
        dev::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int h = kk >> 2, k4 = kk & 3;
          const uint64_t ad =
              dev::sw128_desc(q_s + h * Lay::kHalfQ + k4 * 32, 16, 1024);
          const uint64_t bd =
              dev::sw128_desc(k_s + h * kTileHalf + k4 * 32, 16, 1024);
          dev::umma_f16(s_tmem, ad, bd, idesc_qk, kk > 0 ? 1u : 0u);
        }
        dev::umma_commit(s_full);
        dev::umma_commit(k_empty);
        if (last) dev::umma_commit(q_empty);
        return true;
      };
      uint32_t g = 0;
      int v = 0;
      for (int n = 0; ok; ++n) {
        Item it;
        if (!read_item(n, it)) {
          ok = false;
          break;
        }
        dev::mbar_arrive(item_empty0 + 8 * (n & 1));
        if (it.state == kEnd) break;
        if (it.state == kSkip) continue;
        const int nt = span_of(it).n_tiles;
        ok = dev::mbar_wait(q_full, v & 1) && issue_s(g, nt == 1);
        for (int j = 0; ok && j < nt; ++j) {
          if (j + 1 < nt) ok = issue_s(g + j + 1, j + 2 == nt);
          if (ok) ok = issue_pv(g + j, j == 0);
        }
        g += nt;
        ++v;
      }
      if (ok && g > 0) ok = dev::mbar_wait(o_ready, (g - 1) & 1);
      if (!ok) dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
      if (!dev::mbar_wait(done, 0))
        dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
    }
    __syncwarp();
    dev::tc_fence_after();
    dev::tmem_dealloc(tbase, kTmemCols);
    return;
  }

  if (warp >= 4) {
    // ---------------- converters: codes -> fp16 tiles ----------------
    regs_dec<kConvRegs>();
    const int ctid = tid - 4 * 32;
    // This thread's 16-code chunk, in rows my_row, my_row + kRowStep, ...:
    // two 16-byte chunks of fp16 in the swizzled tile (kRowStep is a multiple
    // of 8, so their places in the row stay).  Threads of the second half of
    // head_dim store their two in the opposite order: the eight lanes of a
    // store phase then hit eight different bank groups.
    constexpr int kChunks = D / 16;
    constexpr int kRowStep = kConvThreads / kChunks;
    const int my_row = ctid / kChunks;
    const bool swap = (ctid % kChunks) >= 4;
    const int my_dst = (swap ? kTileHalf : 0) + my_row * 128;
    const int my_chunk = 2 * (ctid & 3);
    const int my_e = (my_chunk ^ (my_row & 7)) << 4;
    const int my_o = ((my_chunk + 1) ^ (my_row & 7)) << 4;
    const int my_a = swap ? my_o : my_e, my_b = swap ? my_e : my_o;
    uint32_t u = 0, g = 0;
    bool ok = true;
    auto warp_wait = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, dev::mbar_wait(bar, parity));
    };
    // Raw tile u into the fp16 tile at offset `dst`, once `empty` says that
    // tile t - 1 there was read; rows from `limit` on become zeros (a key
    // past the context has weight 0, but 0 * NaN is NaN in the MMA).
    auto convert = [&](int dst, uint32_t full, uint32_t empty, uint32_t t,
                       int limit) -> bool {
      const uint32_t slot = u % kRaw;
      if (!warp_wait(raw_full0 + 8 * slot, (u / kRaw) & 1) ||
          (t >= 1 && !warp_wait(empty, (t - 1) & 1)))
        return false;
      const uint8_t* raw = smem + Lay::kOffRaw + slot * Lay::kRawTile +
                           ctid * 16;
      uint8_t* d = smem + dst + my_dst;
#pragma unroll
      for (int i = 0; i < kKeys / kRowStep; ++i) {
        uint4 w = *reinterpret_cast<const uint4*>(raw + i * kConvThreads * 16);
        if (my_row + i * kRowStep >= limit) w = make_uint4(0u, 0u, 0u, 0u);
        const uint4 lo = make_uint4(
            dev::e4m3x2_to_f16x2(w.x), dev::e4m3x2_to_f16x2_hi(w.x),
            dev::e4m3x2_to_f16x2(w.y), dev::e4m3x2_to_f16x2_hi(w.y));
        const uint4 hi = make_uint4(
            dev::e4m3x2_to_f16x2(w.z), dev::e4m3x2_to_f16x2_hi(w.z),
            dev::e4m3x2_to_f16x2(w.w), dev::e4m3x2_to_f16x2_hi(w.w));
        *reinterpret_cast<uint4*>(d + i * kRowStep * 128 + my_a) =
            swap ? hi : lo;
        *reinterpret_cast<uint4*>(d + i * kRowStep * 128 + my_b) =
            swap ? lo : hi;
      }
      dev::fence_proxy_async_smem();  // visible to the tensor cores
      __syncwarp();
      if (lane == 0) {
        dev::mbar_arrive(full);
        dev::mbar_arrive(raw_empty0 + 8 * slot);
      }
      ++u;
      return true;
    };
    for (int n = 0; ok; ++n) {
      Item it;
      ok = next_item(n, it);
      if (!ok || it.state == kEnd) break;
      if (it.state == kSkip) continue;
      const Span sp = span_of(it);
      for (int t = 0; ok && t <= sp.n_tiles; ++t) {
        if (t < sp.n_tiles)
          ok = convert(Lay::kOffK, k_full, k_empty, g + t, kKeys);
        if (ok && t >= 1)
          ok = convert(Lay::kOffV, v_full, v_empty, g + t - 1,
                       it.L - (t - 1) * kKeys);
      }
      g += sp.n_tiles;
    }
    if (!ok) dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
    return;
  }

  // ---------------- softmax warps (thread = query row) ----------------
  regs_inc<kSoftmaxRegs>();
  const int quarter = warp;  // tensor-memory lane quarter of this warp
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const int r = quarter * 32 + lane;
  const int t_loc = r / G;
  const int hg = r - t_loc * G;
  auto wait_pv = [&](uint32_t t) {
    return __all_sync(0xffffffffu, dev::mbar_wait(o_ready, t & 1));
  };
  bool ok = true;
  uint32_t g = 0;
  int v = 0;
  for (int n = 0; ok; ++n) {
    Item it;
    ok = next_item(n, it);
    if (!ok || it.state == kEnd) break;
    if (it.state == kSkip) continue;
    const Span sp = span_of(it);
    const int tok = sp.tok0 + t_loc;
    const bool valid = t_loc < sp.n_q;
    const int qpos = valid ? it.L - it.q_len + tok : sp.kv_end - 1;
    const bool idle = quarter * 32 >= sp.n_q * G;
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
      if (v >= 1 && !__all_sync(0xffffffffu,
                                dev::mbar_wait(q_empty, (v - 1) & 1))) {
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
          const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top = __vmaxu2(top, x[e] & 0x7fff7fffu);
        }
        const float2 top2 = dev::Mma<T>::unpack(top);
        const float amax = fmaxf(top2.x, top2.y);
        const int k = min(14 - dev::floor_log2(amax), 100);
        // a negative scale turns the sign of q, so that scores can be
        // compared before they are scaled
        const float up =
            a.scale_log2 < 0.f ? -dev::exp2_int(k) : dev::exp2_int(k);
        c_row = fabsf(a.scale_log2) * dev::exp2_int(-k);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = dev::Mma<T>::unpack(x[e]);
            y[e] = M::pack(f.x * up, f.y * up);
          }
          *reinterpret_cast<uint4*>(smem + Lay::kOffQ +
                                    (i >> 3) * Lay::kHalfQ + r * 128 +
                                    (((i & 7) ^ (r & 7)) << 4)) =
              make_uint4(y[0], y[1], y[2], y[3]);
        }
        dev::fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(q_full);
      ++v;
    }
    float m_ref = -INFINITY, l = 0.f;
    int e_ref = 0;  // E
    for (int j = 0; j < sp.n_tiles && ok; ++j) {
      const uint32_t t = g + j;
      ok = __all_sync(0xffffffffu, dev::mbar_wait(s_full, t & 1));
      if (!ok) break;
      float sv[kKeys];
      if (!idle) {
        dev::tc_fence_after();
        const uint32_t sa = s_tmem + lane_off;
        float (&lo)[32] = *reinterpret_cast<float(*)[32]>(sv);
        float (&hi)[32] = *reinterpret_cast<float(*)[32]>(sv + 32);
        dev::tmem_ld32(sa, lo);
        dev::tmem_ld32(sa + 32, hi);
        dev::tmem_ld_wait();
        dev::tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(s_free);
      if (idle) {
        // Arrives for tile t only once P(t-1).V is done: an arrival a tile
        // ahead would count toward tile t-1 on the single p_full barrier.
        if (t >= 1 && !wait_pv(t - 1)) {
          ok = false;
          break;
        }
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(p_full);
        continue;
      }
      const int k0 = j * kKeys;
      const int lim = qpos - k0;
      if (lim < kKeys - 1) {
#pragma unroll
        for (int k = 0; k < kKeys; ++k)
          if (k > lim) sv[k] = -INFINITY;
      }
      // The tile's scales: a factor and an exponent per block.
      float cb[kNB], lv[kNB];
      const float* sc = scale_s + (t % kScaleSlots) * 8;
      float mx = -INFINITY, top = -100.f;
#pragma unroll
      for (int b = 0; b < kNB; ++b) {
        cb[b] = fmaxf(c_row * sc[b], 1.1754944e-38f);  // -inf * 0 is NaN
        lv[b] = sc[kNB + b];
        top = fmaxf(top, lv[b]);
        float m4[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          m4[u] = dev::fmax3(sv[b * BS + u], sv[b * BS + 4 + u],
                             sv[b * BS + 8 + u]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          m4[u] = fmaxf(m4[u], sv[b * BS + 12 + u]);
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
      float factor = 1.f;
      const int e_top = static_cast<int>(floorf(top));
      if (j == 0) {
        m_ref = mx;  // O is still empty: the first P.V overwrites it
        e_ref = e_top;
      } else {
        if (mx > m_ref + kRescaleLog2) {
          factor = dev::fast_exp2(m_ref - mx);
          m_ref = mx;
          l *= factor;
        }
        if (e_top > e_ref + kVsSlack) {
          factor *= dev::exp2_int(max(e_ref - e_top, -126));
          e_ref = e_top;
        }
      }
      if (__any_sync(0xffffffffu, factor != 1.f)) {
        ok = wait_pv(t - 1);
        if (!ok) break;
        dev::tc_fence_after();
        // Rare (the maxima settle): a rolled loop over 16 columns, which
        // leaves the scores in their registers.
#pragma unroll 1
        for (int col = 0; col < D; col += 16) {
          uint32_t ov[16];
          dev::tmem_ld16u(o_tmem + lane_off + col, ov);
          dev::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            ov[e] = __float_as_uint(__uint_as_float(ov[e]) * factor);
          dev::tmem_st16u(o_tmem + lane_off + col, ov);
        }
        dev::tmem_st_wait();
      }
      // w = 2^(s c_b + log2(vs_b) - E + shift - m), two keys per
      // instruction; the sum of p from the block sums of w.
      {
        uint32_t hw[kKeys / 2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int b = h * kNB / 2; b < (h + 1) * kNB / 2; ++b) {
            const float lvn =
                fmaxf(lv[b] - static_cast<float>(e_ref), -96.f) + kShift;
            const float off = lvn - m_ref;
            const float2 c2 = make_float2(cb[b], cb[b]);
            const float2 o2 = make_float2(off, off);
            float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int e = b * BS / 2; e < (b + 1) * BS / 2; ++e) {
              const float2 x =
                  dev::ffma2(make_float2(sv[2 * e], sv[2 * e + 1]), c2, o2);
              const float w0 = dev::fast_exp2(x.x), w1 = dev::fast_exp2(x.y);
              l2[e & 1] = dev::fadd2(l2[e & 1], make_float2(w0, w1));
              hw[e] = M::pack(w0, w1);
            }
            const float2 lb = dev::fadd2(l2[0], l2[1]);
            l = fmaf(lb.x + lb.y, dev::fast_exp2(-lvn), l);
          }
          if (h == 0) {
            // P(t-1).V must have read the P buffer before it is overwritten.
            if (t >= 1 && !wait_pv(t - 1)) ok = false;
            if (!ok) break;
            dev::tc_fence_after();
          }
          dev::tmem_st16u(
              p_tmem + lane_off + 16 * h,
              *reinterpret_cast<const uint32_t(*)[16]>(hw + 16 * h));
        }
      }
      if (!ok) break;
      dev::tmem_st_wait();
      dev::tc_fence_before();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(p_full);
    }
    // The item's output: O 2^(E - shift) / l -> out[token, query head].
    if (ok && !idle) ok = wait_pv(g + sp.n_tiles - 1);
    if (ok && !idle) {
      dev::tc_fence_after();
      // l is above 0 (each row sees a key) or NaN, which is passed on
      const float inv = dev::exp2_int(e_ref - static_cast<int>(kShift)) / l;
      T* dst = static_cast<T*>(a.out) + row_at;
      float* dst32 = static_cast<float*>(a.out) + row_at;  // out_f32 only
#pragma unroll
      for (int col = 0; col < D; col += 32) {
        float ov[32];
        dev::tmem_ld32(o_tmem + lane_off + col, ov);
        dev::tmem_ld_wait();
        if (valid && a.out_f32) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(dst32 + col + e) =
                make_float4(ov[e] * inv, ov[e + 1] * inv, ov[e + 2] * inv,
                            ov[e + 3] * inv);
        } else if (valid) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 w;
            w.x = dev::Mma<T>::pack(ov[e] * inv, ov[e + 1] * inv);
            w.y = dev::Mma<T>::pack(ov[e + 2] * inv, ov[e + 3] * inv);
            w.z = dev::Mma<T>::pack(ov[e + 4] * inv, ov[e + 5] * inv);
            w.w = dev::Mma<T>::pack(ov[e + 6] * inv, ov[e + 7] * inv);
            *reinterpret_cast<uint4*>(dst + col + e) = w;
          }
        }
      }
    }
    g += sp.n_tiles;
  }
  if (!ok) dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
  dev::tc_fence_before();
  __syncwarp();
  if (lane == 0) dev::mbar_arrive(done);
}

// ---------------------------------------------------------------------------
// Host side.

template <typename T, int BS, int G, int D>
pa_status launch(const PrefillQ8Args& a, cudaStream_t st) {
  auto kern = prefill_q8_kernel<T, BS, G, D>;
  const size_t smem = LayoutQ8<D>::kSmemBytes;
  // The warpgroups' shares of the registers assume kLaunchRegs a thread.
  cudaFuncAttributes attrs;
  cudaError_t e = cudaFuncGetAttributes(&attrs, kern);
  if (e != cudaSuccess || attrs.numRegs != kLaunchRegs)
    return fail(PA_ERR_CUDA, "pa_prefill_q8: built with %d registers, not %d",
                e == cudaSuccess ? attrs.numRegs : -1, kLaunchRegs);
  e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
      static_cast<int>(smem));
  if (e != cudaSuccess)
    return fail(PA_ERR_CUDA, "pa_prefill_q8: cudaFuncSetAttribute(%zu): %s",
                smem, cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  const int64_t slots = 2LL * std::max(device_sm_count(), 1);
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

template <typename T, int BS, int D>
pa_status dispatch_group(const pa_prefill_desc* d, const PrefillQ8Args& a,
                         cudaStream_t st) {
  switch (d->num_q_heads / d->num_kv_heads) {
    case 1: return launch<T, BS, 1, D>(a, st);
    case 2: return launch<T, BS, 2, D>(a, st);
    case 4: return launch<T, BS, 4, D>(a, st);
    default: return launch<T, BS, 8, D>(a, st);
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
  a.num_items = static_cast<int>(pagedkv::tile_cap(d) * d->num_kv_heads);
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
                           max_ctx, workspace, dev_err, s);
  if (planned != PA_OK) return planned;
  return d->dtype == PA_BF16
             ? pagedkv::dispatch_shape<__nv_bfloat16>(d, a, s)
             : pagedkv::dispatch_shape<__half>(d, a, s);
}
