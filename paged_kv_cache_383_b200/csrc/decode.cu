// Paged decode attention for sm_100a: pa_decode and its partition reduce.
//
// What is computed ([Taming the Tail] "Under the Hood: The CUDA Kernel
// Engineering"; [KV-cache chapter] "PagedAttention: borrowing virtual memory
// ..." and "Common misconception..."): for each sequence b and query head h,
// softmax(scale * K_b q) V_b over the sequence's tokens, K_b / V_b gathered
// block by block through the block table.  The pages ask three things of the
// kernel: look the physical block up in the table, keep the accesses
// coalesced despite the scattered blocks, and handle a partly filled last
// block.  Their sketch (one fp32 element per thread) is prior art only.
//
// B200 design.
//  * Work unit = (partition of <= partition_size tokens, KV head, sequence):
//    one CTA.  All G = Hq/Hkv query heads of the KV head are served by the
//    same CTA, so each K/V byte leaves HBM once.
//  * Warp 0, lane 0 is the producer.  It stages the unit's slice of the block
//    table in shared memory and issues 2-D TMA tile loads of whole pages
//    (block_size rows x 128 B, 128-byte swizzle, no multicast) into an
//    S-stage ring, each stage one K page + one V page, signalled by mbarriers
//    with transaction counts.  Waits are bounded (1 s) and report
//    PA_ERR_DEVICE_TIMEOUT instead of hanging.
//  * Warps 1..4 are consumers; consumer w takes pages w, w+4, ... and keeps
//    its own online-softmax state (running max m, sum l, accumulator o) for
//    all G heads.  At the end the four states are merged through shared
//    memory.
//  * Compute variant MMA (default): S^T = K_page . Q^T and O^T += V^T . P^T as
//    m16n8k16 tensor-core MMAs, N = 8 = the (padded) query-head group.  K
//    fragments come from ldmatrix, V fragments from ldmatrix.trans, P moves
//    from the score accumulator layout to the B-operand layout with
//    movmatrix.  P is split into a rounded part and its residual (two
//    16-bit operands) so PV keeps ~16 mantissa bits; accumulation is fp32.
//  * Compute variant SIMT: fp32 FMA dot products on the CUDA cores (kept to
//    show what the tensor-core mapping buys).
//  * A sequence that needs more than one partition writes (m, l, o/l) per
//    partition to the workspace.  With at most 16 partitions the partition
//    CTA that finishes last combines them (fence + ticket, nobody waits);
//    otherwise, or on request, a separate reduce kernel does.  A sequence
//    that fits one partition is written straight to `out`.
//  * With the reduce kernel and partitions of <= 1024 tokens, a CTA serves
//    four consecutive partitions, one per consumer warp (pages interleaved
//    so each warp still owns its ring stages): no cross-warp merge.
//  * A one-CTA prep kernel runs first: it orders the sequences longest
//    first (grid row z serves order[z], so the grid ends on short work) and
//    resets the partition counters.  Kernels are chained by programmatic
//    dependent launch.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "decode_common.cuh"
#include "device_utils.cuh"
#include "pagedkv.h"
#include "status.h"

// Built-in scratch for pa_decode_noalloc: a fixed device array that lives in
// this library's module on every GPU that loads it, for callers that cannot
// allocate device memory.  In host code this name is only a stand-in, not a
// device address: scratch_address() below asks the runtime for the address,
// once per CUDA context.
static __device__ __align__(256) unsigned char
    g_noalloc_scratch[PA_NOALLOC_SCRATCH_BYTES];

namespace pagedkv {
namespace {

// Shared-memory geometry of one (block_size, head_dim, stages) instance.
// A page (one block, one KV head) is head_dim/64 TMA boxes of block_size
// rows x 128 bytes; within a box, 16-byte chunk c of row r sits at chunk
// c ^ (r % 8) (the TMA 128-byte swizzle), so eight consecutive rows read at
// the same logical chunk hit eight different bank groups.
template <int BS, int D, int S>
struct Geometry {
  // Consumer warp w takes pages w, w+4, ... and page i sits in stage i % S.
  // With S a multiple of the consumer count a warp owns its stages, so it
  // waits on every use of them in order and a parity wait can never run two
  // phases ahead (a parity test cannot tell phase m from m-2).
  static_assert(S % kConsumers == 0, "stages must be a multiple of consumers");
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = BS * 128;
  static constexpr int kPageBytes = kBoxes * kBoxBytes;
  static constexpr int kStageBytes = 2 * kPageBytes;  // K page then V page
  static constexpr int kRingBytes = S * kStageBytes;
  static constexpr int kBarBytes = 2 * S * 8;         // full[S], empty[S]
  // Per consumer warp: o[8][kORow], m[8], l[8] (fp32); aliases the ring.
  // Rows are padded by 4 floats so the four head pairs a warp writes at
  // once land in different banks.
  static constexpr int kORow = D + 4;
  static constexpr int kEpiWarpFloats = kMaxGroup * kORow + 2 * kMaxGroup;
  static_assert(kConsumers * kEpiWarpFloats * 4 <= kRingBytes,
                "epilogue must fit in the ring");
  // SIMT scratch: q in fp32 with a 4-float skew between the two halves of a
  // row (bank spread), then per warp scores[BS][8], alpha[8], m_new[8].
  static constexpr int kQRow = D + 8;
  static constexpr int kSimtQFloats = kMaxGroup * kQRow;
  static constexpr int kSimtWarpFloats = BS * kMaxGroup + 2 * kMaxGroup;
  static constexpr int kSimtBytes =
      (kSimtQFloats + kConsumers * kSimtWarpFloats) * 4;

  // Byte offset of element (row, col) inside a page.
  static __device__ __forceinline__ uint32_t offset(int row, int col) {
    return (col >> 6) * kBoxBytes + row * 128 +
           ((((col & 63) >> 3) ^ (row & 7)) << 4) + (col & 7) * 2;
  }
};

// Bytes of the staged block-table slice, rounded to 16.
__host__ __device__ constexpr int bt_bytes(int pages_per_part) {
  return (pages_per_part * 4 + 15) & ~15;
}

// Dynamic shared memory of one CTA: alignment slack, ring, barriers, the
// block-table slice and (SIMT only) the fp32 scratch.
template <int BS, int D, int S, bool kMma>
constexpr size_t smem_bytes_for(int pages_per_part) {
  using G = Geometry<BS, D, S>;
  return 1024 + G::kRingBytes + G::kBarBytes + bt_bytes(pages_per_part) +
         (kMma ? 0 : G::kSimtBytes);
}

// ---------------------------------------------------------------------------
// The decode kernel.
template <typename T, int BS, int D, int S, bool kMma>
__global__ void __launch_bounds__(kThreads)
    decode_kernel(const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap,
                  const DecodeArgs a) {
  using Geo = Geometry<BS, D, S>;
  extern __shared__ uint8_t smem_dyn[];
  // The TMA swizzle is a function of shared-memory address bits, so the ring
  // must start on a 1024-byte boundary of the shared window.
  uint8_t* smem = smem_dyn + ((1024u - (dev::smem_u32(smem_dyn) & 1023u)) & 1023u);

  // Partitions this CTA serves: one, or (warp_parts) kConsumers consecutive
  // ones, consumer warp w taking partition part + w.
  const int nsub = a.warp_parts ? kConsumers : 1;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  dev::pdl_trigger();  // the reduce may start its prologue early
  // Grid rows are handed out longest first (the order the prep kernel wrote,
  // which this grid may only read after waiting for it), so the last CTAs
  // to start are short ones and the tail of the grid is short: partition
  // units by their token count (all KV heads of a unit side by side), or
  // sequences by length (their partitions side by side).
  int part, kvh, b;
  if (a.units) {
    kvh = blockIdx.x;
    dev::pdl_wait();
    const int u = a.units[blockIdx.y];
    b = u / a.max_parts;
    part = u - b * a.max_parts;
  } else {
    part = blockIdx.x * nsub;
    kvh = blockIdx.y;
    b = blockIdx.z;
    if (a.order) {
      dev::pdl_wait();
      b = a.order[blockIdx.z];
    }
  }
  const int PS = a.partition_size;
  const int pages_per_part = PS / BS;
  const int page0 = part * pages_per_part;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Geo::kRingBytes);
  int32_t* bt_s = reinterpret_cast<int32_t*>(bars + 2 * S);
  const uint32_t ring = dev::smem_u32(smem);
  const uint32_t full0 = dev::smem_u32(bars);
  const uint32_t empty0 = full0 + S * 8;

  // The context length and this partition's slice of the block table are
  // fetched together: the slice is read as if the partition were full (clipped
  // to the table row) so the two loads do not wait on each other; entries past
  // the sequence's end are never used.
  const int32_t* bt_row =
      a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq + page0;
  const int row_left = a.max_blocks_per_seq - page0;
  const int ctx = a.context_lens[b];
  for (int i = tid; i < nsub * pages_per_part && i < row_left; i += kThreads)
    bt_s[i] = bt_row[i];
  if (ctx < 0 || ctx > a.max_blocks_per_seq * BS || ctx > a.max_context_len) {
    if (part == 0 && kvh == 0 && tid == 0)
      dev::set_error(a.dev_err, PA_ERR_DEVICE_OOB);
    return;
  }
  const int n_parts = ctx > 0 ? (ctx + PS - 1) / PS : 1;
  if (part >= n_parts) return;
  const int tok0 = part * PS;
  // Tokens (and staged pages) of this CTA's partitions; 0 only when ctx == 0.
  const int n_tok = min(ctx - tok0, nsub * PS);
  const int n_pages = (n_tok + BS - 1) / BS;
  const int G = a.group;

  // Check every block id the partition uses (each thread the entries it
  // staged itself).
  int bad = 0;
  for (int i = tid; i < n_pages; i += kThreads)
    bad |= (bt_s[i] < 0 || bt_s[i] >= a.num_blocks);
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      dev::mbar_init(full0 + s * 8, 1);
      dev::mbar_init(empty0 + s * 8, 1);
    }
    dev::fence_mbar_init();
  }
  bad = __syncthreads_or(bad);
  // Everything above reads only host-written inputs; the K/V pages and the
  // outputs may belong to the previous kernel in the stream.
  dev::pdl_wait();
  __shared__ int s_last;
  if (bad) {
    if (tid == 0) dev::set_error(a.dev_err, PA_ERR_DEVICE_OOB);
    if (n_parts > 1) {
      // mark the CTA's partitions empty for the combine
      for (int k = 0; k < nsub && part + k < n_parts; ++k)
        if (tid < G) {
          const int64_t row =
              (static_cast<int64_t>(b) * a.num_q_heads + kvh * G + tid) *
                  a.max_parts + part + k;
          a.ws_ml[2 * row] = -INFINITY;
          a.ws_ml[2 * row + 1] = 0.f;
        }
      if (a.fused) {  // still counts as finished: the others may be fine
        __threadfence();
        __syncthreads();
        if (tid == 0)
          s_last = atomicAdd(a.counters + b * a.num_kv_heads + kvh, 1) ==
                   n_parts - 1;
        __syncthreads();
        if (s_last) {
          __threadfence();
          combine_partials<T, D>(a, b, kvh, n_parts, tid, kThreads);
        }
      }
    }
    return;
  }

  // ---------------- producer ----------------
  if (warp == 0) {
    if (lane == 0 && n_pages > 0) {
      dev::prefetch_tmap(&kmap);
      dev::prefetch_tmap(&vmap);
      // warp_parts: pages are interleaved across the partitions (index i is
      // page i / kConsumers of partition i % kConsumers), so consumer warp w
      // still gets every page i = w (mod kConsumers) and owns its stages;
      // pages past a shorter partition's end are skipped, which only ever
      // stops the reuse of that warp's stages.
      const int n_iter =
          a.warp_parts ? kConsumers * min(n_pages, pages_per_part) : n_pages;
      for (int i = 0; i < n_iter; ++i) {
        int slot = i;
        if (a.warp_parts) {
          slot = (i % kConsumers) * pages_per_part + i / kConsumers;
          if (slot >= n_pages) continue;
        }
        const int s = i % S;
        if (i >= S && !dev::mbar_wait(empty0 + s * 8, ((i / S) - 1) & 1)) {
          dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
          break;
        }
        const uint32_t full = full0 + s * 8;
        dev::mbar_arrive_expect_tx(full, Geo::kStageBytes);
        const int y = (bt_s[slot] * a.num_kv_heads + kvh) * BS;
        const uint32_t kdst = ring + s * Geo::kStageBytes;
#pragma unroll
        for (int bx = 0; bx < Geo::kBoxes; ++bx) {
          dev::tma_load_2d(kdst + bx * Geo::kBoxBytes, &kmap, bx * 64, y, full);
          dev::tma_load_2d(kdst + Geo::kPageBytes + bx * Geo::kBoxBytes, &vmap,
                           bx * 64, y, full);
        }
      }
    }
    return;
  }

  // ---------------- consumers ----------------
  const int cw = warp - 1;
  const int ctid = tid - 32;  // 0 .. kConsumers*32-1
  const T* qrow = static_cast<const T*>(a.q) +
                  (static_cast<int64_t>(b) * a.num_q_heads + kvh * G) * D;
  float m_fin[2], l_fin[2];  // per-lane head state handed to the epilogue

  if constexpr (kMma) {
    using M = dev::Mma<T>;
    const int g4 = lane >> 2;  // fragment row group
    const int t4 = lane & 3;   // thread in group
    // B fragments of Q^T (K = head_dim, N = 8 heads): head g4, dims
    // kk*16 + 2*t4 (+1) and +8.  Heads past G are zero.
    uint32_t qf[D / 16][2];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        qf[kk][r] = 0u;
        if (g4 < G)
          qf[kk][r] = *reinterpret_cast<const uint32_t*>(
              qrow + g4 * D + kk * 16 + r * 8 + 2 * t4);
      }
    }
    float o[D / 16][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY};
    float l_run[2] = {0.f, 0.f};

    // ldmatrix lane roles: matrix mi = lane/8, row j = lane%8.
    const int mi = lane >> 3;
    const int j = lane & 7;

    // Tokens this warp's pages cover: the CTA's partition (the warps share
    // it), or with warp_parts this warp's own partition part + cw.
    const int w_tok = a.warp_parts ? max(0, min(n_tok - cw * PS, PS)) : n_tok;
    const int w_iter =
        a.warp_parts ? kConsumers * ((w_tok + BS - 1) / BS) : n_pages;
    for (int i = cw; i < w_iter; i += kConsumers) {
      const int s = i % S;
      if (!dev::mbar_wait(full0 + s * 8, (i / S) & 1)) {
        dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
        break;
      }
      const uint32_t kb = ring + s * Geo::kStageBytes;
      const uint32_t vb = kb + Geo::kPageBytes;
      const int pg = a.warp_parts ? i / kConsumers : i;  // page of w_tok
      const int nv = min(BS, w_tok - pg * BS);
      if (nv < BS) {
        // Slots past the context get P = 0, but 0 * NaN is NaN in the MMA:
        // clear the V rows the sequence never wrote (last page only).
        for (int idx = lane; idx < (BS - nv) * Geo::kBoxes * 8; idx += 32) {
          const int row = nv + idx / (Geo::kBoxes * 8);
          const int c = idx % (Geo::kBoxes * 8);
          dev::st_shared_zero16(vb + (c >> 3) * Geo::kBoxBytes + row * 128 +
                                (c & 7) * 16);
        }
        dev::fence_proxy_async_smem();  // before TMA reuses the stage
        __syncwarp();
      }

      // S^T (tokens x heads) for each 16-token slice of the page.
      float sc[BS / 16][4];
#pragma unroll
      for (int mt = 0; mt < BS / 16; ++mt) {
        float acc0[4] = {0.f, 0.f, 0.f, 0.f};
        float acc1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t af[4];
          dev::ldsm_x4(kb + Geo::offset(mt * 16 + j + (mi & 1) * 8,
                                        kk * 16 + (mi >> 1) * 8),
                       af);
          if (kk & 1)
            M::run(acc1, af, qf[kk][0], qf[kk][1]);
          else
            M::run(acc0, af, qf[kk][0], qf[kk][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = mt * 16 + g4 + (e >> 1) * 8;
          const float x = (acc0[e] + acc1[e]) * a.scale_log2;
          sc[mt][e] = tok < nv ? x : -INFINITY;
        }
      }
      // Online softmax; this lane holds heads 2*t4 and 2*t4+1.
      float alpha[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < BS / 16; ++mt)
          mx = fmaxf(mx, fmaxf(sc[mt][h], sc[mt][h + 2]));
        mx = warp_max_xor(mx, 4, 16);
        const float m_new = fmaxf(m_run[h], mx);
        alpha[h] = dev::fast_exp2(m_run[h] - m_new);
        float sum = 0.f;
#pragma unroll
        for (int mt = 0; mt < BS / 16; ++mt) {
          sc[mt][h] = dev::fast_exp2(sc[mt][h] - m_new);
          sc[mt][h + 2] = dev::fast_exp2(sc[mt][h + 2] - m_new);
          sum += sc[mt][h] + sc[mt][h + 2];
        }
        l_run[h] = l_run[h] * alpha[h] + sum;
        m_run[h] = m_new;
      }
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[dt][e] *= alpha[e & 1];

      // P^T as B fragments (K = tokens, N = heads): rounded part and residual.
      uint32_t bh[BS / 16][2], bl[BS / 16][2];
#pragma unroll
      for (int ks = 0; ks < BS / 16; ++ks) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p0 = sc[ks][2 * r], p1 = sc[ks][2 * r + 1];
          const uint32_t hi = M::pack(p0, p1);
          const float2 hf = M::unpack(hi);
          const uint32_t lo = M::pack(p0 - hf.x, p1 - hf.y);
          bh[ks][r] = dev::movmatrix_trans(hi);
          bl[ks][r] = dev::movmatrix_trans(lo);
        }
      }
      // O^T (head_dim x heads) += V^T . P^T
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) {
#pragma unroll
        for (int ks = 0; ks < BS / 16; ++ks) {
          uint32_t af[4];
          dev::ldsm_x4_trans(vb + Geo::offset(ks * 16 + j + (mi >> 1) * 8,
                                              dt * 16 + (mi & 1) * 8),
                             af);
          M::run(o[dt], af, bh[ks][0], bh[ks][1]);
          M::run(o[dt], af, bl[ks][0], bl[ks][1]);
        }
      }
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(empty0 + s * 8);
    }

    if (a.warp_parts) {
      // This warp's partition is complete: write its partial directly
      // (no merge with the other warps, which hold other partitions).
      const int mypart = part + cw;
      if (mypart < n_parts) {
        float lt[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float l = l_run[h];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          lt[h] = l;
        }
        const int64_t row0 =
            static_cast<int64_t>(b) * a.num_q_heads + kvh * G;
        if (n_parts == 1) {
          // The reduce kernel skips single-partition rows: write the output.
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int g = 2 * t4 + (e & 1);
              if (g < G) {
                const float l = lt[e & 1];
                store_out<T>(a, (row0 + g) * D + dt * 16 + g4 + (e >> 1) * 8,
                             l > 0.f ? o[dt][e] / l : 0.f);
              }
            }
          return;
        }
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int g = 2 * t4 + (e & 1);
            if (g < G) {
              const int64_t row = (row0 + g) * a.max_parts + mypart;
              const float l = lt[e & 1];
              a.ws_o[row * D + dt * 16 + g4 + (e >> 1) * 8] =
                  l > 0.f ? o[dt][e] / l : 0.f;
            }
          }
        if (g4 == 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int g = 2 * t4 + h;
            if (g < G) {
              const int64_t row = (row0 + g) * a.max_parts + mypart;
              a.ws_ml[2 * row] = m_run[h];
              a.ws_ml[2 * row + 1] = lt[h];
            }
          }
        }
      }
      return;
    }
    // Hand this warp's state to the epilogue area (aliases the ring).
    dev::named_barrier(1, kConsumers * 32);
    float* ep = reinterpret_cast<float*>(smem) + cw * Geo::kEpiWarpFloats;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float l = l_run[h];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      m_fin[h] = m_run[h];
      l_fin[h] = l;
    }
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        ep[(2 * t4 + (e & 1)) * Geo::kORow + dt * 16 + g4 + (e >> 1) * 8] =
            o[dt][e];
    if (g4 == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ep[kMaxGroup * Geo::kORow + 2 * t4 + h] = m_fin[h];
        ep[kMaxGroup * Geo::kORow + kMaxGroup + 2 * t4 + h] = l_fin[h];
      }
    }
  } else {
    // ---------------- SIMT variant ----------------
    float* q_s = reinterpret_cast<float*>(
        reinterpret_cast<uint8_t*>(bt_s) + bt_bytes(PS / BS));
    float* wsp = q_s + Geo::kSimtQFloats + cw * Geo::kSimtWarpFloats;
    float* sp = wsp;                      // scores / probabilities [BS][8]
    float* alpha_s = wsp + BS * kMaxGroup;
    float* mnew_s = alpha_s + kMaxGroup;

    // q -> fp32 shared copy; half h of a row is skewed by 4h floats.
    for (int idx = ctid; idx < kMaxGroup * D; idx += kConsumers * 32) {
      const int g = idx / D, d = idx % D;
      const float v = g < G ? to_float<T>(qrow[g * D + d]) : 0.f;
      q_s[g * Geo::kQRow + d + (d >= D / 2 ? 4 : 0)] = v;
    }
    dev::named_barrier(1, kConsumers * 32);

    // QK roles: BS=16 -> token lane%16, half lane/16; BS=32 -> token lane.
    constexpr int kHalves = 32 / BS;       // 2 or 1
    constexpr int kDPer = D / kHalves;     // dims per lane in QK
    const int qtok = lane % BS;
    const int qhalf = lane / BS;
    // PV roles: lane owns dims [lane*D/32, +D/32).
    constexpr int kDPV = D / 32;           // 4 or 2
    const int d0 = lane * kDPV;

    float acc_o[kMaxGroup][kDPV];
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g)
#pragma unroll
      for (int e = 0; e < kDPV; ++e) acc_o[g][e] = 0.f;
    float m_run = -INFINITY, l_run = 0.f;  // lanes 0..7: head `lane`

    for (int i = cw; i < n_pages; i += kConsumers) {
      const int s = i % S;
      if (!dev::mbar_wait(full0 + s * 8, (i / S) & 1)) {
        dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
        break;
      }
      const uint8_t* kpg = smem + s * Geo::kStageBytes;
      const uint8_t* vpg = kpg + Geo::kPageBytes;
      const int nv = min(BS, n_tok - i * BS);

      float acc[kMaxGroup];
#pragma unroll
      for (int g = 0; g < kMaxGroup; ++g) acc[g] = 0.f;
#pragma unroll 2
      for (int c = 0; c < kDPer / 8; ++c) {
        const int d = qhalf * kDPer + c * 8;
        const uint4 raw = *reinterpret_cast<const uint4*>(
            kpg + Geo::offset(qtok, d));
        const T* kv = reinterpret_cast<const T*>(&raw);
        float kf[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) kf[e] = to_float<T>(kv[e]);
        const float* qd = q_s + d + (d >= D / 2 ? 4 : 0);
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) {
          const float4 qa = *reinterpret_cast<const float4*>(qd + g * Geo::kQRow);
          const float4 qb =
              *reinterpret_cast<const float4*>(qd + g * Geo::kQRow + 4);
          acc[g] += qa.x * kf[0] + qa.y * kf[1] + qa.z * kf[2] + qa.w * kf[3] +
                    qb.x * kf[4] + qb.y * kf[5] + qb.z * kf[6] + qb.w * kf[7];
        }
      }
      if (kHalves == 2) {
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g)
          acc[g] += __shfl_xor_sync(0xffffffffu, acc[g], 16);
      }
      if (qhalf == 0) {
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g)
          sp[qtok * kMaxGroup + g] =
              qtok < nv ? acc[g] * a.scale_log2 : -INFINITY;
      }
      __syncwarp();
      if (lane < kMaxGroup) {
        float mx = -INFINITY;
        for (int t = 0; t < BS; ++t) mx = fmaxf(mx, sp[t * kMaxGroup + lane]);
        const float m_new = fmaxf(m_run, mx);
        alpha_s[lane] = dev::fast_exp2(m_run - m_new);
        mnew_s[lane] = m_new;
        m_run = m_new;
      }
      __syncwarp();
      for (int idx = lane; idx < BS * kMaxGroup; idx += 32)
        sp[idx] = dev::fast_exp2(sp[idx] - mnew_s[idx % kMaxGroup]);
      __syncwarp();
      if (lane < kMaxGroup) {
        float sum = 0.f;
        for (int t = 0; t < BS; ++t) sum += sp[t * kMaxGroup + lane];
        l_run = l_run * alpha_s[lane] + sum;
      }
#pragma unroll
      for (int g = 0; g < kMaxGroup; ++g) {
        const float al = alpha_s[g];
#pragma unroll
        for (int e = 0; e < kDPV; ++e) acc_o[g][e] *= al;
      }
      for (int t = 0; t < nv; ++t) {
        float vf[kDPV];
        if constexpr (kDPV == 4) {
          const uint2 raw = *reinterpret_cast<const uint2*>(
              vpg + Geo::offset(t, d0));
          const T* vv = reinterpret_cast<const T*>(&raw);
#pragma unroll
          for (int e = 0; e < 4; ++e) vf[e] = to_float<T>(vv[e]);
        } else {
          const uint32_t raw = *reinterpret_cast<const uint32_t*>(
              vpg + Geo::offset(t, d0));
          const T* vv = reinterpret_cast<const T*>(&raw);
#pragma unroll
          for (int e = 0; e < 2; ++e) vf[e] = to_float<T>(vv[e]);
        }
        const float4 pa =
            *reinterpret_cast<const float4*>(sp + t * kMaxGroup);
        const float4 pb =
            *reinterpret_cast<const float4*>(sp + t * kMaxGroup + 4);
        const float p[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g)
#pragma unroll
          for (int e = 0; e < kDPV; ++e) acc_o[g][e] += p[g] * vf[e];
      }
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(empty0 + s * 8);
    }

    dev::named_barrier(1, kConsumers * 32);
    float* ep = reinterpret_cast<float*>(smem) + cw * Geo::kEpiWarpFloats;
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g)
#pragma unroll
      for (int e = 0; e < kDPV; ++e)
        ep[g * Geo::kORow + d0 + e] = acc_o[g][e];
    if (lane < kMaxGroup) {
      ep[kMaxGroup * Geo::kORow + lane] = m_run;
      ep[kMaxGroup * Geo::kORow + kMaxGroup + lane] = l_run;
    }
    (void)m_fin;
    (void)l_fin;
  }

  // ---------------- merge the consumer warps, write the result -------------
  dev::named_barrier(1, kConsumers * 32);
  const float* ep0 = reinterpret_cast<const float*>(smem);
  const bool split = n_parts > 1;
  for (int idx = ctid; idx < G * D; idx += kConsumers * 32) {
    const int g = idx / D, d = idx % D;
    float mmax = -INFINITY;
#pragma unroll
    for (int w = 0; w < kConsumers; ++w)
      mmax = fmaxf(mmax,
                   ep0[w * Geo::kEpiWarpFloats + kMaxGroup * Geo::kORow + g]);
    float val = 0.f, wsum = 0.f;
    if (mmax != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) {
        const float* e = ep0 + w * Geo::kEpiWarpFloats;
        const float mw = e[kMaxGroup * Geo::kORow + g];
        const float sc = mw == -INFINITY ? 0.f : dev::fast_exp2(mw - mmax);
        wsum += e[kMaxGroup * Geo::kORow + kMaxGroup + g] * sc;
        val += e[g * Geo::kORow + d] * sc;
      }
      val = wsum > 0.f ? val / wsum : 0.f;
    }
    const int qh = kvh * G + g;
    if (!split) {
      store_out<T>(a, (static_cast<int64_t>(b) * a.num_q_heads + qh) * D + d,
                   val);
    } else {
      const int64_t row =
          (static_cast<int64_t>(b) * a.num_q_heads + qh) * a.max_parts + part;
      a.ws_o[row * D + d] = val;
      if (d == 0) {
        a.ws_ml[2 * row] = mmax;
        a.ws_ml[2 * row + 1] = wsum;
      }
    }
  }
  if (split && a.fused) {
    // Publish this partition; the partition CTA that finishes last combines
    // all of them (fence + ticket: nobody waits for anybody).
    __threadfence();
    dev::named_barrier(1, kConsumers * 32);
    if (ctid == 0)
      s_last = atomicAdd(a.counters + b * a.num_kv_heads + kvh, 1) ==
               n_parts - 1;
    dev::named_barrier(1, kConsumers * 32);
    if (s_last) {
      __threadfence();
      combine_partials<T, D>(a, b, kvh, n_parts, ctid, kConsumers * 32);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.

// The cache viewed as a 2-D tensor of rows (block, kv head, slot) x head_dim;
// one TMA box is block_size rows x 64 elements (128 bytes), swizzled.
bool encode_cache_map(CUtensorMap* map, const void* base, uint64_t rows,
                      int head_dim, int block_size, pa_dtype dtype) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(head_dim), rows};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(head_dim) * 2};
  cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(block_size)};
  cuuint32_t estr[2] = {1u, 1u};
  CUresult r = enc(map,
                   dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                   2, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

#ifndef PAGEDKV_RING_BYTES
#define PAGEDKV_RING_BYTES 65536
#endif
constexpr int stages_for(int bs, int d) {
  // 64 KB ring per CTA: three CTAs fit one SM's shared memory.  Whole
  // multiples of the consumer count (see Geometry).
  return (PAGEDKV_RING_BYTES / (2 * 2 * bs * d)) / kConsumers * kConsumers;
}

template <typename T, int BS, int D, bool kMma>
pa_status launch(const pa_decode_desc* d, DecodeArgs& a, const CUtensorMap& km,
                 const CUtensorMap& vm, cudaStream_t stream) {
  constexpr int S = stages_for(BS, D);
  auto kern = decode_kernel<T, BS, D, S, kMma>;
  const size_t smem = smem_bytes_for<BS, D, S, kMma>(
      (a.warp_parts ? kConsumers : 1) * a.partition_size / BS);
  int dev = 0;
  cudaGetDevice(&dev);
  static bool configured[64] = {false};
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(
        kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
        static_cast<int>(smem_bytes_for<BS, D, S, kMma>(kMaxPartition / BS)));
    if (e != cudaSuccess)
      return fail(PA_ERR_CUDA, "pa_decode: cudaFuncSetAttribute: %s",
                  cudaGetErrorString(e));
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  return launch_chain<T, D, BS>(
      "pa_decode", d, a, smem, stream, [&](const cudaLaunchConfig_t& cfg) {
        return cudaLaunchKernelEx(&cfg, kern, km, vm, a);
      });
}

template <typename T, bool kMma>
pa_status dispatch_shape(const pa_decode_desc* d, DecodeArgs& a,
                         const CUtensorMap& km, const CUtensorMap& vm,
                         cudaStream_t st) {
  if (d->block_size == 16)
    return d->head_dim == 128 ? launch<T, 16, 128, kMma>(d, a, km, vm, st)
                              : launch<T, 16, 64, kMma>(d, a, km, vm, st);
  return d->head_dim == 128 ? launch<T, 32, 128, kMma>(d, a, km, vm, st)
                            : launch<T, 32, 64, kMma>(d, a, km, vm, st);
}

// The built-in scratch's device address belongs to a CUDA context, not to a
// device ordinal: after cudaDeviceReset, or under a context the caller made
// current through the driver API, the module is loaded again and the array
// may sit elsewhere.  So the cache is keyed on the current context's unique
// id (cuCtxGetId, never reused within a process), filled under a mutex.
using PFN_ctxGetCurrent = CUresult (*)(CUcontext*);
using PFN_ctxGetId = CUresult (*)(CUcontext, unsigned long long*);

template <typename F>
F driver_fn(const char* name) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault,
                                       &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    return reinterpret_cast<F>(p);
  return nullptr;
}

// Unique id of the calling thread's current context; false if there is none.
bool current_context_id(unsigned long long* id) {
  static const PFN_ctxGetCurrent get_current =
      driver_fn<PFN_ctxGetCurrent>("cuCtxGetCurrent");
  static const PFN_ctxGetId get_id = driver_fn<PFN_ctxGetId>("cuCtxGetId");
  CUcontext ctx = nullptr;
  return get_current && get_id && get_current(&ctx) == CUDA_SUCCESS && ctx &&
         get_id(ctx, id) == CUDA_SUCCESS;
}

void* scratch_address(pa_status* st) {
  struct Entry {
    unsigned long long ctx_id;
    void* addr;
  };
  constexpr int kMaxEntries = 64;
  static std::mutex mu;
  static Entry cache[kMaxEntries];
  static int used = 0;
  unsigned long long id = 0;
  if (current_context_id(&id)) {
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
      if (cache[i].ctx_id == id) {
        *st = PA_OK;
        return cache[i].addr;
      }
  }
  // First call in this context (or no context yet: the runtime creates the
  // device's primary context here).
  void* p = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&p, ::g_noalloc_scratch);
  if (e != cudaSuccess || !p) {
    *st = fail(PA_ERR_CUDA,
               "pa_decode_noalloc: cudaGetSymbolAddress of the built-in "
               "scratch failed: %s", cudaGetErrorString(e));
    return nullptr;
  }
  if (current_context_id(&id)) {
    std::lock_guard<std::mutex> lock(mu);
    bool known = false;
    for (int i = 0; i < used; ++i) known |= cache[i].ctx_id == id;
    if (!known && used < kMaxEntries) cache[used++] = Entry{id, p};
  }
  *st = PA_OK;
  return p;
}

}  // namespace
}  // namespace pagedkv

using pagedkv::fail;

extern "C" {

pa_status pa_decode_noalloc(void* out, const void* q, const void* k_cache,
                            const void* v_cache, const int32_t* block_tables,
                            const int32_t* context_lens, float scale,
                            const pa_decode_desc* desc, int32_t* dev_err,
                            void* stream) {
  pagedkv::clear_error();
  pa_status st = pagedkv::check_desc(desc, "pa_decode");
  if (st != PA_OK) return st;
  const size_t need = pagedkv::workspace_bytes(desc);
  if (need > PA_NOALLOC_SCRATCH_BYTES)
    return fail(PA_ERR_WORKSPACE,
                "pa_decode_noalloc: this shape needs %zu bytes of scratch but "
                "the built-in area holds %llu; use a larger partition_size, "
                "fewer sequences, or pa_decode with a caller workspace", need,
                static_cast<unsigned long long>(PA_NOALLOC_SCRATCH_BYTES));
  void* scratch = pagedkv::scratch_address(&st);
  if (st != PA_OK) return st;
  return pa_decode(out, q, k_cache, v_cache, block_tables, context_lens,
                   scale, desc, scratch, PA_NOALLOC_SCRATCH_BYTES, dev_err,
                   stream);
}

size_t pa_decode_workspace_bytes(const pa_decode_desc* desc) {
  pagedkv::clear_error();
  if (pagedkv::check_desc(desc, "pa_decode") != PA_OK) return 0;
  return pagedkv::workspace_bytes(desc);
}

int pa_decode_partition_size(const pa_decode_desc* desc) {
  pagedkv::clear_error();
  if (pagedkv::check_desc(desc, "pa_decode") != PA_OK) return -1;
  return pagedkv::resolve_partition(desc, pagedkv::resolve_max_ctx(desc));
}

pa_status pa_decode(void* out, const void* q, const void* k_cache,
                    const void* v_cache, const int32_t* block_tables,
                    const int32_t* context_lens, float scale,
                    const pa_decode_desc* desc, void* workspace,
                    size_t workspace_bytes, int32_t* dev_err, void* stream) {
  pagedkv::clear_error();
  pa_status st = pagedkv::check_desc(desc, "pa_decode");
  if (st != PA_OK) return st;
  st = pagedkv::check_call("pa_decode", out, q, k_cache, v_cache, block_tables,
                           context_lens, scale, desc, workspace,
                           workspace_bytes);
  if (st != PA_OK || desc->num_seqs == 0) return st;
  pagedkv::DecodeArgs a =
      pagedkv::make_args(out, q, block_tables, context_lens, scale, desc,
                         workspace, dev_err);
  CUtensorMap kmap, vmap;
  const uint64_t rows = static_cast<uint64_t>(desc->num_blocks) *
                        desc->num_kv_heads * desc->block_size;
  if (!pagedkv::encode_cache_map(&kmap, k_cache, rows, desc->head_dim,
                                 desc->block_size, desc->dtype) ||
      !pagedkv::encode_cache_map(&vmap, v_cache, rows, desc->head_dim,
                                 desc->block_size, desc->dtype))
    return fail(PA_ERR_CUDA, "pa_decode: cuTensorMapEncodeTiled failed");

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool mma = desc->kernel != PA_KERNEL_SIMT;
  if (desc->dtype == PA_BF16)
    return mma ? pagedkv::dispatch_shape<__nv_bfloat16, true>(desc, a, kmap,
                                                              vmap, s)
               : pagedkv::dispatch_shape<__nv_bfloat16, false>(desc, a, kmap,
                                                               vmap, s);
  return mma ? pagedkv::dispatch_shape<__half, true>(desc, a, kmap, vmap, s)
             : pagedkv::dispatch_shape<__half, false>(desc, a, kmap, vmap, s);
}

}  // extern "C"
