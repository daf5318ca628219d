// pa_decode_q8: paged decode attention over the 8-bit cache (e4m3 codes, one
// fp32 scale for each block and KV head of K and of V).
//
// What is computed: for sequence b, query head h of KV head g, token t in
// block n(t),
//   s_t = scale * ks[n, g] * (q . kcode_t),   p_t = exp(s_t - max s),
//   out = sum_t p_t vs[n, g] vcode_t / sum_t p_t.
//
// What bounds it: one byte per cached element, so a context streams at twice
// the tokens per second of the 16-bit cache for the same HBM rate, and the
// work per byte on the SM doubles.  The kernel keeps that work small:
//  * Codes become fp16 in registers (exact: every e4m3 value is an fp16
//    value), two per conversion, and the products run as m16n8k16
//    tensor-core MMAs with fp32 accumulation.  The scales never touch the
//    elements: ks joins the score's factor (once per page), vs joins the
//    weight.
//  * q is put into fp16 too, multiplied by the power of two that takes its
//    largest element to [2^14, 2^15): exact for elements above 2^-28 of the
//    largest, and to 2^-39 of it for smaller ones.
//  * K fragments: an 8x8 ldmatrix of 16-bit pairs gives a lane four
//    consecutive codes of one row; the MMA's inner index may be any
//    permutation of head_dim that both operands share, so the lane's codes
//    0, 1 take the places 2t, 2t+1 and its codes 2, 3 the places 2t+8, 2t+9.
//    V fragments: ldmatrix.trans moves pairs of codes (dims 2g, 2g+1) of
//    tokens 2t and 2t+1; one byte permutation puts the two tokens of a dim
//    side by side, and output rows g and g+8 are dims 2g and 2g+1.
//  * Weights w = p vs 2^(10-E) are rounded to fp16 for the second product.
//    E follows the exponent of the largest vs met so far (o is rescaled when
//    it grows by more than 3), so w stays below 2^14 and small weights stay
//    normal down to 2^-24.  The rounding is 2^-11 of a weight, an eighth of a
//    bf16 output's own 2^-8 (which hides it: against fp64 the bf16 outputs
//    of 256 sequences are off by 1.6e-3 with and without; a float32 output of
//    a bf16 call carries it).  With fp16 outputs it would show, so there the
//    weight's residual is a second MMA operand, as in the 16-bit kernel; for
//    bf16 it would take 197 us instead of 190 (batch 256 at 486k tokens).
//
// The split of the work, the ring of TMA pages (swizzled 128 bytes wide at
// head_dim 128, 64 at 64), the bounded waits, the longest-first order and the
// combination of partitions are those of the 16-bit decode
// (decode_common.cuh): warp 0 produces, warps 1..4 take pages in turn.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "decode_common.cuh"
#include "device_utils.cuh"
#include "e4m3.cuh"
#include "pagedkv.h"
#include "status.h"

namespace pagedkv {
namespace {

// A page is block_size rows of head_dim bytes, one TMA box; 16-byte chunk c of
// row r sits where the TMA swizzle of that width puts it, so eight
// consecutive rows read at one chunk hit eight different bank groups.
template <int BS, int D, int S>
struct GeometryQ8 {
  static_assert(S % kConsumers == 0, "stages must be a multiple of consumers");
  static constexpr int kPageBytes = BS * D;
  static constexpr int kStageBytes = 2 * kPageBytes;  // K page then V page
  static constexpr int kRingBytes = S * kStageBytes;
  static constexpr int kBarBytes = 2 * S * 8;         // full[S], empty[S]
  static constexpr int kORow = D + 4;
  static constexpr int kEpiWarpFloats = kMaxGroup * kORow + 2 * kMaxGroup;
  static_assert(kConsumers * kEpiWarpFloats * 4 <= kRingBytes,
                "epilogue must fit in the ring");
  static __device__ __forceinline__ uint32_t offset(int row, int chunk) {
    if constexpr (D == 128)
      return row * 128 + ((chunk ^ (row & 7)) << 4);
    else
      return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
  }
};

// Dynamic shared memory: alignment slack, ring, barriers, then the block ids
// and the K and V scales of the CTA's pages.
template <int BS, int D, int S>
constexpr size_t smem_bytes_q8(int pages) {
  using G = GeometryQ8<BS, D, S>;
  return 1024 + G::kRingBytes + G::kBarBytes +
         ((static_cast<size_t>(pages) * 12 + 15) & ~size_t(15));
}

// CTAs per SM and the ring of one.  The consumers' work per byte is twice the
// 16-bit cache's, so warps matter more than bytes in flight: blocks of 16 run
// five CTAs of 32 KB, whose 72 registers spill 132 to 148 bytes at head_dim
// 128.  Blocks of 32 hold two slices of scores and need the registers of three
// CTAs of 64 KB.  Measured, us, three CTAs of 64 KB / four of 48 / five of 32
// (bf16; fp16 is the same to 3 %; 432k tokens in 256 contexts, and 481k in 8):
//   blocks of 16, head_dim 128   196 / 177 / 173   224 / 204 / 220
//   blocks of 16, head_dim 64    149 / 128 / 116   198 / 151 / 151
//   blocks of 32, head_dim 128   159 / 169 / 175   191 / 188 / 216
//   blocks of 32, head_dim 64    104 / 101 / 95    124 / 118 / 130
constexpr int ctas_q8(int bs) { return bs == 16 ? 5 : 3; }
constexpr int ring_bytes_q8(int bs) { return bs == 16 ? 32768 : 65536; }

struct Q8Scales {
  const float* k;  // [num_blocks, num_kv_heads]
  const float* v;
};

template <typename T, int BS, int D, int S>
__global__ void __launch_bounds__(kThreads, ctas_q8(BS))
    decode_q8_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap,
                     const DecodeArgs a, const Q8Scales scales) {
  using Geo = GeometryQ8<BS, D, S>;
  using M = dev::Mma<__half>;
  // fp16 outputs: the weights' residual as a second operand (see above).
  constexpr bool kResidual = std::is_same<T, __half>::value;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem =
      smem_dyn + ((1024u - (dev::smem_u32(smem_dyn) & 1023u)) & 1023u);
  const int nsub = a.warp_parts ? kConsumers : 1;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  dev::pdl_trigger();
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
    dev::pdl_wait();
    b = a.order[blockIdx.z];
  }
  const int PS = a.partition_size;
  const int pages_per_part = PS / BS;
  const int page0 = part * pages_per_part;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Geo::kRingBytes);
  int32_t* bt_s = reinterpret_cast<int32_t*>(bars + 2 * S);
  float* ks_s = reinterpret_cast<float*>(bt_s + nsub * pages_per_part);
  float* vs_s = ks_s + nsub * pages_per_part;
  const uint32_t ring = dev::smem_u32(smem);
  const uint32_t full0 = dev::smem_u32(bars);
  const uint32_t empty0 = full0 + S * 8;

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
  const int n_tok = min(ctx - tok0, nsub * PS);
  const int n_pages = (n_tok + BS - 1) / BS;
  const int G = a.group;

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
        dev::tma_load_2d(kdst, &kmap, 0, y, full);
        dev::tma_load_2d(kdst + Geo::kPageBytes, &vmap, 0, y, full);
      }
    }
    return;
  }

  // ---------------- consumers ----------------
  const int cw = warp - 1;
  const int ctid = tid - 32;  // 0 .. kConsumers*32-1
  // The pages' scales, while the first pages are in flight.
  for (int i = ctid; i < n_pages; i += kConsumers * 32) {
    const int64_t at = static_cast<int64_t>(bt_s[i]) * a.num_kv_heads + kvh;
    ks_s[i] = scales.k[at];
    vs_s[i] = scales.v[at];
  }
  const T* qrow = static_cast<const T*>(a.q) +
                  (static_cast<int64_t>(b) * a.num_q_heads + kvh * G) * D;
  const int g4 = lane >> 2;  // fragment row group
  const int t4 = lane & 3;   // thread in group
  // B fragments of Q^T (K = head_dim, N = 8 heads): head g4, dims
  // 16 c + 4 t4 .. + 3 of chunk c, in fp16 times a power of two.  Heads past
  // G are zero.
  uint32_t qf[D / 16][2];
  float qs[2];  // scale_log2 / that power, for heads 2 t4 and 2 t4 + 1
  {
    float amax = 0.f;
    uint2 raw[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      raw[c] = make_uint2(0u, 0u);
      if (g4 < G)
        raw[c] = *reinterpret_cast<const uint2*>(qrow + g4 * D + c * 16 +
                                                 4 * t4);
      const float2 u = dev::Mma<T>::unpack(raw[c].x);
      const float2 v = dev::Mma<T>::unpack(raw[c].y);
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)),
                               fmaxf(fabsf(v.x), fabsf(v.y))));
    }
    amax = warp_max_xor(amax, 1, 2);
    const int k = min(14 - dev::floor_log2(amax), 100);
    const float up = dev::exp2_int(k), down = dev::exp2_int(-k);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const float2 u = dev::Mma<T>::unpack(raw[c].x);
      const float2 v = dev::Mma<T>::unpack(raw[c].y);
      qf[c][0] = M::pack(u.x * up, u.y * up);
      qf[c][1] = M::pack(v.x * up, v.y * up);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      qs[h] = a.scale_log2 *
              __shfl_sync(0xffffffffu, down, (2 * t4 + h) * 4);
  }
  float o[D / 16][4];
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY};
  float l_run[2] = {0.f, 0.f};
  int e_run = -1000;  // E: o is in units of 2^(E - 10)
  // ldmatrix lane roles: matrix mi = lane / 8, row j = lane % 8.
  const int mi = lane >> 3;
  const int j = lane & 7;
  dev::named_barrier(1, kConsumers * 32);  // the scales are staged

  const int w_tok = a.warp_parts ? max(0, min(n_tok - cw * PS, PS)) : n_tok;
  const int w_iter =
      a.warp_parts ? kConsumers * ((w_tok + BS - 1) / BS) : n_pages;
  for (int i = cw; i < w_iter; i += kConsumers) {
    const int s = i % S;
    const int pg = a.warp_parts ? i / kConsumers : i;  // page of w_tok
    const int sp = a.warp_parts ? cw * pages_per_part + pg : pg;
    const float ks = ks_s[sp], vs = vs_s[sp];
    if (!dev::mbar_wait(full0 + s * 8, (i / S) & 1)) {
      dev::set_error(a.dev_err, PA_ERR_DEVICE_TIMEOUT);
      break;
    }
    const uint32_t kb = ring + s * Geo::kStageBytes;
    const uint32_t vb = kb + Geo::kPageBytes;
    const int nv = min(BS, w_tok - pg * BS);
    if (nv < BS) {
      // Slots past the context get a weight of 0, but 0 * NaN is NaN in the
      // MMA: clear the V rows the sequence never wrote (last page only; the
      // stage is not loaded again).
      for (int idx = lane; idx < (BS - nv) * (D / 16); idx += 32) {
        const int row = nv + idx / (D / 16);
        dev::st_shared_zero16(vb + Geo::offset(row, idx % (D / 16)));
      }
      __syncwarp();
    }

    // S^T (tokens x heads) for each 16-token slice of the page.
    float sc[BS / 16][4];
    const float f0 = qs[0] * ks, f1 = qs[1] * ks;
#pragma unroll
    for (int mt = 0; mt < BS / 16; ++mt) {
      float acc0[4] = {0.f, 0.f, 0.f, 0.f};
      float acc1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c2 = 0; c2 < D / 32; ++c2) {
        uint32_t r[4];  // rows 0-7, 8-15 of chunk 2 c2, then of 2 c2 + 1
        dev::ldsm_x4(kb + Geo::offset(mt * 16 + j + (mi & 1) * 8,
                                      2 * c2 + (mi >> 1)),
                     r);
        const uint32_t a0[4] = {
            dev::e4m3x2_to_f16x2(r[0]), dev::e4m3x2_to_f16x2(r[1]),
            dev::e4m3x2_to_f16x2_hi(r[0]), dev::e4m3x2_to_f16x2_hi(r[1])};
        const uint32_t a1[4] = {
            dev::e4m3x2_to_f16x2(r[2]), dev::e4m3x2_to_f16x2(r[3]),
            dev::e4m3x2_to_f16x2_hi(r[2]), dev::e4m3x2_to_f16x2_hi(r[3])};
        M::run(acc0, a0, qf[2 * c2][0], qf[2 * c2][1]);
        M::run(acc1, a1, qf[2 * c2 + 1][0], qf[2 * c2 + 1][1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = mt * 16 + g4 + (e >> 1) * 8;
        const float x = (acc0[e] + acc1[e]) * ((e & 1) ? f1 : f0);
        sc[mt][e] = tok < nv ? x : -INFINITY;
      }
    }
    // Online softmax; this lane holds heads 2*t4 and 2*t4+1.  o also
    // follows E, the running exponent of vs.
    float o_scale = 1.f;
    // -100 and 127 keep E - 10 and 10 - E in exp2_int's range.
    const int e_vs = max(-100, min(127, dev::floor_log2(vs)));
    if (e_vs > e_run + 3) {  // the same in every lane
      o_scale = dev::exp2_int(max(e_run - e_vs, -126));
      e_run = e_vs;
    }
    const float wv = vs * dev::exp2_int(10 - e_run);
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
      alpha[h] *= o_scale;
    }
    // Rarely needed on long contexts: the maxima settle early.
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[dt][e] *= alpha[e & 1];
    }

    // The weights as B fragments (K = tokens, N = heads).
    uint32_t bh[BS / 16][2], bl[BS / 16][2];
#pragma unroll
    for (int ks2 = 0; ks2 < BS / 16; ++ks2) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p0 = sc[ks2][2 * r] * wv, p1 = sc[ks2][2 * r + 1] * wv;
        const uint32_t hi = M::pack(p0, p1);
        bh[ks2][r] = dev::movmatrix_trans(hi);
        if constexpr (kResidual) {
          const float2 hf = M::unpack(hi);
          bl[ks2][r] = dev::movmatrix_trans(M::pack(p0 - hf.x, p1 - hf.y));
        }
      }
    }
    // O^T (head_dim x heads) += V^T . W^T
#pragma unroll
    for (int ks2 = 0; ks2 < BS / 16; ++ks2) {
#pragma unroll
      for (int c2 = 0; c2 < D / 32; ++c2) {
        uint32_t r[4];  // tokens 0-7, 8-15 of chunk 2 c2, then of 2 c2 + 1
        dev::ldsm_x4_trans(vb + Geo::offset(ks2 * 16 + j + (mi & 1) * 8,
                                            2 * c2 + (mi >> 1)),
                           r);
#pragma unroll
        for (int u = 0; u < 4; ++u) r[u] = __byte_perm(r[u], 0u, 0x3120);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t af[4] = {dev::e4m3x2_to_f16x2(r[2 * h]),
                                  dev::e4m3x2_to_f16x2_hi(r[2 * h]),
                                  dev::e4m3x2_to_f16x2(r[2 * h + 1]),
                                  dev::e4m3x2_to_f16x2_hi(r[2 * h + 1])};
          M::run(o[2 * c2 + h], af, bh[ks2][0], bh[ks2][1]);
          if constexpr (kResidual)
            M::run(o[2 * c2 + h], af, bl[ks2][0], bl[ks2][1]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(empty0 + s * 8);
  }

  // This warp's state in plain units: the row sums over the lanes, o times
  // its power of two.
  float l_fin[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float l = l_run[h];
    l += __shfl_xor_sync(0xffffffffu, l, 4);
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    l_fin[h] = l;
  }
  float unit[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    unit[h] = e_run > -1000 ? dev::exp2_int(e_run - 10) : 0.f;
    // A NaN or infinite score: the combinations divide by sums above 0 only,
    // so the NaN travels in o.
    if (isnan(l_fin[h])) {
      l_fin[h] = 1.f;
      m_run[h] = fmaxf(m_run[h], 0.f);
      unit[h] = NAN;
    }
  }
  // o[c][e] is head 2 t4 + (e & 1), dim 16 c + 2 g4 + (e >> 1).
  if (a.warp_parts) {
    const int mypart = part + cw;
    if (mypart >= n_parts) return;
    const int64_t row0 = static_cast<int64_t>(b) * a.num_q_heads + kvh * G;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = 2 * t4 + h;
      if (g >= G) continue;
      const float f = l_fin[h] > 0.f ? unit[h] / l_fin[h] : 0.f;
      const int64_t row = (row0 + g) * a.max_parts + mypart;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const int d = c * 16 + 2 * g4;
        if (n_parts == 1) {  // the reduce kernel skips these rows
          store_out<T>(a, (row0 + g) * D + d, o[c][h] * f);
          store_out<T>(a, (row0 + g) * D + d + 1, o[c][h + 2] * f);
        } else {
          *reinterpret_cast<float2*>(a.ws_o + row * D + d) =
              make_float2(o[c][h] * f, o[c][h + 2] * f);
        }
      }
      if (n_parts > 1 && g4 == 0) {
        a.ws_ml[2 * row] = m_run[h];
        a.ws_ml[2 * row + 1] = l_fin[h];
      }
    }
    return;
  }
  // Hand the state to the epilogue area (aliases the ring).
  dev::named_barrier(1, kConsumers * 32);
  float* ep = reinterpret_cast<float*>(smem) + cw * Geo::kEpiWarpFloats;
#pragma unroll
  for (int c = 0; c < D / 16; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float2*>(ep + (2 * t4 + h) * Geo::kORow + c * 16 +
                                 2 * g4) =
          make_float2(o[c][h] * unit[h], o[c][h + 2] * unit[h]);
  if (g4 == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      ep[kMaxGroup * Geo::kORow + 2 * t4 + h] = m_run[h];
      ep[kMaxGroup * Geo::kORow + kMaxGroup + 2 * t4 + h] = l_fin[h];
    }
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
        const float f = mw == -INFINITY ? 0.f : dev::fast_exp2(mw - mmax);
        wsum += e[kMaxGroup * Geo::kORow + kMaxGroup + g] * f;
        val += e[g * Geo::kORow + d] * f;
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

// The cache as rows (block, KV head, slot) x head_dim bytes; one box is a page.
bool encode_q8_map(CUtensorMap* map, const void* base, uint64_t rows,
                   int head_dim, int block_size) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(head_dim), rows};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(head_dim)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(head_dim),
                       static_cast<cuuint32_t>(block_size)};
  cuuint32_t estr[2] = {1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                             : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Stages in whole multiples of the consumer count.
constexpr int stages_q8(int bs, int d) {
  return ring_bytes_q8(bs) / (2 * bs * d) / kConsumers * kConsumers;
}

template <typename T, int BS, int D>
pa_status launch_q8(const pa_decode_desc* d, const DecodeArgs& a,
                    const Q8Scales& sc, const CUtensorMap& km,
                    const CUtensorMap& vm, cudaStream_t stream) {
  constexpr int S = stages_q8(BS, D);
  auto kern = decode_q8_kernel<T, BS, D, S>;
  const size_t smem = smem_bytes_q8<BS, D, S>(
      (a.warp_parts ? kConsumers : 1) * a.partition_size / BS);
  static OncePerDevice configured;
  if (configured.needed()) {
    const cudaError_t e = cudaFuncSetAttribute(
        kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
        static_cast<int>(smem_bytes_q8<BS, D, S>(kMaxPartition / BS)));
    if (e != cudaSuccess)
      return fail(PA_ERR_CUDA, "pa_decode_q8: cudaFuncSetAttribute: %s",
                  cudaGetErrorString(e));
    configured.mark();
  }
  return launch_chain<T, D, BS>(
      "pa_decode_q8", d, a, smem, stream, [&](const cudaLaunchConfig_t& cfg) {
        return cudaLaunchKernelEx(&cfg, kern, km, vm, a, sc);
      });
}

template <typename T>
pa_status dispatch_q8(const pa_decode_desc* d, const DecodeArgs& a,
                      const Q8Scales& sc, const CUtensorMap& km,
                      const CUtensorMap& vm, cudaStream_t st) {
  if (d->block_size == 16)
    return d->head_dim == 128 ? launch_q8<T, 16, 128>(d, a, sc, km, vm, st)
                              : launch_q8<T, 16, 64>(d, a, sc, km, vm, st);
  return d->head_dim == 128 ? launch_q8<T, 32, 128>(d, a, sc, km, vm, st)
                            : launch_q8<T, 32, 64>(d, a, sc, km, vm, st);
}

}  // namespace
}  // namespace pagedkv

using pagedkv::fail;

extern "C" pa_status pa_decode_q8(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const float* k_scales, const float* v_scales, const int32_t* block_tables,
    const int32_t* context_lens, float scale, const pa_decode_desc* desc,
    void* workspace, size_t workspace_bytes, int32_t* dev_err, void* stream) {
  pagedkv::clear_error();
  pa_status st = pagedkv::check_desc(desc, "pa_decode_q8");
  if (st != PA_OK) return st;
  if (desc->kernel == PA_KERNEL_SIMT)
    return fail(PA_ERR_UNSUPPORTED,
                "pa_decode_q8: no SIMT kernel for the 8-bit cache");
  st = pagedkv::check_call("pa_decode_q8", out, q, k_cache, v_cache,
                           block_tables, context_lens, scale, desc, workspace,
                           workspace_bytes);
  if (st != PA_OK || desc->num_seqs == 0) return st;
  if (!k_scales || !v_scales)
    return fail(PA_ERR_INVALID_ARG, "pa_decode_q8: NULL scales");
  const pagedkv::DecodeArgs a =
      pagedkv::make_args(out, q, block_tables, context_lens, scale, desc,
                         workspace, dev_err);
  CUtensorMap km, vm;
  const uint64_t rows = static_cast<uint64_t>(desc->num_blocks) *
                        desc->num_kv_heads * desc->block_size;
  if (!pagedkv::encode_q8_map(&km, k_cache, rows, desc->head_dim,
                              desc->block_size) ||
      !pagedkv::encode_q8_map(&vm, v_cache, rows, desc->head_dim,
                              desc->block_size))
    return fail(PA_ERR_CUDA, "pa_decode_q8: cuTensorMapEncodeTiled failed");
  const pagedkv::Q8Scales sc{k_scales, v_scales};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return desc->dtype == PA_BF16
             ? pagedkv::dispatch_q8<__nv_bfloat16>(desc, a, sc, km, vm, s)
             : pagedkv::dispatch_q8<__half>(desc, a, sc, km, vm, s);
}
