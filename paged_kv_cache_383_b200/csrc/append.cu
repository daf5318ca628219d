// pa_append and pa_append_q8: what a layer does with its new queries, keys and
// values before attention, in one launch: the norm of each query and key head
// (optional), the position rotation, and the write of K and V into the paged
// cache, in the cache's own 16-bit type or as e4m3 codes with one scale for
// each (block, KV head).
//
// Row t of sequence b (i-th of its q_len new tokens) sits at position
// p = L_b - q_len + i, in block table[b][p / block_size].  With x a head:
//   norm      x <- w x / sqrt(mean(x^2) + eps)
//   rotation  (u, w) <- (u cos - w sin, w cos + u sin) for pair j of the first
//             rot_dim elements, at the angle p f_j; the pairs are (j, j +
//             rot_dim/2) or (2j, 2j + 1).
// All in fp32 with one rounding at the end; the angle is reduced to a
// fraction of a turn in fp64 (an fp32 product is off by a tenth of a radian at
// position 10^6), so any position below 2^31 is exact to about 2^-24 turns
// and no table is read.
//
// What bounds it: bytes (each element is read and written once; about ten
// operations for each), or, for a decode step, the latency of the chain
// lengths -> block id -> store.  The rows' loads do not depend on that chain
// and are issued first; a token's sines and cosines are computed once per CTA
// and shared by its heads.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "device_utils.cuh"
#include "e4m3.cuh"
#include "pagedkv.h"
#include "status.h"

namespace pagedkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxWindow = 16;  // rows whose blocks one K/V CTA looks after
constexpr int kMaxBlock = 32;   // block_size
constexpr int kMaxPairs = 64;   // rotated pairs: head_dim / 2
constexpr int kMaxTokens = 4;   // tokens whose rows one CTA streams
// Scales written by pa_append_q8: 2^e with e in this range.
constexpr int kMinScaleExp = -64, kMaxScaleExp = 120;

struct AppendArgs {
  void* q_out;
  const void* q;
  const void* k;
  const void* v;
  const void* q_norm;  // nullable
  const void* k_norm;
  const double* freqs;
  void* k_cache;
  void* v_cache;
  float* k_scales;  // pa_append_q8 only
  float* v_scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;  // nullable: row t is sequence t's only one
  int32_t* dev_err;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int num_seqs, num_q_heads, num_kv_heads;
  int block_size, max_blocks_per_seq, num_blocks;
  int total_q, max_q_len;
  int rot_pairs;  // rot_dim / 2
  int interleaved;
  float rope_scale, norm_eps;
  int tokens;       // tokens per CTA (1 with row_splits > 1)
  int row_splits;   // CTAs that share a token's rows
  int kv_ctas;      // pa_append_q8: CTAs 0 .. kv_ctas - 1 write K and V
  int window;       // rows per K/V window
  int unit_groups;  // CTAs per window (kWarps (K or V, head) units each)
};

// Where a sequence's new rows are; `ok` false: nothing of it is written.
struct Seq {
  int q0, q_len, L;
  bool ok;
};
__device__ __forceinline__ Seq read_seq(const AppendArgs& a, int b) {
  Seq s;
  s.q0 = a.query_start ? a.query_start[b] : b;
  s.q_len = a.query_start ? a.query_start[b + 1] - s.q0 : 1;
  s.L = a.context_lens[b];
  s.ok = false;
  if (s.L == 0) return s;  // padding
  const bool bad =
      s.L < 0 ||
      s.L > static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size ||
      s.q_len < 0 || s.q_len > s.L || s.q_len > a.max_q_len || s.q0 < 0 ||
      s.q0 > a.total_q - s.q_len;
  if (bad)
    dev::set_error(a.dev_err, PA_ERR_DEVICE_OOB);
  else
    s.ok = s.q_len > 0;
  return s;
}

// cos and sin of the pair's angle at position p, times rope_scale.
__device__ __forceinline__ float2 turn(const AppendArgs& a, int pair, int p) {
  const double t = static_cast<double>(p) *
                   (a.freqs[pair] * 0.15915494309189533577);  // 1 / (2 pi)
  float s, c;
  sincospif(2.f * static_cast<float>(t - rint(t)), &s, &c);
  return make_float2(c * a.rope_scale, s * a.rope_scale);
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = dev::Mma<T>::unpack(r[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// A head row is spread over D / 16 lanes; a lane holds two chunks of eight
// elements (16 bytes).  With h = rot_dim / 16 lanes' worth of rotated pairs,
// lane l < h holds both sides of pairs 8l .. 8l + 7: chunks l and l + h in the
// half layout, 2l and 2l + 1 in the interleaved one; the lanes past them hold
// chunks 2l and 2l + 1, which do not turn.  So the rotation needs no other
// lane, and its eight sines serve the lane for every head of a token.
struct Chunks {
  int a, b;
  bool turns;
};
__device__ __forceinline__ Chunks chunks_of(const AppendArgs& a, int l) {
  const int h = a.rot_pairs / 8;
  const bool apart = l < h && !a.interleaved;
  return Chunks{apart ? l : 2 * l, apart ? l + h : 2 * l + 1, l < h};
}

// Shared memory holds a token's pairs in groups of eight, 80 bytes apart: the
// eight lanes of a 16-byte load phase then read all 32 banks.
constexpr int kGroupStride = 10;  // float2
__device__ __forceinline__ int pair_at(int pair) {
  return (pair >> 3) * kGroupStride + (pair & 7);
}
constexpr int kTokenStride = kMaxPairs / 8 * kGroupStride;  // float2 per token

// Norm (weight non-null) and rotation (turn) of a head row; x[0 .. 7] is this
// lane's chunk ch.a, x[8 .. 15] its chunk ch.b, z its pairs' cos and sin.
// Every lane takes part in the shuffles.
template <typename T, int D>
__device__ __forceinline__ void norm_rotate(float (&x)[16], const T* weight,
                                            bool turn, const float2 (&z)[8],
                                            const AppendArgs& a,
                                            const Chunks& ch) {
  if (a.q_norm || a.k_norm) {  // uniform over the grid
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int m = 1; m < D / 16; m <<= 1)
      ss += __shfl_xor_sync(0xffffffffu, ss, m);
    if (weight) {
      const float r = rsqrtf(ss * (1.f / D) + a.norm_eps);
      float w[8];
      unpack8<T>(reinterpret_cast<const uint4*>(weight)[ch.a], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
      unpack8<T>(reinterpret_cast<const uint4*>(weight)[ch.b], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[8 + e] = x[8 + e] * r * w[e];
    }
  }
  if (!turn) return;
  if (a.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = x[2 * e], w = x[2 * e + 1];
      x[2 * e] = u * z[e].x - w * z[e].y;
      x[2 * e + 1] = w * z[e].x + u * z[e].y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = x[e], w = x[8 + e];
      x[e] = u * z[e].x - w * z[e].y;
      x[8 + e] = w * z[e].x + u * z[e].y;
    }
  }
}

__device__ __forceinline__ void load_pairs(const float2* cs, int l,
                                           float2 (&z)[8]) {
  const float4* from =
      reinterpret_cast<const float4*>(cs + l * kGroupStride);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float4 v = from[e];
    z[2 * e] = make_float2(v.x, v.y);
    z[2 * e + 1] = make_float2(v.z, v.w);
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(dev::Mma<T>::pack(x[0], x[1]), dev::Mma<T>::pack(x[2], x[3]),
                    dev::Mma<T>::pack(x[4], x[5]),
                    dev::Mma<T>::pack(x[6], x[7]));
}

// Rows that keep 16 bits, the query heads and (16-bit cache) the key and value
// heads, of tokens t0 .. t0 + a.tokens - 1; `split` of the row_splits CTAs
// that share them.  What hangs on the chain sequence -> length -> block id
// and the sines is looked up once for all the tokens, behind the first loads;
// then the rows stream through.
template <typename T, int D, bool kQ8>
__device__ __forceinline__ void token_rows(const AppendArgs& a, int t0,
                                           int split, float2* cs) {
  constexpr int LPR = D / 16;              // lanes per row
  constexpr int kSlots = kThreads / LPR;   // rows per pass of the CTA
  constexpr int kBatch = 2;                // passes loaded together
  __shared__ int s_seq[kMaxTokens];
  __shared__ int s_pos[kMaxTokens];  // -1: no such row, or padding
  __shared__ int s_blk[kMaxTokens];  // -1: K and V are not written
  const int tid = threadIdx.x;
  const int l = tid % LPR, slot = tid / LPR;
  const Chunks ch = chunks_of(a, l);
  const int rows = a.num_q_heads + (kQ8 ? 0 : 2 * a.num_kv_heads);
  const int n_tok = min(a.tokens, a.total_q - t0);
  const int step = kSlots * a.row_splits;
  // A row of this CTA: token i, row r of it.
  struct Row {
    int i, r;
  };
  auto advance = [&](Row& w) {
    w.r += step;
    while (w.r >= rows && w.i < n_tok) {
      w.r -= rows;
      ++w.i;
    }
  };
  auto src = [&](const Row& w) -> const uint4* {
    const int64_t t = t0 + w.i;
    const T* p;
    if (w.r < a.num_q_heads)
      p = static_cast<const T*>(a.q) + t * a.q_stride + w.r * D;
    else if (w.r < a.num_q_heads + a.num_kv_heads)
      p = static_cast<const T*>(a.k) + t * a.k_stride +
          (w.r - a.num_q_heads) * D;
    else
      p = static_cast<const T*>(a.v) + t * a.v_stride +
          (w.r - a.num_q_heads - a.num_kv_heads) * D;
    return reinterpret_cast<const uint4*>(p);
  };
  Row w{0, split * kSlots + slot - step};
  advance(w);
  auto load = [&](Row& first, uint4 (&raw)[kBatch][2]) {
    first = w;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (w.i < n_tok) {
        const uint4* p = src(w);
        raw[u][0] = p[ch.a];
        raw[u][1] = p[ch.b];
      }
      advance(w);
    }
  };
  Row at;
  uint4 raw[kBatch][2];
  load(at, raw);

  if (tid < kMaxTokens) {
    s_seq[tid] = a.query_start ? -1 : t0 + tid;
  }
  if (a.query_start) {
    __syncthreads();
    for (int j = tid; j < a.num_seqs; j += kThreads) {
      // The first CTA checks every sequence: one whose range holds no row is
      // met by no token.
      if (!kQ8 && blockIdx.x == 0) read_seq(a, j);
      const int lo = max(a.query_start[j], t0);
      const int hi = min(a.query_start[j + 1], t0 + n_tok);
      for (int t = lo; t < hi; ++t) s_seq[t - t0] = j;
    }
  }
  __syncthreads();
  if (tid < n_tok) {
    const int b = s_seq[tid];
    int pos = -1, blk = -1;
    if (b >= 0) {  // else a row behind the last sequence
      const Seq sq = read_seq(a, b);
      if (sq.ok) {
        pos = sq.L - sq.q_len + t0 + tid - sq.q0;
        if constexpr (!kQ8) {
          blk = a.block_tables[static_cast<int64_t>(b) *
                                   a.max_blocks_per_seq +
                               pos / a.block_size];
          if (blk < 0 || blk >= a.num_blocks) {
            dev::set_error(a.dev_err, PA_ERR_DEVICE_OOB);
            blk = -1;
          }
        }
      }
    }
    s_pos[tid] = pos;
    s_blk[tid] = blk;
  }
  __syncthreads();
  for (int j = tid; j < n_tok * a.rot_pairs; j += kThreads) {
    const int i = j / a.rot_pairs;
    const int pair = j - i * a.rot_pairs;
    if (s_pos[i] >= 0)
      cs[i * kTokenStride + pair_at(pair)] = turn(a, pair, s_pos[i]);
  }
  __syncthreads();

  // Passes of the whole CTA (every thread takes part in the shuffles).
  const int passes = (n_tok * rows + step - 1) / step;
  int z_tok = -1;  // whose pairs are in z
  float2 z[8];
  for (int p0 = 0; p0 < passes; p0 += kBatch) {
    if (p0 > 0) load(at, raw);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (p0 + u >= passes) break;
      const bool live = at.i < n_tok;
      const int r = at.r;
      const int pos = live ? s_pos[at.i] : -1;
      const bool is_q = r < a.num_q_heads;
      const int kv = r - a.num_q_heads;  // key heads, then value heads
      const bool is_v = kv >= a.num_kv_heads;
      float x[16] = {};
      if (live) {
        unpack8<T>(raw[u][0], x);
        unpack8<T>(raw[u][1], x + 8);
        if (z_tok != at.i && ch.turns) {
          load_pairs(cs + at.i * kTokenStride, l, z);
          z_tok = at.i;
        }
      }
      norm_rotate<T, D>(x,
                        static_cast<const T*>(is_q ? a.q_norm
                                              : is_v ? nullptr : a.k_norm),
                        ch.turns && (is_q || !is_v), z, a, ch);
      if (pos >= 0) {
        T* dst = nullptr;
        if (is_q) {
          dst = static_cast<T*>(a.q_out) + (t0 + at.i) * a.q_out_stride +
                r * D;
        } else if (s_blk[at.i] >= 0) {
          const int h = is_v ? kv - a.num_kv_heads : kv;
          dst = static_cast<T*>(is_v ? a.v_cache : a.k_cache) +
                ((static_cast<int64_t>(s_blk[at.i]) * a.num_kv_heads + h) *
                     a.block_size + pos % a.block_size) * D;
        }
        if (dst) {
          // V unchanged: the very bits (a NaN's payload too).
          const bool copy = !is_q && is_v;
          reinterpret_cast<uint4*>(dst)[ch.a] =
              copy ? raw[u][0] : pack8<T>(x);
          reinterpret_cast<uint4*>(dst)[ch.b] =
              copy ? raw[u][1] : pack8<T>(x + 8);
        }
      }
      advance(at);
    }
  }
}

// The smallest power of two s with amax <= 448 s, from amax's bits: with
// amax = 2^x m, 448 = 2^8 * 1.75.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t w = __float_as_uint(amax);
  const int e = static_cast<int>(w >> 23) - 127 - 8 +
                ((w & 0x7fffffu) > 0x600000u ? 1 : 0);
  return dev::exp2_int(max(kMinScaleExp, min(kMaxScaleExp, e)));
}

// One warp: new rows [row, row + n) of one sequence, all in block `blk` from
// offset o on, of one KV head's K (weight / rotation) or V, into codes and
// the scale.  The warp alone touches this (block, head).
template <typename T, int D>
__device__ __forceinline__ void quantise_unit(const AppendArgs& a, bool is_k,
                                              int h, int row, int n, int blk,
                                              int o, const float2* cs) {
  constexpr int LPR = D / 16, kRows = 32 / LPR;  // rows per pass
  constexpr int kKeep = 4;                       // passes held in registers
  const int lane = threadIdx.x & 31;
  const int l = lane % LPR, sub = lane / LPR;
  const Chunks ch = chunks_of(a, l);
  const T* base = is_k ? static_cast<const T*>(a.k) + row * a.k_stride
                       : static_cast<const T*>(a.v) + row * a.v_stride;
  const int64_t stride = is_k ? a.k_stride : a.v_stride;
  const T* weight = is_k ? static_cast<const T*>(a.k_norm) : nullptr;
  const int64_t unit = static_cast<int64_t>(blk) * a.num_kv_heads + h;
  float* sp = (is_k ? a.k_scales : a.v_scales) + unit;
  const float s_old = o > 0 ? *sp : 0.f;
  uint8_t* page = static_cast<uint8_t*>(is_k ? a.k_cache : a.v_cache) +
                  unit * a.block_size * D;
  uint4 raw[kKeep][2];
  auto load = [&](int p0) {
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
      const int r = (p0 + u) * kRows + sub;
      const uint4* p =
          reinterpret_cast<const uint4*>(base + r * stride + h * D);
      raw[u][0] = r < n ? p[ch.a] : make_uint4(0u, 0u, 0u, 0u);
      raw[u][1] = r < n ? p[ch.b] : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  auto value = [&](int u, int r, float (&x)[16]) {
    unpack8<T>(raw[u][0], x);
    unpack8<T>(raw[u][1], x + 8);
    if (is_k) {  // uniform over the warp
      float2 z[8];
      if (ch.turns) load_pairs(cs + min(r, n - 1) * kTokenStride, l, z);
      norm_rotate<T, D>(x, weight, ch.turns, z, a, ch);
    }
  };
  float amax = 0.f;
  const int passes = (n + kRows - 1) / kRows;
  // Up to kKeep passes stay in registers as they were read; longer runs (a
  // block of 32 at head_dim 128) are read again for their codes, from L1 or
  // L2.  Norm and rotation are done twice either way: keeping their fp32
  // results would take twice the registers.
  for (int p0 = 0; p0 < passes; p0 += kKeep) {
    load(p0);
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
      if (p0 + u >= passes) break;
      float x[16];
      value(u, (p0 + u) * kRows + sub, x);
      if ((p0 + u) * kRows + sub < n)
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
    }
  }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  const float s = fmaxf(s_old, scale_for(amax));
  if (lane == 0 && s != s_old) *sp = s;
  if (o > 0 && s > s_old) {
    // Older codes of the block follow the scale: exact for powers of two but
    // where a code becomes subnormal.
    const float ratio = s_old / s;
    uint4* old = reinterpret_cast<uint4*>(page);
    for (int i = lane; i < o * (D / 16); i += 32) {
      uint4 w = old[i];
      uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = dev::e4m3x2_to_f16x2(r[e]);
        const uint32_t hi = dev::e4m3x2_to_f16x2_hi(r[e]);
        const float2 f = dev::Mma<__half>::unpack(lo);
        const float2 g = dev::Mma<__half>::unpack(hi);
        r[e] = dev::f32x4_to_e4m3x4(f.x * ratio, f.y * ratio, g.x * ratio,
                                    g.y * ratio);
      }
      old[i] = make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
  // x / s; times the reciprocal where that is exact (a power of two).
  const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0u;
  const float inv = 1.f / s;
  auto store = [&](const float (&x)[16], int r) {
    if (r >= n) return;
    float y[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = pow2 ? x[e] * inv : x[e] / s;
    uint8_t* to = page + static_cast<int64_t>(o + r) * D;
    *reinterpret_cast<uint2*>(to + 8 * ch.a) =
        make_uint2(dev::f32x4_to_e4m3x4(y[0], y[1], y[2], y[3]),
                   dev::f32x4_to_e4m3x4(y[4], y[5], y[6], y[7]));
    *reinterpret_cast<uint2*>(to + 8 * ch.b) =
        make_uint2(dev::f32x4_to_e4m3x4(y[8], y[9], y[10], y[11]),
                   dev::f32x4_to_e4m3x4(y[12], y[13], y[14], y[15]));
  };
  for (int p0 = 0; p0 < passes; p0 += kKeep) {
    if (passes > kKeep) load(p0);
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
      if (p0 + u >= passes) break;
      float x[16];
      value(u, (p0 + u) * kRows + sub, x);
      store(x, (p0 + u) * kRows + sub);
    }
  }
}

// K and V of the runs of rows that start a block (or their sequence) in rows
// [window * w, window * (w + 1)): each run lies in one block.
template <typename T, int D>
__device__ __forceinline__ void window_kv(const AppendArgs& a, int w,
                                          int group, float2* cs) {
  __shared__ int s_run[kMaxWindow][2];  // sequence, first row
  __shared__ int s_n;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int64_t lo64 = static_cast<int64_t>(w) * a.window;
  const int lo = static_cast<int>(lo64);
  const int hi = static_cast<int>(
      min(lo64 + a.window, static_cast<int64_t>(a.total_q)));
  if (tid == 0) s_n = 0;
  __syncthreads();
  auto push = [&](int b, int row) {
    const int i = atomicAdd(&s_n, 1);
    if (i < kMaxWindow) {
      s_run[i][0] = b;
      s_run[i][1] = row;
    } else {  // sequences whose rows overlap
      dev::set_error(a.dev_err, PA_ERR_DEVICE_OOB);
    }
  };
  if (!a.query_start) {
    for (int t = lo + tid; t < hi; t += kThreads) push(t, t);
  } else {
    for (int j = tid; j < a.num_seqs; j += kThreads) {
      const int q0 = a.query_start[j], q1 = a.query_start[j + 1];
      if (q1 <= lo || q0 >= hi) {
        // The first CTA checks every sequence: one whose range holds no row
        // is met by no window.
        if (blockIdx.x == 0) read_seq(a, j);
        continue;
      }
      const Seq sq = read_seq(a, j);
      if (!sq.ok) continue;
      const int from = max(q0, lo);
      if (from == q0) push(j, q0);
      // then the rows at a block's first slot
      const int p = sq.L - sq.q_len + from - q0;
      int r = from + (a.block_size - p % a.block_size) % a.block_size;
      if (r == q0) r += a.block_size;
      for (; r < min(hi, q1); r += a.block_size) push(j, r);
    }
  }
  __syncthreads();
  const int runs = min(s_n, kMaxWindow);
  const int unit = group * kWarps + warp;
  const bool any_k = group * kWarps < a.num_kv_heads;
  for (int i = 0; i < runs; ++i) {
    const int b = s_run[i][0], row = s_run[i][1];
    const Seq sq = read_seq(a, b);
    if (!sq.ok) continue;  // uniform
    const int pos = sq.L - sq.q_len + row - sq.q0;
    const int o = pos % a.block_size;
    const int n = min(a.block_size - o, sq.q0 + sq.q_len - row);
    const int blk =
        a.block_tables[static_cast<int64_t>(b) * a.max_blocks_per_seq +
                       pos / a.block_size];
    if (blk < 0 || blk >= a.num_blocks) {
      if (tid == 0) dev::set_error(a.dev_err, PA_ERR_DEVICE_OOB);
      continue;  // uniform
    }
    if (any_k) {
      __syncthreads();  // the previous run's sines are read
      for (int j = tid; j < n * a.rot_pairs; j += kThreads) {
        const int r = j / a.rot_pairs;
        const int pair = j - r * a.rot_pairs;
        cs[r * kTokenStride + pair_at(pair)] = turn(a, pair, pos + r);
      }
      __syncthreads();
    }
    if (unit < 2 * a.num_kv_heads) {
      const bool is_k = unit < a.num_kv_heads;
      quantise_unit<T, D>(a, is_k, is_k ? unit : unit - a.num_kv_heads, row,
                          n, blk, o, cs);
    }
  }
}

// Four CTAs per SM (three for the 8-bit cache's kernel, which needs more
// registers): loads in flight carry the bandwidth (7728 rows of 80 heads 88 us
// with three, 77 us with four).  K/V CTAs come first: they are the longer
// chains (spread among the others they ended the grid: 7322 prompt rows 75 us
// instead of 59).
template <typename T, int D, bool kQ8>
__global__ void __launch_bounds__(kThreads, kQ8 ? 3 : 4)
    append_kernel(const AppendArgs a) {
  // cos/sin: the pairs of the CTA's tokens, or of a block's.
  __shared__ __align__(16) float2
      cs[(kQ8 ? kMaxBlock : kMaxTokens) * kTokenStride];
  dev::pdl_wait();  // q, k and v may be the previous kernel's output
  // A following attention may run its prologue now.  Not before the wait: it
  // reads lengths, which a kernel before this one may still be writing.
  dev::pdl_trigger();
  if (kQ8 && static_cast<int>(blockIdx.x) < a.kv_ctas) {
    window_kv<T, D>(a, blockIdx.x / a.unit_groups, blockIdx.x % a.unit_groups,
                    cs);
  } else {
    const unsigned i = blockIdx.x - (kQ8 ? a.kv_ctas : 0);
    token_rows<T, D, kQ8>(a, static_cast<int>(i / a.row_splits) * a.tokens,
                          i % a.row_splits, cs);
  }
}

pa_status check_append(const char* fn, const pa_append_desc* d) {
  if (!d) return fail(PA_ERR_INVALID_ARG, "%s: desc is NULL", fn);
  if (d->num_seqs < 0 || d->num_q_heads < 0 || d->num_kv_heads <= 0 ||
      d->max_blocks_per_seq <= 0 || d->num_blocks < 0 || d->total_q < 0 ||
      d->max_q_len < 0 || (d->dtype != PA_F16 && d->dtype != PA_BF16))
    return fail(PA_ERR_INVALID_ARG,
                "%s: num_seqs=%d num_q_heads=%d num_kv_heads=%d "
                "max_blocks_per_seq=%d num_blocks=%d total_q=%d max_q_len=%d "
                "dtype=%d", fn, d->num_seqs, d->num_q_heads, d->num_kv_heads,
                d->max_blocks_per_seq, d->num_blocks, d->total_q,
                d->max_q_len, static_cast<int>(d->dtype));
  if ((d->head_dim != 64 && d->head_dim != 128) ||
      (d->block_size != 16 && d->block_size != 32))
    return fail(PA_ERR_UNSUPPORTED,
                "%s: needs head_dim 64 or 128 (got %d) and block_size 16 or "
                "32 (got %d)", fn, d->head_dim, d->block_size);
  if (d->rot_dim < 0 || d->rot_dim > d->head_dim)
    return fail(PA_ERR_INVALID_ARG, "%s: rot_dim %d not in 0 .. head_dim %d",
                fn, d->rot_dim, d->head_dim);
  if (d->rot_dim % 16)
    return fail(PA_ERR_UNSUPPORTED, "%s: rot_dim %d is not a multiple of 16",
                fn, d->rot_dim);
  if (d->rope_layout != PA_ROPE_HALF && d->rope_layout != PA_ROPE_INTERLEAVED)
    return fail(PA_ERR_INVALID_ARG, "%s: rope_layout %d", fn, d->rope_layout);
  if (!std::isfinite(d->rope_scale) || !std::isfinite(d->norm_eps) ||
      d->norm_eps < 0.f)
    return fail(PA_ERR_INVALID_ARG, "%s: rope_scale or norm_eps", fn);
  if (static_cast<int64_t>(d->max_blocks_per_seq) * d->block_size >
      0x7fffffffLL)
    return fail(PA_ERR_INVALID_ARG, "%s: max_blocks_per_seq too large", fn);
  const int64_t strides[4] = {d->q_stride, d->k_stride, d->v_stride,
                              d->q_out_stride};
  const char* names[4] = {"q_stride", "k_stride", "v_stride", "q_out_stride"};
  for (int i = 0; i < 4; ++i) {
    const bool is_q = i == 0 || i == 3;
    if (is_q && d->num_q_heads == 0) continue;
    const int64_t row = static_cast<int64_t>(is_q ? d->num_q_heads
                                                  : d->num_kv_heads) *
                        d->head_dim;
    if (strides[i] % 8 || (d->total_q > 1 && strides[i] < row))
      return fail(PA_ERR_INVALID_ARG,
                  "%s: %s %lld must be a multiple of 8 elements and at least "
                  "a row (%lld)", fn, names[i],
                  static_cast<long long>(strides[i]),
                  static_cast<long long>(row));
  }
  return PA_OK;
}

template <typename T, int D, bool kQ8>
pa_status launch(const char* fn, const AppendArgs& a, int64_t ctas,
                 cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, append_kernel<T, D, kQ8>, a);
  count_launch();
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(PA_ERR_CUDA, "%s: launch failed: %s", fn,
                cudaGetErrorString(e));
  return PA_OK;
}

template <bool kQ8>
pa_status append(const char* fn, void* q_out, void* k_cache, void* v_cache,
                 float* k_scales, float* v_scales, const void* q,
                 const void* k, const void* v, const void* q_norm,
                 const void* k_norm, const double* rope_freqs,
                 const int32_t* block_tables, const int32_t* context_lens,
                 const int32_t* query_start, const pa_append_desc* d,
                 int32_t* dev_err, void* stream) {
  clear_error();
  const pa_status st = check_append(fn, d);
  if (st != PA_OK) return st;
  if (!query_start && d->total_q != d->num_seqs)
    return fail(PA_ERR_INVALID_ARG,
                "%s: without query_start every sequence has one row, but "
                "total_q %d != num_seqs %d", fn, d->total_q, d->num_seqs);
  // (one row per sequence needs no bound)
  const int max_q_len = query_start ? d->max_q_len : 1;
  if (d->num_seqs == 0 || d->total_q == 0 || max_q_len == 0) return PA_OK;
  if (!k_cache || !v_cache || !k || !v || !block_tables || !context_lens ||
      (d->num_q_heads > 0 && (!q || !q_out)) ||
      (kQ8 && (!k_scales || !v_scales)))
    return fail(PA_ERR_INVALID_ARG, "%s: NULL tensor pointer", fn);
  if (d->rot_dim > 0 && !rope_freqs)
    return fail(PA_ERR_INVALID_ARG, "%s: rot_dim %d without rope_freqs", fn,
                d->rot_dim);
  if (q && q_out == q && d->total_q > 1 && d->q_stride != d->q_out_stride)
    return fail(PA_ERR_INVALID_ARG,
                "%s: q_out is q, but their strides %lld and %lld differ", fn,
                static_cast<long long>(d->q_out_stride),
                static_cast<long long>(d->q_stride));
  const void* aligned[8] = {q_out, k_cache, v_cache, q, k, v, q_norm, k_norm};
  for (const void* p : aligned)
    if (!aligned16(p))
      return fail(PA_ERR_INVALID_ARG,
                  "%s: q, k, v, q_out, the norm weights and the caches must "
                  "be 16-byte aligned", fn);
  if (d->num_blocks == 0)
    return fail(PA_ERR_INVALID_ARG, "%s: empty block pool", fn);
  AppendArgs a;
  a.q_out = q_out;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_norm = d->num_q_heads > 0 ? q_norm : nullptr;
  a.k_norm = k_norm;
  a.freqs = rope_freqs;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.query_start = query_start;
  a.dev_err = dev_err;
  a.q_stride = d->q_stride;
  a.k_stride = d->k_stride;
  a.v_stride = d->v_stride;
  a.q_out_stride = d->q_out_stride;
  a.num_seqs = d->num_seqs;
  a.num_q_heads = d->num_q_heads;
  a.num_kv_heads = d->num_kv_heads;
  a.block_size = d->block_size;
  a.max_blocks_per_seq = d->max_blocks_per_seq;
  a.num_blocks = d->num_blocks;
  a.total_q = d->total_q;
  a.max_q_len = max_q_len;
  a.rot_pairs = d->rot_dim / 2;
  a.interleaved = d->rope_layout == PA_ROPE_INTERLEAVED;
  a.rope_scale = d->rope_scale;
  a.norm_eps = d->norm_eps;
  // Rows of one token: a CTA takes them in passes of 32 (head_dim 128) or 64.
  // With few tokens the passes are dealt out to several CTAs, as long as the
  // grid stays within about four CTAs per SM; with many a CTA streams up to
  // four tokens, as long as it leaves that many.
  const int slots = kThreads / (d->head_dim / 16);
  const int rows = d->num_q_heads + (kQ8 ? 0 : 2 * d->num_kv_heads);
  const int passes = (rows + slots - 1) / slots;
  const int64_t room = 4LL * device_sm_count();
  a.row_splits = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>(passes, room / d->total_q)));
  a.tokens = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>(kMaxTokens, d->total_q / room)));
  int64_t ctas = (static_cast<int64_t>(d->total_q) + a.tokens - 1) /
                 a.tokens * a.row_splits;
  if (rows == 0) ctas = 0;
  a.kv_ctas = 0;
  a.window = 1;
  a.unit_groups = 1;
  if (kQ8) {
    // A window of one row per CTA when every row starts a run (a decode
    // step) or rows are few; with many rows most start none, and windows of
    // up to 16 rows keep the CTAs that find nothing to do few.
    a.unit_groups = (2 * d->num_kv_heads + kWarps - 1) / kWarps;
    const int64_t units = static_cast<int64_t>(d->total_q) * a.unit_groups;
    while (query_start && a.window < kMaxWindow &&
           units / a.window > 8LL * device_sm_count())
      a.window *= 2;
    const int64_t windows =
        (static_cast<int64_t>(d->total_q) + a.window - 1) / a.window;
    if (windows * a.unit_groups + ctas > 0x7fffffffLL)
      return fail(PA_ERR_UNSUPPORTED, "%s: %d rows are too many", fn,
                  d->total_q);
    a.kv_ctas = static_cast<int>(windows * a.unit_groups);
    ctas += a.kv_ctas;
  }
  if (ctas > 0x7fffffffLL)
    return fail(PA_ERR_UNSUPPORTED, "%s: %d rows are too many", fn,
                d->total_q);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->dtype == PA_BF16)
    return d->head_dim == 128
               ? launch<__nv_bfloat16, 128, kQ8>(fn, a, ctas, s)
               : launch<__nv_bfloat16, 64, kQ8>(fn, a, ctas, s);
  return d->head_dim == 128 ? launch<__half, 128, kQ8>(fn, a, ctas, s)
                            : launch<__half, 64, kQ8>(fn, a, ctas, s);
}

}  // namespace
}  // namespace pagedkv

using pagedkv::fail;

extern "C" {

pa_status pa_append(void* q_out, void* k_cache, void* v_cache, const void* q,
                    const void* k, const void* v, const void* q_norm,
                    const void* k_norm, const double* rope_freqs,
                    const int32_t* block_tables, const int32_t* context_lens,
                    const int32_t* query_start, const pa_append_desc* desc,
                    int32_t* dev_err, void* stream) {
  return pagedkv::append<false>("pa_append", q_out, k_cache, v_cache, nullptr,
                                nullptr, q, k, v, q_norm, k_norm, rope_freqs,
                                block_tables, context_lens, query_start, desc,
                                dev_err, stream);
}

pa_status pa_append_q8(void* q_out, void* k_cache, void* v_cache,
                       float* k_scales, float* v_scales, const void* q,
                       const void* k, const void* v, const void* q_norm,
                       const void* k_norm, const double* rope_freqs,
                       const int32_t* block_tables,
                       const int32_t* context_lens,
                       const int32_t* query_start, const pa_append_desc* desc,
                       int32_t* dev_err, void* stream) {
  return pagedkv::append<true>("pa_append_q8", q_out, k_cache, v_cache,
                               k_scales, v_scales, q, k, v, q_norm, k_norm,
                               rope_freqs, block_tables, context_lens,
                               query_start, desc, dev_err, stream);
}

// Host only: the angular frequencies of the rotation (see pagedkv.h).
pa_status pa_rope_freqs(const pa_rope_desc* d, double* freqs_out,
                        float* scale_out) {
  pagedkv::clear_error();
  if (!d || !freqs_out || !scale_out)
    return fail(PA_ERR_INVALID_ARG, "pa_rope_freqs: NULL pointer");
  if (d->rot_dim <= 0 || d->rot_dim % 2 || !(d->base > 1.0) ||
      !std::isfinite(d->base))
    return fail(PA_ERR_INVALID_ARG, "pa_rope_freqs: rot_dim=%d base=%g",
                d->rot_dim, d->base);
  const bool scaled = d->scaling != PA_ROPE_PLAIN;
  const bool banded = d->scaling == PA_ROPE_WAVELENGTH ||
                      d->scaling == PA_ROPE_YARN;
  if (d->scaling < PA_ROPE_PLAIN || d->scaling > PA_ROPE_YARN ||
      (scaled && !(std::isfinite(d->factor) && d->factor >= 1.0)) ||
      (banded && (d->original_len <= 0 || !(d->low > 0.0) ||
                  !(d->high > d->low) || !std::isfinite(d->high))))
    return fail(PA_ERR_INVALID_ARG,
                "pa_rope_freqs: scaling=%d factor=%g original_len=%d low=%g "
                "high=%g", d->scaling, d->factor, d->original_len, d->low,
                d->high);
  const double two_pi = 6.283185307179586477;
  // Yarn's ramp over the pairs: pair(r) turns r times in original_len.
  double first = 0.0, last = 0.0;
  if (d->scaling == PA_ROPE_YARN) {
    auto pair = [&](double turns) {
      return d->rot_dim * std::log(d->original_len / (turns * two_pi)) /
             (2.0 * std::log(d->base));
    };
    first = std::max(std::floor(pair(d->high)), 0.0);
    last = std::min(std::ceil(pair(d->low)), d->rot_dim - 1.0);
    if (last <= first) last = first + 0.001;
  }
  for (int j = 0; j < d->rot_dim / 2; ++j) {
    const double f = std::pow(d->base, -2.0 * j / d->rot_dim);
    double w = 0.0;  // how much of f is divided by the factor
    if (d->scaling == PA_ROPE_LINEAR) {
      w = 1.0;
    } else if (d->scaling == PA_ROPE_WAVELENGTH) {
      const double turns = d->original_len * f / two_pi;
      w = std::min(1.0, std::max(0.0, (d->high - turns) / (d->high - d->low)));
    } else if (d->scaling == PA_ROPE_YARN) {
      w = std::min(1.0, std::max(0.0, (j - first) / (last - first)));
    }
    freqs_out[j] = scaled ? w * (f / d->factor) + (1.0 - w) * f : f;
  }
  *scale_out = d->scaling == PA_ROPE_YARN && d->factor > 1.0
                   ? static_cast<float>(0.1 * std::log(d->factor) + 1.0)
                   : 1.f;
  return PA_OK;
}

}  // extern "C"
