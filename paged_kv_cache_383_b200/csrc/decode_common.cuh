// What the decode kernels share (the 16-bit cache's in decode.cu, the 8-bit
// cache's in decode_q8.cu): the arguments and the workspace, the longest-first
// prep kernel, the combination of a sequence's partitions (in the decode
// kernel or by a separate reduce kernel), the choice of the partition size,
// the checks of a call, and the launch of the chain.  Each translation unit
// gets its own copy (anonymous namespace).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "device_utils.cuh"
#include "order.cuh"
#include "pagedkv.h"
#include "status.h"

namespace pagedkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kConsumers = 4;                      // consumer warps per CTA
constexpr int kThreads = (kConsumers + 1) * 32;    // + one producer warp
constexpr int kMaxGroup = 8;                       // query heads per KV head
constexpr int kMaxPartition = 8192;
constexpr int kMaxParts = 16384;                   // partitions per sequence
constexpr int kFusedMaxParts = 16;  // up to this many: combine in the decode
constexpr int kWarpPartsMaxPartition = 1024;  // warp_parts up to this size

struct DecodeArgs {
  void* out;
  const void* q;
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* ws_o;   // [num_seqs, num_q_heads, max_parts, head_dim]
  float* ws_ml;  // [num_seqs, num_q_heads, max_parts, 2] = (max, sum), log2 units
  int* counters; // [num_seqs, num_kv_heads] finished partitions (fused mode)
  const int32_t* order;  // [num_seqs] sequence served by grid row z
  // [num_seqs * max_parts] partition units longest first (entry u: sequence
  // u / max_parts, partition u % max_parts); non-null when the grid is
  // (KV head, unit) rather than (partition, KV head, sequence)
  const int32_t* units;
  int fused;     // 1: the last partition CTA combines; 0: the reduce kernel
  int warp_parts;  // 1: a CTA serves kConsumers consecutive partitions, one
                   // per consumer warp (reduce kernel path, short partitions)
  int32_t* dev_err;
  float scale_log2;  // scale * log2(e): scores are kept in base-2 units
  int num_q_heads;
  int num_kv_heads;
  int group;
  int max_blocks_per_seq;
  int num_blocks;
  int partition_size;
  int max_parts;
  int max_context_len;
  int out_f32;   // 1: out is float32 (the value before the cast to T)
};

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float(float x) {
  return __float2half_rn(x);
}

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float to_float(__half x) {
  return __half2float(x);
}

__device__ __forceinline__ float warp_max_xor(float v, int lo_mask,
                                              int hi_mask) {
  for (int m = lo_mask; m <= hi_mask; m <<= 1)
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
  return v;
}

// Final store of one output element: rounded once to the output dtype, or,
// on request, the fp32 value itself (lets tests separate the kernel's error
// from the output rounding).
template <typename T>
__device__ __forceinline__ void store_out(const DecodeArgs& a, int64_t idx,
                                          float v) {
  if (a.out_f32)
    static_cast<float*>(a.out)[idx] = v;
  else
    static_cast<T*>(a.out)[idx] = from_float<T>(v);
}

// ---------------------------------------------------------------------------
// Fused combine of one (sequence, KV head)'s partitions, run by threads
// [t, ...) step nt of the partition CTA that finished last:
//   out = sum_j w_j o_j / sum_j w_j,  w_j = l_j 2^(m_j - M),  M = max_j m_j.
// Thread item = (query head g, 16-lane slice of head_dim); four partitions
// are loaded before they are folded.
template <typename T, int D>
__device__ __forceinline__ void combine_partials(const DecodeArgs& a, int b,
                                                 int kvh, int n_parts, int t,
                                                 int nt) {
  constexpr int kDT = D / 16;  // dims per thread: 8 or 4
  const int G = a.group;
  const float2* ml2 = reinterpret_cast<const float2*>(a.ws_ml);
  for (int item = t; item < G * 16; item += nt) {
    const int g = item >> 4;
    const int d0 = (item & 15) * kDT;
    const int64_t row0 =
        (static_cast<int64_t>(b) * a.num_q_heads + kvh * G + g) * a.max_parts;
    float M = -INFINITY, W = 0.f;
    float acc[kDT];
#pragma unroll
    for (int e = 0; e < kDT; ++e) acc[e] = 0.f;
    for (int j0 = 0; j0 < n_parts; j0 += 4) {
      float2 mlj[4];
      float oj[4][kDT];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + u;
        mlj[u] = j < n_parts ? __ldcg(ml2 + row0 + j)
                             : make_float2(-INFINITY, 0.f);
        const float4* src =
            reinterpret_cast<const float4*>(a.ws_o + (row0 + j) * D + d0);
#pragma unroll
        for (int v = 0; v < kDT / 4; ++v) {
          const float4 x = j < n_parts ? __ldcg(src + v)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
          oj[u][4 * v] = x.x;
          oj[u][4 * v + 1] = x.y;
          oj[u][4 * v + 2] = x.z;
          oj[u][4 * v + 3] = x.w;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (mlj[u].x == -INFINITY) continue;  // empty or skipped partition
        if (mlj[u].x > M) {
          const float sc = dev::fast_exp2(M - mlj[u].x);  // 0 when M = -inf
          W *= sc;
#pragma unroll
          for (int e = 0; e < kDT; ++e) acc[e] *= sc;
          M = mlj[u].x;
        }
        const float w = mlj[u].y * dev::fast_exp2(mlj[u].x - M);
        W += w;
#pragma unroll
        for (int e = 0; e < kDT; ++e) acc[e] += w * oj[u][e];
      }
    }
    const int64_t dst =
        (static_cast<int64_t>(b) * a.num_q_heads + kvh * G + g) * D + d0;
#pragma unroll
    for (int e = 0; e < kDT; ++e)
      store_out<T>(a, dst + e, W > 0.f ? acc[e] / W : 0.f);
  }
}
// ---------------------------------------------------------------------------
// Prep kernel (one CTA), run before every decode: orders the sequences
// longest first (a counting sort on context_len >> shift, 1024 buckets,
// descending) into `order` (with a unit grid: the (sequence, partition)
// units by token count into `units` instead), and zeroes the per-(sequence,
// KV head) partition counters when the decode combines in place.  Launched
// with programmatic stream serialization: it sorts while the previous kernel
// drains (it reads only host-written lengths), then waits for that kernel,
// which may still read `order`, the counters and `units`, before writing
// them.  The decode's own wait covers the prep kernel.  Within one bucket the
// order follows the atomics; results do not depend on it (each unit is
// computed on its own and partials are combined in partition order).
__global__ void __launch_bounds__(kOrderThreads)
    prep_kernel(const int32_t* __restrict__ context_lens, int num_seqs,
                int shift, int32_t* __restrict__ order, int* counters,
                int n_counters, int32_t* __restrict__ units, int max_parts,
                int partition_size, int unit_shift) {
  dev::pdl_trigger();
  if (units) {
    // Partition units by token count, largest first: unit u is partition
    // u % max_parts of sequence u / max_parts (empty past the sequence).
    // The unit grid does not read `order`.
    counting_sort_desc(
        num_seqs * max_parts,
        [&](int u) {
          const int b = u / max_parts;
          const int p = u - b * max_parts;
          const int left = context_lens[b] - p * partition_size;
          const int n = left <= 0 ? 0 : min(left, partition_size);
          return n >> unit_shift;
        },
        units, [] { dev::pdl_wait(); });
  } else {
    sort_longest_first(context_lens, num_seqs, shift, order,
                       [] { dev::pdl_wait(); });
  }
  for (int i = threadIdx.x; i < n_counters; i += kOrderThreads)
    counters[i] = 0;
}

// ---------------------------------------------------------------------------
// Partition reduce: out = sum_j w_j o_j / sum_j w_j, w_j = l_j 2^(m_j - M),
// M = max_j m_j (all in base-2 units).
// One CTA per (query head, sequence); warp w folds partitions w, w+8, ...
// with a running max, sixteen partitions in flight per warp (eight at
// head_dim 64; one 16- or 8-byte load per lane each), and the eight warp
// states are merged through shared memory.  The partials were just written
// by the decode and are read once, so the time is the latency of a few
// rounds of loads: 128 partitions in flight per CTA keep that to one or two
// rounds for the longest sequences, and 256 threads let two CTAs share an SM
// (the grid, one CTA per query head and sequence, is a few waves).  Used
// when a sequence has many partitions (the fused combine handles few).
constexpr int kReduceWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kReduceWarps * 32)
    reduce_kernel(const DecodeArgs a, int block_size) {
  constexpr int kPer = D / 32;  // dims per lane
  __shared__ float s_m[kReduceWarps], s_w[kReduceWarps];
  __shared__ float s_acc[kReduceWarps][D];
  const int qh = blockIdx.x;
  const int b = blockIdx.y;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  dev::pdl_trigger();
  const int ctx = a.context_lens[b];
  // The decode kernel has completed and its partials are visible.  CTAs with
  // nothing to do wait too: were they to leave at once, this grid could be
  // over before the decode is, and the kernel launched behind it, which waits
  // for this grid only, would overwrite what the decode still reads.
  dev::pdl_wait();
  if (ctx < 0 || ctx > a.max_blocks_per_seq * block_size ||
      ctx > a.max_context_len)
    return;  // flagged by the decode kernel
  const int n_parts = ctx > 0 ? (ctx + a.partition_size - 1) / a.partition_size
                              : 1;
  if (n_parts <= 1) return;  // the decode kernel wrote this row itself

  const int64_t row0 =
      (static_cast<int64_t>(b) * a.num_q_heads + qh) * a.max_parts;
  const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) + row0;
  const float* o = a.ws_o + row0 * D + lane * kPer;
  float M = -INFINITY, W = 0.f;
  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  // partitions in flight per warp (head_dim 64: 8, which needs no spill)
  constexpr int kBatch = kPer == 4 ? 16 : 8;
  static_assert(kPer == 4 || kPer == 2, "head_dim 128 or 64");
  for (int j0 = warp; j0 < n_parts; j0 += kBatch * kReduceWarps) {
    float2 mlj[kBatch];
    float oj[kBatch][kPer];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = j0 + u * kReduceWarps;
      mlj[u] = j < n_parts ? __ldcg(ml + j) : make_float2(-INFINITY, 0.f);
      // this lane's kPer consecutive dims: one 16- (or 8-) byte load; a
      // partial row is D floats, 16-byte aligned
      const float* src = o + static_cast<int64_t>(j) * D;
      if constexpr (kPer == 4) {
        const float4 v = j < n_parts
                             ? __ldcg(reinterpret_cast<const float4*>(src))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
        oj[u][0] = v.x;
        oj[u][1] = v.y;
        oj[u][2] = v.z;
        oj[u][3] = v.w;
      } else {
        const float2 v = j < n_parts
                             ? __ldcg(reinterpret_cast<const float2*>(src))
                             : make_float2(0.f, 0.f);
        oj[u][0] = v.x;
        oj[u][1] = v.y;
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (mlj[u].x == -INFINITY) continue;  // empty or skipped partition
      if (mlj[u].x > M) {
        const float sc = dev::fast_exp2(M - mlj[u].x);  // 0 when M = -inf
        W *= sc;
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] *= sc;
        M = mlj[u].x;
      }
      const float w = mlj[u].y * dev::fast_exp2(mlj[u].x - M);
      W += w;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] += w * oj[u][e];
    }
  }
  if (lane == 0) {
    s_m[warp] = M;
    s_w[warp] = W;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) s_acc[warp][lane * kPer + e] = acc[e];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kReduceWarps * 32) {
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kReduceWarps; ++w) mx = fmaxf(mx, s_m[w]);
    float tw = 0.f, tv = 0.f;
    if (mx != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kReduceWarps; ++w) {
        const float sc =
            s_m[w] == -INFINITY ? 0.f : dev::fast_exp2(s_m[w] - mx);
        tw += s_w[w] * sc;
        tv += s_acc[w][d] * sc;
      }
    }
    store_out<T>(a, (static_cast<int64_t>(b) * a.num_q_heads + qh) * D + d,
                 tw > 0.f ? tv / tw : 0.f);
  }
}

// ---------------------------------------------------------------------------
// Host side.

#ifndef PAGEDKV_PDL
#define PAGEDKV_PDL 1  // programmatic dependent launch between the kernels
#endif
constexpr int kUsePdl = PAGEDKV_PDL;

int resolve_partition(const pa_decode_desc* d, int max_ctx) {
  if (d->partition_size > 0) return d->partition_size;
  const int64_t pairs = static_cast<int64_t>(d->num_seqs) * d->num_kv_heads;
  const int64_t target = 3LL * device_sm_count();
  // Long partitions (fewer CTAs, less ramp-up and fewer partials) as long as
  // the grid keeps at least 6 units per SM were every sequence max_ctx long;
  // the prep kernel's longest-first order keeps the tail short.  Measured:
  // 4096 is best on the batch-256 and 8-sequence long-context mixes, 2048 on
  // the batch-64 mix (8192 loses everywhere).
  for (int big = 4096; big >= 2048; big /= 2)
    if (pairs * ((max_ctx + big - 1) / big) >= 6LL * device_sm_count() &&
        big % d->block_size == 0)
      return big;
  int ps = 1024;
  while (ps > 2 * d->block_size && ps > 64 &&
         pairs * ((max_ctx + ps - 1) / ps) < target)
    ps /= 2;
  if (ps < d->block_size) ps = d->block_size;
  return ps;
}

int resolve_max_ctx(const pa_decode_desc* d) {
  return d->max_context_len > 0 ? d->max_context_len
                                : d->max_blocks_per_seq * d->block_size;
}

pa_status check_desc(const pa_decode_desc* d, const char* fn) {
  if (!d) return fail(PA_ERR_INVALID_ARG, "%s: desc is NULL", fn);
  if (d->num_seqs < 0 || d->num_q_heads <= 0 || d->num_kv_heads <= 0 ||
      d->max_blocks_per_seq <= 0 || d->num_blocks < 0 ||
      d->max_context_len < 0 || d->partition_size < 0)
    return fail(PA_ERR_INVALID_ARG,
                "%s: num_seqs=%d num_q_heads=%d num_kv_heads=%d "
                "max_blocks_per_seq=%d num_blocks=%d max_context_len=%d "
                "partition_size=%d", fn, d->num_seqs, d->num_q_heads,
                d->num_kv_heads, d->max_blocks_per_seq, d->num_blocks,
                d->max_context_len, d->partition_size);
  if (d->num_q_heads % d->num_kv_heads)
    return fail(PA_ERR_INVALID_ARG,
                "%s: num_q_heads %d is not a multiple of num_kv_heads %d", fn,
                d->num_q_heads, d->num_kv_heads);
  if (d->num_q_heads / d->num_kv_heads > kMaxGroup)
    return fail(PA_ERR_UNSUPPORTED, "%s: group size %d > %d", fn,
                d->num_q_heads / d->num_kv_heads, kMaxGroup);
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(PA_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128}", fn,
                d->head_dim);
  if (d->block_size != 16 && d->block_size != 32)
    return fail(PA_ERR_UNSUPPORTED, "%s: block_size %d not in {16, 32}", fn,
                d->block_size);
  if (d->dtype != PA_F16 && d->dtype != PA_BF16)
    return fail(PA_ERR_INVALID_ARG, "%s: dtype %d", fn,
                static_cast<int>(d->dtype));
  if (d->reduce != PA_REDUCE_AUTO && d->reduce != PA_REDUCE_KERNEL)
    return fail(PA_ERR_INVALID_ARG, "%s: reduce %d", fn,
                static_cast<int>(d->reduce));
  if (d->out_fp32 != 0 && d->out_fp32 != 1)
    return fail(PA_ERR_INVALID_ARG, "%s: out_fp32 %d", fn, d->out_fp32);
  if (d->kernel != PA_KERNEL_AUTO && d->kernel != PA_KERNEL_SIMT &&
      d->kernel != PA_KERNEL_MMA)
    return fail(PA_ERR_INVALID_ARG, "%s: kernel %d", fn,
                static_cast<int>(d->kernel));
  if (d->partition_size > 0 &&
      (d->partition_size % d->block_size || d->partition_size > kMaxPartition))
    return fail(PA_ERR_INVALID_ARG,
                "%s: partition_size %d must be a multiple of block_size "
                "%d and <= %d", fn, d->partition_size, d->block_size,
                kMaxPartition);
  if (static_cast<int64_t>(d->max_blocks_per_seq) * d->block_size >
      0x7fffffffLL)
    return fail(PA_ERR_INVALID_ARG, "%s: max_blocks_per_seq too large", fn);
  if (static_cast<int64_t>(d->num_blocks) * d->num_kv_heads * d->block_size >
      0x7fffffffLL)
    return fail(PA_ERR_UNSUPPORTED,
                "%s: num_blocks * num_kv_heads * block_size exceeds "
                "2^31 rows", fn);
  if (d->num_seqs > 65535 || d->num_kv_heads > 65535)
    return fail(PA_ERR_UNSUPPORTED,
                "%s: num_seqs and num_kv_heads must be <= 65535", fn);
  return PA_OK;
}

// Workspace layout, in bytes from the start: partials o and (m, l) and the
// partition counters (only with more than one partition), then the sequence
// order; each piece 16-byte aligned.
struct WsLayout {
  size_t o = 0, ml = 0, counters = 0, units = 0, order = 0, total = 0;
};

WsLayout ws_layout(const pa_decode_desc* d) {
  auto up16 = [](size_t x) { return (x + 15) & ~size_t(15); };
  const int max_ctx = resolve_max_ctx(d);
  const int ps = resolve_partition(d, max_ctx);
  const int64_t parts = max_ctx > 0 ? (max_ctx + ps - 1) / ps : 1;
  WsLayout w;
  size_t at = 0;
  if (parts > 1) {
    const size_t rows = static_cast<size_t>(d->num_seqs) * d->num_q_heads *
                        static_cast<size_t>(parts);
    w.o = at;
    at += up16(rows * d->head_dim * sizeof(float));
    w.ml = at;
    at += up16(rows * 2 * sizeof(float));
    w.counters = at;
    at += up16(static_cast<size_t>(d->num_seqs) * d->num_kv_heads *
               sizeof(int));
    w.units = at;
    at += up16(static_cast<size_t>(d->num_seqs) * static_cast<size_t>(parts) *
               sizeof(int32_t));
  }
  w.order = at;
  at += up16(static_cast<size_t>(d->num_seqs) * sizeof(int32_t));
  w.total = at;
  return w;
}

size_t workspace_bytes(const pa_decode_desc* d) { return ws_layout(d).total; }


// Combine partitions inside the decode kernel (few partitions) or with the
// separate reduce kernel.
bool use_fused(const pa_decode_desc* d, int parts) {
  return d->reduce == PA_REDUCE_AUTO && parts <= kFusedMaxParts;
}

// Launch one call's kernels: the prep kernel, the decode (launch_decode is
// given its launch configuration) and, when partitions are not combined in
// the decode, the reduce kernel.
template <typename T, int D, int BS, typename LaunchDecode>
pa_status launch_chain(const char* fn, const pa_decode_desc* d,
                       const DecodeArgs& a, size_t smem, cudaStream_t stream,
                       LaunchDecode launch_decode) {
  // Every kernel here (the prep, the decode, the reduce) is
  // launched with programmatic stream serialization: each may start while
  // its predecessor drains and waits (griddepcontrol.wait) before touching
  // memory the predecessor writes.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = kUsePdl;
  {
    const int n = (a.max_parts > 1 && a.fused)
                      ? d->num_seqs * d->num_kv_heads
                      : 0;
    cudaLaunchConfig_t pcfg = {};
    pcfg.gridDim = dim3(1);
    pcfg.blockDim = dim3(kOrderThreads);
    pcfg.stream = stream;
    pcfg.attrs = attr;
    pcfg.numAttrs = 1;
    const cudaError_t pe = cudaLaunchKernelEx(
        &pcfg, prep_kernel, a.context_lens, d->num_seqs,
        order_shift(a.max_context_len), const_cast<int32_t*>(a.order),
        a.counters, n, const_cast<int32_t*>(a.units), a.max_parts,
        a.partition_size, order_shift(a.partition_size));
    count_launch();
    if (pe != cudaSuccess)
      return fail(PA_ERR_CUDA, "%s: prep launch failed: %s", fn,
                  cudaGetErrorString(pe));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim =
      a.units ? dim3(d->num_kv_heads, d->num_seqs * a.max_parts, 1)
              : dim3(a.warp_parts ? (a.max_parts + kConsumers - 1) / kConsumers
                                  : a.max_parts,
                     d->num_kv_heads, d->num_seqs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = launch_decode(cfg);
  count_launch();
  if (e != cudaSuccess)
    return fail(PA_ERR_CUDA, "%s: decode launch failed: %s", fn,
                cudaGetErrorString(e));
  if (a.max_parts > 1 && !a.fused) {
    cudaLaunchConfig_t rcfg = {};
    rcfg.gridDim = dim3(d->num_q_heads, d->num_seqs);
    rcfg.blockDim = dim3(kReduceWarps * 32);
    rcfg.dynamicSmemBytes = 0;
    rcfg.stream = stream;
    rcfg.attrs = attr;
    rcfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&rcfg, reduce_kernel<T, D>, a, BS);
    count_launch();
    if (e != cudaSuccess)
      return fail(PA_ERR_CUDA, "%s: reduce launch failed: %s", fn,
                  cudaGetErrorString(e));
  }
  return PA_OK;
}


// The checks of one call past its descriptor's (num_seqs 0: nothing to do).
pa_status check_call(const char* fn, const void* out, const void* q,
                     const void* k_cache, const void* v_cache,
                     const int32_t* block_tables, const int32_t* context_lens,
                     float scale, const pa_decode_desc* desc,
                     const void* workspace, size_t workspace_size) {
  if (!std::isfinite(scale))
    return fail(PA_ERR_INVALID_ARG, "%s: scale is not finite", fn);
  if (desc->num_seqs == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens)
    return fail(PA_ERR_INVALID_ARG, "%s: NULL tensor pointer", fn);
  if (!aligned16(out) || !aligned16(q) ||
      !aligned16(k_cache) || !aligned16(v_cache))
    return fail(PA_ERR_INVALID_ARG,
                "%s: out, q and the caches must be 16-byte aligned", fn);
  if (desc->num_blocks == 0)
    return fail(PA_ERR_INVALID_ARG, "%s: empty block pool", fn);

  const int max_ctx = resolve_max_ctx(desc);
  const int ps = resolve_partition(desc, max_ctx);
  const int parts = max_ctx > 0 ? (max_ctx + ps - 1) / ps : 1;
  if (parts > kMaxParts)
    return fail(PA_ERR_UNSUPPORTED,
                "%s: %d partitions of %d tokens exceed %d; use a "
                "larger partition_size", fn, parts, ps, kMaxParts);
  const size_t need = workspace_bytes(desc);
  if (need > 0 && (!workspace || workspace_size < need ||
                   !aligned16(workspace)))
    return fail(PA_ERR_WORKSPACE,
                "%s: workspace of %zu bytes (16-byte aligned) needed, "
                "got %zu at %p", fn, need, workspace_size, workspace);
  return PA_OK;
}

// The arguments of one checked call (out, q and the workspace's pieces).
DecodeArgs make_args(void* out, const void* q, const int32_t* block_tables,
                     const int32_t* context_lens, float scale,
                     const pa_decode_desc* desc, void* workspace,
                     int32_t* dev_err) {
  const int max_ctx = resolve_max_ctx(desc);
  const int ps = resolve_partition(desc, max_ctx);
  const int parts = max_ctx > 0 ? (max_ctx + ps - 1) / ps : 1;
  DecodeArgs a;
  a.out = out;
  a.q = q;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  const WsLayout wl = ws_layout(desc);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.ws_o = parts > 1 ? reinterpret_cast<float*>(ws + wl.o) : nullptr;
  a.ws_ml = parts > 1 ? reinterpret_cast<float*>(ws + wl.ml) : nullptr;
  a.counters = parts > 1 ? reinterpret_cast<int*>(ws + wl.counters) : nullptr;
  a.order = reinterpret_cast<const int32_t*>(ws + wl.order);
  a.fused = use_fused(desc, parts) ? 1 : 0;
  // Short partitions combined by the reduce kernel: one partition per
  // consumer warp, kConsumers per CTA (fewer, longer CTAs; no merge).
  a.warp_parts = (desc->kernel != PA_KERNEL_SIMT && !a.fused && parts > 1 &&
                  ps <= kWarpPartsMaxPartition)
                     ? 1
                     : 0;
  a.dev_err = dev_err;
  a.scale_log2 = scale * kLog2e;
  a.num_q_heads = desc->num_q_heads;
  a.num_kv_heads = desc->num_kv_heads;
  a.group = desc->num_q_heads / desc->num_kv_heads;
  a.max_blocks_per_seq = desc->max_blocks_per_seq;
  a.num_blocks = desc->num_blocks;
  a.partition_size = ps;
  a.max_parts = parts;
  a.max_context_len = max_ctx;
  a.out_f32 = desc->out_fp32;
  // Long partitions, one per CTA, in a grid of a few waves: the grid runs
  // (KV head, unit) with the units longest first, so the last CTAs hold the
  // shortest partitions.  Ordered by sequence instead, the second wave can
  // start full-length partitions of mid-length sequences and end on a long
  // tail (batch 64 at 2048-token partitions: 6.12 -> 6.24 TB/s).  With many
  // waves the sequence order already ends on short work, and with short
  // partitions the extra sort in the prep kernel costs more than the tail
  // (gridDim.y caps the unit count).
  const int64_t n_units = static_cast<int64_t>(desc->num_seqs) * parts;
  a.units = (parts > 1 && !a.warp_parts && ps >= 1024 && n_units <= 65535 &&
             // at most four waves of three CTAs per SM
             n_units * desc->num_kv_heads <= 12LL * device_sm_count())
                ? reinterpret_cast<const int32_t*>(ws + wl.units)
                : nullptr;
  return a;
}

}  // namespace
}  // namespace pagedkv
