// What the prefill kernels share (the 16-bit cache's in prefill.cu, the 8-bit
// cache's in prefill_q8.cu): the plan kernel that orders the sequences and
// lists their query tiles, the workspace, and the checks of a call.  Each
// translation unit gets its own copy (anonymous namespace).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "device_utils.cuh"
#include "order.cuh"
#include "pagedkv.h"
#include "status.h"

namespace pagedkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 128;  // query rows per tile (tensor memory lanes)

// One CTA: the longest-first order of the sequences (by context length),
// then the prefill's tile map in that order.  Sequence b's new tokens fill
// ceil(q_len / tok) query tiles of tok tokens; the map lists them, the last
// (the one that sees the most keys) first, as (b, tile) pairs, and (-1, 0)
// after the last one up to its capacity `cap`.  A sequence whose rows fall
// outside q, or that has more new tokens than its context or than
// max_q_len, gets no tiles and sets PA_ERR_DEVICE_OOB; so does a map that
// would overflow (rows of several sequences overlapping), which is cut at
// `cap`.  Launched by programmatic stream serialization: it reads the
// lengths and rows and sorts while the kernel before it drains, then waits
// for that kernel (which may still read the workspace: the previous
// prefill) before writing; the prefill launches early behind it.
__global__ void __launch_bounds__(kOrderThreads)
    prefill_plan_kernel(const int32_t* __restrict__ context_lens,
                        const int32_t* __restrict__ query_start, int num_seqs,
                        int total_q, int max_q_len, int shift, int tok,
                        int cap, int32_t* __restrict__ order,
                        int2* __restrict__ tiles, int* counter,
                        int32_t* dev_err) {
  dev::pdl_trigger();
  // Tile counts and their running sum in 64 bits: sequences whose rows
  // overlap (each range valid on its own) may list more than 2^31 tiles.
  __shared__ int s_b[kOrderThreads];
  __shared__ long long s_n[kOrderThreads], s_start[kOrderThreads];
  __shared__ long long s_warp[kOrderThreads / 32];
  __shared__ long long s_carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  auto tiles_of = [&](int b) -> long long {  // 0 (flagged) if invalid
    const int q0 = query_start[b], q1 = query_start[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > total_q || q1 - q0 > context_lens[b] ||
        q1 - q0 > max_q_len) {
      bad = true;
      return 0;
    }
    return (static_cast<long long>(q1 - q0) + tok - 1) / tok;
  };
  // Up to kOrderThreads sequences, one per thread: a sequence's tile count
  // is loaded with its length and the sort places both at its rank in
  // shared memory (the order itself is not stored); the ranks are scanned
  // there too, so after the wait for the previous kernel only the map's
  // stores are left.  More sequences go through `order` in global memory.
  const bool one_pass = num_seqs <= kOrderThreads;
  const long long my_n = one_pass && tid < num_seqs ? tiles_of(tid) : 0;
  auto key = [&](int i) {
    const int L = context_lens[i];
    return L <= 0 ? 0 : (L >> shift);
  };
  if (one_pass) {
    counting_sort_desc_place(
        num_seqs, key,
        [&](int pos, int i) {  // i == tid
          s_b[pos] = i;
          s_n[pos] = my_n;
        },
        [] {});
  } else {
    counting_sort_desc_place(
        num_seqs, key, [&](int pos, int i) { order[pos] = i; },
        [] { dev::pdl_wait(); });
  }
  if (tid == 0) s_carry = 0;
  __syncthreads();  // the placed ranks (and the order, for more sequences)
  for (int base = 0; base < num_seqs; base += kOrderThreads) {
    const int z = base + tid;
    int b = -1;
    long long n = 0;
    if (z < num_seqs) {
      if (one_pass) {
        b = s_b[z];
        n = s_n[z];
      } else {
        b = order[z];
        n = tiles_of(b);
      }
    }
    // Where sequence z's tiles start: a scan of the tile counts over the
    // CTA, after those of the earlier chunks (s_carry).
    long long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
      long long w = s_warp[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
      }
      s_warp[lane] = w;
    }
    __syncthreads();
    const long long incl = x + (warp > 0 ? s_warp[warp - 1] : 0);
    s_b[tid] = b;
    s_n[tid] = n;
    s_start[tid] = s_carry + incl - n;
    __syncthreads();
    // The previous kernel may still read the workspace (a no-op when
    // already waited for).
    dev::pdl_wait();
    // A warp per sequence writes its tiles, a lane per tile.
    const int cnt = min(kOrderThreads, num_seqs - base);
    for (int i = warp; i < cnt; i += kOrderThreads / 32) {
      const long long st = s_start[i];
      const int sb = s_b[i];
      // Only the tiles that fit the map: slots st .. min(st + n, cap) - 1.
      const long long end = min(st + s_n[i], static_cast<long long>(cap));
      for (long long slot = st + lane; slot < end; slot += 32)
        tiles[slot] = make_int2(sb, static_cast<int>(st + s_n[i] - 1 - slot));
    }
    __syncthreads();  // every thread has read s_carry and the chunk's rows
    if (tid == kOrderThreads - 1) s_carry += incl;
    __syncthreads();
  }
  dev::pdl_wait();
  const long long total = s_carry;
  if (total > cap) bad = true;
  for (long long i = total + tid; i < cap; i += kOrderThreads)
    tiles[i] = make_int2(-1, 0);
  if (tid == 0) *counter = 0;  // the prefill's work items start at 0
  if (bad) dev::set_error(dev_err, PA_ERR_DEVICE_OOB);
}

// New tokens per query tile (tile rows / query group) and the tile map's
// capacity: the map holds sum over sequences of ceil(q_len / tok) tiles,
// which is at most total_q / tok + num_seqs when the sequences' rows do not
// overlap, and at most num_seqs * ceil(max_q_len / tok) as the plan kernel
// drops a sequence above max_q_len.
int tile_tokens(const pa_prefill_desc* d) {
  return kRows / (d->num_q_heads / d->num_kv_heads);
}
int64_t tile_cap(const pa_prefill_desc* d, int tok) {
  return std::min(static_cast<int64_t>(d->total_q) / tok + d->num_seqs,
                  static_cast<int64_t>(d->num_seqs) *
                      ((static_cast<int64_t>(d->max_q_len) + tok - 1) / tok));
}

int64_t tile_cap(const pa_prefill_desc* d) {
  return tile_cap(d, tile_tokens(d));
}

// The sequence order (num_seqs int32, rounded up to 16 bytes), the work
// counter (16 bytes), then the tile map (int2 entries, rounded up to 16).
size_t order_bytes(const pa_prefill_desc* d) {
  return (static_cast<size_t>(d->num_seqs) * sizeof(int32_t) + 15) &
         ~size_t(15);
}
constexpr size_t kCounterBytes = 16;
size_t prefill_workspace_bytes(const pa_prefill_desc* d) {
  const size_t order = order_bytes(d);
  const int G = d->num_kv_heads > 0 ? d->num_q_heads / d->num_kv_heads : 0;
  if (d->num_q_heads <= 0 || d->num_kv_heads <= 0 || d->total_q < 0 ||
      d->max_q_len < 0 || d->num_q_heads % d->num_kv_heads || G <= 0 ||
      G > kRows)
    return order;  // the call rejects this shape
  return order + kCounterBytes +
         ((static_cast<size_t>(tile_cap(d)) * sizeof(int2) + 15) &
          ~size_t(15));
}
int* work_counter(const pa_prefill_desc* d, void* workspace) {
  return reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) +
                                order_bytes(d));
}
int2* tile_map(const pa_prefill_desc* d, void* workspace) {
  return reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) +
                                 order_bytes(d) + kCounterBytes);
}

bool nothing_to_do(const pa_prefill_desc* d) {
  return d->num_seqs == 0 || d->total_q == 0 || d->max_q_len == 0;
}

pa_status check_prefill(const char* fn, const void* out, const void* q,
                        const void* k_cache, const void* v_cache,
                        const int32_t* block_tables,
                        const int32_t* context_lens,
                        const int32_t* query_start, float scale,
                        const pa_prefill_desc* d, const void* workspace,
                        size_t workspace_bytes) {
  if (!d) return fail(PA_ERR_INVALID_ARG, "%s: desc is NULL", fn);
  if (d->num_seqs < 0 || d->num_q_heads <= 0 || d->num_kv_heads <= 0 ||
      d->max_blocks_per_seq <= 0 || d->num_blocks < 0 || d->total_q < 0 ||
      d->max_q_len < 0 || d->max_context_len < 0 ||
      d->num_q_heads % d->num_kv_heads ||
      (d->dtype != PA_F16 && d->dtype != PA_BF16) || !std::isfinite(scale))
    return fail(PA_ERR_INVALID_ARG,
                "%s: num_seqs=%d num_q_heads=%d num_kv_heads=%d "
                "max_blocks_per_seq=%d total_q=%d max_q_len=%d dtype=%d", fn,
                d->num_seqs, d->num_q_heads, d->num_kv_heads,
                d->max_blocks_per_seq, d->total_q, d->max_q_len,
                static_cast<int>(d->dtype));
  const int G = d->num_q_heads / d->num_kv_heads;
  if (d->kernel != PA_PREFILL_AUTO && d->kernel != PA_PREFILL_TILE)
    return fail(PA_ERR_INVALID_ARG, "%s: kernel %d", fn, d->kernel);
  if (d->out_fp32 != 0 && d->out_fp32 != 1)
    return fail(PA_ERR_INVALID_ARG, "%s: out_fp32 %d", fn, d->out_fp32);
  if (d->pv < PA_PV_AUTO || d->pv > PA_PV_SINGLE)
    return fail(PA_ERR_INVALID_ARG, "%s: pv %d", fn, d->pv);
  if ((d->head_dim != 64 && d->head_dim != 128) ||
      (d->block_size != 16 && d->block_size != 32) ||
      (G != 1 && G != 2 && G != 4 && G != 8))
    return fail(PA_ERR_UNSUPPORTED,
                "%s: needs head_dim 64 or 128 (got %d), block_size "
                "16 or 32 (got %d) and a query group of 1, 2, 4 or 8 (got %d)", fn,
                d->head_dim, d->block_size, G);
  if (static_cast<int64_t>(d->max_blocks_per_seq) * d->block_size >
      0x7fffffffLL)
    return fail(PA_ERR_INVALID_ARG, "%s: max_blocks_per_seq too large", fn);
  if (nothing_to_do(d)) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens ||
      !query_start)
    return fail(PA_ERR_INVALID_ARG, "%s: NULL tensor pointer", fn);
  if (!aligned16(out) || !aligned16(q) ||
      !aligned16(k_cache) || !aligned16(v_cache))
    return fail(PA_ERR_INVALID_ARG,
                "%s: out, q and the caches must be 16-byte aligned", fn);
  // Work items (tile-map entry, KV head) are counted in an int.
  if (tile_cap(d) * d->num_kv_heads > 0x7fffffffLL)
    return fail(PA_ERR_UNSUPPORTED,
                "%s: %lld query tiles x %d KV heads exceed 2^31 - 1 "
                "work items", fn,
                static_cast<long long>(tile_cap(d)),
                d->num_kv_heads);
  const size_t need = prefill_workspace_bytes(d);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return fail(PA_ERR_WORKSPACE,
                "%s: workspace of %zu bytes (16-byte aligned) needed, "
                "got %zu at %p", fn, need, workspace_bytes, workspace);
  if (d->num_blocks == 0 || d->num_seqs > 65535 || d->num_kv_heads > 65535)
    return fail(PA_ERR_INVALID_ARG, "%s: bad pool or batch size", fn);
  if (static_cast<int64_t>(d->num_blocks) * d->num_kv_heads * d->block_size >
      0x7fffffffLL)
    return fail(PA_ERR_UNSUPPORTED, "%s: pool exceeds 2^31 rows", fn);
  return PA_OK;
}

// The map lists tiles of `tok` tokens (at least tile_tokens(d), whose map the
// workspace holds).
pa_status launch_plan(const char* fn, const pa_prefill_desc* d,
                      const int32_t* context_lens, const int32_t* query_start,
                      int max_ctx, int tok, void* workspace,
                      int32_t* dev_err, cudaStream_t s) {
  int2* tiles = tile_map(d, workspace);
  int* counter = work_counter(d, workspace);
  cudaLaunchConfig_t pcfg = {};
  pcfg.gridDim = dim3(1);
  pcfg.blockDim = dim3(kOrderThreads);
  pcfg.stream = s;
  cudaLaunchAttribute pattr[1];
  pattr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pattr[0].val.programmaticStreamSerializationAllowed = 1;
  pcfg.attrs = pattr;
  pcfg.numAttrs = 1;
  cudaError_t oe = cudaLaunchKernelEx(
      &pcfg, prefill_plan_kernel, context_lens, query_start,
      d->num_seqs, d->total_q, d->max_q_len, order_shift(max_ctx),
      tok, static_cast<int>(tile_cap(d, tok)),
      static_cast<int32_t*>(workspace), tiles, counter, dev_err);
  count_launch();
  if (oe == cudaSuccess) oe = cudaGetLastError();
  if (oe != cudaSuccess)
    return fail(PA_ERR_CUDA, "%s: plan launch failed: %s", fn,
                cudaGetErrorString(oe));
  return PA_OK;
}

}  // namespace
}  // namespace pagedkv
