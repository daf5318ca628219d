// pa_copy_blocks_q8 and pa_swap_blocks_q8: whole blocks of the 8-bit cache,
// their codes and their scales, within one pool (copy-on-write) or between
// two pools either of which may sit in page-locked host memory.
//
// A byte move: a CTA moves one block's K or V (num_kv_heads x block_size x
// head_dim bytes, contiguous) in 16-byte loads, kInFlight of them per thread
// before their stores, and the block's num_kv_heads scales.  Bound by HBM (or
// the host link); ids are checked on the device, a bad pair records
// PA_ERR_DEVICE_OOB and is skipped.
#include <cuda_runtime.h>

#include <cstdint>

#include "device_utils.cuh"
#include "pagedkv.h"
#include "status.h"

namespace pagedkv {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;

struct PoolQ8 {
  uint4 *k, *v;
  float *ks, *vs;
};

// No __restrict__: copy-on-write moves within one pool.
__global__ void __launch_bounds__(kThreads)
    move_blocks_q8_kernel(const PoolQ8 dst, const PoolQ8 src,
                          const int32_t* __restrict__ pairs,
                          int64_t block_chunks, int num_kv_heads, int num_src,
                          int num_dst, int32_t* dev_err) {
  dev::pdl_wait();
  // A following attention may run its prologue now.  Not before the wait: it
  // reads lengths, which a kernel before this one may still be writing.
  dev::pdl_trigger();
  const int32_t s = pairs[2 * blockIdx.x];
  const int32_t d = pairs[2 * blockIdx.x + 1];
  if (s < 0 || s >= num_src || d < 0 || d >= num_dst) {
    if (threadIdx.x == 0 && blockIdx.y == 0)
      dev::set_error(dev_err, PA_ERR_DEVICE_OOB);
    return;
  }
  const bool is_v = blockIdx.y;
  const uint4* from = (is_v ? src.v : src.k) + s * block_chunks;
  uint4* to = (is_v ? dst.v : dst.k) + d * block_chunks;
  const float* from_s =
      (is_v ? src.vs : src.ks) + static_cast<int64_t>(s) * num_kv_heads;
  float* to_s =
      (is_v ? dst.vs : dst.ks) + static_cast<int64_t>(d) * num_kv_heads;
  for (int i = threadIdx.x; i < num_kv_heads; i += kThreads)
    to_s[i] = from_s[i];
  for (int64_t i0 = threadIdx.x; i0 < block_chunks;
       i0 += static_cast<int64_t>(kThreads) * kInFlight) {
    uint4 v[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int64_t i = i0 + u * kThreads;
      if (i < block_chunks) v[u] = from[i];
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int64_t i = i0 + u * kThreads;
      if (i < block_chunks) to[i] = v[u];
    }
  }
}

pa_status move(const char* fn, const PoolQ8& dst, const PoolQ8& src,
               const int32_t* pairs, int num_pairs, int num_kv_heads,
               int head_dim, int block_size, int num_src, int num_dst,
               int32_t* dev_err, void* stream) {
  const int64_t block_chunks =
      static_cast<int64_t>(num_kv_heads) * block_size * head_dim / 16;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_pairs, 2);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e =
      cudaLaunchKernelEx(&cfg, move_blocks_q8_kernel, dst, src, pairs,
                         block_chunks, num_kv_heads, num_src, num_dst,
                         dev_err);
  count_launch();
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(PA_ERR_CUDA, "%s: launch failed: %s", fn,
                cudaGetErrorString(e));
  return PA_OK;
}

pa_status check_shape(const char* fn, int num_pairs, int num_kv_heads,
                      int head_dim, int block_size, int num_src,
                      int num_dst) {
  if (num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_src < 0 ||
      num_dst < 0 || num_pairs < 0)
    return fail(PA_ERR_INVALID_ARG,
                "%s: num_kv_heads=%d head_dim=%d block_size=%d "
                "num_src_blocks=%d num_dst_blocks=%d num_pairs=%d", fn,
                num_kv_heads, head_dim, block_size, num_src, num_dst,
                num_pairs);
  if (head_dim % 16)
    return fail(PA_ERR_UNSUPPORTED,
                "%s: head_dim %d is not a multiple of 16", fn, head_dim);
  return PA_OK;
}

}  // namespace
}  // namespace pagedkv

using pagedkv::fail;

extern "C" {

pa_status pa_copy_blocks_q8(void* k_cache, void* v_cache, float* k_scales,
                            float* v_scales, const int32_t* pairs,
                            int num_pairs, int num_kv_heads, int head_dim,
                            int block_size, int num_blocks, int32_t* dev_err,
                            void* stream) {
  pagedkv::clear_error();
  const pa_status st =
      pagedkv::check_shape("pa_copy_blocks_q8", num_pairs, num_kv_heads,
                           head_dim, block_size, num_blocks, num_blocks);
  if (st != PA_OK) return st;
  if (num_pairs == 0) return PA_OK;
  if (!k_cache || !v_cache || !k_scales || !v_scales || !pairs)
    return fail(PA_ERR_INVALID_ARG, "pa_copy_blocks_q8: NULL pointer");
  if (!pagedkv::aligned16(k_cache) || !pagedkv::aligned16(v_cache))
    return fail(PA_ERR_INVALID_ARG,
                "pa_copy_blocks_q8: caches must be 16-byte aligned");
  const pagedkv::PoolQ8 pool{
      static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), k_scales,
      v_scales};
  return pagedkv::move("pa_copy_blocks_q8", pool, pool, pairs, num_pairs,
                       num_kv_heads, head_dim, block_size, num_blocks,
                       num_blocks, dev_err, stream);
}

pa_status pa_swap_blocks_q8(void* dst_k_cache, void* dst_v_cache,
                            float* dst_k_scales, float* dst_v_scales,
                            const void* src_k_cache, const void* src_v_cache,
                            const float* src_k_scales,
                            const float* src_v_scales, const int32_t* pairs,
                            int num_pairs, int num_kv_heads, int head_dim,
                            int block_size, int num_src_blocks,
                            int num_dst_blocks, int32_t* dev_err,
                            void* stream) {
  pagedkv::clear_error();
  const pa_status st = pagedkv::check_shape(
      "pa_swap_blocks_q8", num_pairs, num_kv_heads, head_dim, block_size,
      num_src_blocks, num_dst_blocks);
  if (st != PA_OK) return st;
  if (num_pairs == 0) return PA_OK;
  const void* ptrs[9] = {dst_k_cache, dst_v_cache, src_k_cache, src_v_cache,
                         dst_k_scales, dst_v_scales, src_k_scales,
                         src_v_scales, pairs};
  const char* names[9] = {"dst_k_cache", "dst_v_cache", "src_k_cache",
                          "src_v_cache", "dst_k_scales", "dst_v_scales",
                          "src_k_scales", "src_v_scales", "pairs"};
  void* view[9];
  for (int i = 0; i < 9; ++i) {
    if (!ptrs[i])
      return fail(PA_ERR_INVALID_ARG, "pa_swap_blocks_q8: %s is NULL",
                  names[i]);
    view[i] = pagedkv::device_view(ptrs[i]);
    if (!view[i])
      return fail(PA_ERR_INVALID_ARG,
                  "pa_swap_blocks_q8: %s is neither memory of the current "
                  "device nor mapped page-locked host memory", names[i]);
    if (i < 4 && !pagedkv::aligned16(view[i]))
      return fail(PA_ERR_INVALID_ARG,
                  "pa_swap_blocks_q8: %s must be 16-byte aligned", names[i]);
  }
  int32_t* err_view = nullptr;
  if (dev_err) {
    err_view = static_cast<int32_t*>(pagedkv::device_view(dev_err));
    if (!err_view)
      return fail(PA_ERR_INVALID_ARG,
                  "pa_swap_blocks_q8: dev_err is not reachable from the "
                  "device");
  }
  const pagedkv::PoolQ8 dst{
      static_cast<uint4*>(view[0]), static_cast<uint4*>(view[1]),
      static_cast<float*>(view[4]), static_cast<float*>(view[5])};
  const pagedkv::PoolQ8 src{
      static_cast<uint4*>(view[2]), static_cast<uint4*>(view[3]),
      static_cast<float*>(view[6]), static_cast<float*>(view[7])};
  return pagedkv::move("pa_swap_blocks_q8", dst, src,
                       static_cast<const int32_t*>(view[8]), num_pairs,
                       num_kv_heads, head_dim, block_size, num_src_blocks,
                       num_dst_blocks, err_view, stream);
}

}  // extern "C"
