// Internal declarations of the block operators (mrf_rms_norm, mrf_rope, mrf_attention).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/mrf.h"

namespace mrf {

// The text mrf_last_error(NULL) gives on this thread (mrf_api.cu).
void set_thread_error(const char *msg) noexcept;

// One value of a tensor of type T as fp32, and back (rounded to nearest even).
template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// One value of a dtype known at run time.
__device__ __forceinline__ float load_any(const void *p, int dtype, long long i) {
  if (dtype == MRF_DTYPE_F32) return static_cast<const float *>(p)[i];
  if (dtype == MRF_DTYPE_F16) return __half2float(static_cast<const __half *>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

// The current device's SMs, asked once a device (k_attn_packed_tc.cu).
int sm_count();

// Each queues its kernels on st; the arguments have been checked (op_api.cu).
cudaError_t launch_rms_norm(const mrf_rms_norm_args &a, cudaStream_t st);
cudaError_t launch_rope(const mrf_rope_args &a, cudaStream_t st);
// How the keys of few tiles are split: the keys of a range (0: no splits) and the most ranges a sequence can
// have.  A tile has `tokens` tokens for one of `sets` sets of heads and takes `block` us for 128 keys.
struct AttentionSplit {
  int chunk, most;
};
AttentionSplit attention_split(const mrf_attention_args &a, int tokens, long long sets, double block);
// CUDA-core attention (k_attn_rows.cu): any type, width and stride; the workspace it needs.
size_t attention_rows_workspace(const mrf_attention_args &a);
cudaError_t launch_attention_rows(const mrf_attention_args &a, cudaStream_t st);
// Tensor-core attention (k_attn_packed_tc.cu): whether it takes these arguments, the workspace it
// needs for them, and its launches (false: a tensor map was refused and nothing was queued).
bool attention_tc_takes(const mrf_attention_args &a);
size_t attention_tc_workspace(const mrf_attention_args &a);
bool launch_attention_packed_tc(const mrf_attention_args &a, cudaStream_t st, cudaError_t *err);
// Its status word (0, or 1 and the site of a wait that expired) after the work queued on st; cleared.
cudaError_t attention_tc_status(unsigned *word, cudaStream_t st);

}  // namespace mrf
