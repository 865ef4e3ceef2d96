// Root-mean-square norm of rows with the residual's addition and an optional e4m3 output with
// scales (mrf_rms_norm).
#include <cuda_fp8.h>

#include <algorithm>
#include <climits>

#include "block_ops.h"

namespace mrf {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v, float *red) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < kThreads / 32; ++i) s += red[i];
  __syncthreads();
  return s;
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <class T>
__global__ void __launch_bounds__(kThreads) rms_norm_kernel(const mrf_rms_norm_args a) {
  extern __shared__ float row[];
  __shared__ float red[kThreads / 32];
  const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float ss = 0.f;
    for (int j = threadIdx.x; j < a.dim; j += kThreads) {
      float h = to_f32(x[r * a.x_stride + j]);
      if (res) h += to_f32(res[r * a.residual_stride + j]);
      if (a.residual_out) static_cast<T *>(a.residual_out)[r * a.residual_out_stride + j] = from_f32<T>(h);
      row[j] = h;
      ss = fmaf(h, h, ss);
    }
    const float mean = block_sum(ss, red) / (float)a.dim;
    const float s = a.clamp ? 1.f / fmaxf(sqrtf(mean), a.eps) : 1.f / sqrtf(mean + a.eps);
    for (int j = threadIdx.x; j < a.dim; j += kThreads) {
      row[j] *= s;
      if (a.weight) row[j] *= load_any(a.weight, a.weight_dtype, j);
    }
    __syncthreads();
    if (a.out_dtype != MRF_DTYPE_E4M3) {
      for (int j = threadIdx.x; j < a.dim; j += kThreads)
        static_cast<T *>(a.out)[r * a.out_stride + j] = from_f32<T>(row[j]);
    } else {
      const int group = a.group ? a.group : a.dim, groups = (a.dim + group - 1) / group;
      for (int g = threadIdx.x >> 5; g < groups; g += kThreads / 32) {
        const int j1 = min(a.dim, (g + 1) * group);
        float m = 0.f;
        for (int j = g * group + (threadIdx.x & 31); j < j1; j += 32) m = max_nan(m, fabsf(row[j]));
        for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float scale = m / 448.f;
        if ((threadIdx.x & 31) == 0) a.scales[r * groups + g] = scale;
        for (int j = g * group + (threadIdx.x & 31); j < j1; j += 32)
          static_cast<__nv_fp8_e4m3 *>(a.out)[r * a.out_stride + j] = __nv_fp8_e4m3(scale == 0.f ? 0.f : row[j] / scale);
      }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_rms_norm(const mrf_rms_norm_args &a, cudaStream_t st) {
  const int grid = (int)std::min<long long>(a.rows, INT_MAX);
  const size_t smem = (size_t)a.dim * sizeof(float);
#define MRF_NORM(T)                                                                                               \
  do {                                                                                                            \
    cudaError_t e = cudaFuncSetAttribute(rms_norm_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 65536); \
    if (e != cudaSuccess) return e;                                                                               \
    rms_norm_kernel<T><<<grid, kThreads, smem, st>>>(a);                                                          \
  } while (0)
  if (a.dtype == MRF_DTYPE_F32) MRF_NORM(float);
  else if (a.dtype == MRF_DTYPE_F16) MRF_NORM(__half);
  else MRF_NORM(__nv_bfloat16);
#undef MRF_NORM
  return cudaGetLastError();
}

}  // namespace mrf
