// Rotary positions on the heads of q and k (mrf_rope).
#include <algorithm>
#include <climits>

#include "block_ops.h"

namespace mrf {
namespace {

// cos and sin of `phase`, a 64-bit binary fraction of a turn.  Its upper 32 bits, read as signed, are
// half turns of [-1, 1) scaled by 2^31, so no argument reduction is left to do and a position of
// millions keeps the same accuracy (2^-24 of a half turn) as a small one.
__device__ __forceinline__ void turn(unsigned long long phase, float *sn, float *cs) {
  sincospif((float)(int)(phase >> 32) * 4.656612873077393e-10f, sn, cs);
}

template <class T>
__global__ void rope_kernel(const mrf_rope_args a) {
  const int half = a.part / 2, rest = a.width - a.part, items = half + rest;
  const long long n = a.tokens * (a.heads + a.kv_heads) * (long long)items;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const int e = (int)(i % items);
    const long long th = i / items, tok = th / (a.heads + a.kv_heads);
    int h = (int)(th % (a.heads + a.kv_heads));
    const bool isk = h >= a.heads;
    if (isk) h -= a.heads;
    const T *x = static_cast<const T *>(isk ? a.k : a.q) +
                 (isk ? tok * a.k_token_stride + h * a.k_head_stride : tok * a.q_token_stride + h * a.q_head_stride);
    T *y = static_cast<T *>(isk ? a.k_out : a.q_out) + (isk ? tok * a.k_out_token_stride + h * a.k_out_head_stride
                                                             : tok * a.q_out_token_stride + h * a.q_out_head_stride);
    if (e >= half) {
      y[a.part + e - half] = x[a.part + e - half];
      continue;
    }
    const long long pos = a.positions_wide ? static_cast<const long long *>(a.positions)[tok]
                                           : static_cast<const int *>(a.positions)[tok];
    float sn, cs;
    turn((unsigned long long)pos * a.turns[e], &sn, &cs);
    sn *= a.scale;
    cs *= a.scale;
    const int i0 = a.interleaved ? 2 * e : e, i1 = a.interleaved ? 2 * e + 1 : e + half;
    const float u = to_f32(x[i0]), v = to_f32(x[i1]);
    y[i0] = from_f32<T>(u * cs - v * sn);
    y[i1] = from_f32<T>(v * cs + u * sn);
  }
}

}  // namespace

cudaError_t launch_rope(const mrf_rope_args &a, cudaStream_t st) {
  const long long n = a.tokens * (a.heads + a.kv_heads) * (long long)(a.width - a.part / 2);
  const int grid = (int)std::min<long long>((n + 255) / 256, 148 * 32);
  if (a.dtype == MRF_DTYPE_F32) rope_kernel<float><<<grid, 256, 0, st>>>(a);
  else if (a.dtype == MRF_DTYPE_F16) rope_kernel<__half><<<grid, 256, 0, st>>>(a);
  else rope_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace mrf
