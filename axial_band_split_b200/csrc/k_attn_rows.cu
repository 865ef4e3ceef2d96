// Packed attention on the CUDA cores (mrf_attention): one warp per (query row, head), 32 keys at a
// time, one key a lane, online softmax.  It takes any type, width and stride; the tensor-core
// kernel takes the shapes that matrix instructions and bulk tensor loads can.
#include <algorithm>
#include <climits>

#include "block_ops.h"

namespace mrf {
namespace {

constexpr int kWarps = 4, kMaxWidth = 256;

// The sequence whose query rows hold `tok`, or -1.
__device__ __forceinline__ int find_seq(const int32_t *off, int seqs, long long tok) {
  int lo = 0, hi = seqs;  // the last b with off[b] <= tok
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= tok) lo = mid;
    else hi = mid;
  }
  return off[lo] <= tok && tok < off[lo + 1] ? lo : -1;
}

template <class T>
__global__ void __launch_bounds__(32 * kWarps) attention_rows_kernel(const mrf_attention_args a) {
  __shared__ float qs[kWarps][kMaxWidth];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long n = a.q_rows * a.heads;
  float *q = qs[warp];
  for (long long i = (long long)blockIdx.x * kWarps + warp; i < n; i += (long long)gridDim.x * kWarps) {
    const long long tok = i / a.heads;
    const int h = (int)(i % a.heads), hk = h / (a.heads / a.kv_heads);
    const int b = find_seq(a.q_offsets, a.seqs, tok);
    if (b < 0) continue;
    const long long q0 = a.q_offsets[b] < 0 ? 0 : a.q_offsets[b];
    const long long nq = min((long long)a.q_offsets[b + 1], (long long)a.q_rows) - q0;
    const long long k0 = min(max(a.k_len ? (long long)a.k_start[b] : q0, 0ll), (long long)a.k_rows);
    const long long nk = min(max(a.k_len ? (long long)a.k_len[b] : nq, 0ll), a.k_rows - k0);
    const long long seen = a.causal ? min(nk, max(0ll, tok - q0 + 1 + nk - nq)) : nk;
    const T *qp = static_cast<const T *>(a.q) + tok * a.q_token_stride + h * a.q_head_stride;
    const T *kp = static_cast<const T *>(a.k) + k0 * a.k_token_stride + hk * a.k_head_stride;
    const T *vp = static_cast<const T *>(a.v) + k0 * a.v_token_stride + hk * a.v_head_stride;
    __syncwarp();
    for (int d = lane; d < a.width; d += 32) q[d] = to_f32(qp[d]);
    __syncwarp();
    float o[kMaxWidth / 32];
#pragma unroll
    for (int u = 0; u < kMaxWidth / 32; ++u) o[u] = 0.f;
    float m = -INFINITY, l = 0.f;
    for (long long j = 0; j < seen; j += 32) {
      const long long key = j + lane;
      float s = -INFINITY;
      if (key < seen) {
        const T *kr = kp + key * a.k_token_stride;
        s = 0.f;
        for (int d = 0; d < a.width; ++d) s = fmaf(q[d], to_f32(kr[d]), s);
        s *= a.scale;
      }
      float bm = s;
      for (int w = 16; w; w >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, w));
      const float m1 = fmaxf(m, bm), m0 = m1 == -INFINITY ? 0.f : m1;
      const float alpha = expf(m - m0), p = key < seen ? expf(s - m0) : 0.f;
      float ps = p;
      for (int w = 16; w; w >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, w);
      l = l * alpha + ps;
      m = m1;
#pragma unroll
      for (int u = 0; u < kMaxWidth / 32; ++u) o[u] *= alpha;
      const int cnt = (int)min(32ll, seen - j);
      for (int w = 0; w < cnt; ++w) {
        const float pw = __shfl_sync(0xffffffffu, p, w);
        const T *vr = vp + (j + w) * a.v_token_stride;
#pragma unroll
        for (int u = 0; u < kMaxWidth / 32; ++u)
          if (lane + 32 * u < a.v_width) o[u] = fmaf(pw, to_f32(vr[lane + 32 * u]), o[u]);
      }
    }
    const float inv = seen > 0 ? 1.f / l : 0.f;
    T *op = static_cast<T *>(a.out) + tok * a.out_token_stride + h * a.out_head_stride;
#pragma unroll
    for (int u = 0; u < kMaxWidth / 32; ++u)
      if (lane + 32 * u < a.v_width) op[lane + 32 * u] = from_f32<T>(seen > 0 ? o[u] * inv : 0.f);
    if (a.lse && lane == 0) a.lse[tok * a.heads + h] = seen > 0 ? m + logf(l) : -INFINITY;
  }
}

}  // namespace

cudaError_t launch_attention_rows(const mrf_attention_args &a, cudaStream_t st) {
  const long long n = a.q_rows * a.heads;
  const int grid = (int)std::min<long long>((n + kWarps - 1) / kWarps, 148 * 64);
  if (a.dtype == MRF_DTYPE_F32) attention_rows_kernel<float><<<grid, 32 * kWarps, 0, st>>>(a);
  else if (a.dtype == MRF_DTYPE_F16) attention_rows_kernel<__half><<<grid, 32 * kWarps, 0, st>>>(a);
  else attention_rows_kernel<__nv_bfloat16><<<grid, 32 * kWarps, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace mrf
