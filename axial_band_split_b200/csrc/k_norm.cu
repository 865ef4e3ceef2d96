// Root-mean-square norm of rows with the residual's addition and an optional e4m3 output with
// scales (mrf_rms_norm): h = x + residual, y = h * weight * s, s from the row's mean square.
//
// Bound by memory: x and residual are read once and h and y written once; a row stays in registers
// between its sums and its output.  s is common to a row, so max |y| = s max |h * weight|: the
// row's sum of squares and the maxima that the 8-bit scales need come from the same pass over the
// registers, and one exchange between the warps serves both.
//
// Rows up to 512 wide take a warp each (no exchange between warps), wider ones a block; a thread
// holds V vectors of 8 values.  What hides a row's load latency is the other rows on the SM, so the
// register budget is 64 a thread (1024 threads an SM).
#include <cuda_fp8.h>

#include <algorithm>

#include "block_ops.h"

namespace mrf {
namespace {

constexpr int kMaxWarps = 16;

__device__ __forceinline__ float max_nan(float a, float b) {  // keeps a NaN
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float warp_max(float v, int width) {
  for (int o = width / 2; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// 8 values of a row as they lie in memory.
template <class T>
struct Raw {
  T v[8];
};

// Columns of value e of this lane's vector, whose warp's 256 columns begin at c0.  kVec: 8 neighbours
// (16-byte accesses); else 32 apart, so that a warp's accesses of one value are neighbours.
template <bool kVec>
__device__ __forceinline__ int column(int c0, int lane, int e) {
  return kVec ? c0 + 8 * lane + e : c0 + 32 * e + lane;
}

template <class T, bool kVec>
__device__ __forceinline__ void load8(const T *row, int c0, int lane, int dim, Raw<T> &r) {
  if constexpr (kVec) {
    const int c = c0 + 8 * lane;
    if (c < dim) {
      const uint4 *p = reinterpret_cast<const uint4 *>(row + c);
      uint4 *q = reinterpret_cast<uint4 *>(r.v);
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) q[i] = p[i];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (column<false>(c0, lane, e) < dim) r.v[e] = row[column<false>(c0, lane, e)];
  }
}

template <class T, bool kVec>
__device__ __forceinline__ void store8(T *row, int c0, int lane, int dim, const float (&f)[8]) {
  if constexpr (kVec) {
    const int c = c0 + 8 * lane;
    if (c < dim) {
      Raw<T> r;
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e] = from_f32<T>(f[e]);
      uint4 *p = reinterpret_cast<uint4 *>(row + c);
      const uint4 *q = reinterpret_cast<const uint4 *>(r.v);
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) p[i] = q[i];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (column<false>(c0, lane, e) < dim) row[column<false>(c0, lane, e)] = from_f32<T>(f[e]);
  }
}

// The weight's 8 values at this lane's columns.
template <bool kVec>
__device__ __forceinline__ void load_weight(const mrf_rms_norm_args &a, bool wide, int c0, int lane, float (&w)[8]) {
  if (!a.weight) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
  } else if (kVec && wide) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.weight) + c0 + 8 * lane);
    const bool in = c0 + 8 * lane < a.dim;
    const float4 u = in ? __ldg(p) : make_float4(0.f, 0.f, 0.f, 0.f), v = in ? __ldg(p + 1) : u;
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<kVec>(c0, lane, e);
      w[e] = c < a.dim ? load_any(a.weight, a.weight_dtype, c) : 0.f;
    }
  }
}

// kWarpRow: a warp a row; else a block a row.  wide: the weight is fp32 and 16-byte aligned.
template <class T, int V, bool kWarpRow, bool kVec>
__global__ void __launch_bounds__(32 * kMaxWarps, V <= 2 ? 2 : 1) rms_norm_kernel(const mrf_rms_norm_args a, const bool wide) {
  __shared__ float red[2][2][kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
  const bool quant = a.out_dtype == MRF_DTYPE_E4M3, row_scale = quant && a.group == 0;
  const int groups = a.group ? (a.dim + a.group - 1) / a.group : 1;
  const long long step = kWarpRow ? gridDim.x * (long long)warps : gridDim.x;
  int buf = 0;
  for (long long r = kWarpRow ? blockIdx.x * (long long)warps + warp : blockIdx.x; r < a.rows; r += step, buf ^= 1) {
    float h[V][8], ss = 0.f, top = 0.f;
    Raw<T> xr[V], rr[V];
    auto first_column = [&](int v) { return 256 * (kWarpRow ? v : v * warps + warp); };
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) xr[v].v[e] = rr[v].v[e] = from_f32<T>(0.f);
      load8<T, kVec>(x + r * a.x_stride, first_column(v), lane, a.dim, xr[v]);
      if (res) load8<T, kVec>(res + r * a.residual_stride, first_column(v), lane, a.dim, rr[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[v][e] = to_f32(xr[v].v[e]) + to_f32(rr[v].v[e]);
        ss = fmaf(h[v][e], h[v][e], ss);
      }
      if (a.residual_out)
        store8<T, kVec>(static_cast<T *>(a.residual_out) + r * a.residual_out_stride, first_column(v), lane, a.dim, h[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float w[8];
      load_weight<kVec>(a, wide, first_column(v), lane, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] *= w[e];
    }
    // the row's sum of squares and, for one scale a row, its largest |h w|
    if (row_scale) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(h[v][e]));
      top = warp_max(top, 32);
    }
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if constexpr (!kWarpRow) {
      if (lane == 0) {
        red[buf][0][warp] = ss;
        red[buf][1][warp] = top;
      }
      __syncthreads();  // (the other buffer is read before the next one's barrier)
      ss = 0.f;
      for (int i = 0; i < warps; ++i) ss += red[buf][0][i];
      if (row_scale)
        for (int i = 0; i < warps; ++i) top = max_nan(top, red[buf][1][i]);
    }
    const float mean = ss / (float)a.dim;
    const float s = a.clamp ? 1.f / fmaxf(sqrtf(mean), a.eps) : 1.f / sqrtf(mean + a.eps);
    if (!quant) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] *= s;
        store8<T, kVec>(static_cast<T *>(a.out) + r * a.out_stride, first_column(v), lane, a.dim, h[v]);
      }
      continue;
    }
    // scale = s max |h w| / 448 over the group, code = h w * (448 / max |h w|): s drops out of the codes.
    // A scale of 0 gives codes 0, a NaN one NaN.
    if (row_scale && lane == 0 && (kWarpRow || warp == 0)) a.scales[r] = s * top * (1.f / 448.f);
    auto factor = [&](float m) {
      const float scaled = s * m;
      return scaled == 0.f ? 0.f : scaled != scaled ? scaled : 448.f / m;
    };
    uint8_t *o = static_cast<uint8_t *>(a.out) + r * a.out_stride;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c0 = first_column(v);
      if (c0 >= a.dim) break;
      float q[8];
      if (kVec || row_scale) {
        float m = top;
        if (!row_scale) {  // group / 8 neighbouring lanes
          m = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(h[v][e]));
          m = warp_max(m, a.group / 8);
          const int c = c0 + 8 * lane;
          if (c < a.dim && (lane & (a.group / 8 - 1)) == 0) a.scales[r * groups + c / a.group] = s * m * (1.f / 448.f);
        }
        if (m < 1e-30f) {  // 448 / m would pass fp32
          m *= 0x1p90f;
#pragma unroll
          for (int e = 0; e < 8; ++e) h[v][e] *= 0x1p90f;
        }
        const float f = factor(m);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = h[v][e] * f;
      } else {  // group / 32 values of every lane
        const int n = a.group / 32;
        float gm[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float m = warp_max(fabsf(h[v][e]), 32);
          gm[e] = e % n ? max_nan(gm[e ? e - 1 : 0], m) : m;
        }
#pragma unroll
        for (int e = 6; e >= 0; --e)
          if ((e + 1) % n) gm[e] = gm[e + 1];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (lane == 0 && e % n == 0 && c0 + 32 * e < a.dim)
            a.scales[r * groups + (c0 + 32 * e) / a.group] = s * gm[e] * (1.f / 448.f);
          const float up = gm[e] < 1e-30f ? 0x1p90f : 1.f;
          q[e] = h[v][e] * up * factor(gm[e] * up);
        }
      }
      if constexpr (kVec) {
        const int c = c0 + 8 * lane;
        if (c < a.dim) {
          unsigned short b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) b[e] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * e], q[2 * e + 1]), __NV_SATFINITE, __NV_E4M3);
          *reinterpret_cast<uint2 *>(o + c) = make_uint2(b[0] | (unsigned)b[1] << 16, b[2] | (unsigned)b[3] << 16);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (column<false>(c0, lane, e) < a.dim) o[column<false>(c0, lane, e)] = __nv_cvt_float_to_fp8(q[e], __NV_SATFINITE, __NV_E4M3);
      }
    }
  }
}

bool vec_ok(const void *p, long long rows, long long stride, int size) {
  // 8 values: 16-byte accesses, 8 bytes for e4m3
  const int n = size == 1 ? 8 : 16 / size;
  return reinterpret_cast<uintptr_t>(p) % (n * size) == 0 && (rows <= 1 || stride % n == 0);
}

template <class T, bool kVec>
void launch(const mrf_rms_norm_args &a, cudaStream_t st) {
  const bool wide = a.weight_dtype == MRF_DTYPE_F32 && reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
  const int chunks = (a.dim + 255) / 256;  // of 256 columns: a vector of each lane of a warp
  if (chunks <= 2) {
    const int warps = a.rows >= 148 * 16 ? 8 : 1;  // few rows: an SM each
    const int grid = (int)std::min<long long>((a.rows + warps - 1) / warps, 148 * 32 / warps);
    if (chunks == 1) rms_norm_kernel<T, 1, true, kVec><<<grid, 32 * warps, 0, st>>>(a, wide);
    else rms_norm_kernel<T, 2, true, kVec><<<grid, 32 * warps, 0, st>>>(a, wide);
    return;
  }
  const int vecs = chunks <= 2 * kMaxWarps ? 2 : 4, warps = (chunks + vecs - 1) / vecs;
  const int grid = (int)std::min<long long>(a.rows, 148 * std::max(1, (vecs == 2 ? 32 : 16) / warps));
  if (vecs == 2) rms_norm_kernel<T, 2, false, kVec><<<grid, 32 * warps, 0, st>>>(a, wide);
  else rms_norm_kernel<T, 4, false, kVec><<<grid, 32 * warps, 0, st>>>(a, wide);
}

}  // namespace

cudaError_t launch_rms_norm(const mrf_rms_norm_args &a, cudaStream_t st) {
  const int size = a.dtype == MRF_DTYPE_F32 ? 4 : 2;
  const bool vec = a.dim % 8 == 0 && vec_ok(a.x, a.rows, a.x_stride, size) &&
                   (!a.residual || vec_ok(a.residual, a.rows, a.residual_stride, size)) &&
                   (!a.residual_out || vec_ok(a.residual_out, a.rows, a.residual_out_stride, size)) &&
                   vec_ok(a.out, a.rows, a.out_stride, a.out_dtype == MRF_DTYPE_E4M3 ? 1 : size);
#define MRF_NORM(T) (vec ? launch<T, true>(a, st) : launch<T, false>(a, st))
  if (a.dtype == MRF_DTYPE_F32) MRF_NORM(float);
  else if (a.dtype == MRF_DTYPE_F16) MRF_NORM(__half);
  else MRF_NORM(__nv_bfloat16);
#undef MRF_NORM
  return cudaGetLastError();
}

}  // namespace mrf
