// Root-mean-square norm of rows with the residual's addition and an optional e4m3 output with
// scales (mrf_rms_norm): h = x + residual, y = h * weight * s, s from the row's mean square.
//
// Bound by memory: x and residual are read once and h and y written once; a row stays in registers
// between its sums and its output.  s is common to a row, so max |y| = s max |h * weight|: the
// row's sum of squares and the maxima that the 8-bit scales need come from the same pass over the
// registers, and one exchange between the warps serves both.
//
// Rows in 16-byte pieces: up to 256 columns, and up to 512 while every row finds a warp at once, take a warp each (no
// exchange between warps), few rows of up to 2048 columns and all above 8192 a block each in the same
// rms_norm_kernel; the others stream through rms_norm_stream_kernel.  Rows without that alignment go through
// rms_norm_odd_kernel, many of up to 2048 columns with a warp each, else with a block.  launch() has the borders and
// what both sides measured.  The arithmetic, about 10 instructions a value with the conversions, is the next bound:
// it runs on packed fp32 pairs, and the work that a row costs every thread (the sums' exchange, the root, the scales)
// is spread over its 16 values.
// 16384 x 4096 bf16 with residual and an e4m3 output (472 MB): 87.5 us, 5.4 TB/s, 0.82 of the measured copy
// (a first form with 64-bit index products and a division a value executed 40 instructions a value: 113 us).
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "block_ops.h"

namespace mrf {
namespace {

__device__ __forceinline__ float max_nan(float a, float b) {  // keeps a NaN
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float warp_max(float v, int width) {
  for (int o = width / 2; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Two 16-bit values as fp32, and back.
template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
  return __half22float2(*reinterpret_cast<__half2 *>(&u));
}
template <class T>
__device__ __forceinline__ uint32_t pack2(float2 f);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float2 f) {
  const __nv_bfloat162 h = __float22bfloat162_rn(f);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float2 f) {
  const __half2 h = __float22half2_rn(f);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// 8 neighbouring values of a row as they lie in memory.
template <class T>
struct Raw {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T *p, bool in) {  // zeros past the row's end
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = in ? reinterpret_cast<const uint4 *>(p)[i] : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float2 pair(int i) const {
    const uint4 u = v[sizeof(T) == 4 ? i / 2 : 0];
    if constexpr (sizeof(T) == 4)
      return i & 1 ? make_float2(__uint_as_float(u.z), __uint_as_float(u.w)) : make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    else
      return unpack2<T>(i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w);
  }
};

template <class T>
__device__ __forceinline__ void store8(T *p, const float2 (&f)[4]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  } else {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack2<T>(f[0]), pack2<T>(f[1]), pack2<T>(f[2]), pack2<T>(f[3]));
  }
}
__device__ __forceinline__ void store8_e4m3(void *p, const float2 (&f)[4]) {
  unsigned b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __nv_cvt_float2_to_fp8x2(f[i], __NV_SATFINITE, __NV_E4M3);
  *static_cast<uint2 *>(p) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
}

// f *= the weight at columns c .. c + 7 (inside the row).  wide: the weight is fp32 and 16-byte aligned.
__device__ __forceinline__ void times_weight(const mrf_rms_norm_args &a, bool wide, int c, float2 (&f)[4]) {
  if (!a.weight) return;
  if (wide) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.weight) + c);
    const float4 u = __ldg(p), v = __ldg(p + 1);
    f[0] = __fmul2_rn(f[0], make_float2(u.x, u.y));
    f[1] = __fmul2_rn(f[1], make_float2(u.z, u.w));
    f[2] = __fmul2_rn(f[2], make_float2(v.x, v.y));
    f[3] = __fmul2_rn(f[3], make_float2(v.z, v.w));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = __fmul2_rn(f[i], make_float2(load_any(a.weight, a.weight_dtype, c + 2 * i), load_any(a.weight, a.weight_dtype, c + 2 * i + 1)));
  }
}

__device__ __forceinline__ float max8(float m, const float2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_nan(max_nan(m, fabsf(f[i].x)), fabsf(f[i].y));
  return m;
}

// Asynchronous copies of a thread's own vectors into its own places in shared memory: nobody else
// reads them, so the thread's own wait is all the ordering they need.
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 load_shared(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct Plan {
  bool wide;        // the weight is fp32 and 16-byte aligned
  float inv_dim, inv_eps;
  int log2_group;   // of a.group
};

// s of a row with this sum of squares.  clamp: 1 / max(sqrt(mean), eps) = min(1 / sqrt(mean), 1 / eps); a NaN stays.
__device__ __forceinline__ float row_factor(const mrf_rms_norm_args &a, const Plan &plan, float ss) {
  const float mean = ss * plan.inv_dim;
  const float s = rsqrtf(a.clamp ? mean : mean + a.eps);
  return a.clamp && s > plan.inv_eps ? plan.inv_eps : s;
}

// An 8-bit group whose largest |h w| is m: scale = s m / 448 and code = h w * (448 / m); s drops out of the codes.
struct Code {
  float up, f;  // code = (h w * up) * f
};
__device__ __forceinline__ float code_scale(float s, float m) { return s * m * (1.f / 448.f); }
__device__ __forceinline__ Code code_factor(float s, float m) {
  const float scaled = s * m;
  if (scaled > 0.f && m > 1e-30f && m < 1e30f) {
    // The quotient within 2 units in the last place and one step of Newton's method, q + (448 - q m) / m with 1 / m = q / 448:
    // codes on or near a tie round as those of the exact quotient.
    const float q = __fdividef(448.f, m);
    return {1.f, fmaf(fmaf(-q, m, 448.f), q * (1.f / 448.f), q)};
  }
  // a scale of 0 gives codes 0, a NaN one NaN; where the quotient would leave fp32's range h w moves first
  if (scaled == 0.f || scaled != scaled) return {1.f, scaled};
  const float up = m < 1.f ? 0x1p90f : 0x1p-30f;
  return {up, 448.f / (m * up)};
}
__device__ __forceinline__ void to_codes(float2 (&h)[4], Code c) {
  if (c.up != 1.f)
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __fmul2_rn(h[i], make_float2(c.up, c.up));
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __fmul2_rn(h[i], make_float2(c.f, c.f));
}

// Rows in 16-byte pieces held in registers, V vectors of 8 a thread.  kWarpRow: a warp a row; else a block a row.
template <class T, int V, bool kWarpRow>
__global__ void __launch_bounds__(512, V <= 2 ? 2 : 1) rms_norm_kernel(const mrf_rms_norm_args a, const Plan plan) {
  __shared__ float red[2][2][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
  const bool quant = a.out_dtype == MRF_DTYPE_E4M3, row_scale = quant && a.group == 0;
  const int groups = a.group ? (a.dim + a.group - 1) / a.group : 1;
  const long long step = kWarpRow ? gridDim.x * (long long)warps : gridDim.x;
  int buf = 0;
  for (long long r = kWarpRow ? blockIdx.x * (long long)warps + warp : blockIdx.x; r < a.rows; r += step, buf ^= 1) {
    auto column = [&](int v) { return 256 * (kWarpRow ? v : v * warps + warp) + 8 * lane; };
    float2 h[V][4];
    {
      Raw<T> xr[V], rr[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        xr[v].load(x + r * a.x_stride + column(v), column(v) < a.dim);
        if (res) rr[v].load(res + r * a.residual_stride + column(v), column(v) < a.dim);
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) h[v][i] = res ? __fadd2_rn(xr[v].pair(i), rr[v].pair(i)) : xr[v].pair(i);
    }
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s2 = __ffma2_rn(h[v][i], h[v][i], s2);
      if (column(v) < a.dim) {
        if (a.residual_out) store8<T>(static_cast<T *>(a.residual_out) + r * a.residual_out_stride + column(v), h[v]);
        times_weight(a, plan.wide, column(v), h[v]);
      }
    }
    // the row's sum of squares and, for one scale a row, its largest |h w|
    float ss = s2.x + s2.y, top = 0.f;
    if (row_scale) {
#pragma unroll
      for (int v = 0; v < V; ++v) top = max8(top, h[v]);
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
    const float s = row_factor(a, plan, ss);
    if (row_scale && lane == 0 && (kWarpRow || warp == 0)) a.scales[r] = code_scale(s, top);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = column(v);
      if (c - 8 * lane >= a.dim) break;
      if (!quant) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[v][i] = __fmul2_rn(h[v][i], make_float2(s, s));
        if (c < a.dim) store8<T>(static_cast<T *>(a.out) + r * a.out_stride + c, h[v]);
      } else {
        float m = top;
        if (!row_scale) {  // group / 8 neighbouring lanes
          m = warp_max(max8(0.f, h[v]), a.group / 8);
          if (c < a.dim && (lane & (a.group / 8 - 1)) == 0) a.scales[r * groups + (c >> plan.log2_group)] = code_scale(s, m);
        }
        to_codes(h[v], code_factor(s, m));
        if (c < a.dim) store8_e4m3(static_cast<uint8_t *>(a.out) + r * a.out_stride + c, h[v]);
      }
    }
  }
}

// The codes of values j, j + step ... below n, two at a time.
__device__ __forceinline__ void codes_of(const float *row, uint8_t *o, int j, int n, int step, Code c) {
  for (; j < n; j += 2 * step) {
    const bool two = j + step < n;
    float2 v = make_float2(row[j], two ? row[j + step] : 0.f);
    if (c.up != 1.f) v = __fmul2_rn(v, make_float2(c.up, c.up));
    const unsigned b = __nv_cvt_float2_to_fp8x2(__fmul2_rn(v, make_float2(c.f, c.f)), __NV_SATFINITE, __NV_E4M3);
    o[j] = (uint8_t)b;
    if (two) o[j + step] = (uint8_t)(b >> 8);
  }
}

// Rows whose width, stride or address allows no 16-byte pieces: h w in fp32 in shared memory, value by value in
// coalesced order; a team of a warp (kWarpRow) or a block for each row.
// 16000 x 4097 with a residual and one scale per 128 values 195 us, 20000 x 1003 49 us, 20000 x 131 13 us: 2.4, 2.9 and
// 1.4 TB/s, bound by the instructions that single values take.
constexpr int kBatch = 8;  // loads of x and the residual each in flight (4: 16000 x 4097 30% slower; 16: twice as slow, spills)
template <class T, bool kWarpRow>
__global__ void __launch_bounds__(256, 4) rms_norm_odd_kernel(const mrf_rms_norm_args a, const Plan plan) {
  extern __shared__ float odd_rows[];
  __shared__ float red[2][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int me = kWarpRow ? lane : threadIdx.x, team = kWarpRow ? 32 : blockDim.x;
  float *row = odd_rows + (kWarpRow ? warp * a.dim : 0);
  const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
  const bool quant = a.out_dtype == MRF_DTYPE_E4M3;
  auto team_sync = [&]() {
    if constexpr (kWarpRow) __syncwarp();
    else __syncthreads();
  };
  // over the team's threads
  auto reduce = [&](float v, bool sum) {
    for (int o = 16; o; o >>= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, v, o);
      v = sum ? v + u : max_nan(v, u);
    }
    if constexpr (!kWarpRow) {
      __syncthreads();
      if (lane == 0) red[sum][warp] = v;
      __syncthreads();
      v = red[sum][0];
      for (int i = 1; i < warps; ++i) v = sum ? v + red[sum][i] : max_nan(v, red[sum][i]);
    }
    return v;
  };
  const long long step = kWarpRow ? gridDim.x * (long long)warps : gridDim.x;
  for (long long r = kWarpRow ? blockIdx.x * (long long)warps + warp : blockIdx.x; r < a.rows; r += step) {
    float ss = 0.f, top = 0.f;
    const T *xr = x + r * a.x_stride, *rr = res ? res + r * a.residual_stride : nullptr;
    T *ho = a.residual_out ? static_cast<T *>(a.residual_out) + r * a.residual_out_stride : nullptr;
    // values j0, j0 + team ...; kFull: all of a batch lie in the row
    auto batch = [&](int j0, auto full) {
      constexpr bool kFull = decltype(full)::value;
      T v[kBatch], u[kBatch];
      float h[kBatch];
      auto in = [&](int i) { return kFull || j0 + i * team < a.dim; };
#pragma unroll
      for (int i = 0; i < kBatch; ++i) v[i] = in(i) ? xr[j0 + i * team] : from_f32<T>(0.f);
      if (rr) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) u[i] = in(i) ? rr[j0 + i * team] : from_f32<T>(0.f);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) h[i] = to_f32(v[i]) + to_f32(u[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) h[i] = to_f32(v[i]);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) ss = fmaf(h[i], h[i], ss);
      if (ho) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (in(i)) ho[j0 + i * team] = from_f32<T>(h[i]);
      }
      auto weigh = [&](auto *w) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (in(i)) h[i] *= to_f32(w[j0 + i * team]);
      };
      if (!a.weight) {
      } else if (a.weight_dtype == MRF_DTYPE_F32) weigh(static_cast<const float *>(a.weight));
      else if (a.weight_dtype == MRF_DTYPE_F16) weigh(static_cast<const __half *>(a.weight));
      else weigh(static_cast<const __nv_bfloat16 *>(a.weight));
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (in(i)) {
          top = max_nan(top, fabsf(h[i]));
          row[j0 + i * team] = h[i];
        }
    };
    int j0 = me;
    for (; j0 + (kBatch - 1) * team < a.dim; j0 += kBatch * team) batch(j0, std::true_type());
    if (j0 < a.dim) batch(j0, std::false_type());
    const float s = row_factor(a, plan, reduce(ss, true));
    if (!quant) {
      T *o = static_cast<T *>(a.out) + r * a.out_stride;
#pragma unroll 4
      for (int j = me; j < a.dim; j += team) o[j] = from_f32<T>(row[j] * s);
    } else {
      uint8_t *o = static_cast<uint8_t *>(a.out) + r * a.out_stride;
      if (a.group == 0) {
        top = reduce(top, false);
        if (me == 0) a.scales[r] = code_scale(s, top);
        const Code c = code_factor(s, top);
        codes_of(row, o, me, a.dim, team, c);
      } else {
        team_sync();  // a group's values are other threads'
        const int groups = (a.dim + a.group - 1) / a.group;
        for (int g = kWarpRow ? 0 : warp; g < groups; g += kWarpRow ? 1 : warps) {
          const int j0 = g * a.group, j1 = min(a.dim, j0 + a.group);
          float m = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i)  // (a group is 128 at most)
            if (j0 + 32 * i + lane < j1) m = max_nan(m, fabsf(row[j0 + 32 * i + lane]));
          m = warp_max(m, 32);
          if (lane == 0) a.scales[r * groups + g] = code_scale(s, m);
          codes_of(row, o, j0 + lane, j1, 32, code_factor(s, m));
        }
      }
    }
    team_sync();  // before the next row's values
  }
}

// Rows of 257 to 8192 columns in 16-byte pieces, but for those that launch() finds faster elsewhere: a block a row,
// two vectors a thread.  The loads of kAhead rows are in flight at any time (asynchronous copies into shared memory,
// 48 KB a block at 4096 columns of 16 bits), the weight stays in registers, and addresses advance by additions.
// kMode: 0 the output is T, 1 e4m3 with a scale a row, 2 with a scale a group.
constexpr int kAhead = 3;

template <class T, int kMode, bool kRes>
__global__ void __launch_bounds__(512, 2) rms_norm_stream_kernel(const mrf_rms_norm_args a, const Plan plan) {
  constexpr int P = (int)sizeof(T) / 2;                  // 16-byte pieces of a vector
  constexpr int kPieces = 2 * P * (kRes ? 2 : 1);        // of a thread's share of a row
  extern __shared__ uint4 ring[];
  __shared__ float red[2][2][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int c0 = 256 * warp + 8 * lane, c1 = c0 + 256 * warps;
  const bool in0 = c0 < a.dim, in1 = c1 < a.dim;
  const long long first = blockIdx.x, step = gridDim.x;
  const T *x = static_cast<const T *>(a.x) + first * a.x_stride + c0;
  const T *res = kRes ? static_cast<const T *>(a.residual) + first * a.residual_stride + c0 : nullptr;
  T *res_out = kRes && a.residual_out ? static_cast<T *>(a.residual_out) + first * a.residual_out_stride + c0 : nullptr;
  const int out_size = kMode == 0 ? (int)sizeof(T) : 1;
  char *out = static_cast<char *>(a.out) + (first * a.out_stride + c0) * out_size;
  const int far = c1 - c0;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16, pstep = blockDim.x * 16;

  int todo = (int)((a.rows - first + step - 1) / step), ahead = todo;  // rows to work on, rows to load
  auto copy_row = [&](uint32_t at) {
    if (ahead > 0) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (in0) copy_async(at + i * pstep, reinterpret_cast<const uint4 *>(x) + i);
        if (in1) copy_async(at + (P + i) * pstep, reinterpret_cast<const uint4 *>(x + far) + i);
        if constexpr (kRes) {
          if (in0) copy_async(at + (2 * P + i) * pstep, reinterpret_cast<const uint4 *>(res) + i);
          if (in1) copy_async(at + (3 * P + i) * pstep, reinterpret_cast<const uint4 *>(res + far) + i);
        }
      }
      --ahead;
      x += step * a.x_stride;
      if constexpr (kRes) res += step * a.residual_stride;
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) copy_row(mine + i * kPieces * pstep);
  // zeros past the row's end, once
  for (int i = 0; i < kAhead * kPieces; ++i)
    if (!(i / P % 2 ? in1 : in0)) asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(mine + i * pstep), "r"(0));
  float2 w[2][4];
#pragma unroll
  for (int v = 0; v < 2; ++v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[v][i] = make_float2(1.f, 1.f);
    if (v ? in1 : in0) times_weight(a, plan.wide, v ? c1 : c0, w[v]);
  }
  const int groups = kMode == 2 ? (a.dim + a.group - 1) / a.group : 1;
  float *scales = kMode == 0 ? nullptr : a.scales + first * groups;
  uint32_t at = mine;
  const uint32_t end = mine + kAhead * kPieces * pstep;
  for (int buf = 0; todo > 0; --todo, buf ^= 1) {
    copy_wait<kAhead - 1>();
    float2 h[2][4], s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      Raw<T> xr, rr;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        xr.v[i] = load_shared(at + (v * P + i) * pstep);
        if constexpr (kRes) rr.v[i] = load_shared(at + ((2 + v) * P + i) * pstep);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[v][i] = kRes ? __fadd2_rn(xr.pair(i), rr.pair(i)) : xr.pair(i);
        s2 = __ffma2_rn(h[v][i], h[v][i], s2);
      }
    }
    if constexpr (kRes)
      if (res_out) {
        if (in0) store8<T>(res_out, h[0]);
        if (in1) store8<T>(res_out + far, h[1]);
        res_out += step * a.residual_out_stride;
      }
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) h[v][i] = __fmul2_rn(h[v][i], w[v][i]);
    float ss = s2.x + s2.y, top = 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if constexpr (kMode == 1) {
      top = max8(max8(0.f, h[0]), h[1]);
#pragma unroll
      for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (lane == 0) {
      red[buf][0][warp] = ss;
      if constexpr (kMode == 1) red[buf][1][warp] = top;
    }
    __syncthreads();  // (the other buffer is read before the next one's barrier)
    copy_row(at);     // into the place just read
    at += kPieces * pstep;
    if (at == end) at = mine;
    ss = (lane & 15) < warps ? red[buf][0][lane & 15] : 0.f;
#pragma unroll
    for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if constexpr (kMode == 1) {
      top = (lane & 15) < warps ? red[buf][1][lane & 15] : 0.f;
#pragma unroll
      for (int o = 8; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    const float s = row_factor(a, plan, ss);
    if constexpr (kMode == 0) {
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) h[v][i] = __fmul2_rn(h[v][i], make_float2(s, s));
      T *o = reinterpret_cast<T *>(out);
      if (in0) store8<T>(o, h[0]);
      if (in1) store8<T>(o + far, h[1]);
    } else {
      if (kMode == 1 && threadIdx.x == 0) scales[0] = code_scale(s, top);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        float m = top;
        const bool in = v ? in1 : in0;
        if constexpr (kMode == 2) {  // group / 8 neighbouring lanes
          m = max8(0.f, h[v]);
          m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
          if (plan.log2_group > 5) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 4));
          if (plan.log2_group > 6) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 8));
          const int c = v ? c1 : c0;
          if (in && (c & (a.group - 1)) == 0) scales[c >> plan.log2_group] = code_scale(s, m);
        }
        to_codes(h[v], code_factor(s, m));
        if (in) store8_e4m3(out + (v ? far : 0), h[v]);
      }
      scales += step * groups;
    }
    out += step * a.out_stride * out_size;
  }
  copy_wait<0>();
}

// Lets kernel K's launches have up to 200 KB of shared memory, once a device (asking takes longer than a launch's checks).
template <auto *K>
cudaError_t allow_smem() {
  static std::atomic<unsigned long long> ready{0};  // devices that were asked
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && ready.load(std::memory_order_relaxed) >> dev & 1)) return e;
  e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e == cudaSuccess && dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

template <class T, int kMode, bool kRes>
cudaError_t launch_stream(const mrf_rms_norm_args &a, const Plan &p, cudaStream_t st) {
  auto *k = rms_norm_stream_kernel<T, kMode, kRes>;
  const int warps = ((a.dim + 255) / 256 + 1) / 2;
  const int smem = kAhead * (kRes ? 2 : 1) * 2 * (int)sizeof(T) / 2 * 16 * 32 * warps;
  if (const cudaError_t e = allow_smem<rms_norm_stream_kernel<T, kMode, kRes>>()) return e;
  const int blocks = std::max(1, std::min(32 / warps, 220 * 1024 / (smem + 1280)));  // on an SM, at 64 registers a thread
  k<<<(int)std::min<long long>(a.rows, sm_count() * blocks), 32 * warps, smem, st>>>(a, p);
  return cudaGetLastError();
}

bool vec_ok(const void *p, long long rows, long long stride, int size) {
  // 8 values: 16-byte accesses, 8 bytes for e4m3
  const int n = size == 1 ? 8 : 16 / size;
  return reinterpret_cast<uintptr_t>(p) % (n * size) == 0 && (rows <= 1 || stride % n == 0);
}

template <class T>
cudaError_t launch(const mrf_rms_norm_args &a, bool vec, cudaStream_t st) {
  Plan p;
  p.wide = a.weight_dtype == MRF_DTYPE_F32 && reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
  p.inv_dim = 1.f / (float)a.dim;
  p.inv_eps = std::min(1.f / a.eps, 3.4e38f);  // finite: a row of zeros stays zeros
  p.log2_group = a.group == 32 ? 5 : a.group == 64 ? 6 : 7;
  const int chunks = (a.dim + 255) / 256;  // of 256 columns: a vector of each lane of a warp
  const int sms = sm_count();
  const bool few = a.rows < sms * 4;       // rows that do not fill the SMs
  if (!vec) {
    // a warp a row up to 2048 columns where there are rows for every warp (20000 x 2001: 101 us against 153 with a block a row,
    // x 131: 13 and 52; but 16000 x 4097: 286 and 195, and 300 x 131: 4.0 and 2.9)
    if (chunks <= 8 && !few) {
      const int warps = 4, smem = warps * a.dim * (int)sizeof(float);
      if (const cudaError_t e = allow_smem<rms_norm_odd_kernel<T, true>>()) return e;
      rms_norm_odd_kernel<T, true><<<(int)std::min<long long>((a.rows + warps - 1) / warps, sms * 64), 32 * warps, smem, st>>>(a, p);
    } else {
      const int smem = a.dim * (int)sizeof(float);
      if (const cudaError_t e = allow_smem<rms_norm_odd_kernel<T, false>>()) return e;
      rms_norm_odd_kernel<T, false><<<(int)std::min<long long>(a.rows, sms * 64), 256, smem, st>>>(a, p);
    }
  } else if (chunks == 1) {  // a warp a row (40000 x 64: 10.7 us against 14.5 with blocks; x 256: 15.5 and 15.3)
    const int warps = few ? 1 : 8;
    const int grid = (int)std::min<long long>((a.rows + warps - 1) / warps, sms * 64 / warps);
    rms_norm_kernel<T, 1, true><<<grid, 32 * warps, 0, st>>>(a, p);
  } else if (chunks == 2 && !few && a.rows <= sms * 64) {
    // a warp a row while every row finds a warp at once (4201 x 384: 3.4 us against 4.9 streamed, x 512: 3.8 and
    // 5.0; 9472 x 384: 5.5 and 6.2; 40000 x 384: 24 and 20, so not there; 4201 x 1024: 6.3 and 5.5, nor there)
    rms_norm_kernel<T, 2, true><<<(int)((a.rows + 7) / 8), 256, 0, st>>>(a, p);
  } else if (few && chunks <= 8) {
    // more threads a row and shorter chains, up to 2048 columns (1 x 1024: 2.3 us against 2.6; 592 rows: 3.0 and
    // 3.15; 1 x 8192: 4.4 against 3.6, so not there)
    rms_norm_kernel<T, 1, false><<<(int)a.rows, 32 * chunks, 0, st>>>(a, p);
  } else if (chunks <= 32) {
    const int mode = a.out_dtype != MRF_DTYPE_E4M3 ? 0 : a.group == 0 ? 1 : 2;
    if (a.residual) return mode == 0 ? launch_stream<T, 0, true>(a, p, st) : mode == 1 ? launch_stream<T, 1, true>(a, p, st) : launch_stream<T, 2, true>(a, p, st);
    return mode == 0 ? launch_stream<T, 0, false>(a, p, st) : mode == 1 ? launch_stream<T, 1, false>(a, p, st) : launch_stream<T, 2, false>(a, p, st);
  } else {
    rms_norm_kernel<T, 5, false><<<(int)std::min<long long>(a.rows, sms), 32 * ((chunks + 4) / 5), 0, st>>>(a, p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_norm(const mrf_rms_norm_args &a, cudaStream_t st) {
  const int size = a.dtype == MRF_DTYPE_F32 ? 4 : 2;
  const bool vec = a.dim % 8 == 0 && vec_ok(a.x, a.rows, a.x_stride, size) &&
                   (!a.residual || vec_ok(a.residual, a.rows, a.residual_stride, size)) &&
                   (!a.residual_out || vec_ok(a.residual_out, a.rows, a.residual_out_stride, size)) &&
                   vec_ok(a.out, a.rows, a.out_stride, a.out_dtype == MRF_DTYPE_E4M3 ? 1 : size);
  if (a.dtype == MRF_DTYPE_F32) return launch<float>(a, vec, st);
  if (a.dtype == MRF_DTYPE_F16) return launch<__half>(a, vec, st);
  return launch<__nv_bfloat16>(a, vec, st);
}

}  // namespace mrf
