// Rotary positions on the heads of q and k (mrf_rope).
//
// Bound by memory: every value is read and written once.  A block takes a few tokens: it first
// computes their cos and sin into shared memory (part / 2 pairs a token, whatever the number of
// heads), then walks over (token, head, unit) with a unit of 8 pairs or 8 untouched values, in
// 16-byte accesses; where widths, strides or addresses do not allow those a unit is one pair or value.
// 16384 tokens of 40 heads of 128 in bf16 (336 MB): 60 us, 5.6 TB/s, 0.85 of the measured copy (a pair a
// thread with its own cos and sin: 288 us; a token a block: 75 us).
#include <algorithm>

#include "block_ops.h"

namespace mrf {
namespace {

constexpr int kThreads = 256, kMaxPairs = 512;  // pairs of the table in shared memory

// cos and sin of `phase`, a 64-bit binary fraction of a turn.  Its upper 32 bits, read as signed, are
// half turns of [-1, 1) scaled by 2^31, so no argument reduction is left to do and a position of
// millions keeps the same accuracy (2^-24 of a half turn) as a small one.
__device__ __forceinline__ float2 turn(unsigned long long phase, float scale) {
  float sn, cs;
  sincospif((float)(int)(phase >> 32) * 4.656612873077393e-10f, &sn, &cs);
  return make_float2(cs * scale, sn * scale);
}

struct Shape {
  int rot;     // units of one head that turn, of 8 pairs (or one)
  int units;   // and all its units
  int tokens;  // of one block
};

template <class T>
struct Raw {
  T v[8];
};
template <class T>
__device__ __forceinline__ void load8(const T *p, Raw<T> &r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(r.v)[i] = reinterpret_cast<const uint4 *>(p)[i];
}
template <class T>
__device__ __forceinline__ void store8(T *p, const Raw<T> &r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(r.v)[i];
}

template <class T, bool kVec>
__global__ void __launch_bounds__(kThreads) rope_kernel(const mrf_rope_args a, const Shape s) {
  __shared__ float2 table[kMaxPairs];
  const int half = a.part / 2, all_heads = a.heads + a.kv_heads;
  const long long tok0 = blockIdx.x * (long long)s.tokens;
  const int tokens = (int)min((long long)s.tokens, a.tokens - tok0);
  for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
    const long long tok = tok0 + i / half;
    const long long pos = a.positions_wide ? static_cast<const long long *>(a.positions)[tok]
                                           : static_cast<const int *>(a.positions)[tok];
    table[i] = turn((unsigned long long)pos * a.turns[i % half], a.scale);
  }
  __syncthreads();
  const unsigned n = (unsigned)(tokens * all_heads) * s.units;
#pragma unroll 2
  for (unsigned i = threadIdx.x; i < n; i += kThreads) {
    const unsigned th = i / s.units, u = i - th * s.units;
    const unsigned t = th / all_heads;
    int h = (int)(th - t * all_heads);
    const long long tok = tok0 + t;
    const bool isk = h >= a.heads;
    if (isk) h -= a.heads;
    const T *x = static_cast<const T *>(isk ? a.k : a.q) +
                 (isk ? tok * a.k_token_stride + h * a.k_head_stride : tok * a.q_token_stride + h * a.q_head_stride);
    T *y = static_cast<T *>(isk ? a.k_out : a.q_out) + (isk ? tok * a.k_out_token_stride + h * a.k_out_head_stride
                                                             : tok * a.q_out_token_stride + h * a.q_out_head_stride);
    if constexpr (kVec) {
      if (u < (unsigned)s.rot) {
        const int i0 = a.interleaved ? 16 * u : 8 * u, i1 = a.interleaved ? i0 + 8 : i0 + half;
        Raw<T> p, q;
        load8(x + i0, p);
        load8(x + i1, q);
        const float2 *cs = table + t * half + 8 * u;
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 c = cs[e], d = cs[e + 4];
            const float p0 = to_f32(p.v[2 * e]), p1 = to_f32(p.v[2 * e + 1]), q0 = to_f32(q.v[2 * e]), q1 = to_f32(q.v[2 * e + 1]);
            p.v[2 * e] = from_f32<T>(p0 * c.x - p1 * c.y);
            p.v[2 * e + 1] = from_f32<T>(p1 * c.x + p0 * c.y);
            q.v[2 * e] = from_f32<T>(q0 * d.x - q1 * d.y);
            q.v[2 * e + 1] = from_f32<T>(q1 * d.x + q0 * d.y);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 c = cs[e];
            const float a0 = to_f32(p.v[e]), b0 = to_f32(q.v[e]);
            p.v[e] = from_f32<T>(a0 * c.x - b0 * c.y);
            q.v[e] = from_f32<T>(b0 * c.x + a0 * c.y);
          }
        }
        store8(y + i0, p);
        store8(y + i1, q);
      } else {
        const int i0 = a.part + 8 * (u - s.rot);
        Raw<T> p;
        load8(x + i0, p);
        store8(y + i0, p);
      }
    } else if (u < (unsigned)half) {
      const int i0 = a.interleaved ? 2 * u : u, i1 = a.interleaved ? i0 + 1 : i0 + half;
      const float2 c = table[t * half + u];
      const float a0 = to_f32(x[i0]), b0 = to_f32(x[i1]);
      y[i0] = from_f32<T>(a0 * c.x - b0 * c.y);
      y[i1] = from_f32<T>(b0 * c.x + a0 * c.y);
    } else {
      y[u + half] = x[u + half];
    }
  }
}

bool vec_ok(const void *p, long long n1, long long s1, long long n2, long long s2, int size) {
  const int n = 16 / size;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (n1 <= 1 || s1 % n == 0) && (n2 <= 1 || s2 % n == 0);
}

template <class T>
void launch(const mrf_rope_args &a, bool vec, bool in_place, cudaStream_t st) {
  Shape s;
  s.rot = vec ? a.part / 16 : a.part / 2;
  // dimensions that do not turn are copied, unless they are where they should be
  s.units = s.rot + (in_place ? 0 : vec ? (a.width - a.part) / 8 : a.width - a.part);
  // about 1024 units a block, as long as there are blocks enough for every SM
  const long long per = (long long)(a.heads + a.kv_heads) * s.units;
  long long t = std::max(1ll, std::min<long long>({1024 / per, a.tokens / (148 * 4), kMaxPairs / (a.part / 2)}));
  s.tokens = (int)t;
  const int grid = (int)((a.tokens + t - 1) / t);
  if (vec) rope_kernel<T, true><<<grid, kThreads, 0, st>>>(a, s);
  else rope_kernel<T, false><<<grid, kThreads, 0, st>>>(a, s);
}

}  // namespace

cudaError_t launch_rope(const mrf_rope_args &a, cudaStream_t st) {
  const int size = a.dtype == MRF_DTYPE_F32 ? 4 : 2;
  const bool vec = a.part % 16 == 0 && a.width % 8 == 0 &&
                   vec_ok(a.q, a.tokens, a.q_token_stride, a.heads, a.q_head_stride, size) &&
                   vec_ok(a.q_out, a.tokens, a.q_out_token_stride, a.heads, a.q_out_head_stride, size) &&
                   (a.kv_heads == 0 || (vec_ok(a.k, a.tokens, a.k_token_stride, a.kv_heads, a.k_head_stride, size) &&
                                        vec_ok(a.k_out, a.tokens, a.k_out_token_stride, a.kv_heads, a.k_out_head_stride, size)));
  const bool in_place = a.q_out == a.q && (a.kv_heads == 0 || a.k_out == a.k);
  if (a.dtype == MRF_DTYPE_F32) launch<float>(a, vec, in_place, st);
  else if (a.dtype == MRF_DTYPE_F16) launch<__half>(a, vec, in_place, st);
  else launch<__nv_bfloat16>(a, vec, in_place, st);
  return cudaGetLastError();
}

}  // namespace mrf
