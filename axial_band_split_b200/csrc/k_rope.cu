// Rotary positions on the heads of q and k (mrf_rope).
//
// Bound by memory: every value is read and written once.  A block takes a few tokens: it first
// computes their cos and sin into shared memory (part / 2 pairs a token, whatever the number of
// heads), then walks over (token, head, unit) with a unit of N pairs or 2 N untouched values.  N is the
// most of 8, 4, 2 and 1 whose pieces divide half the turned part and fit strides and addresses: 40 heads of 80
// with 40 turned take 54 us with N = 4, 185 with 1; of 96 with 24 turned 59 and 224; of 80 with 20 turned 88 (N = 2)
// and 200.
// 16384 tokens of 40 heads of 128 in bf16 (336 MB): 60 us, 5.6 TB/s, 0.85 of the measured copy (a pair a
// thread with its own cos and sin: 288 us; a token a block: 75 us).
#include <algorithm>
#include <type_traits>

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
  int rot;     // units of one head that turn, of N pairs
  int units;   // and all its units; the others copy 2 N values
  int tokens;  // of one block
};

// N neighbouring values, in accesses of up to 16 bytes.
template <class T, int N>
struct Piece {
  static constexpr int kBytes = N * (int)sizeof(T) < 16 ? N * (int)sizeof(T) : 16;
  using Word = std::conditional_t<kBytes == 16, uint4, std::conditional_t<kBytes == 8, uint2, std::conditional_t<kBytes == 4, uint32_t, uint16_t>>>;
  alignas(16) T v[N];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < N * (int)sizeof(T) / kBytes; ++i) reinterpret_cast<Word *>(v)[i] = reinterpret_cast<const Word *>(p)[i];
  }
  __device__ __forceinline__ void store(T *p) const {
#pragma unroll
    for (int i = 0; i < N * (int)sizeof(T) / kBytes; ++i) reinterpret_cast<Word *>(p)[i] = reinterpret_cast<const Word *>(v)[i];
  }
};
template <class T>
__device__ __forceinline__ void turn_pair(T &a, T &b, float2 c) {
  const float a0 = to_f32(a), b0 = to_f32(b);
  a = from_f32<T>(a0 * c.x - b0 * c.y);
  b = from_f32<T>(b0 * c.x + a0 * c.y);
}

template <class T, int N>
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
    Piece<T, N> p, q;
    if (u < (unsigned)s.rot) {
      const int i0 = a.interleaved ? 2 * N * u : N * u, i1 = a.interleaved ? i0 + N : i0 + half;
      p.load(x + i0);
      q.load(x + i1);
      const float2 *cs = table + t * half + N * u;
      if (a.interleaved && N > 1) {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          turn_pair(p.v[2 * e], p.v[(2 * e + 1) % N], cs[e]);
          turn_pair(q.v[2 * e], q.v[(2 * e + 1) % N], cs[e + N / 2]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) turn_pair(p.v[e], q.v[e], cs[e]);
      }
      p.store(y + i0);
      q.store(y + i1);
    } else {
      const int i0 = a.part + 2 * N * (u - s.rot), i1 = i0 + N;
      p.load(x + i0);
      if (i1 < a.width) q.load(x + i1);
      p.store(y + i0);
      if (i1 < a.width) q.store(y + i1);
    }
  }
}

// A [n1, n2, .] tensor takes pieces of n values.
bool takes(const void *p, long long n1, long long s1, long long n2, long long s2, int size, int n) {
  const int bytes = std::min(16, n * size);
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (n1 <= 1 || s1 * size % bytes == 0) && (n2 <= 1 || s2 * size % bytes == 0);
}

template <class T, int N>
void launch(const mrf_rope_args &a, cudaStream_t st) {
  Shape s;
  s.rot = a.part / 2 / N;
  // dimensions that do not turn are copied, unless they are where they should be
  const bool in_place = a.q_out == a.q && (a.kv_heads == 0 || a.k_out == a.k);
  s.units = s.rot + (in_place ? 0 : (a.width - a.part + 2 * N - 1) / (2 * N));
  // about 1024 units a block, as long as there are blocks enough for every SM
  const long long per = (long long)(a.heads + a.kv_heads) * s.units;
  long long t = std::max(1ll, std::min<long long>({1024 / per, a.tokens / (4 * sm_count()), kMaxPairs / (a.part / 2)}));
  s.tokens = (int)t;
  rope_kernel<T, N><<<(int)((a.tokens + t - 1) / t), kThreads, 0, st>>>(a, s);
}
template <class T>
void launch(const mrf_rope_args &a, cudaStream_t st) {
  constexpr int size = sizeof(T);
  auto fits = [&](int n) {
    return a.part / 2 % n == 0 && a.width % n == 0 && takes(a.q, a.tokens, a.q_token_stride, a.heads, a.q_head_stride, size, n) &&
           takes(a.q_out, a.tokens, a.q_out_token_stride, a.heads, a.q_out_head_stride, size, n) &&
           (a.kv_heads == 0 || (takes(a.k, a.tokens, a.k_token_stride, a.kv_heads, a.k_head_stride, size, n) &&
                                takes(a.k_out, a.tokens, a.k_out_token_stride, a.kv_heads, a.k_out_head_stride, size, n)));
  };
  if (fits(8)) launch<T, 8>(a, st);
  else if (fits(4)) launch<T, 4>(a, st);
  else if (fits(2)) launch<T, 2>(a, st);
  else launch<T, 1>(a, st);
}

}  // namespace

cudaError_t launch_rope(const mrf_rope_args &a, cudaStream_t st) {
  if (a.dtype == MRF_DTYPE_F32) launch<float>(a, st);
  else if (a.dtype == MRF_DTYPE_F16) launch<__half>(a, st);
  else launch<__nv_bfloat16>(a, st);
  return cudaGetLastError();
}

}  // namespace mrf
