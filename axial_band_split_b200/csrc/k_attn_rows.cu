// Packed attention on the CUDA cores (mrf_attention): fp32, widths up to 256, any width, stride and number of
// heads; the tensor-core kernel takes the shapes that matrix instructions and bulk tensor loads can.
//
// A block of 256 threads (tx, ty) = 16 x 16 has a tile of 16 RI rows, row = token * G + head like the tensor-core
// kernel's, so that heads that share a key head share its loads, and goes over its keys 64 at a time with a running
// maximum and sum.  A thread has rows ty + 16 i and of the scores keys tx + 16 j, of the output columns
// 4 tx + 64 n: a row's maxima and sums are exchanged within half a warp, and its probabilities pass through shared
// memory within its warp.  Both products read 16 bytes at a time along the summed or the output dimension; with
// RI = 8 that is 16 wavefronts of shared memory for 128 multiply-adds a thread, so the multiply-adds (128 a clk and
// SM) bound it; with RI = 1 (new tokens) the loads of keys do.  fp32 keys and values come by asynchronous copies,
// values under the scores, the next keys under the second product.  Few tiles with long keys are split into ranges
// of keys, joined by rows_join_kernel.
//
// Measured in fp32: 8 x 1100 tokens both ways, 8 heads, 64 wide 0.67 ms (30 TFLOP/s), 128 wide 1.14 ms (35, nearly half
// of the multiply-adds' peak; shared memory bounds the rest); a token of each of 32 sequences of 500 to 2000 keys, 32
// heads of 128 over 8 0.28 ms (1.2 TB/s).  (A warp a row with a key a lane: 20.5 ms and 2.7 ms.)
#include <algorithm>
#include <atomic>

#include "block_ops.h"

namespace mrf {
namespace {

constexpr int kKeys = 64;         // keys of a step
constexpr int kPad = kKeys + 4;   // stride of a row of probabilities

struct Tiles {
  int G1, parts, TQ;  // heads of a tile, tiles that a group of heads needs, tokens of a tile
  int ld;             // stride of q and k rows in shared memory: 4 x an odd number, so that rows hit different banks
  int chunk, most;    // keys of a range (0: no splits), ranges that the workspace holds
  int vec;            // fp32 keys and values in 16-byte pieces
  long long units;
  float *part, *part_lse;  // [range][row][head][v_width] and their log-sums
};

__device__ __forceinline__ void copy16(float *dst, const float *src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(float *dst, const float *src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src), "r"(in ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// `live` rows of kKeys (zeros after them), `width` columns padded with zeros to a multiple of 4.
template <class T>
__device__ __forceinline__ void load_keys(float *dst, int ld, const T *src, long long stride, int live, int width, int vec) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  if constexpr (sizeof(T) == 4) {
    if (vec) {
      for (int d = 4 * tx; d < width; d += 64)
#pragma unroll
        for (int r = ty; r < kKeys; r += 16) copy16(dst + r * ld + d, r < live ? src + r * stride + d : src, r < live);
    } else {
      for (int d = tx; d < (width + 3) / 4 * 4; d += 16)
#pragma unroll
        for (int r = ty; r < kKeys; r += 16) {
          const bool in = r < live && d < width;
          copy4(dst + r * ld + d, in ? src + r * stride + d : src, in);
        }
    }
  } else {
    for (int d0 = tx; d0 < (width + 3) / 4 * 4; d0 += 64) {  // 16 loads in flight
      T v[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int r = ty + 16 * i, d = d0 + 16 * n;
          v[i][n] = r < live && d < width ? src[r * stride + d] : from_f32<T>(0.f);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if (d0 + 16 * n < (width + 3) / 4 * 4) dst[(ty + 16 * i) * ld + d0 + 16 * n] = to_f32(v[i][n]);
    }
  }
}

// Half a warp's threads.
__device__ __forceinline__ float max16(float v) {
  for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float sum16(float v) {
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Span {
  long long q0, nq, k0, nk;
};
// Sequence b's rows, held to the tensors' whatever the offsets say.
__device__ __forceinline__ long long clamped(long long v, long long hi) { return min(max(v, 0ll), hi); }
__device__ __forceinline__ Span load_span(const mrf_attention_args &a, int b) {
  Span s;
  s.q0 = clamped(a.q_offsets[b], a.q_rows);
  s.nq = max(0ll, clamped(a.q_offsets[b + 1], a.q_rows) - s.q0);
  s.k0 = a.k_len ? clamped(a.k_start[b], a.k_rows) : s.q0;
  s.nk = a.k_len ? clamped(a.k_len[b], a.k_rows - s.k0) : s.nq;
  return s;
}
// Keys of a sequence's ranges: more than `chunk` only where the workspace would not hold them (max_k was too low).
__device__ __forceinline__ long long range_keys(const Tiles &g, long long nk) {
  if (g.chunk == 0) return max(nk, 1ll);
  return max((long long)g.chunk, ((nk + g.most - 1) / g.most + kKeys - 1) / kKeys * kKeys);
}

template <class T, int RI, int NE>
__global__ void __launch_bounds__(256) attention_rows_kernel(const mrf_attention_args a, const Tiles g) {
  extern __shared__ float4 smem[];
  constexpr int R = 16 * RI, kV = 64 * NE;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, ld = g.ld, width4 = (a.width + 3) / 4 * 4;
  float *qs = reinterpret_cast<float *>(smem), *ks = qs + R * ld, *vs = ks + kKeys * ld, *ps = vs + kKeys * kV;
  const int G = a.heads / a.kv_heads, sets = a.kv_heads * g.parts;
  for (long long u = blockIdx.x; u < g.units; u += gridDim.x) {
    const int range = (int)(u % g.most), set = (int)(u / g.most % sets);
    const long long x = u / g.most / sets;
    // Sequence b's tiles are x = q0 / TQ + b and on: places enough for all, whatever the lengths.
    auto first = [&](int b) { return clamped(a.q_offsets[b], a.q_rows) / g.TQ + b; };
    int b = 0;
    for (int hi = a.seqs; hi - b > 1;) {
      const int mid = (b + hi) >> 1;
      if (first(mid) <= x) b = mid;
      else hi = mid;
    }
    const Span s = load_span(a, b);
    const long long t = (s.nq + g.TQ - 1) / g.TQ - 1 - (x - first(b));  // last tiles (the most keys) first
    const long long chunk = range_keys(g, s.nk), r0 = range * chunk;
    const bool split = s.nk > chunk;
    if (x < first(b) || t < 0 || (range > 0 && r0 >= s.nk)) continue;
    const int ntok = (int)min((long long)g.TQ, s.nq - t * g.TQ);
    const int hk = set / g.parts, h0 = hk * G + set % g.parts * g.G1, nh = min(g.G1, (hk + 1) * G - h0);
    const long long tok0 = s.q0 + t * g.TQ, klen = min(s.nk - r0, chunk);
    const long long lim0 = a.causal ? t * g.TQ - s.nq + 1 + s.nk - r0 : klen;  // keys that the tile's first token sees
    const long long seen = max(0ll, min(klen, lim0 + ntok - 1));
    const T *kp = static_cast<const T *>(a.k) + (s.k0 + r0) * a.k_token_stride + hk * a.k_head_stride;
    const T *vp = static_cast<const T *>(a.v) + (s.k0 + r0) * a.v_token_stride + hk * a.v_head_stride;

    __syncthreads();  // the last tile's reads of shared memory
    for (int r = ty; r < R; r += 16) {
      const int tok = r / g.G1, h = r - tok * g.G1;
      const T *qp = static_cast<const T *>(a.q) + (tok0 + tok) * a.q_token_stride + (h0 + h) * a.q_head_stride;
      for (int d = tx; d < width4; d += 16) qs[r * ld + d] = tok < ntok && h < nh && d < a.width ? to_f32(qp[d]) : 0.f;
    }
    long long vis[RI];
    float m[RI], l[RI], o[RI][4 * NE];
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int r = ty + 16 * i, tok = r / g.G1;
      vis[i] = tok < ntok && r - tok * g.G1 < nh ? min(klen, lim0 + tok) : 0;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int n = 0; n < 4 * NE; ++n) o[i][n] = 0.f;
    }
    if (seen > 0) load_keys<T>(ks, ld, kp, a.k_token_stride, (int)min(klen, (long long)kKeys), a.width, g.vec);
    for (long long j = 0; j < seen; j += kKeys) {
      copies_landed();
      __syncthreads();
      load_keys<T>(vs, kV, vp + j * a.v_token_stride, a.v_token_stride, (int)min(klen - j, (long long)kKeys), a.v_width, g.vec);
      float sc[RI][4] = {};
#pragma unroll 2
      for (int d = 0; d < width4; d += 4) {
        float4 k[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) k[c] = *reinterpret_cast<const float4 *>(ks + (tx + 16 * c) * ld + d);
#pragma unroll
        for (int i = 0; i < RI; ++i) {
          const float4 q = *reinterpret_cast<const float4 *>(qs + (ty + 16 * i) * ld + d);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            sc[i][c] = fmaf(q.w, k[c].w, fmaf(q.z, k[c].z, fmaf(q.y, k[c].y, fmaf(q.x, k[c].x, sc[i][c]))));
        }
      }
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        const long long left = vis[i] - j;
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[i][c] = tx + 16 * c < left ? sc[i][c] * a.scale : -INFINITY;
        const float m1 = fmaxf(m[i], max16(fmaxf(fmaxf(sc[i][0], sc[i][1]), fmaxf(sc[i][2], sc[i][3]))));
        const float m0 = m1 == -INFINITY ? 0.f : m1, alpha = expf(m[i] - m0);
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float p = expf(sc[i][c] - m0);
          sum += p;
          ps[(ty + 16 * i) * kPad + tx + 16 * c] = p;
        }
        l[i] = l[i] * alpha + sum16(sum);
        m[i] = m1;
#pragma unroll
        for (int n = 0; n < 4 * NE; ++n) o[i][n] *= alpha;
      }
      copies_landed();
      __syncthreads();
      if (j + kKeys < seen)
        load_keys<T>(ks, ld, kp + (j + kKeys) * a.k_token_stride, a.k_token_stride, (int)min(klen - j - kKeys, (long long)kKeys), a.width,
                     g.vec);
      for (int c = 0; c < kKeys; c += 4) {
        float4 p[RI];
#pragma unroll
        for (int i = 0; i < RI; ++i) p[i] = *reinterpret_cast<const float4 *>(ps + (ty + 16 * i) * kPad + c);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int n = 0; n < NE; ++n) {
            const float4 v = *reinterpret_cast<const float4 *>(vs + (c + e) * kV + 64 * n + 4 * tx);
#pragma unroll
            for (int i = 0; i < RI; ++i) {
              const float w = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
              o[i][4 * n] = fmaf(w, v.x, o[i][4 * n]);
              o[i][4 * n + 1] = fmaf(w, v.y, o[i][4 * n + 1]);
              o[i][4 * n + 2] = fmaf(w, v.z, o[i][4 * n + 2]);
              o[i][4 * n + 3] = fmaf(w, v.w, o[i][4 * n + 3]);
            }
          }
      }
    }
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int r = ty + 16 * i, tok = r / g.G1, h = h0 + r - tok * g.G1;
      if (tok >= ntok || h >= h0 + nh) continue;
      const bool any = l[i] > 0.f || l[i] != l[i];
      const float inv = any ? 1.f / l[i] : 0.f;
      const float lse = any ? m[i] + logf(l[i]) : -INFINITY;
      const long long row = (tok0 + tok) * a.heads + h, at = (range * a.q_rows * a.heads + row) * a.v_width;
      T *op = static_cast<T *>(a.out) + (tok0 + tok) * a.out_token_stride + h * a.out_head_stride;
#pragma unroll
      for (int n = 0; n < 4 * NE; ++n) {
        const int e = 64 * (n / 4) + 4 * tx + n % 4;
        const float v = any ? o[i][n] * inv : 0.f;
        if (e < a.v_width) {
          if (split) g.part[at + e] = v;
          else op[e] = from_f32<T>(v);
        }
      }
      if (tx == 0) {
        if (split) g.part_lse[range * a.q_rows * a.heads + row] = lse;
        else if (a.lse) a.lse[row] = lse;
      }
    }
  }
}

// Joins the ranges of the sequences that were split: a warp a (row, head), weights e^(L - max L), in their order.
template <class T>
__global__ void __launch_bounds__(128) rows_join_kernel(const mrf_attention_args a, const Tiles g) {
  const int lane = threadIdx.x & 31;
  const long long n = a.q_rows * a.heads;
  for (long long i = blockIdx.x * 4ll + (threadIdx.x >> 5); i < n; i += gridDim.x * 4ll) {
    const long long tok = i / a.heads;
    int b = 0;
    for (int hi = a.seqs; hi - b > 1;) {
      const int mid = (b + hi) >> 1;
      if (a.q_offsets[mid] <= tok) b = mid;
      else hi = mid;
    }
    const Span s = load_span(a, b);
    const long long chunk = range_keys(g, s.nk);
    if (tok < s.q0 || tok >= s.q0 + s.nq || s.nk <= chunk) continue;  // of no sequence, or already written
    const int ranges = (int)((s.nk + chunk - 1) / chunk);
    float top = -INFINITY, total = 0.f, o[8] = {};
    for (int k = lane; k < ranges; k += 32) top = fmaxf(top, g.part_lse[k * n + i]);
    for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
#pragma unroll 4
    for (int k = 0; k < ranges; ++k) {
      const float L = g.part_lse[k * n + i];
      if (L == -INFINITY) continue;  // it saw no key
      const float w = expf(L - top);
      total += w;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (lane + 32 * e < a.v_width) o[e] = fmaf(w, g.part[(k * n + i) * a.v_width + lane + 32 * e], o[e]);
    }
    const bool any = total > 0.f || total != total;
    T *op = static_cast<T *>(a.out) + tok * a.out_token_stride + (i - tok * a.heads) * a.out_head_stride;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (lane + 32 * e < a.v_width) op[lane + 32 * e] = from_f32<T>(any ? o[e] / total : 0.f);
    if (a.lse && lane == 0) a.lse[i] = any ? top + logf(total) : -INFINITY;
  }
}

// 16 RI rows a tile, by the rows that a sequence has for a key head.  fp32, RI = 1, 4, 8, in us: a token after 16000
// keys (4 rows) 106, 174, 271; 40 sequences of 30 to 60 tokens 36, 34, 48, of 17 to 300 83, 72, 84; 8 of 1100 tokens
// 1500, 840, 668.  Wide heads leave room in shared memory for 64 rows.
int rows_of(const mrf_attention_args &a) {
  const long long rows = a.q_rows * (a.heads / a.kv_heads) / a.seqs;
  return rows <= 16 ? 1 : rows <= 192 || a.width > 128 || a.v_width > 128 ? 4 : 8;
}

Tiles tiles_of(const mrf_attention_args &a) {
  Tiles g = {};
  const int R = 16 * rows_of(a), G = a.heads / a.kv_heads;
  g.G1 = std::min(G, R);
  g.parts = (G + g.G1 - 1) / g.G1;
  g.TQ = R / g.G1;
  g.ld = (a.width + 3) / 4 * 4;
  if (g.ld / 4 % 2 == 0) g.ld += 4;
  auto pieces = [](const void *p, long long token, long long head, int width) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && token % 4 == 0 && head % 4 == 0 && width % 4 == 0;
  };
  g.vec = pieces(a.k, a.k_token_stride, a.k_head_stride, a.width) && pieces(a.v, a.v_token_stride, a.v_head_stride, a.v_width);
  // a range's 128 keys take the tile's multiply-adds, 128 a clk, and what stands beside them
  const double block = std::max(2.0, 1.3 * R * (a.width + a.v_width) / 1900.);
  const AttentionSplit s = attention_split(a, g.TQ, (long long)a.kv_heads * g.parts, block);
  g.chunk = s.chunk;
  g.most = s.most;
  g.units = (a.q_rows / g.TQ + a.seqs) * a.kv_heads * g.parts * g.most;
  g.part = static_cast<float *>(a.workspace);
  g.part_lse = g.part + (g.chunk ? (size_t)g.most * a.q_rows * a.heads * a.v_width : 0);
  return g;
}

size_t workspace_of(const mrf_attention_args &a, const Tiles &g) {
  return g.chunk ? (size_t)g.most * a.q_rows * a.heads * (a.v_width + 1) * sizeof(float) : 0;
}

template <class T, int RI, int NE>
cudaError_t launch(const mrf_attention_args &a, const Tiles &g, cudaStream_t st) {
  const int smem = (int)sizeof(float) * (16 * RI * (g.ld + kPad) + kKeys * (g.ld + 64 * NE));
  auto *k = attention_rows_kernel<T, RI, NE>;
  static std::atomic<unsigned long long> ready{0};  // devices whose limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1))) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e == cudaSuccess && dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  k<<<(unsigned)std::min<long long>(g.units, 1 << 30), 256, smem, st>>>(a, g);
  e = cudaGetLastError();
  if (e != cudaSuccess || g.chunk == 0) return e;
  rows_join_kernel<T><<<(unsigned)std::min<long long>((a.q_rows * a.heads + 3) / 4, 16 * sm_count()), 128, 0, st>>>(a, g);
  return cudaGetLastError();
}
template <class T>
cudaError_t launch(const mrf_attention_args &a, cudaStream_t st) {
  Tiles g = tiles_of(a);
  if (a.workspace_bytes < workspace_of(a, g)) {  // (sized for the tensor-core kernel, whose tensor maps were refused)
    g.units /= g.most;
    g.chunk = 0;
    g.most = 1;
  }
  const int ri = rows_of(a), ne = a.v_width <= 64 ? 1 : a.v_width <= 128 ? 2 : 4;
  if (ri == 1) return ne == 1 ? launch<T, 1, 1>(a, g, st) : ne == 2 ? launch<T, 1, 2>(a, g, st) : launch<T, 1, 4>(a, g, st);
  if (ri == 4) return ne == 1 ? launch<T, 4, 1>(a, g, st) : ne == 2 ? launch<T, 4, 2>(a, g, st) : launch<T, 4, 4>(a, g, st);
  return ne == 1 ? launch<T, 8, 1>(a, g, st) : launch<T, 8, 2>(a, g, st);
}

}  // namespace

size_t attention_rows_workspace(const mrf_attention_args &a) {
  return workspace_of(a, tiles_of(a));
}

cudaError_t launch_attention_rows(const mrf_attention_args &a, cudaStream_t st) {
  if (a.dtype == MRF_DTYPE_F32) return launch<float>(a, st);
  if (a.dtype == MRF_DTYPE_F16) return launch<__half>(a, st);
  return launch<__nv_bfloat16>(a, st);
}

}  // namespace mrf
