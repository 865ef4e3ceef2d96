// C ABI of the block operators (include/mrf.h: mrf_rms_norm, mrf_rope_table, mrf_rope,
// mrf_attention): argument checks and kernel choice.  Nothing here allocates or throws.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "block_ops.h"
#include "op_status.h"

using namespace mrf;

namespace {

mrf_status op_fail(mrf_status s, const char *fmt, ...) noexcept {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_thread_error(buf);
  return s;
}

// What a launch (or a sync) of `what` left behind.
mrf_status op_done(cudaError_t e, const char *what) noexcept {
  if (e == cudaSuccess) return MRF_OK;
  cudaGetLastError();
  return op_fail(MRF_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool real_type(int t) { return t == MRF_DTYPE_F32 || t == MRF_DTYPE_F16 || t == MRF_DTYPE_BF16; }
uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }
int type_size(int t) { return t == MRF_DTYPE_F32 ? 4 : t == MRF_DTYPE_E4M3 ? 1 : 2; }
bool aligned(const void *p, int t) { return addr(p) % type_size(t) == 0; }

// a [n, inner] tensor whose rows are written: they must not overlap
bool rows_apart(long long n, long long stride, long long inner) { return n <= 1 || stride >= inner || stride <= -inner; }

// a written [n1, n2, inner] tensor: one of the two outer dimensions lies inside the other's stride
bool apart(long long n1, long long s1, long long n2, long long s2, long long inner) {
  if (!rows_apart(n1, s1, inner) || !rows_apart(n2, s2, inner)) return false;
  if (n1 <= 1 || n2 <= 1) return true;
  const long long a1 = std::llabs(s1), a2 = std::llabs(s2);
  return a1 >= a2 ? a1 >= (n2 - 1) * a2 + inner : a2 >= (n1 - 1) * a1 + inner;
}

}  // namespace

extern "C" {

mrf_status mrf_rms_norm(const mrf_rms_norm_args *a, void *stream) {
  if (!a) return op_fail(MRF_EINVAL, "mrf_rms_norm: null arguments");
  if (!real_type(a->dtype) || (a->weight && !real_type(a->weight_dtype)))
    return op_fail(MRF_EINVAL, "mrf_rms_norm: dtype and weight_dtype must be F32, F16 or BF16");
  if (a->out_dtype != a->dtype && a->out_dtype != MRF_DTYPE_E4M3)
    return op_fail(MRF_EINVAL, "mrf_rms_norm: out_dtype must be dtype or E4M3");
  if (a->rows < 0 || a->dim < 1) return op_fail(MRF_ESHAPE, "mrf_rms_norm: rows >= 0 and dim >= 1 required");
  if (a->dim > 16384) return op_fail(MRF_EUNSUPPORTED, "mrf_rms_norm: dim %d is above 16384", a->dim);
  const bool quant = a->out_dtype == MRF_DTYPE_E4M3;
  if (quant ? a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128 : a->group != 0)
    return op_fail(MRF_EINVAL, "mrf_rms_norm: group must be 0, or 32, 64 or 128 with an E4M3 output");
  if (!(a->eps > 0.f) || !std::isfinite(a->eps)) return op_fail(MRF_EINVAL, "mrf_rms_norm: eps must be positive and finite");
  if (a->residual_out && !a->residual) return op_fail(MRF_EINVAL, "mrf_rms_norm: residual_out without residual");
  if (quant ? a->rows > 0 && !a->scales : a->scales != nullptr)
    return op_fail(MRF_EINVAL, "mrf_rms_norm: scales go with an E4M3 output, and only with one");
  if (a->rows == 0) return MRF_OK;
  if (!a->x || !a->out) return op_fail(MRF_EINVAL, "mrf_rms_norm: null x or out pointer");
  if (!aligned(a->x, a->dtype) || !aligned(a->residual, a->dtype) || !aligned(a->residual_out, a->dtype) ||
      !aligned(a->out, a->out_dtype) || (a->weight && !aligned(a->weight, a->weight_dtype)) ||
      !aligned(a->scales, MRF_DTYPE_F32))
    return op_fail(MRF_EINVAL, "mrf_rms_norm: a pointer is not aligned to its type");
  if (!rows_apart(a->rows, a->out_stride, a->dim) ||
      (a->residual_out && !rows_apart(a->rows, a->residual_out_stride, a->dim)))
    return op_fail(MRF_ESHAPE, "mrf_rms_norm: output rows overlap");
  if (a->residual_out && (a->residual_out == a->out || a->residual_out == a->x))
    return op_fail(MRF_EINVAL, "mrf_rms_norm: residual_out overlaps out or x");
  if (a->out == a->residual || (a->out == a->x && (quant || (a->rows > 1 && a->out_stride != a->x_stride))))
    return op_fail(MRF_EINVAL, "mrf_rms_norm: out may be x only with the same stride and type, and never residual");
  if (a->residual_out && a->residual_out == a->residual && a->rows > 1 && a->residual_out_stride != a->residual_stride)
    return op_fail(MRF_EINVAL, "mrf_rms_norm: residual_out may be residual only with the same stride");
  return op_done(launch_rms_norm(*a, static_cast<cudaStream_t>(stream)), "mrf_rms_norm");
}

mrf_status mrf_rope_table(const mrf_rope_config *c, uint64_t *turns, float *scale) {
  if (!c || !turns || !scale) return op_fail(MRF_EINVAL, "mrf_rope_table: null pointer");
  if (c->part < 2 || c->part > 1024 || (c->part & 1)) return op_fail(MRF_ESHAPE, "mrf_rope_table: part must be even, 2 to 1024");
  if (!(c->theta > 1.0) || !std::isfinite(c->theta)) return op_fail(MRF_EINVAL, "mrf_rope_table: theta must be > 1");
  if (c->scaling < MRF_ROPE_NONE || c->scaling > MRF_ROPE_YARN) return op_fail(MRF_EINVAL, "mrf_rope_table: unknown scaling");
  if (c->scaling != MRF_ROPE_NONE && (!(c->factor >= 1.0) || !std::isfinite(c->factor)))
    return op_fail(MRF_EINVAL, "mrf_rope_table: factor must be >= 1");
  if (c->scaling == MRF_ROPE_NTK && c->part == 2) return op_fail(MRF_EINVAL, "mrf_rope_table: NTK needs part > 2");
  // Frequencies in long double (64 bits of fraction): a double's 53 would be off by 2^-56 of a turn a position.
  // The border dimensions of YARN are whole numbers, which double gives as their definition's usual form does.
  const long double pi2 = 6.283185307179586476925286766559005768L, n = c->part, factor = c->factor;
  long double theta = c->theta;
  double lo = 0, hi = 0;
  if (c->scaling == MRF_ROPE_NTK) theta *= std::pow(factor, n / (n - 2));
  if (c->scaling == MRF_ROPE_YARN) {
    const double fast = c->beta_fast == 0 && c->beta_slow == 0 ? 32 : c->beta_fast;
    const double slow = c->beta_fast == 0 && c->beta_slow == 0 ? 1 : c->beta_slow;
    if (!(c->original >= 1.0) || !std::isfinite(c->original) || !(slow > 0) || !(fast > slow) || !std::isfinite(fast))
      return op_fail(MRF_EINVAL, "mrf_rope_table: original >= 1 and beta_fast > beta_slow > 0 required");
    auto dim = [&](double t) { return c->part * std::log(c->original / (t * (double)pi2)) / (2 * std::log(c->theta)); };
    lo = std::fmax(std::floor(dim(fast)), 0.0);
    hi = std::fmin(std::ceil(dim(slow)), c->part - 1.0);
  }
  *scale = 1.f;
  if (c->scaling == MRF_ROPE_YARN && c->factor > 1.0) *scale = (float)(0.1 * std::log(c->factor) + 1.0);
  for (int i = 0; i < c->part / 2; ++i) {
    long double f = std::pow(theta, -2 * i / n);
    if (c->scaling == MRF_ROPE_LINEAR) f /= factor;
    if (c->scaling == MRF_ROPE_YARN) {
      const long double r = std::fmin(std::fmax((i - lo) / (long double)std::fmax(hi - lo, 0.001), 0.0L), 1.0L);
      f = f / factor * r + f * (1 - r);
    }
    turns[i] = (uint64_t)std::llround(std::ldexp(f / pi2, 64));  // f <= 1 radian: below 2^64 * 0.16
  }
  return MRF_OK;
}

mrf_status mrf_rope(const mrf_rope_args *a, void *stream) {
  if (!a) return op_fail(MRF_EINVAL, "mrf_rope: null arguments");
  if (!real_type(a->dtype)) return op_fail(MRF_EINVAL, "mrf_rope: dtype must be F32, F16 or BF16");
  if (a->tokens < 0 || a->tokens > INT32_MAX || a->heads < 1 || a->heads > 65536 || a->kv_heads < 0 ||
      a->kv_heads > 65536 || (a->tokens > 0 && a->kv_heads > 0 && !a->k))
    return op_fail(MRF_ESHAPE, "mrf_rope: tokens in [0, 2^31), heads >= 1 and kv_heads >= 0 (0 without k) required");
  if (a->width < 2 || a->width > 1024 || a->part < 2 || a->part > a->width || (a->part & 1))
    return op_fail(MRF_ESHAPE, "mrf_rope: width up to 1024 and an even part in [2, width] required");
  if (!std::isfinite(a->scale)) return op_fail(MRF_EINVAL, "mrf_rope: scale must be finite");
  if (a->tokens == 0) return MRF_OK;
  if (!a->q || !a->q_out || !a->positions || !a->turns || (a->kv_heads > 0 && (!a->k || !a->k_out)))
    return op_fail(MRF_EINVAL, "mrf_rope: null q, k, output, positions or turns pointer");
  if (!aligned(a->q, a->dtype) || !aligned(a->q_out, a->dtype) || !aligned(a->k, a->dtype) || !aligned(a->k_out, a->dtype) ||
      addr(a->positions) % (a->positions_wide ? 8 : 4) || addr(a->turns) % 8)
    return op_fail(MRF_EINVAL, "mrf_rope: a pointer is not aligned to its type");
  if (!apart(a->tokens, a->q_out_token_stride, a->heads, a->q_out_head_stride, a->width) ||
      (a->kv_heads > 0 && !apart(a->tokens, a->k_out_token_stride, a->kv_heads, a->k_out_head_stride, a->width)))
    return op_fail(MRF_ESHAPE, "mrf_rope: output heads overlap");
  if (a->q_out == a->q && ((a->tokens > 1 && a->q_out_token_stride != a->q_token_stride) ||
                           (a->heads > 1 && a->q_out_head_stride != a->q_head_stride)))
    return op_fail(MRF_EINVAL, "mrf_rope: q_out may be q only with the same strides");
  if (a->kv_heads > 0 && a->k_out == a->k &&
      ((a->tokens > 1 && a->k_out_token_stride != a->k_token_stride) ||
       (a->kv_heads > 1 && a->k_out_head_stride != a->k_head_stride)))
    return op_fail(MRF_EINVAL, "mrf_rope: k_out may be k only with the same strides");
  return op_done(launch_rope(*a, static_cast<cudaStream_t>(stream)), "mrf_rope");
}

namespace {

mrf_status check_attention(const mrf_attention_args *a) {
  if (!a) return op_fail(MRF_EINVAL, "mrf_attention: null arguments");
  if (!real_type(a->dtype)) return op_fail(MRF_EINVAL, "mrf_attention: dtype must be F32, F16 or BF16");
  if (a->seqs < 0 || a->q_rows < 0 || a->k_rows < 0 || a->q_rows > INT32_MAX || a->k_rows > INT32_MAX || a->max_k < 0)
    return op_fail(MRF_ESHAPE, "mrf_attention: seqs, q_rows, k_rows and max_k must be >= 0, rows below 2^31");
  if (a->heads < 1 || a->kv_heads < 1 || a->heads > 65536 || a->heads % a->kv_heads)
    return op_fail(MRF_ESHAPE, "mrf_attention: heads (up to 65536) must be a multiple of kv_heads >= 1");
  if (a->width < 1 || a->v_width < 1) return op_fail(MRF_ESHAPE, "mrf_attention: width and v_width must be >= 1");
  if (a->width > 256 || a->v_width > 256)
    return op_fail(MRF_EUNSUPPORTED, "mrf_attention: width %d or v_width %d is above 256", a->width, a->v_width);
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return op_fail(MRF_EINVAL, "mrf_attention: scale must be positive and finite");
  if ((a->k_start != nullptr) != (a->k_len != nullptr))
    return op_fail(MRF_EINVAL, "mrf_attention: k_start and k_len go together");
  if (a->q_rows == 0 || a->seqs == 0) return MRF_OK;
  if (!a->q || !a->out || !a->q_offsets || (a->k_rows > 0 && (!a->k || !a->v)))
    return op_fail(MRF_EINVAL, "mrf_attention: null q, k, v, out or q_offsets pointer");
  if (!aligned(a->q, a->dtype) || !aligned(a->k, a->dtype) || !aligned(a->v, a->dtype) || !aligned(a->out, a->dtype) ||
      addr(a->lse) % 4 || addr(a->q_offsets) % 4 || addr(a->k_start) % 4 || addr(a->k_len) % 4)
    return op_fail(MRF_EINVAL, "mrf_attention: a pointer is not aligned to its type");
  if (!a->k_len && a->k_rows < a->q_rows)
    return op_fail(MRF_ESHAPE, "mrf_attention: without k_start and k_len the keys need q_rows rows");
  if (!apart(a->q_rows, a->out_token_stride, a->heads, a->out_head_stride, a->v_width))
    return op_fail(MRF_ESHAPE, "mrf_attention: output rows overlap");
  if (a->out == a->q || a->out == a->k || a->out == a->v)
    return op_fail(MRF_EINVAL, "mrf_attention: out must not overlap the inputs");
  return MRF_OK;
}

}  // namespace

mrf_status mrf_attention_workspace(const mrf_attention_args *a, size_t *bytes) {
  if (!bytes) return op_fail(MRF_EINVAL, "mrf_attention_workspace: null bytes pointer");
  *bytes = 0;
  const mrf_status s = check_attention(a);
  if (s == MRF_OK && a->q_rows > 0 && a->seqs > 0) *bytes = attention_tc_takes(*a) ? attention_tc_workspace(*a) : attention_rows_workspace(*a);
  return s;
}

mrf_status mrf_attention(const mrf_attention_args *a, void *stream) {
  const mrf_status s = check_attention(a);
  if (s != MRF_OK || a->q_rows == 0 || a->seqs == 0) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool tc = attention_tc_takes(*a);
  const size_t need = tc ? attention_tc_workspace(*a) : attention_rows_workspace(*a);
  if (need > 0 && (!a->workspace || addr(a->workspace) % 16 || a->workspace_bytes < need))
    return op_fail(MRF_EINVAL, "mrf_attention: the workspace must hold %zu bytes, 16-byte aligned", need);
  cudaError_t e = cudaSuccess;
  if (tc && launch_attention_packed_tc(*a, st, &e)) return op_done(e, "mrf_attention");
  mrf_attention_args rest = *a;
  if (tc) rest.workspace_bytes = need;  // what was checked, for a kernel that would like more
  return op_done(launch_attention_rows(rest, st), "mrf_attention");
}

mrf_status mrf_ops_sync_status(void *stream) {
  static ExpiredWaits waits[64];
  static thread_local unsigned seen[64] = {};
  int dev = 0;
  unsigned word[2] = {0, 0};
  mrf_status s = op_done(cudaGetDevice(&dev), "mrf_ops_sync_status");
  if (s == MRF_OK) s = op_done(attention_tc_status(word, static_cast<cudaStream_t>(stream)), "mrf_ops_sync_status");
  if (s != MRF_OK) return s;
  ExpiredWaits &w = waits[dev % 64];
  if (word[0] != 0) w.found(word[1]);
  if (!w.since(seen[dev % 64])) return MRF_OK;
  return op_fail(MRF_ETIMEOUT, "mrf_attention: a bounded wait expired on the device (site %u)", w.site.load());
}

}  // extern "C"
