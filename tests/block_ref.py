"""The block operators (norm, rotary positions, packed attention) in 64 bits, written from their
formulas, and how far a kernel that follows them may be off."""
import math

import torch

U32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rms_norm(x, weight, eps, residual=None, clamp=False):
    """(y, h) in 64 bits."""
    h = x.double() if residual is None else x.double() + residual.double()
    r = h.square().mean(-1, keepdim=True).sqrt()
    s = 1 / r.clamp(min=eps) if clamp else 1 / (r.square() + eps).sqrt()
    return h * s * (1.0 if weight is None else weight.double()), h


def norm_slack(dim):
    """Relative error of y before its rounding: h rounds once; the sum of squares runs in chains of at
    most dim / 32 + 16 additions, each half a step (its root halves that); the mean, the root, the
    reciprocal, two products and the weight's product round once each."""
    return ((dim / 32 + 16) / 2 + 8) * U32


def rope_frequencies(part, theta=10000.0, scaling="none", factor=1.0, original=0):
    n = part
    f = [theta ** (-2 * i / n) for i in range(n // 2)]
    if scaling == "linear":
        f = [v / factor for v in f]
    if scaling == "ntk":
        t = theta * factor ** (n / (n - 2))
        f = [t ** (-2 * i / n) for i in range(n // 2)]
    mul = 1.0
    if scaling == "yarn":
        dim = lambda turns: n * math.log(original / (2 * math.pi * turns)) / (2 * math.log(theta))
        lo, hi = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), n - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0), 1) for i in range(n // 2)]
        f = [v * (1 - r) + v / factor * r for v, r in zip(f, ramp)]
        mul = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    return f, mul


def rope(x, positions, frequencies, mul, interleaved):
    """x [tokens, heads, width] turned, in 64 bits, and each output's |a| + |b| (its pair's size)."""
    n = 2 * len(frequencies)
    f = torch.tensor(frequencies, dtype=torch.float64, device=x.device)
    angle = positions.double()[:, None, None] * f
    c, s = torch.cos(angle) * mul, torch.sin(angle) * mul
    y, size = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    even, odd = (slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2), slice(n // 2, n))
    a, b = x[..., even].double(), x[..., odd].double()
    y[..., even], y[..., odd] = a * c - b * s, b * c + a * s
    size[..., even] = size[..., odd] = (a.abs() + b.abs()) * abs(mul)
    return y, size


def rope_slack(size):
    """The angle is off by at most half a step of fp32 at one half turn, pi 2^-25 < 2 U32; cos and sin
    are within 2 U32; the factor, the product and the fused sum round once each."""
    return size * 8 * U32


def attention(q, k, v, spans, causal, scale):
    """q [nq, H, D], k [nk, K, D], v [nk, K, E]; spans: (q0, nq, k0, nk) for each sequence.  out and lse in
    64 bits (NaN in rows of no sequence), and per output sum p |v| and the row's largest sum |q k| scale."""
    nq, H = q.shape[:2]
    G = H // k.shape[1]
    out = torch.full((nq, H, v.shape[2]), math.nan, dtype=torch.float64, device=q.device)
    size, lse = out.clone(), out[..., 0].clone()
    big = lse.clone()
    for q0, n, k0, m in spans:
        a = q[q0 : q0 + n].double().transpose(0, 1)  # [H, n, D]
        b = k[k0 : k0 + m].double().transpose(0, 1).repeat_interleave(G, 0)
        c = v[k0 : k0 + m].double().transpose(0, 1).repeat_interleave(G, 0)
        s = a @ b.transpose(1, 2) * scale
        sizes = a.abs() @ b.abs().transpose(1, 2) * scale
        if causal:
            hidden = torch.arange(m, device=q.device) > torch.arange(n, device=q.device)[:, None] + (m - n)
            s = s.masked_fill(hidden, -math.inf)
            sizes = sizes.masked_fill(hidden, 0.0)
        if m == 0:
            s, sizes = s.new_zeros(H, n, 0), s.new_zeros(H, n, 0)
        top = s.amax(-1, keepdim=True) if m else s.new_full((H, n, 1), -math.inf)
        top = torch.where(top == -math.inf, 0.0, top)
        p = (s - top).exp()
        l = p.sum(-1, keepdim=True)
        p = p / torch.where(l > 0, l, 1.0)
        out[q0 : q0 + n] = (p @ c).transpose(0, 1)
        size[q0 : q0 + n] = (p @ c.abs()).transpose(0, 1)
        lse[q0 : q0 + n] = (top + l.log())[..., 0].T
        big[q0 : q0 + n] = (sizes.amax(-1) if m else s.new_zeros(H, n)).T
    return out, lse, size, big


def attention_slack(dtype, out, size, big, keys, width):
    """(bound of out, bound of lse).  A score is a sum of `width` products in fp32, whose error is at most
    width 2^-23 of its absolute sum (each addition a whole step); its exponential is within 2^-22 and
    rounds to the type for the second product (half a step; not for fp32); sums over the keys run in
    fp32, whole steps of 2^-23 over chains of at most keys / 16 + 64; the output rounds once."""
    score = big * width * 2.0**-23 + 2.0**-22 + 4 * U32
    sums = (keys / 16 + 64) * 2.0**-23
    weights = half_step(dtype) if dtype != torch.float32 else 0.0
    # an error of `score` in the exponents moves every weight by that factor, above and below the line
    bound = size * (2 * score[..., None] + 2 * sums + weights) + half_step(dtype) * out.abs() + 2.0**-24 * size
    return bound, score + sums + lse_step(keys)


def lse_step(keys):
    """The logarithm's own rounding and the sum with the largest score: magnitudes up to about 32."""
    return 32 * 2 * U32
