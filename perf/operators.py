"""What the transformer-block operators are measured on: cases, inputs, plain forms and 64-bit results.

The operators are what stands between the matrix products of a causal transformer block over packed
sequences: the root-mean-square norm with the residual's addition (and an 8-bit output with scales),
rotary positions, and attention with grouped heads over packed sequences or a cache.

`run` computes an operator in plain torch operations in 32 bits (`own` false) or through the
package's public calls (`own` true); `exact` gives its result from the definition in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}
E4M3_MAX = 448.0


# ----------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a decoder block: the smallest call, latency counts
        dict(name="norm_token", op="norm", rows=1, dim=4096, dtype="bf16", residual=True, quant=True, group=0, clamp=False),
        # the vocals model's own width over the tokens of a short window (70 frames x 60 bands and one row more)
        dict(name="norm_window", op="norm", rows=4201, dim=384, dtype="fp16", residual=True, quant=False, group=0, clamp=True),
        # a long prompt before an 8-bit product: a scale for each 128 columns
        dict(name="norm_prompt", op="norm", rows=16384, dim=4096, dtype="bf16", residual=True, quant=True, group=128, clamp=False),
        # one token of each of 32 requests far into long contexts, frequencies scaled by parts
        dict(name="rope_tokens", op="rope", tokens=32, heads=32, kv_heads=8, width=128, part=128, interleaved=False, scaling="yarn",
             far=1 << 20, dtype="bf16"),
        # the vocals model's heads and pair layout with half of each head rotated, an odd number of tokens
        dict(name="rope_part", op="rope", tokens=4099, heads=8, kv_heads=8, width=64, part=32, interleaved=True, scaling="none",
             far=4099, dtype="fp16"),
        # a long prompt with grouped heads
        dict(name="rope_prompt", op="rope", tokens=16384, heads=32, kv_heads=8, width=128, part=128, interleaved=False, scaling="linear",
             far=16384, dtype="bf16"),
        # many short clips packed without padding, the vocals model's heads
        dict(name="attn_clips", op="attention", seqs=40, q_min=17, q_max=300, past_min=0, past_max=0, heads=8, kv_heads=8, width=64,
             v_width=64, causal=True, lse=False, dtype="fp16", lengths=1),
        # packed prompts of mixed length, grouped heads
        dict(name="attn_prompts", op="attention", seqs=7, q_min=200, q_max=4096, past_min=0, past_max=0, heads=32, kv_heads=8, width=128,
             v_width=128, causal=True, lse=False, dtype="bf16", lengths=2),
        # one long prompt
        dict(name="attn_long", op="attention", seqs=1, q_min=16384, q_max=16384, past_min=0, past_max=0, heads=16, kv_heads=4, width=128,
             v_width=128, causal=True, lse=True, dtype="bf16", lengths=3),
        # one window's frames looking both ways, as the time axis of the vocals model at T = 1100 does
        dict(name="attn_window", op="attention", seqs=8, q_min=1100, q_max=1100, past_min=0, past_max=0, heads=8, kv_heads=8, width=64,
             v_width=64, causal=False, lse=False, dtype="fp16", lengths=4),
        # one new token of each of 32 requests over their caches
        dict(name="attn_tokens", op="attention", seqs=32, q_min=1, q_max=1, past_min=500, past_max=8191, heads=32, kv_heads=8, width=128,
             v_width=128, causal=True, lse=False, dtype="bf16", lengths=5),
        # one new token of a single request over a long cache
        dict(name="attn_token", op="attention", seqs=1, q_min=1, q_max=1, past_min=65536, past_max=65536, heads=32, kv_heads=8, width=128,
             v_width=128, causal=True, lse=False, dtype="bf16", lengths=6),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("norm", "rope", "attention", "attention"))
    if op == "norm":
        dim = _log(rng, 64, 8192)
        dim = dim if rng.random() < 0.25 else max(64, dim // 64 * 64)  # most widths are whole vectors, some are not
        rows = _log(rng, 1, max(1, min(20000, 16384 * 4096 // dim)))
        quant = rng.random() < 0.5
        return dict(op=op, rows=rows, dim=dim, dtype=rng.choice(("fp16", "bf16") if quant else ("fp16", "bf16", "fp32")),
                    residual=rng.random() < 0.7, quant=quant, group=rng.choice((0, 32, 64, 128)) if quant else 0, clamp=rng.random() < 0.3)
    if op == "rope":
        width = rng.choice((32, 64, 80, 96, 128, 256))
        kv = rng.choice((1, 2, 4, 8))
        heads = kv * rng.choice((1, 2, 3, 4, 7))
        tokens = _log(rng, 1, max(1, min(20000, 16384 * 40 * 128 // ((heads + kv) * width))))
        return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv, width=width, part=rng.choice((width, width, width // 2, width // 4 // 2 * 2)),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(("none", "linear", "ntk", "yarn")), far=_log(rng, 100, 1 << 20),
                    dtype=rng.choice(("fp16", "bf16", "fp32")))
    width = rng.choice((64, 64, 128, 128, 96, 80))
    kv = rng.choice((1, 2, 4, 8))
    heads = kv * rng.choice((1, 1, 2, 3, 4, 5, 7, 8))
    v_width = 64 if width == 128 and rng.random() < 0.2 else width
    c = dict(op=op, heads=heads, kv_heads=kv, width=width, v_width=v_width, causal=rng.random() < 0.8, lse=rng.random() < 0.3,
             dtype=rng.choice(("fp16", "bf16")), lengths=rng.randrange(1 << 20))
    kind = rng.choice(("prompt", "prompt", "tokens", "chunk"))
    if kind == "prompt":
        q_max = _log(rng, 2, 8192)
        seqs = _log(rng, 1, max(1, min(64, (1 << 30) // (heads * q_max * q_max))))
        c.update(seqs=seqs, q_min=max(1, q_max // rng.choice((1, 4, 16))), q_max=q_max, past_min=0, past_max=0)
    elif kind == "tokens":
        past = _log(rng, 16, 65536)
        seqs = _log(rng, 1, max(1, min(128, (1 << 18) // past)))
        c.update(seqs=seqs, q_min=1, q_max=1, past_min=past // rng.choice((1, 4, 16)), past_max=past)
    else:  # a prompt's next piece over what the cache holds
        q_max, past = _log(rng, 2, 1024), _log(rng, 16, 16384)
        seqs = _log(rng, 1, max(1, min(16, (1 << 30) // (heads * q_max * (q_max + past)))))
        c.update(seqs=seqs, q_min=max(1, q_max // 4), q_max=q_max, past_min=past // 4, past_max=past)
    return c


def _lengths(case):
    """Each sequence's number of queries and of keys: part of the case, whatever the inputs' seed."""
    r = random.Random(case["lengths"])
    q = [_log(r, case["q_min"], case["q_max"]) for _ in range(case["seqs"])]
    past = [r.randint(case["past_min"], case["past_max"]) for _ in range(case["seqs"])]
    return q, [a + b for a, b in zip(q, past)]


def work(case):
    es = SIZE[case["dtype"]]
    if case["op"] == "norm":
        n = case["rows"] * case["dim"]
        groups = -(-case["dim"] // case["group"]) if case["group"] else 1
        moved = n * es + (2 * n * es if case["residual"] else 0) + (n + 4 * case["rows"] * groups if case["quant"] else n * es)
        return {"bytes": moved + 4 * case["dim"], "flops": 5 * n}
    if case["op"] == "rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["width"]
        return {"bytes": 2 * n * es + 4 * case["tokens"] + 4 * case["part"], "flops": 3 * n}
    q, k = _lengths(case)
    pairs = sum(a * b - (a * (a - 1) // 2 if case["causal"] else 0) for a, b in zip(q, k))
    moved = sum(q) * case["heads"] * (case["width"] + case["v_width"]) * es + sum(k) * case["kv_heads"] * (case["width"] + case["v_width"]) * es
    return {"bytes": moved + (4 * sum(q) * case["heads"] if case["lse"] else 0) + 12 * case["seqs"] + 4,
            "flops": 2 * pairs * case["heads"] * (case["width"] + case["v_width"])}


# ---------------------------------------------------------------------------------------- inputs
YARN = dict(factor=32.0, original=4096)


def _tensors(case, seed):
    """The case's input tensors, from the seed alone."""
    g = torch.Generator("cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "norm":
        # activations have a few columns far larger than the others
        big = 1 + 20 * (torch.rand(case["dim"], generator=g, device="cuda") < 0.01).float()
        x = {"x": (normal(case["rows"], case["dim"]) * big).to(t), "weight": 1 + 0.1 * normal(case["dim"])}
        if case["residual"]:
            x["residual"] = (2 * normal(case["rows"], case["dim"]) * big).to(t)
        return x
    if case["op"] == "rope":
        pos = torch.randint(0, case["far"], (case["tokens"],), generator=g, device="cuda", dtype=torch.int32)
        # q and k are column ranges of one projection's rows
        row = normal(case["tokens"], case["heads"] + 2 * case["kv_heads"], case["width"]).to(t)
        return {"q": row[:, : case["heads"]], "k": row[:, case["heads"] : case["heads"] + case["kv_heads"]], "positions": pos}
    ql, kl = _lengths(case)
    room = [n if case["past_max"] == 0 else -(-n // 256) * 256 for n in kl]  # a cache's sequences have room to grow
    q = normal(sum(ql), case["heads"], case["width"])
    k = normal(sum(room), case["kv_heads"], case["width"]) * (0.5 + torch.rand(case["kv_heads"], case["width"], generator=g, device="cuda"))
    v = normal(sum(room), case["kv_heads"], case["v_width"]) + 0.2 * normal(case["kv_heads"], case["v_width"])
    start = [sum(room[:i]) for i in range(len(room))]
    first = torch.tensor(start, device="cuda")
    k[first] *= 2  # first keys that draw more than their share
    offsets = torch.tensor([sum(ql[:i]) for i in range(len(ql) + 1)], device="cuda", dtype=torch.int32)
    x = {"q": q.to(t), "k": k.to(t), "v": v.to(t), "offsets": offsets}
    if case["past_max"]:
        x["start"] = first.to(torch.int32)
        x["len"] = torch.tensor(kl, device="cuda", dtype=torch.int32)
    return x


def _frequencies(case):
    """The rotary frequencies in 64 bits (radians a position) and the factor on cos and sin."""
    n = case["part"]
    i = torch.arange(0, n, 2, device="cuda", dtype=torch.float64) / n
    if case["scaling"] == "ntk":
        return (10000.0 * YARN["factor"] ** (n / (n - 2))) ** -i, 1.0
    f = 10000.0**-i
    if case["scaling"] == "linear":
        return f / YARN["factor"], 1.0
    if case["scaling"] == "yarn":
        # dimensions that turn 32 times or more in the original length keep their frequency, those that turn
        # less than once are divided by the factor, a ramp between
        def dim(turns):
            return n * math.log(YARN["original"] / (turns * 2 * math.pi)) / (2 * math.log(10000.0))

        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), n - 1)
        ramp = ((torch.arange(n // 2, device="cuda", dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / YARN["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(YARN["factor"]) + 1.0
    return f, 1.0


def prepare(case, seed):
    state = {"case": case, **_tensors(case, seed)}
    if case["op"] == "rope":
        f, mul = _frequencies(case)
        state["frequencies"], state["mul"] = f, mul
        if own:
            from axial_band_split_b200 import mrf

            state["table"] = mrf.rope_table(case["part"], theta=10000.0, scaling=case["scaling"], factor=YARN["factor"], original=YARN["original"])
    if case["op"] == "attention":
        q, k = _lengths(case)
        state["max_q"], state["max_k"] = max(q), max(k)  # a program knows its requests' lengths
    return state


# ----------------------------------------------------------------------------------- plain forms
def _plain_norm(s, case):
    h = s["x"].float()
    if case["residual"]:
        h = h + s["residual"].float()
    mean = h.square().mean(-1, keepdim=True)
    eps = _eps(case)
    y = h * (1 / mean.sqrt().clamp(min=eps) if case["clamp"] else torch.rsqrt(mean + eps)) * s["weight"]
    out = {}
    if case["residual"]:
        out["residual"] = h.to(s["x"].dtype)
    if not case["quant"]:
        return {"out": y.to(s["x"].dtype), **out}
    rows, dim = y.shape
    group = case["group"] or dim
    groups = -(-dim // group)
    blocks = torch.nn.functional.pad(y, (0, groups * group - dim)).view(rows, groups, group)
    scales = blocks.abs().amax(-1) / E4M3_MAX
    codes = (blocks / torch.where(scales > 0, scales, 1.0)[..., None]).view(rows, groups * group)[:, :dim]
    return {"out": codes.to(torch.float8_e4m3fn), "scales": scales, **out}


def _eps(case):
    """1e-6 under the root; or the model's own floor of 1e-12 on the row's 2-norm."""
    return 1e-12 / math.sqrt(case["dim"]) if case["clamp"] else 1e-6


def _rotated(x, cos, sin, case):
    n = case["part"]
    r, rest = x[..., :n], x[..., n:]
    if case["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., : n // 2], r[..., n // 2 :]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def _plain_rope(s, case):
    angle = s["positions"].double()[:, None] * s["frequencies"]  # far positions lose their turns in 32 bits
    cos, sin = ((f(angle) * s["mul"]).float()[:, None] for f in (torch.cos, torch.sin))
    return {n: _rotated(s[n].float(), cos, sin, case).to(s[n].dtype) for n in ("q", "k")}


def _plain_attention(s, case):
    q, k, v, offsets = s["q"], s["k"], s["v"], s["offsets"].long()
    kv, group = case["kv_heads"], case["heads"] // case["kv_heads"]
    n_q = offsets[1:] - offsets[:-1]
    start, n_k = (s["start"].long(), s["len"].long()) if "len" in s else (offsets[:-1], n_q)
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_k"], device="cuda")
    rows_q = (offsets[:-1, None] + i).clamp(max=q.shape[0] - 1)
    rows_k = (start[:, None] + j).clamp(max=k.shape[0] - 1)
    inside = j < n_k[:, None]
    # [sequence, kv head, group x query, width] against [sequence, kv head, width, key]
    a = q[rows_q].float().unflatten(2, (kv, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    b = k[rows_k].float().permute(0, 2, 3, 1)
    scores = (a @ b).unflatten(2, (group, -1)) * (case["width"] ** -0.5)
    seen = inside[:, None, :]
    if case["causal"]:
        seen = seen & (j <= (i[:, None] + (n_k - n_q)[:, None, None]))
    scores = scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    values = torch.where(inside[..., None, None], v[rows_k].float(), 0.0).permute(0, 2, 1, 3)
    o = (p.flatten(2, 3) @ values).unflatten(2, (group, -1)) / torch.where(total > 0, total, 1.0)
    # back to the packed rows
    of = torch.repeat_interleave(torch.arange(case["seqs"], device="cuda"), n_q, output_size=q.shape[0])
    at = torch.arange(q.shape[0], device="cuda") - offsets[of]
    out = {"out": o.permute(0, 3, 1, 2, 4)[of, at].flatten(1, 2).to(q.dtype)}
    if case["lse"]:
        out["lse"] = (top + total.log())[..., 0].permute(0, 3, 1, 2)[of, at].flatten(1, 2)
    return out


# -------------------------------------------------------------------------------- the own calls
def _own_norm(s, case):
    from axial_band_split_b200 import mrf

    r = mrf.rms_norm(s["x"], s["weight"], eps=_eps(case), clamp=case["clamp"], residual=s.get("residual"),
                     out_dtype=torch.float8_e4m3fn if case["quant"] else None, group=case["group"])
    out = {"out": r.out}
    if case["quant"]:
        out["scales"] = r.scales
    if case["residual"]:
        out["residual"] = r.residual
    return out


def _own_rope(s, case):
    from axial_band_split_b200 import mrf

    q, k = mrf.rope(s["q"], s["k"], s["positions"], s["table"], interleaved=case["interleaved"])
    return {"q": q, "k": k}


def _own_attention(s, case):
    from axial_band_split_b200 import mrf

    r = mrf.attention_packed(s["q"], s["k"], s["v"], s["offsets"], k_start=s.get("start"), k_len=s.get("len"), max_k=s["max_k"],
                             causal=case["causal"], return_lse=case["lse"])
    return {"out": r[0], "lse": r[1]} if case["lse"] else {"out": r}


def run(state):
    case = state["case"]
    if own:
        return {"norm": _own_norm, "rope": _own_rope, "attention": _own_attention}[case["op"]](state, case)
    return {"norm": _plain_norm, "rope": _plain_rope, "attention": _plain_attention}[case["op"]](state, case)


# ---------------------------------------------------------------------------------- in 64 bits
def _to_e4m3(v):
    """The nearest values with three bits of fraction and exponents from -6 on, ties to even, in 64 bits."""
    exponent = torch.frexp(v)[1] - 1
    step = torch.exp2((exponent.clamp(min=-6) - 3).double())
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = _tensors(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if case["residual"]:
            h += s["residual"].double()
        power = torch.linalg.vector_norm(h, dim=1) / math.sqrt(case["dim"])
        low = torch.clamp(power, min=_eps(case)) if case["clamp"] else torch.sqrt(power**2 + _eps(case))
        y = h / low[:, None] * s["weight"].double()
        out = {"residual": h} if case["residual"] else {}
        if not case["quant"]:
            return {"out": y, **out}
        scales, codes = [], torch.empty_like(y)
        for c in range(0, case["dim"], case["group"] or case["dim"]):
            part = y[:, c : c + (case["group"] or case["dim"])]
            scale = part.abs().max(dim=1).values / E4M3_MAX
            scales.append(scale)
            codes[:, c : c + part.shape[1]] = _to_e4m3(part / torch.where(scale == 0, 1.0, scale)[:, None])
        return {"out": codes, "scales": torch.stack(scales, 1), **out}
    if case["op"] == "rope":
        f, mul = _frequencies(case)
        n, out = case["part"], {}
        turn = torch.polar(torch.full((), mul, device="cuda", dtype=torch.float64), s["positions"].double()[:, None, None] * f)
        for name in ("q", "k"):
            x = s[name].double()
            y = x.clone()
            if case["interleaved"]:
                z = torch.complex(x[..., 0:n:2], x[..., 1:n:2]) * turn
                y[..., 0:n:2], y[..., 1:n:2] = z.real, z.imag
            else:
                z = torch.complex(x[..., : n // 2], x[..., n // 2 : n]) * turn
                y[..., : n // 2], y[..., n // 2 : n] = z.real, z.imag
            out[name] = y
        return out
    ql, kl = _lengths(case)
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(sum(ql), case["heads"], case["v_width"], device="cuda", dtype=torch.float64)
    lse = torch.full((sum(ql), case["heads"]), -math.inf, device="cuda", dtype=torch.float64)
    at = 0
    for b, (n_q, n_k) in enumerate(zip(ql, kl)):
        first = int(s["start"][b]) if "start" in s else at
        for h in range(case["heads"]):
            key = s["k"][first : first + n_k, h // group].double()
            value = s["v"][first : first + n_k, h // group].double()
            for r in range(0, n_q, 4096):
                e = min(r + 4096, n_q)
                w = s["q"][at + r : at + e, h].double() @ key.T / math.sqrt(case["width"])
                if case["causal"]:
                    w += torch.full_like(w, -math.inf).triu(n_k - n_q + r + 1)
                lse[at + r : at + e, h] = torch.logsumexp(w, -1)
                out[at + r : at + e, h] = torch.softmax(w, -1) @ value
        at += n_q
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
