"""The block operators (norm, rotary positions, packed attention) on the GPU against their formulas in
64 bits, with the bounds that block_ref derives from the roundings."""
import dataclasses
import math

import pytest

import block_ref
from axial_band_split_b200 import mrf

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, F16, BF16, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def within(got, ref, bound, what=""):
    d = (got.double() - ref).abs()
    bad = ~(d <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((d / bound).nan_to_num(9e9).max()):.2f} of the bound"


# ------------------------------------------------------------------------------------------ norm
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 64), (1, 384), (301, 384), (2, 1000), (33, 1536), (7, 2049), (130, 4096),
                                      (3, 8200), (2, 16384), (700, 1000), (601, 4104), (1500, 520), (593, 8192), (640, 1003)])
def test_norm(dtype, rows, dim):
    g = gen(rows * dim)
    x, res = randn(g, rows, dim, dtype=dtype), 3 * randn(g, rows, dim)
    res = res.to(dtype)
    w = 1 + 0.1 * randn(g, dim)
    for weight, residual, clamp in ((None, None, False), (w, res, False), (w.to(BF16), None, True), (w.to(F16), res, True)):
        eps = 1e-12 / math.sqrt(dim) if clamp else 1e-5
        r = mrf.rms_norm(x, weight, eps, residual, clamp=clamp)
        y, h = block_ref.rms_norm(x, weight, eps, residual, clamp)
        assert r.scales is None and r.out.dtype == dtype and (r.residual is None) == (residual is None)
        within(r.out, y, y.abs() * (block_ref.norm_slack(dim) + block_ref.half_step(dtype)) + 2.0**-25, "out")
        if residual is not None:
            within(r.residual, h, h.abs() * (block_ref.U32 + block_ref.half_step(dtype)) * 1.001 + 2.0**-25, "h")


def check_quant(r, y, group, dim):
    """The scale is max |y| / 448; a code is off its y by half a step of e4m3 (2^-4, or 2^-10 below the
    normal range), in units of the scale; y and the scale carry the norm's fp32 roundings."""
    size = group or dim
    slack = block_ref.norm_slack(dim) + 4 * block_ref.U32
    for c in range(0, dim, size):
        part, scale = y[:, c : c + size], r.scales[:, c // size].double()[:, None]
        top = part.abs().amax(-1, keepdim=True) / 448
        within(scale, top, top * slack, "scales")
        v = (part / torch.where(top > 0, top, 1.0)).abs()
        bound = torch.clamp(v * (2.0**-4 + 2 * slack), min=2.0**-10) * top
        within(r.out[:, c : c + size].float().double() * scale, part, bound + slack * part.abs(), "codes")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,dim,group", [(1, 4096, 0), (9, 384, 128), (5, 1000, 64), (3, 77, 32), (2, 130, 128), (65, 2048, 32),
                                            (4, 8192, 128), (2, 16384, 0), (17, 64, 0), (650, 1000, 64), (600, 2048, 0), (1201, 640, 32),
                                            (600, 8192, 128), (700, 1003, 128), (2500, 192, 64)])
def test_norm_e4m3(dtype, rows, dim, group):
    g = gen(dim + group)
    x, res = randn(g, rows, dim, dtype=dtype), randn(g, rows, dim, dtype=dtype)
    w = 1 + 0.5 * randn(g, dim)
    r = mrf.rms_norm(x, w, 1e-6, res, out_dtype=E4M3, group=group)
    y, h = block_ref.rms_norm(x, w, 1e-6, res)
    check_quant(r, y, group, dim)
    within(r.residual, h, h.abs() * (block_ref.U32 + block_ref.half_step(dtype)) * 1.001 + 2.0**-25, "h")


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("rows,dim", [(700, 131), (613, 2047), (600, 2049), (20, 4097)])
def test_norm_of_odd_widths(dtype, rows, dim):
    """A warp and a block a row, whole batches of values and their ends, every kind of scale and of weight."""
    g = gen(rows + dim)
    x, res, w = randn(g, rows, dim, dtype=dtype), randn(g, rows, dim, dtype=dtype), 1 + 0.5 * randn(g, dim)
    for group, residual, weight in ((0, res, w), (32, None, w.to(F16)), (64, res, None), (128, res, w.to(BF16))):
        r = mrf.rms_norm(x, weight, 1e-6, residual, out_dtype=E4M3, group=group)
        y, h = block_ref.rms_norm(x, weight, 1e-6, residual)
        check_quant(r, y, group, dim)
        r = mrf.rms_norm(x, weight, 1e-6, residual)
        within(r.out, y, y.abs() * (block_ref.norm_slack(dim) + block_ref.half_step(dtype)) + 2.0**-25, "out")
        if residual is not None:
            within(r.residual, h, h.abs() * (block_ref.U32 + block_ref.half_step(dtype)) * 1.001 + 2.0**-25, "h")
            again = mrf.rms_norm(x.clone(), weight, 1e-6, residual, residual_out=residual.clone())
            assert torch.equal(again.out, r.out) and torch.equal(again.residual, r.residual)


def test_norm_zero_nan_and_infinity():
    x = torch.zeros(4, 256, device="cuda", dtype=BF16)
    x[1, 5] = math.nan
    x[2, 7] = math.inf
    x[3] = 1
    r = mrf.rms_norm(x, None, 1e-6, out_dtype=E4M3, group=64)
    assert torch.equal(r.out[0].float(), torch.zeros(256, device="cuda")) and torch.equal(r.scales[0], torch.zeros(4, device="cuda"))
    assert r.scales[1].isnan().all() and r.out[1].float().isnan().all()
    assert r.scales[2, 0].isnan() and r.out[2, :64].float().isnan().all()
    assert torch.equal(r.out[3].float(), torch.full((256,), 448.0, device="cuda"))
    many = torch.cat((x.repeat(1, 3), torch.full((4, 768), 2.0**-100, device="cuda", dtype=BF16)) * 100)  # rows enough for the streaming kernel
    q = mrf.rms_norm(many, None, 1e-6, out_dtype=E4M3, group=64)
    assert not q.out[0].float().any() and not q.scales[0].any() and q.out[1].float().isnan().all() and q.scales[2, 0].isnan()
    assert not q.out[2, 64:256].float().any() and torch.equal(q.out[3].float(), torch.full((768,), 448.0, device="cuda"))
    # 2^-100 / sqrt(1e-6): a scale of 1000 * 2^-100 / 448 and full codes
    assert torch.equal(q.out[4].float(), torch.full((768,), 448.0, device="cuda"))
    within(q.scales[4], torch.full((12,), 1000 * 2.0**-100 / 448, device="cuda", dtype=torch.float64), torch.tensor(1000 * 2.0**-100 / 448 * 2.0**-18, device="cuda"))
    y = mrf.rms_norm(x, None, 1e-6).out
    assert torch.equal(y[0].float(), torch.zeros(256, device="cuda")) and y[1].isnan().all() and y[2, 7].isnan()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_strides_in_place_and_leading_dims(dtype):
    g = gen(5)
    wide = randn(g, 40, 1111, dtype=dtype)
    for x in (wide[:, :640], wide[:, 3:643], wide[::2, 1:641], wide[:1, :640].expand(40, 640)):
        y, _ = block_ref.rms_norm(x, None, 1e-6)
        tol = y.abs() * (block_ref.norm_slack(640) + block_ref.half_step(dtype)) + 2.0**-25
        within(mrf.rms_norm(x).out, y, tol)
        out = torch.zeros(x.shape[0], 700, device="cuda", dtype=dtype)
        mrf.rms_norm(x, out=out[:, 5:645])
        within(out[:, 5:645], y, tol)
        assert not out[:, :5].any() and not out[:, 645:].any()
    x, res = randn(g, 6, 5, 128, dtype=dtype), randn(g, 6, 5, 128, dtype=dtype)
    want = mrf.rms_norm(x, residual=res)
    assert want.out.shape == x.shape
    h, same = res.clone(), x.clone()
    got = mrf.rms_norm(same, residual=h, residual_out=h, out=same)
    assert got.out.data_ptr() == same.data_ptr() and got.residual.data_ptr() == h.data_ptr()
    assert torch.equal(same, want.out) and torch.equal(h, want.residual)
    assert mrf.rms_norm(x[:0]).out.shape == (0, 5, 128)
    q = mrf.rms_norm(x[:0], out_dtype=E4M3, group=32)
    assert q.scales.shape == (0, 5, 4)


# ------------------------------------------------------------------------------------------ rope
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("tokens,heads,kv,width,part", [(1, 1, 1, 64, 64), (37, 8, 2, 64, 32), (5, 3, 1, 80, 20), (130, 7, 1, 128, 128),
                                                        (3, 2, 2, 33, 6), (9, 4, 0, 96, 96), (2, 1, 1, 256, 128), (65, 32, 8, 128, 128)])
def test_rope(dtype, interleaved, tokens, heads, kv, width, part):
    g = gen(tokens * width)
    q = randn(g, tokens, heads, width, dtype=dtype)
    k = randn(g, tokens, kv, width, dtype=dtype) if kv else None
    pos = torch.randint(-5, 1 << 20, (tokens,), generator=g, device="cuda", dtype=torch.int64)
    table = mrf.rope_table(part, 10000.0, "yarn", 32.0, 4096)
    f, mul = block_ref.rope_frequencies(part, 10000.0, "yarn", 32.0, 4096)
    for positions in (pos, pos.int()):
        got = mrf.rope(q, k, positions, table, interleaved)
        assert (got[1] is None) == (k is None)
        for x, y in zip((q, k), got):
            if x is not None:
                ref, size = block_ref.rope(x, positions, f, mul, interleaved)
                within(y, ref, block_ref.rope_slack(size) + block_ref.half_step(dtype) * ref.abs() * 1.01 + (size > 0) * 2.0**-25)


def test_rope_far_positions_wide():
    g = gen(8)
    q = randn(g, 6, 2, 64)
    pos = torch.tensor([0, 1, (1 << 31) - 1, 1 << 31, 1 << 36, -(1 << 33)], device="cuda")
    f, mul = block_ref.rope_frequencies(64)
    # the table's fraction of a turn against exact whole-number arithmetic: no error grows with the position
    turns = mrf.rope_table(64, device="cpu").turns.numpy().view("uint64")
    angle = torch.tensor([[(int(p) * int(t) % 2**64) / 2.0**64 * 2 * math.pi for t in turns] for p in pos.tolist()], device="cuda", dtype=torch.float64)
    a, b = q[..., 0::2].double(), q[..., 1::2].double()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    got, _ = mrf.rope(q, None, pos, mrf.rope_table(64))
    size = block_ref.rope_slack(a.abs() + b.abs())
    within(got[..., 0::2], a * c - b * s, size)
    within(got[..., 1::2], b * c + a * s, size)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("width,part", [(80, 40), (96, 24), (32, 8), (28, 8), (44, 40), (6, 4), (18, 12), (48, 16), (24, 16)])
def test_rope_pieces(dtype, interleaved, width, part):
    """Parts whose half is a multiple of 8, 4, 2 or 1, an odd number of pieces that do not turn, and rows that start off 16 bytes."""
    g = gen(width + part)
    pos = torch.arange(700, device="cuda", dtype=torch.int32)
    table = mrf.rope_table(part)
    f, mul = block_ref.rope_frequencies(part)
    for lead in (0, 1, 2, 4):
        row = randn(g, 700, lead + 5 * width + (-(lead + 5 * width)) % 8, dtype=dtype)
        view = row[:, lead : lead + 5 * width].unflatten(1, (5, width))
        for x, y in zip((view[:, :4], view[:, 4:]), mrf.rope(view[:, :4], view[:, 4:], pos, table, interleaved)):
            ref, size = block_ref.rope(x, pos, f, mul, interleaved)
            within(y, ref, block_ref.rope_slack(size) + block_ref.half_step(dtype) * ref.abs() * 1.01 + (size > 0) * 2.0**-25)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_in_place_in_projection_rows(dtype, interleaved):
    """q and k as column ranges of one projection's rows, aligned or not, turned in place: v and the rest stay."""
    g = gen(9)
    for width, part, lead in ((64, 64, 0), (64, 32, 3), (20, 10, 1)):
        row = randn(g, 50, lead + (4 + 2 + 2) * width, dtype=dtype)
        before = row.clone()
        view = row[:, lead:].unflatten(1, (8, width))
        q, k = view[:, :4], view[:, 4:6]
        pos = torch.arange(50, device="cuda", dtype=torch.int32)
        table = mrf.rope_table(part)
        want = mrf.rope(q, k, pos, table, interleaved)
        got = mrf.rope(q, k, pos, table, interleaved, q_out=q, k_out=k)
        assert got[0].data_ptr() == q.data_ptr() and torch.equal(q, want[0]) and torch.equal(k, want[1])
        assert torch.equal(row[:, :lead], before[:, :lead]) and torch.equal(row[:, lead + 6 * width :], before[:, lead + 6 * width :])
        back = mrf.rope(q, k, -pos, table, interleaved)  # the inverse
        f, mul = block_ref.rope_frequencies(part)
        ref, size = block_ref.rope(q, -pos, f, mul, interleaved)
        within(back[0], ref, block_ref.rope_slack(size) + block_ref.half_step(dtype) * ref.abs() * 1.01 + 2.0**-25)
    heads_first = randn(g, 4, 50, 64, dtype=dtype).transpose(0, 1)
    got, _ = mrf.rope(heads_first, None, pos, mrf.rope_table(64), interleaved)
    want, _ = mrf.rope(heads_first.contiguous(), None, pos, mrf.rope_table(64), interleaved)
    assert torch.equal(got, want)


# ------------------------------------------------------------------------------------- attention
@dataclasses.dataclass
class Shape:
    spans: list  # (queries, keys) of each sequence; keys None: a whole prompt
    heads: int = 4
    kv: int = 2
    width: int = 64
    v_width: int = 64
    dtype: torch.dtype = BF16
    causal: bool = True
    max_k: int = 0
    junk: float = math.nan  # what the rows of no sequence hold
    gap: int = 3


def make(s, seed=0):
    """q, k, v, offsets, start, length and the oracle's spans; a cache has gaps of junk between the sequences."""
    g = gen(seed)
    nq = sum(n for n, _ in s.spans)
    q = randn(g, nq + 2, s.heads, s.width, dtype=s.dtype)  # two rows behind the last sequence
    off = [0]
    for n, _ in s.spans:
        off.append(off[-1] + n)
    offsets = torch.tensor(off, device="cuda", dtype=torch.int32)
    if s.spans[0][1] is None:
        spans = [(off[i], n, off[i], n) for i, (n, _) in enumerate(s.spans)]
        rows, start, length = nq + 2, None, None
    else:
        at, spans = s.gap, []
        for i, (n, m) in enumerate(s.spans):
            spans.append((off[i], n, at, m))
            at += m + s.gap
        rows = at
        start = torch.tensor([p[2] for p in spans], device="cuda", dtype=torch.int32)
        length = torch.tensor([p[3] for p in spans], device="cuda", dtype=torch.int32)
    k = torch.full((rows, s.kv, s.width), s.junk, device="cuda", dtype=s.dtype)
    v = torch.full((rows, s.kv, s.v_width), s.junk, device="cuda", dtype=s.dtype)
    for _, _, k0, m in spans:
        k[k0 : k0 + m] = randn(g, m, s.kv, s.width, dtype=s.dtype)
        v[k0 : k0 + m] = randn(g, m, s.kv, s.v_width, dtype=s.dtype)
    return q, k, v, offsets, start, length, spans


def check_attention(s, q, k, v, spans, out, lse, scale):
    ref, rlse, size, big = block_ref.attention(q, k, v, spans, s.causal, scale)
    keys = max([m for _, _, _, m in spans] + [1])
    bound, lbound = block_ref.attention_slack(s.dtype, ref, size, big, keys, s.width)
    n = sum(p[1] for p in spans)
    within(out[:n], ref[:n], bound[:n] + 2.0**-25, "out")
    empty = rlse[:n] == -math.inf
    assert torch.equal(lse[:n][empty], rlse[:n][empty].float()) and not out[:n][empty].any()
    within(torch.where(empty, 0, lse[:n]), torch.where(empty, 0, rlse[:n]), lbound[:n], "lse")


def run(s, seed=0, **more):
    q, k, v, offsets, start, length, spans = make(s, seed)
    n = sum(p[1] for p in spans)
    out = torch.full((q.shape[0], s.heads, s.v_width), 7.0, device="cuda", dtype=s.dtype)
    scale = s.width**-0.5
    o, lse = mrf.attention_packed(q, k, v, offsets, start, length, s.max_k, s.causal, out=out, return_lse=True, **more)
    assert o.data_ptr() == out.data_ptr()
    mrf.ops_sync_status()
    check_attention(s, q, k, v, spans, out, lse, scale)
    assert (out[n:] == 7).all()  # rows behind the last sequence
    again = mrf.attention_packed(q, k, v, offsets, start, length, s.max_k, s.causal, scale=scale)
    assert torch.equal(again[:n], out[:n])  # the same bits on every run


PROMPTS = [[(1, None)], [(5, None)], [(128, None)], [(129, None), (1, None)], [(17, None), (0, None), (300, None), (64, None)],
           [(0, None), (257, None), (0, None), (0, None), (640, None), (0, None)], [(33, None)] * 9]
CACHES = [[(1, 1)], [(1, 128)], [(1, 1000), (1, 0), (1, 129)], [(1, 5000)], [(3, 300), (130, 131), (0, 50), (64, 2000)],
          [(200, 150), (4, 0), (300, 1)], [(1, m) for m in range(1, 200, 7)], [(128, 128), (16, 17), (127, 255)]]


@pytest.mark.parametrize("spans", PROMPTS + CACHES, ids=lambda v: "-".join(f"{a}.{b}" for a, b in v)[:40])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_lengths(spans, dtype, causal):
    run(Shape(spans, dtype=dtype, causal=causal))
    run(Shape(spans, heads=8, kv=1, width=128, v_width=128, dtype=dtype, causal=causal, max_k=max(m or n for n, m in spans)))


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (6, 2), (5, 5), (14, 2), (7, 1), (32, 8), (12, 1), (40, 1), (128, 1), (130, 1), (200, 2)])
@pytest.mark.parametrize("width,v_width", [(64, 64), (128, 128)])
def test_attention_grouped_heads(heads, kv, width, v_width):
    run(Shape([(70, None), (1, None), (200, None)], heads, kv, width, v_width))
    run(Shape([(1, 300), (2, 17), (9, 700)], heads, kv, width, v_width, F16))


@pytest.mark.parametrize("width,v_width", [(128, 64), (64, 128), (96, 96), (80, 80), (8, 8), (16, 64), (40, 104), (72, 64), (33, 20),
                                           (1, 1), (160, 160), (256, 256), (192, 128)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_widths(width, v_width, dtype):
    run(Shape([(150, None), (37, None)], 4, 2, width, v_width, dtype))
    run(Shape([(1, 450), (20, 33)], 4, 2, width, v_width, dtype, causal=False))


@pytest.mark.parametrize("causal", [True, False])
def test_attention_fp32(causal):
    run(Shape([(150, None), (1, None), (0, None)], 4, 2, 64, 64, F32, causal))
    run(Shape([(1, 450), (20, 13)], 6, 2, 80, 96, F32, causal))


@pytest.mark.parametrize("dtype,width,v_width", [(F32, 64, 64), (F32, 128, 128), (F32, 256, 256), (F32, 65, 67), (F16, 36, 36), (BF16, 250, 9)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_of_other_types_and_widths(dtype, width, v_width, causal):
    """fp32, odd and wide heads: every size of tile, split keys, ends inside a step, heads that fill several tiles."""
    run(Shape([(1, None), (63, None), (64, None), (65, None), (300, None)], 2, 2, width, v_width, dtype, causal))
    run(Shape([(1, 64), (1, 65), (3, 1000), (0, 9), (2, 0), (1, 4001)], 8, 2, width, v_width, dtype, causal, max_k=4001))
    run(Shape([(1, 9000)], 8, 1, width, v_width, dtype, causal))
    run(Shape([(40, 3000)], 4, 2, width, v_width, dtype, causal))
    run(Shape([(1, 100), (3, 5)], 300, 2, width, v_width, dtype, causal))


def test_attention_of_other_types_in_many_sequences():
    """Empty sequences between others, and a key bound that is too low for the ranges that it sizes."""
    run(Shape([(n % 5, None) for n in range(333)], 4, 2, dtype=F32))
    run(Shape([(0, 5)] * 40 + [(130, 2000)] + [(0, 0)] * 40 + [(1, 4097)], 2, 1, 128, 128, F32, max_k=4097))
    run(Shape([(1, 6000), (1, 100), (2, 1025)], 8, 1, 128, 128, F32, max_k=1024))
    run(Shape([(1, 6000)], 8, 1, 100, 36, BF16, max_k=1024))


def test_attention_of_other_types_and_strides():
    """Heads that start off 16 bytes, and rows of no sequence that hold NaN."""
    for width, off in ((64, 1), (64, 4), (30, 2)):
        s = Shape([(70, None), (1, None)], 4, 2, width, width, F32)
        q, k, v, offsets, _, _, spans = make(s, 5)
        wide = torch.full((q.shape[0], 8 * (width + off) + off), math.nan, device="cuda")
        parts = wide[:, off:].unflatten(1, (8, width + off))[..., :width]
        parts[:, :4], parts[:, 4:6], parts[:, 6:] = q, k[: q.shape[0]], v[: q.shape[0]]
        n = sum(p[1] for p in spans)
        parts[n:] = math.nan
        out, lse = mrf.attention_packed(parts[:, :4], parts[:, 4:6], parts[:, 6:], offsets, return_lse=True)
        check_attention(s, q, k, v, spans, out, lse, width**-0.5)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_long(causal):
    run(Shape([(2100, None), (1300, None)], 2, 1, 128, 128, BF16, causal))
    run(Shape([(1500, 4000)], 4, 4, 64, 64, F16, causal))
    run(Shape([(1, 70001), (2, 9000)], 8, 1, 128, 128, BF16, causal, max_k=70001))
    run(Shape([(1, 70001)], 2, 2, 64, 64, F16, causal))


def test_attention_cold_inputs_give_the_same_bits():
    """The first call on inputs that no cache holds yet (slow loads, units that run apart) against the calls after it."""
    for i in range(6):
        for s in (Shape([(1, 7000)] * 32, 32, 8, 128, 128, max_k=7000), Shape([(1, 30000), (2, 9000)], 8, 1, 128, 128, max_k=30000),
                  Shape([(1, 5000)] * 40 + [(1, 10)] * 40, 6, 3, 64, 64, max_k=5000)):
            q, k, v, offsets, start, length, spans = make(s, 100 + i)
            torch.cuda.synchronize()
            outs = [mrf.attention_packed(q, k, v, offsets, start, length, s.max_k) for _ in range(4)]
            n = sum(p[1] for p in spans)
            assert all(torch.equal(o[:n], outs[-1][:n]) for o in outs[:-1])


def test_attention_many_sequences():
    """More sequences than the 32 that are looked at together, empty ones among them, and a key bound that is too low."""
    run(Shape([(n % 5, None) for n in range(333)], 4, 2))
    run(Shape([(n % 3, 7 * n % 400) for n in range(150)], 8, 2, 128, 128, F16, causal=False))
    run(Shape([(1, 13 * n % 3000) for n in range(70)], 4, 4, 64, 64, BF16, max_k=3000))
    run(Shape([(0, 5)] * 40 + [(130, 2000)] + [(0, 0)] * 40 + [(1, 4097)], 2, 1, 128, 128, max_k=4097))
    run(Shape([(1, 6000), (1, 100), (2, 1025)], 8, 1, 128, 128, max_k=1024))
    run(Shape([(1, 6000)], 8, 1, 64, 64, max_k=1024))


def test_attention_from_two_threads():
    """Calls of two threads on their own streams do not disturb one another."""
    import threading
    cases = [make(Shape([(1, 9000 + 77 * i), (1, 50)], 8, 1, 128, 128), 40 + i) for i in range(2)]
    want = [mrf.attention_packed(*c[:6], 9100) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        for _ in range(30):
            got = mrf.attention_packed(*cases[i][:6], 9100, stream=stream)
            stream.synchronize()
            bad.append(not torch.equal(got[:2], want[i][:2]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(bad) == 60 and not any(bad)


def test_attention_large_scores_and_peaks():
    """Scores of hundreds (running maxima that jump between key blocks) and one key that takes all the weight."""
    for width in (64, 128):
        s = Shape([(300, None), (90, None)], 4, 2, width, width, F16)
        q, k, v, offsets, _, _, spans = make(s, 3)
        k[:390] *= torch.linspace(0.1, 8, 390, device="cuda")[:, None, None].to(F16)
        q *= 6
        out, lse = mrf.attention_packed(q, k, v, offsets, return_lse=True)
        check_attention(s, q, k, v, spans, out, lse, width**-0.5)


def test_attention_masked_keys_may_be_anything():
    """Infinities and NaN in keys that causality hides do not reach the rows that do not see them."""
    for value in (math.inf, -math.inf, math.nan):
        for width in (64, 128):
            s = Shape([(200, None), (60, None)], 4, 2, width, width)
            q, k, v, offsets, _, _, spans = make(s, 4)
            want = mrf.attention_packed(q, k, v, offsets)
            k[150] = value
            got = mrf.attention_packed(q, k, v, offsets)
            assert torch.equal(got[:150], want[:150]) and torch.equal(got[200:260], want[200:260])


def test_attention_strides():
    """q, k and v as column ranges of projection rows, head-major caches, misaligned rows, an output inside wider rows."""
    s = Shape([(100, None), (31, None)], 4, 2, 64, 64)
    q, k, v, offsets, _, _, spans = make(s, 5)
    want = mrf.attention_packed(q, k, v, offsets)
    n = 131
    for lead in (0, 8, 3):
        row = torch.zeros(q.shape[0], lead + 8 * 64 + 5 * 8, device="cuda", dtype=BF16)
        view = row[:, lead : lead + 512].unflatten(1, (8, 64))
        view[:, :4], view[:, 4:6], view[:, 6:] = q, k, v
        wide = torch.full((q.shape[0], 4, 80), 7.0, device="cuda", dtype=BF16)
        got = mrf.attention_packed(view[:, :4], view[:, 4:6], view[:, 6:], offsets, out=wide[..., 8:72])
        ref, rlse, size, big = block_ref.attention(q, k, v, spans, True, 0.125)
        bound, _ = block_ref.attention_slack(BF16, ref, size, big, 100, 64)
        within(got[:n], ref[:n], bound[:n] + 2.0**-25)
        assert (wide[..., :8] == 7).all() and (wide[..., 72:] == 7).all()
    hk, hv = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (k, v))
    assert torch.equal(mrf.attention_packed(q, hk, hv, offsets)[:n], want[:n])
    one = mrf.attention_packed(q, k[:, :1].expand(-1, 2, -1), v[:, :1].expand(-1, 2, -1), offsets)  # a broadcast head
    ref, rlse, size, big = block_ref.attention(q, k[:, :1], v[:, :1], spans, True, 0.125)
    bound, _ = block_ref.attention_slack(BF16, ref, size, big, 100, 64)
    within(one[:n], ref[:n], bound[:n] + 2.0**-25)


def test_attention_offsets_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements: the sequences at its far end."""
    rows, kv, width = (1 << 31) // (8 * 128) + 5000, 8, 128
    k = torch.empty(rows, kv, width, device="cuda", dtype=F16)
    v = torch.empty(rows, kv, width, device="cuda", dtype=F16)
    g = gen(6)
    spans = [(0, 1, rows - 700, 700), (1, 40, rows - 2000, 333)]
    for _, _, k0, m in spans:
        k[k0 : k0 + m] = randn(g, m, kv, width, dtype=F16)
        v[k0 : k0 + m] = randn(g, m, kv, width, dtype=F16)
    q = randn(g, 41, 16, width, dtype=F16)
    offsets, start, length = (torch.tensor(t, device="cuda", dtype=torch.int32) for t in ([0, 1, 41], [rows - 700, rows - 2000], [700, 333]))
    out, lse = mrf.attention_packed(q, k, v, offsets, start, length, 700, return_lse=True)
    check_attention(Shape([], 16, 8, 128, 128, F16), q, k, v, spans, out, lse, width**-0.5)


def test_attention_wrong_offsets_stay_inside():
    """Offsets beyond the tensors are held to their rows: the call ends, and rows outside the spans are not written."""
    s = Shape([(40, None)], 4, 2, 64, 64, junk=0.0)
    q, k, v, _, _, _, _ = make(s, 7)
    i32 = lambda *t: torch.tensor(t, device="cuda", dtype=torch.int32)
    for offsets, start, length in ((i32(0, 1000), None, None), (i32(-5, 20), None, None), (i32(0, 42), i32(-9), i32(1 << 30)),
                                   (i32(0, 42), i32(1 << 30), i32(5)), (i32(0, 42), i32(3), i32(-4)), (i32(10, 5), None, None),
                                   (i32(2**31 - 1, 2**31 - 1), None, None), (i32(30, 10, 42), None, None)):
        for width in (64, 128):
            qq, kk, vv = (t if width == 64 else torch.cat((t, t), -1) for t in (q, k, v))
            mrf.attention_packed(qq, kk, vv, offsets, start, length)
            mrf.ops_sync_status()


def test_attention_empty_calls():
    q = torch.zeros(5, 4, 64, device="cuda", dtype=F16)
    none = torch.zeros(0, 2, 64, device="cuda", dtype=F16)
    i32 = lambda *t: torch.tensor(t, device="cuda", dtype=torch.int32)
    out, lse = mrf.attention_packed(q, none, none, i32(0, 5), i32(0), i32(0), return_lse=True)
    assert not out.any() and (lse == -math.inf).all()
    assert mrf.attention_packed(q[:0], none, none, i32(0, 0), i32(0), i32(0)).shape == (0, 4, 64)
    assert mrf.attention_packed(q, none, none, i32(0), i32(), i32()).shape == (5, 4, 64)


# ------------------------------------------------------------------- streams, graphs, the whole run
def test_refusals_of_the_binding():
    x = torch.zeros(4, 2, 64, device="cuda", dtype=F16)
    i32 = lambda *t: torch.tensor(t, device="cuda", dtype=torch.int32)
    off, table = i32(0, 4), mrf.rope_table(64)
    bad = [lambda: mrf.rms_norm(x.double()), lambda: mrf.rms_norm(x, out_dtype=F32), lambda: mrf.rms_norm(x, weight=torch.ones(65, device="cuda")),
           lambda: mrf.rms_norm(x, residual=x.float()), lambda: mrf.rms_norm(x, residual=x[:2]), lambda: mrf.rms_norm(x, group=32),
           lambda: mrf.rms_norm(x, residual_out=x), lambda: mrf.rms_norm(x[..., ::2]), lambda: mrf.rms_norm(x.transpose(0, 1)),
           lambda: mrf.rms_norm(x.requires_grad_()), lambda: mrf.rms_norm(x.detach(), out=x.detach().cpu()),
           lambda: mrf.rope(x.detach(), None, i32(1, 2, 3), table), lambda: mrf.rope(x.detach(), None, i32(1, 2, 3, 4).float(), table),
           lambda: mrf.rope(x.detach(), None, i32(1, 2, 3, 4), mrf.rope_table(66)), lambda: mrf.rope(x.detach(), None, i32(1, 2, 3, 4), table.turns),
           lambda: mrf.rope(x.detach(), None, i32(1, 2, 3, 4), mrf.rope_table(64, device="cpu")),
           lambda: mrf.attention_packed(x.detach(), x.detach().float(), x.detach(), off), lambda: mrf.attention_packed(x.detach(), x.detach(), x.detach(), off.long()),
           lambda: mrf.attention_packed(x.detach(), x.detach(), x.detach(), off, k_start=off), lambda: mrf.attention_packed(x.detach(), x.detach(), x.detach(), off, off, off),
           lambda: mrf.attention_packed(x.detach(), x.detach()[:, :, ::2], x.detach(), off), lambda: mrf.attention_packed(x.detach(), x.detach(), x.detach(), off, scale=0.0),
           lambda: mrf.attention_packed(x.detach(), x.detach(), x.detach(), off, out=x.detach()), lambda: mrf.attention_packed(x.detach(), x.detach(), x.detach(), off.cpu())]
    for i, call in enumerate(bad):
        with pytest.raises(mrf.MrfError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_windows_over_one_signal():
    """Inputs whose rows overlap (token and head strides below the width) give new outputs of their own layout."""
    signal = randn(gen(8), 64 * 9, dtype=F16)
    for strides in ((1, 2, 1), (8, 16, 1), (0, 0, 1), (2, 1, 1)):
        x = signal.as_strided((20, 2, 64), strides)
        dense = x.clone(memory_format=torch.contiguous_format)
        off, pos = torch.tensor([0, 20], device="cuda", dtype=torch.int32), torch.arange(20, device="cuda")
        table = mrf.rope_table(64)
        assert all(torch.equal(a, b) for a, b in zip(mrf.rope(x, x, pos, table), mrf.rope(dense, dense, pos, table)))
        got, want = mrf.attention_packed(x, x, x, off), mrf.attention_packed(dense, dense, dense, off)
        # (strides that are no multiples of 8 go to the CUDA cores, without the probabilities' rounding to fp16 and with
        # sums in another order: each side is within half a step of its weights and of the output)
        assert (got.float() - want.float()).abs().max() <= 4 * 2.0**-11 * dense.float().abs().max()
        got, want = mrf.rms_norm(x[:, 0]).out.float(), mrf.rms_norm(dense[:, 0]).out.float()
        assert ((got - want).abs() <= 2 * 2.0**-11 * want.abs() + 2.0**-24).all()  # (the sums' order may move a rounding)


def test_refusals_of_what_is_no_tensor():
    x = torch.zeros(4, 2, 64, device="cuda", dtype=F16)
    off, table = torch.tensor([0, 4], device="cuda", dtype=torch.int32), mrf.rope_table(64)
    for call in (lambda: mrf.attention_packed(x, x, None, off), lambda: mrf.attention_packed(x, None, x, off), lambda: mrf.attention_packed(None, x, x, off),
                 lambda: mrf.attention_packed(x, x, x, [0, 4]), lambda: mrf.rope(x, 3, off, table), lambda: mrf.rms_norm([1.0]),
                 lambda: mrf.rms_norm(x, residual=1.0)):
        with pytest.raises(mrf.MrfError):
            call()


def test_other_streams():
    """Calls on side streams, given as torch streams, raw pointers or the current one, at the same time."""
    s = Shape([(200, None), (300, None)], 8, 2, 128, 128)
    q, k, v, offsets, _, _, _ = make(s, 8)
    want = mrf.attention_packed(q, k, v, offsets)
    long = make(Shape([(1, 40000)], 8, 1, 128, 128), 9)
    want_long = mrf.attention_packed(*long[:6], 40000)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append((mrf.attention_packed(q, k, v, offsets, stream=a), want))
        got.append((mrf.attention_packed(*long[:6], 40000, stream=b.cuda_stream), want_long))
        with torch.cuda.stream(a):
            got.append((mrf.attention_packed(*long[:6], 40000), want_long))
    torch.cuda.synchronize()
    for i, (x, y) in enumerate(got):
        n = 500 if y is want else 1
        assert torch.equal(x[:n], y[:n]), i


def test_graph_replay_with_new_lengths():
    """A captured token step replayed after the cache grew; two graphs captured in a row keep their own workspaces."""
    g = gen(10)
    seqs, heads, kv, width, room = 3, 8, 2, 128, 6000
    k, v = randn(g, seqs * room, kv, width, dtype=BF16), randn(g, seqs * room, kv, width, dtype=BF16)
    q = randn(g, seqs, heads, width, dtype=BF16)
    offsets = torch.arange(seqs + 1, device="cuda", dtype=torch.int32)
    start = torch.arange(seqs, device="cuda", dtype=torch.int32) * room
    length = torch.tensor([10, 4000, 300], device="cuda", dtype=torch.int32)
    step = lambda: mrf.attention_packed(q, k, v, offsets, start, length, room)
    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step()
        graphs.append((gr, out))
    for lens in ([10, 4000, 300], [11, 4001, 301], [6000, 1, 0], [0, 5999, 129]):
        length.copy_(torch.tensor(lens, dtype=torch.int32))
        want = step().clone()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        for (gr, _), st in zip(graphs, (s1, s2)):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][1], want) and torch.equal(graphs[1][1], want)
        ref = block_ref.attention(q, k, v, [(i, 1, i * room, n) for i, n in enumerate(lens)], True, width**-0.5)
        bound, _ = block_ref.attention_slack(BF16, ref[0], ref[2], ref[3], room, width)
        within(want, ref[0], bound + 2.0**-25)


def block(p, x, h, positions, table, offsets, cache=None):
    """One block of a causal transformer over packed rows: norm, projection, rotary positions, attention,
    projection, the residual's norm, an 8-bit copy for the next product.  cache: (k, v, start, length, slots)."""
    n = mrf.rms_norm(x, p["g1"], residual=h)
    qkv = (n.out @ p["wqkv"]).unflatten(1, (8, 64))
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    mrf.rope(q, k, positions, table, q_out=q, k_out=k)
    if cache is None:
        o = mrf.attention_packed(q, k, v, offsets)
    else:
        ck, cv, start, length, slots = cache
        ck[slots], cv[slots] = k, v
        o = mrf.attention_packed(q, ck, cv, offsets, start, length)
    return mrf.rms_norm(o.flatten(1) @ p["wo"], p["g2"], residual=n.residual, out_dtype=E4M3, group=64)


def test_a_block_as_it_is_used():
    """A packed prompt at once, the same in pieces over a cache, then token by token, and all against 64 bits."""
    g = gen(11)
    dim, lens = 192, [70, 1, 133]
    p = {"g1": 1 + 0.1 * randn(g, dim), "g2": 1 + 0.1 * randn(g, dim), "wqkv": (randn(g, dim, 512) / dim**0.5).to(F16), "wo": (randn(g, 256, dim) / 16).to(F16)}
    x, h = randn(g, sum(lens), dim, dtype=F16), randn(g, sum(lens), dim, dtype=F16)
    table = mrf.rope_table(64)
    i32 = lambda t: torch.tensor(t, device="cuda", dtype=torch.int32)
    offsets = i32([0, 70, 71, 204])
    positions = torch.cat([torch.arange(n, device="cuda") for n in lens]).int()
    whole = block(p, x, h, positions, table, offsets)
    # 64 bits
    n, h2 = block_ref.rms_norm(x, p["g1"], 1e-6, h)
    qkv = (n @ p["wqkv"].double()).unflatten(1, (8, 64))
    f, mul = block_ref.rope_frequencies(64)
    q, k = (block_ref.rope(t, positions, f, mul, True)[0] for t in (qkv[:, :4], qkv[:, 4:6]))
    o = block_ref.attention(q, k, qkv[:, 6:], [(0, 70, 0, 70), (70, 1, 70, 1), (71, 133, 71, 133)], True, 0.125)[0]
    y, h3 = block_ref.rms_norm(o.flatten(1) @ p["wo"].double(), p["g2"], 1e-6, h2)
    # five roundings to fp16 (half a step 2^-11 each) of values of size about 1 pass through sums that spread
    # them as the values themselves: 16 half steps of the output's size cover them with room
    scale = whole.scales.double().repeat_interleave(64, 1)
    within(whole.residual, h3, 16 * 2.0**-11 * (1 + h3.abs()), "residual")
    within(whole.out.float().double() * scale, y, (2.0**-4 + 2.0**-8) * y.abs() + 2.0**-10 * scale + 16 * 2.0**-11 * (1 + y.abs()), "codes")
    # pieces: every sequence's first half, then the rest but the last token, then the last tokens
    room = 160
    ck, cv = (torch.full((3 * room, 2, 64), math.nan, device="cuda", dtype=F16) for _ in range(2))
    first = [0, 70, 71]
    done = [0, 0, 0]
    for to in ([35, 0, 64], [69, 0, 132], lens):
        rows = [torch.arange(first[b] + done[b], first[b] + to[b], device="cuda") for b in range(3)]
        pick = torch.cat(rows)
        slots = torch.cat([torch.arange(done[b], to[b], device="cuda") + b * room for b in range(3)])
        off = [0]
        for r in rows:
            off.append(off[-1] + len(r))
        got = block(p, x[pick], h[pick], positions[pick], table, i32(off), (ck, cv, i32([0, room, 2 * room]), i32(to), slots))
        # the same sums in another order: one rounding of the attention's output and of the product may fall the other way
        within(got.residual, whole.residual[pick].double(), 8 * 2.0**-11 * (1 + h3[pick].abs()), f"residual of a piece to {to}")
        done = list(to)
