"""The block operators where their loops turn more than once, where offsets are wrong and where a graph captures the
first call, against their formulas in 64 bits with the bounds that block_ref derives."""
import os
import subprocess
import sys

import pytest

import block_ref
from axial_band_split_b200 import mrf

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_block_ops_gpu import BF16, E4M3, F16, F32, check_quant, gen, randn, within  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------------------------------ rope
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("tokens", [1301, 4099, 20001])
@pytest.mark.parametrize("width,part", [(64, 64), (64, 32), (80, 40), (80, 20), (33, 6), (256, 128)])
def test_rope_of_several_tokens_a_block(dtype, interleaved, tokens, width, part):
    """From 1184 tokens on a block has several, the last one fewer: units of 8, 4, 2 and 1 pairs, heads that turn in part."""
    g = gen(tokens + width)
    heads, kv = (3, 1) if tokens < 20000 else (1, 1)
    q, k = randn(g, tokens, heads, width, dtype=dtype), randn(g, tokens, kv, width, dtype=dtype)
    pos = torch.randint(0, 100000, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    table = mrf.rope_table(part)
    f, mul = block_ref.rope_frequencies(part)
    got = mrf.rope(q, k, pos, table, interleaved)
    alone, _ = mrf.rope(k, None, pos, table, interleaved)
    assert torch.equal(alone, got[1])
    for x, y in zip((q, k), got):
        ref, size = block_ref.rope(x, pos, f, mul, interleaved)
        within(y, ref, block_ref.rope_slack(size) + block_ref.half_step(dtype) * ref.abs() * 1.01 + (size > 0) * 2.0**-25)
    mrf.rope(q, k, pos, table, interleaved, q_out=q, k_out=k)
    assert torch.equal(q, got[0]) and torch.equal(k, got[1])


def test_rope_far_positions_against_fifty_digits():
    """Angles at positions up to 2^37 from frequencies that are not the table's: off by position * 2^-63 of a turn at most."""
    from decimal import Decimal, localcontext
    from test_block_ops_edges import PI, exact_turns
    g = gen(12)
    places = [0, 1, 4097, (1 << 20) + 3, (1 << 31) - 1, 1 << 31, (1 << 36) + 12345, (1 << 37) - 1, -(1 << 33), -(1 << 37)]
    q = randn(g, len(places), 2, 128)
    with localcontext() as ctx:
        ctx.prec = 50
        fractions = [[p * f % 1 for f in exact_turns(128, 10000.0)] for p in map(Decimal, places)]
        angle = torch.tensor([[float(2 * PI * t) for t in row] for row in fractions], dtype=torch.float64, device="cuda")[:, None]
    far = torch.tensor([abs(p) for p in places], dtype=torch.float64, device="cuda")[:, None, None] * 2.0**-63 * 6.2832
    got, _ = mrf.rope(q, None, torch.tensor(places, device="cuda"), mrf.rope_table(128, 10000.0), interleaved=False)
    a, b = q[..., :64].double(), q[..., 64:].double()
    size = a.abs() + b.abs()
    bound = block_ref.rope_slack(size) + size * far
    within(got[..., :64], a * angle.cos() - b * angle.sin(), bound)
    within(got[..., 64:], b * angle.cos() + a * angle.sin(), bound)


def test_rope_of_no_tokens():
    """A step without new tokens, new outputs and in place: q and k of no rows, whose tensors have null pointers."""
    x = torch.zeros(4, 8, 64, device="cuda", dtype=F16)
    pos, table = torch.arange(4, device="cuda"), mrf.rope_table(64)
    for q, k in ((x[:0, :6], x[:0, 6:]), (x[:0], None)):
        a, b = mrf.rope(q, k, pos[:0], table)
        assert a.shape == q.shape and (b is None if k is None else b.shape == k.shape)
        assert mrf.rope(q, k, pos[:0], table, q_out=q, k_out=k)[0] is q


# ------------------------------------------------------------------------------------------ norm
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,dim", [(10001, 64), (9601, 200), (10001, 384), (10001, 520), (200, 8200), (331, 16384), (10001, 2049), (40001, 131),
                                      (1500, 4096), (600, 16383)])
def test_norm_of_several_rows_a_team(dtype, rows, dim):
    """More rows than the launch has warps or blocks, so that each takes several: every kernel, plain and 8-bit."""
    g = gen(rows + dim)
    x, res, w = randn(g, rows, dim, dtype=dtype), randn(g, rows, dim, dtype=dtype), 1 + 0.1 * randn(g, dim)
    for residual in (None, res):
        y, h = block_ref.rms_norm(x, w, 1e-6, residual)
        r = mrf.rms_norm(x, w, 1e-6, residual)
        within(r.out, y, y.abs() * (block_ref.norm_slack(dim) + block_ref.half_step(dtype)) + 2.0**-25, "out")
        if residual is not None:
            within(r.residual, h, h.abs() * (block_ref.U32 + block_ref.half_step(dtype)) * 1.001 + 2.0**-25, "h")
        for group in (0, 128):
            q = mrf.rms_norm(x, w, 1e-6, residual, out_dtype=E4M3, group=group)
            check_quant(q, y, group, dim)
            if residual is not None:
                assert torch.equal(q.residual, r.residual)


# ------------------------------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype,width", [(F16, 64), (BF16, 128), (F32, 64), (F16, 36)])
@pytest.mark.parametrize("cache", [0, 9000])
def test_attention_wrong_offsets_write_no_other_rows(dtype, width, cache):
    """Offsets beyond the tensors or descending: rows of the output that no clamped span holds, and what lies before and
    behind it, stay as they were, on both kernels, with and without ranges of keys."""
    g = gen(width)
    q_rows = 12 if cache else 300
    heads, kv = (8, 1) if cache else (4, 2)
    k_rows = cache or q_rows
    q, k, v = randn(g, q_rows, heads, width, dtype=dtype), randn(g, k_rows, kv, width, dtype=dtype), randn(g, k_rows, kv, width, dtype=dtype)
    i32 = lambda t: torch.tensor(t, device="cuda", dtype=torch.int32)
    big = 2**31 - 1
    for off in ([0, 5], [-5, 4], [0, 1000], [10, 5], [big, big], [9, 3, 11], [2, 2, 2], [7, big, 3], [-big, -1, 6], [3, 8, 8, big]):
        seqs = len(off) - 1
        spans = [(min(max(a, 0), q_rows), min(max(b, 0), q_rows)) for a, b in zip(off, off[1:])]
        lengths = [(None, None)] if not cache else [([3] * seqs, [cache - 10] * seqs), ([-9] * seqs, [1 << 30] * seqs), ([1 << 30] * seqs, [5] * seqs),
                                                   ([7] * seqs, [-4] * seqs)]
        for start, length in lengths:
            pad = 40
            whole = torch.full((q_rows + 2 * pad, heads, width), 7.0, device="cuda", dtype=dtype)
            out = whole[pad : pad + q_rows]
            mrf.attention_packed(q, k, v, i32(off), start and i32(start), length and i32(length), out=out)
            mrf.ops_sync_status()
            inside = torch.zeros(q_rows, dtype=torch.bool, device="cuda")
            for a, b in spans:
                inside[a:b] = True
            assert (whole[:pad] == 7).all() and (whole[pad + q_rows :] == 7).all() and (out[~inside] == 7).all(), (off, start, length)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("width", [64, 128])
@pytest.mark.parametrize("queries,heads,kv", [(1, 8, 1), (300, 2, 1)])
def test_attention_of_many_small_weights(dtype, width, queries, heads, kv):
    """A key in every 1500 takes the weight and has no value; the others have 2^-24.5 to 2^-26.5 of it each, and all of the
    output.  Beside the relative half steps a weight may be off by 2^-32 of the largest, half a step of fp16's smallest
    numbers with the factor of 2^7; unscaled ones would lose most of the output."""
    g = gen(width)
    keys = 20000
    x = 24.5 + 2 * torch.rand(keys, generator=g, device="cuda")
    x[::1500] = 0
    q = torch.zeros(queries, heads, width, device="cuda", dtype=dtype)
    q[..., 0] = 1
    k = torch.zeros(keys, kv, width, device="cuda", dtype=dtype)
    k[..., 0] = (-x * 0.6931471805599453)[:, None].to(dtype)
    v = (0.5 + torch.rand(keys, kv, width, generator=g, device="cuda")).to(dtype)
    v[::1500] = 0
    i32 = lambda *t: torch.tensor(t, device="cuda", dtype=torch.int32)
    out, lse = mrf.attention_packed(q, k, v, i32(0, queries), i32(0), i32(keys), keys, causal=False, scale=1.0, return_lse=True)
    ref, rlse, size, big = block_ref.attention(q, k, v, [(0, queries, 0, keys)], False, 1.0)
    bound, lbound = block_ref.attention_slack(dtype, ref, size, big, keys, width)
    share = keys * 2.0**-32 / rlse.exp()[..., None] * 1.5  # (values up to 1.5)
    # the output itself is a small number of its type
    step = 2.0**-25 if dtype == F16 else 0.0
    within(out, ref, bound + share + step)
    within(lse, rlse, lbound)


# ------------------------------------------------------------------------------------- refusals
def test_tangents_are_refused():
    """Forward-mode derivatives: a tensor with a tangent is refused as one that requires a gradient, the others are not."""
    import torch.autograd.forward_ad as forward_ad
    x = torch.ones(4, 2, 64, device="cuda", dtype=F16)
    off, pos, table = torch.tensor([0, 4], device="cuda", dtype=torch.int32), torch.arange(4, device="cuda"), mrf.rope_table(64)
    w = torch.ones(64, device="cuda")
    with forward_ad.dual_level():
        d, dw = forward_ad.make_dual(x, torch.ones_like(x)), forward_ad.make_dual(w, torch.ones_like(w))
        for call in (lambda: mrf.rms_norm(d), lambda: mrf.rms_norm(x, dw), lambda: mrf.rms_norm(x, residual=d), lambda: mrf.rope(d, None, pos, table),
                     lambda: mrf.rope(x, d, pos, table), lambda: mrf.attention_packed(d, x, x, off), lambda: mrf.attention_packed(x, d, x, off),
                     lambda: mrf.attention_packed(x, x, d, off)):
            with pytest.raises(mrf.MrfError, match="gradient"):
                call()
        assert mrf.rms_norm(x, w, residual=x).out.shape == x.shape and mrf.attention_packed(x, x, x, off).shape == x.shape
        assert mrf.rope(x, x, pos, table)[1].shape == x.shape


def test_rotary_tables_that_do_not_hold_their_pairs_are_refused():
    """A table with another part than its values, or values of another kind, would be read past its end."""
    x, pos, table = torch.ones(4, 2, 128, device="cuda", dtype=F16), torch.arange(4, device="cuda"), mrf.rope_table(64)
    for bad in (table._replace(part=128), table._replace(part=66), table._replace(part=62), table._replace(part=-64), table._replace(turns=table.turns[::2]),
                table._replace(turns=table.turns[::2], part=32), table._replace(turns=table.turns.int()),
                table._replace(turns=None), table._replace(turns=table.turns.cpu()), tuple(table)):
        with pytest.raises(mrf.MrfError):
            mrf.rope(x, None, pos, bad)
    part = mrf.rope(x, None, pos, table._replace(turns=table.turns[:16].clone(), part=32))[0]
    assert torch.equal(part[..., 32:], x[..., 32:])


def test_attention_without_a_tensor_map_uses_no_unchecked_workspace():
    """A token stride that no tensor map takes (the row behind it is of no sequence): the CUDA cores compute, and a null
    workspace is not written although workspace_bytes names some, because the call needs none."""
    import ctypes
    from test_block_ops import attention_args
    g = gen(3)
    q, k, v = randn(g, 2, 64, 128, dtype=F16), randn(g, 384, 1, 128, dtype=F16), randn(g, 384, 1, 128, dtype=F16)
    i32 = lambda *t: torch.tensor(t, device="cuda", dtype=torch.int32)
    out, off, start, length = torch.full_like(q, 7.0), i32(0, 1), i32(0), i32(384)
    a = attention_args(q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), out=out.data_ptr(), q_offsets=off.data_ptr(), k_start=start.data_ptr(),
                       k_len=length.data_ptr(), workspace=None, workspace_bytes=1 << 40, q_rows=2, k_rows=384, q_token_stride=1 << 41, q_head_stride=128,
                       k_token_stride=128, k_head_stride=128, v_token_stride=128, v_head_stride=128, out_token_stride=64 * 128, out_head_stride=128,
                       seqs=1, heads=64, kv_heads=1, width=128, v_width=128, scale=128**-0.5)
    need = ctypes.c_size_t(1)
    assert mrf.lib().mrf_attention_workspace(ctypes.byref(a), ctypes.byref(need)) == 0 and need.value == 0
    assert mrf.lib().mrf_attention(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    ref, _, size, big = block_ref.attention(q, k, v, [(0, 1, 0, 384)], True, 128**-0.5)
    bound, _ = block_ref.attention_slack(F16, ref, size, big, 384, 128)
    within(out[:1], ref[:1], bound[:1] + 2.0**-25)
    assert (out[1:] == 7).all()


FIRST = """
import torch
from axial_band_split_b200 import mrf
torch.manual_seed(0)
x = torch.randn(700, 8, 128, device="cuda", dtype=torch.float16)
k, v = x[:, :2].contiguous(), x[:, 2:4].contiguous()
wide = torch.randn(50, 4, 200, device="cuda", dtype=torch.float16)
i32 = lambda *t: torch.tensor(t, device="cuda", dtype=torch.int32)
off, off1, one, start, length, offw = i32(0, 300, 700), i32(0, 1), x[:1].contiguous(), i32(0), i32(700), i32(0, 50)
pos, table = torch.arange(700, device="cuda"), mrf.rope_table(128)
w = torch.ones(1024, device="cuda")
def step():
    n = mrf.rms_norm(x.flatten(1), w, residual=x.flatten(1), out_dtype=torch.float8_e4m3fn, group=128)
    odd = mrf.rms_norm(x.flatten(1)[:, :1001])
    q, kk = mrf.rope(x, k, pos, table, interleaved=False)
    a = mrf.attention_packed(q, kk, v, off)
    b = mrf.attention_packed(one, kk, v, off1, start, length)
    c = mrf.attention_packed(wide, wide, wide, offw)
    return [n.out.float(), n.scales, n.residual, odd.out, q, kk, a, b, c]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
want = step()
mrf.ops_sync_status()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("equal")
"""


def test_first_calls_of_a_process_are_captured():
    """No call of the process came before the capture: what a first call sets up is set up inside it."""
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stdout + r.stderr
