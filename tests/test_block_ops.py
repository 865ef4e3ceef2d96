"""Refusals and host tables of the block operators (no GPU): every bad call is answered with its
status before anything is launched, so the pointers here are never read."""
import ctypes
import math

import numpy as np
import pytest

import block_ref
from axial_band_split_b200 import mrf

P = 1 << 20  # an address that is aligned for every type


def norm_args(**change):
    a = dict(x=P, residual=None, weight=None, out=2 * P, residual_out=None, scales=None, rows=4, x_stride=64,
             residual_stride=64, out_stride=64, residual_out_stride=64, dim=64, dtype=1, weight_dtype=0, out_dtype=1,
             group=0, clamp=0, eps=1e-6)
    a.update(change)
    return mrf.mrf_rms_norm_args(**a)


def rope_args(**change):
    a = dict(q=P, k=2 * P, q_out=3 * P, k_out=4 * P, positions=5 * P, turns=6 * P, tokens=4, q_token_stride=256,
             q_head_stride=64, k_token_stride=128, k_head_stride=64, q_out_token_stride=256, q_out_head_stride=64,
             k_out_token_stride=128, k_out_head_stride=64, heads=4, kv_heads=2, width=64, part=64, dtype=1,
             positions_wide=0, interleaved=1, scale=1.0)
    a.update(change)
    return mrf.mrf_rope_args(**a)


def attention_args(**change):
    a = dict(q=P, k=2 * P, v=3 * P, out=4 * P, lse=None, q_offsets=5 * P, k_start=None, k_len=None, workspace=None,
             workspace_bytes=0, q_rows=8, k_rows=8, max_k=0, q_token_stride=256, q_head_stride=64, k_token_stride=128,
             k_head_stride=64, v_token_stride=128, v_head_stride=64, out_token_stride=256, out_head_stride=64, seqs=2,
             heads=4, kv_heads=2, width=64, v_width=64, dtype=1, causal=1, scale=0.125)
    a.update(change)
    return mrf.mrf_attention_args(**a)


EINVAL, ESHAPE, EUNSUPPORTED = -1, -2, -5


@pytest.mark.parametrize("change,status", [
    (dict(dtype=7), EINVAL), (dict(dtype=3, out_dtype=3, scales=P), EINVAL), (dict(out_dtype=0), EINVAL),
    (dict(weight=P, weight_dtype=9), EINVAL), (dict(rows=-1), ESHAPE), (dict(dim=0), ESHAPE),
    (dict(dim=16385, x_stride=16385, out_stride=16385), EUNSUPPORTED), (dict(group=32), EINVAL),
    (dict(out_dtype=3, scales=P, group=48), EINVAL), (dict(out_dtype=3, scales=P, group=-1), EINVAL),
    (dict(eps=0.0), EINVAL), (dict(eps=math.nan), EINVAL), (dict(eps=math.inf), EINVAL), (dict(eps=-1e-6), EINVAL),
    (dict(residual_out=7 * P), EINVAL), (dict(out_dtype=3), EINVAL), (dict(scales=P), EINVAL), (dict(x=None), EINVAL),
    (dict(out=None), EINVAL), (dict(x=P + 1), EINVAL), (dict(weight=P + 2), EINVAL), (dict(out=P + 1), EINVAL),
    (dict(out_stride=63), ESHAPE), (dict(out_stride=0), ESHAPE),
    (dict(residual=7 * P, residual_out=8 * P, residual_out_stride=10), ESHAPE),
    (dict(residual=7 * P, residual_out=2 * P), EINVAL), (dict(residual=7 * P, residual_out=P), EINVAL),
    (dict(residual=2 * P), EINVAL), (dict(out=P, out_stride=128), EINVAL), (dict(out=P, out_dtype=3, scales=7 * P), EINVAL),
    (dict(residual=7 * P, residual_out=7 * P, residual_out_stride=128), EINVAL),
])
def test_norm_refusals(change, status):
    assert mrf.lib().mrf_rms_norm(ctypes.byref(norm_args(**change)), None) == status
    assert b"mrf_rms_norm" in mrf.lib().mrf_last_error(None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), EINVAL), (dict(tokens=-1), ESHAPE), (dict(tokens=1 << 31), ESHAPE), (dict(heads=0), ESHAPE), (dict(kv_heads=-1), ESHAPE),
    (dict(k=None), ESHAPE), (dict(width=1, part=2), ESHAPE), (dict(width=1026), ESHAPE), (dict(part=0), ESHAPE),
    (dict(part=66), ESHAPE), (dict(part=33), ESHAPE), (dict(scale=math.nan), EINVAL), (dict(q=None), EINVAL),
    (dict(q_out=None), EINVAL), (dict(k_out=None), EINVAL), (dict(positions=None), EINVAL), (dict(turns=None), EINVAL),
    (dict(q=P + 1), EINVAL), (dict(positions=P + 2), EINVAL), (dict(positions=P + 4, positions_wide=1), EINVAL),
    (dict(turns=P + 4), EINVAL), (dict(q_out_token_stride=128), ESHAPE), (dict(q_out_head_stride=32), ESHAPE),
    (dict(k_out_token_stride=0), ESHAPE), (dict(q_out=P, q_out_token_stride=512), EINVAL),
    (dict(k_out=2 * P, k_out_token_stride=512), EINVAL),
])
def test_rope_refusals(change, status):
    assert mrf.lib().mrf_rope(ctypes.byref(rope_args(**change)), None) == status
    assert b"mrf_rope" in mrf.lib().mrf_last_error(None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), EINVAL), (dict(seqs=-1), ESHAPE), (dict(q_rows=-1), ESHAPE), (dict(k_rows=-1), ESHAPE),
    (dict(q_rows=1 << 31), ESHAPE), (dict(k_rows=1 << 31), ESHAPE), (dict(max_k=-1), ESHAPE), (dict(heads=3), ESHAPE),
    (dict(heads=0), ESHAPE), (dict(kv_heads=0), ESHAPE), (dict(width=0), ESHAPE), (dict(v_width=0), ESHAPE),
    (dict(width=257), EUNSUPPORTED), (dict(v_width=300), EUNSUPPORTED), (dict(scale=0.0), EINVAL),
    (dict(scale=math.nan), EINVAL), (dict(scale=-1.0), EINVAL), (dict(k_start=P), EINVAL), (dict(k_len=P), EINVAL),
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(out=None), EINVAL),
    (dict(q_offsets=None), EINVAL), (dict(q=P + 1), EINVAL), (dict(lse=P + 2), EINVAL), (dict(q_offsets=P + 1), EINVAL),
    (dict(k_rows=7), ESHAPE), (dict(out_token_stride=128), ESHAPE), (dict(out_head_stride=32), ESHAPE),
    (dict(out=P), EINVAL), (dict(out=3 * P), EINVAL),
])
def test_attention_refusals(change, status):
    need = ctypes.c_size_t(7)
    assert mrf.lib().mrf_attention(ctypes.byref(attention_args(**change)), None) == status
    assert b"mrf_attention" in mrf.lib().mrf_last_error(None)
    assert mrf.lib().mrf_attention_workspace(ctypes.byref(attention_args(**change)), ctypes.byref(need)) == status
    assert need.value == 0


@pytest.mark.parametrize("packer,args", [(mrf._NORM, norm_args()), (mrf._ROPE, rope_args()), (mrf._ATTENTION, attention_args())])
def test_packed_arguments_are_the_structures(packer, args):
    values = [getattr(args, n) or 0 for n, _ in args._fields_]
    assert packer.pack(*values) == bytes(args)


def test_null_and_empty_calls():
    L = mrf.lib()
    assert L.mrf_rms_norm(None, None) == L.mrf_rope(None, None) == L.mrf_attention(None, None) == EINVAL
    assert L.mrf_attention_workspace(ctypes.byref(attention_args()), None) == EINVAL
    assert L.mrf_rope_table(None, None, None) == EINVAL
    # nothing to do: nothing is launched, whatever the pointers
    assert L.mrf_rms_norm(ctypes.byref(norm_args(rows=0, x=None, out=None)), None) == 0
    assert L.mrf_rope(ctypes.byref(rope_args(tokens=0, q=None, q_out=None, positions=None)), None) == 0
    assert L.mrf_attention(ctypes.byref(attention_args(q_rows=0, q=None, out=None)), None) == 0
    assert L.mrf_attention(ctypes.byref(attention_args(seqs=0)), None) == 0


@pytest.mark.parametrize("change,status", [
    (dict(part=0), ESHAPE), (dict(part=3), ESHAPE), (dict(part=1026), ESHAPE), (dict(theta=1.0), EINVAL),
    (dict(theta=math.inf), EINVAL), (dict(scaling="linear", factor=0.5), EINVAL), (dict(scaling="ntk", part=2), EINVAL),
    (dict(scaling="yarn", factor=2.0), EINVAL), (dict(scaling="yarn", factor=2.0, original=4096, beta_fast=1, beta_slow=2), EINVAL),
    (dict(scaling="other"), EINVAL),
])
def test_rope_table_refusals(change, status):
    with pytest.raises(mrf.MrfError) as e:
        mrf.rope_table(**{"part": 64, "device": "cpu", **change})
    assert e.value.status == status


@pytest.mark.parametrize("part,theta,scaling,factor,original", [
    (64, 10000.0, "none", 1.0, 0), (2, 10000.0, "none", 1.0, 0), (128, 5e5, "linear", 4.0, 0), (96, 10000.0, "ntk", 8.0, 0),
    (128, 1e6, "yarn", 32.0, 4096), (32, 10000.0, "yarn", 16.0, 2048), (128, 10000.0, "yarn", 1.0, 4096),
])
def test_rope_table_against_the_formulas(part, theta, scaling, factor, original):
    t = mrf.rope_table(part, theta, scaling, factor, original, device="cpu")
    f, mul = block_ref.rope_frequencies(part, theta, scaling, factor, original)
    got = t.turns.numpy().view(np.uint64).astype(np.float64) / 2.0**64 * 2 * math.pi
    # 53-bit arithmetic on both sides (powers and logarithms within a few steps), 2^-62 of a turn in the table
    assert np.all(np.abs(got - np.array(f)) <= 64 * 2.0**-53 * np.array(f) + 2.0**-59)
    assert t.scale == pytest.approx(mul, rel=2.0**-23) and t.part == part


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64)
    with pytest.raises(mrf.MrfError):
        mrf.rms_norm(x)
    with pytest.raises(mrf.MrfError):
        mrf.rope(x[:, None], None, torch.zeros(2, dtype=torch.int32), mrf.rope_table(64, device="cpu"))
    with pytest.raises(mrf.MrfError):
        mrf.attention_packed(x[:, None], x[:, None], x[:, None], torch.zeros(2, dtype=torch.int32))
