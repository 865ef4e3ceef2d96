"""The block operators' smallest calls and their tables against arithmetic that is not theirs (no GPU)."""
import ctypes

from axial_band_split_b200 import mrf
from test_block_ops import rope_args


def test_rope_of_no_tokens_takes_null_heads():
    """A tensor of no tokens has a null pointer: nothing is launched, whatever the pointers."""
    L = mrf.lib()
    assert L.mrf_rope(ctypes.byref(rope_args(tokens=0, q=None, k=None, q_out=None, k_out=None, positions=None)), None) == 0
    assert L.mrf_rope(ctypes.byref(rope_args(tokens=4, k=None)), None) == -2
