"""The block operators' smallest calls and their tables against arithmetic that is not theirs (no GPU)."""
import ctypes
import math
import os
import subprocess
from decimal import Decimal, localcontext

import numpy as np
import pytest

from axial_band_split_b200 import mrf
from test_block_ops import rope_args


def test_rope_of_no_tokens_takes_null_heads():
    """A tensor of no tokens has a null pointer: nothing is launched, whatever the pointers."""
    L = mrf.lib()
    assert L.mrf_rope(ctypes.byref(rope_args(tokens=0, q=None, k=None, q_out=None, k_out=None, positions=None)), None) == 0
    assert L.mrf_rope(ctypes.byref(rope_args(tokens=4, k=None)), None) == -2


PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def exact_turns(part, theta, scaling="none", factor=1.0, original=0):
    """The frequencies in turns a position, in 50 digits."""
    with localcontext() as ctx:
        ctx.prec = 50
        n, t, s = part, Decimal(theta), Decimal(factor)
        if scaling == "ntk":
            t *= s ** (Decimal(n) / (n - 2))
        f = [t ** (Decimal(-2 * i) / n) for i in range(n // 2)]
        if scaling == "linear":
            f = [v / s for v in f]
        if scaling == "yarn":
            dim = lambda turns: n * (Decimal(original) / (2 * PI * turns)).ln() / (2 * t.ln())
            lo, hi = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), n - 1)
            ramp = [min(max(Decimal(i - lo) / (hi - lo), Decimal(0)), Decimal(1)) for i in range(n // 2)]
            f = [v * (1 - r) + v / s * r for v, r in zip(f, ramp)]
        return [v / (2 * PI) for v in f]


@pytest.mark.parametrize("part,theta,scaling,factor,original", [
    (64, 10000.0, "none", 1.0, 0), (128, 5e5, "none", 1.0, 0), (256, 10000.0, "none", 1.0, 0), (1024, 1e6, "none", 1.0, 0), (2, 10000.0, "none", 1.0, 0),
    (128, 10000.0, "linear", 3.0, 0), (96, 10000.0, "ntk", 8.0, 0), (128, 1e6, "yarn", 32.0, 4096), (64, 10000.0, "yarn", 7.0, 2048),
])
def test_rope_table_against_fifty_digits(part, theta, scaling, factor, original):
    """Every entry is within 2^-63 of a turn: a half unit of 2^-64 from its rounding, the rest from the roundings before it
    (64-bit fractions of values below 0.16 of a turn: the power, the ramp's two products and sum, the division)."""
    got = mrf.rope_table(part, theta, scaling, factor, original, device="cpu").turns.numpy().view(np.uint64)
    with localcontext() as ctx:
        ctx.prec = 50
        for t, want in zip(got.tolist(), exact_turns(part, theta, scaling, factor, original)):
            assert abs(Decimal(t) - want * 2**64) <= 2


STATUS = r"""
#include <cassert>
#include <thread>
#include "op_status.h"
int main() {
  mrf::ExpiredWaits w;
  unsigned a = 0, b = 0;
  assert(!w.since(a) && !w.since(b));
  w.found(61);  // one thread read the device's word and cleared it
  assert(w.since(a) && !w.since(a));
  assert(w.since(b) && w.site.load() == 61 && !w.since(b));  // the other learns of it all the same, once
  w.found(53);
  w.found(54);
  assert(w.since(b) && !w.since(b) && w.since(a));
  unsigned told[4] = {};
  std::thread t[4];
  for (int i = 0; i < 4; ++i)
    t[i] = std::thread([&, i] {
      unsigned seen = 0;
      if (i == 0) w.found(7);
      while (!told[i]) told[i] = w.since(seen);
    });
  for (auto &x : t) x.join();
  return told[0] + told[1] + told[2] + told[3] == 4 ? 0 : 1;
}
"""


def test_an_expired_wait_is_told_to_every_thread(tmp_path):
    """The device's word is cleared by the first thread that asks: the others must not lose the answer."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "axial_band_split_b200", "csrc")
    (tmp_path / "status.cpp").write_text(STATUS)
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I" + csrc, "-o", str(tmp_path / "status"), str(tmp_path / "status.cpp")], check=True)
    assert subprocess.run([str(tmp_path / "status")], timeout=60).returncode == 0
