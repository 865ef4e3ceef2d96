"""The work items of the packed attention (csrc/packed_items.cuh), checked on the CPU: the header's whole-number
arithmetic is compiled for the host, and one block after another asks for its item as the kernel's item warp does.
Blocks are taken over in no promised order, so every order has to give the same items, each row of each key head (and
each range of its keys) exactly once and inside the tensors."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "axial_band_split_b200", "csrc")

PROGRAM = r"""
#include "packed_items.cuh"
using namespace mrf;

// out: for each asked block 2 units of (sequence, q_row, ntok, kvh, k_row, klen, lim0, nblk, split, shared, partial);
// sequence -1: the block has no item
extern "C" void items_of(const int32_t *q_offsets, const int32_t *k_start, const int32_t *k_len, const int *shape, const long long *asked,
                         int n, int *out) {
  Batch a = {q_offsets, k_start, k_len, shape[0], shape[1], shape[2], shape[3], shape[4], shape[5], shape[6], shape[7]};
  Walk w = {};
  long long incl[kWindow] = {};
  auto load = [&]() {
    w.total = 0;
    for (int lane = 0; lane < kWindow; ++lane) incl[lane] = w.total += w.base + lane < a.seqs ? seq_items(a, load_seq(a, w.base + lane)) : 0;
  };
  load();
  for (int i = 0; i < n; ++i) {
    int *o = out + 22 * i;
    o[0] = o[11] = -1;
    if (!find_sequences(w, a.seqs, asked[i], load)) continue;
    const long long r = asked[i] - w.before;
    int src = 0;
    while (src < kWindow - 1 && incl[src] <= r) ++src;  // the first lane past r, as a ballot gives it
    const Seq s = load_seq(a, w.base + src);
    const Item it = make_item(a, s, r - (incl[src] - seq_items(a, s)));
    for (int t = 0; t < 2; ++t) {
      const Unit &u = it.u[t];
      const int v[11] = {w.base + src, u.q_row, u.ntok, u.kvh, u.k_row, u.klen, u.lim0, u.nblk, u.split, it.shared, it.partial};
      for (int k = 0; k < 11; ++k) o[11 * t + k] = v[k];
    }
  }
}
"""


@pytest.fixture(scope="module")
def items_of(tmp_path_factory):
    d = tmp_path_factory.mktemp("items")
    (d / "items.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover", "-static-libubsan", "-shared", "-fPIC",
                    "-I" + CSRC, "-o", str(d / "items.so"), str(d / "items.cpp")], check=True)
    f = ctypes.CDLL(str(d / "items.so")).items_of

    def call(q_offsets, k_start, k_len, shape, asked):
        q, s, l = (None if v is None else np.ascontiguousarray(v, np.int32) for v in (q_offsets, k_start, k_len))
        at = lambda v: None if v is None else v.ctypes.data_as(ctypes.c_void_p)
        asked, shape = np.ascontiguousarray(asked, np.int64), np.ascontiguousarray(shape, np.int32)
        out = np.zeros((len(asked), 2, 11), np.int32)
        f(at(q), at(s), at(l), at(shape), at(asked), len(asked), at(out))
        return out

    return call


def batch(rng, seqs, q_most, past, chunk):
    nq = [rng.choice((0, 1, 1, rng.randint(0, q_most))) for _ in range(seqs)]
    off = np.concatenate([[rng.randint(0, 3)], nq]).cumsum()
    nk = [max(0, n + rng.choice((0, rng.randint(-5, past)))) for n in nq]
    start, at = [], 0
    for n in nk:
        at += rng.randint(0, 9)
        start.append(at)
        at += n
    most = max(1, -(-max(nk + [1]) // chunk)) if chunk else 1
    return nq, off, nk, start, at, most


@pytest.mark.parametrize("seqs,q_most,past,chunk", [(1, 300, 0, 0), (5, 700, 0, 0), (33, 200, 500, 0), (100, 60, 300, 128), (200, 3, 3000, 384),
                                                   (65, 1, 2000, 256), (32, 40, 900, 128), (1000, 5, 4, 0)])
@pytest.mark.parametrize("kv_heads,TQ", [(1, 128), (2, 32), (3, 16), (8, 8)])
def test_every_order_of_blocks_gives_every_item_once(items_of, seqs, q_most, past, chunk, kv_heads, TQ):
    rng = random.Random(seqs * 1000 + TQ)
    nq, off, nk, start, k_rows, most = batch(rng, seqs, q_most, past, chunk)
    q_rows = int(off[-1]) + 2
    for causal in (0, 1):
        shape = [q_rows, k_rows + 1, seqs, kv_heads, TQ, causal, chunk, most]
        tiles = q_rows // TQ + seqs
        grid = tiles * kv_heads * ((most + 1) // 2) if chunk else tiles // 2 * kv_heads + min(seqs, tiles) * ((kv_heads + 1) // 2)
        want = items_of(off, start, nk, shape, np.arange(grid))
        check_cover(want, nq, off, nk, start, kv_heads, TQ, causal, chunk, most)
        back, mixed = np.arange(grid)[::-1], rng.sample(range(grid), grid)
        for order in (back, mixed, sorted(mixed, key=lambda i: (i // 7 % 3, -i))):
            got = items_of(off, start, nk, shape, order)
            assert np.array_equal(got, want[order])


def check_cover(items, nq, off, nk, start, kv_heads, TQ, causal, chunk, most):
    seen = {}
    for item in items:
        for b, q_row, ntok, kvh, k_row, klen, lim0, nblk, split, shared, partial in item.tolist():
            if b < 0 or ntok == 0:
                continue
            assert 0 <= kvh < kv_heads and off[b] <= q_row and q_row + ntok <= off[b + 1] and 0 < ntok <= TQ
            assert start[b] <= k_row and k_row + klen <= start[b] + nk[b] and 0 <= split < most
            for i in range(ntok):
                # the keys that the token sees, in this range
                vis = max(0, min(klen, lim0 + i))
                assert nblk * 128 >= vis
                seen.setdefault((q_row + i, kvh), []).append((k_row, k_row + vis, klen, partial, split))
    for b, n in enumerate(nq):
        for i in range(n):
            limit = min(nk[b], i + nk[b] - n + 1) if causal else nk[b]
            for h in range(kv_heads):
                ranges = sorted(seen.pop((off[b] + i, h)))
                assert len({r[4] for r in ranges}) == len(ranges) and (len(ranges) == 1) != bool(ranges[0][3])
                at = start[b]
                for k0, k1, klen, _, _ in ranges:
                    assert k0 == at
                    at += klen
                assert at == start[b] + nk[b]
                assert sum(k1 - k0 for k0, k1, _, _, _ in ranges) == max(0, limit)
    assert not seen


def test_wrong_offsets_stay_inside(items_of):
    """Offsets that descend, pass the tensors or overlap: whatever a block gets lies inside the tensors."""
    rng = random.Random(5)
    for trial in range(200):
        seqs, kv_heads, TQ = rng.randint(1, 80), rng.choice((1, 3, 8)), rng.choice((1, 8, 32))
        q_rows, k_rows, chunk = rng.randint(1, 300), rng.randint(1, 5000), rng.choice((0, 128, 384))
        wild = lambda: rng.choice((rng.randint(-50, 400), 2**31 - 1, -2**31))
        off = [wild() for _ in range(seqs + 1)]
        start, length = ([wild() for _ in range(seqs)] for _ in range(2))
        most = max(1, -(-rng.randint(1, k_rows) // chunk)) if chunk else 1
        shape = [q_rows, k_rows, seqs, kv_heads, TQ, trial % 2, chunk, most]
        for item in items_of(off, start, length, shape, [rng.randrange(4000) for _ in range(60)]):
            for b, q_row, ntok, kvh, k_row, klen, lim0, nblk, split, shared, partial in item.tolist():
                if b < 0 or ntok == 0:
                    continue
                assert 0 <= kvh < kv_heads and 0 <= q_row and 0 < ntok and q_row + ntok <= q_rows
                assert 0 <= k_row and 0 <= klen and k_row + klen <= k_rows and 0 <= split < most
                assert nblk >= 0 and (nblk - 1) * 128 < max(klen, 1)
