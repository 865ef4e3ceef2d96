// Work items of the packed attention on tensor cores (k_attn_packed_tc.cu): which tiles and ranges of keys a block of
// the grid computes, from the sequences' offsets and lengths.  Whole-number arithmetic without CUDA, so that the host
// can check it too.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define MRF_HD __host__ __device__ __forceinline__
#else
#include <algorithm>
#define MRF_HD inline
#endif

namespace mrf {
namespace {

#ifndef __CUDACC__
using std::max;
using std::min;
#endif

constexpr int kKeys = 128;   // of a block
constexpr int kWindow = 32;  // sequences that are looked at together, one a lane

// The sequences of a call.
struct Batch {
  const int32_t *q_offsets, *k_start, *k_len;
  int q_rows, k_rows, seqs, kv_heads, TQ, causal;
  int chunk, max_splits;  // keys of a range (0: no splits), ranges that the workspace holds
};

// One unit of an item.  Token i of the tile sees the first min(klen, lim0 + i) keys of its range.
struct Unit {
  int q_row, ntok;   // the tile's first query row, its tokens (0: no unit)
  int kvh;
  int k_row, klen;   // the range's first key row, its keys
  int lim0;
  int nblk;          // key blocks that any of its tokens sees
  int split;
};
struct Item {
  Unit u[2];
  int shared;  // both units read the same key blocks
  int partial; // one key range of several: outputs go to the workspace
  int last;    // no more items
};

struct Seq {
  int q0, nq, k0, nk;
};
// Sequence b's rows, held to the tensors' whatever the offsets say.
MRF_HD Seq load_seq(const Batch &a, int b) {
  Seq s;
  s.q0 = min(max(a.q_offsets[b], 0), a.q_rows);
  s.nq = min(max(a.q_offsets[b + 1], s.q0), a.q_rows) - s.q0;
  if (a.k_len) {
    s.k0 = min(max(a.k_start[b], 0), a.k_rows);
    s.nk = min(max(a.k_len[b], 0), a.k_rows - s.k0);
  } else {
    s.k0 = s.q0;
    s.nk = s.nq;
  }
  return s;
}
// The keys of a sequence's ranges: whole blocks, more of them than `chunk` only where the workspace would not
// hold the ranges (max_k was too low).
MRF_HD int range_keys(const Batch &a, int nk) {
  if (a.chunk == 0) return nk;
  const int least = ((nk + a.max_splits - 1) / a.max_splits + kKeys - 1) / kKeys * kKeys;
  return max(a.chunk, least);
}
MRF_HD int range_count(const Batch &a, int nk) {
  return a.chunk == 0 ? 1 : max(1, (nk - 1) / range_keys(a, nk) + 1);
}
MRF_HD long long seq_items(const Batch &a, const Seq &s) {
  const int nt = (s.nq + a.TQ - 1) / a.TQ, ns = range_count(a, s.nk);
  if (ns > 1) return (long long)nt * a.kv_heads * ((ns + 1) / 2);
  return (long long)a.kv_heads * (nt / 2) + (nt & 1) * ((a.kv_heads + 1) / 2);
}
MRF_HD Unit make_unit(const Batch &a, const Seq &s, int tile, int kvh, int split) {
  Unit u;
  const int t0 = tile * a.TQ, chunk = range_keys(a, s.nk);
  const int r0 = (int)min((long long)split * chunk, (long long)s.nk);
  u.q_row = s.q0 + t0;
  u.ntok = min(a.TQ, s.nq - t0);
  u.kvh = kvh;
  u.k_row = s.k0 + r0;
  u.klen = min(s.nk - r0, chunk);
  u.lim0 = a.causal ? (t0 - s.nq) + 1 + (s.nk - r0) : u.klen;
  u.nblk = (max(0, min(u.klen, u.lim0 + u.ntok - 1)) + kKeys - 1) / kKeys;
  u.split = split;
  return u;
}
MRF_HD Item make_item(const Batch &a, const Seq &s, long long r) {
  Item it;
  const int nt = (s.nq + a.TQ - 1) / a.TQ, ns = range_count(a, s.nk);
  it.last = 0;
  it.shared = 0;
  it.partial = ns > 1;
  if (ns > 1) {
    const int js = (ns + 1) / 2, j = (int)(r % js), th = (int)(r / js);
    const int tile = nt - 1 - th / a.kv_heads, kvh = th % a.kv_heads;
    it.u[0] = make_unit(a, s, tile, kvh, 2 * j);
    it.u[1] = make_unit(a, s, tile, kvh, 2 * j + 1);
    if (2 * j + 1 >= ns) it.u[1].ntok = it.u[1].nblk = 0;
  } else if (r < (long long)a.kv_heads * (nt / 2)) {
    const int tile = (nt & 1) + 2 * (nt / 2 - 1 - (int)(r / a.kv_heads)), kvh = (int)(r % a.kv_heads);
    it.shared = 1;
    it.u[0] = make_unit(a, s, tile, kvh, 0);
    it.u[1] = make_unit(a, s, tile + 1, kvh, 0);
  } else {
    const int kvh = 2 * (int)(r - (long long)a.kv_heads * (nt / 2));
    it.u[0] = make_unit(a, s, 0, kvh, 0);
    it.u[1] = it.u[0];
    it.u[1].kvh = kvh + 1;
    if (kvh + 1 >= a.kv_heads) it.u[1].ntok = it.u[1].nblk = 0;
  }
  return it;
}

// The sequences base .. base + kWindow - 1 and the items of all before them and of these.
struct Walk {
  int base;
  long long before, total;  // 64 bits: wrong offsets may count rows many times
};
// Moves the walk to the sequences that item `it` is of; false when there are none.  load() sets the total at the walk's
// base.  Items mostly come in ascending order, but a take-over of blocks promises none: one that lies behind starts the
// walk again.
template <class Load>
MRF_HD bool find_sequences(Walk &w, int seqs, long long it, Load load) {
  if (it < w.before) {
    w.base = 0;
    w.before = 0;
    load();
  }
  while (w.base < seqs && it >= w.before + w.total) {
    w.base += kWindow;
    w.before += w.total;
    load();
  }
  return w.base < seqs;
}

}  // namespace
}  // namespace mrf
