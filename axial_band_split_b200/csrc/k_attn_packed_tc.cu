// Packed attention with grouped heads on tcgen05 tensor cores (mrf_attention): o = softmax(scale q
// k^T) v per sequence and head, widths up to 128, fp16 or bf16, causal or not, over the query's own
// rows or a cache.  One pass over the keys with a running maximum and sum; the scores never leave
// the SM.
//
// Tiles.  The G = heads / kv_heads query heads that share a key head are rows of one matrix: a tile
// is TQ = 128 / G tokens (32 / G for single new tokens, see Cfg) x G heads, row = token * G + head, one
// bulk tensor load of a (64, G, 1, TQ) box per 64 dimensions.  So each key block is read once for all of
// them and a single new token already fills G rows.  Key blocks are 128 rows.
//
// Work items.  A CTA runs two units (a tile with a range of keys) t = 0, 1 side by side:
//   pair   - two neighbouring tiles of one sequence and key head: they share every key block;
//   heads  - a sequence's odd tile (its first, which sees the fewest keys) for two key heads, each
//            unit with its own keys: short prompts and single tokens have nothing but these;
//   splits - with few tiles and long keys, two key ranges of one tile: the ranges, of equal size in all
//            sequences, leave their own outputs and log-sums in the workspace, and combine_kernel joins them.
// Items are numbered sequence by sequence, a causal sequence's last tiles (the most keys) first.  The grid
// has a block for each; a running CTA takes over blocks that have not been launched (cluster launch
// control), so that items go to whoever is free, in order.  Lengths live in device memory, so warp 11
// finds each item's sequence by a running prefix sum over the sequences' item counts and hands it to the
// others through shared memory.
//
// Warps 0-3 and 4-7: softmax of unit 0 and 1, one score row per thread; warp 8: bulk tensor loads;
// warps 9, 10: matrix instructions of unit 0, 1; warp 11: items.
//
// Tensor memory (512 columns).  With v up to 64 wide: S_t at 128 t, O_t at 256 + 64 t, P_t (the 16-bit
// probabilities, half as wide) at 384 + 64 t, and the next block's scores compute under this block's
// exponentials.  With wider v S_t at 128 t and O_t at 256 + 128 t fill it.  P is handed over in two
// halves of 64 keys, so P V of the first runs under the second's exponentials; with wider v the first
// half overwrites S_t (the softmax has read it all), the second goes through shared memory, and the
// issuer queues the next block's scores as soon as the first half's P V has ended: they are ready when the
// second half's exponentials are done.  (With both halves over S_t they had to wait for the whole P V,
// about 1200 of a block's 4000 clk.  Queued right behind the first half, without a wait, they were no
// faster: a prompt of 16384 tokens 841 us against 832, token steps 105 against 107.)
//
// K and V blocks stream through one ring in the order of their use (separate keys: the two units'
// streams take turns).  Both issuers acknowledge every slot, their own when its reads have ended and
// the other unit's as it arrives: a phase of a slot's barrier is then never more than one ahead of
// anybody who waits on it by parity.
//
// Key rows past a sequence's end belong to others or were never written: their scores are replaced
// by -inf whatever they are, and their rows of v, whose product with a zero probability could still
// be NaN, are zeroed in shared memory before the second product.
//
// Measured, against a copy of 6.57 TB/s and a matrix product of 1669 TFLOP/s on the same device:
//   a causal prompt of 16384 tokens, 16 heads of 128 over 4   0.84 ms, 1.31 PFLOP/s, 0.78
//   7 causal prompts of 200 to 4096 tokens, 32 over 8         0.29 to 0.34 ms, 0.9 to 1.03 PFLOP/s, 0.54 to 0.62
//   8 x 1100 tokens both ways, 8 heads of 64                  44 to 47 us, 0.42 to 0.45 PFLOP/s
//   a token of each of 32 sequences of 500 to 8191 keys       106 us, 5.0 TB/s, 0.76
//   a token after 65536 keys                                  58.5 us, 4.6 TB/s, 0.70
// A block of 128 keys costs both units together 3400 to 3700 clk, where its matrix instructions need 2800 with widths of
// 128 and its exponentials, at 16 a clk and SM, 2048: each unit's row loads, maxima, conversions and stores stand beside its
// exponentials.  With 64 those phases bound it, and an item's start and output (about 4000 clk each) weigh as much as a block
// or two, as they do in short prompts.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "block_ops.h"
#include "gemm_tc.cuh"
#include "packed_items.cuh"
#include "tc_ptx.cuh"

namespace mrf {
namespace {

constexpr int kRows = 128, kHalf = 64;
constexpr int kLate = 32;           // keys of P's second half whose exponentials run before the first half is handed over
constexpr int kAtom = kRows * 128;  // 64 16-bit values of 128 rows
constexpr int kThreads = 384;
// register split, as in the model's attention: 2 * 128 * 208 + 128 * 72 <= 384 * 168
constexpr int kRegsLaunch = 168, kRegsSoftmax = 208, kRegsIo = 72;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsIo <= kThreads * kRegsLaunch, "register split over budget");
constexpr float kRescaleLog2 = 8.f;  // a row's maximum is raised only when exceeded by more than 2^8
// Probabilities and their sum carry a factor of 2^kUp.  fp16 ends at 2^-24: without the factor weights below 2^-14 of the
// maximum would lose bits and those below 2^-25 vanish from the product while the sum has them, 2^-9 of the output with
// 65536 such keys beside one that takes the weight.  2^7 is what 2^8 above the maximum leaves below 65504.
template <bool kBF>
constexpr float kUp = kBF ? 0.f : 7.f;
// Key blocks of an item that are still to be loaded when the next one is taken: late, so that the longest items, which
// come first, do not also get the first of the rest (a prompt of 4096 tokens, 16 heads: 69 us, 86 when it is taken at
// once), and early enough for the time that taking one needs.
constexpr int kAhead = 4;
constexpr int kItems = 1;            // ring of work items: the next one is taken when everybody has begun this one

// kFew: tiles of 32 rows (new tokens).  The matrix instructions still have 128 rows, but only 32 are stored:
// unit t's are rows 32 t .. 32 t + 31 of an area of 64, which both units' operands start at, and what the
// other rows read (the other unit's, the areas behind) ends in rows that nobody reads.  A unit's rows are one
// warp's, on a scheduler of their own, and the room goes to more key blocks in flight.
template <int QA, int VA, bool kFew>
struct Cfg {
  static constexpr bool overlay = VA == 2;           // P's first half over S, its second in shared memory
  static constexpr int qbufs = QA == 1 ? 2 : 1;      // q buffers of two tiles
  static constexpr int rows = kFew ? 32 : kRows;     // of a tile
  static constexpr int tile = rows * 128;            // 64 16-bit values of a tile's rows
  static constexpr int unit = kFew ? 0 : QA * kAtom; // from unit 0's q operand to unit 1's
  static constexpr int step = kFew ? 2 * tile : kAtom;  // from one 64 values to the next
  static constexpr int qbuf = 2 * QA * tile;
  static constexpr int slot = (QA > VA ? QA : VA) * kAtom;
  static constexpr int q = 0;
  static constexpr int p = q + qbufs * qbuf;         // the second half of P; the output's way out
  static constexpr int kv = p + (overlay ? 2 * tile : 0);
  static constexpr int slots = (14 * kAtom - kv) / slot;  // ring of K or V blocks
  static constexpr int bar = kv + slots * slot;
  static constexpr int item = bar + 512;
  static constexpr int resp = (item + kItems * (int)sizeof(Item) + 15) / 16 * 16;  // taken_block's answer
  static constexpr int total = resp + 16;
  static constexpr int warps = kFew ? 1 : 4;         // softmax warps of a unit
  static_assert(total + 1024 <= 232448, "shared memory over the 227 KB limit");
  static_assert(p + kAtom <= bar && q + qbufs * qbuf + kAtom <= bar, "operands of 128 rows stay inside");
};

struct Args : Batch {
  void *out;
  float *lse;         // or null
  float *part;        // splits: [split][row * heads + head][v_width], then their log2 sums
  float *part_lse;
  long long out_token_stride, out_head_stride;
  int heads, G, width, v_width;
  float scale, scale_log2;
};

// Take over the next block of the grid that has not been launched: the answer arrives at resp (16 bytes) and
// counts on bar.
__device__ __forceinline__ void take_block(void *resp, uint64_t *bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   tc::smem_u32(resp)),
               "r"(tc::smem_u32(bar))
               : "memory");
}
// Its index, or -1 when there was none left (nobody may ask again then).
__device__ __forceinline__ int taken_block(const void *resp) {
  int x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "mov.b32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
      : "=r"(x)
      : "r"(tc::smem_u32(resp))
      : "memory");
  return x;
}

__device__ unsigned g_status[2];  // a bounded wait that expired: 1, site

// ------------------------------------------------------------------ small device helpers
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <bool kBF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (kBF) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
  } else {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
  }
}

// 32 fp32 columns of this thread's lane, not waited for; tmem_landed orders every use after the wait.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_landed(uint32_t *r) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                 "+r"(r[i + 6]), "+r"(r[i + 7]));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// 8 columns of this thread's lane times f (few registers: scores are held while it runs)
__device__ __forceinline__ void tmem_scale8(uint32_t taddr, float f) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Matrix instructions of a whole warp, issued by its `leader` lane alone: without a branch around them
// the operands stay in uniform registers (inside one, each cost about 130 clk to issue).
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p;
}
// D (+)= A * B, both from shared memory.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc), "r"(leader));
}
// D (+)= A * B with A (16-bit pairs) in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(acc), "r"(leader));
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc::smem_u32(bar)), "r"(leader)
      : "memory");
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// V as the MN-major B operand: 64-wide atoms side by side (the leading offset), 8 keys each 1024 bytes
// (the stride offset).
__device__ __forceinline__ uint64_t v_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)(kAtom >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Wait, within the limit, for a phase whose copies are in flight, whatever the abort flag says.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity) {
  const unsigned long long t0 = tc::globaltimer();
  while (!tc::mbar_try_wait(bar, parity) && tc::globaltimer() - t0 < tc::kWaitLimitNs) {
  }
}

// Waits for work items last as long as items do: up to a minute, ended by the abort flag that any other
// expired wait (within seconds) raises.
__device__ __forceinline__ bool wait_item(uint64_t *bar, uint32_t parity, unsigned *status, unsigned site, volatile int *abort) {
  const unsigned long long t0 = tc::globaltimer();
  while (!tc::mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (tc::globaltimer() - t0 > 60000000000ull) return tc::mbar_wait(bar, parity, status, site, abort);
  }
  return true;
}

// A stream of n key blocks in the order of its use, the elements of block j: with wide v K0 V0 K1 V1 ...,
// else K0 K1 V0 K2 V1 ... V(n - 1).
template <bool kOverlay>
__device__ __forceinline__ int k_elem(int j) { return kOverlay ? 2 * j : max(0, 2 * j - 1); }
template <bool kOverlay>
__device__ __forceinline__ int v_elem(int j, int n) { return kOverlay ? 2 * j + 1 : min(2 * j + 2, 2 * n - 1); }

// ------------------------------------------------------------------ softmax of one key block
// This thread's row of scores from tensor memory, those at hi and past it -inf.
__device__ __forceinline__ void load_scores(uint32_t tS, float (&s)[kKeys], bool masked, int hi) {
  uint32_t raw[kKeys];
#pragma unroll
  for (int k = 0; k < kKeys; k += 32) tmem_ld32_async(tS + k, raw + k);
  tmem_wait_ld();
#pragma unroll
  for (int k = 0; k < kKeys; k += 32) tmem_landed(raw + k);
#pragma unroll
  for (int k = 0; k < kKeys; ++k) s[k] = __uint_as_float(raw[k]);
  if (masked) {
#pragma unroll
    for (int k = 0; k < kKeys; ++k)
      if (k >= hi) s[k] = -INFINITY;
  }
}

__device__ __forceinline__ float row_max(const float (&s)[kKeys]) {
  constexpr int n = 8;  // chains
  float m[n];
#pragma unroll
  for (int i = 0; i < n; ++i) m[i] = s[i];
#pragma unroll
  for (int k = n; k < kKeys; k += 2 * n)
#pragma unroll
    for (int i = 0; i < n; ++i) m[i] = k + n + i < kKeys ? max3(m[i], s[k + i], s[k + n + i]) : fmaxf(m[i], s[k + i]);
#pragma unroll
  for (int i = 1; i < n; ++i) m[0] = fmaxf(m[0], m[i]);
  return m[0];
}

// pk <- 2^(c s + negm) of the keys kA .. kB, two 16-bit values each, and their unrounded sums
template <bool kBF, int kA, int kB>
__device__ __forceinline__ void exponentials(const float (&s)[kKeys], float c, float negm, float2 (&sum)[2], uint32_t *pk) {
  const float2 c2 = make_float2(c, c), n2 = make_float2(negm, negm);
#pragma unroll
  for (int k = kA; k < kB; k += 2) {
    const float2 d = __ffma2_rn(make_float2(s[k], s[k + 1]), c2, n2);
    const float2 p = make_float2(ex2(d.x), ex2(d.y));
    sum[k / 2 % 2] = __fadd2_rn(sum[k / 2 % 2], p);
    pk[(k - kA) / 2] = pack2<kBF>(p.x, p.y);
  }
}
// ------------------------------------------------------------------ the kernel
template <bool kBF, int QA, int VA, bool kFew>
__global__ void __launch_bounds__(kThreads, 1)
    attn_packed_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const Args a) {
  using C = Cfg<QA, VA, kFew>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::bar);
  uint64_t *q_full = bars, *q_empty = bars + 2;          // [qbufs]
  uint64_t *s_full = bars + 4, *s_free = bars + 6;       // [2]: scores written / read (not with P over S)
  uint64_t *p_full = bars + 8;                           // [2 t + half]
  uint64_t *pv_done = bars + 12, *o_free = bars + 14;    // [2]
  uint64_t *item_full = bars + 16, *item_empty = bars + 20;  // [kItems]
  uint64_t *done = bars + 24, *block_full = bars + 25;
  uint64_t *kv_full = bars + 26, *kv_empty = kv_full + C::slots;
  uint64_t *half_done = bars + 60;                       // [2]: the first half's P V has ended (with P over S)
  static_assert(26 + 2 * C::slots <= 60, "barrier area");
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 62);
  volatile int *abort = reinterpret_cast<int *>(bars + 63);
  Item *items = reinterpret_cast<Item *>(smem + C::item);
  unsigned *status = g_status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    *abort = 0;
    for (int b = 0; b < C::qbufs; ++b) { tc::mbar_init(q_full + b, 1); tc::mbar_init(q_empty + b, 2); }
    for (int s = 0; s < C::slots; ++s) { tc::mbar_init(kv_full + s, 1); tc::mbar_init(kv_empty + s, 2); }
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(s_full + t, 1);
      tc::mbar_init(s_free + t, C::warps);
      tc::mbar_init(p_full + 2 * t, C::warps);
      tc::mbar_init(p_full + 2 * t + 1, C::warps);
      tc::mbar_init(pv_done + t, 1);
      tc::mbar_init(half_done + t, 1);
      tc::mbar_init(o_free + t, C::warps);
    }
    for (int i = 0; i < kItems; ++i) { tc::mbar_init(item_full + i, 1); tc::mbar_init(item_empty + i, 3 + 2 * C::warps); }
    tc::mbar_init(done, 2);
    tc::mbar_init(block_full, 1);
    tc::fence_barrier_init();
  }
  if (warp == 8) tc::tmem_alloc(tmem_slot, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  tc::griddep_wait();
  if (a.chunk) tc::griddep_launch_dependents();  // combine_kernel
  constexpr uint32_t kOCol = 256, kOStep = 64 * VA;

  // the n-th item, copied from the ring (release: and acknowledged); false when there is none left or a wait expired
  auto next_item = [&](int n, Item &it, bool release = true) {
    if (!wait_item(item_full + n % kItems, (n / kItems) & 1, status, 50, abort)) return false;
    it = items[n % kItems];
    __syncwarp();
    if (release && lane == 0) tc::mbar_arrive(item_empty + n % kItems);
    return !it.last;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIo));
    if (warp == 11) {
      // ---------------- items: a running prefix sum over 32 sequences at a time
      Walk walk = {};
      long long incl = 0;
      Seq s = {};
      auto load = [&]() {
        long long cnt = 0;
        if (walk.base + lane < a.seqs) {
          s = load_seq(a, walk.base + lane);
          cnt = seq_items(a, s);
        }
        incl = cnt;
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        walk.total = __shfl_sync(0xffffffffu, incl, 31);
      };
      load();
      long long it = blockIdx.x;
      for (int n = 0, asked = 0;; ++n) {
        if (!wait_item(item_empty + n % kItems, ((n / kItems) & 1) ^ 1, status, 51, abort)) break;
        Item item;
        item.last = 1;
        // the next block that has an item (the grid may have more blocks than there are items: those are
        // taken over too, and dropped)
        for (bool first = n == 0; it >= 0 && item.last; first = false) {
          if (!first) {
            if (lane == 0) {
              tc::fence_proxy_async();  // after the last answer was read
              tc::mbar_arrive_expect_tx(block_full, 16);
              take_block(smem + C::resp, block_full);
            }
            if (!tc::mbar_wait(block_full, asked & 1, status, 64, abort)) {
              drain(block_full, asked & 1);
              break;
            }
            ++asked;
            it = taken_block(smem + C::resp);
            __syncwarp();
            if (it < 0) break;
          }
          if (!find_sequences(walk, a.seqs, it, load)) continue;
          const long long r = it - walk.before;
          const int src = __ffs(__ballot_sync(0xffffffffu, incl > r)) - 1;
          Seq q;
          q.q0 = __shfl_sync(0xffffffffu, s.q0, src);
          q.nq = __shfl_sync(0xffffffffu, s.nq, src);
          q.k0 = __shfl_sync(0xffffffffu, s.k0, src);
          q.nk = __shfl_sync(0xffffffffu, s.nk, src);
          item = make_item(a, q, r - (__shfl_sync(0xffffffffu, incl, src) - seq_items(a, q)));
        }
        if (lane == 0) {
          items[n % kItems] = item;
          tc::mbar_arrive(item_full + n % kItems);
        }
        __syncwarp();
        if (item.last) break;
      }
    } else if (warp == 8) {
      // ---------------- bulk tensor loads
      Item it;
      int g = 0, qn = 0;  // ring slots filled, q buffers filled
      const uint32_t q_bytes = (uint32_t)(a.TQ * a.G) * 128 * QA;
      bool ok = true;
      for (int n = 0; ok && next_item(n, it, false); ++n) {
        const int n0 = it.u[0].nblk, n1 = it.u[1].nblk;
        // the acknowledgement lets the next item be taken: only when this one nears its end
        const int near_end = max(0, 2 * (max(n0, n1) - kAhead));
        if (lane == 0 && n0 + n1 == 0) tc::mbar_arrive(item_empty + n % kItems);
        if (lane == 0 && n0 + n1 > 0) {
          const int qb = qn % C::qbufs;
          if (!tc::mbar_wait(q_empty + qb, ((qn / C::qbufs) & 1) ^ 1, status, 52, abort)) ok = false;
          if (ok) {
            tc::mbar_arrive_expect_tx(q_full + qb, q_bytes * ((n0 > 0) + (n1 > 0)));
            for (int t = 0; t < 2; ++t)
              if (it.u[t].nblk > 0)
#pragma unroll
                for (int c = 0; c < QA; ++c)
                  tc::tma_load_4d(smem + C::q + qb * C::qbuf + (kFew ? 2 * c + t : t * QA + c) * C::tile, &tq, q_full + qb, 64 * c, 0,
                                  it.u[t].kvh, it.u[t].q_row);
          }
          // element e of unit t's stream into the next slot
          auto fill = [&](int t, int e, int nb) {
            const int s = g % C::slots;
            if (!tc::mbar_wait(kv_empty + s, ((g / C::slots) & 1) ^ 1, status, 53, abort)) return false;
            const bool is_k = C::overlay ? !(e & 1) : e == 0 || ((e & 1) && e != 2 * nb - 1);
            const int j = C::overlay ? e / 2 : is_k ? (e + 1) / 2 : e == 2 * nb - 1 ? nb - 1 : e / 2 - 1;
            const int atoms = is_k ? QA : VA;
            // a range's last block of up to 64 keys loads no more
            const int halves = it.u[t].klen - j * kKeys > kHalf ? 2 : 1;
            tc::mbar_arrive_expect_tx(kv_full + s, atoms * halves * (kAtom / 2));
            for (int c = 0; c < atoms; ++c)
              for (int h = 0; h < halves; ++h)
                tc::tma_load_3d(smem + C::kv + s * C::slot + c * kAtom + h * (kAtom / 2), is_k ? &tk : &tv, kv_full + s, 64 * c,
                                it.u[t].kvh, it.u[t].k_row + j * kKeys + h * kHalf);
            ++g;
            return true;
          };
          const int nmax = max(n0, n1);
          for (int e = 0; ok && e < 2 * nmax; ++e) {
            if (e == near_end) tc::mbar_arrive(item_empty + n % kItems);
            if (it.shared || e < 2 * n0) ok = fill(0, e, it.shared ? nmax : n0);
            if (ok && !it.shared && e < 2 * n1) ok = fill(1, e, n1);
          }
          ++qn;
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      }
      if (*abort && lane == 0) {  // gave up: the copies in flight land before the memory is given back
        for (int b = 0; b < C::qbufs && b < qn; ++b) drain(q_full + b, ((qn - 1 - b) / C::qbufs) & 1);
        for (int i = 0; i < C::slots && i < g; ++i) drain(kv_full + (g - 1 - i) % C::slots, ((g - 1 - i) / C::slots) & 1);
      }
    } else {
      // ---------------- matrix instructions of unit t
      const int t = uniform(warp - 9);
      const uint32_t leader = elect_lane();
      Item it;
      const uint32_t id_s = tc::idesc_f16(kRows, kKeys, false, kBF), id_s64 = tc::idesc_f16(kRows, kHalf, false, kBF);
      const uint32_t id_pv = tc::idesc_f16(kRows, (a.v_width + 15) / 16 * 16, true, kBF);
      const int qk_steps = (a.width + 15) / 16;
      const uint32_t tS = tmem + 128 * t, tO = tmem + kOCol + kOStep * t;
      const uint32_t tP = C::overlay ? tS : tmem + 384 + 64 * t;
      int ring = 0, qn = 0;             // next ring slot, q buffer
      uint32_t ring_phase = 0, q_phase = 0, units = 0, blocks = 0;  // parities: of those, and of this unit's
      uint32_t half_phase = 0;
      bool half_open = false;  // a P V that reads P over S was queued and not waited for
      const uint64_t p_desc = tc::sw128_kmajor_desc(tc::smem_u32(smem + C::p) + (kFew ? 0 : t * C::tile));
      // operand descriptors at the first byte of their areas: an offset adds to the address field (bytes
      // / 16, below 2^14 within shared memory)
      const uint64_t q_desc = tc::sw128_kmajor_desc(tc::smem_u32(smem + C::q) + t * C::unit);
      const uint64_t k_desc = tc::sw128_kmajor_desc(tc::smem_u32(smem + C::kv)), v_desc0 = v_desc(tc::smem_u32(smem + C::kv));
      bool ok = true;
      for (int n = 0; ok && next_item(n, it); ++n) {
        const int n0 = uniform(it.u[0].nblk), n1 = uniform(it.u[1].nblk), shared = uniform(it.shared);
        const int nb = t ? n1 : n0;
        const int all = shared ? max(n0, n1) : nb;                   // blocks of the stream
        const int others = shared ? 0 : 2 * (t ? n0 : n1);           // ring slots of the other unit's
        const int used = 2 * all + others;
        if (used == 0) continue;
        const int klen = uniform(t ? it.u[1].klen : it.u[0].klen);
        // the keys that any token of the tile sees
        const int seen = uniform(min(klen, t ? it.u[1].lim0 + it.u[1].ntok - 1 : it.u[0].lim0 + it.u[0].ntok - 1));
        int at = 0;  // slots of this item acknowledged or taken
        auto full = [&]() { return tc::mbar_wait(kv_full + ring, ring_phase, status, 54, abort); };
        auto advance = [&]() {
          ++at;
          if (++ring == C::slots) {
            ring = 0;
            ring_phase ^= 1;
          }
        };
        // acknowledges the slots before place `to`, which this unit does not read, as they arrive
        auto pass = [&](int to) {
          while (at < to) {
            if (!full()) return false;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(kv_empty + ring);
            advance();
          }
          return true;
        };
        // waits for element e of the own stream (the two streams take turns while both last): its
        // slot, or -1
        auto take = [&](int e) {
          if (!pass(e + min(e + t, others)) || !full()) return -1;
          const int sl = ring;
          advance();
          return sl;
        };
        // scores of block j.  With wide v they overwrite the half of P that the P V queued before reads: matrix
        // instructions of one thread are only promised to run in order where they share an accumulator, so that P V is
        // waited for (its 64 keys, while the softmax works on the second half).
        auto issue_s = [&](int j, int sl) {
          if (half_open) {
            if (!tc::mbar_wait(half_done + t, half_phase, status, 65, abort)) return false;
            half_phase ^= 1;
            half_open = false;
          }
          tc::tc_fence_after();
          const uint32_t id = klen - j * kKeys > kHalf ? id_s : id_s64;
          const uint64_t qd = q_desc + ((qn * C::qbuf) >> 4), kd = k_desc + ((sl * C::slot) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4 * QA; ++kk)
            if (kk < qk_steps)
              mma_ss(leader, tS, qd + (((kk / 4) * C::step + (kk % 4) * 32) >> 4),
                     kd + (((kk / 4) * kAtom + (kk % 4) * 32) >> 4), id, kk != 0);
          commit(leader, s_full + t);
          commit(leader, kv_empty + sl);
          if (j == nb - 1) commit(leader, q_empty + qn);
          return true;
        };
        if (!tc::mbar_wait(q_full + qn, q_phase, status, 55, abort)) { ok = false; break; }
        if (nb == 0 && lane == 0) tc::mbar_arrive(q_empty + qn);
        if (nb > 0) {
          const int sk = take(k_elem<C::overlay>(0));
          // (S_t was read by the previous unit's last softmax: its P V has been queued)
          if (sk < 0 || !issue_s(0, sk)) { ok = false; break; }
        }
        for (int j = 0; j < nb; ++j) {
          int sk = 0, sl = 0;
          if (!C::overlay && j + 1 < nb) {
            sk = take(k_elem<false>(j + 1));
            if (sk < 0 || !tc::mbar_wait(s_free + t, blocks, status, 57, abort) || !issue_s(j + 1, sk)) { ok = false; break; }
          }
          sl = take(v_elem<C::overlay>(j, all));
          if (C::overlay && sl >= 0 && j + 1 < nb) sk = take(k_elem<true>(j + 1));  // ahead of the wait for P
          if (sl < 0 || sk < 0) { ok = false; break; }
          const int live = min(kKeys, klen - j * kKeys);               // the range's rows of this block
          const int steps = (min(kKeys, seen - j * kKeys) + 15) / 16;  // 16-key steps that some token sees
          if (live < 16 * steps) {
            // rows of no sequence: zeros, whatever they hold (both units of a pair write the same zeros)
            uint8_t *vs = smem + C::kv + sl * C::slot;
            const int rows = 16 * steps - live;
            for (int c = lane; c < rows * 8 * VA; c += 32)
              *reinterpret_cast<uint4 *>(vs + (c / (rows * 8)) * kAtom + (live + (c / 8) % rows) * 128 + (c % 8) * 16) =
                  make_uint4(0, 0, 0, 0);
            tc::fence_proxy_async();
            __syncwarp();
          }
          const uint64_t vd = v_desc0 + ((sl * C::slot) >> 4);
          if ((j == 0 && !tc::mbar_wait(o_free + t, units ^ 1, status, 59, abort)) ||
              !tc::mbar_wait(p_full + 2 * t, blocks, status, 58, abort)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (kk < steps) mma_ts(leader, tO, tP + 8 * kk, vd + ((kk * 2048) >> 4), id_pv, j != 0 || kk != 0);
          if (C::overlay) {
            commit(leader, half_done + t);
            half_open = true;
            if (j + 1 < nb && !issue_s(j + 1, sk)) { ok = false; break; }
          }
          if (!tc::mbar_wait(p_full + 2 * t + 1, blocks, status, 58, abort)) { ok = false; break; }
          tc::tc_fence_after();
#pragma unroll
          for (int kk = 4; kk < 8; ++kk)
            if (kk < steps) {
              if (C::overlay) mma_ss(leader, tO, p_desc + (((kk - 4) * 32) >> 4), vd + ((kk * 2048) >> 4), id_pv, 1);
              else mma_ts(leader, tO, tP + 8 * kk, vd + ((kk * 2048) >> 4), id_pv, 1);
            }
          commit(leader, pv_done + t);
          commit(leader, kv_empty + sl);
          blocks ^= 1;
        }
        // what is left of the item is the other unit's
        if (ok && !pass(used)) ok = false;
        qn = qn + 1 == C::qbufs ? 0 : qn + 1;
        q_phase ^= qn == 0;
        units ^= nb > 0;
      }
      commit(leader, done);
      tc::mbar_wait(done, 0, status, 60, abort);
      if (*abort && lane == 0) drain(done, 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ---------------- softmax and output of unit t: row r of the tile, in tensor memory's lanes from `first` on
    const int t = warp >> 2, first = 32 * (warp & 3), r = kFew ? lane : first + lane;
    const int tok = r / a.G, head = r - tok * a.G;
    const uint32_t lane_off = (uint32_t)first << 16;
    const uint32_t tS = tmem + 128 * t + lane_off, tO = tmem + kOCol + kOStep * t + lane_off;
    const uint32_t tP = C::overlay ? tS : tmem + 384 + 64 * t + lane_off;
    const float c = a.scale_log2;
    uint32_t blocks = 0;  // of this unit in all
    Item it;
    for (int n = 0; (!kFew || (warp & 3) == t) && next_item(n, it); ++n) {
      const int nb = it.u[t].nblk;
      const bool row = tok < it.u[t].ntok && r < a.TQ * a.G;
      const bool live = __any_sync(0xffffffffu, row);  // a warp without rows only keeps the barriers going
      // the keys this row sees (a row that is none needs no mask)
      const int vis = row ? max(0, min(it.u[t].klen, it.u[t].lim0 + tok)) : 0x7fffffff;
      const int min_vis = __reduce_min_sync(0xffffffffu, vis);
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < nb; ++j, ++blocks) {
        if (!tc::mbar_wait(s_full + t, blocks & 1, status, 61, abort)) { ok = false; break; }
        tc::tc_fence_after();
        if (!live) {
          // its arrival for this block must not count for the one before: that block's P V has ended
          if (!C::overlay && lane == 0) tc::mbar_arrive(s_free + t);
          if (j > 0 && !tc::mbar_wait(pv_done + t, (blocks - 1) & 1, status, 62, abort)) { ok = false; break; }
          __syncwarp();
          if (lane == 0) {
            tc::mbar_arrive(p_full + 2 * t);
            tc::mbar_arrive(p_full + 2 * t + 1);
          }
          continue;
        }
        const int hi = vis - j * kKeys;
        const bool masked = min_vis - j * kKeys < kKeys;
        float sv[kKeys];
        load_scores(tS, sv, masked, hi);
        if (!C::overlay) {
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(s_free + t);
        }
        const float bm = row_max(sv);
        bool need = false;
        float alpha = 1.f;
        if (j == 0) {
          m = bm;
        } else {
          need = row && (bm - m) * c > kRescaleLog2;  // also from -inf, whose l and O are zero
          if (need) {
            alpha = ex2((m - bm) * c);
            l *= alpha;
            m = bm;
          }
        }
        const bool any_need = __any_sync(0xffffffffu, need);
        // p = 2^(c s - c m + kUp), rounded to the type's pairs for the second product; l sums them unrounded
        const float negm = m == -INFINITY ? 0.f : fmaf(-m, c, kUp<kBF>);
        float2 sum[2] = {};
        uint32_t pk[kHalf / 2];
        exponentials<kBF, 0, kHalf>(sv, c, negm, sum, pk);
        // What P and O were used for before: with narrow v the previous block's P V read all of P_t; with
        // wide v it read the second half's place, while the first half's is this block's own S_t.
        auto previous_pv = [&]() { return j == 0 || tc::mbar_wait(pv_done + t, (blocks - 1) & 1, status, 62, abort); };
        if ((!C::overlay || any_need) && !previous_pv()) { ok = false; break; }
        tc::tc_fence_after();
#pragma unroll
        for (int k = 0; k < kHalf / 2; k += 8) tmem_st8(tP + k, pk + k);
        if (any_need) {  // O_t moves to the new maximum
#pragma unroll
          for (int k = 0; k < 64 * VA; k += 8) tmem_scale8(tO + k, alpha);
        }
        uint32_t pk1[kHalf / 2];
        // (the store's latency under the second half's first exponentials)
        exponentials<kBF, kHalf, kHalf + kLate>(sv, c, negm, sum, pk1);
        tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_full + 2 * t);
        exponentials<kBF, kHalf + kLate, kKeys>(sv, c, negm, sum, pk1 + kLate / 2);
        if (C::overlay) {
          if (!previous_pv()) { ok = false; break; }
          uint8_t *pr = smem + C::p + ((kFew ? 0 : t * kRows) + first + lane) * 128;  // 128-byte rows of 64 keys, 16-byte chunk i of row r at i ^ (r % 8)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4 *>(pr + ((k ^ (r & 7)) << 4)) = make_uint4(pk1[4 * k], pk1[4 * k + 1], pk1[4 * k + 2], pk1[4 * k + 3]);
          tc::fence_proxy_async();
        } else {
#pragma unroll
          for (int k = 0; k < kHalf / 2; k += 8) tmem_st8(tP + kHalf / 2 + k, pk1 + k);
          tmem_wait_st();
          tc::tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_full + 2 * t + 1);
        const float2 s2 = __fadd2_rn(sum[0], sum[1]);
        l += s2.x + s2.y;
      }
      if (!ok) break;
      if (nb > 0) {
        if (!tc::mbar_wait(pv_done + t, (blocks - 1) & 1, status, 63, abort)) break;
        tc::tc_fence_after();
      }
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // a row that saw no key: zeros
      const long long at = (long long)it.u[t].q_row + tok;
      const int h = it.u[t].kvh * a.G + head, size = it.partial ? 4 : 2;
      // With whole tiles and wide v the output goes by 128 bytes of each row through this warp's rows of the P area (the
      // last P V has read it), so that a store instruction writes whole pieces of 4 rows: 16 bytes of 32 rows
      // at a time took 9000 clk a tile of 128 columns.  Otherwise rows are stored as they are.
      constexpr bool kStage = VA == 2 && !kFew;
      unsigned long long mine = 0;
      if (row)
        mine = it.partial ? reinterpret_cast<unsigned long long>(a.part + (((long long)it.u[t].split * a.q_rows + at) * a.heads + h) * a.v_width)
                          : reinterpret_cast<unsigned long long>(static_cast<uint16_t *>(a.out) + at * a.out_token_stride + h * a.out_head_stride);
      uint8_t *stage = smem + C::p + (t * kRows + first) * 128;
#pragma unroll 1
      for (int i = 0; i < 64 * VA; i += 32) {
        if (!live || i >= a.v_width) break;
        float v[32];
        if (nb > 0) tc::tmem_ld32(tO + i, v);
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = inv == 0.f ? 0.f : v[k] * inv;
        // chunk: 16 bytes of the row from this pass's first
        auto put = [&](int chunk, uint4 u) {
          if constexpr (!kStage) {
            const int byte = i * size + chunk * 16;
            if (mine != 0 && byte < a.v_width * size) *reinterpret_cast<uint4 *>(mine + byte) = u;
          } else {
            const int c = it.partial ? chunk : (i & 32) / 8 + chunk;
            *reinterpret_cast<uint4 *>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) = u;
          }
        };
        if (it.partial) {
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            put(k / 4, make_uint4(__float_as_uint(v[k]), __float_as_uint(v[k + 1]), __float_as_uint(v[k + 2]), __float_as_uint(v[k + 3])));
        } else {
#pragma unroll
          for (int k = 0; k < 32; k += 8)
            put(k / 8, make_uint4(pack2<kBF>(v[k], v[k + 1]), pack2<kBF>(v[k + 2], v[k + 3]), pack2<kBF>(v[k + 4], v[k + 5]),
                                  pack2<kBF>(v[k + 6], v[k + 7])));
        }
        __syncwarp();
        if (kStage && (it.partial || (i & 32) || i + 32 >= a.v_width)) {
          const int byte = (it.partial ? i * 4 : (i & ~63) * 2) + (lane & 7) * 16;  // within the row
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += 4) {
            const int rr = r0 + (lane >> 3);
            const unsigned long long to = __shfl_sync(0xffffffffu, mine, rr);
            if (to != 0 && byte < a.v_width * size)
              *reinterpret_cast<uint4 *>(to + byte) = *reinterpret_cast<const uint4 *>(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
          }
          __syncwarp();
        }
      }
      if (nb > 0) {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(o_free + t);
      }
      if (row) {
        if (it.partial)
          a.part_lse[((long long)it.u[t].split * a.q_rows + at) * a.heads + h] = l > 0.f || l != l ? m * c + (log2f(l) - kUp<kBF>) : -INFINITY;
        else if (a.lse)
          a.lse[at * a.heads + h] = l > 0.f || l != l ? m * a.scale + logf(l * exp2f(-kUp<kBF>)) : -INFINITY;
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins the key ranges of the sequences that were split: kWarps warps a (query row, head), each taking every
// kWarps-th range; weights 2^(L_s - max L) of the ranges' log2 sums, added in a fixed order.
template <bool kBF, int kWarps>
__global__ void __launch_bounds__(128) combine_kernel(const Args a) {
  __shared__ float4 part[4][32];
  __shared__ float weight[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long n = (long long)a.q_rows * a.heads;
  constexpr int kRowsBlock = 4 / kWarps;
  tc::griddep_wait();
  for (long long i0 = (long long)blockIdx.x * kRowsBlock; i0 < n; i0 += (long long)gridDim.x * kRowsBlock) {
    const long long i = i0 + warp / kWarps;
    const long long tok = min(i, n - 1) / a.heads;
    int lo = 0, hi = a.seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.q_offsets[mid] <= tok) lo = mid;
      else hi = mid;
    }
    const Seq s = load_seq(a, lo);
    const int ns = range_count(a, s.nk);
    const bool row = i < n && tok >= s.q0 && tok < s.q0 + s.nq && ns > 1;  // else of no sequence, or already written
    float top = -INFINITY, total = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row) {
      for (int k = lane; k < ns; k += 32) top = fmaxf(top, a.part_lse[k * n + i]);
      for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const float base = top == -INFINITY ? 0.f : top;
      for (int k0 = 0; k0 < ns; k0 += 32) {
        const float mine = k0 + lane < ns ? a.part_lse[(k0 + lane) * n + i] : -INFINITY;
        const float wl = mine == -INFINITY ? 0.f : ex2(mine - base);  // NaN stays
        const int cnt = min(32, ns - k0);
#pragma unroll 4
        for (int k = warp % kWarps; k < cnt; k += kWarps) {
          const float w = __shfl_sync(0xffffffffu, wl, k);
          if (w != 0.f) {  // (a range without keys left no output)
            total += w;
            if (4 * lane < a.v_width) {
              const float4 p = *reinterpret_cast<const float4 *>(a.part + ((k0 + k) * n + i) * a.v_width + 4 * lane);
              o.x = fmaf(w, p.x, o.x);
              o.y = fmaf(w, p.y, o.y);
              o.z = fmaf(w, p.z, o.z);
              o.w = fmaf(w, p.w, o.w);
            }
          }
        }
      }
    }
    if constexpr (kWarps > 1) {
      __syncthreads();
      part[warp][lane] = o;
      if (lane == 0) weight[warp] = total;
      __syncthreads();
      if (warp == 0) {
        for (int w = 1; w < 4; ++w) {
          const float4 p = part[w][lane];
          o.x += p.x, o.y += p.y, o.z += p.z, o.w += p.w;
          total += weight[w];
        }
      }
    }
    if (!row || warp % kWarps) continue;
    const bool any = total > 0.f || total != total;
    const float inv = any ? 1.f / total : 0.f;
    const long long h = i - tok * a.heads;
    if (4 * lane < a.v_width)
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + tok * a.out_token_stride + h * a.out_head_stride + 4 * lane) =
          make_uint2(pack2<kBF>(o.x * inv, o.y * inv), pack2<kBF>(o.z * inv, o.w * inv));
    if (a.lse && lane == 0) a.lse[i] = any ? (top + log2f(total)) * 0.6931471805599453f : -INFINITY;
  }
}

int current_device() {
  int dev = 0;
  cudaGetDevice(&dev);
  return dev;
}

template <bool kBF, int QA, int VA, bool kFew>
cudaError_t launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const Args &a, int grid, cudaStream_t st) {
  auto *k = attn_packed_kernel<kBF, QA, VA, kFew>;
  const int smem = Cfg<QA, VA, kFew>::total + 1024;
  static std::atomic<unsigned long long> ready{0};  // devices whose limits are set
  const int dev = current_device();
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, k);
    if (e == cudaSuccess && fa.numRegs < kRegsLaunch) e = cudaErrorLaunchOutOfResources;  // the register split would wait for good
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  k<<<grid, kThreads, smem, st>>>(tq, tk, tv, a);
  return cudaGetLastError();
}

// Sequences whose queries fill no more than 32 rows of a tile on average (single new tokens) take tiles of 32 (32 tokens
// over 500 to 8191 keys 106 us against 145 with 128 rows, 64 over 2000 92 and 116; with a piece of 256 more among them
// 116 and 117).
bool few_rows(const mrf_attention_args &a) { return a.q_rows * (a.heads / a.kv_heads) <= 32ll * a.seqs && a.heads / a.kv_heads <= 32; }
int tile_tokens(const mrf_attention_args &a) { return (few_rows(a) ? 32 : kRows) / (a.heads / a.kv_heads); }

// (about 2 us a block: see the head of this file)
AttentionSplit split_of(const mrf_attention_args &a) { return attention_split(a, tile_tokens(a), a.kv_heads, 2.0); }

bool mult8(long long n, long long stride) { return n <= 1 || (stride > 0 && stride % 8 == 0); }

}  // namespace

int sm_count() {
  static std::atomic<int> known[64];
  const int dev = current_device();
  int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 148;
  }
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

bool attention_tc_takes(const mrf_attention_args &a) {
  if (a.dtype != MRF_DTYPE_F16 && a.dtype != MRF_DTYPE_BF16) return false;
  if (a.width > 128 || a.v_width > 128 || a.width % 8 || a.v_width % 8 || a.heads / a.kv_heads > kRows) return false;
  const long long big = INT32_MAX - 65536;
  if (a.k_rows < 1 || a.k_rows > big || a.q_rows * a.heads > big || (a.q_rows + a.seqs) * (long long)a.kv_heads * 64 > big) return false;
  for (const void *p : {a.q, a.k, a.v, (const void *)a.out})
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return mult8(a.q_rows, a.q_token_stride) && mult8(a.heads, a.q_head_stride) && mult8(a.k_rows, a.k_token_stride) &&
         mult8(a.kv_heads, a.k_head_stride) && mult8(a.k_rows, a.v_token_stride) && mult8(a.kv_heads, a.v_head_stride) &&
         mult8(a.q_rows, a.out_token_stride) && mult8(a.heads, a.out_head_stride);
}

AttentionSplit attention_split(const mrf_attention_args &a, int tokens, long long sets, double block) {
  const long long tiles = std::max<long long>(a.seqs, (a.q_rows + tokens - 1) / tokens), units = tiles * sets, sms = sm_count();
  const long long keys = a.max_k ? std::min(a.max_k, a.k_rows) : a.k_rows, blocks = (keys + kKeys - 1) / kKeys;
  // More units than SMs: only single tiles (new tokens) of long sequences whose lengths only the device knows,
  // where the longest would keep its SM while the others are done (32 sequences up to 8192 keys, 8 key
  // heads: 110 us against 142; up to 1024: 34 against 26).
  if (units > (tiles > a.seqs || a.seqs == 1 || blocks < 32 ? sms : 4 * sms)) return {0, 1};
  // One sequence: as many equal ranges as give every SM one item (two units).  Several: smaller ranges,
  // about eight rounds if all were as long as the longest.
  long long wanted = a.seqs == 1 ? 2 * (sms / units) : 16 * sms / units;
  // A range's output is written and read again in fp32, at about 2.5 TB/s, against the time of a key block:
  // the number of ranges where their sum is least.
  const double range = (double)a.q_rows * a.heads * a.v_width * 8 / 2.5e6;
  wanted = std::min<long long>(wanted, (long long)std::sqrt(blocks * block / range));
  if (wanted < 2) return {0, 1};
  long long chunk = (blocks + wanted - 1) / wanted;
  // (several sequences, 4 up to 8192 keys: at least 1, 2, 3, 4 blocks a range 36, 32, 31, 34 us)
  chunk = std::max<long long>({chunk, a.seqs == 1 ? 1 : 3, (blocks + 127) / 128});
  const long long most = (blocks + chunk - 1) / chunk;
  // and only where they gain on one range; 4 us for the joining launch (one sequence, 8 key heads: a token after 1024
  // keys 12 us against 22, 128 after 4000 34 and 65; a prompt of 1024 tokens would take 34 against 24)
  if (chunk * block + most * range + 4 >= blocks * block) return {0, 1};
  return {(int)(chunk * kKeys), (int)most};
}

size_t attention_tc_workspace(const mrf_attention_args &a) {
  const AttentionSplit s = split_of(a);
  return s.chunk ? (size_t)s.most * a.q_rows * a.heads * (a.v_width + 1) * sizeof(float) : 0;
}

bool launch_attention_packed_tc(const mrf_attention_args &m, cudaStream_t st, cudaError_t *err) {
  Args a;
  a.out = m.out;
  a.lse = m.lse;
  a.q_offsets = m.q_offsets;
  a.k_start = m.k_start;
  a.k_len = m.k_len;
  a.out_token_stride = m.out_token_stride;
  a.out_head_stride = m.out_head_stride;
  a.q_rows = (int)m.q_rows;
  a.k_rows = (int)m.k_rows;
  a.seqs = m.seqs;
  a.heads = m.heads;
  a.kv_heads = m.kv_heads;
  a.G = m.heads / m.kv_heads;
  a.TQ = tile_tokens(m);
  a.width = m.width;
  a.v_width = m.v_width;
  a.causal = m.causal != 0;
  const AttentionSplit split = split_of(m);
  a.chunk = split.chunk;
  a.max_splits = split.most;
  a.scale = m.scale;
  a.scale_log2 = m.scale * 1.4426950408889634f;
  a.part = static_cast<float *>(m.workspace);
  a.part_lse = a.part + (size_t)a.max_splits * a.q_rows * a.heads * a.v_width;

  // a dimension of one row needs no stride; the maps want a valid one
  auto st1 = [](long long n, long long s, int inner) { return (unsigned long long)(n <= 1 ? (inner + 7) / 8 * 8 : s); };
  using ull = unsigned long long;
  const ull qs_h = st1(m.heads, m.q_head_stride, m.width), qs_t = st1(m.q_rows, m.q_token_stride, m.width);
  const ull qd[4] = {(ull)m.width, (ull)a.G, (ull)m.kv_heads, (ull)m.q_rows}, qst[3] = {qs_h, qs_h * a.G, qs_t};
  const ull kd[3] = {(ull)m.width, (ull)m.kv_heads, (ull)m.k_rows};
  const ull kst[2] = {st1(m.kv_heads, m.k_head_stride, m.width), st1(m.k_rows, m.k_token_stride, m.width)};
  const ull vd[3] = {(ull)m.v_width, (ull)m.kv_heads, (ull)m.k_rows};
  const ull vst[2] = {st1(m.kv_heads, m.v_head_stride, m.v_width), st1(m.k_rows, m.v_token_stride, m.v_width)};
  const unsigned qbox[4] = {64, (unsigned)a.G, 1, (unsigned)a.TQ}, kbox[3] = {64, 1, kHalf};
  CUtensorMap tq, tk, tv;
  if (!make_tmap(&tq, m.q, kTmF16, 4, qd, qst, qbox, 128) || !make_tmap(&tk, m.k, kTmF16, 3, kd, kst, kbox, 128) ||
      !make_tmap(&tv, m.v, kTmF16, 3, vd, vst, kbox, 128))
    return false;
  // At least a block for each item.  Without splits: with at most q_rows / TQ + seqs tiles, pairs of them
  // for each key head and for every sequence's odd one half as many.  With splits, pairs of ranges.
  const long long tiles = m.q_rows / a.TQ + m.seqs;
  const long long items = a.chunk ? tiles * m.kv_heads * ((a.max_splits + 1) / 2)
                                  : tiles / 2 * m.kv_heads + std::min<long long>(m.seqs, tiles) * ((m.kv_heads + 1) / 2);
  const int grid = (int)std::max(1ll, items);
  const bool bf = m.dtype == MRF_DTYPE_BF16, few = few_rows(m), q2 = m.width > 64, v2 = m.v_width > 64;
#define MRF_ATTN(BF, FEW)                                                                                        \
  (q2 ? (v2 ? launch<BF, 2, 2, FEW>(tq, tk, tv, a, grid, st) : launch<BF, 2, 1, FEW>(tq, tk, tv, a, grid, st))   \
      : (v2 ? launch<BF, 1, 2, FEW>(tq, tk, tv, a, grid, st) : launch<BF, 1, 1, FEW>(tq, tk, tv, a, grid, st)))
  *err = bf ? (few ? MRF_ATTN(true, true) : MRF_ATTN(true, false)) : (few ? MRF_ATTN(false, true) : MRF_ATTN(false, false));
#undef MRF_ATTN
  if (*err != cudaSuccess || a.chunk == 0) return true;
  cudaLaunchConfig_t cfg = {};
  // many ranges: a block a row; few: a warp
  const bool wide = a.max_splits > 8;
  const long long rows = m.q_rows * m.heads;
  cfg.gridDim = dim3((unsigned)std::min<long long>(wide ? rows : (rows + 3) / 4, 16 * sm_count()));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (wide) *err = bf ? cudaLaunchKernelEx(&cfg, combine_kernel<true, 4>, a) : cudaLaunchKernelEx(&cfg, combine_kernel<false, 4>, a);
  else *err = bf ? cudaLaunchKernelEx(&cfg, combine_kernel<true, 1>, a) : cudaLaunchKernelEx(&cfg, combine_kernel<false, 1>, a);
  return true;
}

cudaError_t attention_tc_status(unsigned *word, cudaStream_t st) {
  unsigned w[2] = {0, 0};
  cudaError_t e = cudaMemcpyFromSymbolAsync(w, g_status, sizeof w, 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && w[0] != 0) {
    const unsigned zero[2] = {0, 0};
    e = cudaMemcpyToSymbolAsync(g_status, zero, sizeof zero, 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  word[0] = w[0];
  word[1] = w[1];
  return e;
}

}  // namespace mrf
