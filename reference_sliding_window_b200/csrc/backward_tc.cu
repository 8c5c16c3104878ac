// Gradient of the teacher-forced R-SWA attention on the 5th-generation tensor
// cores (tcgen05 + TMEM): bf16 tensors, head dim 64 or 128, float32
// accumulation.  The formulas, the mask and the work items are in backward.h.
//
// One CTA per SM, which takes (work item, head) pairs off a counter, heaviest
// first; tiles of 128 queries x 128 keys.  Bound: the tensor pipe (4 tile
// products per tile pair in a dK, dV item, 3 in a dQ item) and the operands it
// reads from shared memory, with the exponentials close behind.  Measured at
// 12832 + 19936 rows, 10 heads, d = 128: 3320 cycles a tile pair in dK, dV
// items and 2440 in dQ items, of 2048 and 1536 at the MMA's rate; 5.5 to 5.8 ms
// in a stream of calls, whose clock the power limit lowers (4.9 to 5.3 ms for the
// first ones): 750 to 790 TFLOP/s of the five products that the gradient cannot
// do without.
//
// * A dK, dV item keeps its K and V tiles in shared memory and streams Q and
//   dO tiles.  S and dP are formed transposed (keys on TMEM lanes), so that P
//   and dS, bf16 pairs written over S's columns, are at once the A operands
//   (read from TMEM) of dV += P^T dO and dK += dS^T Q, whose B operands are
//   the streamed tiles themselves.
// * A dQ item keeps its Q and dO rows in TMEM, as the A operands of S = Q K^T and
//   dP = dO V^T, streams K and V, and adds dQ += dS K with dS written over dP.
//   An MMA that reads both operands from shared memory takes 90 cycles
//   instead of 64 (16 KB of operands at 128 bytes a cycle, and the ring's
//   writes); with A in TMEM it takes 68.  A dK, dV item has no TMEM left for it.
// * Warp 0 streams tiles with TMA (128-byte swizzle) through two rings, warp
//   1 issues the MMAs, warp 2 stages the row statistics (dK, dV items, where
//   they vary along a thread's columns), warps 3-18 are the softmax: four
//   groups of 128 threads, each for a quarter of the 128 score columns.
// * Issue order of a dK, dV item, two score regions X, Y taking turns: S(i)
//   in one, dP(i) in the other, then dV(i), which runs while the softmax reads
//   dP(i), S(i+1) over the dP(i) just read, dK(i) and dP(i+1), under which it forms
//   P(i+1).  (S(i+1) before dV(i) left the tensor pipe idle while dP(i) was read:
//   4100 cycles a tile pair.)  A dQ item: S(i+1) as soon as S(i) is read, dQ(i),
//   dP(i+1) over the dS(i) just used.
// * P and dS are rounded to bf16 for the products, as the tensor cores take
//   them (relative error 2^-8 at most on each term of sums of independent
//   terms); dS is formed from the float32 P.
// * Rows of a streamed tile past the document's end belong to the next
//   document.  Their weights are exactly 0, but 0 times an infinity is NaN, so
//   the softmax clears them in shared memory before the products read them.
// * The producer takes the next item while the last tiles of the current one are
//   computed and starts its loads (a load under way from memory takes 2 to 3
//   us, as long as a short document's whole item): every role walks the items
//   by itself, and barriers, not the CTA's start, order one item's use of a tile,
//   a region or an accumulator before the next one's.
// * Every wait is bounded.  A CTA in which one ran out writes the rows of the
//   items that it holds as NaN, and then those of every item still on the list
//   (which other CTAs may not live to take): no row keeps what was there before.

#include <math.h>

#include <algorithm>

#include "backward.h"
#include "launch.cuh"
#include "tc.cuh"

namespace rswa {
namespace tc {
namespace {

constexpr int kThreads = 608;
constexpr int kSoftmaxWarp = 3;
constexpr int kSoftmaxThreads = 512;
constexpr int kCols = 32;  // score columns of a softmax thread's fragments
constexpr int kTmemCols = 512;
constexpr uint32_t kColA = 256;  // dQ items: the rows of Q, then of dO, bf16 pairs

struct BwdTcParams {
  CUtensorMap tmQ, tmK, tmV, tmG;  // packed [L][H][D] maps; G is dO
  BackwardParams b;
  float scale_log2;
  int n_items;  // work entries x heads
};

template <int D>
struct Cfg {
  static constexpr int kBoxes = D / kBox;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  // Ring A: K tiles (dQ items) or Q tiles, read by S and again, a tile's
  // softmax later, by dQ or dK; ring B: V or dO tiles.  Two stages of ring A are
  // too few: the tile after next then waits for its load (a dK, dV tile pair
  // took 4560 cycles with two stages).
  static constexpr int kA = D == 128 ? 3 : 4, kB = D == 128 ? 2 : 4;
  static constexpr int kSmRes = 0;
  static constexpr int kSmA = kSmRes + 2 * kTileBytes;
  static constexpr int kSmB = kSmA + kA * kTileBytes;
  // statistics of two streamed query tiles (dK, dV items)
  static constexpr int kSmStats = kSmB + kB * kTileBytes;
  static constexpr int kSmBar = kSmStats + 2 * 1024;
  static constexpr int kSmBytes = kSmBar + 512;
};
static_assert(Cfg<128>::kSmBytes <= 232448 && Cfg<64>::kSmBytes <= 232448, "shared memory of an SM");

// A wait names one of a barrier's two phases, so a barrier's next phase but one
// must not complete while a waiter has still to see this one.  S, P and dS take
// two barriers in turn; everything else is ordered by the next use of the ring,
// region, tile or slot that it guards.  Phases count over all items of the CTA.
enum : int {
  kBarRes = 0,        // 2: the item's own tiles have landed (K, V or Q, dO)
  kBarResFree = 2,    // they may be overwritten
  kBarRows = 3,       // dQ items: Q and dO are in TMEM
  kBarAccFree = 4,    // the item's accumulators have been read
  kBarItem = 5,       // 2: the next item's number is in its slot
  kBarItemFree = 7,   // 2: every role is done with the item
  kBarAFull = 9,      // 4
  kBarAFree = 13,     // 4
  kBarBFull = 17,     // 4
  kBarBFree = 21,     // 4
  kBarS = 25,         // 2
  kBarP = 27,         // 2 (dK, dV items)
  kBarDS = 29,        // 2
  kBarDP = 31,
  kBarRead = 32,      // dK, dV items: dP is read; dQ items: S is
  kBarFinal = 33,     // the item's last MMA is done
  kBarFinalV = 34,    // dK, dV items: the last into dV is
  kBarStats = 35,     // 2 (dK, dV items)
  kBarStatsFree = 37, // 2
  kBarEnd = 39,
  kSlotTmem = 40, kSlotAbort = 41, kSlotItem = 42,  // 2 x 64 bytes: Item::Slot
  kSlotLeft = 58      // an item that was taken and not announced, or -1
};

constexpr uint32_t idesc(int n, bool b_n_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24) |
         (b_n_major ? 1u << 16 : 0u);
}

// The MMA warp runs these with all lanes, so that descriptors and addresses
// stay in uniform registers; the instruction itself issues on the one lane
// with lead != 0 (always the same: a commit covers its own thread's MMAs).
__device__ __forceinline__ void mma_ss(int lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(int lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit(int lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(lead)
      : "memory");
}

// D (TMEM) = A B^T over the head dim, both tiles K-major in shared memory.
template <int D>
__device__ __forceinline__ void mma_scores(int lead, uint32_t tmem_d, uint32_t a, uint32_t b) {
  const uint64_t da = smem_desc(a, 16, 1024), db = smem_desc(b, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4;
    mma_ss(lead, tmem_d, da + off, db + off, idesc(kTile, false), kk > 0);
  }
}

// The same with A's rows (bf16 pairs) in TMEM.
template <int D>
__device__ __forceinline__ void mma_scores_ta(int lead, uint32_t tmem_d, uint32_t tmem_a, uint32_t b) {
  const uint64_t db = smem_desc(b, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    mma_ts(lead, tmem_d, tmem_a + kk * 8, db + (((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4), idesc(kTile, false),
           kk > 0);
}

// D (TMEM, 128 x D) += A B: A 128 x 128 bf16 pairs in TMEM, 32 columns of it at
// tmem_a, the next 32 kCols TMEM columns on, ...; B a tile's rows.
template <int D>
__device__ __forceinline__ void mma_grad(int lead, uint32_t tmem_d, uint32_t tmem_a, uint32_t b, bool acc) {
  const uint64_t db = smem_desc(b, kBoxBytes, 1024);
#pragma unroll
  for (int kk = 0; kk < kTile / 16; ++kk)
    mma_ts(lead, tmem_d, tmem_a + (kk >> 1) * kCols + (kk & 1) * 8, db + ((kk * 2048) >> 4), idesc(D, true),
           kk > 0 ? 1u : acc);
}

// A warp's 32 lanes x 32 TMEM columns as MMA fragments: with g = lane / 4 and t
// = lane % 4, v[16 h + 4 k + r] is TMEM lane 16 h + 8 (r / 2) + g, column 8 k +
// 2 t + r % 2.  A thread then holds 4 rows of 8 columns, so a value that
// belongs to a column is read from shared memory once for 4 elements (one row
// of 32 columns a thread read 128 bits for 4 elements, and those reads,
// 1024 cycles a tile pair, delayed the MMAs' own).
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float* v) {
  uint32_t r[32];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[16 * h]), "=r"(r[16 * h + 1]), "=r"(r[16 * h + 2]), "=r"(r[16 * h + 3]), "=r"(r[16 * h + 4]),
          "=r"(r[16 * h + 5]), "=r"(r[16 * h + 6]), "=r"(r[16 * h + 7]), "=r"(r[16 * h + 8]), "=r"(r[16 * h + 9]),
          "=r"(r[16 * h + 10]), "=r"(r[16 * h + 11]), "=r"(r[16 * h + 12]), "=r"(r[16 * h + 13]),
          "=r"(r[16 * h + 14]), "=r"(r[16 * h + 15])
        : "r"(taddr + ((uint32_t)(16 * h) << 16)));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// The same elements rounded to bf16 pairs, into 16 columns of the 32 lanes.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const float* v) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[16 * h + 2 * i], v[16 * h + 2 * i + 1]);
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                     taddr + ((uint32_t)(16 * h) << 16)),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  }
}

// Two floats at a time (the same roundings per element).
__device__ __forceinline__ void fma2(float& x0, float& x1, float m, float a0, float a1) {
  unsigned long long x, mm, a;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(mm) : "f"(m));
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(x) : "l"(mm), "l"(a));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(x));
}
// p *= x + a
__device__ __forceinline__ void addmul2(float& p0, float& p1, float x0, float x1, float a0, float a1) {
  unsigned long long p, x, a;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(p0), "f"(p1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(a));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(p) : "l"(x));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(p0), "=f"(p1) : "l"(p));
}

// Bits [lo, hi) of 32.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  const uint32_t below_hi = hi <= 0 ? 0u : hi >= 32 ? ~0u : (1u << hi) - 1;
  const uint32_t below_lo = lo <= 0 ? 0u : lo >= 32 ? ~0u : (1u << lo) - 1;
  return below_hi & ~below_lo;
}
// A fragment's row i (of 4): its elements zeroed (whatever they hold, NaN
// included) where the bit of their column is clear.
__device__ __forceinline__ void keep_row(float* x, int i, uint32_t bits) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float& y = x[16 * (i >> 1) + 2 * (i & 1) + 4 * (e >> 1) + (e & 1)];
    y = bits & (1u << (8 * (e >> 1) + (e & 1))) ? y : 0.f;
  }
}

// Transposes the 4 x 4 words of a quad of lanes: q[j] of lane t becomes q[t] of lane j.
__device__ __forceinline__ void quad_transpose(uint32_t* q, int t) {
#pragma unroll
  for (int b = 1; b <= 2; b <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(i & b)) {
        const uint32_t x = __shfl_xor_sync(0xffffffffu, t & b ? q[i] : q[i | b], b);
        if (t & b) q[i] = x;
        else q[i | b] = x;
      }
}

__device__ __forceinline__ int ld_shared(uint32_t addr) {
  int v;
  asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared(uint32_t addr, int v) {
  asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void ld_shared4(uint32_t addr, int& a, int& b, int& c, int& d) {
  asm volatile("ld.volatile.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void st_shared4(uint32_t addr, int a, int b, int c, int d) {
  asm volatile("st.volatile.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ float2 ld_shared2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// A bounded wait (bar0: the barriers' base) that ends early once the CTA has
// given up.  What follows a failed first try is out of line: inlined at every
// wait it made up much of the kernel's code, which a launch fetches cold.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, uint32_t abort) {
  return !ld_shared(abort) && mbar_wait_bounded(bar, parity);
}
__device__ __forceinline__ bool wait_phase(uint32_t bar0, int slot, int phase) {
  const uint32_t bar = bar0 + 8u * slot;
  return mbar_try_wait(bar, phase & 1) || wait_on(bar, phase & 1, bar0 + 8u * kSlotAbort);
}

// What the producer announces of an item, four words at a time.  Every other
// role reads it from here: working it out of the launch's list takes a role
// hundreds of cycles, twice an item.
struct Item {
  int number, T, U, kq;      // -1: no more; tiles before it; of them dK, dV items' tiles; dQ items before it
  int start, len, ref, h;    // document and head
  int tile, dq, nt, part;    // its tile, kind, tiles of its sequence, partial
  int A, B0, lo, pad;        // tile lo + j of the sequence: its own number below A, B0 + (lo + j - A) from there on

  static __device__ __forceinline__ uint32_t slot(uint32_t bar0, int k) { return bar0 + 8u * kSlotItem + 64u * (k & 1); }
  __device__ __forceinline__ int at(int j) const { return lo + j < A ? lo + j : B0 + lo + j - A; }

  // Item k, read by all lanes of a warp; false: there is none.
  __device__ __forceinline__ bool next(uint32_t bar0, int k) {
    if (!__all_sync(0xffffffffu, wait_phase(bar0, kBarItem + (k & 1), k >> 1))) return false;
    read(slot(bar0, k));
    return number >= 0;
  }
  __device__ __forceinline__ void read(uint32_t s) {
    ld_shared4(s, number, T, U, kq);
    ld_shared4(s + 16, start, len, ref, h);
    ld_shared4(s + 32, tile, dq, nt, part);
    ld_shared4(s + 48, A, B0, lo, pad);
  }
  __device__ __forceinline__ void announce(uint32_t s) const {
    st_shared4(s + 16, start, len, ref, h);
    st_shared4(s + 32, tile, dq, nt, part);
    st_shared4(s + 48, A, B0, lo, pad);
    st_shared4(s, number, T, U, kq);
  }
  // Gives the slot back (one arrival per warp).
  static __device__ __forceinline__ void done(uint32_t bar0, int k, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar0 + 8u * (kBarItemFree + (k & 1)));
  }
};

// The softmax warps of an item: P and dS of every tile of its sequence, then
// the finished gradient tile from TMEM to memory.
template <int D, bool DQ>
__device__ __forceinline__ void softmax_item(uint32_t bar0, uint32_t tmem, const BwdTcParams& p, int item_k, bool& ok) {
  using C = Cfg<D>;
  constexpr int nA = C::kA, nB = C::kB;
  Item w;
  w.read(Item::slot(bar0, item_k));
  // Opaque, so that what follows from it is worked out per item, not kept in
  // registers over all of them for both kinds.
  int tid = threadIdx.x;
  asm volatile("" : "+r"(tid), "+r"(bar0), "+r"(tmem));
  const int warp = tid >> 5, lane = tid & 31;
  const int g = (warp - kSoftmaxWarp) >> 2;  // column quarter
  const int quarter = warp & 3;              // TMEM lanes 32 * quarter .. +31
  const int fg = lane >> 2, ft = lane & 3;   // the fragments' row and column pair
  const int c0 = kCols * g;
  const int own0 = w.tile * kTile + quarter * 32 + fg;  // the thread's local rows own0 + 8 i: queries (DQ) or keys
  const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16) + c0;
  const float sl2 = p.scale_log2;
  const bool bidir = p.b.bidir != 0;
  // After a timed-out wait a thread stops waiting but keeps arriving, so
  // the MMA thread is not left waiting on it; its rows are written as NaN.
  auto wait = [&](int slot, int phase) {
    if (ok && !wait_phase(bar0, slot, phase)) ok = false;
  };
  // A warp's arrival, once all of its lanes are there: an arrival per lane
  // costs an operation on the barrier's word each.
  auto arrive = [&](int slot) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar0 + 8u * slot);
  };
  if (DQ) {
    // The rows of Q and dO from their staged tiles into TMEM, as A operands: bf16
    // pairs as they lie in memory; a group takes an equal share of the words.
    constexpr int kWords = D * 128 / kSoftmaxThreads;  // of the D words of both rows
    const int row = quarter * 32 + lane, word0 = g * kWords, which = word0 / (D / 2);
    const uint32_t tile = bar0 - C::kSmBar + C::kSmRes + which * C::kTileBytes;
    const uint32_t dst = tmem + ((uint32_t)(quarter * 32) << 16) + kColA + word0;
    if (item_k > 0) wait(kBarAccFree, item_k - 1);  // (over the last item's dV)
    wait(kBarRes + which, item_k);
    tc_fence_after();
#pragma unroll
    for (int k = 0; k < kWords; k += 16) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int chunk = (word0 % (D / 2) + k) / 4 + i;  // 16 bytes of the row, 8 to a box row
        const uint32_t u = tile + (chunk >> 3) * kBoxBytes + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[4 * i]), "=f"(v[4 * i + 1]), "=f"(v[4 * i + 2]), "=f"(v[4 * i + 3])
                     : "r"(u)
                     : "memory");
      }
      tmem_st16(dst + k, v);
    }
    tmem_wait_st();
    tc_fence_before();
    arrive(kBarRows);
  }
  // The row statistics come from the kernel before this one; Q, K, V and dO
  // are older than that kernel's start.
  dependency_wait();
  float nlse[4], ndelta[4];
  if (DQ) {
    const int one_key = bwd_one_key_rows(w.len, w.ref, p.b.n, bidir);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 st = own0 + 8 * i < w.len ? p.b.stats[(size_t)w.h * p.b.stat_stride + w.start + own0 + 8 * i]
                                             : make_float2(0.f, 0.f);
      // (a row that sees one key has no dS, and P serves nothing else here)
      nlse[i] = own0 + 8 * i < one_key ? -INFINITY : st.x;
      ndelta[i] = st.y;
    }
  }
  // Tiles [full0, full1) of the sequence have every pair visible.
  int full0, full1;
  if (DQ) {  // reference keys alone, none after the first query unless all prefix rows see them
    const int q0 = w.tile * kTile;
    full0 = 0;
    full1 = (bidir || q0 >= w.ref ? w.ref : min(w.ref, q0 + 1)) / kTile;
  } else {   // no query before the last key, past the document, or past the first key's window
    const int k0 = w.tile * kTile, first = w.B0 * kTile;
    const bool all_ref = k0 + kTile <= w.ref;
    const int from = all_ref && bidir ? 0 : k0 + kTile - 1;
    const long long to = all_ref ? w.len : min((long long)w.len, (long long)k0 + p.b.n);
    full0 = max(0, from - first + kTile - 1) / kTile;
    full1 = (int)((to - first) / kTile);
  }
  // (what only a masked tile needs is read back from the item's slot)
  const int nt = w.nt, T = w.T, U = w.U, f0 = full0 - w.lo, f1 = full1 - w.lo;
  const int lo = w.lo, A = w.A - w.lo, B0 = w.B0 + (DQ ? 0 : w.lo);
#pragma unroll 1
  for (int j = 0; j < nt; ++j) {
    const int odd = j & 1, it = T + j, iu = U + j;
    // first local row of the streamed tile
    const int o0 = (DQ ? (j < A ? j + lo : B0 + j - A) : B0 + j) * kTile;
    const uint32_t tS = base + (DQ ? 0 : odd * 128);
    const uint32_t tP = base + (DQ ? 128 : (odd ^ 1) * 128);
    const bool full = j >= f0 && j < f1;
    const uint32_t slot = Item::slot(bar0, item_k);
    // Zeroes what the thread's rows do not see.
    auto mask = [&](float* y, int len, int ref) {
      const int x0 = o0 + c0, n = min(p.b.n, len);  // (own + n stays small)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int own = own0 + 8 * i;
        uint32_t vis;
        if (DQ)
          vis = own < ref ? bit_range(0, (bidir ? ref : own + 1) - x0)
                          : bit_range(0, ref - x0) | bit_range(max(ref, own - n + 1) - x0, own + 1 - x0);
        else
          vis = bit_range((own < ref && bidir ? 0 : own) - x0, (own < ref ? len : min(len, own + n)) - x0);
        keep_row(y, i, vis >> (2 * ft));
      }
    };
    const uint32_t st = bar0 - C::kSmBar + C::kSmStats + (iu & 1) * 1024 + (c0 + 2 * ft) * 4;
    if (!DQ) wait(kBarStats + (iu & 1), iu >> 1);
    wait(kBarS + (it & 1), it >> 1);
    tc_fence_after();
    float x[kCols];
    tmem_ld_frag(tS, x);
    tmem_wait_ld();
    if (DQ) {
      tc_fence_before();
      arrive(kBarRead);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 l = make_float2(0.f, 0.f);
      if (!DQ) l = ld_shared2(st + 32 * k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float* y = x + 16 * (i >> 1) + 2 * (i & 1) + 4 * k;
        fma2(y[0], y[1], sl2, DQ ? nlse[i] : l.x, DQ ? nlse[i] : l.y);
        y[0] = ex2(y[0]);
        y[1] = ex2(y[1]);
      }
    }
    bool past_end = false;
    if (!full) {
      const int len = ld_shared(slot + 20), ref = ld_shared(slot + 24);
      mask(x, len, ref);
      past_end = o0 + kTile > len;
      // Rows [from, to) of a streamed tile cleared in shared memory.
      auto clear = [&](int stage, int from, int to) {
        for (int i = tid - kSoftmaxWarp * 32; i < (to - from) * 8 * C::kBoxes; i += kSoftmaxThreads) {
          const int row = from + i / (8 * C::kBoxes), chunk = i % (8 * C::kBoxes);
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                           bar0 - C::kSmBar + stage + (chunk >> 3) * kBoxBytes + row * 128 + (chunk & 7) * 16),
                       "r"(0)
                       : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      };
      const int stage_a = C::kSmA + (it % nA) * C::kTileBytes;
      if (past_end) {  // rows of the streamed tiles past the document's end
        clear(stage_a, len - o0, kTile);
        // The tile on ring A has landed: S, complete, has read it.  Nothing so
        // far says that of the dO tile on ring B, and a load that landed after
        // the clear would bring the next document's rows back.  Its stage is
        // filled again only after dV(j), which waits for this warp's P: the
        // phase that is waited for cannot be overtaken.  dP(j) may read the
        // tile before, under or after the clear: these rows are its columns of
        // masked pairs alone, and dP is zeroed there below whatever it holds.
        if (!DQ) {
          wait(kBarBFull + it % nB, it / nB);
          clear(C::kSmB + (it % nB) * C::kTileBytes, len - o0, kTile);
        }
      }
      // Queries that see one key: dS = 0 in effect, as dK, the last to read their
      // rows of Q, finds zeros there.
      if (!DQ && (o0 == 0 || p.b.n == 1))
        clear(stage_a, 0, min(kTile, bwd_one_key_rows(len, ref, p.b.n, bidir) - o0));
    }
    if (!DQ) {
      tmem_st_frag(tS, x);
      tmem_wait_st();
      tc_fence_before();
      arrive(kBarP + (iu & 1));
    }
    wait(kBarDP, it);
    tc_fence_after();
    float dp[kCols];
    tmem_ld_frag(tP, dp);
    tmem_wait_ld();
    if (past_end) {  // a masked weight of 0 times a NaN of another document's row
#pragma unroll
      for (int e = 0; e < kCols; ++e) dp[e] = x[e] == 0.f ? 0.f : dp[e];
    }
    if (!DQ) {
      tc_fence_before();
      arrive(kBarRead);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 d = make_float2(0.f, 0.f);
      if (!DQ) d = ld_shared2(st + 4 * kTile + 32 * k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 16 * (i >> 1) + 2 * (i & 1) + 4 * k;
        addmul2(x[e], x[e + 1], dp[e], dp[e + 1], DQ ? ndelta[i] : d.x, DQ ? ndelta[i] : d.y);
      }
    }
    tmem_st_frag(DQ ? tP : tS + kCols / 2, x);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(bar0 + 8u * (kBarDS + (it & 1)));
      if (!DQ) mbar_arrive(bar0 + 8u * (kBarStatsFree + (iu & 1)));
    }
  }
  // -------------------------------------------------- the tile's gradient
  // The item again from its slot: nothing of it but the loop's own stays in
  // registers over the loop.
  Item out;
  out.read(Item::slot(bar0, item_k));
  const int own = out.tile * kTile + quarter * 32 + fg;
  // Blocks of 32 columns, a group each in turn: those of dQ, or of dV (complete
  // before the last dS is), then dK.
  constexpr int kBlocks = D / 32;
  const int H = p.b.H;
#pragma unroll 1
  for (int blk = g; blk < (DQ ? 1 : 2) * kBlocks; blk += 4) {
    const int which = blk / kBlocks, col = blk % kBlocks * 32;
    if (!DQ && which == 0) wait(kBarFinalV, item_k - out.kq);
    else wait(kBarFinal, item_k);
    tc_fence_after();
    float o[32];
    tmem_ld_frag(tmem + ((uint32_t)(quarter * 32) << 16) + (DQ ? 384 : 256 + 128 * which) + col, o);
    tmem_wait_ld();
    const bool good = ok && !ld_shared(bar0 + 8u * kSlotAbort);
    if (DQ || which == 1 || !good) {
      const float mul = !good ? __int_as_float(0x7fc00000)
                        : out.part >= 0 ? 1.f : p.b.scale;
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] *= mul;
    }
    if (out.part < 0) {
      __nv_bfloat16* grad = static_cast<__nv_bfloat16*>(DQ ? p.b.dQ : which == 0 ? p.b.dV : p.b.dK) +
                            ((size_t)(out.start + own) * H + out.h) * D + col + 8 * ft;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* v = o + 16 * (i >> 1) + 2 * (i & 1);
        uint32_t q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = pack_bf16x2(v[4 * k], v[4 * k + 1]);
        // Words to the lane that holds their 16 bytes: a warp then writes 64
        // bytes of 8 rows at a time (a row per lane costs a pass per line).
        quad_transpose(q, ft);
        if (own + 8 * i < out.len)
          *reinterpret_cast<uint4*>(grad + (size_t)(8 * i) * H * D) = make_uint4(q[0], q[1], q[2], q[3]);
      }
    } else {
      float* part = p.b.partials + (((size_t)out.part * H + out.h) * 2 + which) * kTile * D +
                    (quarter * 32 + fg) * D + col + 2 * ft;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float* v = o + 16 * (i >> 1) + 2 * (i & 1) + 4 * k;
          *reinterpret_cast<float2*>(part + 8 * i * D + 8 * k) = make_float2(v[0], v[1]);
        }
    }
  }
  if (!ok) st_shared(bar0 + 8u * kSlotAbort, 1);
  tc_fence_before();
  arrive(kBarAccFree);
}

// What an item would have written, as NaN (all threads of the CTA).
__device__ __forceinline__ void write_nan(const BwdWork& w, int h, const BackwardParams& b) {
  const int first = w.tile * kTile, rows = w.part >= 0 ? kTile : min(kTile, w.len - first);
  for (int which = 0; which < (w.kind == kBwdDQ ? 1 : 2); ++which) {
    __nv_bfloat16* grad = static_cast<__nv_bfloat16*>(w.kind == kBwdDQ ? b.dQ : which == 0 ? b.dV : b.dK) +
                          ((size_t)(w.start + first) * b.H + h) * b.D;
    float* part = b.partials + (((size_t)max(w.part, 0) * b.H + h) * 2 + which) * kTile * b.D;
    for (int i = threadIdx.x; i < rows * b.D; i += kThreads) {
      if (w.part >= 0) part[i] = __int_as_float(0x7fc00000);
      else grad[(size_t)(i / b.D) * b.H * b.D + i % b.D] = __ushort_as_bfloat16(0x7fc0);
    }
  }
}

template <int D, int N>
__global__ void __launch_bounds__(kThreads, 1)
    backward_tc_kernel(const __grid_constant__ BwdLaunch<BwdTcParams, N> p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];  // (the swizzle's period)
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kSmBar);
  const uint32_t bar0 = smem_u32(bars);
  auto B = [&](int slot) { return bar0 + 8u * slot; };
  volatile uint32_t* s_tmem = reinterpret_cast<volatile uint32_t*>(&bars[kSlotTmem]);
  volatile int* s_abort = reinterpret_cast<volatile int*>(&bars[kSlotAbort]);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  constexpr int nA = C::kA, nB = C::kB;

  launch_dependents();
  if (threadIdx.x < 4) {
    const CUtensorMap* map = threadIdx.x == 0 ? &p.tmQ : threadIdx.x == 1 ? &p.tmK : threadIdx.x == 2 ? &p.tmV : &p.tmG;
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
  }
  if (threadIdx.x == 0) {
    constexpr int kWarps = kSoftmaxThreads / 32;
    for (int s = 0; s < kBarEnd + 1; ++s) {
      const bool per_warp = s == kBarRows || s == kBarAccFree || s == kBarP || s == kBarP + 1 || s == kBarDS ||
                            s == kBarDS + 1 || s == kBarRead || s == kBarStatsFree || s == kBarStatsFree + 1;
      // the roles that read an item's number: MMA, statistics, softmax
      mbar_init(B(s), per_warp ? kWarps : s == kBarItemFree || s == kBarItemFree + 1 ? kWarps + 2 : 1);
    }
    *s_abort = (sbase & 1023) != 0 || (int)blockIdx.x < p.b.give_up;
    st_shared(Item::slot(bar0, 1), -1);
    st_shared(B(kSlotLeft), -1);
    fence_barrier_init();
  }
  const uint32_t smA = sbase + C::kSmA, smB = sbase + C::kSmB, smRes = sbase + C::kSmRes;
  // The producer's steps (thread 0).  The first item's first loads are issued
  // before the CTA has set itself up: they need the barriers, which thread 0
  // has just made, and nothing else.
  Item item;
  int a = 0, b = 0;  // tiles issued on each ring
  auto load = [&](uint32_t dst, const CUtensorMap* map, int tile, uint32_t bar) {
    mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
    for (int x = 0; x < C::kBoxes; ++x)
      tma_load_3d(dst + x * kBoxBytes, map, kBox * x, item.h, item.start + tile * kTile, bar);
  };
  auto load_a = [&](int j) {
    load(smA + (a % nA) * C::kTileBytes, item.dq ? &p.tmK : &p.tmQ, item.at(j), B(kBarAFull + a % nA));
    ++a;
  };
  auto load_b = [&](int j) {
    load(smB + (b % nB) * C::kTileBytes, item.dq ? &p.tmV : &p.tmG, item.at(j), B(kBarBFull + b % nB));
    ++b;
  };
  auto load_res = [&] {
    load(smRes, item.dq ? &p.tmQ : &p.tmK, item.tile, B(kBarRes));
    load(smRes + C::kTileBytes, item.dq ? &p.tmG : &p.tmV, item.tile, B(kBarRes + 1));
  };
  auto announce = [&](int k) {  // item.number's description, or the end
    if (item.number >= p.n_items) {
      item.number = -1;
    } else {
      const BwdWork& w = p.work[item.number / p.b.H];
      item.h = item.number % p.b.H;
      item.start = w.start;
      item.len = w.len;
      item.ref = w.ref;
      item.tile = w.tile;
      item.dq = w.kind == kBwdDQ;
      item.nt = w.hi - w.lo;
      item.part = w.part;
      const BwdTiles seq = item.dq ? bwd_key_tiles(kTile, w.tile, w.len, w.ref, p.b.n, p.b.bidir != 0)
                                   : bwd_query_tiles(kTile, w.tile, w.len, w.ref, p.b.n, p.b.bidir != 0);
      item.A = seq.A;
      item.B0 = seq.B0;
      item.lo = w.lo;
      item.pad = 0;
    }
    item.announce(Item::slot(bar0, k));
    mbar_arrive(B(kBarItem + (k & 1)));
  };
  if (threadIdx.x == 0) {
    item.T = item.U = item.kq = 0;
    item.number = blockIdx.x;
    announce(0);
    load_a(0);
    load_res();
    load_b(0);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32((const void*)s_tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      auto wait = [&](int slot, int phase) { return wait_phase(bar0, slot, phase); };
      bool ok = true;
      int r = 1;  // items whose own tiles were issued
      for (int k = 0; ok; ++k) {
        if (k > 0) {
          ok = wait(kBarItemFree + (k & 1), (k >> 1) + 1);
          if (!ok) {
            st_shared(B(kSlotLeft), item.number);
            break;
          }
          announce(k);
          if (item.number < 0) break;
        }
        for (int j = k == 0 ? 1 : 0; j < item.nt; ++j) {
          ok = wait(kBarAFree + a % nA, a / nA + 1);
          if (!ok) break;
          load_a(j);
          if (j == 0) {
            ok = wait(kBarResFree, k - 1);
            if (!ok) break;
            load_res();
            ++r;
          }
          ok = wait(kBarBFree + b % nB, b / nB + 1);
          if (!ok) break;
          load_b(j);
        }
        if (!ok) break;
        item.T += item.nt;
        if (item.dq) ++item.kq;
        else item.U += item.nt;
        // The counter is zeroed by the kernel before this one.
        dependency_wait();
        item.number = (int)gridDim.x + atomicAdd(p.b.counter, 1);
      }
      if (!ok) *s_abort = 1;
      // drain: every issued copy has landed before the CTA may exit
      mbar_wait_bounded(B(kBarRes), (r - 1) & 1);
      mbar_wait_bounded(B(kBarRes + 1), (r - 1) & 1);
      for (int j = max(0, a - nA); j < a; ++j) mbar_wait_bounded(B(kBarAFull + j % nA), (j / nA) & 1);
      for (int j = max(0, b - nB); j < b; ++j) mbar_wait_bounded(B(kBarBFull + j % nB), (j / nB) & 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const int lead = lane == 0;
    // (every lane of the warp answers the same)
    auto wait = [&](int slot, int phase) {
      return __all_sync(0xffffffffu, wait_phase(bar0, slot, phase)) != 0;
    };
    bool ok = true;
    for (int k = 0; ok && item.next(bar0, k); ++k) {
      const int nt = item.nt, T = item.T, U = item.U;
      // stages of ring A: of the next S and of the next gradient product; of ring B: of the next dP
      int sa = T % nA, pa = T / nA & 1, ga = sa, sb = T % nB, pb = T / nB & 1, gb = sb;
      auto step = [](int& s, int n) { s = s + 1 == n ? 0 : s + 1; };
      // the accumulators of the item before have been read
      auto acc_free = [&](int j) { return j > 0 || k == 0 || wait(kBarAccFree, k - 1); };
      if (item.dq) {
        const uint32_t S = tmem, dP = tmem + 128, dQ = tmem + 384, aQ = tmem + kColA, aG = aQ + D / 2;
        auto scores = [&](int j) -> bool {  // S(j) = Q K_j^T
          if (!wait(kBarAFull + sa, pa)) return false;
          tc_fence_after();
          mma_scores_ta<D>(lead, S, aQ, smA + sa * C::kTileBytes);
          commit(lead, B(kBarS + ((T + j) & 1)));
          step(sa, nA);
          pa ^= sa == 0;
          return true;
        };
        auto dprob = [&](int j) -> bool {  // dP(j) = dO V_j^T
          if (!wait(kBarBFull + sb, pb)) return false;
          tc_fence_after();
          mma_scores_ta<D>(lead, dP, aG, smB + sb * C::kTileBytes);
          commit(lead, B(kBarDP));
          commit(lead, B(kBarBFree + sb));
          step(sb, nB);
          pb ^= sb == 0;
          return true;
        };
        ok = wait(kBarRows, item.kq);
        if (ok && lane == 0) mbar_arrive(B(kBarResFree));
        ok = ok && scores(0) && dprob(0);
        for (int j = 0; j < nt && ok; ++j) {
          if (j + 1 < nt) ok = wait(kBarRead, T + j) && scores(j + 1);
          ok = ok && wait(kBarDS + ((T + j) & 1), (T + j) >> 1) && acc_free(j);
          if (!ok) break;
          tc_fence_after();
          mma_grad<D>(lead, dQ, dP, smA + ga * C::kTileBytes, j > 0);
          commit(lead, B(kBarAFree + ga));
          step(ga, nA);
          if (j + 1 < nt) ok = dprob(j + 1);
        }
      } else {
        const uint32_t dV = tmem + 256, dK = tmem + 384;
        auto scores = [&](int j) -> bool {  // S(j)^T = K Q_j^T
          if (!wait(kBarAFull + sa, pa)) return false;
          tc_fence_after();
          mma_scores<D>(lead, tmem + (j & 1) * 128, smRes, smA + sa * C::kTileBytes);
          commit(lead, B(kBarS + ((T + j) & 1)));
          step(sa, nA);
          pa ^= sa == 0;
          return true;
        };
        auto dprob = [&](int j) -> bool {  // dP(j)^T = V dO_j^T
          if (!wait(kBarBFull + sb, pb)) return false;
          tc_fence_after();
          mma_scores<D>(lead, tmem + ((j & 1) ^ 1) * 128, smRes + C::kTileBytes, smB + sb * C::kTileBytes);
          commit(lead, B(kBarDP));
          if (j == nt - 1) commit(lead, B(kBarResFree));
          step(sb, nB);
          pb ^= sb == 0;
          return true;
        };
        ok = wait(kBarRes, k) && scores(0) && wait(kBarRes + 1, k) && dprob(0);
        for (int j = 0; j < nt && ok; ++j) {
          ok = wait(kBarP + ((U + j) & 1), (U + j) >> 1) && acc_free(j);
          if (!ok) break;
          tc_fence_after();
          mma_grad<D>(lead, dV, tmem + (j & 1) * 128, smB + gb * C::kTileBytes, j > 0);
          commit(lead, B(kBarBFree + gb));
          if (j == nt - 1) commit(lead, B(kBarFinalV));
          step(gb, nB);
          if (j + 1 < nt) ok = wait(kBarRead, T + j) && scores(j + 1);
          ok = ok && wait(kBarDS + ((T + j) & 1), (T + j) >> 1);
          if (!ok) break;
          tc_fence_after();
          mma_grad<D>(lead, dK, tmem + (j & 1) * 128 + kCols / 2, smA + ga * C::kTileBytes, j > 0);
          commit(lead, B(kBarAFree + ga));
          step(ga, nA);
          if (j + 1 < nt) ok = dprob(j + 1);
        }
      }
      commit(lead, B(kBarFinal));
      Item::done(bar0, k, lane);
    }
    if (!ok) *s_abort = 1;
    // every MMA issued by this thread has completed before TMEM is freed
    commit(lead, B(kBarEnd));
    mbar_wait_bounded(B(kBarEnd), 0);
  } else if (warp == 2) {
    // -------------------------------------------------- row statistics
    dependency_wait();
    bool ok = true;
    for (int k = 0; ok && item.next(bar0, k); ++k) {
      for (int j = 0; !item.dq && j < item.nt; ++j) {
        const int u = item.U + j, s = u & 1;
        ok = __all_sync(0xffffffffu, wait_phase(bar0, kBarStatsFree + s, (u >> 1) + 1));
        if (!ok) break;
        // (rows past the document's end are another's: zeros in their place)
        const int q0 = item.at(j) * kTile;
        const float2* src = p.b.stats + (size_t)item.h * p.b.stat_stride + item.start + q0;
        float* dst = reinterpret_cast<float*>(smem + C::kSmStats) + s * 2 * kTile;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = q0 + lane + 32 * i < item.len ? src[lane + 32 * i] : make_float2(0.f, 0.f);
          dst[lane + 32 * i] = v.x;
          dst[kTile + lane + 32 * i] = v.y;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(B(kBarStats + s));
      }
      Item::done(bar0, k, lane);
    }
  } else if (warp >= kSoftmaxWarp) {
    bool ok = true;
    for (int k = 0;; ++k) {
      if (!__all_sync(0xffffffffu, wait_phase(bar0, kBarItem + (k & 1), k >> 1))) break;
      const uint32_t slot = Item::slot(bar0, k);
      if (ld_shared(slot) < 0) break;
      if (ld_shared(slot + 36)) softmax_item<D, true>(bar0, tmem, p, k, ok);
      else softmax_item<D, false>(bar0, tmem, p, k, ok);
      Item::done(bar0, k, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                              : "memory");
  if (*s_abort) {
    // The two announced last may be unfinished (one is announced when every role
    // is done with the one before the last), one may be taken and not announced.
    dependency_wait();
    const uint32_t held[3] = {Item::slot(bar0, 0), Item::slot(bar0, 1), B(kSlotLeft)};
    for (uint32_t slot : held) {
      const int number = ld_shared(slot);
      if (number >= 0 && number < p.n_items) write_nan(p.work[number / p.b.H], number % p.b.H, p.b);
    }
    while (true) {
      __syncthreads();
      if (threadIdx.x == 0) st_shared(B(kSlotLeft), (int)gridDim.x + atomicAdd(p.b.counter, 1));
      __syncthreads();
      const int number = ld_shared(B(kSlotLeft));
      if (number >= p.n_items) break;
      write_nan(p.work[number / p.b.H], number % p.b.H, p.b);
    }
  }
}

template <int D, int N>
cudaError_t launch(const BwdTcParams& common, const BwdWork* work, int n_work, cudaStream_t stream) {
  static PerContextOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(backward_tc_kernel<D, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmBytes);
  });
  if (e != cudaSuccess) return e;
  BwdLaunch<BwdTcParams, N> p;
  static_cast<BwdTcParams&>(p) = common;
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  for (int w0 = 0; w0 < n_work; w0 += N) {
    const int m = std::min(N, n_work - w0);
    std::copy_n(work + w0, m, p.work);
    p.n_items = m * p.b.H;
    e = launch_dependent(backward_tc_kernel<D, N>, std::min(p.n_items, sms), kThreads, Cfg<D>::kSmBytes, stream, p);
    if (e != cudaSuccess) return e;
    ++p.b.counter;
  }
  return cudaSuccess;
}

template <int D>
cudaError_t launch(const BwdTcParams& p, const BwdWork* work, int n_work, cudaStream_t stream) {
  return n_work <= kBwdFewWork ? launch<D, kBwdFewWork>(p, work, n_work, stream)
                               : launch<D, kBwdMaxWork>(p, work, n_work, stream);
}

}  // namespace
}  // namespace tc

cudaError_t launch_backward_tc(const BackwardParams& b, const BwdWork* work, int n_work, cudaStream_t stream) {
  using namespace tc;
  BwdTcParams p;
  if (!make_packed_map(&p.tmQ, b.Q, b.L, b.H, b.D) || !make_packed_map(&p.tmK, b.K, b.L, b.H, b.D) ||
      !make_packed_map(&p.tmV, b.V, b.L, b.H, b.D) || !make_packed_map(&p.tmG, b.dO, b.L, b.H, b.D))
    return cudaErrorInvalidValue;
  p.b = b;
  p.scale_log2 = b.scale * 1.4426950408889634f;
  return b.D == 64 ? launch<64>(p, work, n_work, stream) : launch<128>(p, work, n_work, stream);
}

}  // namespace rswa
