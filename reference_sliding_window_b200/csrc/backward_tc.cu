// Gradient of the teacher-forced R-SWA attention on the 5th-generation tensor
// cores (tcgen05 + TMEM): bf16 tensors, head dim 64 or 128, float32
// accumulation.  The formulas, the mask and the work items are in backward.h.
//
// One CTA per work item and head, tiles of 128 queries x 128 keys.  Bound: the
// tensor pipe (4 tile products per key tile and query tile in a dK, dV item, 3
// in a dQ item), with the exponentials and the products' operand reads from
// shared memory close behind.
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
//   they vary along a thread's columns), warps 4-19 are the softmax: four
//   groups of 128 threads, one thread per TMEM lane and a quarter of its 128
//   columns.
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
// * Every wait is bounded; on a timeout the item's rows are written as NaN.

#include <algorithm>

#include "backward.h"
#include "common.cuh"
#include "tc.cuh"

namespace rswa {
namespace tc {
namespace {

constexpr int kThreads = 640;
constexpr int kSoftmaxWarp = 4;
constexpr int kSoftmaxThreads = 512;
constexpr int kCols = 32;  // score columns of a softmax thread
constexpr int kTmemCols = 512;
constexpr uint32_t kColA = 256;  // dQ items: the rows of Q, then of dO, bf16 pairs

struct BwdTcParams {
  CUtensorMap tmQ, tmK, tmV, tmG;  // packed [L][H][D] maps; G is dO
  BackwardParams b;
  float scale_log2;
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
// two barriers in turn; everything else is ordered by the ring's or the region's
// next use.  (Warp 2's wait for dS(j) comes before it stages the statistics that
// dS(j+2) needs.)
enum : int {
  kBarRes = 0,      // 2: the item's own tiles; dQ items: both have landed, both are in TMEM
  kBarAFull = 2,    // 4
  kBarAFree = 6,    // 4
  kBarBFull = 10,   // 4
  kBarBFree = 14,   // 4
  kBarS = 18,       // 2
  kBarP = 20,       // 2
  kBarDS = 22,      // 2
  kBarDP = 24,
  kBarRead = 25,    // dK, dV items: dP is read; dQ items: S is
  kBarFinal = 26,
  kBarStats = 27,   // 2
  kSlotTmem = 29, kSlotAbort = 30
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
// Fragment elements zeroed (whatever they hold, NaN included) where the bit of
// their column, vis[i] for row 8 i + g, is clear.
__device__ __forceinline__ void keep(float* x, const uint32_t* vis, int t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t bits = vis[i] >> (2 * t);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float& y = x[16 * (i >> 1) + 2 * (i & 1) + 4 * (e >> 1) + (e & 1)];
      y = bits & (1u << (8 * (e >> 1) + (e & 1))) ? y : 0.f;
    }
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

// A bounded wait that ends early once the CTA has given up.
__device__ __forceinline__ bool wait_phase(uint32_t bar, int phase, volatile int* abort) {
  return mbar_try_wait(bar, phase & 1) || (!*abort && mbar_wait_bounded(bar, phase & 1));
}

struct Ctx {
  const BwdTcParams& p;
  const BwdWork& w;
  const BwdTiles& seq;
  uint8_t* smem;
  uint32_t bar0, tmem;
  volatile int* abort;
  int h;
};

// The softmax warps of an item: P and dS of every tile of its sequence, then
// the finished gradient tile from TMEM to memory.
template <int D, bool DQ>
__device__ __forceinline__ void softmax_warps(const Ctx& c) {
  using C = Cfg<D>;
  constexpr int nA = C::kA, nB = C::kB;
  const BwdTcParams& p = c.p;
  const BwdWork& w = c.w;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = (warp - kSoftmaxWarp) >> 2;  // column quarter
  const int quarter = warp & 3;              // TMEM lanes 32 * quarter .. +31
  const int fg = lane >> 2, ft = lane & 3;   // the fragments' row and column pair
  const int c0 = kCols * g;
  const int own0 = w.tile * kTile + quarter * 32 + fg;  // the thread's local rows own0 + 8 i: queries (DQ) or keys
  const uint32_t base = c.tmem + ((uint32_t)(quarter * 32) << 16) + c0;
  const float sl2 = p.scale_log2;
  const bool bidir = p.b.bidir != 0;
  bool ok = true;
  // After a timed-out wait a thread stops waiting but keeps arriving, so
  // the MMA thread is not left waiting on it; its rows are written as NaN.
  auto wait = [&](int slot, int phase) {
    if (ok && !wait_phase(c.bar0 + 8u * slot, phase, c.abort)) ok = false;
  };
  // A warp's arrival, once all of its lanes are there: an arrival per lane
  // costs an operation on the barrier's word each.
  auto arrive = [&](int slot) {
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar0 + 8u * slot);
  };
  if (DQ) {
    // The rows of Q (groups 0, 1) and dO (2, 3) from their staged tiles into
    // TMEM, as A operands: bf16 pairs as they lie in memory.
    constexpr int kWords = D / 4;
    const int row = quarter * 32 + lane;
    const uint8_t* tile = c.smem + C::kSmRes + (g >> 1) * C::kTileBytes;
    const uint32_t dst = c.tmem + ((uint32_t)(quarter * 32) << 16) + kColA + (g >> 1) * (D / 2) + (g & 1) * kWords;
    wait(kBarRes, 0);
#pragma unroll
    for (int k = 0; k < kWords; k += 16) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int chunk = ((g & 1) * kWords + k) / 4 + i;  // 16 bytes of the row, 8 to a box row
        const float4 u = *reinterpret_cast<const float4*>(tile + (chunk >> 3) * kBoxBytes + row * 128 +
                                                          (((chunk & 7) ^ (row & 7)) << 4));
        v[4 * i] = u.x;
        v[4 * i + 1] = u.y;
        v[4 * i + 2] = u.z;
        v[4 * i + 3] = u.w;
      }
      tmem_st16(dst + k, v);
    }
    tmem_wait_st();
    tc_fence_before();
    arrive(kBarRes + 1);
  }
  // The row statistics come from the kernel before this one; Q, K, V and dO
  // are older than that kernel's start.
  dependency_wait();
  float nlse[4], ndelta[4];
  if (DQ) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 st = own0 + 8 * i < w.len ? p.b.stats[(size_t)c.h * p.b.stat_stride + w.start + own0 + 8 * i]
                                             : make_float2(0.f, 0.f);
      nlse[i] = st.x;
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
    const int k0 = w.tile * kTile, first = c.seq.at(0) * kTile;
    const bool all_ref = k0 + kTile <= w.ref;
    const int from = all_ref && bidir ? 0 : k0 + kTile - 1;
    const long long to = all_ref ? w.len : min((long long)w.len, (long long)k0 + p.b.n);
    full0 = max(0, from - first + kTile - 1) / kTile;
    full1 = (int)((to - first) / kTile);
  }
  for (int j = w.lo; j < w.hi; ++j) {
    const int it = j - w.lo;
    const int o0 = c.seq.at(j) * kTile;  // first local row of the streamed tile
    const uint32_t tS = base + (DQ ? 0 : (it & 1) * 128);
    const uint32_t tP = base + (DQ ? 128 : ((it & 1) ^ 1) * 128);
    const bool full = j >= full0 && j < full1;
    uint32_t vis[4];  // otherwise: the visible columns of the thread's rows
    if (!full) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int own = own0 + 8 * i, x0 = o0 + c0;
        if (DQ)
          vis[i] = own < w.ref ? bit_range(0, (bidir ? w.ref : own + 1) - x0)
                               : bit_range(0, w.ref - x0) | bit_range(max(w.ref, own - p.b.n + 1) - x0, own + 1 - x0);
        else
          vis[i] = bit_range((own < w.ref && bidir ? 0 : own) - x0,
                             (own < w.ref ? w.len : (int)min((long long)w.len, (long long)own + p.b.n)) - x0);
      }
    }
    const float* st = reinterpret_cast<const float*>(c.smem + C::kSmStats) + (it & 1) * 2 * kTile + c0;
    if (!DQ) wait(kBarStats + (it & 1), it >> 1);
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
      if (!DQ) l = *reinterpret_cast<const float2*>(st + 8 * k + 2 * ft);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float* y = x + 16 * (i >> 1) + 2 * (i & 1) + 4 * k;
        fma2(y[0], y[1], sl2, DQ ? nlse[i] : l.x, DQ ? nlse[i] : l.y);
        y[0] = ex2(y[0]);
        y[1] = ex2(y[1]);
      }
    }
    const bool past_end = o0 + kTile > w.len;
    if (!full) keep(x, vis, ft);
    if (past_end) {  // rows of the streamed tiles past the document's end
      const int valid = w.len - o0;
      for (int i = threadIdx.x - kSoftmaxWarp * 32; i < (kTile - valid) * 8 * C::kBoxes; i += kSoftmaxThreads) {
        const int row = valid + i / (8 * C::kBoxes), chunk = i % (8 * C::kBoxes);
        const int off = (chunk >> 3) * kBoxBytes + row * 128 + (chunk & 7) * 16;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(c.smem + C::kSmA + (it % nA) * C::kTileBytes + off) = zero;
        if (!DQ) *reinterpret_cast<uint4*>(c.smem + C::kSmB + (it % nB) * C::kTileBytes + off) = zero;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (!DQ) {
      tmem_st_frag(tS, x);
      tmem_wait_st();
      tc_fence_before();
      arrive(kBarP + (it & 1));
    }
    wait(kBarDP, it);
    tc_fence_after();
    float dp[kCols];
    tmem_ld_frag(tP, dp);
    tmem_wait_ld();
    if (!DQ) {
      tc_fence_before();
      arrive(kBarRead);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 d = make_float2(0.f, 0.f);
      if (!DQ) d = *reinterpret_cast<const float2*>(st + kTile + 8 * k + 2 * ft);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 16 * (i >> 1) + 2 * (i & 1) + 4 * k;
        addmul2(x[e], x[e + 1], dp[e], dp[e + 1], DQ ? ndelta[i] : d.x, DQ ? ndelta[i] : d.y);
      }
    }
    // a masked weight of 0 times a NaN of another document's row
    if (past_end) keep(x, vis, ft);
    tmem_st_frag(DQ ? tP : tS + kCols / 2, x);
    tmem_wait_st();
    tc_fence_before();
    arrive(kBarDS + (it & 1));
  }
  // -------------------------------------------------- the tile's gradient
  wait(kBarFinal, 0);
  tc_fence_after();
  if (!ok) *c.abort = 1;
  const bool good = ok && !*c.abort;
  // Blocks of 32 columns, a group each in turn: those of dQ, or of dV, then dK.
  constexpr int kBlocks = D / 32;
  const int H = p.b.H;
#pragma unroll 1
  for (int blk = g; blk < (DQ ? 1 : 2) * kBlocks; blk += 4) {
    const int which = blk / kBlocks, col = blk % kBlocks * 32;
    float o[32];
    tmem_ld_frag(c.tmem + ((uint32_t)(quarter * 32) << 16) + (DQ ? 384 : 256 + 128 * which) + col, o);
    tmem_wait_ld();
    if (w.part < 0) {
      const float mul = !good ? __int_as_float(0x7fc00000) : !DQ && which == 0 ? 1.f : p.b.scale;
      __nv_bfloat16* grad = static_cast<__nv_bfloat16*>(DQ ? p.b.dQ : which == 0 ? p.b.dV : p.b.dK) +
                            ((size_t)(w.start + own0) * H + c.h) * D + col + 8 * ft;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* v = o + 16 * (i >> 1) + 2 * (i & 1);
        uint32_t q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = pack_bf16x2(v[4 * k] * mul, v[4 * k + 1] * mul);
        // Words to the lane that holds their 16 bytes: a warp then writes 64
        // bytes of 8 rows at a time (a row per lane costs a pass per line).
        quad_transpose(q, ft);
        if (own0 + 8 * i < w.len)
          *reinterpret_cast<uint4*>(grad + (size_t)(8 * i) * H * D) = make_uint4(q[0], q[1], q[2], q[3]);
      }
    } else {
      float* part = p.b.partials + (((size_t)w.part * H + c.h) * 2 + which) * kTile * D +
                    (quarter * 32 + fg) * D + col + 2 * ft;
      const float mul = good ? 1.f : __int_as_float(0x7fc00000);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float* v = o + 16 * (i >> 1) + 2 * (i & 1) + 4 * k;
          *reinterpret_cast<float2*>(part + 8 * i * D + 8 * k) = make_float2(v[0] * mul, v[1] * mul);
        }
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

  const int H = p.b.H, h = blockIdx.x % H;
  const BwdWork w = p.work[blockIdx.x / H];
  const bool dq = w.kind == kBwdDQ;
  const bool bidir = p.b.bidir != 0;
  const BwdTiles seq = dq ? bwd_key_tiles(kTile, w.tile, w.len, w.ref, p.b.n, bidir)
                          : bwd_query_tiles(kTile, w.tile, w.len, w.ref, p.b.n, bidir);
  const int nt = w.hi - w.lo;
  constexpr int nA = C::kA, nB = C::kB;

  launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(B(kBarRes + s), dq && s == 1 ? kSoftmaxThreads / 32 : 1);
      mbar_init(B(kBarS + s), 1);
      mbar_init(B(kBarStats + s), 1);
      mbar_init(B(kBarP + s), kSoftmaxThreads / 32);
      mbar_init(B(kBarDS + s), kSoftmaxThreads / 32);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(B(kBarAFull + s), 1);
      mbar_init(B(kBarAFree + s), 1);
      mbar_init(B(kBarBFull + s), 1);
      mbar_init(B(kBarBFree + s), 1);
    }
    mbar_init(B(kBarDP), 1);
    mbar_init(B(kBarRead), kSoftmaxThreads / 32);
    mbar_init(B(kBarFinal), 1);
    *s_abort = (sbase & 1023) != 0;
    fence_barrier_init();
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
  const uint32_t smA = sbase + C::kSmA, smB = sbase + C::kSmB, smRes = sbase + C::kSmRes;

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      auto load = [&](uint32_t dst, const CUtensorMap* map, int tile, uint32_t bar) {
        mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
        for (int x = 0; x < C::kBoxes; ++x)
          tma_load_3d(dst + x * kBoxBytes, map, kBox * x, h, w.start + tile * kTile, bar);
      };
      const CUtensorMap* mapA = dq ? &p.tmK : &p.tmQ;
      const CUtensorMap* mapB = dq ? &p.tmV : &p.tmG;
      if (dq) {
        mbar_arrive_expect_tx(B(kBarRes), 2 * C::kTileBytes);
        for (int x = 0; x < C::kBoxes; ++x) {
          tma_load_3d(smRes + x * kBoxBytes, &p.tmQ, kBox * x, h, w.start + w.tile * kTile, B(kBarRes));
          tma_load_3d(smRes + C::kTileBytes + x * kBoxBytes, &p.tmG, kBox * x, h, w.start + w.tile * kTile, B(kBarRes));
        }
      } else {
        load(smRes, &p.tmK, w.tile, B(kBarRes));
      }
      int a = 0, b = 0;  // tiles issued on each ring
      bool ok = true;
      for (int j = 0; j < nt && ok; ++j) {
        const int tile = seq.at(w.lo + j);
        ok = !*s_abort && mbar_wait_bounded(B(kBarAFree + j % nA), ((j / nA) & 1) ^ 1);
        if (!ok) break;
        load(smA + (j % nA) * C::kTileBytes, mapA, tile, B(kBarAFull + j % nA));
        ++a;
        if (j == 0 && !dq) load(smRes + C::kTileBytes, &p.tmV, w.tile, B(kBarRes + 1));
        ok = !*s_abort && mbar_wait_bounded(B(kBarBFree + j % nB), ((j / nB) & 1) ^ 1);
        if (!ok) break;
        load(smB + (j % nB) * C::kTileBytes, mapB, tile, B(kBarBFull + j % nB));
        ++b;
      }
      if (!ok) *s_abort = 1;
      // drain: every issued copy has landed before the CTA may exit
      mbar_wait_bounded(B(kBarRes), 0);
      if (!dq && a > 0) mbar_wait_bounded(B(kBarRes + 1), 0);
      for (int j = max(0, a - nA); j < a; ++j) mbar_wait_bounded(B(kBarAFull + j % nA), (j / nA) & 1);
      for (int j = max(0, b - nB); j < b; ++j) mbar_wait_bounded(B(kBarBFull + j % nB), (j / nB) & 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    {
      const int lead = lane == 0;
      // (every lane of the warp answers the same)
      auto wait = [&](int slot, int phase) {
        return __all_sync(0xffffffffu, wait_phase(B(slot), phase, s_abort)) != 0;
      };
      auto tileA = [&](int j) { return smA + (j % nA) * C::kTileBytes; };
      auto tileB = [&](int j) { return smB + (j % nB) * C::kTileBytes; };
      bool ok;
      if (dq) {
        const uint32_t S = tmem, dP = tmem + 128, dQ = tmem + 384, aQ = tmem + kColA, aG = aQ + D / 2;
        auto scores = [&](int j) -> bool {  // S(j) = Q K_j^T
          if (!wait(kBarAFull + j % nA, j / nA)) return false;
          tc_fence_after();
          mma_scores_ta<D>(lead, S, aQ, tileA(j));
          commit(lead, B(kBarS + (j & 1)));
          return true;
        };
        auto dprob = [&](int j) -> bool {  // dP(j) = dO V_j^T
          if (!wait(kBarBFull + j % nB, j / nB)) return false;
          tc_fence_after();
          mma_scores_ta<D>(lead, dP, aG, tileB(j));
          commit(lead, B(kBarDP));
          commit(lead, B(kBarBFree + j % nB));
          return true;
        };
        ok = wait(kBarRes + 1, 0) && scores(0) && dprob(0);
        for (int j = 0; j < nt && ok; ++j) {
          if (j + 1 < nt) ok = wait(kBarRead, j) && scores(j + 1);
          ok = ok && wait(kBarDS + (j & 1), j >> 1);
          if (!ok) break;
          tc_fence_after();
          mma_grad<D>(lead, dQ, dP, tileA(j), j > 0);
          commit(lead, B(kBarAFree + j % nA));
          if (j + 1 < nt) ok = dprob(j + 1);
        }
      } else {
        const uint32_t dV = tmem + 256, dK = tmem + 384;
        auto scores = [&](int j) -> bool {  // S(j)^T = K Q_j^T
          if (!wait(kBarAFull + j % nA, j / nA)) return false;
          tc_fence_after();
          mma_scores<D>(lead, tmem + (j & 1) * 128, smRes, tileA(j));
          commit(lead, B(kBarS + (j & 1)));
          return true;
        };
        auto dprob = [&](int j) -> bool {  // dP(j)^T = V dO_j^T
          if (!wait(kBarBFull + j % nB, j / nB)) return false;
          tc_fence_after();
          mma_scores<D>(lead, tmem + ((j & 1) ^ 1) * 128, smRes + C::kTileBytes, tileB(j));
          commit(lead, B(kBarDP));
          return true;
        };
        ok = wait(kBarRes, 0) && scores(0) && wait(kBarRes + 1, 0) && dprob(0);
        for (int j = 0; j < nt && ok; ++j) {
          ok = wait(kBarP + (j & 1), j >> 1);
          if (!ok) break;
          tc_fence_after();
          mma_grad<D>(lead, dV, tmem + (j & 1) * 128, tileB(j), j > 0);
          commit(lead, B(kBarBFree + j % nB));
          if (j + 1 < nt) ok = wait(kBarRead, j) && scores(j + 1);
          ok = ok && wait(kBarDS + (j & 1), j >> 1);
          if (!ok) break;
          tc_fence_after();
          mma_grad<D>(lead, dK, tmem + (j & 1) * 128 + kCols / 2, tileA(j), j > 0);
          commit(lead, B(kBarAFree + j % nA));
          if (j + 1 < nt) ok = dprob(j + 1);
        }
      }
      if (!ok) *s_abort = 1;
      // every MMA issued by this thread has completed before TMEM is read or freed
      commit(lead, B(kBarFinal));
      mbar_wait_bounded(B(kBarFinal), 0);
    }
  } else if (warp == 2) {
    // -------------------------------------------------- row statistics
    if (!dq) {
      dependency_wait();
      for (int j = 0; j < nt; ++j) {
        const int s = j & 1;
        // the softmax has read the statistics of tile j - 2 once its dS is there
        const bool free = j < 2 || (!*s_abort && mbar_wait_bounded(B(kBarDS + s), ((j - 2) >> 1) & 1));
        if (!__all_sync(0xffffffffu, free)) break;
        // rows past the document's end are another's, or padding of the array
        const float2* src = p.b.stats + (size_t)h * p.b.stat_stride + w.start + seq.at(w.lo + j) * kTile;
        float* dst = reinterpret_cast<float*>(smem + C::kSmStats) + s * 2 * kTile;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = src[lane + 32 * i];
          dst[lane + 32 * i] = v.x;
          dst[kTile + lane + 32 * i] = v.y;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(B(kBarStats + s));
      }
    }
  } else if (warp >= kSoftmaxWarp) {
    const Ctx c{p, w, seq, smem, bar0, tmem, s_abort, h};
    if (dq) softmax_warps<D, true>(c);
    else softmax_warps<D, false>(c);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                              : "memory");
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
  for (int w0 = 0; w0 < n_work; w0 += N) {
    const int m = std::min(N, n_work - w0);
    std::copy_n(work + w0, m, p.work);
    e = launch_dependent(backward_tc_kernel<D, N>, m * p.b.H, kThreads, Cfg<D>::kSmBytes, stream, p);
    if (e != cudaSuccess) return e;
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
