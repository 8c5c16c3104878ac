// Gradient of the teacher-forced R-SWA attention for float32 tensors (the
// formulas, the mask and the work items are in backward.h).
//
// Every product runs on the tensor cores in three tf32 MMAs: an operand x is
// split into hi = tf32(x), rounded, and lo = x - hi, exact, of which the MMA
// takes the leading 11 bits; x y is taken as hi hi + hi lo + lo hi, accumulated
// in float32.  |lo| is at most 2^-11 |x|, so lo's cut leaves 2^-21 |x| and the
// dropped lo lo 2^-22 |x y|: a product is off by at most 1.25 2^-20, a few
// float32 roundings.  Plain FMAs are bound by shared memory, not by the FMA
// pipes: the register file takes 128 bytes a cycle from it, half of what 4x4
// blocks a thread need (2011 rows, 10 heads, d = 128: 925 us, this kernel 598).
// The tensor pipe is busy 53 % of that time (its rate for these MMAs, 1024
// operations a cycle and SM, measured); loading the next tiles under this pair's
// work saved under 1 %, so they are loaded plainly.
//
// One CTA of 16 warps per work item and head, tiles of 64 queries x 64 keys.
// Per tile pair warps 0-7 form S (32 x 16 each) and write P to shared memory,
// warps 8-15 form dP and write dP - delta, transposed for a dK, dV item; then
// warps 0-7 add their 32 x D/4 blocks of dV and warps 8-15 theirs of dK, taking
// dS as the product of the two tiles (a dQ item: all warps, 32 x D/8 of the
// tile).  m16n8k8 fragments: a lane (g = lane / 4, t = lane % 4) holds k = t and t +
// 4; which elements those are is free as long as A and B agree, so the score
// products take 2t and 2t + 1 and read both with one 64-bit load.  Rows are
// padded to 8 floats modulo the 32 banks (the weight tiles to 4): every fragment
// load then touches each bank once.

#include <math.h>

#include <algorithm>

#include "backward.h"
#include "launch.cuh"

namespace rswa {
namespace {

constexpr int kT = kBwdTileF32;
constexpr int kThreads = 512;
constexpr int kPS = kT + 4;  // row stride of the P and dS tiles

template <int D>
constexpr int smem_bytes() {
  return 4 * (4 * kT * (D + 8) + 2 * kT * kPS);
}

struct F32Params {
  BackwardParams b;
  float scale_log2;
};

// Rows [row0, row0 + 64) of a packed [L][H][D] tensor's head h, asynchronously;
// rows at or past row_end are zero.
template <int D>
__device__ __forceinline__ void load_tile(float* dst, const void* src, int row0, int row_end, int H, int h) {
  for (int c = threadIdx.x; c < kT * (D / 4); c += kThreads) {
    const int r = c / (D / 4), e = (c % (D / 4)) * 4;
    const bool in = row0 + r < row_end;
    const float* p = static_cast<const float*>(src) + ((size_t)(in ? row0 + r : row0) * H + h) * D + e;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst + r * (D + 8) + e)), "l"(p),
                 "r"(in ? 16 : 0)
                 : "memory");
  }
}
__device__ __forceinline__ void load_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

struct Split {
  uint32_t hi, lo;
};
__device__ __forceinline__ Split split(float x) {
  Split s;
  // to the nearest 11 bits, in integers (605 us; with the conversion
  // instruction 675).  A NaN may be lost here, but lo keeps it.
  s.hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  s.lo = __float_as_uint(x - __uint_as_float(s.hi));
  return s;
}

__device__ __forceinline__ void mma_tf32(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c += a b over 8 k.  a: rows g, g + 8 at k = t, then at k = t + 4; b: k = t, t +
// 4.  The MMA truncates where it adds, a bias that a long chain of them would
// collect, so each starts from zero, small terms first, and its sum is added
// with rounding (the FMA pipes are idle).
__device__ __forceinline__ void mma3(float* c, const Split* a, const Split* b) {
  float s[4];
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(s[0]), "=f"(s[1]), "=f"(s[2]), "=f"(s[3])
      : "r"(a[0].lo), "r"(a[1].lo), "r"(a[2].lo), "r"(a[3].lo), "r"(b[0].hi), "r"(b[1].hi), "f"(0.f));
  mma_tf32(s, a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[0].lo, b[1].lo);
  mma_tf32(s, a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[0].hi, b[1].hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] += s[i];
}

__device__ __forceinline__ float2 ld2(const float* p) { return *reinterpret_cast<const float2*>(p); }

// c (32 x 16) += the warp's rows of A and B over the head dim.
template <int D>
__device__ __forceinline__ void scores(float (*c)[2][4], const float* a_rows, const float* b_rows, int g, int t) {
  constexpr int S = D + 8;
#pragma unroll 2
  for (int k = 0; k < D; k += 8) {
    Split a[2][4], b[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const float2 x = ld2(a_rows + (16 * m + g) * S + k + 2 * t), y = ld2(a_rows + (16 * m + 8 + g) * S + k + 2 * t);
      a[m][0] = split(x.x);
      a[m][1] = split(y.x);
      a[m][2] = split(x.y);
      a[m][3] = split(y.y);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float2 x = ld2(b_rows + (8 * n + g) * S + k + 2 * t);
      b[n][0] = split(x.x);
      b[n][1] = split(x.y);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < 2; ++n) mma3(c[m][n], a[m], b[n]);
  }
}

// NT consecutive floats of shared memory, split: row i of B's fragments.
template <int NT>
__device__ __forceinline__ void split_row(Split (*b)[2], int i, const float* row) {
  if constexpr (NT == 4) {
    const float4 x = *reinterpret_cast<const float4*>(row);
    b[0][i] = split(x.x);
    b[1][i] = split(x.y);
    b[2][i] = split(x.z);
    b[3][i] = split(x.w);
  } else if constexpr (NT == 2) {
    const float2 x = ld2(row);
    b[0][i] = split(x.x);
    b[1][i] = split(x.y);
  } else {
    b[0][i] = split(*row);
  }
}

// acc (32 x 8 NT) += W (rows of a [64][kPS] weight tile, the warp's 32; DS: times
// the tile at w2) x the tile's columns from `cols` on.  Column n of block i is
// column NT n + i.
template <int D, int NT, bool DS>
__device__ __forceinline__ void gradient(float (*acc)[NT][4], const float* w1, const float* w2, const float* cols, int g,
                                         int t) {
  constexpr int S = D + 8;
#pragma unroll 2
  for (int k = 0; k < kT; k += 8) {
    Split a[2][4], b[NT][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = (16 * m + 8 * (i & 1) + g) * kPS + k + t + 4 * (i >> 1);
        a[m][i] = split(DS ? w1[e] * w2[e] : w1[e]);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) split_row<NT>(b, i, cols + (k + t + 4 * i) * S + NT * g);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) mma3(acc[m][n], a[m], b[n]);
  }
}

// The warp's 32 x 8 NT block (rows r0 ..., columns c0 ...) to the gradient or to a partial.
template <int D, int NT>
__device__ __forceinline__ void write_block(const float (*acc)[NT][4], void* grad, float* part, float mul, int row0,
                                            int row_end, int H, int h, int r0, int c0, int g, int t) {
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = r0 + 16 * m + 8 * half + g;
      if (row0 + r >= row_end) continue;
      float* dst = part ? part + r * D : static_cast<float*>(grad) + ((size_t)(row0 + r) * H + h) * D;
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {  // the fragment's columns 2t, 2t + 1 of every block
        float v[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) v[n] = acc[m][n][2 * half + odd] * (part ? 1.f : mul);
        float* d = dst + c0 + NT * (2 * t + odd);
        if constexpr (NT == 4) *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
        else if constexpr (NT == 2) *reinterpret_cast<float2*>(d) = make_float2(v[0], v[1]);
        else *d = v[0];
      }
    }
}

// An item of one kind: the streamed tiles' work, then the finished block.
template <int D, bool DQ>
__device__ __forceinline__ void run_item(const F32Params& p, const BwdWork& w, int h, float* sm) {
  constexpr int S = D + 8, NT = DQ ? D / 64 : D / 32;
  const BackwardParams& b = p.b;
  float* res0 = sm;               // DQ: Q, dO; otherwise K, V
  float* res1 = sm + kT * S;
  float* str0 = sm + 2 * kT * S;  // DQ: K, V; otherwise Q, dO
  float* str1 = sm + 3 * kT * S;
  float* t0 = sm + 4 * kT * S;    // P, DQ: [query][key], otherwise [key][query]
  float* t1 = t0 + kT * kPS;      // dP - delta likewise
  const int own0 = w.tile * kT;   // local rows of the owned tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int team = warp >> 3, wt = warp & 7;  // team 0: S and dV, team 1: dP and dK
  const int sq = (wt & 1) * 32, sk = (wt >> 1) * 16;                        // scores: 32 queries x 16 keys
  const int gr = (wt & 1) * 32, gc = (DQ ? warp >> 1 : wt >> 1) * 8 * NT;  // gradient: 32 rows x 8 NT columns
  const bool bidir = b.bidir != 0;
  const BwdTiles seq = DQ ? bwd_key_tiles(kT, w.tile, w.len, w.ref, b.n, bidir)
                          : bwd_query_tiles(kT, w.tile, w.len, w.ref, b.n, bidir);
  const int end = w.start + w.len;
  load_tile<D>(res0, DQ ? b.Q : b.K, w.start + own0, end, b.H, h);
  load_tile<D>(res1, DQ ? b.dO : b.V, w.start + own0, end, b.H, h);
  dependency_wait();  // for the row statistics; Q, K, V and dO are older than the kernel that forms them
  // team 0: rows of Q, columns of K; team 1: rows of dO, columns of V
  const float* rows = DQ ? (team ? res1 : res0) : (team ? str1 : str0);
  const float* cols = DQ ? (team ? str1 : str0) : (team ? res1 : res0);
  float* mine = team ? t1 : t0;

  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;

  for (int j = w.lo; j < w.hi; ++j) {
    const int other0 = seq.at(j) * kT;
    load_tile<D>(str0, DQ ? b.K : b.Q, w.start + other0, end, b.H, h);
    load_tile<D>(str1, DQ ? b.V : b.dO, w.start + other0, end, b.H, h);
    const int q0 = DQ ? own0 : other0, k0 = DQ ? other0 : own0;
    float stat[2][2];  // team 0: -lse log2 e, team 1: -delta
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = q0 + sq + 16 * m + 8 * half + g;
        const float* x = reinterpret_cast<const float*>(b.stats + (size_t)h * b.stat_stride + w.start + i) + team;
        stat[m][half] = i < w.len ? *x : 0.f;
      }
    load_wait();
    __syncthreads();
    float s[2][2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[m][n][i] = 0.f;
    scores<D>(s, rows + sq * S, cols + sk * S, g, t);
    // every pair of the tiles visible (a tile past the document's end never is)
    const bool full = k0 + kT <= w.ref && q0 + kT <= w.len && (bidir || k0 + kT - 1 <= q0);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = sq + 16 * m + 8 * (i >> 1) + g, c = sk + 8 * n + 2 * t + (i & 1);
          const int row = q0 + r, key = k0 + c;
          const bool vis = full || (row < w.len && ((key <= row && (row < w.ref || key < w.ref || key > row - b.n)) ||
                                                    (bidir && row < w.ref && key < w.ref)));
          const float x = stat[m][i >> 1];
          const float y = team ? s[m][n][i] + x : exp2f(fmaf(s[m][n][i], p.scale_log2, x));
          mine[DQ ? r * kPS + c : c * kPS + r] = vis ? y : 0.f;
        }
    if (!full && team && q0 < bwd_one_key_rows(w.len, w.ref, b.n, bidir)) {  // (the same elements again)
      const int one_key = bwd_one_key_rows(w.len, w.ref, b.n, bidir) - q0;
#pragma unroll 1
      for (int r = sq + g; r < min(sq + 32, one_key); r += 8)
        for (int c = sk + 2 * t; c < sk + 16; c += (c & 1) ? 7 : 1) mine[DQ ? r * kPS + c : c * kPS + r] = 0.f;
    }
    __syncthreads();
    const float *w1 = t0 + gr * kPS, *w2 = t1 + gr * kPS;
    if (DQ) gradient<D, NT, true>(acc, w1, w2, str0 + gc, g, t);
    else if (team == 0) gradient<D, NT, false>(acc, w1, w2, str1 + gc, g, t);
    else gradient<D, NT, true>(acc, w1, w2, str0 + gc, g, t);
    __syncthreads();
  }
  float* part = w.part < 0 ? nullptr : b.partials + (((size_t)w.part * b.H + h) * 2 + (DQ ? 0 : team)) * kT * D;
  const float scale = !DQ && team == 0 ? 1.f : b.scale;
  write_block<D, NT>(acc, DQ ? b.dQ : team ? b.dK : b.dV, part, scale, w.start + own0, end, b.H, h, gr, gc, g, t);
}

template <int D, int N>
__global__ void __launch_bounds__(kThreads) backward_f32_kernel(const __grid_constant__ BwdLaunch<F32Params, N> p) {
  extern __shared__ __align__(16) float sm[];
  launch_dependents();
  const BwdWork w = p.work[blockIdx.x / p.b.H];
  const int h = blockIdx.x % p.b.H;
  if (w.kind == kBwdDQ) run_item<D, true>(p, w, h, sm);
  else run_item<D, false>(p, w, h, sm);
}

template <int D, int N>
cudaError_t launch(const F32Params& common, const BwdWork* work, int n_work, cudaStream_t stream) {
  static PerContextOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(backward_f32_kernel<D, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D>());
  });
  if (e != cudaSuccess) return e;
  BwdLaunch<F32Params, N> p;
  static_cast<F32Params&>(p) = common;
  for (int w0 = 0; w0 < n_work; w0 += N) {
    const int m = std::min(N, n_work - w0);
    std::copy_n(work + w0, m, p.work);
    e = launch_dependent(backward_f32_kernel<D, N>, m * p.b.H, kThreads, smem_bytes<D>(), stream, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int D>
cudaError_t launch(const F32Params& p, const BwdWork* work, int n_work, cudaStream_t stream) {
  return n_work <= kBwdFewWork ? launch<D, kBwdFewWork>(p, work, n_work, stream)
                               : launch<D, kBwdMaxWork>(p, work, n_work, stream);
}

}  // namespace

cudaError_t launch_backward_f32(const BackwardParams& b, const BwdWork* work, int n_work, cudaStream_t stream) {
  F32Params p;
  p.b = b;
  p.scale_log2 = b.scale * 1.4426950408889634f;
  return b.D == 64 ? launch<64>(p, work, n_work, stream) : launch<128>(p, work, n_work, stream);
}

}  // namespace rswa
