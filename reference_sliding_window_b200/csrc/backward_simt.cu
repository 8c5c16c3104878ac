// Gradient of the teacher-forced R-SWA attention on CUDA cores: float32
// arithmetic throughout (float32 tensors; the formulas and the mask are in
// backward.h).
//
// One CTA of 256 threads per work item and head, tiles of 64 queries x 64
// keys.  Bound: the FMA pipes.  Per tile pair a thread forms 4x4 scores and
// 4x4 dP from rows staged in shared memory (16 128-bit loads for 128 FMAs),
// writes P and dS to shared memory, and adds its 4 x D/16 block of the
// gradient tile (6 128-bit loads for 64 FMAs in the dK, dV items).  Rows are
// padded by 4 floats so that the 128-bit loads of 8 consecutive rows fall on
// distinct banks.

#include <math.h>

#include "backward.h"
#include "common.cuh"

namespace rswa {
namespace {

constexpr int kT = kBwdTileSimt;
constexpr int kThreads = 256;
constexpr int kPS = kT + 4;  // row stride of the P and dS tiles

template <int D>
constexpr int smem_bytes() {
  return 4 * (4 * kT * (D + 4) + 2 * kT * kPS);
}

struct SimtParams {
  BackwardParams b;
  float scale_log2;
  BwdWork work[kBwdMaxWork];
};

// Rows [row0, row0 + 64) of a packed [L][H][D] tensor's head h as float32;
// rows at or past row_end are zero.
template <int D>
__device__ __forceinline__ void load_tile(float* dst, const void* src, int row0, int row_end, int H, int h) {
  for (int c = threadIdx.x; c < kT * (D / 4); c += kThreads) {
    const int r = c / (D / 4), e = (c % (D / 4)) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row0 + r < row_end)
      v = *reinterpret_cast<const float4*>(static_cast<const float*>(src) + ((size_t)(row0 + r) * H + h) * D + e);
    *reinterpret_cast<float4*>(dst + r * (D + 4) + e) = v;
  }
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

__device__ __forceinline__ void fma4(float& a, float4 x, float4 y) {
  a = fmaf(x.x, y.x, a);
  a = fmaf(x.y, y.y, a);
  a = fmaf(x.z, y.z, a);
  a = fmaf(x.w, y.w, a);
}

template <int NC>
__device__ __forceinline__ void outer(float (*acc)[NC], float4 w, const float* row, int tx) {
  const float wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < NC; e += 4) {
    const float4 x = ld4(row + tx * 4 + 16 * e);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      acc[a][e] = fmaf(wv[a], x.x, acc[a][e]);
      acc[a][e + 1] = fmaf(wv[a], x.y, acc[a][e + 1]);
      acc[a][e + 2] = fmaf(wv[a], x.z, acc[a][e + 2]);
      acc[a][e + 3] = fmaf(wv[a], x.w, acc[a][e + 3]);
    }
  }
}

// A thread's 4 x NC block of a gradient tile (rows 4*ty .. +3, columns
// tx*4 + 16*e .. +3), to the gradient or to a partial.
template <int D, int NC>
__device__ __forceinline__ void write_tile(const float (*acc)[NC], void* grad, float* part, float mul, int row0,
                                           int row_end, int H, int h, int tx, int ty) {
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int r = 4 * ty + a;
    if (row0 + r >= row_end) continue;
#pragma unroll
    for (int e = 0; e < NC; ++e) {
      const int c = tx * 4 + 16 * (e & ~3) + (e & 3);
      if (part) part[r * D + c] = acc[a][e];
      else static_cast<float*>(grad)[((size_t)(row0 + r) * H + h) * D + c] = acc[a][e] * mul;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) backward_simt_kernel(const __grid_constant__ SimtParams p) {
  extern __shared__ __align__(16) float sm[];
  constexpr int S = D + 4, NC = D / 16;
  float* res0 = sm;                // dQ items: Q, dO; dK, dV items: K, V
  float* res1 = sm + kT * S;
  float* str0 = sm + 2 * kT * S;   // dQ items: K, V; dK, dV items: Q, dO
  float* str1 = sm + 3 * kT * S;
  float* t0 = sm + 4 * kT * S;     // dS [key][query] (dQ items) or P [query][key]
  float* t1 = t0 + kT * kPS;       // dS [query][key] (dK, dV items)
  const BackwardParams& b = p.b;
  const BwdWork w = p.work[blockIdx.x / b.H];
  const int h = blockIdx.x % b.H;
  const bool dq = w.kind == kBwdDQ;
  const int own0 = w.tile * kT;  // local rows of the owned tile
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const BwdTiles seq = dq ? bwd_key_tiles(kT, w.tile, w.len, w.ref, b.n, b.bidir != 0)
                          : bwd_query_tiles(kT, w.tile, w.len, w.ref, b.n, b.bidir != 0);
  const int end = w.start + w.len;
  load_tile<D>(res0, dq ? b.Q : b.K, w.start + own0, end, b.H, h);
  load_tile<D>(res1, dq ? b.dO : b.V, w.start + own0, end, b.H, h);
  const float* qs = dq ? res0 : str0;
  const float* gs = dq ? res1 : str1;
  const float* ks = dq ? str0 : res0;
  const float* vs = dq ? str1 : res1;

  float acc0[4][NC], acc1[4][NC];  // dQ; or dV, dK
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int e = 0; e < NC; ++e) acc0[a][e] = acc1[a][e] = 0.f;

  for (int j = w.lo; j < w.hi; ++j) {
    const int other0 = seq.at(j) * kT;
    load_tile<D>(str0, dq ? b.K : b.Q, w.start + other0, end, b.H, h);
    load_tile<D>(str1, dq ? b.V : b.dO, w.start + other0, end, b.H, h);
    __syncthreads();
    const int q0 = dq ? own0 : other0, k0 = dq ? other0 : own0;
    float s[4][4], dp[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[a][c] = dp[a][c] = 0.f;
#pragma unroll 2
    for (int e = 0; e < D; e += 4) {
      float4 q[4], g[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        q[a] = ld4(qs + (ty + 16 * a) * S + e);
        g[a] = ld4(gs + (ty + 16 * a) * S + e);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 k = ld4(ks + (tx + 16 * c) * S + e), v = ld4(vs + (tx + 16 * c) * S + e);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          fma4(s[a][c], q[a], k);
          fma4(dp[a][c], g[a], v);
        }
      }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = ty + 16 * a, i = q0 + r;  // query row
      const float2 st = i < w.len ? b.stats[(size_t)h * b.stat_stride + w.start + i] : make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int kr = tx + 16 * c, key = k0 + kr;
        const bool vis = i < w.len && ((key <= i && (i < w.ref || key < w.ref || key > i - b.n)) ||
                                       (b.bidir && i < w.ref && key < w.ref));
        const float pr = vis ? exp2f(fmaf(s[a][c], p.scale_log2, st.x)) : 0.f;
        const float ds = vis ? pr * (dp[a][c] + st.y) : 0.f;
        if (dq) {
          t0[kr * kPS + r] = ds;
        } else {
          t0[r * kPS + kr] = pr;
          t1[r * kPS + kr] = ds;
        }
      }
    }
    __syncthreads();
    if (dq) {
#pragma unroll 4
      for (int k = 0; k < kT; ++k) outer<NC>(acc0, ld4(t0 + k * kPS + 4 * ty), ks + k * S, tx);
    } else {
#pragma unroll 4
      for (int q = 0; q < kT; ++q) {
        outer<NC>(acc0, ld4(t0 + q * kPS + 4 * ty), gs + q * S, tx);
        outer<NC>(acc1, ld4(t1 + q * kPS + 4 * ty), qs + q * S, tx);
      }
    }
    __syncthreads();
  }
  float* part = w.part < 0 ? nullptr : b.partials + ((size_t)w.part * b.H + h) * 2 * kT * D;
  if (dq) {
    write_tile<D, NC>(acc0, b.dQ, part, b.scale, w.start + own0, end, b.H, h, tx, ty);
  } else {
    write_tile<D, NC>(acc0, b.dV, part, 1.f, w.start + own0, end, b.H, h, tx, ty);
    write_tile<D, NC>(acc1, b.dK, part ? part + kT * D : nullptr, b.scale, w.start + own0, end, b.H, h, tx, ty);
  }
}

template <int D>
cudaError_t launch(const SimtParams& p, int n_work, cudaStream_t stream) {
  static PerContextOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(backward_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D>());
  });
  if (e != cudaSuccess) return e;
  backward_simt_kernel<D><<<n_work * p.b.H, kThreads, smem_bytes<D>(), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_backward_simt(const BackwardParams& b, const BwdWork* work, int n_work, cudaStream_t stream) {
  SimtParams p;
  p.b = b;
  p.scale_log2 = b.scale * 1.4426950408889634f;
  for (int w0 = 0; w0 < n_work; w0 += kBwdMaxWork) {
    const int m = n_work - w0 < kBwdMaxWork ? n_work - w0 : kBwdMaxWork;
    for (int i = 0; i < m; ++i) p.work[i] = work[w0 + i];
    const cudaError_t e = b.D == 64 ? launch<64>(p, m, stream) : launch<128>(p, m, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace rswa
