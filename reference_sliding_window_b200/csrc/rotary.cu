// Rotary positions on queries and keys: pair i of a head, at position m, turns
// by the angle m * theta_i (and is scaled by the plan's mscale):
//   y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin,
// pairs (x_i, x_{i + dim/2}) in the half layout, (x_2i, x_2i+1) interleaved;
// elements from dim on pass through.  The gradient is the turn by the
// opposite angle.
//
// Bound: memory (each element read and written once).  The angle needs no
// table: theta_i is stored as a fraction of a turn in units of 2^-64, so
// position * theta_i modulo one turn is the low 64 bits of an integer
// product, exact however far the position; its nearest quarter turn is taken
// off as an integer and only the rest, at most an eighth of a turn, is
// rounded to float32.  A thread forms the angles of its pairs once and uses
// them for every head that it visits (heads g, g + groups, ...).

#include "rotary.h"

#include "launch.cuh"

namespace rswa {
namespace {

constexpr int kThreads = 128;

struct Turn {
  float c, s;
};

__device__ __forceinline__ Turn turn_at(int pos, unsigned long long turn, float mscale, float sign) {
  const unsigned t = (unsigned)((unsigned long long)(long long)pos * turn >> 32);  // 2^-32 turns
  const unsigned quarter = (t + (1u << 29)) >> 30;
  const int rest = (int)(t - (quarter << 30));                        // within an eighth of a turn
  float s, c;
  sincospif((float)rest * 4.6566128730773926e-10f, &s, &c);           // 2^-31: half turns
  const float cq = (quarter & 1) ? s : c, sq = (quarter & 1) ? c : s;
  Turn r;
  r.c = ((quarter + 1) & 2) ? -cq : cq;                               // quarters 1, 2
  r.s = (quarter & 2) ? -sq : sq;                                     // quarters 2, 3
  r.c *= mscale;
  r.s *= mscale * sign;
  return r;
}

__device__ __forceinline__ void rotate(float& x0, float& x1, Turn t) {
  const float y0 = x0 * t.c - x1 * t.s;
  x1 = x1 * t.c + x0 * t.s;
  x0 = y0;
}

// One unit: kPairs pairs of every head, as one or two 16-byte vectors
// (VEC), or one pair element by element; units past the pairs copy.
template <typename T, bool VEC, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p, int units, int groups) {
  constexpr int V = Vec16<T>::N;
  constexpr int kPairs = !VEC ? 1 : INTER ? V / 2 : V;
  int u, g;
  long long row;
  if (gridDim.x <= 0xffffffffu / kThreads) {  // (a 64-bit division costs as much as a head's turn)
    const unsigned idx = blockIdx.x * kThreads + threadIdx.x, rg = idx / (unsigned)units;
    u = (int)(idx - rg * (unsigned)units);
    row = rg / (unsigned)groups;
    g = (int)(rg - (unsigned)row * (unsigned)groups);
  } else {
    const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x, rg = idx / units;
    u = (int)(idx % units);
    row = rg / groups;
    g = (int)(rg % groups);
  }
  dependency_wait();
  if (row >= p.rows) return;
  const int dim = p.plan.dim, half = dim / 2;
  const bool turns = u * kPairs < half;
  // first element of the unit; half layout: and of its partners
  const int e0 = turns ? (INTER ? 2 * u * kPairs : u * kPairs) : dim + (u - half / kPairs) * (VEC ? V : 2);
  const int e1 = half + e0;
  Turn t[kPairs];
  if (turns) {
    const int pos = p.positions ? p.positions[row] : p.step_T ? p.step_Lm[row] + p.step_T[0] : p.first + (int)row;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) t[i] = turn_at(pos, p.plan.turn[u * kPairs + i], p.plan.mscale, p.sign);
  }
  const int heads = p.x[0].heads + p.x[1].heads;
  // In place, a load may not pass a store as far as the compiler knows, so a
  // thread loads kBatch heads before it stores any (each element has one reader
  // and writer).
  constexpr int kBatch = 4;
  for (int h0 = g; h0 < heads; h0 += kBatch * groups) {
    const T* in[kBatch];
    T* out[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = min(h0 + j * groups, heads - 1);
      const bool second = h >= p.x[0].heads;
      const RotaryTensor& x = p.x[second];
      const long long at = (long long)(second ? h - p.x[0].heads : h) * p.plan.d;
      in[j] = static_cast<const T*>(x.in) + row * x.in_stride + at;
      out[j] = static_cast<T*>(x.out) + row * x.out_stride + at;
    }
    if constexpr (VEC) {
      uint4 a[kBatch], b[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (h0 + j * groups < heads) {
          a[j] = *reinterpret_cast<const uint4*>(in[j] + e0);
          if (!INTER && turns) b[j] = *reinterpret_cast<const uint4*>(in[j] + e1);
        }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (h0 + j * groups < heads) {
          if (turns) {
            float f[V];
            Vec16<T>::unpack(a[j], f);
            if constexpr (INTER) {
#pragma unroll
              for (int i = 0; i < kPairs; ++i) rotate(f[2 * i], f[2 * i + 1], t[i]);
            } else {
              float f1[V];
              Vec16<T>::unpack(b[j], f1);
#pragma unroll
              for (int i = 0; i < V; ++i) rotate(f[i], f1[i], t[i]);
              *reinterpret_cast<uint4*>(out[j] + e1) = pack16<T>(f1);
            }
            a[j] = pack16<T>(f);
          }
          *reinterpret_cast<uint4*>(out[j] + e0) = a[j];
        }
    } else {
      const int eb = turns && !INTER ? e1 : e0 + 1;
      T a[kBatch], b[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (h0 + j * groups < heads) {
          a[j] = in[j][e0];
          b[j] = in[j][eb];
        }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (h0 + j * groups < heads) {
          if (turns) {
            float x0 = load_elem(&a[j]), x1 = load_elem(&b[j]);
            rotate(x0, x1, t[0]);
            store_elem(&a[j], x0);
            store_elem(&b[j], x1);
          }
          out[j][e0] = a[j];
          out[j][eb] = b[j];
        }
    }
  }
}

template <typename T, bool VEC, bool INTER>
cudaError_t launch(const RotaryParams& p, cudaStream_t stream) {
  constexpr int V = Vec16<T>::N;
  constexpr int kPairs = !VEC ? 1 : INTER ? V / 2 : V;
  const int units = p.plan.dim / 2 / kPairs + (p.plan.d - p.plan.dim) / (VEC ? V : 2);
  const int heads = p.x[0].heads + p.x[1].heads;
  // Enough threads to fill the SMs; beyond that, more heads a thread.
  const long long fill = 148 * 2048, per_group = (long long)p.rows * units;
  long long groups = (fill + per_group - 1) / per_group;
  groups = groups < 1 ? 1 : groups > heads ? heads : groups;
  const long long blocks = (per_group * groups + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  // The kernel may be scheduled while its predecessor ends; it reads nothing
  // before its dependency wait.
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotary_kernel<T, VEC, INTER>, p, units, (int)groups);
}

template <typename T>
cudaError_t dispatch(const RotaryParams& p, cudaStream_t stream) {
  // 16-byte vectors need the pairs to fill them: half a rotary dim (or, with
  // interleaved pairs, the dim) that is a multiple of a vector.
  if (p.plan.interleaved)
    return p.plan.dim % Vec16<T>::N == 0 ? launch<T, true, true>(p, stream) : launch<T, false, true>(p, stream);
  return p.plan.dim / 2 % Vec16<T>::N == 0 ? launch<T, true, false>(p, stream) : launch<T, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, int elem, cudaStream_t stream) {
  return elem == kF32 ? dispatch<float>(p, stream) : dispatch<__nv_bfloat16>(p, stream);
}

}  // namespace rswa
