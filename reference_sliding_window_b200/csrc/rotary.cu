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

#include "common.cuh"

namespace rswa {
namespace {

constexpr int kThreads = 256;

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
  const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int u = (int)(idx % units);
  const long long rg = idx / units;
  const int g = (int)(rg % groups);
  const long long row = rg / groups;
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
#pragma unroll 4
  for (int h = g; h < heads; h += groups) {
    const bool second = h >= p.x[0].heads;
    const RotaryTensor& x = p.x[second];
    const int hh = second ? h - p.x[0].heads : h;
    const T* in = static_cast<const T*>(x.in) + row * x.in_stride + (long long)hh * p.plan.d;
    T* out = static_cast<T*>(x.out) + row * x.out_stride + (long long)hh * p.plan.d;
    if constexpr (VEC) {
      const uint4 a = *reinterpret_cast<const uint4*>(in + e0);
      if (!turns) {
        *reinterpret_cast<uint4*>(out + e0) = a;
        continue;
      }
      float f[V];
      Vec16<T>::unpack(a, f);
      if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) rotate(f[2 * i], f[2 * i + 1], t[i]);
      } else {
        float f1[V];
        Vec16<T>::unpack(*reinterpret_cast<const uint4*>(in + e1), f1);
#pragma unroll
        for (int i = 0; i < V; ++i) rotate(f[i], f1[i], t[i]);
        *reinterpret_cast<uint4*>(out + e1) = pack16<T>(f1);
      }
      *reinterpret_cast<uint4*>(out + e0) = pack16<T>(f);
    } else if (turns) {
      const int ea = e0, eb = INTER ? e0 + 1 : e1;
      float x0 = load_elem(in + ea), x1 = load_elem(in + eb);
      rotate(x0, x1, t[0]);
      store_elem(out + ea, x0);
      store_elem(out + eb, x1);
    } else {
      const T a = in[e0], b = in[e0 + 1];
      out[e0] = a;
      out[e0 + 1] = b;
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
