// Gradient of the teacher-forced R-SWA attention: the work planner, the row
// statistics every item reads, the sums of split tiles, and the launches.

#include "backward.h"

#include <algorithm>
#include <vector>

#include "launch.cuh"

namespace rswa {
namespace {

constexpr int kSMs = 148;

struct Plan {
  std::vector<BwdWork> work;  // heaviest first
  std::vector<BwdJoin> joins;
  int parts = 0;
};

// Tile products of an item of `tiles` tile pairs: S, dP and the gradient's own
// (one in a dQ item, two in a dK, dV item), and a start of about kStart.
constexpr long long kStart = 6;
long long item_cost(int kind, long long tiles) { return tiles * (kind == kBwdDQ ? 3 : 4) + kStart; }

Plan make_plan(int size, const int32_t* cu, const int32_t* refs, int n_docs, int n, int H, bool bidir) {
  Plan plan;
  long long total = 0;
  for (int d = 0; d < n_docs; ++d) {
    const int len = cu[d + 1] - cu[d];
    for (int t = 0; t * (long long)size < len; ++t)
      for (int kind : {kBwdDQ, kBwdDKV}) {
        const int tiles = (kind == kBwdDQ ? bwd_key_tiles(size, t, len, refs[d], n, bidir)
                                          : bwd_query_tiles(size, t, len, refs[d], n, bidir)).count();
        plan.work.push_back({cu[d], len, refs[d], t, kind, 0, tiles, -1});
        total += item_cost(kind, tiles);
      }
  }
  // An item longer than the SMs' equal share would end last, alone: it is cut
  // into shares of the tile sequence whose partial sums a second kernel adds in
  // order.  Shorter limits cost more in partials than they even out (2592 + 4001
  // rows, d = 128: 10 heads 255 us uncut against 283 with limits of a third of
  // the share; one head of 288 + 19712 rows 62 us cut against 113 uncut).
  const long long limit = std::max<long long>(total * H / kSMs, 60);
  std::vector<BwdWork> cut;
  for (const BwdWork& w : plan.work) {
    const long long cost = item_cost(w.kind, w.hi);
    const int shares = (int)std::min<long long>((cost + limit - 1) / limit, w.hi);
    if (shares <= 1) {
      cut.push_back(w);
      continue;
    }
    plan.joins.push_back({w.start, w.len, w.tile, w.kind, plan.parts, shares});
    for (int s = 0; s < shares; ++s) {
      BwdWork x = w;
      x.lo = (int)((long long)w.hi * s / shares);
      x.hi = (int)((long long)w.hi * (s + 1) / shares);
      x.part = plan.parts++;
      cut.push_back(x);
    }
  }
  plan.work.swap(cut);
  std::stable_sort(plan.work.begin(), plan.work.end(), [](const BwdWork& a, const BwdWork& b) {
    return item_cost(a.kind, a.hi - a.lo) > item_cost(b.kind, b.hi - b.lo);
  });
  return plan;
}

int tile_size(int elem) { return elem == kBF16 ? kBwdTileTc : kBwdTileF32; }

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }
// Launches of a plan's items (never more than the threads that form the statistics).
int n_launches(const Plan& plan) { return (int)((plan.work.size() + kBwdMaxWork - 1) / kBwdMaxWork); }
size_t counter_bytes(const Plan& plan) { return align_up(sizeof(int32_t) * (size_t)n_launches(plan)); }
size_t stats_bytes(int L, int H) { return align_up(sizeof(float2) * (size_t)H * (L + 128)); }

// Row statistics, float32: D/N lanes per row
// and head, 16 bytes of O and of dO each.  Bound by the reads of O and dO.
template <typename T, int D>
__global__ void __launch_bounds__(256) backward_stats_kernel(const BackwardParams p) {
  constexpr int N = Vec16<T>::N, G = D / N;
  dependency_wait();
  // The items may load their tiles while the statistics form: whatever wrote
  // their tensors is done.
  launch_dependents();
  const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
  if (idx < p.n_counters) p.counter[idx] = 0;
  const long long rh = idx / G;  // row * H + head
  const int e = (int)(idx % G) * N;
  const bool in = rh < (long long)p.L * p.H;
  float sum = 0.f;
  if (in) {
    float o[N], g[N];
    Vec16<T>::unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(p.O) + rh * D + e), o);
    Vec16<T>::unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(p.dO) + rh * D + e), g);
#pragma unroll
    for (int i = 0; i < N; ++i) sum = fmaf(o[i], g[i], sum);
  }
#pragma unroll
  for (int off = G / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (in && e == 0) {
    const int row = (int)(rh / p.H), h = (int)(rh % p.H);
    p.stats[(size_t)h * p.stat_stride + row] = make_float2(p.lse[(size_t)h * p.L + row] * -1.4426950408889634f, -sum);
  }
}

template <typename T, int D>
cudaError_t launch_stats(const BackwardParams& p, cudaStream_t stream) {
  const long long threads = (long long)p.L * p.H * (D / Vec16<T>::N);
  return launch_dependent(backward_stats_kernel<T, D>, (unsigned)((threads + 255) / 256), 256, 0, stream, p);
}

constexpr int kMaxJoin = 1000;
struct JoinParams {
  BackwardParams b;
  int size;
  BwdJoin join[kMaxJoin];
};

// Adds a split tile's partials in order.  One CTA per (tile, head, gradient and
// slice of the tile's rows): few tiles are split, so a tile has many CTAs.
constexpr int kJoinSlices = 8;
template <typename T>
__global__ void __launch_bounds__(256) backward_join_kernel(const __grid_constant__ JoinParams p) {
  dependency_wait();
  const BackwardParams& b = p.b;
  const int which = blockIdx.x & 1, slice = (blockIdx.x >> 1) % kJoinSlices;
  const int tile_head = blockIdx.x / (2 * kJoinSlices);
  const BwdJoin w = p.join[tile_head / b.H];
  if (which == 1 && w.kind == kBwdDQ) return;
  const int h = tile_head % b.H;
  const int tile_elems = p.size * b.D;
  const int first = w.tile * p.size, slice_rows = p.size / kJoinSlices;
  const int rows = min(slice_rows, w.len - first - slice * slice_rows);  // may be <= 0
  const size_t stride = (size_t)b.H * 2 * tile_elems;
  T* grad = static_cast<T*>(w.kind == kBwdDQ ? b.dQ : which == 0 ? b.dV : b.dK) +
            ((size_t)(w.start + first + slice * slice_rows) * b.H + h) * b.D;
  const float mul = w.kind == kBwdDKV && which == 0 ? 1.f : b.scale;
  const float* part = b.partials + (((size_t)w.part * b.H + h) * 2 + which) * tile_elems + slice * slice_rows * b.D;
  for (int c = threadIdx.x * 4; c < rows * b.D; c += 256 * 4) {
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < w.n_parts; ++s) {
      const float4 x = *reinterpret_cast<const float4*>(part + s * stride + c);
      sum.x += x.x;
      sum.y += x.y;
      sum.z += x.z;
      sum.w += x.w;
    }
    T* dst = grad + (size_t)(c / b.D) * b.H * b.D + c % b.D;
    store_elem(dst, sum.x * mul);
    store_elem(dst + 1, sum.y * mul);
    store_elem(dst + 2, sum.z * mul);
    store_elem(dst + 3, sum.w * mul);
  }
}

thread_local int give_up_ctas = 0;

}  // namespace

extern "C" void rswa_testing_backward_give_up(int ctas) { give_up_ctas = ctas; }

size_t backward_workspace_bytes(const int32_t* cu, const int32_t* refs, int n_docs, int n, int H, int D, int elem,
                                bool bidir) {
  const int size = tile_size(elem);
  const Plan plan = make_plan(size, cu, refs, n_docs, n, H, bidir);
  return counter_bytes(plan) + stats_bytes(cu[n_docs], H) + sizeof(float) * (size_t)plan.parts * H * 2 * size * D;
}

cudaError_t launch_backward(BackwardParams p, int elem, void* workspace, cudaStream_t stream) {
  const int size = tile_size(elem);
  const Plan plan = make_plan(size, p.cu, p.refs, p.n_docs, p.n, p.H, p.bidir != 0);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.counter = reinterpret_cast<int32_t*>(ws);
  p.n_counters = n_launches(plan);
  p.give_up = give_up_ctas;
  p.stats = reinterpret_cast<float2*>(ws + counter_bytes(plan));
  p.stat_stride = p.L + 128;
  p.partials = reinterpret_cast<float*>(ws + counter_bytes(plan) + stats_bytes(p.L, p.H));
  cudaError_t e = elem == kF32 ? (p.D == 64 ? launch_stats<float, 64>(p, stream) : launch_stats<float, 128>(p, stream))
                  : p.D == 64  ? launch_stats<__nv_bfloat16, 64>(p, stream)
                               : launch_stats<__nv_bfloat16, 128>(p, stream);
  if (e != cudaSuccess) return e;
  e = elem == kBF16 ? launch_backward_tc(p, plan.work.data(), (int)plan.work.size(), stream)
                    : launch_backward_f32(p, plan.work.data(), (int)plan.work.size(), stream);
  if (e != cudaSuccess) return e;
  JoinParams j;
  j.b = p;
  j.size = size;
  for (size_t w0 = 0; w0 < plan.joins.size(); w0 += kMaxJoin) {
    const int m = (int)std::min<size_t>(kMaxJoin, plan.joins.size() - w0);
    std::copy_n(plan.joins.begin() + w0, m, j.join);
    e = launch_dependent(elem == kF32 ? backward_join_kernel<float> : backward_join_kernel<__nv_bfloat16>, m * p.H * 2 * kJoinSlices,
                         256, 0, stream, j);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace rswa
