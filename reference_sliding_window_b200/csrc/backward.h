// The gradient of the teacher-forced R-SWA attention: work items, their tile
// ranges and the kernels' interfaces.
//
// Per head, over the visible (query i, key j) pairs (0 elsewhere):
//   P = exp(scale q_i.k_j - lse_i),  delta_i = O_i . dO_i,
//   dS = P (dO_i . v_j - delta_i),
//   dV_j = sum_i P dO_i,  dQ_i = scale sum_j dS k_j,  dK_j = scale sum_i dS q_i.
// P is recomputed from Q, K and lse.  Two kinds of work item share a launch:
// a query tile sums its dQ over key tiles, a key tile sums its dK and dV over
// query tiles.  Each sum has one owner and one order, so results repeat bit
// for bit; the price is that S and dP are formed twice (7 tile products
// instead of the 5 of a form that adds dQ to memory with atomics).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace rswa {

enum BwdKind : int { kBwdDQ = 0, kBwdDKV = 1 };

// One CTA's work (for each head): tiles [lo, hi) of the sequence that its
// query tile (kBwdDQ: key tiles) or key tile (kBwdDKV: query tiles) visits.
struct BwdWork {
  int32_t start, len, ref;  // the document: first pack row, rows, reference rows
  int32_t tile;             // tile of local rows [tile * size, (tile + 1) * size)
  int32_t kind;             // BwdKind
  int32_t lo, hi;           // its share of the tile sequence
  int32_t part;             // split-sum partial this share writes, or -1: the gradient itself
};

// A tile whose sum was split: partials [part, part + n_parts) added in order.
struct BwdJoin {
  int32_t start, len, tile, kind, part, n_parts;
};

// Key tiles of a query tile: [0, A), then [B0, B0 + nB).
struct BwdTiles {
  int A, B0, nB;
  __host__ __device__ int count() const { return A + nB; }
  __host__ __device__ int at(int j) const { return j < A ? j : B0 + (j - A); }
};

__host__ __device__ inline BwdTiles bwd_key_tiles(int size, int tile, int len, int ref, int n, bool bidir) {
  const int q0 = tile * size;
  const int q_last = (q0 + size < len ? q0 + size : len) - 1;
  if (q_last < ref)  // prefix rows only: causal, or every reference key
    return {bidir ? (ref + size - 1) / size : q_last / size + 1, 0, 0};
  BwdTiles r;
  r.A = (ref + size - 1) / size;
  const int qs = q0 > ref ? q0 : ref;
  const int lo = (long long)qs - n + 1 > ref ? qs - n + 1 : ref;
  r.B0 = lo / size > r.A ? lo / size : r.A;
  r.nB = q_last / size - r.B0 + 1;
  if (r.nB < 0) r.nB = 0;
  return r;
}

// Query tiles of a key tile: one contiguous run (B0, nB), A = 0.  A tile with
// a reference key is seen by every later row (and, bidirectional, by every
// prefix row); an output key by the n rows from its own on.
__host__ __device__ inline BwdTiles bwd_query_tiles(int size, int tile, int len, int ref, int n, bool bidir) {
  const int k0 = tile * size;
  const int k_last = (k0 + size < len ? k0 + size : len) - 1;
  int last = len - 1, first = tile;
  if (k0 < ref) {
    if (bidir) first = 0;
  } else if ((long long)k_last + n - 1 < last) {
    last = k_last + n - 1;
  }
  return {0, first, last / size - first + 1};
}

// The first so many of a document's rows see one key (its first row, unless a
// bidirectional prefix shows it more; every row of a window of one without a
// prefix): P is 1 whatever the score, so dS = 0.  The difference of two equal sums
// formed in two orders would leave their rounding error; the kernels set such a
// row's dS to 0.  A tile with such a pair is never visible as a whole.
__host__ __device__ inline int bwd_one_key_rows(int len, int ref, int n, bool bidir) {
  return ref == 0 && n == 1 ? len : bidir && ref > 1 ? 0 : 1;
}

struct BackwardParams {
  const void *dO, *Q, *K, *V, *O;
  const float* lse;  // [H][L]
  void *dQ, *dK, *dV;
  int L, n, H, D;
  float scale;
  int bidir;
  // documents of the pack, HOST arrays
  const int32_t* cu;
  const int32_t* refs;
  int n_docs;
  // workspace
  float2* stats;    // [H][stat_stride]: (-lse log2 e, -delta) of each row
  int stat_stride;  // L and a tile of padding
  float* partials;  // [parts][H][2][tile][D]
  int32_t* counter; // one per launch: items taken off its list, zeroed with the statistics
  int n_counters;
  int give_up;      // CTAs of the bf16 kernel whose waits run out at once (tests)
};

constexpr int kBwdTileTc = 128, kBwdTileF32 = 64;
// Work entries per launch, which travel in the kernel's parameters: up to 30
// KB, or 2 KB where that holds them (a launch with the large ones costs the
// host about 2 us more).
constexpr int kBwdMaxWork = 960, kBwdFewWork = 64;
template <typename Common, int N>
struct BwdLaunch : Common {
  BwdWork work[N];  // heaviest first
};

// Failure injection for the tests of the bf16 kernel's bounded waits: in the
// calling thread's gradient calls from here on, each launch's first `ctas` CTAs
// behave as if a wait had run out.  0, the default: none.
extern "C" void rswa_testing_backward_give_up(int ctas);

size_t backward_workspace_bytes(const int32_t* cu, const int32_t* refs, int n_docs, int n, int H, int D, int elem,
                                bool bidir);
// Fills the workspace fields of p from `workspace` (backward_workspace_bytes).
cudaError_t launch_backward(BackwardParams p, int elem, void* workspace, cudaStream_t stream);

// float32: three tf32 MMAs per product.
cudaError_t launch_backward_f32(const BackwardParams& p, const BwdWork* work, int n_work,
                                 cudaStream_t stream);

// bf16, head dim 64 or 128: the tcgen05 kernel.
cudaError_t launch_backward_tc(const BackwardParams& p, const BwdWork* work, int n_work, cudaStream_t stream);

}  // namespace rswa
