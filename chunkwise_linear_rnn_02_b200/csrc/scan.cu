// Elementwise gated linear recurrence (C ABI in include/gla.h, gla_scan_*):
//
//     h_t = a_t h_{t-1} + b_t,   a_t = exp g_t,   b_t = x_t  or  (1 - a_t) x_t
//
// HBM-bound: g and x are read once and o written once.  A run of tokens acts on the state in front of it as
// h -> A h + H with A the product of its a's and H its end state from zero, and two runs one after the other
// act as (A2 A1, A2 H1 + H2).  So every thread reduces a run of R tokens of VEC neighbouring channels to (A, H),
// the pairs are joined in token order across the lanes of a warp (shuffles), the warps of a block (shared
// memory) and the blocks of a cluster (their shared memory), and then each thread walks its run again from the
// state that enters it.
//
// Split: a block owns a slab of LPR * VEC channels and steps through the tokens; a step is a tile of
// 8 (32 / LPR) R tokens.  Where there are too few slabs to fill the SMs, K blocks of a cluster share a slab and take
// its tiles in turn.  Each step every block sends its (A, H) to all blocks of the cluster (st.async onto an
// mbarrier in the receiver's shared memory); every block folds all K of them, in token order, into a carry of its
// own.  So nothing goes through global memory, nothing waits outside the cluster, whose blocks run together, and the
// order of all operations is fixed by the sizes.
//
// The tiles are copied asynchronously, two steps ahead, into places of shared memory that only the copying
// thread reads, so they need no barrier; a step takes one __syncthreads.
//
// The backward walks the tiles in reverse with e_t = a_t d_t as the state: d_t = dO_t + e_{t+1}, so a run acts as
// e -> A e + E with the same A.  The states h_{t-1} that dg needs are recomputed in fp32 inside the tile, from
// the fp32 state that the forward keeps every 64 tokens (1/16 byte a value): as many bytes as reading o would
// take, without its rounding.
#include <limits.h>
#include <math.h>

#include <atomic>

#include "../../include/gla.h"
#include "fast_path.cuh"
#include "scan_cluster.cuh"
#include "vec.cuh"

namespace {

using gla::bf16;
using gla::ldf;
using gla::Pack;
using gla::stf;
namespace cl = gla::cluster;

constexpr int kKeep = 64;   // tokens between the kept states
constexpr int kWarps = 8;   // warps a block
constexpr int kMaxK = 8;    // blocks a cluster
constexpr int kStages = 2;  // tiles in flight or in use

// a = exp g and 1 - a.  Near g = 0 both come from exp g - 1 = g (1 + g/2 (1 + g/3 (...))), so that neither the
// 1 - a of a slow gate nor a long product of a's loses its leading digits; the series ends five terms in, where
// |g| < 1/8 leaves a relative error below g^5/720 < 2^-24.  Elsewhere a state forgets within a few dozen tokens,
// and the exponential's own error (2^-22 for the approximate one at bf16) has no time to add up.
template <typename T>
__device__ __forceinline__ float decay(float g, float* rest) {
  float p = fmaf(g, 1.f / 120.f, 1.f / 24.f);
  p = fmaf(g, p, 1.f / 6.f);
  p = fmaf(g, p, 0.5f);
  p = fmaf(g, p, 1.f) * g;
  const float e = sizeof(T) == 2 ? __expf(g) : expf(g);
  const bool slow = fabsf(g) < 0.125f;
  *rest = slow ? -p : 1.f - e;
  return slow ? 1.f + p : e;
}

struct Args {
  const void *g, *x, *dO;
  const float *first;  // h0 (forward), dhT (backward), or null
  const float* hc_in;  // backward: kept states
  void *o, *dg, *dx;
  float *last, *hc;    // hT (forward), dh0 (backward); kept states (forward); or null
  int T, D, slabs;     // slabs of channels a head
  int steps, tiles, K;
  unsigned int* latch;
};

// A thread's place: VEC channels from `c` of the block's slab, run `run` of the tile.
template <int VEC, int LPR>
struct Place {
  int lane_c, run_in_warp, warp, c;
  size_t bh;
  uint32_t rank;
  __device__ __forceinline__ Place(const Args& a, bool clustered) {
    const int lane = threadIdx.x & 31;
    lane_c = lane % LPR, run_in_warp = lane / LPR, warp = threadIdx.x >> 5;
    const uint32_t col = clustered ? blockIdx.x / (uint32_t)a.K : blockIdx.x;
    rank = clustered ? cl::block_rank() : 0;
    bh = col / (uint32_t)a.slabs;
    c = ((int)(col - (uint32_t)bh * (uint32_t)a.slabs) * LPR + lane_c) * VEC;
  }
};

// Copy this thread's VEC channels of a token into its own place: asynchronously where the piece has 4 bytes or more.
template <typename T, int VEC>
__device__ __forceinline__ void fetch(char* place, const T* src, bool in) {
  constexpr int BYTES = VEC * (int)sizeof(T);
  if constexpr (BYTES >= 4) {
    cl::copy_async<BYTES>(gla::sm100::smem_u32(place), src, in);
  } else {
    T v;
    stf(&v, 0.f);
    if (in) v = *src;
    *reinterpret_cast<T*>(place) = v;
  }
}

// The pair (A, H) of VEC channels, and what follows it.
template <int VEC>
struct Pair {
  float A[VEC], H[VEC];
  __device__ __forceinline__ void identity() {
#pragma unroll
    for (int j = 0; j < VEC; ++j) A[j] = 1.f, H[j] = 0.f;
  }
  // this := n after this
  __device__ __forceinline__ void then(const Pair& n) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      H[j] = fmaf(n.A[j], H[j], n.H[j]);
      A[j] *= n.A[j];
    }
  }
};

// Exclusive join over the runs of a warp, in token order (or against it): `p` becomes what lies before this
// lane's run, `all` the whole warp's.
template <int VEC, int LPR, bool REVERSE>
__device__ __forceinline__ void join_warp(Pair<VEC>& p, Pair<VEC>& all, int run) {
  constexpr int RUNS = 32 / LPR;
  if constexpr (RUNS == 1) {
    all = p;
    p.identity();
  } else {
    const int at = REVERSE ? RUNS - 1 - run : run;
#pragma unroll
    for (int d = 1; d < RUNS; d *= 2) {
      Pair<VEC> q;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        q.A[j] = REVERSE ? __shfl_down_sync(0xffffffffu, p.A[j], d * LPR) : __shfl_up_sync(0xffffffffu, p.A[j], d * LPR);
        q.H[j] = REVERSE ? __shfl_down_sync(0xffffffffu, p.H[j], d * LPR) : __shfl_up_sync(0xffffffffu, p.H[j], d * LPR);
      }
      if (at >= d) {
        q.then(p);
        p = q;
      }
    }
    const int src = (threadIdx.x & 31) % LPR + (REVERSE ? 0 : (RUNS - 1) * LPR);
    Pair<VEC> q;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      all.A[j] = __shfl_sync(0xffffffffu, p.A[j], src);
      all.H[j] = __shfl_sync(0xffffffffu, p.H[j], src);
      q.A[j] = REVERSE ? __shfl_down_sync(0xffffffffu, p.A[j], LPR) : __shfl_up_sync(0xffffffffu, p.A[j], LPR);
      q.H[j] = REVERSE ? __shfl_down_sync(0xffffffffu, p.H[j], LPR) : __shfl_up_sync(0xffffffffu, p.H[j], LPR);
    }
    if (at == 0) p.identity();
    else p = q;
  }
}

// Shared memory of the cluster's exchange: two slots, each with every rank's pair.
template <int VEC, int LPR>
struct Exchange {
  float slot[2][kMaxK][LPR][2 * VEC];
  uint64_t bar[2];
};

// Sends the block's pair to the cluster, waits for all pairs, moves `carry` over all of them and leaves in
// `enter` the state that enters this block's tile.  A slot is used again two steps later: a block sends for step
// s + 2 after it has taken everybody's pair of step s + 1, and a block sends that only after the __syncthreads
// behind its reads of step s.
template <int VEC, int LPR>
__device__ __forceinline__ void exchange(Exchange<VEC, LPR>& ex, const Pair<VEC>& block, float (&carry)[VEC],
                                         float (&enter)[VEC], int step, int K, uint32_t rank, int warp, int run,
                                         int lane_c, bool& alive, unsigned int* latch) {
  const int s = step & 1;
  if (warp < K && run == 0) {
    float v[2 * VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = block.A[j], v[VEC + j] = block.H[j];
    cl::store_async(cl::peer(gla::sm100::smem_u32(&ex.slot[s][rank][lane_c][0]), warp), v,
                    cl::peer(gla::sm100::smem_u32(&ex.bar[s]), warp));
  }
  if (alive) {
    alive = cl::wait(gla::sm100::smem_u32(&ex.bar[s]), (step >> 1) & 1, latch);
    // the slot's next use, two steps on
    if (alive && threadIdx.x == 0)
      gla::sm100::mbar_arrive_expect_tx(&ex.bar[s], (uint32_t)(K * LPR * 2 * VEC * sizeof(float)));
  }
  for (int r = 0; r < K; ++r) {
    if (r == (int)rank)
#pragma unroll
      for (int j = 0; j < VEC; ++j) enter[j] = carry[j];
    const float* v = ex.slot[s][r][lane_c];
#pragma unroll
    for (int j = 0; j < VEC; ++j) carry[j] = fmaf(v[j], carry[j], v[VEC + j]);
  }
}

template <int VEC, int LPR>
__device__ __forceinline__ void open_exchange(Exchange<VEC, LPR>& ex, int K) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) gla::sm100::mbar_init(&ex.bar[s], 1);
    gla::sm100::fence_mbar_init();
    for (int s = 0; s < 2; ++s)
      gla::sm100::mbar_arrive_expect_tx(&ex.bar[s], (uint32_t)(K * LPR * 2 * VEC * sizeof(float)));
  }
  cl::sync();
}

template <typename T, int VEC, int LPR, int R, bool COMP, bool CLUSTER>
__global__ void __launch_bounds__(kWarps * 32, 2) scan_fwd_kernel(const Args a) {
  constexpr int NT = kWarps * 32, RUNS = 32 / LPR, TILE = kWarps * RUNS * R, PIECE = VEC * (int)sizeof(T);
  extern __shared__ __align__(16) char stage[];  // [kStages][2][R][NT] pieces
  __shared__ __align__(16) float tot[2][kWarps][LPR][2 * VEC];
  __shared__ __align__(16) Exchange<VEC, CLUSTER ? LPR : 1> ex;
  const Place<VEC, LPR> at(a, CLUSTER);
  if constexpr (CLUSTER) open_exchange(ex, a.K);
  const T *g = (const T*)a.g, *x = (const T*)a.x;
  const bool mine = at.c < a.D;
  const size_t base = at.bh * (size_t)a.T * a.D + (mine ? at.c : 0);
  float carry[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) carry[j] = mine && a.first ? a.first[at.bh * a.D + at.c + j] : 0.f;
  bool alive = true;

  auto first_token = [&](int step) {
    return ((long long)step * a.K + at.rank) * TILE + (at.warp * RUNS + at.run_in_warp) * R;
  };
  auto place = [&](int step, int which, int i) {
    return stage + ((((step % kStages) * 2 + which) * R + i) * NT + threadIdx.x) * PIECE;
  };
  auto prefetch = [&](int step) {
    if (step < a.steps) {
      const long long t0 = first_token(step);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bool in = mine && t0 + i < a.T;
        const size_t p = in ? base + (size_t)(t0 + i) * a.D : 0;
        fetch<T, VEC>(place(step, 0, i), g + p, in);
        fetch<T, VEC>(place(step, 1, i), x + p, in);
      }
    }
    cl::copy_commit();
  };
  for (int s = 0; s < kStages; ++s) prefetch(s);

  for (int step = 0; step < a.steps; ++step) {
    cl::copy_wait<kStages - 1>();
    float ai[R][VEC], bi[R][VEC];
    Pair<VEC> p, warp_all;
    p.identity();
#pragma unroll
    for (int i = 0; i < R; ++i) {  // tokens behind the end have g = x = 0: they leave the state as it is
      const Pack<T, VEC> pg = *reinterpret_cast<const Pack<T, VEC>*>(place(step, 0, i));
      const Pack<T, VEC> px = *reinterpret_cast<const Pack<T, VEC>*>(place(step, 1, i));
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float rest;
        ai[i][j] = decay<T>(pg.get(j), &rest);
        bi[i][j] = COMP ? rest * px.get(j) : px.get(j);
        p.H[j] = fmaf(ai[i][j], p.H[j], bi[i][j]);
        p.A[j] *= ai[i][j];
      }
    }
    prefetch(step + kStages);
    join_warp<VEC, LPR, false>(p, warp_all, at.run_in_warp);
    if (at.run_in_warp == 0) {
      float* t = tot[step & 1][at.warp][at.lane_c];
#pragma unroll
      for (int j = 0; j < VEC; ++j) t[j] = warp_all.A[j], t[VEC + j] = warp_all.H[j];
    }
    __syncthreads();
    Pair<VEC> before, block;  // the block's warps in front of this one; all of them
    block.identity();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == at.warp) before = block;
      Pair<VEC> n;
      const float* t = tot[step & 1][w][at.lane_c];
#pragma unroll
      for (int j = 0; j < VEC; ++j) n.A[j] = t[j], n.H[j] = t[VEC + j];
      block.then(n);
    }
    float h[VEC];
    if constexpr (CLUSTER) {
      exchange(ex, block, carry, h, step, a.K, at.rank, at.warp, at.run_in_warp, at.lane_c, alive, a.latch);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        h[j] = carry[j];
        carry[j] = fmaf(block.A[j], carry[j], block.H[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) h[j] = fmaf(p.A[j], fmaf(before.A[j], h[j], before.H[j]), p.H[j]);
    const long long t0 = first_token(step);
    if (a.hc && mine && t0 < a.T && t0 % kKeep == 0) {
      const size_t n = (at.bh * (size_t)((a.T + (long long)kKeep - 1) / kKeep) + (size_t)(t0 / kKeep)) * a.D + at.c;
#pragma unroll
      for (int j = 0; j < VEC; ++j) a.hc[n + j] = h[j];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      Pack<T, VEC> out;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        h[j] = fmaf(ai[i][j], h[j], bi[i][j]);
        out.set(j, h[j]);
      }
      if (a.o && mine && t0 + i < a.T) out.store((T*)a.o + base + (size_t)(t0 + i) * a.D);
    }
  }
  if (a.last && mine && at.rank == 0 && at.warp == 0 && at.run_in_warp == 0)
#pragma unroll
    for (int j = 0; j < VEC; ++j) a.last[at.bh * a.D + at.c + j] = carry[j];
  if constexpr (CLUSTER) cl::sync();  // no block leaves while others may still send to it
}

template <typename T, int VEC, int LPR, int R, bool COMP, bool CLUSTER>
__global__ void __launch_bounds__(kWarps * 32, 2) scan_bwd_kernel(const Args a) {
  constexpr int NT = kWarps * 32, RUNS = 32 / LPR, TILE = kWarps * RUNS * R, PIECE = VEC * (int)sizeof(T);
  static_assert(TILE % kKeep == 0, "every tile starts at a kept state");
  extern __shared__ __align__(16) char stage[];  // [kStages][3][R][NT] pieces, then [kStages][VEC][NT] floats
  __shared__ __align__(16) float tot[2][kWarps][LPR][3 * VEC];
  __shared__ __align__(16) Exchange<VEC, CLUSTER ? LPR : 1> ex;
  float* kept = reinterpret_cast<float*>(stage + kStages * 3 * R * NT * PIECE);
  const Place<VEC, LPR> at(a, CLUSTER);
  if constexpr (CLUSTER) open_exchange(ex, a.K);
  const T *g = (const T*)a.g, *x = (const T*)a.x, *dO = (const T*)a.dO;
  const bool mine = at.c < a.D;
  const size_t base = at.bh * (size_t)a.T * a.D + (mine ? at.c : 0);
  const size_t kept_rows = at.bh * (size_t)((a.T + (long long)kKeep - 1) / kKeep);
  float carry[VEC];  // e behind the tiles still to come
#pragma unroll
  for (int j = 0; j < VEC; ++j) carry[j] = mine && a.first ? a.first[at.bh * a.D + at.c + j] : 0.f;
  bool alive = true;

  auto tile_token = [&](int step) {  // negative in front of the sequence (the last step of some ranks)
    return ((long long)a.tiles - 1 - ((long long)step * a.K + at.rank)) * TILE;
  };
  auto place = [&](int step, int which, int i) {
    return stage + ((((step % kStages) * 3 + which) * R + i) * NT + threadIdx.x) * PIECE;
  };
  auto keep_at = [&](int step, int j) { return kept + ((step % kStages) * VEC + j) * NT + threadIdx.x; };
  auto prefetch = [&](int step) {
    if (step < a.steps) {
      const long long tile = tile_token(step), t0 = tile + (at.warp * RUNS + at.run_in_warp) * R;
      const bool real = mine && tile >= 0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bool in = real && t0 + i < a.T;
        const size_t p = in ? base + (size_t)(t0 + i) * a.D : 0;
        fetch<T, VEC>(place(step, 0, i), g + p, in);
        fetch<T, VEC>(place(step, 1, i), x + p, in);
        fetch<T, VEC>(place(step, 2, i), dO + p, in);
      }
      const size_t n = real ? (kept_rows + (size_t)(tile / kKeep)) * a.D + at.c : 0;
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        cl::copy_async<4>(gla::sm100::smem_u32(keep_at(step, j)), a.hc_in + (real ? n + j : 0), real);
    }
    cl::copy_commit();
  };
  for (int s = 0; s < kStages; ++s) prefetch(s);

  for (int step = 0; step < a.steps; ++step) {
    cl::copy_wait<kStages - 1>();
    float ai[R][VEC], ri[COMP ? R : 1][VEC];  // a, and 1 - a where it is needed
    Pair<VEC> f, e, warp_f, warp_e;           // forward and reverse action of the run
    f.identity();
    e.identity();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const Pack<T, VEC> pg = *reinterpret_cast<const Pack<T, VEC>*>(place(step, 0, i));
      const Pack<T, VEC> px = *reinterpret_cast<const Pack<T, VEC>*>(place(step, 1, i));
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float rest;
        ai[i][j] = decay<T>(pg.get(j), &rest);
        if constexpr (COMP) ri[i][j] = rest;
        f.H[j] = fmaf(ai[i][j], f.H[j], COMP ? rest * px.get(j) : px.get(j));
        f.A[j] *= ai[i][j];
      }
    }
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
      const Pack<T, VEC> pd = *reinterpret_cast<const Pack<T, VEC>*>(place(step, 2, i));
#pragma unroll
      for (int j = 0; j < VEC; ++j) e.H[j] = ai[i][j] * (pd.get(j) + e.H[j]);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) e.A[j] = f.A[j];
    join_warp<VEC, LPR, false>(f, warp_f, at.run_in_warp);
    join_warp<VEC, LPR, true>(e, warp_e, at.run_in_warp);
    if (at.run_in_warp == 0) {
      float* t = tot[step & 1][at.warp][at.lane_c];
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        t[j] = warp_f.A[j], t[VEC + j] = warp_f.H[j], t[2 * VEC + j] = warp_e.H[j];
    }
    __syncthreads();
    float h[VEC];  // the state that enters this run
    Pair<VEC> behind, block;
#pragma unroll
    for (int j = 0; j < VEC; ++j) h[j] = *keep_at(step, j);
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w) {
      const float* t = tot[step & 1][w][at.lane_c];
      if (w < at.warp)
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[j] = fmaf(t[j], h[j], t[VEC + j]);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) h[j] = fmaf(f.A[j], h[j], f.H[j]);
    block.identity();
#pragma unroll
    for (int w = kWarps - 1; w >= 0; --w) {
      if (w == at.warp) behind = block;
      Pair<VEC> n;
      const float* t = tot[step & 1][w][at.lane_c];
#pragma unroll
      for (int j = 0; j < VEC; ++j) n.A[j] = t[j], n.H[j] = t[2 * VEC + j];
      block.then(n);
    }
    float back[VEC];
    if constexpr (CLUSTER) {
      exchange(ex, block, carry, back, step, a.K, at.rank, at.warp, at.run_in_warp, at.lane_c, alive, a.latch);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        back[j] = carry[j];
        carry[j] = fmaf(block.A[j], carry[j], block.H[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) back[j] = fmaf(e.A[j], fmaf(behind.A[j], back[j], behind.H[j]), e.H[j]);
    float hp[R][VEC];  // the states before the run's tokens
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const Pack<T, VEC> px = *reinterpret_cast<const Pack<T, VEC>*>(place(step, 1, i));
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float in = px.get(j);
        hp[i][j] = COMP ? h[j] - in : h[j];
        h[j] = fmaf(ai[i][j], h[j], COMP ? ri[i][j] * in : in);
      }
    }
    const long long tile = tile_token(step), t0 = tile + (at.warp * RUNS + at.run_in_warp) * R;
    const bool real = mine && tile >= 0;
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
      const Pack<T, VEC> pd = *reinterpret_cast<const Pack<T, VEC>*>(place(step, 2, i));
      Pack<T, VEC> og, ox;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = pd.get(j) + back[j];
        back[j] = ai[i][j] * d;
        ox.set(j, COMP ? ri[i][j] * d : d);
        og.set(j, back[j] * hp[i][j]);
      }
      if (real && t0 + i < a.T) {
        const size_t p = base + (size_t)(t0 + i) * a.D;
        ox.store((T*)a.dx + p);
        og.store((T*)a.dg + p);
      }
    }
    prefetch(step + kStages);
  }
  if (a.last && mine && at.rank == 0 && at.warp == 0 && at.run_in_warp == 0)
#pragma unroll
    for (int j = 0; j < VEC; ++j) a.last[at.bh * a.D + at.c + j] = carry[j];
  if constexpr (CLUSTER) cl::sync();
}

template <typename T, bool COMP>
__global__ void scan_step_kernel(const T* __restrict__ g, const T* __restrict__ x, float* __restrict__ S,
                                 T* __restrict__ o, long long n) {
  const long long c = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= n) return;
  float rest;
  const float a = decay<T>(ldf(g + c), &rest), in = ldf(x + c);
  const float h = fmaf(a, S[c], COMP ? rest * in : in);
  S[c] = h;
  stf(o + c, h);
}

#define SCAN_TRY(expr)           \
  do {                           \
    const int _s = (expr);       \
    if (_s != GLA_OK) return _s; \
  } while (0)

int check_sizes(int B, int H, int T, int D, int input, int dtype) {
  if (B <= 0 || H <= 0 || T < 0 || D <= 0) return GLA_ERR_INVALID_ARG;
  if ((long long)B * H > INT_MAX || (long long)B * H * (long long)(T > 0 ? T : 1) > (1LL << 40))
    return GLA_ERR_INVALID_ARG;
  if ((long long)B * H * (((long long)D + 15) / 16) > (1LL << 27)) return GLA_ERR_UNSUPPORTED;
  if (dtype != GLA_DTYPE_F32 && dtype != GLA_DTYPE_BF16) return GLA_ERR_UNSUPPORTED;
  if (input != GLA_SCAN_ADD && input != GLA_SCAN_COMPLEMENT) return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}

// A pointer to per-token values (esize bytes each) or fp32 states (esize = 4).
int check_ptr(const void* p, size_t esize, bool required) {
  if (!p) return required ? GLA_ERR_INVALID_ARG : GLA_OK;
  return gla::aligned_to(p, esize) ? GLA_OK : GLA_ERR_INVALID_ARG;
}

size_t esize(int dtype) { return dtype == GLA_DTYPE_BF16 ? 2 : 4; }
int launched() { return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_CUDA; }

constexpr int kRun = 8;          // tokens a thread
constexpr int kFill = 148 * 2;   // blocks that run at once: two an SM

// Launches one variant; K blocks of a cluster share a slab.  K is the largest power of two that keeps all blocks
// running at once, and no more than there are tiles.
template <typename T, int VEC, int LPR, bool COMP, bool BWD>
int launch(Args a, long long BH, cudaStream_t st) {
  constexpr int TILE = kWarps * (32 / LPR) * kRun, PIECE = VEC * (int)sizeof(T);
  constexpr int SMEM = kStages * (BWD ? 3 * kRun * PIECE + 4 * VEC : 2 * kRun * PIECE) * kWarps * 32;
  a.slabs = (a.D + LPR * VEC - 1) / (LPR * VEC);
  a.tiles = (int)(((long long)a.T + TILE - 1) / TILE);
  const long long cols = BH * a.slabs;
  int K = 1;
  while (K < kMaxK && K * 2 <= a.tiles && cols * K * 2 <= kFill) K *= 2;
  a.K = K;
  a.steps = (a.tiles + K - 1) / K;
  void (*kernel)(const Args);
  if constexpr (BWD)
    kernel = K > 1 ? scan_bwd_kernel<T, VEC, LPR, kRun, COMP, true> : scan_bwd_kernel<T, VEC, LPR, kRun, COMP, false>;
  else
    kernel = K > 1 ? scan_fwd_kernel<T, VEC, LPR, kRun, COMP, true> : scan_fwd_kernel<T, VEC, LPR, kRun, COMP, false>;
  // Shared memory above 48 KB is asked for once per device (and kernel).
  static std::atomic<unsigned long long> allowed[2] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GLA_ERR_CUDA;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(allowed[K > 1].load(std::memory_order_relaxed) & bit) || dev > 63) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess) return GLA_ERR_CUDA;
    allowed[K > 1].fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(cols * K));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = K;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = K > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, (const Args)a) != cudaSuccess) {
    (void)cudaGetLastError();
    return GLA_ERR_CUDA;
  }
  return GLA_OK;
}

// Slabs: rows of 32 pieces (8 bytes each) make the longest requests; where even clusters of them leave most SMs
// idle, slabs of 8 pieces, whose tiles are four times as long, give four times the blocks.
template <typename T, int VEC, bool COMP, bool BWD>
int choose(const Args& a, long long BH, cudaStream_t st) {
  const long long wide = BH * ((a.D + 32 * VEC - 1) / (32 * VEC));
  const long long tiles = ((long long)a.T + 63) / 64;
  const long long blocks = wide * (tiles < kMaxK ? tiles : kMaxK);
  if (blocks * 2 <= kFill && tiles > kMaxK) return launch<T, VEC, 8, COMP, BWD>(a, BH, st);
  return launch<T, VEC, 32, COMP, BWD>(a, BH, st);
}

template <bool BWD>
int run(const Args& a, long long BH, int input, int dtype, cudaStream_t st) {
  const size_t es = esize(dtype);
  // The widest piece that divides a row and every address: at most 8 bytes, or 4 in the backward, whose third
  // array and reverse pairs would otherwise leave room for one block an SM.
  int vec = (int)((BWD ? 4 : 8) / es);
  auto fits = [&](int v) {
    if (a.D % v != 0) return false;
    for (const void* p : {a.g, a.x, a.dO, (const void*)a.o, (const void*)a.dg, (const void*)a.dx})
      if (!gla::aligned_to(p, v * es)) return false;
    return true;
  };
  while (vec > 1 && !fits(vec)) vec /= 2;
  const bool comp = input == GLA_SCAN_COMPLEMENT;
#define SCAN_CHOOSE(TYPE, VEC) (comp ? choose<TYPE, VEC, true, BWD>(a, BH, st) : choose<TYPE, VEC, false, BWD>(a, BH, st))
  if (dtype == GLA_DTYPE_BF16) {
    if constexpr (!BWD)
      if (vec == 4) return SCAN_CHOOSE(bf16, 4);
    return vec == 2 ? SCAN_CHOOSE(bf16, 2) : SCAN_CHOOSE(bf16, 1);
  }
  if constexpr (!BWD)
    if (vec == 2) return SCAN_CHOOSE(float, 2);
  return SCAN_CHOOSE(float, 1);
#undef SCAN_CHOOSE
}

int fwd(const void* g, const void* x, const float* h0, void* o, float* hT, float* hc, int B, int H, int T, int D,
        int input, int dtype, cudaStream_t st) {
  Args a = {};
  a.g = g, a.x = x, a.first = h0, a.o = o, a.last = hT, a.hc = hc;
  a.T = T, a.D = D, a.latch = gla::device_error_latch();
  return run<false>(a, (long long)B * H, input, dtype, st);
}

}  // namespace

extern "C" int gla_scan_fwd(const void* g, const void* x, const float* h0, void* o, float* hT, float* hc, int B,
                            int H, int T, int D, int input, int dtype, void* stream) {
  SCAN_TRY(check_sizes(B, H, T, D, input, dtype));
  const size_t es = esize(dtype);
  SCAN_TRY(check_ptr(g, es, T > 0));
  SCAN_TRY(check_ptr(x, es, T > 0));
  SCAN_TRY(check_ptr(o, es, T > 0));
  SCAN_TRY(check_ptr(h0, 4, false));
  SCAN_TRY(check_ptr(hT, 4, false));
  SCAN_TRY(check_ptr(hc, 4, false));
  return fwd(g, x, h0, o, hT, hc, B, H, T, D, input, dtype, static_cast<cudaStream_t>(stream));
}

extern "C" size_t gla_scan_bwd_workspace(int B, int H, int T, int D, int have_hc) {
  if (have_hc || check_sizes(B, H, T, D, GLA_SCAN_ADD, GLA_DTYPE_F32) != GLA_OK) return 0;
  return gla::align256((size_t)B * H * ((T + (size_t)kKeep - 1) / kKeep) * D * sizeof(float));
}

extern "C" int gla_scan_bwd(const void* g, const void* x, const float* h0, const float* hc, const void* dO,
                            const float* dhT, void* dg, void* dx, float* dh0, int B, int H, int T, int D, int input,
                            int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  SCAN_TRY(check_sizes(B, H, T, D, input, dtype));
  const size_t es = esize(dtype);
  SCAN_TRY(check_ptr(g, es, T > 0));
  SCAN_TRY(check_ptr(x, es, T > 0));
  SCAN_TRY(check_ptr(dO, es, T > 0));
  SCAN_TRY(check_ptr(dg, es, T > 0));
  SCAN_TRY(check_ptr(dx, es, T > 0));
  SCAN_TRY(check_ptr(h0, 4, false));
  SCAN_TRY(check_ptr(hc, 4, false));
  SCAN_TRY(check_ptr(dhT, 4, false));
  SCAN_TRY(check_ptr(dh0, 4, false));
  const size_t need = gla_scan_bwd_workspace(B, H, T, D, hc != nullptr);
  if (need > 0 && (!workspace || !gla::aligned_to(workspace, 256) || workspace_bytes < need)) return GLA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (need > 0) {
    SCAN_TRY(fwd(g, x, h0, nullptr, nullptr, static_cast<float*>(workspace), B, H, T, D, input, dtype, st));
    hc = static_cast<const float*>(workspace);
  }
  Args a = {};
  a.g = g, a.x = x, a.dO = dO, a.hc_in = hc, a.first = dhT, a.dg = dg, a.dx = dx, a.last = dh0;
  a.T = T, a.D = D, a.latch = gla::device_error_latch();
  return run<true>(a, (long long)B * H, input, dtype, st);
}

extern "C" int gla_scan_step(const void* g, const void* x, float* S, void* o, int B, int H, int D, int input,
                             int dtype, void* stream) {
  SCAN_TRY(check_sizes(B, H, 1, D, input, dtype));
  const size_t es = esize(dtype);
  SCAN_TRY(check_ptr(g, es, true));
  SCAN_TRY(check_ptr(x, es, true));
  SCAN_TRY(check_ptr(S, 4, true));
  SCAN_TRY(check_ptr(o, es, true));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long n = (long long)B * H * D;
  const unsigned grid = (unsigned)((n + 127) / 128);
#define SCAN_STEP(TYPE, COMP) \
  scan_step_kernel<TYPE, COMP><<<grid, 128, 0, st>>>((const TYPE*)g, (const TYPE*)x, S, (TYPE*)o, n)
  const bool comp = input == GLA_SCAN_COMPLEMENT;
  if (dtype == GLA_DTYPE_BF16) {
    if (comp) SCAN_STEP(bf16, true);
    else SCAN_STEP(bf16, false);
  } else {
    if (comp) SCAN_STEP(float, true);
    else SCAN_STEP(float, false);
  }
#undef SCAN_STEP
  return launched();
}
