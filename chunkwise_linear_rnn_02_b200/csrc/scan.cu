// Elementwise gated linear recurrence (C ABI in include/gla.h, gla_scan_*):
//
//     h_t = a_t h_{t-1} + b_t,   a_t = exp g_t,   b_t = x_t  or  (1 - a_t) x_t
//
// Measured, bf16: B=8, T=2048, C=2048 forward 34 us (5.9 TB/s), backward 63 us (5.3 TB/s), for the complement 40 and
// 72 us; B=1, T=32768, C=1024 (clusters of eight) forward 47 us, backward 91 us; one token of 32 x 2048 1.4 us.
// fp32, B=8, T=2048, C=2048: 66 us (6.1 TB/s) and 110 us (6.1 TB/s).
//
// HBM-bound: g and x are read once and o written once.  A run of tokens acts on the state in front of it as
// h -> A h + H with A the product of its a's and H its end state from zero, and two runs one after the other
// act as (A2 A1, A2 H1 + H2).  So every thread reduces a run of R tokens of two neighbouring channels to (A, H), the
// pairs are joined in token order across the lanes of a warp (shuffles), the warps of a block (shared memory) and the
// blocks of a cluster (their shared memory), and then each thread walks its run again from the state that enters it.
//
// Split: a block owns a slab of 2 LPR channels and steps through the tokens; a step is a tile of 4 (32 / LPR) R
// tokens.  Where there are too few slabs to fill the SMs, K blocks of a cluster share a slab and take its tiles in
// turn.  Each step every block sends its (A, H) to all blocks of the cluster (st.async onto an mbarrier in the
// receiver's shared memory); every block folds all K of them, in token order, into a carry of its own.  So nothing
// goes through global memory, nothing waits outside the cluster, whose blocks run together, and the order of all
// operations is fixed by the sizes, the type and the alignment (which also chooses between TMA and copies by the threads, and
// so between slabs and clusters: scan_plan.cuh).
//
// (All times here and below: replays of a CUDA graph of 20 calls, inputs larger than L2 except where they are small.)
// What a step costs is instructions (a value has 6 bytes to move at bf16, about 30 issue slots an SM at full
// bandwidth): two channels a thread go through the packed fp32 pair arithmetic of sm_100a, tiles come by TMA, and a
// step has one __syncthreads, which also says that the tile's values are in registers and its place can be filled
// again.
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
#include "fused_common.cuh"
#include "pair_math.cuh"
#include "scan_cluster.cuh"
#include "scan_plan.cuh"
#include "vec.cuh"

namespace {

using gla::add2;
using gla::bf16;
using gla::f2;
using gla::F2;
using gla::fma2;
using gla::hi;
using gla::ldf;
using gla::lo;
using gla::mul2;
using gla::stf;
using gla::Two;
using gla::scan::kByThread;
using gla::scan::kKeep;
using gla::scan::kTma;
using gla::scan::Plan;
namespace cl = gla::cluster;
namespace sm = gla::sm100;

constexpr float kLog2e = gla::fast::kLog2e;
constexpr double kLn2Exact = 0.693147180559945309417;
constexpr float kLn2 = (float)kLn2Exact, kLn2Rest = (float)(kLn2Exact - (double)kLn2);

__device__ __forceinline__ F2 shfl2(F2 a, int src) {
  return f2(__shfl_sync(0xffffffffu, lo(a), src), __shfl_sync(0xffffffffu, hi(a), src));
}

__device__ __forceinline__ float max_nan(float x, float y) {  // NaN where either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// x -> (e^x - 1) / x by a polynomial with c0 = 1 and the coefficients that keep its largest relative error smallest (found by
// Lawson's reweighted least squares, rounded to fp32): 2^-25.8 for |x| <= ln 2 / 2 (WIDE), 2^-23.3 for -1/2 <= x <= 0.
template <bool WIDE>
__device__ __forceinline__ F2 rise(F2 x) {
  F2 t;
  if constexpr (WIDE) {
    t = fma2(x, f2(0.0013882521f), f2(0.0083665224f));
    t = fma2(x, t, f2(0.0416672006f));
    t = fma2(x, t, f2(0.1666654348f));
    t = fma2(x, t, f2(0.4999999702f));
  } else {
    t = fma2(x, f2(0.0068076085f), f2(0.0410424843f));
    t = fma2(x, t, f2(0.1665636003f));
    t = fma2(x, t, f2(0.4999946356f));
  }
  return fma2(x, t, f2(1.f));
}

// a = exp g and, with REST, 1 - a.  Neither the 1 - a of a slow gate nor a long product of a's may lose its leading digits,
// so that near g = 0 both come from exp g - 1.
//   fp32   g = n ln 2 + f with n whole and |f| <= ln 2 / 2 (the reduction of Cody and Waite), s = 2^n, p = exp f - 1:
//          a = s + s p is off by 2.5 2^-24 and 1 - a = (1 - s) - s p, which is -p for n = 0, by 5 2^-24, however strong the gate.
//          n is in the low bits of a sum with 2^23 + 2^22 + 127; these, moved up, are s.  From g = -88 on (and where a would be
//          below 2^-126) n is -127 and s zero.
//   bf16   the approximate exponential, off by 2^-22 and by |g| 2^-24 for its argument, but near 0 the polynomial: with REST for
//          |g| < 1/2, since beyond it a / (1 - a) < 1.55 and 1 - a is off by 2^-20.8 at most; for a alone for |g| < 1/32, where
//          three terms of the series do (g^4/24 < 2^-24).  (As at fp32 it takes a fifteenth longer, B=8, T=2048, C=2048 forward.)
template <typename T, bool REST>
__device__ __forceinline__ F2 decay(F2 g, F2* rest) {
  if constexpr (sizeof(T) == 4) {
    constexpr float kWhole = 12582912.f + 127.f;
    g = f2(max_nan(lo(g), -88.f), max_nan(hi(g), -88.f));
    const F2 r = fma2(g, f2(kLog2e), f2(kWhole)), n = add2(r, f2(-kWhole));
    const F2 f = fma2(n, f2(-kLn2Rest), fma2(n, f2(-kLn2), g)), t = rise<true>(f);
    const F2 s = f2(__uint_as_float(__float_as_uint(lo(r)) << 23), __uint_as_float(__float_as_uint(hi(r)) << 23));
    const F2 sf = mul2(s, f);
    if constexpr (!REST) return fma2(sf, t, s);
    const F2 sp = mul2(sf, t);
    *rest = fma2(sp, f2(-1.f), fma2(s, f2(-1.f), f2(1.f)));
    return add2(s, sp);
  } else {
    constexpr float kNear = REST ? 0.5f : 0.03125f;
    const F2 t = REST ? rise<false>(g) : fma2(g, fma2(g, f2(1.f / 6.f), f2(0.5f)), f2(1.f)), near = fma2(t, g, f2(1.f));
    const F2 y = mul2(g, f2(kLog2e)), far = f2(gla::fast_ex2(lo(y)), gla::fast_ex2(hi(y)));
    const bool s0 = fabsf(lo(g)) < kNear, s1 = fabsf(hi(g)) < kNear;
    if constexpr (REST) {
      const F2 rn = mul2(t, mul2(g, f2(-1.f))), rf = fma2(far, f2(-1.f), f2(1.f));
      *rest = f2(s0 ? lo(rn) : lo(rf), s1 ? hi(rn) : hi(rf));
    }
    return f2(s0 ? lo(near) : lo(far), s1 ? hi(near) : hi(far));
  }
}

// The action h -> A h + H of a run on two channels.
struct Pair {
  F2 A, H;
  __device__ __forceinline__ void identity() { A = f2(1.f), H = f2(0.f); }
  // this := n after this
  __device__ __forceinline__ void then(const Pair& n) {
    H = fma2(n.A, H, n.H);
    A = mul2(A, n.A);
  }
  __device__ __forceinline__ F2 of(F2 h) const { return fma2(A, h, H); }
};

// Exclusive join over the runs of a warp, in token order (or against it): `p` becomes what lies before this
// lane's run, `all` the whole warp's.
template <int LPR, bool REVERSE>
__device__ __forceinline__ void join_warp(Pair& p, Pair& all, int run) {
  constexpr int RUNS = 32 / LPR;
  if constexpr (RUNS == 1) {
    all = p;
    p.identity();
  } else {
    const int lane = threadIdx.x & 31, at = REVERSE ? RUNS - 1 - run : run;
    auto from = [&](int d) { return (lane + (REVERSE ? d : -d) * LPR) & 31; };
#pragma unroll
    for (int d = 1; d < RUNS; d *= 2) {
      Pair q;
      q.A = shfl2(p.A, from(d)), q.H = shfl2(p.H, from(d));
      if (at >= d) {
        q.then(p);
        p = q;
      }
    }
    const int last = lane % LPR + (REVERSE ? 0 : (RUNS - 1) * LPR);
    Pair q;
    q.A = shfl2(p.A, from(1)), q.H = shfl2(p.H, from(1));
    all.A = shfl2(p.A, last), all.H = shfl2(p.H, last);
    if (at == 0) p.identity();
    else p = q;
  }
}

struct Args {
  const void* in[3];   // g, x and, in the backward, dO
  const float* first;  // h0 (forward), dhT (backward), or null
  const float* hc_in;  // backward: kept states
  void *out0, *out1;   // o (may be null), or dx and dg
  float *last, *hc;    // hT (forward), dh0 (backward); kept states (forward); or null
  int T, D, slabs;     // slabs of channels a head
  int steps, tiles, K;
  int pairs;           // rows and tensors are aligned to two values
  unsigned int* latch;
};
struct Maps {
  CUtensorMap m[3];
};

// Cluster exchange: two slots with every rank's pair, each on an mbarrier.
template <int LPR, int MAXK>
struct Exchange {
  float4 slot[2][MAXK][LPR];
  uint64_t bar[2];
};

template <typename T, int W, int LPR, int R, int NIN, int STAGES, int MAXK, bool CLUSTER, int LOAD>
struct Block {
  static constexpr int RUNS = 32 / LPR, TILE = W * RUNS * R, CW = 2 * LPR;
  static constexpr int ROW = CW * (int)sizeof(T), ARRAY = TILE * ROW, STAGE = NIN * ARRAY;
  typedef typename Two<T>::Raw Raw;
  typedef Exchange<CLUSTER ? LPR : 1, CLUSTER ? MAXK : 1> Ex;

  const Args& a;
  char* stage;
  uint64_t* full;  // [STAGES]
  Ex& ex;
  int lane_c, run, warp, c, slab;
  size_t bh;
  uint32_t rank;
  int gave_up;  // after a wait has run out, the step whose tile came last or never; kNever before
  bool mine0, mine1;
  static constexpr int kNever = INT_MAX;

  __device__ __forceinline__ Block(const Args& args, char* smem, uint64_t* bars, Ex& e)
      : a(args), stage(smem), full(bars), ex(e), gave_up(kNever) {
    const int lane = threadIdx.x & 31;
    lane_c = lane % LPR, run = lane / LPR, warp = threadIdx.x >> 5;
    const uint32_t col = CLUSTER ? blockIdx.x / (uint32_t)a.K : blockIdx.x;
    rank = CLUSTER ? cl::block_rank() : 0;
    bh = col / (uint32_t)a.slabs;
    slab = (int)(col - (uint32_t)bh * (uint32_t)a.slabs);
    c = slab * CW + lane_c * 2;
    mine0 = c < a.D, mine1 = c + 1 < a.D;
    if (threadIdx.x == 0) {
      if constexpr (LOAD == kTma)
        for (int s = 0; s < STAGES; ++s) sm::mbar_init(&full[s], 1);
      if constexpr (CLUSTER)
        for (int s = 0; s < 2; ++s) sm::mbar_init(&ex.bar[s], 1);
      sm::fence_mbar_init();
      if constexpr (CLUSTER)
        for (int s = 0; s < 2; ++s) sm::mbar_arrive_expect_tx(&ex.bar[s], (uint32_t)(a.K * LPR * 16));
    }
    if constexpr (CLUSTER) cl::sync();
    else __syncthreads();
  }

  __device__ __forceinline__ size_t row(long long t) const { return (bh * (size_t)a.T + (size_t)t) * a.D + c; }
  __device__ __forceinline__ int first_row() const { return (warp * RUNS + run) * R; }

  // Values of a state row [bh][D].
  __device__ __forceinline__ F2 state(const float* p) const {
    return f2(p && mine0 ? p[bh * a.D + c] : 0.f, p && mine1 ? p[bh * a.D + c + 1] : 0.f);
  }
  __device__ __forceinline__ void keep(float* p, F2 v) const {
    if (mine0) p[0] = lo(v);
    if (mine1) p[1] = hi(v);
  }

  // This thread's values of the R tokens from t0, zeros from T on (INSIDE: there are none such).  Channels behind the
  // last one stay as they are: what is computed for them goes nowhere.
  template <bool INSIDE>
  __device__ __forceinline__ void fetch(char* at, long long t0) const {
    constexpr int ES = (int)sizeof(T);
    if (!mine0) return;
#pragma unroll
    for (int n = 0; n < NIN; ++n) {
      const T* src = (const T*)a.in[n];
      const T* p = src + (INSIDE || t0 < a.T ? row(t0) : 0);
      char* dst = at + n * ARRAY + first_row() * ROW + lane_c * 2 * ES;
      if (a.pairs) {
#pragma unroll
        for (int i = 0; i < R; ++i, p += a.D) {
          const bool in = INSIDE || t0 + i < a.T;
          cl::copy_async<2 * ES>(sm::smem_u32(dst + i * ROW), in ? p : src, in);
        }
      } else if constexpr (ES == 4) {
#pragma unroll
        for (int i = 0; i < R; ++i, p += a.D) {
          const bool in = INSIDE || t0 + i < a.T;
          cl::copy_async<4>(sm::smem_u32(dst + i * ROW), in ? p : src, in);
          if (mine1) cl::copy_async<4>(sm::smem_u32(dst + i * ROW + 4), in ? p + 1 : src, in);
        }
      } else {  // odd rows of bf16: nothing asynchronous is that narrow
        unsigned short v[R], w[R];
        const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
        for (int i = 0; i < R; ++i, u += a.D) {
          const bool in = INSIDE || t0 + i < a.T;
          v[i] = in ? __ldg(u) : (unsigned short)0;
          w[i] = in && mine1 ? __ldg(u + 1) : (unsigned short)0;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) *reinterpret_cast<uint32_t*>(dst + i * ROW) = v[i] | (uint32_t)w[i] << 16;
      }
    }
  }

  // Starts the copy of the tile whose first token is `tile` (a tile outside the sequence reads as zeros) for
  // step `step`; with kTma by one thread, when all threads have taken the values that lay there.
  __device__ __forceinline__ void prefetch(const Maps& maps, int step, long long tile) {
    char* at = stage + (step % STAGES) * STAGE;
    if constexpr (LOAD == kTma) {
      if (step < a.steps && gave_up == kNever && threadIdx.x == 0) {
        uint64_t* bar = &full[step % STAGES];
        sm::mbar_arrive_expect_tx(bar, STAGE);
        const int t = tile < 0 || tile > a.T ? a.T : (int)tile;
        for (int n = 0; n < NIN; ++n) sm::tma_load_3d(at + n * ARRAY, &maps.m[n], bar, slab * CW, t, (int)bh);
      }
    } else {
      if (step < a.steps) {
        const long long t0 = tile + first_row();
        if (tile >= 0 && t0 + R <= a.T) fetch<true>(at, t0);
        else fetch<false>(at, tile < 0 ? a.T : t0);
      }
      cl::copy_commit();
    }
  }
  __device__ __forceinline__ void arrived(int step) {
    if constexpr (LOAD == kTma) {
      if (gave_up == kNever && !sm::mbar_wait(&full[step % STAGES], (step / STAGES) & 1, a.latch)) gave_up = step;
    } else {
      cl::copy_wait<STAGES - 1>();
    }
  }
  // Where this thread's values of `step` lie, and its pair of token i in array `which`.
  __device__ __forceinline__ const char* place(int step) const {
    return stage + (step % STAGES) * STAGE + first_row() * ROW + lane_c * 2 * (int)sizeof(T);
  }
  __device__ __forceinline__ Raw value(const char* at, int which, int i) const {
    return *reinterpret_cast<const Raw*>(at + which * ARRAY + i * ROW);
  }
  __device__ __forceinline__ void store(T* p, F2 v) const {
    if (LOAD == kTma || a.pairs) {
      *reinterpret_cast<Raw*>(p) = Two<T>::narrow(v);
    } else {
      stf(p, lo(v));
      if (mine1) stf(p + 1, hi(v));
    }
  }

  // Sends the block's pair to the cluster, waits for all pairs, moves `carry` over all of them and returns the
  // state that enters this block's tile.  A slot is used again two steps later: a block sends for step s + 2 after
  // it has taken everybody's pair of step s + 1, and a block sends that only after the __syncthreads behind its
  // reads of step s.
  __device__ __forceinline__ F2 exchange(const Pair& block, F2& carry, int step) {
    F2 enter = carry;
    if constexpr (CLUSTER) {
      const int s = step & 1;
      if (run == 0) {
        for (int r = warp; r < a.K; r += W)
          cl::store_async(cl::peer(sm::smem_u32(&ex.slot[s][rank][lane_c]), r), lo(block.A), hi(block.A), lo(block.H),
                          hi(block.H), cl::peer(sm::smem_u32(&ex.bar[s]), r));
      }
      if (gave_up == kNever) {
        if (!cl::wait(sm::smem_u32(&ex.bar[s]), (step >> 1) & 1, a.latch))
          gave_up = step + 1;
        else if (threadIdx.x == 0)  // the slot's next use, two steps on
          sm::mbar_arrive_expect_tx(&ex.bar[s], (uint32_t)(a.K * LPR * 16));
      }
      for (int r = 0; r < a.K; ++r) {
        if (r == (int)rank) enter = carry;
        const float4 v = ex.slot[s][r][lane_c];
        carry = fma2(f2(v.x, v.y), carry, f2(v.z, v.w));
      }
    } else {
      carry = block.of(carry);
    }
    return enter;
  }
  __device__ __forceinline__ void close(F2 carry) {
    if (a.last && rank == 0 && warp == 0 && run == 0) keep(a.last + bh * a.D + c, carry);
    // After a wait that ran out, the copies still on their way are waited for, again with a limit.
    if (LOAD == kTma && gave_up != kNever && threadIdx.x == 0)
      for (int s = gave_up; s < gave_up + STAGES && s < a.steps; ++s)
        sm::mbar_wait(&full[s % STAGES], (s / STAGES) & 1, a.latch);
    if constexpr (CLUSTER) cl::sync();  // no block leaves while others may still send to it
  }
};

template <typename T, int W, int LPR, int R, int STAGES, int MINB, int MAXK, bool COMP, bool CLUSTER, int LOAD>
__global__ void __launch_bounds__(W * 32, MINB) scan_fwd_kernel(const Args a, const __grid_constant__ Maps maps) {
  typedef Block<T, W, LPR, R, 2, STAGES, MAXK, CLUSTER, LOAD> B;
  extern __shared__ __align__(128) char stage[];
  __shared__ float4 tot[2][W][LPR];
  __shared__ __align__(16) typename B::Ex ex;
  __shared__ uint64_t full[STAGES];
  B b(a, stage, full, ex);
  F2 carry = b.state(a.first);
  const size_t kept_rows = b.bh * (size_t)((a.T + (long long)kKeep - 1) / kKeep);
  auto tile_of = [&](int step) { return ((long long)step * a.K + b.rank) * B::TILE; };
  for (int s = 0; s < STAGES; ++s) b.prefetch(maps, s, tile_of(s));

  for (int step = 0; step < a.steps; ++step) {
    b.arrived(step);
    const long long t0 = tile_of(step) + b.first_row();
    const char* in = b.place(step);
    F2 av[R], bv[R];
    Pair p, warp_all;
    p.identity();
#pragma unroll
    for (int i = 0; i < R; ++i) {  // tokens behind the end have g = x = 0: they leave the state as it is
      F2 rest;
      const F2 x = Two<T>::wide(b.value(in, 1, i));
      av[i] = decay<T, COMP>(Two<T>::wide(b.value(in, 0, i)), &rest);
      bv[i] = COMP ? mul2(rest, x) : x;
      p.H = fma2(av[i], p.H, bv[i]);
      p.A = mul2(p.A, av[i]);
    }
    join_warp<LPR, false>(p, warp_all, b.run);
    if (b.run == 0)
      tot[step & 1][b.warp][b.lane_c] = make_float4(lo(warp_all.A), hi(warp_all.A), lo(warp_all.H), hi(warp_all.H));
    __syncthreads();
    b.prefetch(maps, step + STAGES, tile_of(step + STAGES));
    Pair before, block;  // the block's warps in front of this one; all of them
    before.identity();
    block.identity();
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float4 v = tot[step & 1][w][b.lane_c];
      Pair n;
      n.A = f2(v.x, v.y), n.H = f2(v.z, v.w);
      if (w < b.warp) before.then(n);
      block.then(n);
    }
    F2 h = p.of(before.of(b.exchange(block, carry, step)));
    if (a.hc && t0 < a.T && t0 % kKeep == 0) b.keep(a.hc + (kept_rows + (size_t)(t0 / kKeep)) * a.D + b.c, h);
    if (a.out0 && b.mine0) {
      T* out = (T*)a.out0 + b.row(t0);
      if (t0 + R <= a.T) {
#pragma unroll
        for (int i = 0; i < R; ++i, out += a.D) {
          h = fma2(av[i], h, bv[i]);
          b.store(out, h);
        }
      } else {
#pragma unroll
        for (int i = 0; i < R; ++i, out += a.D) {
          h = fma2(av[i], h, bv[i]);
          if (t0 + i < a.T) b.store(out, h);
        }
      }
    }
  }
  b.close(carry);
}

template <typename T, int W, int LPR, int R, int STAGES, int MINB, int MAXK, bool COMP, bool CLUSTER, int LOAD>
__global__ void __launch_bounds__(W * 32, MINB) scan_bwd_kernel(const Args a, const __grid_constant__ Maps maps) {
  typedef Block<T, W, LPR, R, 3, STAGES, MAXK, CLUSTER, LOAD> B;
  static_assert(B::TILE % kKeep == 0, "every tile starts at a kept state");
  extern __shared__ __align__(128) char stage[];
  __shared__ float4 tot[2][W][LPR];   // A and the forward H of every warp
  __shared__ float2 tot_e[2][W][LPR]; // the reverse E
  __shared__ __align__(16) typename B::Ex ex;
  __shared__ uint64_t full[STAGES];
  B b(a, stage, full, ex);
  F2 carry = b.state(a.first);  // e behind the tiles still to come
  const size_t kept_rows = b.bh * (size_t)((a.T + (long long)kKeep - 1) / kKeep);
  // Negative in front of the sequence (the last step of some ranks).
  auto tile_of = [&](int step) { return ((long long)a.tiles - 1 - ((long long)step * a.K + b.rank)) * B::TILE; };
  auto kept_state = [&](int step) {
    const long long tile = tile_of(step);
    if (step >= a.steps || tile < 0) return f2(0.f);
    const float* p = a.hc_in + (kept_rows + (size_t)(tile / kKeep)) * a.D + b.c;
    return f2(b.mine0 ? p[0] : 0.f, b.mine1 ? p[1] : 0.f);
  };
  for (int s = 0; s < STAGES; ++s) b.prefetch(maps, s, tile_of(s));
  F2 kept_next = kept_state(0);

  for (int step = 0; step < a.steps; ++step) {
    F2 h = kept_next;  // becomes the state that enters this run
    kept_next = kept_state(step + 1);
    b.arrived(step);
    const char* in = b.place(step);
    F2 av[R], rv[COMP ? R : 1];  // a, and 1 - a where it is needed
    typename Two<T>::Raw xr[R], dr[R];
    Pair f, e, warp_f, warp_e;  // forward and reverse action of the run
    f.identity();
    e.identity();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      F2 rest;
      av[i] = decay<T, COMP>(Two<T>::wide(b.value(in, 0, i)), &rest);
      xr[i] = b.value(in, 1, i);
      dr[i] = b.value(in, 2, i);
      F2 x = Two<T>::wide(xr[i]);
      if constexpr (COMP) {
        rv[i] = rest;
        x = mul2(rest, x);
      }
      f.H = fma2(av[i], f.H, x);
      f.A = mul2(f.A, av[i]);
    }
#pragma unroll
    for (int i = R - 1; i >= 0; --i) e.H = mul2(av[i], add2(Two<T>::wide(dr[i]), e.H));
    e.A = f.A;
    join_warp<LPR, false>(f, warp_f, b.run);
    join_warp<LPR, true>(e, warp_e, b.run);
    if (b.run == 0) {
      tot[step & 1][b.warp][b.lane_c] = make_float4(lo(warp_f.A), hi(warp_f.A), lo(warp_f.H), hi(warp_f.H));
      tot_e[step & 1][b.warp][b.lane_c] = make_float2(lo(warp_e.H), hi(warp_e.H));
    }
    __syncthreads();
    b.prefetch(maps, step + STAGES, tile_of(step + STAGES));
    Pair behind, block;
    behind.identity();
    block.identity();
#pragma unroll
    for (int w = W - 1; w >= 0; --w) {
      const float4 v = tot[step & 1][w][b.lane_c];
      const float2 r = tot_e[step & 1][w][b.lane_c];
      Pair n;
      n.A = f2(v.x, v.y), n.H = f2(r.x, r.y);
      if (w > b.warp) behind.then(n);
      block.then(n);
    }
#pragma unroll
    for (int w = 0; w < W - 1; ++w) {
      if (w < b.warp) {
        const float4 v = tot[step & 1][w][b.lane_c];
        h = fma2(f2(v.x, v.y), h, f2(v.z, v.w));
      }
    }
    h = f.of(h);
    F2 back = e.of(behind.of(b.exchange(block, carry, step)));
    F2 hp[R];  // the states before the run's tokens (less x for the complement)
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const F2 x = Two<T>::wide(xr[i]);
      hp[i] = COMP ? fma2(x, f2(-1.f), h) : h;
      h = fma2(av[i], h, COMP ? mul2(rv[i], x) : x);
    }
    const long long tile = tile_of(step), t0 = tile + b.first_row();
    const bool real = b.mine0 && tile >= 0, whole = t0 + R <= a.T;
    size_t at = real ? b.row(t0 + R - 1) : 0;  // one offset: a pointer for each output spills the complement's values
#pragma unroll
    for (int i = R - 1; i >= 0; --i, at -= a.D) {
      const F2 d = add2(Two<T>::wide(dr[i]), back);
      back = mul2(av[i], d);
      if (real && (whole || t0 + i < a.T)) {
        b.store((T*)a.out0 + at, COMP ? mul2(rv[i], d) : d);
        b.store((T*)a.out1 + at, mul2(back, hp[i]));
      }
    }
  }
  b.close(carry);
}

template <typename T, bool COMP>
__global__ void scan_step_kernel(const T* __restrict__ g, const T* __restrict__ x, float* __restrict__ S,
                                 T* __restrict__ o, long long n) {
  const long long c = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= n) return;
  F2 rest;
  const float a = lo(decay<T, COMP>(f2(ldf(g + c)), &rest)), in = ldf(x + c);
  const float h = fmaf(a, S[c], COMP ? lo(rest) * in : in);
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


// Tensor map over [BH, T, D] with boxes of (box_d, box_t) values; everything outside reads as zeros.
bool make_map(CUtensorMap* m, const void* base, long long BH, int T, int D, int box_d, int box_t, bool is_bf16) {
  auto fn = gla::fast::encode_fn();
  if (!fn) return false;
  const cuuint64_t es = is_bf16 ? 2 : 4;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)T, (cuuint64_t)BH};
  const cuuint64_t strides[2] = {(cuuint64_t)D * es, (cuuint64_t)D * es * (cuuint64_t)T};
  const cuuint32_t box[3] = {(cuuint32_t)box_d, (cuuint32_t)box_t, 1}, one[3] = {1, 1, 1};
  return fn(m, is_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base),
            dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int LPR, int LOAD, bool COMP, bool BWD>
int launch(Args a, const Plan& p, long long BH, cudaStream_t st) {
  typedef gla::scan::Shape<sizeof(T) == 2, LPR, BWD> S;
  constexpr int W = S::W, MINB = S::MINB, R = S::R, STAGES = S::STAGES, MAXK = S::MAXK;
  typedef Block<T, W, LPR, R, BWD ? 3 : 2, STAGES, MAXK, true, LOAD> B;
  constexpr int SMEM = STAGES * B::STAGE;
  static_assert(B::TILE == S::TILE && B::CW == S::CW && B::STAGE == S::STAGE && sizeof(typename B::Ex) == S::EXCHANGE,
                "the plan counts with what the kernel takes");
  const int K = p.K;
  const long long cols = p.cols;
  a.slabs = p.slabs, a.tiles = p.tiles, a.K = K, a.steps = p.steps;
  Maps maps;
  if (LOAD == kTma && a.T > 0)
    for (int n = 0; n < (BWD ? 3 : 2); ++n)
      if (!make_map(&maps.m[n], a.in[n], BH, a.T, a.D, B::CW, B::TILE, sizeof(T) == 2)) return GLA_ERR_CUDA;
  void (*kernel)(const Args, const Maps);
  if constexpr (BWD)
    kernel = K > 1 ? scan_bwd_kernel<T, W, LPR, R, STAGES, MINB, MAXK, COMP, true, LOAD>
                   : scan_bwd_kernel<T, W, LPR, R, STAGES, MINB, MAXK, COMP, false, LOAD>;
  else
    kernel = K > 1 ? scan_fwd_kernel<T, W, LPR, R, STAGES, MINB, MAXK, COMP, true, LOAD>
                   : scan_fwd_kernel<T, W, LPR, R, STAGES, MINB, MAXK, COMP, false, LOAD>;
  // Shared memory above 48 KB and clusters of 16 are asked for once per device and kernel.
  static std::atomic<bool> done[2][64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GLA_ERR_CUDA;
  if (dev < 0 || dev > 63 || !done[K > 1][dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess ||
        (MAXK > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)) {
      (void)cudaGetLastError();
      return GLA_ERR_CUDA;
    }
    if (dev >= 0 && dev < 64) done[K > 1][dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(cols * K));
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = K;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = K > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, (const Args)a, (const Maps)maps) != cudaSuccess) {
    (void)cudaGetLastError();
    return GLA_ERR_CUDA;
  }
  return GLA_OK;
}

template <typename T, int LOAD, bool COMP, bool BWD>
int launch(const Args& a, long long BH, cudaStream_t st) {
  const Plan p = gla::scan::choose<sizeof(T) == 2, LOAD, COMP, BWD>(BH, a.T, a.D);
  if constexpr (!BWD && (sizeof(T) == 2 || LOAD == kTma))
    if (p.lpr == 32) return launch<T, 32, LOAD, COMP, BWD>(a, p, BH, st);
  if (p.lpr == 16) return launch<T, 16, LOAD, COMP, BWD>(a, p, BH, st);
  return launch<T, 8, LOAD, COMP, BWD>(a, p, BH, st);
}

template <bool BWD>
int run(Args a, long long BH, int input, int dtype, cudaStream_t st) {
  const int es = (int)esize(dtype);
  uintptr_t at = 0;
  for (const void* p : {a.in[0], a.in[1], a.in[2], (const void*)a.out0, (const void*)a.out1}) at |= reinterpret_cast<uintptr_t>(p);
  const bool tma = gla::scan::by_tma(at, a.T, a.D, es);
  a.pairs = gla::scan::fits(at, a.D, es, 2 * es);
  const bool comp = input == GLA_SCAN_COMPLEMENT;
#define SCAN_LAUNCH(TYPE)                                                                                             \
  (tma ? (comp ? launch<TYPE, kTma, true, BWD>(a, BH, st) : launch<TYPE, kTma, false, BWD>(a, BH, st))                \
       : (comp ? launch<TYPE, kByThread, true, BWD>(a, BH, st) : launch<TYPE, kByThread, false, BWD>(a, BH, st)))
  return dtype == GLA_DTYPE_BF16 ? SCAN_LAUNCH(bf16) : SCAN_LAUNCH(float);
#undef SCAN_LAUNCH
}

int fwd(const void* g, const void* x, const float* h0, void* o, float* hT, float* hc, int B, int H, int T, int D,
        int input, int dtype, cudaStream_t st) {
  Args a = {};
  a.in[0] = g, a.in[1] = x, a.first = h0, a.out0 = o, a.last = hT, a.hc = hc;
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
  a.in[0] = g, a.in[1] = x, a.in[2] = dO, a.hc_in = hc, a.first = dhT, a.out0 = dx, a.out1 = dg, a.last = dh0;
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
