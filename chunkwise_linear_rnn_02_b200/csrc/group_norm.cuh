// Group norm with an output gate, channels last (C ABI in include/gla.h, gla_group_norm_*).
//
// A row is one head of one token: D values, normalised on their own in fp32,
//     n = (x - mean) rstd,  u = n w + b,  y = u act(z)  (or act(u) without a gate),
// and, with du = dy act(z), dn = du w,
//     dz = dy u act'(z),   dx = rstd (dn - mean(dn) - n mean(dn n)),   dw = sum du n,   db = sum du
// (without the mean terms of dn for the RMS form; du = dy act'(u) without a gate).
//
// HBM-bound: one pass, a row stays packed in the registers of the lanes that share it, so x, z and dy are read once
// and y, dx, dz written once.  The mean is subtracted before the squares are summed.  What there is to save is
// instructions (at full bandwidth a bf16 value has about 30 issue slots forward, 55 backward) and the latency of two
// dependent row sums: 16 values a lane at bf16, so that D = 512 needs no more than a warp (8 a lane take a third longer
// forward, an eighth backward), packed fp32 pairs for the arithmetic, and the row of the next step loaded before this
// one is worked on.
// A block serves one head and strides over the tokens, so that a lane keeps its channels: w and b are loaded once
// (the backward keeps them in shared memory), and the sums of dw and db stay in registers until the block ends.  They
// are then joined over the block's rows, written as one partial row a block, and a second launch joins the partial
// rows in pairs, in a fixed order (no atomics: the result does not depend on how blocks are scheduled).
//
// Measured (replays of a CUDA graph of 20 calls) with gate and weights: B=8, H=4, T=2048, D=512 bf16 forward 36 us
// (5.7 TB/s), backward 68 us (4.9 TB/s); fp32 72 us (5.6 TB/s) and 133 us (5.0 TB/s); B=8, H=4, D=256, one token 2.0 us.
// That is at the widths that fill a variant (dispatch, below).  Lanes without a channel issue what the others do, so that D = 80
// or 640, 62 % of the places, take 1.3 to 1.5 times as long forward and 1.4 to 1.7 times backward for the same bytes; rows off 16
// bytes have four variants only (bf16 D = 300: 3.5 times as long, D = 1100, a block of 1024 threads a row, 15 times).
#pragma once

#include <limits.h>
#include <math.h>

#include "../../include/gla.h"
#include "pair_math.cuh"
#include "vec.cuh"

namespace gla {
namespace norm {

struct Args {
  const void *x, *z, *dy;
  const float *w, *b;
  void *y, *dx, *dz;
  float *part_w, *part_b;  // backward: [gridDim.x][H][D] partial sums of this launch, or null
  int H, T, D;
  long long tokens;  // B * T
  int shared_w;      // one weight row for all heads
  int rms, head_major;
  float eps, inv_d;
  Divider by_t;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eRest = (float)(1.4426950408889634074 - (double)kLog2e), kLn2 = 0.6931471805599453f;

// 1 / (1 + e^-v) by the approximate base-2 exponential, off by 2^-22, and reciprocal, off by 2^-23.  The exponential's argument
// -y, y = v log2 e, is rounded, which costs |v| 2^-24 of e^-v.  At bf16 that is far below the gate's own 2^-9.  At fp32 what y
// takes too much, r (exact by a fused multiply-add, and the rest of log2 e), is put back as 2^r = 1 + r ln 2 (r^2 is below
// 2^-32), so that the sigmoid is off by 2^-21 for every v.  (r is no number, or infinite, where y is infinite; 1, and below zero
// any r, then leaves the sigmoid at 0 or 1.)
template <typename T>
__device__ __forceinline__ F2 sigmoid2(F2 v) {
  const F2 y = mul2(v, f2(kLog2e)), e = f2(fast_ex2(-lo(y)), fast_ex2(-hi(y)));
  F2 q;
  if constexpr (sizeof(T) == 4) {
    const F2 r = fma2(v, f2(-kLog2eRest), fma2(v, f2(-kLog2e), y));
    q = fma2(e, fma2(f2(fminf(lo(r), 1.f), fminf(hi(r), 1.f)), f2(kLn2), f2(1.f)), f2(1.f));
  } else {
    q = add2(e, f2(1.f));
  }
  return f2(fast_rcp(lo(q)), fast_rcp(hi(q)));
}
// act(v) and its derivative.
template <typename T, int ACT>
__device__ __forceinline__ F2 act2(F2 v, F2* slope) {
  if constexpr (ACT == GLA_ACT_NONE) {
    *slope = f2(1.f);
    return v;
  } else {
    const F2 s = sigmoid2<T>(v), rest = fma2(s, f2(-1.f), f2(1.f));
    if constexpr (ACT == GLA_ACT_SIGMOID) {
      *slope = mul2(s, rest);
      return s;
    } else {
      *slope = mul2(s, fma2(v, rest, f2(1.f)));
      return mul2(v, s);
    }
  }
}

// Sums of N values over the LANES threads that share a row; all of them get the result.  Rows of up to a warp use
// shuffles; wider rows join their warps through shared memory (two buffers in turn, so one barrier a sum is enough).
template <int LANES, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float (*buf)[32][2], int& turn) {
#pragma unroll
  for (int d = (LANES < 32 ? LANES : 32) / 2; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
  if constexpr (LANES > 32) {
    constexpr int W = LANES / 32;
    const int warp = threadIdx.x >> 5, first = warp / W * W;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) buf[turn][warp][i] = s[i];
    __syncthreads();
    float t[N] = {};
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] += buf[turn][first + w][i];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = t[i];
    turn ^= 1;
  }
}

// A lane's values of a row: NV vectors of V neighbouring channels, vector i of lane l being number l + i LANES, kept
// as pairs of values.  A vector is 16 bytes, or 2 values or 1 where rows or tensors are not aligned to more; a pair is
// two values of a vector, or of two vectors where V is 1.
template <typename T, int V, int LANES, int NV>
struct Row {
  static constexpr int E = V * NV, P = E / 2;
  static_assert(E % 2 == 0, "pairs");
  typename Two<T>::Raw v[P];

  static __device__ __forceinline__ int channel(int lane, int e) { return (lane + e / V * LANES) * V + e % V; }

  // Values behind the last channel stay as they are: zero from the start.
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int p = 0; p < P; ++p) v[p] = 0;
  }
  __device__ __forceinline__ void load(const T* row, int lane, int D) {
    if constexpr (V * sizeof(T) == 16) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (channel(lane, i * V) < D)
          reinterpret_cast<uint4*>(v)[i] = __ldg(reinterpret_cast<const uint4*>(row + channel(lane, i * V)));
    } else if constexpr (V == 2) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (channel(lane, 2 * i) < D)
          v[i] = __ldg(reinterpret_cast<const typename Two<T>::Raw*>(row + channel(lane, 2 * i)));
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        T t[2];
        stf(&t[0], 0.f), stf(&t[1], 0.f);
        if (channel(lane, 2 * p) < D) t[0] = __ldg(row + channel(lane, 2 * p));
        if (channel(lane, 2 * p + 1) < D) t[1] = __ldg(row + channel(lane, 2 * p + 1));
        v[p] = Two<T>::narrow(f2(ldf(&t[0]), ldf(&t[1])));
      }
    }
  }
  __device__ __forceinline__ void store(T* row, int lane, int D) const {
    if constexpr (V * sizeof(T) == 16) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (channel(lane, i * V) < D)
          *reinterpret_cast<uint4*>(row + channel(lane, i * V)) = reinterpret_cast<const uint4*>(v)[i];
    } else if constexpr (V == 2) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (channel(lane, 2 * i) < D)
          *reinterpret_cast<typename Two<T>::Raw*>(row + channel(lane, 2 * i)) = v[i];
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const F2 t = get(p);  // v holds rounded values: widening and narrowing again is exact
        if (channel(lane, 2 * p) < D) stf(row + channel(lane, 2 * p), lo(t));
        if (channel(lane, 2 * p + 1) < D) stf(row + channel(lane, 2 * p + 1), hi(t));
      }
    }
  }
  __device__ __forceinline__ F2 get(int p) const { return Two<T>::wide(v[p]); }
  __device__ __forceinline__ void set(int p, F2 x) { v[p] = Two<T>::narrow(x); }  // rounds, once
};

constexpr int threads_of(int lanes) { return lanes < 128 ? 128 : lanes; }
constexpr int rows_of(int lanes) { return threads_of(lanes) / lanes; }

template <typename T, int V, int LANES, int NV, int ACT, bool GATE, bool BWD, int MINB>
__global__ void __launch_bounds__(threads_of(LANES), MINB) norm_kernel(const Args a) {
  constexpr int THREADS = threads_of(LANES), ROWS = rows_of(LANES);
  typedef Row<T, V, LANES, NV> R;
  constexpr int P = R::P, E = R::E;
  __shared__ float buf[2][32][2];
  int turn = 0;
  const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES, h = blockIdx.y, D = a.D;
  // w and b of this lane's channels: in registers, or, where the running sums take those (SHARED), in shared memory,
  // four values of a lane together and the lanes side by side.
  constexpr bool SHARED = (BWD ? E >= 8 : E >= 32) && LANES * E <= 4096;  // 32 KB at most
  __shared__ float4 ws[SHARED ? E / 4 : 1][SHARED ? LANES : 1], bs[SHARED ? E / 4 : 1][SHARED ? LANES : 1];
  F2 wr[SHARED ? 1 : P], br[SHARED ? 1 : P], sw[BWD ? P : 1], sb[BWD ? P : 1];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float t[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = R::channel(lane, 2 * p + j);
      const size_t at = (size_t)(a.shared_w ? 0 : h) * D + c;
      t[j] = c < D && a.w ? a.w[at] : 1.f;
      t[2 + j] = c < D && a.b ? a.b[at] : 0.f;
    }
    if constexpr (SHARED) {
      if (sub == 0) {
        reinterpret_cast<float2*>(&ws[p / 2][lane])[p % 2] = make_float2(t[0], t[1]);
        reinterpret_cast<float2*>(&bs[p / 2][lane])[p % 2] = make_float2(t[2], t[3]);
      }
    } else {
      wr[p] = f2(t[0], t[1]), br[p] = f2(t[2], t[3]);
    }
    if constexpr (BWD) sw[p] = sb[p] = f2(0.f);
  }
  if constexpr (SHARED) __syncthreads();
  auto w_of = [&](int p) {
    if constexpr (!SHARED) return wr[p];
    const float4 v = ws[p / 2][lane];
    return p % 2 ? f2(v.z, v.w) : f2(v.x, v.y);
  };
  auto b_of = [&](int p) {
    if constexpr (!SHARED) return br[p];
    const float4 v = bs[p / 2][lane];
    return p % 2 ? f2(v.z, v.w) : f2(v.x, v.y);
  };
  // Where this thread's rows lie: of y, z, dy at `row`, of x and dx at `xrow`.  Every thread of the block takes the
  // same number of steps (the barriers of wide rows count on it).
  const long long step = (long long)gridDim.x * ROWS;
  const size_t row_step = (size_t)step * a.H * D, x_step = a.head_major ? (size_t)step * D : row_step;
  long long tok = (long long)blockIdx.x * ROWS + sub;
  size_t row = ((size_t)tok * a.H + h) * D, xrow = row;
  uint32_t t = 0;  // head-major: the token's place in its sequence
  if (a.head_major && tok < a.tokens) {
    const uint32_t bb = a.by_t.quot((uint32_t)tok);
    t = (uint32_t)tok - bb * (uint32_t)a.T;
    xrow = (((size_t)bb * a.H + h) * a.T + t) * D;
  }
  R nx, nz, nd;
  nx.zero(), nz.zero(), nd.zero();
  auto load = [&]() {
    if (tok >= a.tokens) return;  // what was loaded last stays and is not used
    nx.load((const T*)a.x + xrow, lane, D);
    if constexpr (GATE) nz.load((const T*)a.z + row, lane, D);
    if constexpr (BWD) nd.load((const T*)a.dy + row, lane, D);
  };
  load();
  for (long long first = (long long)blockIdx.x * ROWS; first < a.tokens; first += step) {
    R px = nx, pz = nz, pd = nd;
    const bool live = tok < a.tokens;
    if (BWD && !live) px.zero(), pz.zero(), pd.zero();  // a row that is none adds nothing to the sums of dw and db
    const size_t out = row, xout = xrow;
    tok += step, row += row_step, xrow += x_step;
    if (a.head_major && tok < a.tokens) {
      t += (uint32_t)step;
      if (t >= (uint32_t)a.T) {
        const uint32_t q = a.by_t.quot(t);
        t -= q * (uint32_t)a.T;
        xrow += (size_t)q * (a.H - 1) * a.T * D;
      }
    }
    load();  // the next step's row

    F2 c[P];  // x less its mean, zero behind the last channel
    if (!a.rms) {
      F2 s2 = px.get(0);
#pragma unroll
      for (int p = 1; p < P; ++p) s2 = add2(s2, px.get(p));
      float s[1] = {lo(s2) + hi(s2)};
      row_sum<LANES>(s, buf, turn);
      const float m = -s[0] * a.inv_d;
#pragma unroll
      for (int p = 0; p < P; ++p)
        c[p] = add2(px.get(p), f2(R::channel(lane, 2 * p) < D ? m : 0.f, R::channel(lane, 2 * p + 1) < D ? m : 0.f));
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) c[p] = px.get(p);
    }
    F2 q2 = mul2(c[0], c[0]);
#pragma unroll
    for (int p = 1; p < P; ++p) q2 = fma2(c[p], c[p], q2);
    float q[1] = {lo(q2) + hi(q2)};
    row_sum<LANES>(q, buf, turn);
    const float rstd = rsqrtf(q[0] * a.inv_d + a.eps);
    R o;
    if constexpr (!BWD) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        F2 slope;
        const F2 u = fma2(mul2(c[p], f2(rstd)), w_of(p), b_of(p));
        o.set(p, GATE ? mul2(u, act2<T, ACT>(pz.get(p), &slope)) : act2<T, ACT>(u, &slope));
      }
      if (live) o.store((T*)a.y + out, lane, D);
    } else {
      F2 dn[P], s1 = f2(0.f), s2 = f2(0.f);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const F2 n = mul2(c[p], f2(rstd)), w = w_of(p), u = fma2(n, w, b_of(p)), d = pd.get(p);
        F2 slope, du;
        if constexpr (GATE) {
          du = mul2(d, act2<T, ACT>(pz.get(p), &slope));
          o.set(p, mul2(mul2(d, u), slope));
        } else {
          act2<T, ACT>(u, &slope);
          du = mul2(d, slope);
        }
        sw[p] = fma2(du, n, sw[p]);
        sb[p] = add2(sb[p], du);
        dn[p] = mul2(du, w);
        s1 = add2(s1, dn[p]);
        s2 = fma2(dn[p], n, s2);
      }
      if (GATE && a.dz && live) o.store((T*)a.dz + out, lane, D);
      float s[2] = {lo(s1) + hi(s1), lo(s2) + hi(s2)};
      row_sum<LANES>(s, buf, turn);
      // dx = rstd dn - rstd mean(dn) - c rstd^2 mean(dn n)
      const F2 m1 = f2(a.rms ? 0.f : -rstd * s[0] * a.inv_d), m2 = f2(-rstd * rstd * s[1] * a.inv_d), r = f2(rstd);
#pragma unroll
      for (int p = 0; p < P; ++p) o.set(p, fma2(c[p], m2, fma2(dn[p], r, m1)));
      if (live) o.store((T*)a.dx + xout, lane, D);
    }
  }
  if constexpr (BWD) {
    // One partial row a block: the block's rows are added in order through shared memory.
    __shared__ float sums[ROWS > 1 ? ROWS : 1][2][ROWS > 1 ? LANES * E : 1];
    const size_t out = ((size_t)blockIdx.x * a.H + h) * D;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int ch = R::channel(lane, 2 * p + j);
        const float vw = j ? hi(sw[p]) : lo(sw[p]), vb = j ? hi(sb[p]) : lo(sb[p]);
        if constexpr (ROWS > 1) {
          sums[sub][0][ch] = vw;
          sums[sub][1][ch] = vb;
        } else if (ch < D) {
          if (a.part_w) a.part_w[out + ch] = vw;
          if (a.part_b) a.part_b[out + ch] = vb;
        }
      }
    if constexpr (ROWS > 1) {
      __syncthreads();
      for (int ch = threadIdx.x; ch < D; ch += THREADS) {
        float tw = 0.f, tb = 0.f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) tw += sums[r][0][ch], tb += sums[r][1][ch];
        if (a.part_w) a.part_w[out + ch] = tw;
        if (a.part_b) a.part_b[out + ch] = tb;
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------------- host
// Threads an SM, and so registers a thread: 96 or 128 at bf16 (16 values a lane), 80 at fp32 (8), 128 in the backward.  These leave
// small spills (nvcc 12.9): 8 to 24 bytes a thread in the gated bf16 backward, 8 or 16 in the gated fp32 forward up to
// D = 512; blocks of 1024 threads have 64 registers, and their backward spills 16 to 168 bytes.  More threads with fewer registers
// lose more than they hide: the D = 512 case above takes 45 instead of 36 us forward with 768 threads; short rows, which
// shuffle less, want the registers (H=8, D=64: 8.6 us with 512 threads, 11.6 us with 640).
constexpr int resident(int lanes, bool bwd, bool wide) { return bwd ? 512 : wide ? 768 : lanes <= 16 ? 512 : 640; }
constexpr int blocks_an_sm(int lanes, bool bwd, bool wide) {
  return resident(lanes, bwd, wide) / threads_of(lanes) < 1 ? 1 : resident(lanes, bwd, wide) / threads_of(lanes);
}
// Blocks a head: enough to fill the 148 SMs of a B200, no more than there are steps, by the lanes that share a row
// of 16 values a lane (8 at fp32).  The same for every alignment and, in the backward, which passes wide = false,
// type, so that the workspace follows from the sizes, and for every device, so that the order of the sums does.
inline int row_blocks(long long tokens, int H, int D, bool bwd, bool wide) {
  const int each = wide ? 8 : 16;
  int lanes = 64 / each;
  while (lanes * each < D) lanes *= 2;
  const long long want = (148LL * blocks_an_sm(lanes, bwd, wide) + H - 1) / H;
  const long long most = (tokens + rows_of(lanes) - 1) / rows_of(lanes);
  return (int)(want < most ? want : most);
}

template <typename T, int V, int LANES, int NV, bool BWD>
int launch(const Args& a, int act, int grid_x, cudaStream_t st) {
  constexpr int MINB = NV > 4 ? 1 : blocks_an_sm(LANES, BWD, sizeof(T) == 4);
  const dim3 grid(grid_x, a.H), block(threads_of(LANES));
  constexpr bool GATED = V * NV < 32;
#define NORM_LAUNCH(ACT)                                                                                     \
  (GATED && a.z ? norm_kernel<T, V, LANES, NV, ACT, GATED, BWD, MINB><<<grid, block, 0, st>>>(a)             \
                : norm_kernel<T, V, LANES, NV, ACT, false, BWD, MINB><<<grid, block, 0, st>>>(a))
  if (act == GLA_ACT_SILU) NORM_LAUNCH(GLA_ACT_SILU);
  else if (act == GLA_ACT_SIGMOID) NORM_LAUNCH(GLA_ACT_SIGMOID);
  else NORM_LAUNCH(GLA_ACT_NONE);
#undef NORM_LAUNCH
  return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

// Launches the variant for rows of D values in vectors of V.
template <typename T, bool BWD>
int dispatch(const Args& a, int V, int act, int grid_x, cudaStream_t st) {
  const int D = a.D;
  if constexpr (sizeof(T) == 2) {
    if (V == 8) {
      if (D <= 64) return launch<T, 8, 4, 2, BWD>(a, act, grid_x, st);
      if (D <= 128) return launch<T, 8, 8, 2, BWD>(a, act, grid_x, st);
      if (D <= 256) return launch<T, 8, 16, 2, BWD>(a, act, grid_x, st);
      if (D <= 512) return launch<T, 8, 32, 2, BWD>(a, act, grid_x, st);
      // Without a gate a warp holds 1024 values (32 a lane, w and b in shared memory): 26 against 28 us for 32768 rows of
      // 1024.  With one it spills (79 against 69 us).
      if constexpr (!BWD)
        if (D <= 1024 && !a.z) return launch<T, 8, 32, 4, BWD>(a, act, grid_x, st);
      if (D <= 1024) return launch<T, 8, 64, 2, BWD>(a, act, grid_x, st);
      if (D <= 2048) return launch<T, 8, 128, 2, BWD>(a, act, grid_x, st);
      if (D <= 4096) return launch<T, 8, 256, 2, BWD>(a, act, grid_x, st);
      if constexpr (BWD) return launch<T, 8, 1024, 1, BWD>(a, act, grid_x, st);
      else return launch<T, 8, 512, 2, BWD>(a, act, grid_x, st);
    }
  } else if constexpr (sizeof(T) == 4) {
    if (V == 4) {
      if (D <= 64) return launch<T, 4, 8, 2, BWD>(a, act, grid_x, st);
      if (D <= 128) return launch<T, 4, 16, 2, BWD>(a, act, grid_x, st);
      if (D <= 256) return launch<T, 4, 32, 2, BWD>(a, act, grid_x, st);
      if (D <= 512) return launch<T, 4, 64, 2, BWD>(a, act, grid_x, st);
      if (D <= 1024) return launch<T, 4, 128, 2, BWD>(a, act, grid_x, st);
      if (D <= 2048) return launch<T, 4, 256, 2, BWD>(a, act, grid_x, st);
      if (D <= 4096) return launch<T, 4, 512, 2, BWD>(a, act, grid_x, st);
      return launch<T, 4, 1024, 2, BWD>(a, act, grid_x, st);
    }
  }
  if (V == 2) {
    if (D <= 64) return launch<T, 2, 32, 1, BWD>(a, act, grid_x, st);
    if (D <= 256) return launch<T, 2, 32, 4, BWD>(a, act, grid_x, st);
    if (D <= 1024) return launch<T, 2, 128, 4, BWD>(a, act, grid_x, st);
    return launch<T, 2, 1024, 4, BWD>(a, act, grid_x, st);
  }
  if (D <= 64) return launch<T, 1, 32, 2, BWD>(a, act, grid_x, st);
  if (D <= 256) return launch<T, 1, 32, 8, BWD>(a, act, grid_x, st);
  if (D <= 1024) return launch<T, 1, 128, 8, BWD>(a, act, grid_x, st);
  return launch<T, 1, 1024, 8, BWD>(a, act, grid_x, st);
}

#define NORM_TRY(expr)           \
  do {                           \
    const int _s = (expr);       \
    if (_s != GLA_OK) return _s; \
  } while (0)

inline int check_ptr(const void* p, size_t es, bool required) {
  if (!p) return required ? GLA_ERR_INVALID_ARG : GLA_OK;
  return aligned_to(p, es) ? GLA_OK : GLA_ERR_INVALID_ARG;
}
inline size_t esize(int dtype) { return dtype == GLA_DTYPE_BF16 ? 2 : 4; }

inline int check_sizes(int B, int H, int T, int D, int weight_rows) {
  if (B <= 0 || H <= 0 || T < 0 || D <= 0) return GLA_ERR_INVALID_ARG;
  if (weight_rows != 1 && weight_rows != H) return GLA_ERR_INVALID_ARG;
  if ((long long)B * (T > 0 ? T : 1) > INT_MAX || H > 65535 || D > 8192) return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}
inline int check_kind(int kind, int act, float eps, int layout, int dtype) {
  if (!(eps > 0.f) || !isfinite(eps)) return GLA_ERR_INVALID_ARG;
  if (kind != GLA_NORM_GROUP && kind != GLA_NORM_RMS) return GLA_ERR_UNSUPPORTED;
  if (act < GLA_ACT_NONE || act > GLA_ACT_SIGMOID) return GLA_ERR_UNSUPPORTED;
  if (layout != GLA_LAYOUT_BHTD && layout != GLA_LAYOUT_BTHD) return GLA_ERR_UNSUPPORTED;
  if (dtype != GLA_DTYPE_F32 && dtype != GLA_DTYPE_BF16) return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}

// The vector length: 16 bytes where rows and every tensor start on them, else 2 or 1 values.
inline int vector_of(const Args& a, size_t es) {
  auto fits = [&](int v, size_t bytes) {
    if (a.D % v != 0 || a.D * es % bytes != 0) return false;
    for (const void* p : {a.x, a.z, a.dy, (const void*)a.y, (const void*)a.dx, (const void*)a.dz})
      if (!aligned_to(p, bytes)) return false;
    return true;
  };
  const int wide = (int)(16 / es);
  return fits(wide, 16) ? wide : fits(2, 2 * es) ? 2 : 1;
}

inline Args make_args(const void* x, const void* z, const float* w, const float* b, int B, int H, int T, int D,
                      int weight_rows, int kind, float eps, int layout) {
  Args a = {};
  a.x = x, a.z = z, a.w = w, a.b = b;
  a.H = H, a.T = T, a.D = D;
  a.tokens = (long long)B * T;
  a.shared_w = weight_rows == 1;
  a.rms = kind == GLA_NORM_RMS, a.head_major = layout == GLA_LAYOUT_BHTD;
  a.eps = eps, a.inv_d = 1.f / (float)D;
  a.by_t = Divider((uint32_t)(T > 0 ? T : 1));
  return a;
}

}  // namespace norm
}  // namespace gla
