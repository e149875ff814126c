// Group norm with an output gate, channels last (C ABI in include/gla.h, gla_group_norm_*).
//
// A row is one head of one token: D values, normalised on their own in fp32,
//     n = (x - mean) rstd,  u = n w + b,  y = u act(z)  (or act(u) without a gate),
// and, with du = dy act(z), dn = du w,
//     dz = dy u act'(z),   dx = rstd (dn - mean(dn) - n mean(dn n)),   dw = sum du n,   db = sum du
// (without the mean terms of dn for the RMS form; du = dy act'(u) without a gate).
//
// HBM-bound: one pass, a row stays packed in the registers of the lanes that share it, so x, z and dy
// are read once and y, dx, dz written once.  The mean is subtracted before the squares are summed.
// A block serves one head and strides over the tokens, so that a lane keeps its channels: w and b are
// loaded once, and the sums of dw and db stay in registers until the block ends.  They are then
// joined over the block's rows, written as one partial row a block, and a second launch adds the
// partial rows in order (no atomics: the result does not depend on how blocks are scheduled).
#include <limits.h>
#include <math.h>

#include "../../include/gla.h"
#include "vec.cuh"

namespace {

using gla::bf16;
using gla::Pack;

struct Args {
  const void *x, *z, *dy;
  const float *w, *b;
  void *y, *dx, *dz;
  float *part_w, *part_b;  // [gridDim.x][H][D] partial sums of this launch (backward)
  int H, T, D;
  long long tokens;  // B * T
  int shared_w;      // one weight row for all heads
  int rms, act, head_major;
  float eps, inv_d;
  gla::Divider by_t;
};

template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
  // bf16 results carry 8 bits: the approximate exponential and quotient (a few 2^-22) do for them.
  if constexpr (sizeof(T) == 2) return __fdividef(1.f, 1.f + __expf(-v));
  return 1.f / (1.f + expf(-v));
}
// act(v) and its derivative.
template <typename T>
__device__ __forceinline__ float act(float v, int kind, float* slope) {
  if (kind == GLA_ACT_NONE) {
    *slope = 1.f;
    return v;
  }
  const float s = sigmoid<T>(v);
  if (kind == GLA_ACT_SIGMOID) {
    *slope = s * (1.f - s);
    return s;
  }
  *slope = s * (1.f + v * (1.f - s));
  return v * s;
}

// Sums of N values over the LANES threads that share a row; all of them get the result.  Rows of up
// to a warp use shuffles; wider rows join their warps through shared memory (two buffers in turn, so
// one barrier a sum is enough).
template <int LANES, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float* buf, int& turn) {
#pragma unroll
  for (int d = (LANES < 32 ? LANES : 32) / 2; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
  if constexpr (LANES > 32) {
    constexpr int W = LANES / 32;
    float* p = buf + turn * W * 2;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) p[(threadIdx.x >> 5) * 2 + i] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) t += p[w * 2 + i];
      s[i] = t;
    }
  }
}

// LANES threads share a row, each with NV vectors of V channels: vector i of lane l is number l + i LANES.
template <typename T, int V, int LANES, int NV, bool BWD>
__global__ void __launch_bounds__(LANES < 256 ? 256 : LANES) norm_kernel(const Args a) {
  constexpr int THREADS = LANES < 256 && LANES != 128 ? 256 : LANES, ROWS = THREADS / LANES;
  __shared__ float buf[LANES > 32 ? LANES / 32 * 4 : 1];
  int turn = 0;
  const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES, h = blockIdx.y;
  const int nvec = a.D / V;
  const T *x = (const T*)a.x, *z = (const T*)a.z, *dy = (const T*)a.dy;
  float w[NV * V], b[NV * V], sw[BWD ? NV * V : 1], sb[BWD ? NV * V : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (lane + i * LANES) * V + j, e = i * V + j;
      const bool in = c < a.D;
      const size_t at = (size_t)(a.shared_w ? 0 : h) * a.D + c;
      w[e] = in && a.w ? a.w[at] : 1.f;
      b[e] = in && a.b ? a.b[at] : 0.f;
      if constexpr (BWD) sw[e] = sb[e] = 0.f;
    }
  // Every thread of the block takes the same number of steps (the barriers of wide rows count on it).
  const long long step = (long long)gridDim.x * ROWS;
  for (long long first = (long long)blockIdx.x * ROWS; first < a.tokens; first += step) {
    const long long tok = first + sub;
    const bool live = tok < a.tokens;
    const size_t row = ((size_t)tok * a.H + h) * a.D;  // of y, z, dy
    size_t xrow = row;
    if (a.head_major && live) {
      const uint32_t bb = a.by_t.quot((uint32_t)tok), t = (uint32_t)tok - bb * (uint32_t)a.T;
      xrow = (((size_t)bb * a.H + h) * a.T + t) * a.D;
    }
    Pack<T, V> px[NV], pz[NV], pd[BWD ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * LANES;
      if (live && v < nvec) {
        px[i].load_const(x + xrow + (size_t)v * V);
        if (z) pz[i].load_const(z + row + (size_t)v * V);
        if constexpr (BWD) pd[i].load_const(dy + row + (size_t)v * V);
      } else {
        px[i].zero();
        pz[i].zero();
        if constexpr (BWD) pd[i].zero();
      }
    }
    float mean = 0.f;
    if (!a.rms) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) s[0] += px[i].get(j);
      row_sum<LANES>(s, buf, turn);
      mean = s[0] * a.inv_d;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + i * LANES < nvec)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = px[i].get(j) - mean;
          q[0] = fmaf(d, d, q[0]);
        }
    row_sum<LANES>(q, buf, turn);
    const float rstd = 1.f / sqrtf(q[0] * a.inv_d + a.eps);
    if constexpr (!BWD) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = lane + i * LANES;
        if (!live || v >= nvec) continue;
        Pack<T, V> out;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float slope;
          const float u = fmaf((px[i].get(j) - mean) * rstd, w[i * V + j], b[i * V + j]);
          out.set(j, z ? u * act<T>(pz[i].get(j), a.act, &slope) : act<T>(u, a.act, &slope));
        }
        out.store((T*)a.y + row + (size_t)v * V);
      }
    } else {
      float dn[NV * V], s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = lane + i * LANES;
        Pack<T, V> out;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int e = i * V + j;
          const float n = (px[i].get(j) - mean) * rstd, u = fmaf(n, w[e], b[e]), d = pd[i].get(j);
          float slope, du;
          if (z) {
            const float f = act<T>(pz[i].get(j), a.act, &slope);
            du = d * f;
            out.set(j, d * u * slope);
          } else {
            act<T>(u, a.act, &slope);
            du = d * slope;
          }
          const bool in = live && v < nvec;
          du = in ? du : 0.f;
          if (in) sw[e] = fmaf(du, n, sw[e]);
          sb[e] += du;
          dn[e] = du * w[e];
          s[0] += dn[e];
          s[1] = in ? fmaf(dn[e], n, s[1]) : s[1];
        }
        if (a.dz && live && v < nvec) out.store((T*)a.dz + row + (size_t)v * V);
      }
      row_sum<LANES>(s, buf, turn);
      const float m1 = a.rms ? 0.f : s[0] * a.inv_d, m2 = s[1] * a.inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = lane + i * LANES;
        if (!live || v >= nvec) continue;
        Pack<T, V> out;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float n = (px[i].get(j) - mean) * rstd;
          out.set(j, rstd * (dn[i * V + j] - m1 - n * m2));
        }
        out.store((T*)a.dx + xrow + (size_t)v * V);
      }
    }
  }
  if constexpr (BWD) {
    // One partial row a block: the block's rows are added in order through shared memory.
    extern __shared__ float sums[];  // [ROWS][2][LANES * NV * V] when ROWS > 1
    constexpr int C = LANES * NV * V;
    const size_t out = ((size_t)blockIdx.x * a.H + h) * a.D;
    if constexpr (ROWS > 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = (lane + i * LANES) * V + j;
          sums[(sub * 2 + 0) * C + c] = sw[i * V + j];
          sums[(sub * 2 + 1) * C + c] = sb[i * V + j];
        }
      __syncthreads();
      for (int c = threadIdx.x; c < a.D; c += THREADS) {
        float tw = 0.f, tb = 0.f;
        for (int r = 0; r < ROWS; ++r) {
          tw += sums[(r * 2 + 0) * C + c];
          tb += sums[(r * 2 + 1) * C + c];
        }
        if (a.part_w) a.part_w[out + c] = tw;
        if (a.part_b) a.part_b[out + c] = tb;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = (lane + i * LANES) * V + j;
          if (c >= a.D) continue;
          if (a.part_w) a.part_w[out + c] = sw[i * V + j];
          if (a.part_b) a.part_b[out + c] = sb[i * V + j];
        }
    }
  }
}

// out[r] = sum over p < P of part[p][r], in order: 8 groups of 32 threads take slices of P, 32 columns a block.
__global__ void join_kernel(const float* __restrict__ part_w, const float* __restrict__ part_b, float* __restrict__ dw,
                            float* __restrict__ db, int P, int cols) {
  __shared__ float s[8][32];
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float* out = blockIdx.y == 0 ? dw : db;
  if (!part) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  float t = 0.f;
  if (c < cols)
    for (int p = g; p < P; p += 8) t += part[(size_t)p * cols + c];
  s[g][threadIdx.x & 31] = t;
  __syncthreads();
  if (g == 0 && c < cols) {
    t = 0.f;
    for (int i = 0; i < 8; ++i) t += s[i][threadIdx.x];
    out[c] = t;
  }
}

// Blocks a head: enough to fill the 148 SMs of a B200 a few times over, no more than there are rows.
// (A constant, so that the sums' order and the workspace do not go by the current device.)
int row_blocks(long long tokens, int H, int rows_a_block, int blocks_an_sm) {
  const long long want = (148LL * blocks_an_sm + H - 1) / H;
  const long long most = (tokens + rows_a_block - 1) / rows_a_block;
  return (int)(want < 1 ? 1 : want < most ? want : most < 1 ? 1 : most);
}

template <typename T, int V, int LANES, int NV, bool BWD>
int launch(const Args& a, int grid_x, cudaStream_t st) {
  constexpr int THREADS = LANES < 256 && LANES != 128 ? 256 : LANES, ROWS = THREADS / LANES;
  const size_t smem = BWD && ROWS > 1 ? sizeof(float) * 2 * ROWS * LANES * NV * V : 0;
  norm_kernel<T, V, LANES, NV, BWD><<<dim3(grid_x, a.H), THREADS, smem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

// The number of rows that a block of the variant for nvec vectors works on together.
int rows_of(int nvec) { return nvec <= 8 ? 32 : nvec <= 16 ? 16 : nvec <= 64 ? 8 : 1; }

template <typename T, int V, bool BWD>
int dispatch(const Args& a, int grid_x, cudaStream_t st) {
  const int nvec = a.D / V;
  if (nvec <= 8) return launch<T, V, 8, 1, BWD>(a, grid_x, st);
  if (nvec <= 16) return launch<T, V, 16, 1, BWD>(a, grid_x, st);
  if (nvec <= 32) return launch<T, V, 32, 1, BWD>(a, grid_x, st);
  if (nvec <= 64) return launch<T, V, 32, 2, BWD>(a, grid_x, st);
  if (nvec <= 128) return launch<T, V, 128, 1, BWD>(a, grid_x, st);
  if (nvec <= 256) return launch<T, V, 256, 1, BWD>(a, grid_x, st);
  if (nvec <= 512) return launch<T, V, 512, 1, BWD>(a, grid_x, st);
  if (nvec <= 1024) return launch<T, V, 512, 2, BWD>(a, grid_x, st);
  if constexpr (V <= 4)  // D <= 8192 is 1024 vectors of 8 bf16 at most
    if (nvec <= 2048) return launch<T, V, 512, 4, BWD>(a, grid_x, st);
  if constexpr (V == 1) return launch<T, V, 512, 16, BWD>(a, grid_x, st);
  return GLA_ERR_UNSUPPORTED;
}

#define NORM_TRY(expr)           \
  do {                           \
    const int _s = (expr);       \
    if (_s != GLA_OK) return _s; \
  } while (0)

int check_ptr(const void* p, size_t es, bool required) {
  if (!p) return required ? GLA_ERR_INVALID_ARG : GLA_OK;
  return gla::aligned_to(p, es) ? GLA_OK : GLA_ERR_INVALID_ARG;
}
size_t esize(int dtype) { return dtype == GLA_DTYPE_BF16 ? 2 : 4; }

int check_sizes(int B, int H, int T, int D, int weight_rows) {
  if (B <= 0 || H <= 0 || T < 0 || D <= 0) return GLA_ERR_INVALID_ARG;
  if (weight_rows != 1 && weight_rows != H) return GLA_ERR_INVALID_ARG;
  if ((long long)B * (T > 0 ? T : 1) > INT_MAX || H > 65535 || D > 8192) return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}
int check_kind(int kind, int act, float eps, int layout, int dtype) {
  if (!(eps > 0.f) || !isfinite(eps)) return GLA_ERR_INVALID_ARG;
  if (kind != GLA_NORM_GROUP && kind != GLA_NORM_RMS) return GLA_ERR_UNSUPPORTED;
  if (act < GLA_ACT_NONE || act > GLA_ACT_SIGMOID) return GLA_ERR_UNSUPPORTED;
  if (layout != GLA_LAYOUT_BHTD && layout != GLA_LAYOUT_BTHD) return GLA_ERR_UNSUPPORTED;
  if (dtype != GLA_DTYPE_F32 && dtype != GLA_DTYPE_BF16) return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}

// Whether 16-byte vectors can be used: rows and every tensor start on 16 bytes.
bool vectors(const Args& a, size_t es) {
  if (a.D * es % 16 != 0) return false;
  for (const void* p : {a.x, a.z, a.dy, (const void*)a.y, (const void*)a.dx, (const void*)a.dz})
    if (!gla::aligned_to(p, 16)) return false;
  return true;
}

constexpr int kFwdBlocks = 8, kBwdBlocks = 4;  // blocks an SM

template <bool BWD>
int run(const Args& a, int grid_x, int dtype, bool vec, cudaStream_t st) {
  if (dtype == GLA_DTYPE_BF16)
    return vec ? dispatch<bf16, 8, BWD>(a, grid_x, st) : dispatch<bf16, 1, BWD>(a, grid_x, st);
  return vec ? dispatch<float, 4, BWD>(a, grid_x, st) : dispatch<float, 1, BWD>(a, grid_x, st);
}

Args make_args(const void* x, const void* z, const float* w, const float* b, int B, int H, int T, int D,
               int weight_rows, int kind, int act, float eps, int layout) {
  Args a = {};
  a.x = x, a.z = z, a.w = w, a.b = b;
  a.H = H, a.T = T, a.D = D;
  a.tokens = (long long)B * T;
  a.shared_w = weight_rows == 1;
  a.rms = kind == GLA_NORM_RMS, a.act = act, a.head_major = layout == GLA_LAYOUT_BHTD;
  a.eps = eps, a.inv_d = 1.f / (float)D;
  a.by_t = gla::Divider((uint32_t)(T > 0 ? T : 1));
  return a;
}

// Blocks a head of the backward: one partial row each, whatever the dtype and alignment.
int bwd_blocks(int B, int H, int T) { return row_blocks((long long)B * T, H, 1, kBwdBlocks); }

}  // namespace

extern "C" int gla_group_norm_fwd(const void* x, const void* z, const float* w, const float* b, void* y, int B, int H,
                                  int T, int D, int weight_rows, int kind, int act, float eps, int layout, int dtype,
                                  void* stream) {
  NORM_TRY(check_sizes(B, H, T, D, weight_rows));
  NORM_TRY(check_kind(kind, act, eps, layout, dtype));
  if (T == 0) return GLA_OK;
  const size_t es = esize(dtype);
  NORM_TRY(check_ptr(x, es, true));
  NORM_TRY(check_ptr(z, es, false));
  NORM_TRY(check_ptr(w, 4, false));
  NORM_TRY(check_ptr(b, 4, false));
  NORM_TRY(check_ptr(y, es, true));
  Args a = make_args(x, z, w, b, B, H, T, D, weight_rows, kind, act, eps, layout);
  a.y = y;
  const bool vec = vectors(a, es);
  const int nvec = vec ? (int)(D * es / 16) : D;
  return run<false>(a, row_blocks(a.tokens, H, rows_of(nvec), kFwdBlocks), dtype, vec,
                    static_cast<cudaStream_t>(stream));
}

extern "C" size_t gla_group_norm_bwd_workspace(int B, int H, int T, int D, int weight_rows, int need_dw,
                                               int need_db) {
  if (check_sizes(B, H, T, D, weight_rows) != GLA_OK || T == 0) return 0;
  const size_t one = gla::align256((size_t)bwd_blocks(B, H, T) * H * D * sizeof(float));
  return one * ((need_dw != 0) + (need_db != 0));
}

extern "C" int gla_group_norm_bwd(const void* x, const void* z, const float* w, const float* b, const void* dy,
                                  void* dx, void* dz, float* dw, float* db, int B, int H, int T, int D,
                                  int weight_rows, int kind, int act, float eps, int layout, int dtype,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  NORM_TRY(check_sizes(B, H, T, D, weight_rows));
  NORM_TRY(check_kind(kind, act, eps, layout, dtype));
  const size_t es = esize(dtype);
  NORM_TRY(check_ptr(x, es, T > 0));
  NORM_TRY(check_ptr(z, es, T > 0 && dz));
  NORM_TRY(check_ptr(w, 4, false));
  NORM_TRY(check_ptr(b, 4, false));
  NORM_TRY(check_ptr(dy, es, T > 0));
  NORM_TRY(check_ptr(dx, es, T > 0));
  NORM_TRY(check_ptr(dz, es, false));
  NORM_TRY(check_ptr(dw, 4, false));
  NORM_TRY(check_ptr(db, 4, false));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t n_w = (size_t)weight_rows * D * sizeof(float);
  if (T == 0) {
    if (dw && cudaMemsetAsync(dw, 0, n_w, st) != cudaSuccess) return GLA_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, n_w, st) != cudaSuccess) return GLA_ERR_CUDA;
    return GLA_OK;
  }
  const size_t need = gla_group_norm_bwd_workspace(B, H, T, D, weight_rows, dw != nullptr, db != nullptr);
  if (need > 0 && (!workspace || !gla::aligned_to(workspace, 256) || workspace_bytes < need)) return GLA_ERR_WORKSPACE;
  Args a = make_args(x, z, w, b, B, H, T, D, weight_rows, kind, act, eps, layout);
  a.dy = dy, a.dx = dx, a.dz = dz;
  const int P = bwd_blocks(B, H, T);
  if (dw) a.part_w = static_cast<float*>(workspace);
  if (db) a.part_b = static_cast<float*>(workspace) + (dw ? need / 2 / sizeof(float) : 0);
  NORM_TRY(run<true>(a, P, dtype, vectors(a, es), st));
  if (!dw && !db) return GLA_OK;
  // A shared weight row also sums over the heads: the partial rows [P][H][D] are P * H rows of D.
  const int rows = weight_rows == 1 ? P * H : P, cols = weight_rows * D;
  join_kernel<<<dim3((cols + 31) / 32, 2), 256, 0, st>>>(a.part_w, a.part_b, dw, db, rows, cols);
  return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}
