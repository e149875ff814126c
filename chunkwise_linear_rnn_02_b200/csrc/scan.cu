// Elementwise gated linear recurrence (C ABI in include/gla.h, gla_scan_*):
//
//     h_t = a_t h_{t-1} + b_t,   a_t = exp g_t,   b_t = x_t  or  (1 - a_t) x_t
//
// First form: one thread a channel walks the tokens.  The backward pass recomputes the states of a
// block of 64 tokens from the state kept in front of it, then walks the block in reverse.
#include <limits.h>
#include <math.h>

#include "../../include/gla.h"
#include "vec.cuh"

namespace {

using gla::bf16;
using gla::ldf;
using gla::stf;

constexpr int kKeep = 64;  // tokens between the kept states

// a = exp g and, when asked for, 1 - a.  Near g = 0 both come from exp g - 1 = g (1 + g/2 (1 + g/3 (...))),
// so that neither the 1 - a of a slow gate nor a long product of a's loses its leading digits; the
// series ends five terms in, where |g| < 1/8 leaves a relative error below g^5/720 < 2^-24.
__device__ __forceinline__ float decay(float g, float* rest) {
  float p = fmaf(g, 1.f / 120.f, 1.f / 24.f);
  p = fmaf(g, p, 1.f / 6.f);
  p = fmaf(g, p, 0.5f);
  p = fmaf(g, p, 1.f) * g;
  const float e = expf(g);
  const bool slow = fabsf(g) < 0.125f;
  *rest = slow ? -p : 1.f - e;
  return slow ? 1.f + p : e;
}

template <typename T, bool COMP>
__global__ void scan_fwd_kernel(const T* __restrict__ g, const T* __restrict__ x, const float* __restrict__ h0,
                                T* __restrict__ o, float* __restrict__ hT, float* __restrict__ hc, long long BH,
                                int T_, int D) {
  const long long c = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= BH * D) return;
  const long long bh = c / D;
  const int d = (int)(c - bh * D);
  const int NC = (T_ + kKeep - 1) / kKeep;
  float h = h0 ? h0[c] : 0.f;
  size_t at = (size_t)bh * T_ * D + d;
  for (int t = 0; t < T_; ++t, at += D) {
    if (hc && t % kKeep == 0) hc[((size_t)bh * NC + t / kKeep) * D + d] = h;
    float rest;
    const float a = decay(ldf(g + at), &rest), in = ldf(x + at);
    h = fmaf(a, h, COMP ? rest * in : in);
    if (o) stf(o + at, h);
  }
  if (hT) hT[c] = h;
}

template <typename T, bool COMP>
__global__ void scan_bwd_kernel(const T* __restrict__ g, const T* __restrict__ x, const float* __restrict__ hc,
                                const T* __restrict__ dO, const float* __restrict__ dhT, T* __restrict__ dg,
                                T* __restrict__ dx, float* __restrict__ dh0, long long BH, int T_, int D) {
  const long long c = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= BH * D) return;
  const long long bh = c / D;
  const int d = (int)(c - bh * D);
  const int NC = (T_ + kKeep - 1) / kKeep;
  float back = dhT ? dhT[c] : 0.f;  // a_{t+1} d_{t+1}
  float h[kKeep];                   // states before the block's tokens
  for (int n = NC - 1; n >= 0; --n) {
    const int t0 = n * kKeep, len = min(kKeep, T_ - t0);
    const size_t base = ((size_t)bh * T_ + t0) * D + d;
    float rest;
    h[0] = hc[((size_t)bh * NC + n) * D + d];
    for (int i = 0; i + 1 < len; ++i) {
      const float a = decay(ldf(g + base + (size_t)i * D), &rest), in = ldf(x + base + (size_t)i * D);
      h[i + 1] = fmaf(a, h[i], COMP ? rest * in : in);
    }
    for (int i = len - 1; i >= 0; --i) {
      const size_t at = base + (size_t)i * D;
      const float a = decay(ldf(g + at), &rest);
      const float dd = ldf(dO + at) + back;
      back = a * dd;
      stf(dx + at, COMP ? rest * dd : dd);
      stf(dg + at, back * (COMP ? h[i] - ldf(x + at) : h[i]));
    }
  }
  if (dh0) dh0[c] = back;
}

template <typename T, bool COMP>
__global__ void scan_step_kernel(const T* __restrict__ g, const T* __restrict__ x, float* __restrict__ S,
                                 T* __restrict__ o, long long n) {
  const long long c = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= n) return;
  float rest;
  const float a = decay(ldf(g + c), &rest), in = ldf(x + c);
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
unsigned blocks(long long n) { return (unsigned)((n + 127) / 128); }

int fwd(const void* g, const void* x, const float* h0, void* o, float* hT, float* hc, int B, int H, int T, int D,
        int input, int dtype, cudaStream_t st) {
  const long long BH = (long long)B * H;
  const unsigned grid = blocks(BH * D);
#define SCAN_FWD(TYPE, COMP) \
  scan_fwd_kernel<TYPE, COMP><<<grid, 128, 0, st>>>((const TYPE*)g, (const TYPE*)x, h0, (TYPE*)o, hT, hc, BH, T, D)
  const bool comp = input == GLA_SCAN_COMPLEMENT;
  if (dtype == GLA_DTYPE_BF16) {
    if (comp) SCAN_FWD(bf16, true);
    else SCAN_FWD(bf16, false);
  } else {
    if (comp) SCAN_FWD(float, true);
    else SCAN_FWD(float, false);
  }
#undef SCAN_FWD
  return launched();
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
  const long long BH = (long long)B * H;
  const unsigned grid = blocks(BH * D);
#define SCAN_BWD(TYPE, COMP)                                                                                     \
  scan_bwd_kernel<TYPE, COMP><<<grid, 128, 0, st>>>((const TYPE*)g, (const TYPE*)x, hc, (const TYPE*)dO, dhT, \
                                                    (TYPE*)dg, (TYPE*)dx, dh0, BH, T, D)
  const bool comp = input == GLA_SCAN_COMPLEMENT;
  if (dtype == GLA_DTYPE_BF16) {
    if (comp) SCAN_BWD(bf16, true);
    else SCAN_BWD(bf16, false);
  } else {
    if (comp) SCAN_BWD(float, true);
    else SCAN_BWD(float, false);
  }
#undef SCAN_BWD
  return launched();
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
  const unsigned grid = blocks(n);
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
