// Rotary positions of q and k (C ABI in include/gla.h, gla_rotary).
//
// The pairs (u, v) of the first R channels of a head turn by A_i = p freq_i; the rest is copied.  HBM-bound:
// each value is read and written once.  A thread owns one token and one vector of pairs (V pairs in the
// half layout, V / 2 in the interleaved one), forms their sines and cosines once and applies them to
// several heads of q and k.  The angle is p freq_i / 2 pi in 64 bits, minus the nearest whole number of
// turns; the remaining part of a turn is rounded to 32 bits (|r| <= 1/2, off by at most 2^-26 turns), so
// the angle's error does not grow with the position.
#include <limits.h>
#include <math.h>

#include "../../include/gla.h"
#include "fast_path.cuh"
#include "vec.cuh"

namespace {

using gla::bf16;
using gla::Pack;

struct Args {
  const void *q, *k;
  void *qo, *ko;
  const double* freq;
  const long long* pos;
  long long pos0;
  int pos_rows;
  int Hq, Hk, T, D, R;
  unsigned tokens;  // B * T
  int items;        // vectors a head: turned ones, then copied ones
  int turned;
  int heads_a_thread;
  float scale, sign;
  int in_head_major, out_head_major;
  gla::Divider by_t, by_items;
};

// Offset of (token (b, t), head h) and the distance between heads.
__device__ __forceinline__ size_t row_of(bool head_major, uint32_t b, uint32_t t, int h, int H, int T, int D) {
  return head_major ? (((size_t)b * H + h) * T + t) * D : (((size_t)b * T + t) * H + h) * D;
}

template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(256) rotary_kernel(const Args a) {
  const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
  const uint32_t tok = a.by_items.quot(idx);
  if (tok >= a.tokens) return;
  const int item = (int)(idx - tok * (uint32_t)a.items);
  const uint32_t b = a.by_t.quot(tok), t = tok - b * (uint32_t)a.T;
  const int h0 = blockIdx.y * a.heads_a_thread, h1 = min(h0 + a.heads_a_thread, a.Hq + a.Hk);

  if (item >= a.turned) {  // copied channels
    const int c = a.R + (item - a.turned) * V;
    for (int h = h0; h < h1; ++h) {
      const bool is_q = h < a.Hq;
      const int hh = is_q ? h : h - a.Hq, H = is_q ? a.Hq : a.Hk;
      Pack<T, V> p;
      p.load((const T*)(is_q ? a.q : a.k) + row_of(a.in_head_major, b, t, hh, H, a.T, a.D) + c);
      p.store((T*)(is_q ? a.qo : a.ko) + row_of(a.out_head_major, b, t, hh, H, a.T, a.D) + c);
    }
    return;
  }
  constexpr int PAIRS = INTERLEAVED ? (V > 1 ? V / 2 : 1) : V;
  long long p = a.pos0;
  if (a.pos_rows == 0) p += t;
  else p += a.pos[a.pos_rows == 1 ? (size_t)t : (size_t)tok];
  float cs[PAIRS], sn[PAIRS];
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) {
    double turns = (double)p * (a.freq[item * PAIRS + i] * 0.15915494309189533577);  // 1 / (2 pi)
    turns -= rint(turns);
    sincospif(2.f * (float)turns, &sn[i], &cs[i]);
    cs[i] *= a.scale;
    sn[i] *= a.scale * a.sign;
  }
  for (int h = h0; h < h1; ++h) {
    const bool is_q = h < a.Hq;
    const int hh = is_q ? h : h - a.Hq, H = is_q ? a.Hq : a.Hk;
    const T* in = (const T*)(is_q ? a.q : a.k) + row_of(a.in_head_major, b, t, hh, H, a.T, a.D);
    T* out = (T*)(is_q ? a.qo : a.ko) + row_of(a.out_head_major, b, t, hh, H, a.T, a.D);
    if constexpr (INTERLEAVED) {
      constexpr int W = V > 1 ? V : 2;  // one pair at a time when nothing wider fits
      Pack<T, W / (V > 1 ? 1 : 2)> u, v;
      if constexpr (V > 1) {
        u.load(in + item * V);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          const float x = u.get(2 * i), y = u.get(2 * i + 1);
          u.set(2 * i, x * cs[i] - y * sn[i]);
          u.set(2 * i + 1, y * cs[i] + x * sn[i]);
        }
        u.store(out + item * V);
      } else {
        u.load(in + item * 2);
        v.load(in + item * 2 + 1);
        const float x = u.get(0), y = v.get(0);
        u.set(0, x * cs[0] - y * sn[0]);
        v.set(0, y * cs[0] + x * sn[0]);
        u.store(out + item * 2);
        v.store(out + item * 2 + 1);
      }
    } else {
      Pack<T, V> u, v;
      u.load(in + item * V);
      v.load(in + a.R / 2 + item * V);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float x = u.get(i), y = v.get(i);
        u.set(i, x * cs[i] - y * sn[i]);
        v.set(i, y * cs[i] + x * sn[i]);
      }
      u.store(out + item * V);
      v.store(out + a.R / 2 + item * V);
    }
  }
}

template <typename T, int V>
int launch(Args a, bool interleaved, cudaStream_t st) {
  a.turned = interleaved ? (V > 1 ? a.R / V : a.R / 2) : a.R / 2 / V;
  a.items = a.turned + (a.D - a.R) / V;
  const long long threads = (long long)a.tokens * a.items;
  if (threads > INT_MAX - 256) return GLA_ERR_UNSUPPORTED;
  a.by_items = gla::Divider((uint32_t)a.items);
  // A thread takes several heads, so that its sines serve all of them, as long as enough threads are left.
  const int heads = a.Hq + a.Hk;
  const long long fill = (long long)gla::fast::sm_count() * 2048;
  long long per = threads * heads / fill;
  per = per < 1 ? 1 : per > heads ? heads : per;
  const long long most_y = 65535;
  if ((heads + per - 1) / per > most_y) per = (heads + most_y - 1) / most_y;
  a.heads_a_thread = (int)per;
  const dim3 grid((unsigned)((threads + 255) / 256), (unsigned)((heads + per - 1) / per));
  if (interleaved) rotary_kernel<T, V, true><<<grid, 256, 0, st>>>(a);
  else rotary_kernel<T, V, false><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

#define ROT_TRY(expr)            \
  do {                           \
    const int _s = (expr);       \
    if (_s != GLA_OK) return _s; \
  } while (0)

int check_ptr(const void* p, size_t es, bool required) {
  if (!p) return required ? GLA_ERR_INVALID_ARG : GLA_OK;
  return gla::aligned_to(p, es) ? GLA_OK : GLA_ERR_INVALID_ARG;
}

}  // namespace

extern "C" int gla_rotary(const void* q, const void* k, void* qo, void* ko, const double* freq, const long long* pos,
                          long long pos0, int pos_rows, int B, int Hq, int Hk, int T, int D, int R, float scale,
                          int interleaved, int inverse, int in_layout, int out_layout, int dtype, void* stream) {
  if (B <= 0 || Hq <= 0 || Hk < 0 || T < 0 || D <= 0 || R <= 0) return GLA_ERR_INVALID_ARG;
  if (R % 2 != 0 || R > D || !isfinite(scale)) return GLA_ERR_INVALID_ARG;
  if (pos_rows != 0 && pos_rows != 1 && pos_rows != B) return GLA_ERR_INVALID_ARG;
  if (dtype != GLA_DTYPE_F32 && dtype != GLA_DTYPE_BF16) return GLA_ERR_UNSUPPORTED;
  for (int l : {in_layout, out_layout})
    if (l != GLA_LAYOUT_BHTD && l != GLA_LAYOUT_BTHD) return GLA_ERR_UNSUPPORTED;
  if (D > 8192 || (long long)Hq + Hk > INT_MAX || (long long)B * (T > 0 ? T : 1) > INT_MAX) return GLA_ERR_UNSUPPORTED;
  if (T == 0) return GLA_OK;
  const size_t es = dtype == GLA_DTYPE_BF16 ? 2 : 4;
  ROT_TRY(check_ptr(q, es, true));
  ROT_TRY(check_ptr(qo, es, true));
  ROT_TRY(check_ptr(k, es, Hk > 0));
  ROT_TRY(check_ptr(ko, es, Hk > 0));
  ROT_TRY(check_ptr(freq, 8, true));
  ROT_TRY(check_ptr(pos, 8, pos_rows > 0));
  if (in_layout != out_layout && (q == qo || (Hk > 0 && k == ko))) return GLA_ERR_INVALID_ARG;
  Args a = {};
  a.q = q, a.k = Hk > 0 ? k : nullptr, a.qo = qo, a.ko = Hk > 0 ? ko : nullptr;
  a.freq = freq, a.pos = pos, a.pos0 = pos0, a.pos_rows = pos_rows;
  a.Hq = Hq, a.Hk = Hk, a.T = T, a.D = D, a.R = R;
  a.tokens = (unsigned)((long long)B * T);
  a.scale = scale, a.sign = inverse ? -1.f : 1.f;
  a.in_head_major = in_layout == GLA_LAYOUT_BHTD, a.out_head_major = out_layout == GLA_LAYOUT_BHTD;
  a.by_t = gla::Divider((uint32_t)T);
  // The widest vector (at most 16 bytes) that divides the turned and the copied channels and every
  // address: one value at a time when nothing else does.
  int V = (int)(16 / es);
  const int piece = interleaved ? R : R / 2;
  while (V > 1) {
    bool fits = piece % V == 0 && D % V == 0;
    for (const void* p : {q, (const void*)qo, a.k, (const void*)a.ko}) fits = fits && gla::aligned_to(p, V * es);
    if (fits && (!interleaved ? true : V >= 2)) break;
    V /= 2;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (es == 2) {
    if (V == 8) return launch<bf16, 8>(a, interleaved != 0, st);
    if (V == 4) return launch<bf16, 4>(a, interleaved != 0, st);
    if (V == 2) return launch<bf16, 2>(a, interleaved != 0, st);
    return launch<bf16, 1>(a, interleaved != 0, st);
  }
  if (V == 4) return launch<float, 4>(a, interleaved != 0, st);
  if (V == 2) return launch<float, 2>(a, interleaved != 0, st);
  return launch<float, 1>(a, interleaved != 0, st);
}
