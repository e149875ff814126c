// Rotary positions of q and k (C ABI in include/gla.h, gla_rotary).
//
// The pairs (u, v) of the first R channels of a head turn by A_i = p freq_i; the rest is copied.  HBM-bound: each value
// is read and written once.  A thread owns one token and two vectors of V channels, forms the sines and cosines of
// their pairs once and applies them to several heads of q and k, whose vectors it loads two heads at a time.  In the
// half layout the two vectors are the first and the second halves of V pairs; in the interleaved one they are
// neighbours.  Copied vectors go the same way without the rotation.
// The angle: |freq_i| / 2 pi, less its whole turns, becomes a 64-bit fraction once a block (and is negated for a negative
// frequency); its product with the position, whose overflow drops exactly the whole turns, rounded to the upper word, is the
// angle's part of a turn.  (64-bit floating point for every token took most of the kernel's time.)  The word's upper bits,
// rounded, are the quadrant; the rest, at most 1/8 turn, goes into the Taylor sums of sine and cosine, to x^9 and x^8: what is
// left out is below (pi/4)^10 / 10! = 2.5e-8.  So the angle is off by |p freq| 2^-52 radians, the rounding of freq / 2 pi, by
// |p| 2^-65 turns, that of the fraction, and by 2^-33 turns, that of the word.
//
// Measured (bf16, replays of a CUDA graph of 20 calls): q and k [8, 2048, 4, 256] channels last to head-major 23 us
// (5.9 TB/s), half as long again with the angles in 64-bit floating point; q, k [1, 8 + 2, 32768, 128], half of it
// turned, 31 us (5.5 TB/s), two fifths longer when turned and copied vectors were different threads' work; 16 x (8 + 8) x 128,
// one token, 2.4 us.  Half layout with odd R / 2 (vectors of one value, in the copied channels too), 8 x 2048 x 8 x 90 with R = 50:
// bf16 17 us for a floor of 7, fp32 20 us for 14.
#include <limits.h>
#include <math.h>

#include "../../include/gla.h"
#include "pair_math.cuh"
#include "vec.cuh"

namespace {

using gla::bf16;
using gla::F2;
using gla::f2;
using gla::fma2;
using gla::hi;
using gla::lo;
using gla::mul2;
using gla::Pack;
using gla::Two;

struct Args {
  const void *q, *k;
  void *qo, *ko;
  const double* freq;
  const long long* pos;
  long long pos0;
  int pos_rows;
  int Hq, Hk, T, D, R;
  unsigned tokens;  // B * T
  int items;        // a head's pairs of vectors: turned ones, then copied ones
  int turned;
  int heads_a_thread;
  float scale, sign;
  int in_head_major, out_head_major;
  int neighbours;  // V = 1: the halves of a pair are channels 2i and 2i + 1
  gla::Divider by_t, by_items;
};

constexpr int kBatch = 2;  // heads loaded together: four leave registers for half the warps and take half as long again

// Sine and cosine of a 64-bit fraction of a turn.
__device__ __forceinline__ void sincos_turns(unsigned long long turns, float* sn, float* cs) {
  const uint32_t w = (uint32_t)((turns + 0x80000000ull) >> 32), k = (w + 0x20000000u) >> 30;  // the nearest quadrant
  const float x = (float)(int)(w - (k << 30)) * 1.4629180792671596e-9f;      // 2 pi / 2^32
  const float y = x * x;
  float s = fmaf(y, 1.f / 362880.f, -1.f / 5040.f), c = fmaf(y, 1.f / 40320.f, -1.f / 720.f);
  s = fmaf(y, s, 1.f / 120.f), c = fmaf(y, c, 1.f / 24.f);
  s = fmaf(y, s, -1.f / 6.f), c = fmaf(y, c, -0.5f);
  s = fmaf(x * y, s, x), c = fmaf(y, c, 1.f);
  const uint32_t p = __float_as_uint(k & 1 ? c : s), q = __float_as_uint(k & 1 ? s : c);
  *sn = __uint_as_float(p ^ ((k << 30) & 0x80000000u));
  *cs = __uint_as_float(q ^ (((k + 1) << 30) & 0x80000000u));
}

template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(256, 4) rotary_kernel(const Args a) {
  // The pairs' turns a position as fractions of 2^64.
  extern __shared__ unsigned long long fraction[];  // [R / 2]
  for (int f = threadIdx.x; f < a.R / 2; f += 256) {
    double turns = fabs(a.freq[f]) * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= floor(turns);                                    // exact, and below 1
    const unsigned long long n = __double2ull_rn(turns * 18446744073709551616.0);
    fraction[f] = __double_as_longlong(a.freq[f]) < 0 ? 0ull - n : n;
  }
  __syncthreads();
  const int h0 = blockIdx.y * a.heads_a_thread, h1 = min(h0 + a.heads_a_thread, a.Hq + a.Hk);
  const uint32_t idx = blockIdx.x * 256u + threadIdx.x, tok = a.by_items.quot(idx);
  if (tok >= a.tokens) return;
  const int item = (int)(idx - tok * (uint32_t)a.items);
  const uint32_t b = a.by_t.quot(tok), t = tok - b * (uint32_t)a.T;

  // The item's two vectors, and which of them turn.
  int c0, c1;
  bool turn0, turn1;
  if constexpr (INTERLEAVED) {
    c0 = item * 2 * V, c1 = c0 + V;
    turn0 = c0 < a.R, turn1 = c1 < a.R;
  } else {
    turn0 = turn1 = item < a.turned;
    c0 = turn0 ? (a.neighbours ? 2 * item : item * V) : a.R + (item - a.turned) * 2 * V;
    c1 = turn0 ? (a.neighbours ? c0 + 1 : c0 + a.R / 2) : c0 + V;
  }
  const bool has1 = c1 < a.D;

  // Of the V pairs: in the half layout pair i turns values i of both vectors, in the interleaved one the first V / 2
  // pairs are those of the first vector.
  float cs[V], sn[V];
  if (turn0) {
    long long p = a.pos0;
    if (a.pos_rows == 0) p += t;
    else p += a.pos[a.pos_rows == 1 ? (size_t)t : (size_t)tok];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int f = item * V + i;
      if (INTERLEAVED && f >= a.R / 2) break;  // of a second vector that does not turn
      sincos_turns(fraction[f] * (unsigned long long)p, &sn[i], &cs[i]);
      cs[i] *= a.scale;
      sn[i] *= a.scale * a.sign;
    }
  }

#pragma unroll 1
  for (int part = 0; part < 2; ++part) {  // heads of q, then heads of k
    const int H = part ? a.Hk : a.Hq, first = max(h0 - (part ? a.Hq : 0), 0), last = min(h1 - (part ? a.Hq : 0), H);
    if (first >= last) continue;
    const size_t in_stride = a.in_head_major ? (size_t)a.T * a.D : (size_t)a.D;
    const size_t out_stride = a.out_head_major ? (size_t)a.T * a.D : (size_t)a.D;
    const T* in = (const T*)(part ? a.k : a.q) +
                  (a.in_head_major ? ((size_t)b * H * a.T + t) * a.D : (size_t)tok * H * a.D) + first * in_stride;
    T* out = (T*)(part ? a.ko : a.qo) +
             (a.out_head_major ? ((size_t)b * H * a.T + t) * a.D : (size_t)tok * H * a.D) + first * out_stride;
    for (int h = first; h < last; h += kBatch, in += kBatch * in_stride, out += kBatch * out_stride) {
      Pack<T, V> u[kBatch], v[kBatch];
#pragma unroll
      for (int n = 0; n < kBatch; ++n)
        if (h + n < last) {
          u[n].load(in + n * in_stride + c0);
          if (has1) v[n].load(in + n * in_stride + c1);
        }
#pragma unroll
      for (int n = 0; n < kBatch; ++n)
        if (h + n < last) {
          if constexpr (V == 1) {
            if (turn0) {
              const float x = u[n].get(0), y = v[n].get(0);
              u[n].set(0, x * cs[0] - y * sn[0]);
              v[n].set(0, y * cs[0] + x * sn[0]);
            }
          } else {
            typedef typename Two<T>::Raw Raw;
            Raw* ur = reinterpret_cast<Raw*>(u[n].v);
            Raw* vr = reinterpret_cast<Raw*>(v[n].v);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
              const F2 x = Two<T>::wide(ur[i]), y = Two<T>::wide(vr[i]);
              if constexpr (INTERLEAVED) {  // (x, y) c + (-y, x) s
                const F2 xs = f2(-hi(x), lo(x)), ys = f2(-hi(y), lo(y));
                if (turn0) ur[i] = Two<T>::narrow(fma2(xs, f2(sn[i]), mul2(x, f2(cs[i]))));
                if (turn1) vr[i] = Two<T>::narrow(fma2(ys, f2(sn[V / 2 + i]), mul2(y, f2(cs[V / 2 + i]))));
              } else if (turn0) {
                const F2 c = f2(cs[2 * i], cs[2 * i + 1]), s = f2(sn[2 * i], sn[2 * i + 1]);
                ur[i] = Two<T>::narrow(fma2(y, f2(-sn[2 * i], -sn[2 * i + 1]), mul2(x, c)));
                vr[i] = Two<T>::narrow(fma2(x, s, mul2(y, c)));
              }
            }
          }
          u[n].store(out + n * out_stride + c0);
          if (has1) v[n].store(out + n * out_stride + c1);
        }
    }
  }
}

template <typename T, int V>
int launch(Args a, bool interleaved, cudaStream_t st) {
  if (interleaved && V > 1) {
    a.items = (a.D / V + 1) / 2;
  } else {
    a.neighbours = interleaved;
    a.turned = a.R / 2 / V;
    a.items = a.turned + ((a.D - a.R) / V + 1) / 2;
  }
  const long long threads = (long long)a.tokens * a.items;
  if (threads > INT_MAX - 256) return GLA_ERR_UNSUPPORTED;
  a.by_items = gla::Divider((uint32_t)a.items);
  // A thread takes several heads, so that its sines serve all of them, as long as enough threads are left.
  const int heads = a.Hq + a.Hk;
  const long long fill = 148LL * 1024;
  long long groups = (fill + threads - 1) / threads;
  if (groups > heads) groups = heads;
  if (groups > 65535) groups = 65535;
  a.heads_a_thread = (int)((heads + groups - 1) / groups);
  const dim3 grid((unsigned)((threads + 255) / 256), (unsigned)((heads + a.heads_a_thread - 1) / a.heads_a_thread));
  const size_t smem = (size_t)(a.R / 2) * sizeof(unsigned long long);  // 32 KB at most
  if constexpr (V > 1) {
    if (interleaved) rotary_kernel<T, V, true><<<grid, 256, smem, st>>>(a);
    else rotary_kernel<T, V, false><<<grid, 256, smem, st>>>(a);
  } else {
    rotary_kernel<T, V, false><<<grid, 256, smem, st>>>(a);
  }
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
    if (fits) break;
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
