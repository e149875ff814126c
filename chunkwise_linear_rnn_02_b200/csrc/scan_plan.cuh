// How the elementwise scan cuts its work: which slab of channels a block has, how many blocks share one, and so which of the
// kernels in scan.cu runs.  Host code only, without CUDA, so that it can be asked without a GPU.
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace gla {
namespace scan {

constexpr int kKeep = 64;  // tokens between the kept states

// How a block's tiles come into shared memory (rows of 2 LPR values, one a token):
//   kTma       one copy of the whole tile by TMA; rows and tensors start on 16 bytes
//   kByThread  every thread copies what it will read itself, two values or one at a time, asynchronously where they
//              have 4 bytes at least
// B=8, T=2048, C=1008 bf16 forward: 20 us by TMA; by thread, C=1002 31 us, C=1001, one value at a time, 44 us.
enum Load { kTma = 0, kByThread = 1 };

// How a variant with slabs of 2 LPR channels is cut: blocks of W warps, MINB of them an SM, R tokens a thread, STAGES
// tiles in shared memory, up to MAXK blocks a cluster.
// Blocks of 4 warps: 8 warps with the same bytes in flight pay for joining twice the warps (B=1, T=32768, C=1024 bf16
// forward a quarter longer).  Forward: 16 tokens a thread at bf16, since 8 make twice the joins an element (B=8, T=2048,
// C=2048 a fifth longer); one tile of g is 8 KB, so three stages of three blocks fit the 227 KB.  fp32 has 8 tokens for
// the same 8 KB; on slabs of 64 channels it has 16 and two stages of 16 KB, which serves many channels by TMA (B=8,
// T=2048, C=2048 65 us, 73 us on slabs of 32) and is too little in flight where the threads copy (C=1002 60 and 39 us).
// Backward: the third array and the recomputed states take the registers of the other 8 tokens (with 16 the complement
// spills and takes two and a half times as long), and a tile has to start at a kept state, so slabs of 64 channels
// would need 8 warps: slabs of 32 are its widest (B=8, T=2048, C=2048 bf16 62 against 65 us).
template <bool BF16, int LPR, bool BWD>
struct Shape {
  static_assert(!BWD || LPR < 32, "a tile of the backward starts at a kept state");
  static constexpr int W = 4, MINB = BWD && BF16 ? 4 : 3;
  static constexpr int R = BWD || (!BF16 && LPR < 32) ? 8 : 16;
  static constexpr int STAGES = !BF16 && LPR == 32 ? 2 : 3;
  static constexpr int MAXK = LPR == 8 ? 16 : LPR == 16 ? 8 : 6;
  // tokens and channels of a tile; bytes of a stage, and of the values that the blocks of a cluster exchange
  static constexpr int TILE = W * (32 / LPR) * R, CW = 2 * LPR, STAGE = (BWD ? 3 : 2) * TILE * CW * (BF16 ? 2 : 4);
  static constexpr int EXCHANGE = 2 * MAXK * LPR * 16 + 16;
};

// How many blocks share a slab, and what that costs.  A step of a block takes a fixed time, more the more blocks
// exchange, and the work of a tile times the blocks of the SM, which differs with the width of the slab (narrow rows
// also join across the warp):
//     cost = steps (fixed + block K + work (R / 16) blocks_an_sm)
// fitted to 53 shapes with every K and slab (both types, 256 to 65,536 tokens, 64 to 6,400 channels in all, rows on
// 16 bytes, even and odd): what it chooses takes 1.02 times as long as the best choice within the limits below on average, 1.34
// times at worst, and 1.05 times as long as the best of all on average, 1.6 times at worst.
// The complement's backward at bf16 takes the narrow slab at many channels (B=8, T=2048, C=2048: 76 us under the profiler, 85 us
// on the wide one): it issues 51 instructions a value instead of 48, but has 6.9 blocks an SM instead of 3.5 and waits a
// quarter as long for loads (long scoreboard 0.3 cycles an issue, 1.3).  Neither spills there; copied by the threads both do,
// 32 to 40 bytes a thread.
// K is 1, 2, 3, 4, 6, 8 or 16, all blocks running at once (in between, clusters leave places free: B=1, T=32768, C=1024
// forward 65 us with 13, 47 us with 8), and clusters of six and more take seven eighths of the places at most, since how
// they fill the GPU's groups of SMs differs from one GPU to the next (2 x 2 x 3000 x 200 bf16 backward: 16 us with 52
// clusters of 8, 13 us with 52 of 6; fp32 3 x 2 x 1531 x 333 forward with 66 of 6: 13 us on one GPU, 18 us on another).
// Clusters of 16 serve where they leave an SM no more than a block (on a GPU that took more of them, 2 x 20000 x 96 bf16 backward
// had 22 us with 192 blocks, 31 us with the clusters of 8 that this rule leaves).
struct Cost {
  double fixed, block, work64, work32, work16;
};
template <bool BF16, int LOAD, bool COMP, bool BWD>
constexpr Cost cost() {
  if (LOAD == kTma) {
    if (!BWD) return BF16 ? Cost{0.3, 0.15, 0.6, 0.72, 1.1} : Cost{0.6, 0.08, 0.6, 0.6, 0.9};
    if (!BF16) return {0.3, 0.11, 0., 0.7, 0.9};
    return COMP ? Cost{0.6, 0.08, 0., 0.7, 0.69} : Cost{0.6, 0.05, 0., 0.5, 0.75};
  }
  if (BF16) return {0.9, 0.08, 0.6, 0.75, BWD ? 1.125 : 1.3};
  return BWD ? Cost{0.4, 0.08, 0., 0.9, 1.6} : Cost{0.5, 0.08, 0., 0.9, 1.5};
}
struct Plan {
  long long cols = 0;
  int lpr = 0, slabs = 0, tiles = 0, K = 0, steps = 0;
  double cost = 0.;
};
template <bool BF16, int LPR, int LOAD, bool COMP, bool BWD>
Plan plan(long long BH, int T, int D) {
  typedef Shape<BF16, LPR, BWD> S;
  constexpr int SHARED = S::STAGES * S::STAGE + S::W * LPR * (BWD ? 48 : 32) + S::EXCHANGE + 1088;
  constexpr int PLACES = 148 * (S::MINB < 233472 / SHARED ? S::MINB : 233472 / SHARED);  // 228 KB an SM
  constexpr Cost C = cost<BF16, LOAD, COMP, BWD>();
  constexpr double work = (LPR == 32 ? C.work64 : LPR == 16 ? C.work32 : C.work16) * S::R / 16;
  Plan best;
  best.lpr = LPR;
  best.slabs = (D - 1) / S::CW + 1;  // D goes up to 2^31 - 1
  best.tiles = (int)(((long long)T + S::TILE - 1) / S::TILE);
  best.cols = BH * best.slabs;
  for (int K : {1, 2, 3, 4, 6, 8, 16}) {
    const long long n = best.cols * K;
    if (K > 1 && (K > S::MAXK || K > best.tiles || n > (K < 6 ? PLACES : K < 16 ? PLACES / 8 * 7 : 148))) break;
    const int steps = (best.tiles + K - 1) / K;
    const double c = (double)steps * (C.fixed + (K > 1 ? C.block * K : 0.) + work * (double)((n + 147) / 148));
    if (K == 1 || c < best.cost) best.K = K, best.steps = steps, best.cost = c;
  }
  return best;
}

// Slabs of 64 (forward, but not fp32 copied by the threads), 32 or 16 channels, whichever costs least.
template <bool BF16, int LOAD, bool COMP, bool BWD>
Plan choose(long long BH, int T, int D) {
  const Plan mid = plan<BF16, 16, LOAD, COMP, BWD>(BH, T, D), narrow = plan<BF16, 8, LOAD, COMP, BWD>(BH, T, D);
  if constexpr (!BWD && (BF16 || LOAD == kTma)) {
    const Plan wide = plan<BF16, 32, LOAD, COMP, BWD>(BH, T, D);
    if (wide.cost <= mid.cost && wide.cost <= narrow.cost) return wide;
  }
  return mid.cost <= narrow.cost ? mid : narrow;
}

// The way a call's tiles are loaded.  `addresses`: all of its tensors' addresses, or'ed together.  TMA counts tokens and heads in
// 32 bits and strides up to 2^40 bytes.
inline bool fits(uintptr_t addresses, int D, int value_bytes, int bytes) {
  return (long long)D * value_bytes % bytes == 0 && addresses % (uintptr_t)bytes == 0;
}
inline bool by_tma(uintptr_t addresses, int T, int D, int value_bytes) {
  return fits(addresses, D, value_bytes, 16) && T < (1 << 30) && (double)D * value_bytes * T < 1099511627776.0;
}

}  // namespace scan
}  // namespace gla
