// Vectors of N neighbouring values kept packed as they lie in memory (2 to 16 bytes, one access),
// and an exact division by a launch constant.  Used by the elementwise operators around the
// recurrences.
#pragma once

#include "common.cuh"

namespace gla {

template <int BYTES>
struct Words;
template <>
struct Words<2> {
  typedef unsigned short type;
};
template <>
struct Words<4> {
  typedef unsigned int type;
};
template <>
struct Words<8> {
  typedef uint2 type;
};
template <>
struct Words<16> {
  typedef uint4 type;
};

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  typedef typename Words<sizeof(T) * N>::type Raw;
  T v[N];

  __device__ __forceinline__ void load(const T* p) { *reinterpret_cast<Raw*>(v) = *reinterpret_cast<const Raw*>(p); }
  // For memory that nothing writes during the launch.
  __device__ __forceinline__ void load_const(const T* p) {
    *reinterpret_cast<Raw*>(v) = __ldg(reinterpret_cast<const Raw*>(p));
  }
  __device__ __forceinline__ void store(T* p) const {
    *reinterpret_cast<Raw*>(p) = *reinterpret_cast<const Raw*>(v);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) stf(&v[i], 0.f);
  }
  __device__ __forceinline__ float get(int i) const { return ldf(&v[i]); }
  // fp32 -> T rounds to nearest even, once, here.
  __device__ __forceinline__ void set(int i, float x) { stf(&v[i], x); }
};

// n / d for 0 <= n < 2^31 and a fixed d >= 1 by one multiplication: with l = ceil(log2 d) and
// m = ceil(2^(31 + l) / d), n / d = floor(n m / 2^(31 + l)), since m d - 2^(31 + l) < d <= 2^l keeps the
// excess n (m d - 2^(31 + l)) / (d 2^(31 + l)) below 1 / d.
struct Divider {
  uint32_t d, m, shift;
  Divider() : d(1), m(0x80000000u), shift(0) {}
  explicit Divider(uint32_t div) : d(div) {
    uint32_t l = 0;
    while ((1ull << l) < div) ++l;
    m = (uint32_t)(((1ull << (31 + l)) + div - 1) / div);
    shift = l;
  }
  __host__ __device__ __forceinline__ uint32_t quot(uint32_t n) const {
    return (uint32_t)(((uint64_t)n * m) >> 31 >> shift);
  }
};

inline bool aligned_to(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace gla
