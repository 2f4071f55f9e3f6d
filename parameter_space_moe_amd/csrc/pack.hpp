// Rows of any width and alignment in packs of eight elements: whole packs move
// as 16-byte (bf16) or 2 x 16-byte (fp32) accesses whatever their alignment
// (global memory takes them at element alignment), a row's last, partial
// pack element by element.
#pragma once
#include "swimba_device.hpp"

namespace swimba {

constexpr int kPack = 8;

// Eight raw elements.
template <typename T>
struct alignas(16) Pack {
  T v[kPack];
};

template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) LoosePack {
  uint32_t w[2 * sizeof(T)];
};

template <typename T>
__device__ __forceinline__ Pack<T> load_pack(const T* p, int n) {
  Pack<T> r;
  if (n >= kPack) {
    const LoosePack<T> l = *reinterpret_cast<const LoosePack<T>*>(p);
    __builtin_memcpy(&r, &l, sizeof(r));
  } else {
#pragma unroll
    for (int i = 0; i < kPack; ++i) r.v[i] = i < n ? p[i] : T(0);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void store_pack(T* p, const Pack<T>& r, int n) {
  if (n >= kPack) {
    LoosePack<T> l;
    __builtin_memcpy(&l, &r, sizeof(r));
    *reinterpret_cast<LoosePack<T>*>(p) = l;
  } else {
#pragma unroll
    for (int i = 0; i < kPack; ++i)
      if (i < n) p[i] = r.v[i];
  }
}

// How the rows of a tensor lie for loads of N elements: whole groups, any width,
// or a tensor of fewer than N elements in all.
enum Rows { kLoose = 0, kWhole = 1, kTiny = 2 };

// N elements of a row on their way: one whole load that stays inside the tensor
// whatever the row width, so that a run of them is issued without branches
// between.  Where the tensor ends inside it the load starts `back`
// elements (back_of) earlier; get() moves the elements up again and clears
// those from `left`, the elements left in the row, on.
template <typename T, int N>
struct Loose {
  static constexpr int kWords = N * (int)sizeof(T) / 4;
  typedef uint32_t raw_t __attribute__((ext_vector_type(kWords > 4 ? 4 : kWords)));
  static constexpr int kRaw = kWords > 4 ? kWords / 4 : 1;
  struct __attribute__((packed, aligned(sizeof(T)))) Mem { raw_t r[kRaw]; };
  raw_t r[kRaw];

  __device__ __forceinline__ void whole(const T* p) {
    const Mem m = *reinterpret_cast<const Mem*>(p);
#pragma unroll
    for (int i = 0; i < kRaw; ++i) r[i] = m.r[i];
  }
  // a tensor of fewer than N elements
  __device__ __forceinline__ void few(const T* p, int left) {
    T v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < left ? p[i] : T(0);
    __builtin_memcpy(r, v, sizeof(v));
  }
  __device__ __forceinline__ void get(int back, int left, T* out) const {
    T m[N];
    __builtin_memcpy(m, r, sizeof(m));
    if (__ballot(back != 0)) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        T v = m[i];
#pragma unroll
        for (int j = i + 1; j < N; ++j) v = back == j - i ? m[j] : v;
        out[i] = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = m[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = i < left ? out[i] : T(0);
  }
};

// How far a load of N elements has to be moved back to stay inside a tensor of at
// least N: `left` (above 0) elements of the row and `behind` rows of `width`
// follow.  Rows narrower than N may need it before the last one.
template <int N>
__host__ __device__ __forceinline__ int back_of(int64_t behind, int width, int left) {
  const int rows = behind < N ? (int)behind : N, w = width < N ? width : N;
  const int rest = rows * w + (left < N ? left : N);
  return left > 0 && rest < N ? N - rest : 0;
}

}  // namespace swimba
