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

}  // namespace swimba
