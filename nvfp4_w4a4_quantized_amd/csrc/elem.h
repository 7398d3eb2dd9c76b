// elem.h -- the element types of the operators on unquantized tensors
// (dtype codes of the C ABI: 0 binary32, 1 bf16, 2 fp16) and 16-byte pieces
// of rows in those types.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4_device.h"

namespace nvfp4 {

template <int DT>
struct Elem;
template <>
struct Elem<0> {
  typedef float type;
  static __device__ __forceinline__ float to_float(float v) { return v; }
  static __device__ __forceinline__ float from_float(float v) { return v; }
};
template <>
struct Elem<1> {
  typedef uint16_t type;   // bf16 bits
  static __device__ __forceinline__ float to_float(uint16_t v) {
    return __uint_as_float((uint32_t)v << 16);
  }
  // round to nearest even; the compiler's conversion keeps NaN a NaN
  static __device__ __forceinline__ uint16_t from_float(float v) {
    const __bf16 b = (__bf16)v;
    uint16_t u;
    __builtin_memcpy(&u, &b, 2);
    return u;
  }
};
template <>
struct Elem<2> {
  typedef _Float16 type;
  static __device__ __forceinline__ float to_float(_Float16 v) { return (float)v; }
  static __device__ __forceinline__ _Float16 from_float(float v) { return (_Float16)v; }
};

// 16 bytes of a row as binary32 values.  Rows may start at any element (odd
// widths and strides), so the copy assumes the element's alignment only.
template <int DT>
struct Piece {
  typedef typename Elem<DT>::type T;
  static constexpr int kN = 16 / (int)sizeof(T);
  T v[kN];
  typedef u32x4_t any16_t __attribute__((aligned(2)));   // 16 bytes at an element's alignment
  __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(v, p, 16); }
  // read once, and written for a later kernel: past the caches' replacement order
  __device__ __forceinline__ void load_once(const T* p) {
    const u32x4_t w = __builtin_nontemporal_load(reinterpret_cast<const any16_t*>(p));
    __builtin_memcpy(v, &w, 16);
  }
  __device__ __forceinline__ void store(T* p) const {
    u32x4_t w;
    __builtin_memcpy(&w, v, 16);
    __builtin_nontemporal_store(w, reinterpret_cast<any16_t*>(p));
  }
  // the first n elements (n < kN): a row's last, partial piece
  __device__ __forceinline__ void load_part(const T* p, int n) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = i < n ? p[i] : (T)0;
  }
  __device__ __forceinline__ void store_part(T* p, int n) const {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i < n) p[i] = v[i];
  }
  __device__ __forceinline__ float get(int i) const { return Elem<DT>::to_float(v[i]); }
  __device__ __forceinline__ void set(int i, float f) { v[i] = Elem<DT>::from_float(f); }
};

}  // namespace nvfp4
