// Row access shared by the token and adapter kernels: vector loads and stores of bf16 or float32
// elements at any element alignment, and the rounding to bf16.
#pragma once

#include "e4b_device.h"

namespace e4b {

// Rows of a matrix with an odd number of columns start at any multiple of the element size; the
// hardware takes 16-byte global accesses at any address, the types say so to the compiler.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// float32 -> bf16 bits, round to nearest even; NaN stays NaN (one conversion instruction).
__device__ __forceinline__ uint16_t bf16_rne(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ uint32_t bf16_rne2(float lo, float hi) {
  return uint32_t(bf16_rne(lo)) | (uint32_t(bf16_rne(hi)) << 16);
}

// Element types of rows: 0 bf16, 1 float32 (the values of e4b_dtype).
template <int DT> struct RowElem;
template <> struct RowElem<0> { typedef uint16_t type; };
template <> struct RowElem<1> { typedef float type; };
template <int DT> using row_elem = typename RowElem<DT>::type;

__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = bf16_rne(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// V consecutive elements as float32 (4 or 8 float32, 8 bf16; 4 or 8 of either written).  Rows are
// written past the caches: kept there they slowed the kernels that followed (7862 slots of 3000
// float32 back to tokens and again: 36 us a call kept, 27 past; measured without a call that reads
// them in between).
template <int V>
__device__ __forceinline__ void load_vec(const uint16_t* p, float (&v)[V]) {
  static_assert(V == 8, "");
  const u32x4 q = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(q[i] << 16);
    v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
  }
}
template <int V>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const f32x4 q = *reinterpret_cast<const f32x4_any*>(p + 4 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * i + j] = q[j];
  }
}
// The same past the caches, for what is read once.
template <int V>
__device__ __forceinline__ void load_once(const uint16_t* p, float (&v)[V]) {
  static_assert(V == 8, "");
  const u32x4 q = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(q[i] << 16);
    v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
  }
}
template <int V>
__device__ __forceinline__ void load_once(const float* p, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const f32x4 q = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(p + 4 * i));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * i + j] = q[j];
  }
}
template <int V>
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&v)[V]) {
  if constexpr (V == 8) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = bf16_rne2(v[2 * i], v[2 * i + 1]);
    __builtin_nontemporal_store(q, reinterpret_cast<u32x4_any*>(p));
  } else {
    u32x2 q;
    q[0] = bf16_rne2(v[0], v[1]);
    q[1] = bf16_rne2(v[2], v[3]);
    __builtin_nontemporal_store(q, reinterpret_cast<u32x2_any*>(p));
  }
}
template <int V>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i)
    __builtin_nontemporal_store(f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]}, reinterpret_cast<f32x4_any*>(p + 4 * i));
}

}  // namespace e4b
