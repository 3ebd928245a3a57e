// Device helpers of the streaming kernels (block norm, act8 checkpoints,
// adapters): eight consecutive values of a row as one or two 16-byte accesses,
// bf16 conversion, and sums over a wave in a fixed order.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace wush {

using f32x4 = float __attribute__((ext_vector_type(4)));
using u32x2 = uint32_t __attribute__((ext_vector_type(2)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));

struct bf16_t {
  uint16_t bits;
};

template <class T>
constexpr bool is_f32 = std::is_same<T, float>::value;

// Eight values as they lie in memory: the loads of several rows are issued
// before any of them is converted.
template <class T>
struct raw8;
template <>
struct raw8<float> {
  f32x4 a, b;
};
template <>
struct raw8<bf16_t> {
  u32x4 a;
};

__device__ __forceinline__ void load8(raw8<float>& r, const float* p) {
  const f32x4* q = reinterpret_cast<const f32x4*>(p);
  r.a = q[0];
  r.b = q[1];
}
__device__ __forceinline__ void load8(raw8<bf16_t>& r, const bf16_t* p) { r.a = *reinterpret_cast<const u32x4*>(p); }

__device__ __forceinline__ void widen8(const raw8<float>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = r.a[i];
    v[4 + i] = r.b[i];
  }
}
__device__ __forceinline__ void widen8(const raw8<bf16_t>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __builtin_bit_cast(float, r.a[i] << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, r.a[i] & 0xffff0000u);
  }
}

// Two fp32 values to bf16, each to the nearest (ties to even); low half first.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  bf16x2 v;
  v[0] = static_cast<__bf16>(lo);
  v[1] = static_cast<__bf16>(hi);
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void store8(float* p, const float* v) {
  f32x4* q = reinterpret_cast<f32x4*>(p);
  q[0] = f32x4{v[0], v[1], v[2], v[3]};
  q[1] = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(bf16_t* p, const float* v) {
  *reinterpret_cast<u32x4*>(p) =
      u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}

// Sum over the wave's 64 lanes, the same value in every lane (butterfly order).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

}  // namespace wush
