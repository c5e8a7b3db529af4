// Rows of bf16, fp16 or fp32 in chunks of eight channels: the row kernels (norms, expert gather and
// combine) hold a chunk as raw words until they need its values, and compute in fp32.
#pragma once

#include "common.cuh"

namespace ss {

// Element types of the row kernels, by their SS_BF16 / SS_F16 / SS_F32 code.
struct Bf16 {
  using Store = uint16_t;
  static constexpr int kWords = 4;   // 32-bit words of eight values
  static __device__ __forceinline__ void unpack(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_bf16(a, b); }
};
struct F16 {
  using Store = uint16_t;
  static constexpr int kWords = 4;
  static __device__ __forceinline__ void unpack(uint32_t w, float& a, float& b) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
    a = v.x;
    b = v.y;
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
struct F32 {
  using Store = float;
  static constexpr int kWords = 8;
};

// Eight channels as raw 32-bit words.
template <class T>
struct Chunk {
  uint32_t w[T::kWords];
};
template <class T>
__device__ __forceinline__ void chunk_zero(Chunk<T>& c) {
#pragma unroll
  for (int i = 0; i < T::kWords; ++i) c.w[i] = 0;
}
// From / to global or shared memory, in 16-byte pieces (p 16-byte aligned).
template <class T>
__device__ __forceinline__ void chunk_load(Chunk<T>& c, const typename T::Store* p) {
#pragma unroll
  for (int i = 0; i < T::kWords / 4; ++i) {
    const uint4 v = reinterpret_cast<const uint4*>(p)[i];
    c.w[4 * i] = v.x;
    c.w[4 * i + 1] = v.y;
    c.w[4 * i + 2] = v.z;
    c.w[4 * i + 3] = v.w;
  }
}
// The same over the read-only path, whose loads the compiler may move ahead of griddep_wait(): only for
// addresses that depend on something loaded plainly behind the wait (an expert's weights), or where the
// work before the wait is known to be done. All else (rows, routes, orders, and the norms' parameters and
// gates, which the launch before may just have written) is loaded plainly, through pointers without
// __restrict__, and so stays behind the wait.
template <class T>
__device__ __forceinline__ void chunk_ldg(Chunk<T>& c, const typename T::Store* p) {
#pragma unroll
  for (int i = 0; i < T::kWords / 4; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
    c.w[4 * i] = v.x;
    c.w[4 * i + 1] = v.y;
    c.w[4 * i + 2] = v.z;
    c.w[4 * i + 3] = v.w;
  }
}
template <class T>
__device__ __forceinline__ void chunk_store(typename T::Store* p, const Chunk<T>& c) {
#pragma unroll
  for (int i = 0; i < T::kWords / 4; ++i)
    reinterpret_cast<uint4*>(p)[i] =
        make_uint4(c.w[4 * i], c.w[4 * i + 1], c.w[4 * i + 2], c.w[4 * i + 3]);
}
template <class T>
__device__ __forceinline__ void chunk_floats(const Chunk<T>& c, float (&f)[8]) {
  if constexpr (T::kWords == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(c.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) T::unpack(c.w[i], f[2 * i], f[2 * i + 1]);
  }
}
// Rounded to the element type (to nearest even), once.
template <class T>
__device__ __forceinline__ void chunk_round(Chunk<T>& c, const float (&f)[8]) {
  if constexpr (T::kWords == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c.w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c.w[i] = T::pack(f[2 * i], f[2 * i + 1]);
  }
}

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Calls f with the type tag of a dtype code (checked by the caller).
template <class F>
auto by_dtype(int dtype, F&& f) {
  switch (dtype) {
    case SS_BF16: return f(Bf16{});
    case SS_F16: return f(F16{});
    default: return f(F32{});
  }
}

}  // namespace ss
