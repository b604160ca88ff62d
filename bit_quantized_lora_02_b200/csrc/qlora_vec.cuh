// qlora_vec.cuh -- 16-byte access to rows of bf16 or fp32 values, and the warp
// reductions that the row kernels (layer norm, token log probabilities) share.
//
// Windows: a row that starts `sh` elements past a 16-byte boundary is covered
// by aligned 16-byte windows; window c holds columns c * N - sh + i, i < N.
// Only a row's first and last window can reach outside [0, cols).  They are written
// element by element, so nothing outside the row ever is.  Loads into registers
// (load_raw) stay in the row as well; those into shared memory (cp.async) stop at
// its end, but take a first window from its 16-byte boundary on: up to 14 bytes
// ahead of the row, in the same aligned 16 bytes as its first element and so in
// mapped memory, whoever owns them.  Their values are dropped before any use.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "qlora_device.cuh"

namespace qlora {

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// Two fp32 values in one 64-bit register (packed f32x2 arithmetic of sm_100, each
// half rounded to nearest even).  ptxas 12.9 contracts f2_add(f2_mul(a, b), c) to
// one f2_fma, its .rn notwithstanding (measured): where both roundings count,
// one of the two has to be the scalar __fmul_rn or __fadd_rn.
using f2 = uint64_t;
__device__ __forceinline__ f2 f2_make(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f2 f2_dup(float x) { return f2_make(x, x); }
__device__ __forceinline__ void f2_get(f2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ float f2_sum(f2 v) {
  float a, b;
  f2_get(v, a, b);
  return a + b;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A 16-byte vector as pairs of fp32.
__device__ __forceinline__ void unpack2(const uint4& v, f2 (&f)[4], __nv_bfloat16) {
  f[0] = f2_make(bf16_lo(v.x), bf16_hi(v.x));
  f[1] = f2_make(bf16_lo(v.y), bf16_hi(v.y));
  f[2] = f2_make(bf16_lo(v.z), bf16_hi(v.z));
  f[3] = f2_make(bf16_lo(v.w), bf16_hi(v.w));
}
__device__ __forceinline__ void unpack2(const uint4& v, f2 (&f)[2], float) {
  f[0] = f2_make(__uint_as_float(v.x), __uint_as_float(v.y));
  f[1] = f2_make(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ uint32_t pack2_bf16(f2 v) {
  float lo, hi;
  f2_get(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint4 pack2(const f2 (&f)[4], __nv_bfloat16) {
  return make_uint4(pack2_bf16(f[0]), pack2_bf16(f[1]), pack2_bf16(f[2]), pack2_bf16(f[3]));
}
__device__ __forceinline__ uint4 pack2(const f2 (&f)[2], float) {
  return make_uint4(static_cast<uint32_t>(f[0]), static_cast<uint32_t>(f[0] >> 32), static_cast<uint32_t>(f[1]),
                    static_cast<uint32_t>(f[1] >> 32));
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Columns col .. col + N - 1 of a row, packed (col may be negative or reach past
// cols: those elements become zero).  `p` is the row's first element; p + col
// is 16-byte aligned.  WHOLE: a window lies in the row or past it, never across
// an end.  The element loads clamp their column, so that their addresses lie in
// the row whether or not the compiler keeps them behind the comparison.
template <typename T, bool WHOLE>
__device__ __forceinline__ uint4 load_raw(const T* p, int col, int cols) {
  constexpr int N = Vec<T>::N;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (WHOLE ? col < cols : (col >= 0 && col + N <= cols)) {
    v = *reinterpret_cast<const uint4*>(p + col);
  } else if (!WHOLE && col < cols && col > -N) {
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = to_f32(p[min(max(col + i, 0), cols - 1)]);
      f[i] = (col + i >= 0 && col + i < cols) ? x : 0.0f;
    }
    v = Vec<T>::pack(f);
  }
  return v;
}

template <typename T, bool WHOLE>
__device__ __forceinline__ void store_raw(T* p, int col, int cols, const uint4& v) {
  constexpr int N = Vec<T>::N;
  if (WHOLE ? col < cols : (col >= 0 && col + N <= cols)) {
    *reinterpret_cast<uint4*>(p + col) = v;
  } else if (!WHOLE) {
    float f[N];
    Vec<T>::unpack(v, f);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (col + i >= 0 && col + i < cols) p[col + i] = from_f32<T>(f[i]);
  }
}

// 16 bytes from global to shared memory without passing through registers; only
// the first `bytes` are read, the rest of the 16 become zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int BYTES>   // 4, 8 or 16
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most `left` of this thread's latest groups are in flight (0..3).
__device__ __forceinline__ void cp_async_wait(int left) {
  if (left >= 3)
    asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (left == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (left == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
template <typename V>
__device__ __forceinline__ V lds(uint32_t a);
template <>
__device__ __forceinline__ uint4 lds<uint4>(uint32_t a) { return lds128(a); }
template <>
__device__ __forceinline__ uint2 lds<uint2>(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
template <>
__device__ __forceinline__ uint32_t lds<uint32_t>(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace qlora
