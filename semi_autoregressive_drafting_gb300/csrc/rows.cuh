// rows.cuh -- rows of fp32 or bf16 logits in 16-byte pieces, shared by the kernels that stream them.
#pragma once

#include <string.h>

#include "common.cuh"

namespace dspark {

__device__ __forceinline__ float ex2p(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values in one 64-bit register pair: one instruction per pair on sm_100 and later.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 un2(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// What a type needs: E entries per 16 bytes, the 32-bit word of fill entries (-inf), the largest
// entry of 16 bytes, and the number of entries above a threshold.
template <typename T>
struct Lg;
template <>
struct Lg<float> {
  static constexpr int E = 4;
  static constexpr uint32_t kFill = 0xFF800000u;
  struct Thr {
    float x;
  };
  struct Cnt {
    int n;
  };
  __device__ __forceinline__ static float max16(float m, const uint4& q) {
    return fmaxf(m, fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)),
                          fmaxf(__uint_as_float(q.z), __uint_as_float(q.w))));
  }
  __device__ __forceinline__ static F2 pair(const uint4& q, int i) {
    return i == 0 ? f2(__uint_as_float(q.x), __uint_as_float(q.y)) : f2(__uint_as_float(q.z), __uint_as_float(q.w));
  }
  __device__ __forceinline__ static Thr thr(float x) { return Thr{x}; }
  __device__ __forceinline__ static void above(Cnt& c, const uint4& q, const Thr& t) {
    c.n += (__uint_as_float(q.x) > t.x ? 1 : 0) + (__uint_as_float(q.y) > t.x ? 1 : 0) +
           (__uint_as_float(q.z) > t.x ? 1 : 0) + (__uint_as_float(q.w) > t.x ? 1 : 0);
  }
  __device__ __forceinline__ static Cnt zero() { return Cnt{0}; }
  __device__ __forceinline__ static int total(const Cnt& c) { return c.n; }
};
template <>
struct Lg<__nv_bfloat16> {
  static constexpr int E = 8;
  static constexpr uint32_t kFill = 0xFF80FF80u;
  struct Thr {
    __nv_bfloat162 x;
  };
  struct Cnt {
    __nv_bfloat162 n;  // counts of up to 2 x 256 entries are exact
  };
  __device__ __forceinline__ static __nv_bfloat162 b2(uint32_t w) {
    __nv_bfloat162 r;
    memcpy(&r, &w, 4);
    return r;
  }
  __device__ __forceinline__ static float max16(float m, const uint4& q) {
    const __nv_bfloat162 a = __hmax2(__hmax2(b2(q.x), b2(q.y)), __hmax2(b2(q.z), b2(q.w)));
    return fmaxf(m, fmaxf(__low2float(a), __high2float(a)));
  }
  __device__ __forceinline__ static F2 pair(const uint4& q, int i) {
    const uint32_t w = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  __device__ __forceinline__ static Thr thr(float x) { return Thr{__float2bfloat162_rn(x)}; }
  __device__ __forceinline__ static void above(Cnt& c, const uint4& q, const Thr& t) {
    c.n = __hadd2(c.n, __hadd2(__hadd2(__hgt2(b2(q.x), t.x), __hgt2(b2(q.y), t.x)),
                               __hadd2(__hgt2(b2(q.z), t.x), __hgt2(b2(q.w), t.x))));
  }
  __device__ __forceinline__ static Cnt zero() { return Cnt{__float2bfloat162_rn(0.f)}; }
  __device__ __forceinline__ static int total(const Cnt& c) {
    return (int)(__low2float(c.n) + __high2float(c.n));
  }
};

// The 16 bytes of a row whose first entry is v0 (16-byte aligned; v0 < 0 in front of a row that
// starts inside them): entries outside [0, V) are not read, and are -inf.
template <typename T>
__device__ __forceinline__ uint4 load16(const T* z, int v0, int V) {
  constexpr int E = Lg<T>::E;
  if (v0 >= 0 && v0 + E <= V) return __ldg((const uint4*)(z + v0));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (E == 4) {
      w[i] = v0 + i >= 0 && v0 + i < V ? ((const uint32_t*)z)[v0 + i] : Lg<T>::kFill;
    } else {
      const int a = v0 + 2 * i;
      const uint32_t lo = a >= 0 && a < V ? ((const uint16_t*)z)[a] : (Lg<T>::kFill & 0xFFFFu);
      const uint32_t hi = a + 1 >= 0 && a + 1 < V ? ((const uint16_t*)z)[a + 1] : (Lg<T>::kFill & 0xFFFFu);
      w[i] = lo | (hi << 16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// entries between the 16-byte boundary at or below a row's start and the start
template <typename T>
__device__ __forceinline__ int row_head(const T* z) {
  return (int)(((uintptr_t)z & 15) / sizeof(T));
}

// 16 bytes of a row from fp32 values, rounded once
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* f);
template <>
__device__ __forceinline__ uint4 pack16<float>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    memcpy(&w[i], &b, 4);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

}  // namespace dspark
