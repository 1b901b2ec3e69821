// elem.cuh -- 16-byte vectors of the element types as floats and back.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moeperm {

// Pairs of floats for the packed 32-bit instructions of sm_100 and later (one
// issue slot for two multiply-adds; each half rounds as the scalar one does).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 halves(f32x2 v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <int TYPE>
struct Vec {
  static constexpr int kBytes = TYPE == kF32 ? 4 : 2;
  static constexpr int kN = 16 / kBytes;  // elements per vector
  __device__ __forceinline__ static void unpack(const uint4& v, float (&f)[kN]) {
    if constexpr (TYPE == kF32) {
      f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
      f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == kBF16) {
          f[2 * i] = bf16_lo(w[i]);
          f[2 * i + 1] = bf16_hi(w[i]);
        } else {
          const float2 p = f16x2_to_float2(w[i]);
          f[2 * i] = p.x;
          f[2 * i + 1] = p.y;
        }
      }
    }
  }
  static constexpr int kP = kN / 2;  // pairs per vector
  __device__ __forceinline__ static void unpack2(const uint4& v, f32x2 (&p)[kP]) {
    float f[kN];
    unpack(v, f);
#pragma unroll
    for (int i = 0; i < kP; ++i) p[i] = pair(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ static uint4 pack2(const f32x2 (&p)[kP]) {
    float f[kN];
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const float2 h = halves(p[i]);
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    }
    return pack(f);
  }
  __device__ __forceinline__ static uint4 pack(const float (&f)[kN]) {
    if constexpr (TYPE == kF32) {
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                        __float_as_uint(f[3]));
    } else if constexpr (TYPE == kBF16) {
      return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                        pack_bf16x2(f[6], f[7]));
    } else {
      return make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]),
                        pack_f16x2(f[6], f[7]));
    }
  }
};

}  // namespace moeperm
