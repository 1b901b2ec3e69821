// elem.cuh -- 16-byte vectors of the element types as floats and back.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moeperm {

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
