// fp4.cuh -- four-bit rows: e2m1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign)
// with one scale byte for each group along the row, and their quantisation.
//
//   e8m0  groups of 32, scale 2^e, e the least with 6 * 2^e >= amax
//   mx    groups of 32, e = floor(log2 amax) - 2, elements above 6 saturate (OCP MX)
//   nv    groups of 16, scale s = e4m3(amax / (6 ts)), elements x / (s * ts), with a
//         float32 scale ts of the whole tensor
//
// A group with a NaN or an infinity gets a scale of NaN and zero elements, so that
// products with it are NaN. Element 2 i is the low half of byte i. The scales of 16
// groups are one 16-byte piece; piece c of row r is at (c * ld + r) * 16, so that
// the pieces of consecutive rows are contiguous: what a tile of a product needs of
// one piece column is a single bulk copy that starts at any row. Bytes of the last
// piece past the row's groups are 0.
#pragma once

#include "elem.cuh"

namespace moeperm {

__host__ __device__ constexpr int fp4_group(int fmt) { return fmt == kFp4NV ? 16 : 32; }
__host__ __device__ constexpr int fp4_pieces(int H, int fmt) { return (H / fp4_group(fmt) + 15) / 16; }

// Eight floats to e2m1 (round to nearest even, saturating), the first in the low bits.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// The way back, as pairs of fp16 (exact).
__device__ __forceinline__ void e2m1x8_to_floats(uint32_t q, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(q));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = f16x2_to_float2(h[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// What a scale byte multiplies elements by: 2^(b - 127) (NaN for 255), or s * ts.
template <int FMT>
__device__ __forceinline__ float fp4_scale(uint32_t byte, float ts) {
  if constexpr (FMT == kFp4NV) return __fmul_rn(e4m3x2_to_float2(byte).x, ts);
  return byte == 0 ? 0x1p-127f : byte == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}

// 32 bytes at once, so that the lanes of a warp read or write one run of memory.
__device__ __forceinline__ void ld_nc_v8(const void* p, uint4& a, uint4& b) {
  asm("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
      : "l"(p));
}
__device__ __forceinline__ void st_v8(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// A chunk of 16 elements as a lane holds it. `wide`: the address is a multiple of 32.
template <int TYPE>
struct Chunk {
  static constexpr int kVecs = TYPE == kF32 ? 4 : 2;
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const void* p, bool valid, bool wide) {
    if (wide) {
#pragma unroll
      for (int i = 0; i < kVecs; i += 2) {
        if (valid) ld_nc_v8(static_cast<const uint8_t*>(p) + 16 * i, v[i], v[i + 1]);
        else v[i] = v[i + 1] = make_uint4(0, 0, 0, 0);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      v[i] = valid ? ld_nc_v4(static_cast<const uint8_t*>(p) + 16 * i) : make_uint4(0, 0, 0, 0);
  }
  // The largest magnitude, as the bits of a float (those of infinity or above for one
  // that holds an infinity or a NaN: the order of the bits is that of the magnitudes).
  __device__ __forceinline__ uint32_t amax() const {
    if constexpr (TYPE == kF32) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        m = max(m, max(max(v[i].x & 0x7FFFFFFFu, v[i].y & 0x7FFFFFFFu), max(v[i].z & 0x7FFFFFFFu, v[i].w & 0x7FFFFFFFu)));
      return m;
    } else {
      const uint32_t m = amax16_bf16(v[0], v[1]);  // (the order of fp16's bits is the same)
      if constexpr (TYPE == kBF16) return m << 16;
      return __float_as_uint(f16x2_to_float2(m).x) & 0x7FFFFFFFu;
    }
  }
  __device__ __forceinline__ void floats(float (&f)[16]) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float p[Vec<TYPE>::kN];
      Vec<TYPE>::unpack(v[i], p);
#pragma unroll
      for (int j = 0; j < Vec<TYPE>::kN; ++j) f[i * Vec<TYPE>::kN + j] = p[j];
    }
  }
};

// Quantises a chunk; every lane of the warp calls it. Returns the 16 elements and the
// byte of the chunk's group (the same in both lanes of a group of 32).
//
// nv divides by d = fl32(s * ts): a product with the reciprocal, corrected once by
// its remainder (Markstein 1990, correct rounding of a division by fused
// multiply-adds), two elements an instruction. That holds while d, 1/d and the
// quotients are far from the ends of the range; otherwise the elements are divided one
// by one. The quotients are formed with the other sign, which the codes then lose: a zero's
// remainder is +0, and fma(+0, 1/d, -0) would be +0 for an element of -0, where fma(+0, -1/d, +0)
// is the +0 that becomes -0.
template <int TYPE, int FMT>
__device__ __forceinline__ uint2 fp4_quant(const Chunk<TYPE>& x, float ts, float ts6, uint32_t& byte) {
  uint32_t am = x.amax();
  if constexpr (FMT != kFp4NV) am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
  const bool finite = am < 0x7F800000u;
  float f[16];
  x.floats(f);
  uint32_t flip = 0;  // signs of eight codes
  if constexpr (FMT == kFp4NV) {
    flip = 0x88888888u;
    // (a group of zeros has scale 0 whatever the tensor's: that of a tensor of zeros is 0, too)
    byte = am == 0 ? 0u : cvt_e4m3x2(__fdiv_rn(__uint_as_float(am), ts6), 0.0f) & 0xFF;
    const float d = fp4_scale<kFp4NV>(byte, ts);
    if (!finite) byte = 0x7F;
    const bool some = finite && d > 0.0f;
    if (some && !(d > 0x1p-100f && d < 0x1p100f && __uint_as_float(am) < 0x1p20f * d)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = __fdiv_rn(f[i], -d);
    } else {
      const float y = some ? __frcp_rn(d) : 0.0f;
      const f32x2 ny = pair(-y, -y), dd = pair(d, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const f32x2 v = pair(f[2 * i], f[2 * i + 1]), q = mul2(v, ny);
        const float2 r = halves(fma2(fma2(q, dd, v), ny, q));
        f[2 * i] = r.x;
        f[2 * i + 1] = r.y;
      }
    }
    if (!some) {  // nothing that a scale reaches, or no numbers
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = -0.0f;
    }
  } else {
    // amax = 1.m * 2^E, 6 = 1.5 * 2^2
    const int E = (int)(am >> 23) - 127;
    const int e = max(E - 2 + (FMT == kFp4E8M0 && (am & 0x7FFFFFu) > 0x400000u ? 1 : 0), -127);
    byte = finite ? (uint32_t)(e + 127) : 255u;
    const float inv = finite ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.0f;  // 2^-e, e in [-127, 126]
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = finite ? __fmul_rn(f[i], inv) : 0.0f;
  }
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = f[i];
    hi[i] = f[8 + i];
  }
  return make_uint2(cvt_e2m1x8(lo) ^ flip, cvt_e2m1x8(hi) ^ flip);
}

// The bytes of four groups as a word, in the first lane of the 4 (nv) or 8 lanes that
// hold them; lane: whether this lane is one of those.
template <int FMT>
__device__ __forceinline__ uint32_t fp4_scale_word(uint32_t byte) {
  constexpr int kStep = FMT == kFp4NV ? 1 : 2;
  byte |= __shfl_down_sync(0xffffffffu, byte, kStep) << 8;
  return byte | (__shfl_down_sync(0xffffffffu, byte, 2 * kStep) << 16);
}
template <int FMT>
__device__ __forceinline__ bool fp4_word_lane(int lane) {
  return lane % (FMT == kFp4NV ? 4 : 8) == 0;
}
// Offset of the word of the groups of chunk c (a multiple of 4 or 8) within a row's
// pieces: piece, and byte in it.
template <int FMT>
__device__ __forceinline__ int fp4_piece_of(int c) {
  return c / (FMT == kFp4NV ? 16 : 32);
}
template <int FMT>
__device__ __forceinline__ int fp4_byte_of(int c) {
  return c % (FMT == kFp4NV ? 16 : 32) / (FMT == kFp4NV ? 1 : 2);
}

}  // namespace moeperm
