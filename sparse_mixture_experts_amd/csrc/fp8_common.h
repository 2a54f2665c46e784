// fp8_common.h -- device helpers of the 8-bit (OCP e4m3) formats: quantising
// a block of values to codes with one fp32 scale, and the K = 128 matrix
// instruction that multiplies the codes.
//
// Blocks hold 128 reduction elements.  With m = max(amax, 448 * 2^-126) of a
// block, scale = m / 448 and code = e4m3(448 x / m), to nearest even; 448 is
// the largest e4m3 value, and the floor keeps the scale a normal number (an
// all-zero block gets codes 0).  The quotient is rounded to fp32 once before
// it is rounded to 4 significant bits: it is computed correctly rounded, so a
// value that lies exactly between two codes (common, because 16-bit inputs
// have few bits) stays exactly between them and goes to the even one.
#pragma once

#include "dequant_f16.h"
#include "device_common.h"

namespace moe {

constexpr int kFp8Block = 128;            // reduction elements per scale, and rows of a weight block
constexpr float kFp8Max = 448.0f;
constexpr float kFp8AmaxFloor = 448.0f * 1.17549435e-38f;  // 448 * 2^-126

// The quantiser of one block: x -> 448 x / m.  m = a * 2^e with a in [1, 2);
// t = x * (448 * 2^-e) is exact for inputs of up to 21 significant bits,
// and t / a follows from the correctly rounded reciprocal y of a by one
// residual step (q0 = t y, q = q0 + (t - q0 a) y), which gives the correctly
// rounded quotient.  An infinite amax sends finite values to 0 and infinite
// ones to NaN.
struct Fp8Quant {
  float a, y, c, scale;
  __device__ __forceinline__ explicit Fp8Quant(float amax) {
    const float m = fmaxf(amax, kFp8AmaxFloor);
    scale = m / kFp8Max;
    const uint32_t b = __float_as_uint(m);
    const bool inf = b >= 0x7f800000u;
    a = __uint_as_float((b & 0x007fffffu) | 0x3f800000u);
    y = 1.0f / a;
    // 448 * 2^-e = 1.75 * 2^(8 - e), e = (b >> 23) - 127 in [-118, 127]
    c = inf ? 0.0f : 1.75f * __uint_as_float((uint32_t(262 - int(b >> 23))) << 23);
  }
  __device__ __forceinline__ float operator()(float x) const {
    const float t = x * c;
    const float q0 = t * y;
    return __builtin_fmaf(__builtin_fmaf(-q0, a, t), y, q0);
  }
};

// Four values (already divided by their scale) as e4m3 codes, nearest even.
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

// The largest magnitude over the 8 lanes of a half row (lanes 8i .. 8i+7),
// in every one of them.
__device__ __forceinline__ float max8_lanes(float v) {
  v = fmaxf(v, dpp_move<kDppQuadSwap1>(v, v));
  v = fmaxf(v, dpp_move<kDppQuadSwap2>(v, v));
  return fmaxf(v, dpp_move<kDppHalfMirror>(v, v));
}

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float fp8_acc __attribute__((ext_vector_type(4)));

// Eight codes as fp16.
__device__ __forceinline__ uint4 fp8_to_f16(uint32_t a, uint32_t b) {
  const h2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false),
                   __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true),
                   __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false),
                   __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true)};
  return make_uint4(__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]),
                    __builtin_bit_cast(uint32_t, v[2]), __builtin_bit_cast(uint32_t, v[3]));
}

// The 32 codes of a 128-element block that a lane holds as an operand of one
// 16x16 tile: row (operand a) or column (operand b) lane % 16.  The lane's
// four results are rows 4 * (lane / 16) + i of column lane % 16.  Any
// assignment of the 128 elements to (lane / 16, place) is right as long as
// both operands use it.
//
// Two instructions multiply them.  The 8-bit one takes the block at once, at
// twice the 16-bit rate, but aligns the products of each 8 neighbouring
// elements to the largest and drops, towards zero, what lies 13 binary places
// below its leading one (measured: beside 2^16, 2^3 is kept and 2^2 lost; the
// sums of eight are then added in fp32): 1.5e-5 of a result's norm on
// normally distributed values.  That is far below half a step of a 16-bit
// result (2^-9 for bf16, 2^-12 for fp16) and is used for those alone.  Where
// a result stays in fp32 or is rounded again later (EXACT), the codes go to
// fp16, which holds every one of them, two per instruction, and four 16-bit
// products sum them in fp32.
template <bool EXACT>
struct Fp8Operand {
  i32x8 v;
  __device__ __forceinline__ explicit Fp8Operand(const i32x8 &c) : v(c) {}
};
template <>
struct Fp8Operand<true> {
  f16x8 v[4];
  __device__ __forceinline__ Fp8Operand(const uint4 &a, const uint4 &b, const uint4 &c, const uint4 &d)
      : v{__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, c),
          __builtin_bit_cast(f16x8, d)} {}
  __device__ __forceinline__ explicit Fp8Operand(const i32x8 &c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __builtin_bit_cast(f16x8, fp8_to_f16(c[2 * j], c[2 * j + 1]));
  }
};
template <bool EXACT>
__device__ __forceinline__ fp8_acc fp8_product(const Fp8Operand<EXACT> &a, const Fp8Operand<EXACT> &b) {
  fp8_acc z = {0.f, 0.f, 0.f, 0.f};
  if constexpr (EXACT) {
#pragma unroll
    for (int j = 0; j < 4; ++j) z = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[j], b.v[j], z, 0, 0, 0);
    return z;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, z, 0, 0, 0, 0, 0, 0);
  }
}

__device__ __forceinline__ i32x8 join8(const uint4 &lo, const uint4 &hi) {
  i32x8 v;
  v[0] = int(lo.x), v[1] = int(lo.y), v[2] = int(lo.z), v[3] = int(lo.w);
  v[4] = int(hi.x), v[5] = int(hi.y), v[6] = int(hi.z), v[7] = int(hi.w);
  return v;
}

}  // namespace moe
