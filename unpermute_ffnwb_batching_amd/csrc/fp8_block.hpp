// Device helpers of the expert operators: e4m3 values with a scale for each 128 elements.
//
// gfx950 holds e4m3 in the OCP form (bias 7, largest 448, NaN 0x7f / 0xff, no infinity).
// Its conversions from FP32 round to nearest even and keep NaN; its conversions to BF16 and
// FP16 are exact.
#pragma once

#include "device_common.hpp"

namespace ffnwb {

constexpr int kBlk = 128;  // elements under one scale

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Loads from global memory: pointers taken out of a structure would be loaded from as "flat".
__device__ __forceinline__ u32x4 load16(const void* p) { return *(const __attribute__((address_space(1))) u32x4*)p; }
__device__ __forceinline__ float load_f32(const float* p) { return *(const __attribute__((address_space(1))) float*)p; }

// The scale of a block whose largest |x| has the FP32 bits `amax_bits`.  Taken as integers
// (monotonic in |x|, NaN above infinity above every finite value), so that a NaN or an
// infinity in the block reaches its scale.  2^-126 keeps the quotients of tiny blocks finite.
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
  const float a = __uint_as_float(amax_bits);
  const float s = a / 448.0f;
  return s < 1.17549435e-38f ? 1.17549435e-38f : s;
}

// x / s rounded to nearest for the values of one block, |x / s| <= 448.  r = RN(1/s), q0 =
// RN(x r); the residual q0 s - x is exact in one FMA, and RN(q0 - residual r) is the quotient
// (the last step of division by Newton's iteration, Markstein 1990): 3 operations where the
// division takes about 10.  With the residual taken this way round, x = -0 gives -0: its residual is +0,
// and -0 - (+0) stays -0, where -0 + (+0) would be +0.  Equal to the division on 4e7 operands, half of them within 3
// steps of a midpoint of e4m3, the only place where the last bit could matter.  Residuals must
// not underflow: quotients below 2^-11 are 0 in e4m3, so s >= 2^-80 is ample; s <= 2^100 keeps
// r normal.  Other blocks, those with infinities and NaN among them, divide.
template <int N>
__device__ __forceinline__ void block_quotients(float (&x)[N], float s) {
  if (s >= 0x1p-80f && s <= 0x1p100f) {
    const float r = 1.0f / s;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float q0 = x[i] * r;
      x[i] = __builtin_fmaf(-__builtin_fmaf(q0, s, -x[i]), r, q0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = x[i] / s;
  }
}

// Four FP32 values -> four e4m3 bytes, x[0] lowest.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return static_cast<uint32_t>(v);
}

// Quantises the block of which each of 16 adjacent lanes holds 8 elements (0 past the row's
// end): returns its scale and leaves the lane's e4m3 bytes in lo, hi.
__device__ __forceinline__ float quant_block(float (&f)[8], uint32_t& lo, uint32_t& hi) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d)));
  const float s = block_scale(m);
  block_quotients(f, s);
  lo = pack_e4m3(f[0], f[1], f[2], f[3]);
  hi = pack_e4m3(f[4], f[5], f[6], f[7]);
  return s;
}

// Matrix products of 16 rows of A by 16 rows of B (row lane % 16, columns split over the four
// groups lane / 16); the result lane holds B row lane % 16 and A rows 4 (lane / 16) + 0..3.
// The order of the columns over lanes and registers only has to be the same for A and B.
//
// In the 16-bit types (32 columns) a product of two e4m3 values is exact and sums are in FP32:
// 3e-9 of the result's size off for 32 columns.  The e4m3 instructions (twice
// the rate) add products in groups of 8 columns, and drop the bits of
// each below 2^-13 of the power of two of the group's largest, whatever the shape of the
// instruction: 1.5e-5 of the result's size for normal data, at most 7 * 2^-13 of each group's largest
// product, which is without bound against a result that large products cancel to.

__device__ __forceinline__ bf16x8 as_bf16(const u32x4& v) { return __builtin_bit_cast(bf16x8, v); }
__device__ __forceinline__ f16x8 as_f16(const u32x4& v) { return __builtin_bit_cast(f16x8, v); }

template <class T> struct Mat;  // 16x16x32 products in the type of the activations
template <> struct Mat<TBF16> {
  __device__ static f32x4 mul(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(a), as_bf16(b), c, 0, 0, 0);
  }
  __device__ static uint32_t widen(uint32_t v, bool hi) {  // two e4m3 -> two BF16
    const bf16x2 r = hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true)
                        : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false);
    return __builtin_bit_cast(uint32_t, r);
  }
};
template <> struct Mat<TF16> {
  __device__ static f32x4 mul(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(as_f16(a), as_f16(b), c, 0, 0, 0);
  }
  __device__ static uint32_t widen(uint32_t v, bool hi) {
    const f16x2 r = hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, true)
                       : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, false);
    return __builtin_bit_cast(uint32_t, r);
  }
};

// Eight e4m3 values (two registers) -> BF16, exactly.
__device__ __forceinline__ u32x4 widen8(uint32_t a, uint32_t b) {
  return u32x4{Mat<TBF16>::widen(a, false), Mat<TBF16>::widen(a, true), Mat<TBF16>::widen(b, false), Mat<TBF16>::widen(b, true)};
}

// silu(g) * u = g * sigmoid(g) * u.  exp(-g) overflows to infinity for very negative g, which
// gives the limit -0; g = -inf is NaN, as in g * sigmoid(g).
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + expf(-g)) * u; }

}  // namespace ffnwb
