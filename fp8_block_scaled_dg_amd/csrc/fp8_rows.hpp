// Device helpers of the kernels that write E4M3 rows with one FP32 scale per 128
// columns (dispatch.hip, swiglu_fp8.hip): the quantiser's codes and scales
// (s = binary32(amax / 448), code = E4M3(binary32(x / s)), dg_device.hpp) in as few
// instructions as they can be had, since these kernels quantise two or three
// values for each one they read and the VALU would bound them (SwiGLU with its
// checkpoint, 32768 rows of 1408 units, 32 rows a workgroup: 88 us with dg_device.hpp's
// encoder and fmaxf, some 54 instructions a unit, 75 with these).
#pragma once

#include "dg_device.hpp"

namespace dg {

// max(m, |x|) in one instruction (fmaxf quiets its operands first); no NaN.
__device__ __forceinline__ float join_top(float m, float x) {
  return __builtin_amdgcn_fmed3f(fabsf(x), m, __builtin_inff());
}
template <int N>
__device__ __forceinline__ float top_of(const float (&v)[N]) {
  float a = fabsf(v[0]), b = fabsf(v[1]);  // two chains
#pragma unroll
  for (int i = 2; i < N; i += 2) {
    a = join_top(a, v[i]);
    b = join_top(b, v[i + 1]);
  }
  return join_top(a, b);
}

// Largest of the values of G = 4, 8 or 16 neighbouring lanes, none negative: their
// bits order like them, and the integer maximum takes its operand across lanes.
template <int G>
__device__ __forceinline__ float group_top(float v) {
  uint32_t u = __float_as_uint(v);
  u = max(u, (uint32_t)__builtin_amdgcn_mov_dpp((int)u, 0xB1, 0xF, 0xF, false));
  u = max(u, (uint32_t)__builtin_amdgcn_mov_dpp((int)u, 0x4E, 0xF, 0xF, false));
  if constexpr (G >= 8) u = max(u, (uint32_t)__builtin_amdgcn_mov_dpp((int)u, 0x141, 0xF, 0xF, false));
  if constexpr (G >= 16) u = max(u, (uint32_t)__builtin_amdgcn_mov_dpp((int)u, 0x140, 0xF, 0xF, false));
  return __uint_as_float(u);
}

// RN(1 / d): v_rcp_f32 (one unit in the last place) and one Newton step.  Not proved
// but shown: for all 2^23 significands of d and exponents from end to end of 2^-64 to
// 2^126 there is no difference from the division (a test compares them).
__device__ __forceinline__ float reciprocal_rn(float d) {
  const float r = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}

// Scale of a block and what its values are divided by.
//   scale : amax / 448, correctly rounded: the product with RN(1/448) and one FMA
//           correction (Markstein; the remainder is exact from 2^-90 up)
//   s, r  : the divisor and RN(1 / s)
// Blocks with amax below 2^-50 (rare, a branch of its own) take the division, and
// where the scale is below 2^-62 their values are lifted by 2^64, as block_scale
// does; r is 0 for an all-zero block.
struct RowScale {
  float scale, s, r;
};

template <int N>
__device__ __forceinline__ RowScale row_scale(float (&v)[N], float amax) {
  constexpr float r448 = 1.0f / 448.0f;
  RowScale b;
  const float q = amax * r448;
  b.scale = __builtin_fmaf(__builtin_fmaf(-q, 448.0f, amax), r448, q);
  b.s = b.scale;
  if (amax < 0x1p-50f) {
    b.scale = b.s = amax / 448.0f;
    if (b.s < 0x1p-62f) {
      b.s *= 0x1p64f;
      // a subnormal scale is rounded by up to half: past 448 the codes saturate
      const float most = b.s > 0.0f ? 448.0f * b.s : __builtin_inff();
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __builtin_amdgcn_fmed3f(v[i] * 0x1p64f, -most, most);
    }
  }
  b.r = b.s == 0.0f ? 0.0f : reciprocal_rn(b.s);
  return b;
}

// Codes of N values.  The quotient is quotient_rn's, its correction taken as
// q - (q s - x) r: that keeps the sign of a zero.  No quotient is above
// 448 (1 + 2^-23), which rounds to 448, so none needs a clamp.
template <int N>
__device__ __forceinline__ void encode_values(const float (&v)[N], const RowScale& b,
                                              uint32_t (&codes)[N / 4]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    float q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = v[i + j], a = x * b.r;
      q[j] = __builtin_fmaf(-__builtin_fmaf(a, b.s, -x), b.r, a);
    }
    const int p = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    codes[i / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], p, true);
  }
}

// Streams that this launch does not read again: they leave the L2 to what it does.
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store_stream(uint8_t* out, const uint32_t (&w)[2]) {
  __builtin_nontemporal_store((u2){w[0], w[1]}, reinterpret_cast<u2*>(out));
}
__device__ __forceinline__ void store_stream(uint8_t* out, const uint32_t (&w)[4]) {
  __builtin_nontemporal_store((u4){w[0], w[1], w[2], w[3]}, reinterpret_cast<u4*>(out));
}

}  // namespace dg
