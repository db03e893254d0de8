// MXFP4 quantiser and its inverse for gfx950.
//
// Every block of 32 values (of a row, or of a column for the transposed
// direction) gets the exponent
//   e = max(floor(log2(amax)) - 2, -127)   (all-zero block: -127)
// which puts its largest magnitude into [4, 8) 2^e, and the codes
//   E2M1(x / 2^e), rounded to nearest, ties to even, at most 6.
// floor(log2(amax)) is amax's exponent field, x / 2^e is exact, so codes and
// exponents do not depend on how they are computed.  A block that holds an
// infinity or a NaN gets the exponent byte 255 (it reads back as NaN) and
// codes 0.  Blocks that reach past the end are filled with zeros; bytes of
// the last scale word past the last block are 0.
//
// Both kernels are bound by HBM: 2 or 4 bytes read and 17/32 written per
// value and direction.
#include "mxfp4_device.hpp"

namespace dg {
namespace {

struct QuantArgs {
  const void* x;
  int64_t rows, cols, ldx;
  uint8_t* q;
  uint8_t* sf;  // little-endian words, written byte by byte or as words
  uint8_t* qt;
  uint8_t* sft;
};

template <bool BF16>
__device__ __forceinline__ float load_value(const void* x, int64_t i) {
  if constexpr (BF16) return bf16_bits_to_f32(static_cast<const uint16_t*>(x)[i]);
  return static_cast<const float*>(x)[i];
}

// Exponent byte of a block with largest magnitude amax (NaN propagates as a
// number with exponent field 255).
__device__ __forceinline__ uint32_t mxfp4_exponent(uint32_t amax_bits) {
  const uint32_t f = amax_bits >> 23;
  return f == 255u ? 255u : (f < 2u ? 0u : f - 2u);
}

// The conversion's scale operand for an exponent byte (its exponent field is
// what counts; 2^-127 is given as that subnormal).
__device__ __forceinline__ float mxfp4_scale(uint32_t e) {
  return __uint_as_float(e == 0u ? 0x00400000u : e << 23);
}

// Codes of eight values, the first in the lowest nibble.
// v_cvt_scalef32_pk_fp4_f32 rounds x / 2^e to nearest even and saturates; it
// was compared on an MI355X with the rounding above on a grid of step 2^-10
// over [0, 8], both neighbours of every tie, +-0, subnormals and infinity, at
// exponents from -127 to 127: no difference.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], uint32_t e) {
  const float s = mxfp4_scale(e);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
  return e == 255u ? 0u : w;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// One thread per block of 32 values along a row (or, TR, along a column).
template <bool BF16, bool TR>
__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(QuantArgs p) {
  const int64_t R = TR ? p.cols : p.rows, C = TR ? p.rows : p.cols;  // of the result
  const int64_t words = (C + 127) / 128;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  // consecutive threads: consecutive rows for TR (coalesced reads)
  const int64_t blocks = words * 4;
  int64_t r, b;
  if (TR) {
    b = idx / R;
    r = idx - b * R;
  } else {
    r = idx / blocks;
    b = idx - r * blocks;
  }
  if (r >= R || b >= blocks) return;
  uint8_t* sf = (TR ? p.sft : p.sf) + ((b >> 2) * R + r) * 4 + (b & 3);
  if (b * 32 >= C) {
    *sf = 0;
    return;
  }
  float v[32];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const int64_t c = b * 32 + j;
    v[j] = c < C ? load_value<BF16>(p.x, TR ? c * p.ldx + r : r * p.ldx + c) : 0.0f;
    m = max(m, abs_bits(v[j]));
  }
  const uint32_t e = mxfp4_exponent(m);
  *sf = (uint8_t)e;
  uint4 w;
  uint32_t* wp = &w.x;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = v[8 * h + j];
    wp[h] = encode8(t, e);
  }
  const int64_t ldq = (C + 31) / 32 * 16;
  *reinterpret_cast<uint4*>((TR ? p.qt : p.q) + r * ldq + b * 16) = w;
}

template <bool BF16>
__global__ void __launch_bounds__(256)
dequantize_mxfp4_kernel(void* out, const uint8_t* q, const uint8_t* sf, int64_t rows,
                        int64_t cols) {
  const int64_t n8 = (cols + 7) / 8;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = idx / n8, c = (idx - r * n8) * 8;
  if (r >= rows) return;
  const int64_t ldq = (cols + 31) / 32 * 16;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(q + r * ldq + c / 2);
  const uint32_t e = sf[((c >> 7) * rows + r) * 4 + ((c >> 5) & 3)];
  const float s = __uint_as_float(e << 23);
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    // exact in BF16 down to its subnormals' last bit, 2^-133; the smallest
    // value is 0.5 2^-127
    const dg_bf16x2 t = h == 0   ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)
                        : h == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)
                        : h == 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)
                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    const uint32_t u = __builtin_bit_cast(uint32_t, t);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t cc = c + 2 * h + j;
      if (cc >= cols) continue;
      const uint32_t bits = j == 0 ? u & 0xFFFFu : u >> 16;
      if constexpr (BF16)
        static_cast<uint16_t*>(out)[r * cols + cc] = (uint16_t)bits;
      else
        static_cast<uint32_t*>(out)[r * cols + cc] = bits << 16;
    }
  }
}

template <bool BF16, bool TR>
hipError_t quantize_way(const QuantArgs& p, hipStream_t stream) {
  const int64_t R = TR ? p.cols : p.rows, C = TR ? p.rows : p.cols;
  const int64_t n = (C + 127) / 128 * 4 * R;
  hipLaunchKernelGGL((quantize_mxfp4_kernel<BF16, TR>), dim3((unsigned)((n + 255) / 256)),
                     dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_mxfp4(uint8_t* q, uint32_t* sf, uint8_t* qt, uint32_t* sft,
                                 const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ldx,
                                 hipStream_t stream) {
  const QuantArgs p{x, rows, cols, ldx, q, reinterpret_cast<uint8_t*>(sf), qt,
                    reinterpret_cast<uint8_t*>(sft)};
  hipError_t e = hipSuccess;
  if (q) e = bf16 ? quantize_way<true, false>(p, stream) : quantize_way<false, false>(p, stream);
  if (e == hipSuccess && qt)
    e = bf16 ? quantize_way<true, true>(p, stream) : quantize_way<false, true>(p, stream);
  return e;
}

hipError_t launch_dequantize_mxfp4(void* out, bool bf16, const uint8_t* q, const uint32_t* sf,
                                   int64_t rows, int64_t cols, hipStream_t stream) {
  const int64_t n = rows * ((cols + 7) / 8);
  const uint8_t* s = reinterpret_cast<const uint8_t*>(sf);
  const dim3 grid((unsigned)((n + 255) / 256));
  if (bf16)
    hipLaunchKernelGGL(dequantize_mxfp4_kernel<true>, grid, dim3(256), 0, stream, out, q, s, rows,
                       cols);
  else
    hipLaunchKernelGGL(dequantize_mxfp4_kernel<false>, grid, dim3(256), 0, stream, out, q, s, rows,
                       cols);
  return hipGetLastError();
}

}  // namespace dg
