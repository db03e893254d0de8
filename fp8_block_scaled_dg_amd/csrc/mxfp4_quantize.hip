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
// value and direction.  MI355X, 8192 x 8192 BF16: both directions from one
// reading 47 us (205 MB, 4.4 TB/s), back to BF16 28 to 31 us (170 MB, 5.5 to
// 6.0 TB/s; a plain copy of 1 GiB moves 5.1); 64 x 4096: 2.5 us, the launch.
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

// Codes of eight values held as BF16 pairs or as FP32, the first in the lowest
// nibble.  v_cvt_scalef32_pk_fp4_f32 rounds x / 2^e to nearest even and
// saturates; it was compared on an MI355X with the rounding above on a grid
// of step 2^-10 over [0, 8], both neighbours of every tie, +-0, subnormals and
// infinity, at exponents from -127 to 127: no difference.  The BF16 form
// takes the same values without widening them first.
__device__ __forceinline__ uint32_t encode8(const uint32_t (&v)[4], float s) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(dg_bf16x2, v[0]), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(dg_bf16x2, v[1]), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(dg_bf16x2, v[2]), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(dg_bf16x2, v[3]), s, 3);
  return w;
}
__device__ __forceinline__ uint32_t encode8(const uint32_t (&v)[8], float s) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(v[0]), __uint_as_float(v[1]), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(v[2]), __uint_as_float(v[3]), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(v[4]), __uint_as_float(v[5]), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(v[6]), __uint_as_float(v[7]), s, 3);
  return w;
}

typedef unsigned short us2 __attribute__((ext_vector_type(2)));

// Largest magnitude of a dword's values (two BF16 or one FP32) joined to m,
// as bits (they order like the magnitudes, NaN above infinity); fold() leaves
// it as FP32 bits.
template <bool BF16>
__device__ __forceinline__ uint32_t join(uint32_t m, uint32_t v) {
  if constexpr (BF16) {
    const us2 r = __builtin_elementwise_max(__builtin_bit_cast(us2, m),
                                            __builtin_bit_cast(us2, v & 0x7FFF7FFFu));
    return __builtin_bit_cast(uint32_t, r);
  }
  return max(m, v & 0x7FFFFFFFu);
}
template <bool BF16>
__device__ __forceinline__ uint32_t fold(uint32_t m) {
  if constexpr (BF16) return max(m << 16, m & 0xFFFF0000u);
  return m;
}

// Eight consecutive values of a row from column c on, zeros from `cols` on.
// The row starts at any element, so the wide load is not aligned to its size
// (the memory path takes that).
template <bool BF16>
__device__ __forceinline__ void load8(const QuantArgs& p, int64_t r, int64_t c,
                                      uint32_t (&v)[BF16 ? 4 : 8]) {
  constexpr int SZ = BF16 ? 2 : 4;
#pragma unroll
  for (int j = 0; j < 2 * SZ; ++j) v[j] = 0;
  if (r >= p.rows || c >= p.cols) return;
  const char* s = static_cast<const char*>(p.x) + (r * p.ldx + c) * SZ;
  if (c + 8 <= p.cols) {
    __builtin_memcpy(v, __builtin_assume_aligned(s, SZ), 8 * SZ);
    return;
  }
  const int n = (int)(p.cols - c);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) {
      if constexpr (BF16)
        v[j >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(s)[j] << (16 * (j & 1));
      else
        v[j] = reinterpret_cast<const uint32_t*>(s)[j];
    }
}

__device__ __forceinline__ uint32_t dpp_ror(uint32_t v, int by4) {  // within 16 lanes
  return by4 == 4 ? (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x124, 0xF, 0xF, false)
                  : (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, false);
}

// Row direction alone: 16 lanes take 128 columns of a row, four lanes a
// block, so codes leave in 64-byte and scale words in 16-byte pieces and
// nothing goes through LDS.  A workgroup takes 16 PASSES rows of 128 columns.
template <bool BF16, int PASSES>
__global__ void __launch_bounds__(256) quantize_mxfp4_rows_kernel(QuantArgs p) {
  const int t = threadIdx.x;
  const int64_t w = blockIdx.x, c = w * 128 + 8 * (t & 15);
  const int64_t ldq = (p.cols + 31) / 32 * 16;
  uint32_t v[PASSES][BF16 ? 4 : 8];
#pragma unroll
  for (int i = 0; i < PASSES; ++i)
    load8<BF16>(p, ((int64_t)blockIdx.y * PASSES + i) * 16 + (t >> 4), c, v[i]);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t r = ((int64_t)blockIdx.y * PASSES + i) * 16 + (t >> 4);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < (BF16 ? 4 : 8); ++j) m = join<BF16>(m, v[i][j]);
    m = fold<BF16>(m);
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));
    const uint32_t e = mxfp4_exponent(m);
    uint32_t word = e << (8 * ((t >> 2) & 3));
    word |= dpp_ror(word, 4);
    word |= dpp_ror(word, 8);
    if (r >= p.rows) continue;
    if ((t & 15) == 0) reinterpret_cast<uint32_t*>(p.sf)[w * p.rows + r] = word;
    const uint32_t codes = encode8(v[i], mxfp4_scale(e));
    if (c / 2 < ldq)
      *reinterpret_cast<uint32_t*>(p.q + r * ldq + c / 2) = e == 255u ? 0u : codes;
  }
}

// The column direction, and both from one reading of x: a tile of 128 x 128
// values goes to LDS.  Rows: a thread takes a block of 32 columns.  Columns: a
// thread takes two neighbouring columns of 32 rows; the codes of the tile are
// put together in LDS first, so they too leave in 64-byte pieces.  The row
// pitch is 16 bytes over the row, which spreads both read patterns over the
// banks.
template <bool BF16, bool ROWS>
__global__ void __launch_bounds__(256) quantize_mxfp4_tile_kernel(QuantArgs p) {
  constexpr int SZ = BF16 ? 2 : 4, PITCH = 128 * SZ + 16, V = 2 * SZ;
  constexpr int CP = 80;  // bytes from one column's codes to the next
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * PITCH];
  __shared__ uint32_t col_e[128];  // one byte per row block
  const int t = threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.y * 128, c0 = (int64_t)blockIdx.x * 128;
  {
    uint32_t v[8][V];
#pragma unroll
    for (int i = 0; i < 8; ++i) load8<BF16>(p, r0 + 16 * i + (t >> 4), c0 + 8 * (t & 15), v[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint8_t* d = tile + (16 * i + (t >> 4)) * PITCH + 8 * (t & 15) * SZ;
#pragma unroll
      for (int h = 0; h < V; h += 4)
        *reinterpret_cast<uint4*>(d + 4 * h) = make_uint4(v[i][h], v[i][h + 1], v[i][h + 2], v[i][h + 3]);
    }
  }
  __syncthreads();
  if constexpr (ROWS) {
    const int64_t ldq = (p.cols + 31) / 32 * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (t >> 2) + 64 * i, b = t & 3;
      uint32_t v[4][V], m = 0;
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          const uint4 q = *reinterpret_cast<const uint4*>(tile + r * PITCH + (32 * b + 8 * h) * SZ + 4 * j);
          v[h][j] = q.x; v[h][j + 1] = q.y; v[h][j + 2] = q.z; v[h][j + 3] = q.w;
        }
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int j = 0; j < V; ++j) m = join<BF16>(m, v[h][j]);
      const uint32_t e = mxfp4_exponent(fold<BF16>(m));
      const float s = mxfp4_scale(e);
      uint32_t word = e << (8 * b);
      word |= (uint32_t)__builtin_amdgcn_mov_dpp((int)word, 0xB1, 0xF, 0xF, false);
      word |= (uint32_t)__builtin_amdgcn_mov_dpp((int)word, 0x4E, 0xF, 0xF, false);
      const int64_t row = r0 + r;
      if (row >= p.rows) continue;
      if (b == 0) reinterpret_cast<uint32_t*>(p.sf)[(int64_t)blockIdx.x * p.rows + row] = word;
      if (c0 + 32 * b < p.cols) {
        const uint32_t keep = e == 255u ? 0u : ~0u;
        *reinterpret_cast<uint4*>(p.q + row * ldq + c0 / 2 + 16 * b) =
            make_uint4(encode8(v[0], s) & keep, encode8(v[1], s) & keep, encode8(v[2], s) & keep,
                       encode8(v[3], s) & keep);
      }
    }
  }
  // columns 2 (t % 64) and + 1, rows 32 (t / 64) .. + 31
  const int cp = t & 63, rb = t >> 6;
  uint32_t x[32][SZ / 2];
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const uint32_t* s = reinterpret_cast<const uint32_t*>(tile + (32 * rb + j) * PITCH + 2 * cp * SZ);
#pragma unroll
    for (int h = 0; h < SZ / 2; ++h) x[j][h] = s[h];
  }
  __syncthreads();  // the tile's room is free: the columns' codes go there
#pragma unroll
  for (int cc = 0; cc < 2; ++cc) {
    uint32_t v[4][V], m = 0;
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (BF16)  // rows 8h + 2j and + 1 of the column, packed
          v[h][j] = cc == 0 ? __builtin_amdgcn_perm(x[8 * h + 2 * j + 1][0], x[8 * h + 2 * j][0], 0x05040100)
                            : __builtin_amdgcn_perm(x[8 * h + 2 * j + 1][0], x[8 * h + 2 * j][0], 0x07060302);
        else
          v[h][j] = x[8 * h + j][cc];
        m = join<BF16>(m, v[h][j]);
      }
    const uint32_t e = mxfp4_exponent(fold<BF16>(m));
    const float s = mxfp4_scale(e);
    const uint32_t keep = e == 255u ? 0u : ~0u;
    *reinterpret_cast<uint4*>(tile + (2 * cp + cc) * CP + 16 * rb) =
        make_uint4(encode8(v[0], s) & keep, encode8(v[1], s) & keep, encode8(v[2], s) & keep,
                   encode8(v[3], s) & keep);
    reinterpret_cast<uint8_t*>(col_e)[(2 * cp + cc) * 4 + rb] = (uint8_t)e;
  }
  __syncthreads();
  const int64_t ldt = (p.rows + 31) / 32 * 16;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = (t >> 2) + 64 * i, b = t & 3;
    if (c0 + c < p.cols && r0 + 32 * b < p.rows)
      *reinterpret_cast<uint4*>(p.qt + (c0 + c) * ldt + r0 / 2 + 16 * b) =
          *reinterpret_cast<const uint4*>(tile + c * CP + 16 * b);
  }
  if (t < 128 && c0 + t < p.cols)
    reinterpret_cast<uint32_t*>(p.sft)[(int64_t)blockIdx.y * p.cols + c0 + t] = col_e[t];
}

// Eight values per thread and pass, four passes; a row of the output starts
// at any element, so the wide store is not aligned to its size.
template <bool BF16>
__global__ void __launch_bounds__(256)
dequantize_mxfp4_kernel(void* out, const uint8_t* q, const uint8_t* sf, int64_t rows, int64_t cols,
                        int64_t n8) {
  constexpr int SZ = BF16 ? 2 : 4, V = 2 * SZ;
  const int64_t ldq = (cols + 31) / 32 * 16, total = rows * n8;
  uint32_t w[4], e[4];
  int64_t r[4], c[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t idx = ((int64_t)blockIdx.x * 4 + u) * 256 + threadIdx.x;
    r[u] = total <= 0xFFFFFFFFll ? (int64_t)((uint32_t)idx / (uint32_t)n8) : idx / n8;
    c[u] = (idx - r[u] * n8) * 8;
    if (r[u] >= rows) continue;
    w[u] = *reinterpret_cast<const uint32_t*>(q + r[u] * ldq + c[u] / 2);
    e[u] = sf[((c[u] >> 7) * rows + r[u]) * 4 + ((c[u] >> 5) & 3)];
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (r[u] >= rows) continue;
    // exact in BF16 down to its subnormals; the smallest value is 2^-128
    const float s = __uint_as_float(e[u] << 23);
    uint32_t b[4], v[V];
    b[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u], s, 0));
    b[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u], s, 1));
    b[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u], s, 2));
    b[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u], s, 3));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if constexpr (BF16) v[j] = b[j];
      else v[j] = (j & 1) ? b[j >> 1] & 0xFFFF0000u : b[j >> 1] << 16;
    }
    char* d = static_cast<char*>(out) + (r[u] * cols + c[u]) * SZ;
    if (c[u] + 8 <= cols) {
      __builtin_memcpy(__builtin_assume_aligned(d, SZ), v, 8 * SZ);
      continue;
    }
    const int n = (int)(cols - c[u]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) {
        if constexpr (BF16)
          reinterpret_cast<uint16_t*>(d)[j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
        else
          reinterpret_cast<uint32_t*>(d)[j] = v[j];
      }
  }
}

template <bool BF16>
hipError_t quantize_any(const QuantArgs& p, hipStream_t stream) {
  const unsigned wx = (unsigned)((p.cols + 127) / 128);
  if (p.qt) {
    const dim3 grid(wx, (unsigned)((p.rows + 127) / 128));
    if (p.q)
      hipLaunchKernelGGL((quantize_mxfp4_tile_kernel<BF16, true>), grid, dim3(256), 0, stream, p);
    else
      hipLaunchKernelGGL((quantize_mxfp4_tile_kernel<BF16, false>), grid, dim3(256), 0, stream, p);
  } else {
    // four passes a workgroup once that still leaves each CU several
    const int64_t groups = (p.rows + 15) / 16;
    if (groups * wx >= 8192)
      hipLaunchKernelGGL((quantize_mxfp4_rows_kernel<BF16, 4>),
                         dim3(wx, (unsigned)((groups + 3) / 4)), dim3(256), 0, stream, p);
    else
      hipLaunchKernelGGL((quantize_mxfp4_rows_kernel<BF16, 1>), dim3(wx, (unsigned)groups),
                         dim3(256), 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_mxfp4(uint8_t* q, uint32_t* sf, uint8_t* qt, uint32_t* sft,
                                 const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ldx,
                                 hipStream_t stream) {
  const QuantArgs p{x, rows, cols, ldx, q, reinterpret_cast<uint8_t*>(sf), qt,
                    reinterpret_cast<uint8_t*>(sft)};
  return bf16 ? quantize_any<true>(p, stream) : quantize_any<false>(p, stream);
}

hipError_t launch_dequantize_mxfp4(void* out, bool bf16, const uint8_t* q, const uint32_t* sf,
                                   int64_t rows, int64_t cols, hipStream_t stream) {
  const int64_t n8 = (cols + 7) / 8, n = rows * n8;
  const uint8_t* s = reinterpret_cast<const uint8_t*>(sf);
  const dim3 grid((unsigned)((n + 1023) / 1024));
  if (bf16)
    hipLaunchKernelGGL(dequantize_mxfp4_kernel<true>, grid, dim3(256), 0, stream, out, q, s, rows,
                       cols, n8);
  else
    hipLaunchKernelGGL(dequantize_mxfp4_kernel<false>, grid, dim3(256), 0, stream, out, q, s, rows,
                       cols, n8);
  return hipGetLastError();
}

}  // namespace dg
