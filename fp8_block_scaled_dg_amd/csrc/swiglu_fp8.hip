// The activation between the grouped products in 8 bits, gfx950: E4M3 codes with
// one FP32 scale per 128 columns of a row.
//
//   forward   h = silu(g) u -> codes for the next product, and (optional) the
//             checkpoint: g and u themselves in codes, in place of their BF16
//   backward  from the checkpoint's values and dh, sig = 1 / (1 + e^-g):
//             dg = dh u sig (1 + g (1 - sig)), du = dh g sig -> codes, and
//             (optional) h again for the weight gradient
//   transpose codes and scales of rows -> those of the transposed matrix with
//             scales over 128 rows: the operands of the weight gradients
//
// g and u of hidden unit i are columns 2i and 2i + 1.  Rows that only fill an
// expert's last 128-row block are written as zeros, blocks without an expert are
// not touched.
//
// All are bound by HBM, the gradient with h again by its VALU as well.  MI355X (a copy
// moves 5.0 TB/s): h alone, 2048 rows of 11008 units 26 us (113 MB and 10 MB of fill);
// with the checkpoint 32768 rows of 1408 and 8 thousand to fill 66 us (366 MB, 5.5
// TB/s), the gradient with h again 76; turned operands 18 thousand rows of 2048 columns
// 15.8 (scales of columns, 75 MB).
#include "dg_device.hpp"
#include "dg_internal.hpp"
#include "fp8_rows.hpp"

namespace dg {
namespace {

typedef float f2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float2 decode2(uint32_t codes, bool high) {
  const f2 v = high ? __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true)
                    : __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
  return make_float2(v.x, v.y);
}
// 1 / (1 + e^-g) of N gates, off by four half steps at most.
//   e^-g : 2^n 2^f, n the integer next to -g log2 e and |f| <= 1/2 what is left of the
//          product, rounded once; v_exp_f32 is off by one unit in the last place.
//          SHORT gates have 8 significant bits (BF16): their product with 15 bits of
//          log2 e is exact, so f takes two instructions, not five (the same f for all
//          of them)
//   1/d  : correctly rounded, d = 1 to 1 + e^87
// Gates beyond 87 in magnitude (rare, a branch of its own) go through the library's
// e^a; below -87 the sigmoid is e^g (1 + e^g is 1 in FP32 from -17 down), where e^-g
// would overflow and its reciprocal leave the normal range.
// With v_exp_f32 of -g log2 e rounded once and v_rcp_f32 alone the sigmoid is off by
// (|g| + 2) half steps, and subnormal ones are lost; that took 0.7 to 1.7 us less in the
// forward (of 48 and 66), 7 to 9 in the gradient (of 63 and 76; 32768 rows of 1408).
template <bool SHORT, int N>
__device__ __forceinline__ void sigmoids(const float (&g)[N], float (&sig)[N]) {
#pragma clang fp contract(off)
  float top = fabsf(g[0]);
#pragma unroll
  for (int j = 1; j < N; ++j) top = fmaxf(top, fabsf(g[j]));
  constexpr float integer = 0x1.8p23f;  // added: the sum's low bits are the nearest integer
  constexpr float log2e = 0x1.715476p+0f, rest = 0x1.4ae0cp-26f;  // log2 e: their sum,
  constexpr float log2e15 = 0x1.7154p+0f, rest15 = 0x1.d94ae0p-18f;  // and theirs
  float e[N], m[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if constexpr (SHORT) {
      m[j] = __builtin_fmaf(g[j], -log2e, integer);
      e[j] = __builtin_fmaf(g[j], -rest15, __builtin_fmaf(g[j], -log2e15, integer - m[j]));
    } else {
      const float p = g[j] * -log2e;
      m[j] = p + integer;
      const float low = __builtin_fmaf(g[j], -rest, __builtin_fmaf(g[j], -log2e, -p));
      e[j] = (p - (m[j] - integer)) + low;
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j) e[j] = __builtin_amdgcn_exp2f(e[j]);
#pragma unroll
  for (int j = 0; j < N; ++j)
    e[j] = 1.0f + __uint_as_float(__float_as_uint(e[j]) + (__float_as_uint(m[j]) << 23));
#pragma unroll
  for (int j = 0; j < N; ++j) sig[j] = reciprocal_rn(e[j]);
  if (top > 87.0f) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (fabsf(g[j]) > 87.0f) sig[j] = g[j] < 0.0f ? expf(g[j]) : 1.0f;  // 1 + e^-87 is 1
  }
}

// A workgroup takes p.tile_rows rows by 512 hidden units, a wave a row at a time,
// eight units a lane: a block of h is 16 lanes, one of gate/up 8.  The scales of
// the tile are put together in LDS and leave in runs along the rows.
constexpr int kUnits = 512, kTileRows = 16;
struct ScaleTile {
  float h[kUnits / 128][kTileRows], g[kUnits / 64][kTileRows];
};

template <int KB>
__device__ __forceinline__ void store_scales(const float (&s)[KB][kTileRows], float* out, int64_t M,
                                             int64_t kbs, int64_t kb0, int64_t r0, int tile_rows) {
  for (int i = threadIdx.x; i < KB * tile_rows; i += 256) {
    const int kb = i / tile_rows, r = i % tile_rows;
    if (kb0 + kb < kbs && r0 + r < M) out[(kb0 + kb) * M + r0 + r] = s[kb][r];
  }
}

// What a lane reads of a row: 16 BF16 gate/up values, or 16 codes with their
// scale and 8 BF16 values of dh.
template <bool FORWARD>
struct RowInput {
  u4 a, b;
  float s;
  __device__ __forceinline__ void load(const SwigluArgs& p, int64_t r, int64_t c) {
    if constexpr (FORWARD) {
      const u4* x = reinterpret_cast<const u4*>(p.gu + r * 2 * p.I + 2 * c);
      a = __builtin_nontemporal_load(x);
      b = __builtin_nontemporal_load(x + 1);
    } else {
      a = __builtin_nontemporal_load(reinterpret_cast<const u4*>(p.kept + r * 2 * p.I + 2 * c));
      b = __builtin_nontemporal_load(reinterpret_cast<const u4*>(p.dh + r * p.I + c));
      s = p.skept[2 * c / 128 * p.M + r];
    }
  }
  // g: gate/up or their gradients, h: silu(gate) * up, every operation rounded by
  // itself: the bits that elementary FP32 operations in this order give
  __device__ __forceinline__ void compute(float (&g)[16], float (&h)[8]) const {
#pragma clang fp contract(off)
    float gate[8], sig[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (FORWARD) {
        const uint32_t u = j < 4 ? a[j & 3] : b[j & 3];
        g[2 * j] = __uint_as_float(u << 16);
        g[2 * j + 1] = __uint_as_float(u & 0xFFFF0000u);
      } else {
        const float2 v = decode2(a[j >> 1], j & 1);
        g[2 * j] = v.x * s;
        g[2 * j + 1] = v.y * s;
      }
      gate[j] = g[2 * j];
    }
    sigmoids<FORWARD>(gate, sig);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float up = g[2 * j + 1], x = gate[j] * sig[j];
      h[j] = x * up;
      if constexpr (!FORWARD) {
        const float dh = __uint_as_float(j & 1 ? b[j >> 1] & 0xFFFF0000u : b[j >> 1] << 16);
        g[2 * j] = dh * up * sig[j] * (1.0f + gate[j] * (1.0f - sig[j]));
        g[2 * j + 1] = dh * x;
      }
    }
  }
};

// FORWARD: h (and KEEP: the checkpoint) from gu; else dgu (and KEEP: h) from dh
// and the checkpoint.  A wave has the next row's values on their way while it
// works on a row.
template <bool FORWARD, bool KEEP>
__global__ void __launch_bounds__(256) swiglu_kernel(SwigluArgs p) {
  constexpr bool H = FORWARD || KEEP, G = !FORWARD || KEEP;
  __shared__ ScaleTile tile;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t parts = (uint32_t)((p.I + kUnits - 1) / kUnits), part = blockIdx.x % parts;
  const int64_t r0 = (int64_t)(blockIdx.x / parts) * p.tile_rows, c0 = (int64_t)part * kUnits + lane * 8;
  if (p.m_indices && p.m_indices[r0 & ~int64_t(127)] < 0) return;
  // lanes past the last column (whole blocks of 16) repeat a lane's work, unstored
  const bool inside = c0 < p.I;
  const int64_t c = inside ? c0 : p.I - 8;
  // this wave's rows are wave, wave + 4, ..; bit i: row r0 + i is real
  const int rows = (int)(p.M - r0 < p.tile_rows ? p.M - r0 : p.tile_rows);
  const uint64_t real = __ballot(lane < rows && (!p.m_indices || p.m_indices[r0 + lane] >= 0));
  uint8_t* const codes = FORWARD ? p.kept : p.dgu;
  RowInput<FORWARD> next;
  if (real >> wave & 1) next.load(p, r0 + wave, c);
  for (int i = wave; i < rows; i += 4) {
    const int64_t r = r0 + i;
    const RowInput<FORWARD> in = next;
    if (i + 4 < rows && (real >> (i + 4) & 1)) next.load(p, r + 4, c);
    uint32_t wh[2] = {0, 0}, wg[4] = {0, 0, 0, 0};
    float sh = 0.0f, sg = 0.0f;
    if (real >> i & 1) {  // the same in every lane
      float g[16], h[8];
      in.compute(g, h);
      if constexpr (H) {
        const RowScale b = row_scale(h, group_top<16>(top_of(h)));
        encode_values(h, b, wh);
        sh = b.scale;
      }
      if constexpr (G) {
        const RowScale b = row_scale(g, group_top<8>(top_of(g)));
        encode_values(g, b, wg);
        sg = b.scale;
      }
    }
    if constexpr (H) {
      if (inside) store_stream(p.h + r * p.I + c, wh);
      if ((lane & 15) == 0) tile.h[lane >> 4][i] = sh;
    }
    if constexpr (G) {
      if (inside) store_stream(codes + r * 2 * p.I + 2 * c, wg);
      if ((lane & 7) == 0) tile.g[lane >> 3][i] = sg;
    }
  }
  __syncthreads();
  if constexpr (H) store_scales(tile.h, p.sh, p.M, p.I / 128, part * 4, r0, p.tile_rows);
  if constexpr (G) store_scales(tile.g, FORWARD ? p.skept : p.sdgu, p.M, p.I / 64, part * 8, r0, p.tile_rows);
}

// A tile of 128 rows by 128 columns; thread: 4 columns by 16 rows, the eight
// threads of a column group next to each other, so that a column's codes leave
// in 128-byte pieces.
template <bool COLUMN>  // scales of single columns, else of the tile
__global__ void __launch_bounds__(256) transpose_blocks_kernel(TransposeArgs p) {
  __shared__ float s_top[4];
  const int t = threadIdx.x, rg = t & 7, cg = t >> 3;
  const uint32_t across = (uint32_t)(p.C / 128), rb = blockIdx.x / across, cb = blockIdx.x % across;
  const int64_t r0 = (int64_t)rb * 128, c0 = (int64_t)cb * 128;
  if (p.m_indices && p.m_indices[r0] < 0) return;
  const float* scales = p.s + cb * p.M + r0 + 16 * rg;
  float v[4][16], top[4];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p.q + (r0 + 16 * rg + i) * p.C + c0 + 4 * cg);
    const float s = scales[i];
    const float2 a = decode2(w, false), b = decode2(w, true);
    v[0][i] = a.x * s;
    v[1][i] = a.y * s;
    v[2][i] = b.x * s;
    v[3][i] = b.y * s;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) top[j] = group_top<8>(top_of(v[j]));
  if constexpr (!COLUMN) {
    float m = wave_max(join_top(join_top(top[0], top[1]), join_top(top[2], top[3])));
    if ((t & 63) == 0) s_top[t >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
#pragma unroll
    for (int j = 0; j < 4; ++j) top[j] = m;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const RowScale b = row_scale(v[j], top[j]);
    uint32_t w[4];
    encode_values(v[j], b, w);
    store_stream(p.qt + (c0 + 4 * cg + j) * p.M + r0 + 16 * rg, w);
    if constexpr (COLUMN) {
      if (rg == 0) p.st[rb * p.C + c0 + 4 * cg + j] = b.scale;
    } else if (t == 0 && j == 0) {
      p.st[(int64_t)rb * across + cb] = b.scale;
    }
  }
}

}  // namespace

hipError_t launch_swiglu(SwigluArgs p, bool backward, hipStream_t stream) {
  const int64_t parts = (p.I + kUnits - 1) / kUnits;
  // Rows a workgroup.  Four (a row a wave) where eight would leave fewer than 600
  // workgroups, two and a bit a CU: h of 512 rows of 4096 units (512 workgroups of 8 rows)
  // 4.5 us, so 4.9 with eight; 256 of 11008 (704) 5.9, so 5.6.  Eight from there on:
  // 32768 rows of 1408 with the checkpoint 60 us, 64 with four, 63 with sixteen.  Sixteen
  // for the gradient from 4096 workgroups on, for longer runs of scales: with h again 70
  // us, so 72 with eight (2048 of 11008, 2816 workgroups: 34.6 and 34.8); with
  // thirty-two no less.
  const auto groups = [&] { return (p.M + p.tile_rows - 1) / p.tile_rows * parts; };
  p.tile_rows = kTileRows;
  if (!backward || groups() < 4096) p.tile_rows = 8;
  if (p.tile_rows == 8 && groups() < 600) p.tile_rows = 4;
  const dim3 grid((unsigned)groups()), block(256);
  if (!backward && !p.kept) hipLaunchKernelGGL((swiglu_kernel<true, false>), grid, block, 0, stream, p);
  else if (!backward) hipLaunchKernelGGL((swiglu_kernel<true, true>), grid, block, 0, stream, p);
  else if (!p.h) hipLaunchKernelGGL((swiglu_kernel<false, false>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((swiglu_kernel<false, true>), grid, block, 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_transpose_blocks(const TransposeArgs& p, bool column, hipStream_t stream) {
  const dim3 grid((unsigned)(p.C / 128 * (p.M / 128)));
  if (column) hipLaunchKernelGGL(transpose_blocks_kernel<true>, grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(transpose_blocks_kernel<false>, grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dg
