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
// not touched.  All are bound by HBM.
#include "dg_device.hpp"
#include "dg_internal.hpp"

namespace dg {
namespace {

typedef float f2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float2 decode2(uint32_t codes, bool high) {
  const f2 v = high ? __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true)
                    : __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
  return make_float2(v.x, v.y);
}
__device__ __forceinline__ float4 decode4(uint32_t codes) {
  const float2 a = decode2(codes, false), b = decode2(codes, true);
  return make_float4(a.x, a.y, b.x, b.y);
}

// 1 real row, 0 a row that fills its block, -1 a row of a block without expert
__device__ __forceinline__ int kind_of(const int32_t* m_indices, int64_t r) {
  if (!m_indices || m_indices[r] >= 0) return 1;
  return m_indices[r & ~int64_t(127)] >= 0 ? 0 : -1;
}

__device__ __forceinline__ float max4(float m, const float* v) {
  return abs_max4(m, make_float4(v[0], v[1], v[2], v[3]));
}

// N values (a multiple of 4) of a block with scale s
template <int N>
__device__ __forceinline__ void encode(const float* v, const BlockScale& s, uint8_t* out) {
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    w[i] = encode4_block(make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]), s);
  __builtin_memcpy(__builtin_assume_aligned(out, N), w, N);
}
template <int N>
__device__ __forceinline__ float top_of(const float* v) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i += 4) m = max4(m, v + i);
  return m;
}

// A wave takes 512 hidden units of a row, eight a lane: a block of h is 16
// lanes, one of gate/up 8.  Four rows a workgroup.
__global__ void __launch_bounds__(256) swiglu_kernel(SwigluArgs p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t parts = (uint32_t)((p.I + 511) / 512);
  const int64_t r = (int64_t)(blockIdx.x / parts) * 4 + wave;
  const int64_t c = (int64_t)(blockIdx.x % parts) * 512 + lane * 8;
  if (r >= p.M || c >= p.I) return;
  const int kind = kind_of(p.m_indices, r);
  if (kind < 0) return;
  float gu[16] = {}, h[8] = {};
  if (kind > 0) {
    const uint4* s = reinterpret_cast<const uint4*>(p.gu + r * 2 * p.I + 2 * c);
    const uint4 a = s[0], b = s[1];
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      gu[2 * i] = __uint_as_float(u[i] << 16);
      gu[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      h[i] = silu_f(gu[2 * i]) * gu[2 * i + 1];
    }
  }
  const BlockScale s = block_scale(lane_group_max<16>(top_of<8>(h)));
  encode<8>(h, s, p.h + r * p.I + c);
  if ((lane & 15) == 0) p.sh[c / 128 * p.M + r] = s.s;
  if (p.kept) {
    const BlockScale g = block_scale(lane_group_max<8>(top_of<16>(gu)));
    encode<16>(gu, g, p.kept + r * 2 * p.I + 2 * c);
    if ((lane & 7) == 0) p.skept[2 * c / 128 * p.M + r] = g.s;
  }
}

__global__ void __launch_bounds__(256) swiglu_backward_kernel(SwigluArgs p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t parts = (uint32_t)((p.I + 511) / 512);
  const int64_t r = (int64_t)(blockIdx.x / parts) * 4 + wave;
  const int64_t c = (int64_t)(blockIdx.x % parts) * 512 + lane * 8;
  if (r >= p.M || c >= p.I) return;
  const int kind = kind_of(p.m_indices, r);
  if (kind < 0) return;
  float d[16] = {}, h[8] = {};
  if (kind > 0) {
    const uint4 codes = *reinterpret_cast<const uint4*>(p.kept + r * 2 * p.I + 2 * c);
    const float s = p.skept[2 * c / 128 * p.M + r];
    const uint4 b = *reinterpret_cast<const uint4*>(p.dh + r * p.I + c);
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w}, u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = decode4(w[i]);
      const float dh[2] = {__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u)};
      const float gate[2] = {v.x * s, v.z * s}, up[2] = {v.y * s, v.w * s};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float sig = 1.0f / (1.0f + expf(-gate[j])), a = gate[j] * sig;
        d[4 * i + 2 * j] = dh[j] * up[j] * (sig + a * (1.0f - sig));
        d[4 * i + 2 * j + 1] = dh[j] * a;
        h[2 * i + j] = a * up[j];
      }
    }
  }
  const BlockScale g = block_scale(lane_group_max<8>(top_of<16>(d)));
  encode<16>(d, g, p.dgu + r * 2 * p.I + 2 * c);
  if ((lane & 7) == 0) p.sdgu[2 * c / 128 * p.M + r] = g.s;
  if (p.h) {
    const BlockScale s = block_scale(lane_group_max<16>(top_of<8>(h)));
    encode<8>(h, s, p.h + r * p.I + c);
    if ((lane & 15) == 0) p.sh[c / 128 * p.M + r] = s.s;
  }
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
  float4 v[16];
  float4 top = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p.q + (r0 + 16 * rg + i) * p.C + c0 + 4 * cg);
    const float s = scales[i];
    v[i] = decode4(w);
    v[i].x *= s; v[i].y *= s; v[i].z *= s; v[i].w *= s;
    top.x = fmaxf(top.x, fabsf(v[i].x));
    top.y = fmaxf(top.y, fabsf(v[i].y));
    top.z = fmaxf(top.z, fabsf(v[i].z));
    top.w = fmaxf(top.w, fabsf(v[i].w));
  }
  if constexpr (COLUMN) {
    top.x = lane_group_max<8>(top.x);
    top.y = lane_group_max<8>(top.y);
    top.z = lane_group_max<8>(top.z);
    top.w = lane_group_max<8>(top.w);
  } else {
    float m = wave_max(abs_max4(0.0f, top));
    if ((t & 63) == 0) s_top[t >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
    top = make_float4(m, m, m, m);
  }
  const float tops[4] = {top.x, top.y, top.z, top.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const BlockScale s = block_scale(tops[j]);
    float col[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) col[i] = j == 0 ? v[i].x : j == 1 ? v[i].y : j == 2 ? v[i].z : v[i].w;
    encode<16>(col, s, p.qt + (c0 + 4 * cg + j) * p.M + r0 + 16 * rg);
    if constexpr (COLUMN) {
      if (rg == 0) p.st[rb * p.C + c0 + 4 * cg + j] = s.s;
    } else if (t == 0 && j == 0) {
      p.st[(int64_t)rb * across + cb] = s.s;
    }
  }
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& p, bool backward, hipStream_t stream) {
  const dim3 grid((unsigned)((p.I + 511) / 512 * ((p.M + 3) / 4)));
  if (backward) hipLaunchKernelGGL(swiglu_backward_kernel, grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(swiglu_kernel, grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_transpose_blocks(const TransposeArgs& p, bool column, hipStream_t stream) {
  const dim3 grid((unsigned)(p.C / 128 * (p.M / 128)));
  if (column) hipLaunchKernelGGL(transpose_blocks_kernel<true>, grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(transpose_blocks_kernel<false>, grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dg
