// Activations into the layout of the grouped products, and the experts' rows
// back to the tokens, gfx950.  row(t, j) is the layout's row of slot j of token
// t (-1: none).
//
//   dispatch          A[row(t, j)] = E4M3(v / s), s = amax(v) / 448 per 128
//                     columns, v = x[t] or the FP32 product w[t][j] x[t]
//   combine           y[t] = sum_j w[t][j] c[row(t, j)] (+ residual[t]), FP32
//                     sums in slot order, rounded to BF16 once
//   combine backward  dc = dispatch of w dy, dw[t][j] = dy[t] . c[row(t, j)]
// (the gradient of dispatch is combine without weights).
//
// All are bound by HBM.  A wave takes 512 columns, eight a lane, so a 128-column
// block is one row of 16 lanes; a token's values are read once and leave k
// times.
#include "dg_device.hpp"
#include "dg_internal.hpp"

namespace dg {
namespace {

constexpr int kCols = 512;  // columns of a wave

// Eight values from an element-aligned address as FP32.
__device__ __forceinline__ void load8(const void* x, bool bf16, int64_t at, float (&v)[8]) {
  if (bf16) {
    uint32_t u[4];
    __builtin_memcpy(u, __builtin_assume_aligned(static_cast<const uint16_t*>(x) + at, 2), 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
    __builtin_memcpy(v, __builtin_assume_aligned(static_cast<const float*>(x) + at, 4), 32);
  }
}

// Eight values of a lane's 128-column block (16 lanes): codes and scale.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float& scale) {
  const float4 a = make_float4(v[0], v[1], v[2], v[3]), b = make_float4(v[4], v[5], v[6], v[7]);
  const BlockScale s = block_scale(row16_max(abs_max4(abs_max4(0.0f, a), b)));
  scale = s.s;
  return make_uint2(encode4_block(a, s), encode4_block(b, s));
}

__device__ __forceinline__ int row_of(const int32_t* rows, int64_t at, int64_t M) {
  const int r = rows[at];
  return r < M ? r : -1;
}

// Workgroups 0 .. token_groups - 1: a wave a (token, 512 columns); the others: the
// rows that fill an expert's last block, 2048 columns each, with zeros.
__global__ void __launch_bounds__(256) dispatch_kernel(DispatchArgs p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (blockIdx.x >= p.token_groups) {
    const uint32_t i = blockIdx.x - p.token_groups, parts = (uint32_t)((p.H + 2047) / 2048);
    const int64_t r0 = (int64_t)(i / parts) * 128, c = (int64_t)(i % parts) * 2048 + threadIdx.x * 8;
    if (p.pairs[r0] < 0 || p.pairs[r0 + 127] >= 0 || c >= p.H) return;
    for (int r = 127; r > 0 && p.pairs[r0 + r] < 0; --r) {
      *reinterpret_cast<uint2*>(p.a + (r0 + r) * p.H + c) = make_uint2(0, 0);
      if ((threadIdx.x & 15) == 0) p.sa[c / 128 * p.M + r0 + r] = 0.0f;
    }
    return;
  }
  const uint32_t unit = blockIdx.x * 4 + wave, units = (uint32_t)((p.H + kCols - 1) / kCols);
  const int64_t t = unit / units, c = (int64_t)(unit % units) * kCols + lane * 8;
  if (t >= p.T || c >= p.H) return;
  float v[8];
  load8(p.x, p.bf16, t * p.ldx + c, v);
  float scale;
  uint2 q = encode8(v, scale);
  for (int j = 0; j < p.k; ++j) {
    const int row = row_of(p.rows, t * p.k + j, p.M);
    if (row < 0) continue;
    if (p.weights) {
      const float w = p.weights[t * p.k + j];
      float wv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) wv[i] = w * v[i];
      q = encode8(wv, scale);
    }
    *reinterpret_cast<uint2*>(p.a + (int64_t)row * p.H + c) = q;
    if ((lane & 15) == 0) p.sa[c / 128 * p.M + row] = scale;
  }
}

__global__ void __launch_bounds__(256) combine_kernel(CombineArgs p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t unit = blockIdx.x * 4 + wave, units = (uint32_t)((p.H + kCols - 1) / kCols);
  const int64_t t = unit / units, c = (int64_t)(unit % units) * kCols + lane * 8;
  if (t >= p.T || c >= p.H) return;
  float y[8] = {};
  for (int j = 0; j < p.k; ++j) {
    const int row = row_of(p.rows, t * p.k + j, p.M);
    if (row < 0) continue;
    const float w = p.weights ? p.weights[t * p.k + j] : 1.0f;
    float v[8];
    load8(p.c, true, (int64_t)row * p.H + c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(w, v[i], y[i]);
  }
  if (p.residual) {
    float v[8];
    load8(p.residual, true, t * p.H + c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += v[i];
  }
  *reinterpret_cast<uint4*>(p.y + t * p.H + c) =
      make_uint4(bf16x2_rne(y[0], y[1]), bf16x2_rne(y[2], y[3]), bf16x2_rne(y[4], y[5]),
                 bf16x2_rne(y[6], y[7]));
}

__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// One workgroup a token: its waves' partial sums meet in LDS, in wave order.
__global__ void __launch_bounds__(256) combine_dot_kernel(CombineArgs p) {
  __shared__ float s_sum[4][kMoeMaxSlots];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  for (int j = 0; j < p.k; ++j) {
    const int row = row_of(p.rows, t * p.k + j, p.M);
    float sum = 0.0f;
    if (row >= 0)
      for (int64_t c = threadIdx.x * 8; c < p.H; c += 2048) {
        float a[8], b[8];
        load8(p.dy, true, t * p.lddy + c, a);
        load8(p.c, true, (int64_t)row * p.H + c, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(a[i], b[i], sum);
      }
    sum = wave_add(sum);
    if (lane == 0) s_sum[wave][j] = sum;
  }
  __syncthreads();
  if (threadIdx.x < p.k) {
    const int j = threadIdx.x;
    p.dweights[t * p.k + j] = (s_sum[0][j] + s_sum[1][j]) + (s_sum[2][j] + s_sum[3][j]);
  }
}

}  // namespace

hipError_t launch_dispatch(DispatchArgs p, hipStream_t stream) {
  const int64_t units = (p.H + kCols - 1) / kCols;
  p.token_groups = (uint32_t)((p.T * units + 3) / 4);
  const int64_t fill = p.M / 128 * ((p.H + 2047) / 2048);
  hipLaunchKernelGGL(dispatch_kernel, dim3((unsigned)(p.token_groups + fill)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs& p, hipStream_t stream) {
  const int64_t units = (p.H + kCols - 1) / kCols;
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((p.T * units + 3) / 4)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_combine_dot(const CombineArgs& p, hipStream_t stream) {
  hipLaunchKernelGGL(combine_dot_kernel, dim3((unsigned)p.T), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dg
