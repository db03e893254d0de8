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
// times.  MI355X, BF16, tokens x columns to k of E experts (a copy moves 5.0 TB/s,
// stores alone to scattered rows 5.1):
//   dispatch 8192 x 7168, 8 of 256      145 us  720 MB, of it 117 MB of zeros
//                                               that fill the experts' blocks;
//                                               times the weights 147
//            4001 x 2048, 4 of 60      12.8 us  times the weights 13.7
//            64 x 7168, 8 of 256         45 us  nearly all of it the zeros (236 MB)
//   combine  8192 x 7168, 8 of 256      184 us  1058 MB, 5.7 TB/s
//            4001 x 2048, 4 of 60      15.0 us
//   its gradient, 4001 x 2048, 4 of 60 22.8 us  113 MB (25.8 in two launches, dy
//                                               read twice)
// One token of 4096 columns takes 4.5 us, 64 tokens' combine 3: a launch and its
// chain of loads (the slots' rows, then what they say).
#include "dg_device.hpp"
#include "dg_internal.hpp"
#include "fp8_rows.hpp"

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

// The slots of token t, one a lane: row in the layout (-1: none) and weight.
// Read at once; slot j is then a lane of a register.
struct Slots {
  int row;
  float weight;
  __device__ __forceinline__ Slots(const int32_t* rows, const float* weights, int64_t t, int k,
                                   int64_t M, int lane) {
    const bool ok = lane < k;
    row = ok ? rows[t * k + lane] : -1;
    weight = ok && weights ? weights[t * k + lane] : 1.0f;
    if (row >= M) row = -1;
  }
  __device__ __forceinline__ int row_of(int j) const { return __builtin_amdgcn_readlane(row, j); }
  __device__ __forceinline__ float weight_of(int j) const {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), j));
  }
};

// f(IntTag<K>) for the smallest K = 1, 2, 4, 8, 16 that is not below k.
template <int K = 1, class F>
__device__ __host__ __forceinline__ void with_slots(int k, F&& f) {
  if constexpr (K == kMoeMaxSlots) {
    f(IntTag<K>{});
  } else {
    if (k <= K) f(IntTag<K>{});
    else with_slots<2 * K>(k, f);
  }
}

// The rows of the 32 from r0 on that no pair has, one bit each; 0 in a 128-row
// block without an expert.
__device__ __forceinline__ uint32_t rows_to_fill(const DispatchArgs& p, int64_t r0) {
  const int lane = threadIdx.x & 63;
  if (p.pairs[r0 & ~int64_t(127)] < 0) return 0;
  return (uint32_t)__ballot(lane < 32 && p.pairs[r0 + (lane & 31)] < 0);
}

// Zero codes for these rows, columns c .. c + 15 of this thread.
__device__ __forceinline__ void fill_rows(const DispatchArgs& p, int64_t r0, uint32_t fill, int64_t c) {
  const uint32_t none[4] = {0, 0, 0, 0};
  for (; fill; fill &= fill - 1) store_stream(p.a + (r0 + __builtin_ctz(fill)) * p.H + c, none);
}

// Part i of the fill: 32 rows by 4096 columns, with their scales.
__device__ __forceinline__ void fill_block(const DispatchArgs& p, uint32_t i) {
  const uint32_t parts = (uint32_t)((p.H + 4095) / 4096);
  const int64_t r0 = (int64_t)(i / parts) * 32, c = (int64_t)(i % parts) * 4096 + threadIdx.x * 16;
  uint32_t fill = rows_to_fill(p, r0);
  if (c >= p.H) return;
  fill_rows(p, r0, fill, c);
  if ((threadIdx.x & 7) == 0)
    for (; fill; fill &= fill - 1) p.sa[c / 128 * p.M + r0 + __builtin_ctz(fill)] = 0.0f;
}

// One slot of a token whose values go out with its weight: columns c .. c + 7 to row
// `row`, a parked scale to place `pair`; top: the largest magnitude of the block of v.
template <bool PARKED>
__device__ __forceinline__ void put_weighted(const DispatchArgs& p, const float (&v)[8], float top,
                                             float w, int64_t pair, int64_t row, int64_t c, int lane) {
  float wv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) wv[i] = w * v[i];
  // rounding is monotone: the largest product is that of the largest value
  const RowScale b = row_scale(wv, fabsf(w) * top);
  uint32_t q[2];
  encode_values(wv, b, q);
  store_stream(p.a + row * p.H + c, q);
  if ((lane & 15) != 0) return;
  if (PARKED) p.parked[pair * (p.H / 128) + c / 128] = b.scale;
  else p.sa[c / 128 * p.M + row] = b.scale;
}

// A wave a (token, 512 columns).  PARKED: the scales go to the workspace, token by
// token ([T][H/128], WEIGHTED [T k][H/128]), and dispatch_scales_kernel takes them
// from there; else each goes to its place, and workgroups from token_groups on fill
// the ends of the experts' last blocks.
template <bool WEIGHTED, bool PARKED>
__global__ void __launch_bounds__(256) dispatch_kernel(DispatchArgs p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (!PARKED && blockIdx.x >= p.token_groups) {
    fill_block(p, blockIdx.x - p.token_groups);
    return;
  }
  const uint32_t unit = blockIdx.x * 4 + wave, units = (uint32_t)((p.H + kCols - 1) / kCols);
  const int64_t t = unit / units, c = (int64_t)(unit % units) * kCols + lane * 8;
  if (t >= p.T) return;
  const Slots slots(p.rows, p.weights, t, p.k, p.M, lane);
  if (c >= p.H) return;  // whole blocks of 16 lanes: the first k, with the slots, stay
  float v[8];
  load8(p.x, p.bf16, t * p.ldx + c, v);
  const float top = group_top<16>(top_of(v));
  if constexpr (WEIGHTED) {
    for (int j = 0; j < p.k; ++j)
      if (slots.row_of(j) >= 0)
        put_weighted<PARKED>(p, v, top, slots.weight_of(j), t * p.k + j, slots.row_of(j), c, lane);
  } else {
    const RowScale b = row_scale(v, top);
    uint32_t q[2];
    encode_values(v, b, q);
    const bool leader = (lane & 15) == 0;
    if (PARKED && leader) p.parked[t * (p.H / 128) + c / 128] = b.scale;
    for (int j = 0; j < p.k; ++j) {
      const int row = slots.row_of(j);
      if (row < 0) continue;
      store_stream(p.a + (int64_t)row * p.H + c, q);
      if (!PARKED && leader) p.sa[c / 128 * p.M + row] = b.scale;
    }
  }
}

// Parked scales to their places, 32 rows by 64 blocks of columns a workgroup
// through LDS (runs of 128 bytes both ways), and zeros where a row only fills its
// block.
template <bool WEIGHTED>
__global__ void __launch_bounds__(256) dispatch_scales_kernel(DispatchArgs p) {
  __shared__ float s_scale[32][65];
  __shared__ int s_from[32];
  const int t = threadIdx.x, lane = t & 63;
  const int64_t kbs = p.H / 128;
  const uint32_t parts = (uint32_t)((kbs + 63) / 64);
  const int64_t r0 = (int64_t)(blockIdx.x / parts) * 32, kb0 = (int64_t)(blockIdx.x % parts) * 64;
  if (p.pairs[r0 & ~int64_t(127)] < 0) return;
  const int n = (int)(kbs - kb0 < 64 ? kbs - kb0 : 64);
  const uint32_t fill = rows_to_fill(p, r0);
  if (t < 32) {
    const int pair = p.pairs[r0 + t];
    s_from[t] = pair < 0 || pair >= p.T * p.k ? -1 : WEIGHTED ? pair : pair / p.k;
  }
  __syncthreads();
#pragma unroll
  for (int r = t >> 6; r < 32; r += 4)
    s_scale[r][lane] = s_from[r] >= 0 && lane < n ? p.parked[(int64_t)s_from[r] * kbs + kb0 + lane] : 0.0f;
  for (int64_t c = kb0 * 128 + t * 16; c < (kb0 + n) * 128; c += 4096) fill_rows(p, r0, fill, c);
  __syncthreads();
#pragma unroll
  for (int kb = t >> 5; kb < 64; kb += 8)
    if (kb < n) p.sa[(kb0 + kb) * p.M + r0 + (t & 31)] = s_scale[t & 31][kb];
}

// All slots' rows are asked for before the first is added.
template <int K>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t unit = blockIdx.x * 4 + wave, units = (uint32_t)((p.H + kCols - 1) / kCols);
  const int64_t t = unit / units, c0 = (int64_t)(unit % units) * kCols + lane * 8;
  if (t >= p.T) return;
  // the first k lanes hold the slots, so all stay; past the end they repeat the
  // last columns, unstored
  const int64_t c = c0 < p.H ? c0 : p.H - 8;
  const Slots slots(p.rows, p.weights, t, p.k, p.M, lane);
  u4 v[K], res = {};
  if (p.residual) res = *reinterpret_cast<const u4*>(p.residual + t * p.H + c);
#pragma unroll
  for (int j = 0; j < K; ++j)
    if (slots.row_of(j) >= 0)
      v[j] = __builtin_nontemporal_load(
          reinterpret_cast<const u4*>(p.c + (int64_t)slots.row_of(j) * p.H + c));
  float y[8] = {};
#pragma unroll
  for (int j = 0; j < K; ++j)
    if (slots.row_of(j) >= 0) {
      const float w = slots.weight_of(j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = fmaf(w, __uint_as_float(v[j][i] << 16), y[2 * i]);
        y[2 * i + 1] = fmaf(w, __uint_as_float(v[j][i] & 0xFFFF0000u), y[2 * i + 1]);
      }
    }
  u4 out;
#pragma unroll
  for (int i = 0; i < 4; ++i)  // without a residual the sum keeps the sign of a zero
    out[i] = p.residual ? bf16x2_rne(y[2 * i] + __uint_as_float(res[i] << 16),
                                     y[2 * i + 1] + __uint_as_float(res[i] & 0xFFFF0000u))
                        : bf16x2_rne(y[2 * i], y[2 * i + 1]);
  if (c0 < p.H) __builtin_nontemporal_store(out, reinterpret_cast<u4*>(p.y + t * p.H + c));
}

__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Gradient of the weights, one workgroup a token: its waves' partial sums meet in
// LDS, in wave order.  DC other than none: with each row of c read, the row's
// gradient (the dispatch of w dy) written, so that dy is read once for both.
enum { DC_NONE, DC_DIRECT, DC_PARKED };
template <int K, int DC>
__global__ void __launch_bounds__(256) combine_backward_kernel(CombineArgs p, DispatchArgs d) {
  __shared__ float s_sum[4][kMoeMaxSlots];
  if (DC == DC_DIRECT && blockIdx.x >= p.T) {
    fill_block(d, blockIdx.x - (uint32_t)p.T);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  const Slots slots(p.rows, d.weights, t, p.k, p.M, lane);
  float sum[K] = {};
  for (int64_t c = threadIdx.x * 8; c < p.H; c += 2048) {  // lanes leave by blocks of 16
    u4 v[K];
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (slots.row_of(j) >= 0)
        v[j] = __builtin_nontemporal_load(
            reinterpret_cast<const u4*>(p.c + (int64_t)slots.row_of(j) * p.H + c));
    float dy[8];
    load8(p.dy, true, t * p.lddy + c, dy);
    const float top = DC != DC_NONE ? group_top<16>(top_of(dy)) : 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (slots.row_of(j) >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[j] = fmaf(dy[2 * i], __uint_as_float(v[j][i] << 16), sum[j]);
          sum[j] = fmaf(dy[2 * i + 1], __uint_as_float(v[j][i] & 0xFFFF0000u), sum[j]);
        }
        if constexpr (DC != DC_NONE)
          put_weighted<DC == DC_PARKED>(d, dy, top, slots.weight_of(j), d.weights ? t * p.k + j : t,
                                       slots.row_of(j), c, lane);
      }
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const float s = wave_add(sum[j]);
    if (lane == 0) s_sum[wave][j] = s;
  }
  __syncthreads();
  if (threadIdx.x < p.k) {
    const int j = threadIdx.x;
    p.dweights[t * p.k + j] = (s_sum[0][j] + s_sum[1][j]) + (s_sum[2][j] + s_sum[3][j]);
  }
}

}  // namespace

// A scale stored by itself is one request to the L2, and with hundreds of experts, whose
// rows grow at the same time, no line of scales fills up there before it leaves.  Few
// experts fill their lines, and the second launch costs more than it saves.  us without
// and with the workspace, in the order of the scales' number:
//   8 of 256, 7168 columns   0.9 million  61, 51   1.1  67, 56   1.3  70, 59   1.8  81, 75
//                            2.2  114, 110         3.7  170, 143
//   8 of 128, 4096           1.0  38.6, 38.3       2.1  65.6, 65.7
//   4 of 60, 2048            0.26 13.0, 15.1  0.5  21.8, 23.1  1.0  39.4, 40.2  2.1  88.4, 87.8
//   6 of 64, 2048            1.6  51.2, 52.0       3.1  122, 114
//   2 of 8, 4096             1.0  52.8, 56.7       2.1  99, 105      4.2  194, 200
//   1 of 8, 8192             1.0  77, 87           2.1  144, 166
// (weighted, the scales of a token k times, 1 to 5 us more with the workspace).  The rule
// knows the scales' number alone: from 2^20 on.
size_t dispatch_workspace_bytes(int64_t T, int k, int64_t H, bool weighted) {
  if (T * k < (int64_t(1) << 20) / (H / 128)) return 0;
  return (size_t)(weighted ? T * k : T) * (H / 128) * sizeof(float);
}

namespace {

int64_t fill_blocks(const DispatchArgs& p) { return p.M / 32 * ((p.H + 4095) / 4096); }

hipError_t launch_scales(const DispatchArgs& p, hipStream_t stream) {
  const dim3 rows((unsigned)(p.M / 32 * ((p.H / 128 + 63) / 64)));
  if (p.weights) hipLaunchKernelGGL(dispatch_scales_kernel<true>, rows, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(dispatch_scales_kernel<false>, rows, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dispatch(DispatchArgs p, void* workspace, hipStream_t stream) {
  const int64_t units = (p.H + kCols - 1) / kCols;
  p.token_groups = (uint32_t)((p.T * units + 3) / 4);
  p.parked = static_cast<float*>(workspace);
  const dim3 grid((unsigned)(p.token_groups + (workspace ? 0 : fill_blocks(p)))), block(256);
  if (!workspace) {
    if (p.weights) hipLaunchKernelGGL((dispatch_kernel<true, false>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((dispatch_kernel<false, false>), grid, block, 0, stream, p);
    return hipGetLastError();
  }
  if (p.weights) hipLaunchKernelGGL((dispatch_kernel<true, true>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((dispatch_kernel<false, true>), grid, block, 0, stream, p);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? launch_scales(p, stream) : e;
}

hipError_t launch_combine(const CombineArgs& p, hipStream_t stream) {
  const int64_t units = (p.H + kCols - 1) / kCols;
  const dim3 grid((unsigned)((p.T * units + 3) / 4));
  with_slots(p.k, [&](auto K) {
    hipLaunchKernelGGL(combine_kernel<decltype(K)::value>, grid, dim3(256), 0, stream, p);
  });
  return hipGetLastError();
}

hipError_t launch_combine_backward(const CombineArgs& p, DispatchArgs d, void* workspace,
                                   hipStream_t stream) {
  d.parked = static_cast<float*>(workspace);
  const int mode = !d.a ? DC_NONE : workspace ? DC_PARKED : DC_DIRECT;
  const dim3 grid((unsigned)(p.T + (mode == DC_DIRECT ? fill_blocks(d) : 0))), block(256);
  with_slots(p.k, [&](auto K) {
    constexpr int k = decltype(K)::value;
    if (mode == DC_NONE) hipLaunchKernelGGL((combine_backward_kernel<k, DC_NONE>), grid, block, 0, stream, p, d);
    else if (mode == DC_DIRECT) hipLaunchKernelGGL((combine_backward_kernel<k, DC_DIRECT>), grid, block, 0, stream, p, d);
    else hipLaunchKernelGGL((combine_backward_kernel<k, DC_PARKED>), grid, block, 0, stream, p, d);
  });
  const hipError_t e = hipGetLastError();
  return e == hipSuccess && mode == DC_PARKED ? launch_scales(d, stream) : e;
}

}  // namespace dg
