// Routing to experts, gfx950: ids, weights of the k experts of each token, and
// the gradient of the logits.
//
//   s   = softmax(l) or 1 / (1 + e^-l)          over the token's E logits
//   c   = s + bias (in 64 bits), or without a bias the order of l itself
//   groups of E / G consecutive experts: a group's value is the sum of its
//         `best` (1 or 2) largest c; the top_groups largest values stay
//   ids = the k largest c of the groups that stay, ties to the lowest index
//   w   = scale s, divided by the sum of the chosen s if renormalised
//
// A logit of -inf or NaN, or a bias of -inf or NaN, is an expert that is never
// chosen; slots left over get id -1 and weight 0.
//
// Gradient of L with g = dL/dw, q = s / (sum of the chosen s), gm = sum g q:
//   renormalised      softmax dl_j = scale q_j (g_j - gm)
//                     sigmoid dl_j = scale q_j (g_j - gm) (1 - s_j)
//   not renormalised  softmax dl_e = scale s_e (g_e [e chosen] - sum s_j g_j)
//                     sigmoid dl_j = scale g_j s_j (1 - s_j)
// The choice itself, and so the bias, has no gradient.
//
// One wave per token, PER consecutive experts a lane.
#include "dg_device.hpp"
#include "dg_internal.hpp"

namespace dg {
namespace {

constexpr int kRouteWaves = 4;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(u >> 32), CTRL, 0xF, 0xF, false);
  return __longlong_as_double((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float lane_of(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t u = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane);
  return __longlong_as_double((uint64_t)hi << 32 | lo);
}

// f over the wave's values, in every lane: within 16 lanes by DPP (swap
// neighbours, swap pairs, rotate by 4, by 8), then the four rows' results.
template <class T, class F>
__device__ __forceinline__ T wave_join(T v, F&& f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x124>(v));
  v = f(v, dpp<0x128>(v));
  return f(f(lane_of(v, 0), lane_of(v, 16)), f(lane_of(v, 32), lane_of(v, 48)));
}
template <class T>
__device__ __forceinline__ T wave_top(T v) {  // no NaN among them
  return wave_join(v, [](T a, T b) { return a > b ? a : b; });
}
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
  return wave_join(v, [](T a, T b) { return a + b; });
}

// Experts lane * PER .. + PER - 1 of a token's logits as FP32, -inf where there
// is none; a row starts at any element.
template <int PER>
__device__ __forceinline__ void load_logits(const void* logits, bool bf16, int64_t at, int E,
                                            int lane, float (&v)[PER]) {
  const int e0 = lane * PER;
#pragma unroll
  for (int q = 0; q < PER; ++q) v[q] = -INFINITY;
  if (e0 >= E) return;
  if (bf16) {
    const uint16_t* s = static_cast<const uint16_t*>(logits) + at + e0;
    uint16_t u[PER];
    if (e0 + PER <= E) {
      __builtin_memcpy(u, __builtin_assume_aligned(s, 2), sizeof u);
#pragma unroll
      for (int q = 0; q < PER; ++q) v[q] = bf16_bits_to_f32(u[q]);
    } else {
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (e0 + q < E) v[q] = bf16_bits_to_f32(s[q]);
    }
  } else {
    const float* s = static_cast<const float*>(logits) + at + e0;
    if (e0 + PER <= E) {
      __builtin_memcpy(v, __builtin_assume_aligned(s, 4), sizeof v);
    } else {
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (e0 + q < E) v[q] = s[q];
    }
  }
}

__device__ __forceinline__ float load_logit(const RouteArgs& p, int64_t at) {
  return p.bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(p.logits)[at])
                : static_cast<const float*>(p.logits)[at];
}

// sig(v) / sig(m) or e^(v - m), formed without overflow or underflow of either:
// sig(v) = e^min(v,0) / (1 + e^-|v|).
__device__ __forceinline__ float relative_score(float v, float m, int scoring) {
  if (scoring == ROUTE_SOFTMAX) return expf(v - m);
  return expf(fminf(v, 0.0f) - fminf(m, 0.0f)) * ((1.0f + expf(-fabsf(m))) / (1.0f + expf(-fabsf(v))));
}

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// Scores in 64 bits: the softmax of the lanes' logits v (largest m) or their
// sigmoid; 0 for v = -inf.
template <int PER>
__device__ __forceinline__ void wide_scores(const float (&v)[PER], float m, int scoring,
                                            double (&c)[PER]) {
  double sum = 0.0;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    if (scoring == ROUTE_SOFTMAX) {
      c[q] = v[q] == m ? 1.0 : exp((double)v[q] - (double)m);
      if (v[q] == -INFINITY) c[q] = 0.0;
      sum += c[q];
    } else {
      c[q] = 1.0 / (1.0 + exp(-(double)v[q]));
    }
  }
  if (scoring == ROUTE_SOFTMAX) {
    sum = wave_sum(sum);
#pragma unroll
    for (int q = 0; q < PER; ++q) c[q] /= sum;
  }
}

template <int PER, bool BIASED, bool GROUPED>
__global__ void __launch_bounds__(64 * kRouteWaves) route_kernel(RouteArgs p) {
  using Key = std::conditional_t<BIASED, double, float>;
  __shared__ double s_value[GROUPED ? kRouteWaves : 1][GROUPED ? 64 * PER : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t >= p.T) return;
  float v[PER];
  load_logits<PER>(p.logits, p.bf16, t * p.ldl, p.E, lane, v);
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    if (v[q] != v[q]) v[q] = -INFINITY;
    m = fmaxf(m, v[q]);
  }
  m = wave_top(m);
  Key key[PER];
  double c[PER];
  if (BIASED || (GROUPED && p.best == 2)) wide_scores<PER>(v, m, p.scoring, c);
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int e = lane * PER + q;
    bool off = v[q] == -INFINITY;
    if constexpr (BIASED) {
      const float b = e < p.E ? p.bias[e] : -INFINITY;
      off = off || !(b > -INFINITY);
      key[q] = off ? (Key)-INFINITY : (Key)(c[q] + (double)b);
    } else {
      key[q] = v[q];
    }
  }
  if constexpr (GROUPED) {
    double* value = s_value[wave];
#pragma unroll
    for (int q = 0; q < PER; ++q)
      value[lane * PER + q] = BIASED || p.best == 1 || key[q] == (Key)-INFINITY ? (double)key[q] : c[q];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    // p.lanes (a power of two) lanes a group
    const int per = p.E / p.groups, g = lane / p.lanes;
    double a = -INFINITY, b = -INFINITY;  // the two largest, a >= b
    if (g < p.groups)
      for (int i = lane % p.lanes; i < per; i += p.lanes) {
        const double x = value[g * per + i];
        if (x > a) {
          b = a;
          a = x;
        } else if (x > b) {
          b = x;
        }
      }
    for (int d = 1; d < p.lanes; d *= 2) {
      const double oa = __shfl_xor(a, d, 64), ob = __shfl_xor(b, d, 64);
      const double lo = oa > a ? a : oa;  // of the two largest the smaller
      a = oa > a ? oa : a;
      b = ob > b ? ob : b;
      b = lo > b ? lo : b;
    }
    if (p.best == 2 && b > -INFINITY) a += b;
    // groups ahead of this one: larger, or equal and before it
    int ahead = 0;
    for (int i = 0; i < p.groups; ++i) {
      const double o = lane_of(a, i * p.lanes);
      ahead += o > a || (o == a && i < g);
    }
    const uint64_t stays = __ballot(g < p.groups && ahead < p.top_groups);
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = lane * PER + q;
      if (e < p.E && !(stays >> (e / per * p.lanes) & 1)) key[q] = (Key)-INFINITY;
    }
  }
  int my_id = -1;
  for (int j = 0; j < p.k; ++j) {
    Key b = key[0];
    int bi = 0;
#pragma unroll
    for (int q = 1; q < PER; ++q)
      if (key[q] > b) {
        b = key[q];
        bi = q;
      }
    const Key top = wave_top(b);
    if (top == (Key)-INFINITY) break;  // the same in every lane
    const int owner = __ffsll((unsigned long long)__ballot(b == top)) - 1;
    const int id = owner * PER + __builtin_amdgcn_readlane(bi, owner);
    if (lane == j) my_id = id;
#pragma unroll
    for (int q = 0; q < PER; ++q)
      if (id == lane * PER + q) key[q] = (Key)-INFINITY;
  }
  // weights: lane j has slot j
  const float l = my_id >= 0 ? load_logit(p, t * p.ldl + my_id) : -INFINITY;
  float w = 0.0f;
  if (p.renormalise) {
    const float top = wave_top(l);
    const float r = my_id >= 0 ? relative_score(l, top, p.scoring) : 0.0f;
    w = p.scale * r / wave_sum(r);
  } else if (p.scoring == ROUTE_SOFTMAX) {
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < PER; ++q) sum += expf(v[q] - m);
    w = p.scale * expf(l - m) / wave_sum(sum);
  } else {
    w = p.scale * sigmoid(l);
  }
  if (p.scoring == ROUTE_SOFTMAX && m == INFINITY) w = NAN;
  if (lane < p.k) {
    p.ids[t * p.k + lane] = my_id;
    p.weights[t * p.k + lane] = my_id >= 0 ? w : 0.0f;
  }
}

template <int PER>
__global__ void __launch_bounds__(64 * kRouteWaves) route_backward_kernel(RouteArgs p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t >= p.T) return;
  float v[PER];
  load_logits<PER>(p.logits, p.bf16, t * p.ldl, p.E, lane, v);
#pragma unroll
  for (int q = 0; q < PER; ++q)
    if (v[q] != v[q]) v[q] = -INFINITY;
  // lane j has slot j; a slot without an expert, or one of an expert that
  // cannot be chosen, gives and gets nothing
  int id = lane < p.k ? p.ids[t * p.k + lane] : -1;
  if (id >= p.E) id = -1;
  float l = id >= 0 ? load_logit(p, t * p.ldl + id) : -INFINITY;
  if (!(l > -INFINITY)) id = -1, l = -INFINITY;
  const float g = id >= 0 ? p.scale * p.dweights[t * p.k + lane] : 0.0f;
  // slot: what is added to the logit of the slot's expert; all: what is
  // subtracted from every logit, times its score
  float slot = 0.0f, all = 0.0f, m = 0.0f, inverse = 0.0f;
  if (p.renormalise) {
    const float top = wave_top(l);
    const float r = id >= 0 ? relative_score(l, top, p.scoring) : 0.0f;
    const float sum = wave_sum(r);
    const float q = sum > 0.0f ? r / sum : 0.0f;
    slot = q * (g - wave_sum(g * q));
    if (p.scoring == ROUTE_SIGMOID) slot *= sigmoid(-l);
  } else if (p.scoring == ROUTE_SOFTMAX) {
    m = -INFINITY;
#pragma unroll
    for (int q = 0; q < PER; ++q) m = fmaxf(m, v[q]);
    m = wave_top(m);
    float sum = 0.0f;
    if (m > -INFINITY) {
#pragma unroll
      for (int q = 0; q < PER; ++q) sum += expf(v[q] - m);
    }
    sum = wave_sum(sum);
    inverse = sum > 0.0f ? 1.0f / sum : 0.0f;
    slot = id >= 0 ? g * expf(l - m) * inverse : 0.0f;
    all = wave_sum(slot);
  } else {
    slot = g * sigmoid(l) * sigmoid(-l);
  }
  if (id < 0) slot = 0.0f;
  float d[PER];
#pragma unroll
  for (int q = 0; q < PER; ++q) d[q] = all != 0.0f && v[q] > -INFINITY ? -all * (expf(v[q] - m) * inverse) : 0.0f;
  for (int j = 0; j < p.k; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const float s = lane_of(slot, j);
#pragma unroll
    for (int q = 0; q < PER; ++q)
      if (e == lane * PER + q) d[q] += s;
  }
  const int e0 = lane * PER;
  if (e0 >= p.E) return;
  if (p.bf16) {
    uint16_t* o = static_cast<uint16_t*>(p.dlogits) + t * p.ldd + e0;
    uint16_t u[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) u[q] = (uint16_t)bf16x2_rne(d[q], 0.0f);
    if (e0 + PER <= p.E) {
      __builtin_memcpy(__builtin_assume_aligned(o, 2), u, sizeof u);
    } else {
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (e0 + q < p.E) o[q] = u[q];
    }
  } else {
    float* o = static_cast<float*>(p.dlogits) + t * p.ldd + e0;
    if (e0 + PER <= p.E) {
      __builtin_memcpy(__builtin_assume_aligned(o, 4), d, sizeof d);
    } else {
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (e0 + q < p.E) o[q] = d[q];
    }
  }
}

template <int PER>
void launch_per(const RouteArgs& p, bool backward, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
  if (backward) {
    hipLaunchKernelGGL(route_backward_kernel<PER>, grid, block, 0, stream, p);
  } else if (p.top_groups < p.groups) {
    if (p.bias) hipLaunchKernelGGL((route_kernel<PER, true, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((route_kernel<PER, false, true>), grid, block, 0, stream, p);
  } else {
    if (p.bias) hipLaunchKernelGGL((route_kernel<PER, true, false>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((route_kernel<PER, false, false>), grid, block, 0, stream, p);
  }
}

hipError_t launch_any(const RouteArgs& p, bool backward, hipStream_t stream) {
  if (p.E <= 64) launch_per<1>(p, backward, stream);
  else if (p.E <= 128) launch_per<2>(p, backward, stream);
  else if (p.E <= 256) launch_per<4>(p, backward, stream);
  else if (p.E <= 512) launch_per<8>(p, backward, stream);
  else launch_per<16>(p, backward, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(RouteArgs p, hipStream_t stream) {
  p.lanes = 1;
  while (2 * p.lanes * p.groups <= 64) p.lanes *= 2;
  return launch_any(p, false, stream);
}

hipError_t launch_route_backward(const RouteArgs& p, hipStream_t stream) {
  return launch_any(p, true, stream);
}

}  // namespace dg
