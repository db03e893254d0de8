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
// Up to 512 experts (in up to 16 groups): 16 lanes per token, four tokens a wave,
// all in FP32 with bounds on its errors; a token whose choice these bounds leave
// open is done again by the whole wave in 64 bits (route_exact).  More of either:
// one wave per token in 64 bits.
//
// What bounds it is the chain of k rounds of a maximum over 16 lanes (45
// instructions a round for 256 experts), not the logits' bytes.  MI355X, 16384 tokens,
// k = 8, in a graph: 256 experts without a bias 8.5 us (FP32; 16.8 MB, 3.4 us at 5.0
// TB/s), with a bias 10.3, and 8 groups by their best two 12.3 (of it about 2 for the
// tokens that are looked at again, since the last wave waits for them; 15.7 with
// route_exact for all of these, 37 with a wave per token in 64 bits); 512 experts in 8
// groups 18.6, 1024 without a bias 32, with one 84; 60 experts, k = 4, 30001 tokens 5.2, the gradient 5.4 (14 and
// 13 with a wave per token; with e^d from v_exp_f32 of a product rounded once, off by
// (d + 2) half steps, it took 5.0).
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
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
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

// PER logits from element `at` on as FP32, -inf from the count-th on (count may be
// negative); they start at any element.
template <int PER>
__device__ __forceinline__ void load_logits(const void* logits, bool bf16, int64_t at, int count,
                                            float (&v)[PER]) {
#pragma unroll
  for (int q = 0; q < PER; ++q) v[q] = -INFINITY;
  if (count <= 0) return;
  if (bf16) {
    const uint16_t* s = static_cast<const uint16_t*>(logits) + at;
    uint16_t u[PER];
    if (count >= PER) {
      __builtin_memcpy(u, __builtin_assume_aligned(s, 2), sizeof u);
#pragma unroll
      for (int q = 0; q < PER; ++q) v[q] = bf16_bits_to_f32(u[q]);
    } else {
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (q < count) v[q] = bf16_bits_to_f32(s[q]);
    }
  } else {
    const float* s = static_cast<const float*>(logits) + at;
    if (count >= PER) {
      __builtin_memcpy(v, __builtin_assume_aligned(s, 4), sizeof v);
    } else {
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (q < count) v[q] = s[q];
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

// The sum of a lane's values in halves: log2 PER roundings deep.
template <int PER>
__device__ __forceinline__ float lane_sum(const float (&v)[PER]) {
  float s[PER];
#pragma unroll
  for (int q = 0; q < PER; ++q) s[q] = v[q];
#pragma unroll
  for (int n = PER / 2; n >= 1; n /= 2)
#pragma unroll
    for (int q = 0; q < n; ++q) s[q] += s[q + n];
  return s[0];
}

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// Scores in 64 bits: the softmax of the lanes' logits v (largest m) or their
// sigmoid; 0 for v = -inf.
__device__ __forceinline__ double wide_score(float v, float m, int scoring) {
  if (scoring == ROUTE_SIGMOID) return 1.0 / (1.0 + exp(-(double)v));
  return v == m ? 1.0 : v == -INFINITY ? 0.0 : exp((double)v - (double)m);
}
template <int PER>
__device__ __forceinline__ void wide_scores(const float (&v)[PER], float m, int scoring, double (&c)[PER],
                                            double* value, int lane) {
  // one exponential in the code, not PER: unrolled they take every register there
  // is (16384 tokens of 1024 experts with a bias 175 us, so 84)
  double sum = 0.0;
#pragma unroll
  for (int q = 0; q < PER; ++q) value[lane * PER + q] = v[q];
#pragma unroll 1
  for (int q = 0; q < PER; ++q)
    sum += value[lane * PER + q] = wide_score((float)value[lane * PER + q], m, scoring);
#pragma unroll
  for (int q = 0; q < PER; ++q) c[q] = value[lane * PER + q];
  if (scoring == ROUTE_SOFTMAX) {
    const double inverse = 1.0 / wave_sum(sum);
#pragma unroll
    for (int q = 0; q < PER; ++q) c[q] *= inverse;
  }
}

// One wave, token t, PER consecutive experts a lane; value: room for 64 * PER
// numbers of this wave (GROUPED or BIASED).
template <int PER, bool BIASED, bool GROUPED>
__device__ __forceinline__ void route_exact(const RouteArgs& p, int64_t t, int lane, double* value) {
  using Key = std::conditional_t<BIASED, double, float>;
  float v[PER];
  load_logits<PER>(p.logits, p.bf16, t * p.ldl + lane * PER, p.E - lane * PER, v);
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    if (v[q] != v[q]) v[q] = -INFINITY;
    m = fmaxf(m, v[q]);
  }
  m = wave_top(m);
  Key key[PER];
  double c[PER];
  if (BIASED || (GROUPED && p.best == 2)) wide_scores<PER>(v, m, p.scoring, c, value, lane);
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
#pragma unroll
    for (int q = 0; q < PER; ++q)
      value[lane * PER + q] = BIASED || p.best == 1 || key[q] == (Key)-INFINITY ? (double)key[q] : c[q];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    // p.wide_lanes (a power of two) lanes a group
    const int lanes = p.wide_lanes, per = p.E / p.groups, g = lane / lanes;
    double a = -INFINITY, b = -INFINITY;  // the two largest, a >= b
    if (g < p.groups)
      for (int i = lane % lanes; i < per; i += lanes) {
        const double x = value[g * per + i];
        if (x > a) {
          b = a;
          a = x;
        } else if (x > b) {
          b = x;
        }
      }
    for (int d = 1; d < lanes; d *= 2) {
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
      const double o = lane_of(a, i * lanes);
      ahead += o > a || (o == a && i < g);
    }
    const uint64_t stays = __ballot(g < p.groups && ahead < p.top_groups);
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = lane * PER + q;
      if (e < p.E && !(stays >> (e / per * lanes) & 1)) key[q] = (Key)-INFINITY;
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
    float e[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) e[q] = expf(v[q] - m);
    w = p.scale * (expf(l - m) / wave_sum(lane_sum(e)));
  } else {
    w = p.scale * sigmoid(l);
  }
  if (p.scoring == ROUTE_SOFTMAX && m == INFINITY) w = NAN;
  if (lane < p.k) {
    p.ids[t * p.k + lane] = my_id;
    p.weights[t * p.k + lane] = my_id >= 0 ? w : 0.0f;
  }
}

template <int PER, bool BIASED, bool GROUPED>
__global__ void __launch_bounds__(64 * kRouteWaves) route_wide_kernel(RouteArgs p) {
  constexpr bool ROOM = GROUPED || BIASED;
  __shared__ double s_value[ROOM ? kRouteWaves : 1][ROOM ? 64 * PER : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t < p.T) route_exact<PER, BIASED, GROUPED>(p, t, threadIdx.x & 63, s_value[ROOM ? wave : 0]);
}

// ---- 16 lanes per token ----

// f over 16 neighbouring lanes, in each of them; like every move across lanes,
// outside of branches that lanes of a row take differently.
template <class T, class F>
__device__ __forceinline__ T row_join(T v, F&& f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  v = f(v, dpp<0x140>(v));
  return v;
}
// One instruction.  Of a NaN and a number the number; the compiler takes it for
// the first operand where that is -inf for certain, so a NaN may come out of the
// first of several values, to go at the next.
__device__ __forceinline__ float larger(float a, float b) {
  return __builtin_amdgcn_fmed3f(a, b, __builtin_inff());
}
__device__ __forceinline__ float row_top(float v) { return row_join(v, larger); }
__device__ __forceinline__ float row_low(float v) { return -row_top(-v); }
__device__ __forceinline__ float row_sum(float v) {
  return row_join(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ uint32_t row_top(uint32_t v) {
  return row_join(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// FP32 as an unsigned number of the same order, and back (no NaN, no -0).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ (uint32_t)((int32_t)u >> 31 | (int32_t)0x80000000);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u);
}

// A token's choice by unsigned keys, value above index, so that one maximum
// gives both and equal values go to the lowest index.  Value 0: cannot be chosen.
//   BF16 logits without a bias: the 16 bits of the logit in their order, exact.
//   else: 24 bits (23 with more than 256 experts), the place of the choice value c
//   on a grid of `steps` to 1 over the `window` below the largest c (what is
//   further below gets 0 as well).
// The value is off from c's place by at most eps steps + 2.5 for an error eps of c: the difference to the window's end is rounded by half a step, its product
// with the steps by one, and the fraction is cut.  eps of the sigmoid s, in 2^-24: the
// argument's product with log2 e 1.22 |l| s (1 - s) <= 0.27, v_exp_f32 (one ulp)
// 2 s (1 - s) <= 0.5, 1 + e rounded 1, v_rcp_f32 (one ulp) 2: below 2^-22.  Of the
// softmax, with d = m - l (rounded): (d + 2) 2^-24 of the numerator, s d <= 0.37 / sum;
// of the sum the same with d's mean, at most ln E <= 6.3, and 9 additions; two more
// roundings: less than 64 2^-24 / sum.  The sum with the bias adds |c| 2^-24.  Two
// keys whose values differ by more than twice that are in c's order.  Where closer
// ones meet among the k first or at their end, all that are that close to the k-th
// or above it, up to 16, are put in order in 64 bits, one a lane; with a bias on the
// softmax (whose sum would be needed in 64 bits), with more than 16, with groups
// that are too close, or where the choice reaches below the window, the token is left
// to route_exact.  With 256 sigmoid scores of normal logits (deviation 2), a bias
// (0.1) and 4 of 8 groups that is one token in thirty thousand; one in 1600 is put in
// order.
template <bool BIASED, int PER>
struct Grid {
  static constexpr uint32_t index_bits = PER > 16 ? 9 : 8, most = (1u << index_bits) - 1;
  static constexpr float top = (float)((1u << (32 - index_bits)) - 1);
  static constexpr float window = BIASED ? 2.0f : 16.0f, steps = 0.95f * top / window;
};

template <int PER, bool BIASED, bool GROUPED>
__global__ void __launch_bounds__(64 * kRouteWaves) route_kernel(RouteArgs p) {
  using G = Grid<BIASED, PER>;
  constexpr int EXACT = PER > 16 ? 8 : 4;  // experts a lane in route_exact
  constexpr bool ROOM = GROUPED || BIASED;
  __shared__ double s_value[ROOM ? kRouteWaves : 1][ROOM ? 64 * EXACT : 1];
  const int lane = threadIdx.x & 63, lane16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * 4;
  if (t0 >= p.T) return;
  const int64_t t = t0 + (lane >> 4) < p.T ? t0 + (lane >> 4) : p.T - 1;
  // p.lanes lanes a group (16: no groups), PER consecutive experts of it each
  const int per = GROUPED ? p.E / p.groups : p.E, group = GROUPED ? lane16 / p.lanes : 0;
  const int sub = (GROUPED ? lane16 % p.lanes : lane16) * PER, base = group * per + sub;
  const int count = GROUPED && group >= p.groups ? 0 : per - sub;
  float v[PER], c[PER];
  load_logits<PER>(p.logits, p.bf16, t * p.ldl + base, count, v);
  if constexpr (BIASED) load_logits<PER>(p.bias, false, base, count, c);
  const bool pairs = GROUPED && p.best == 2;
  const bool exact = !BIASED && p.bf16, softmax = p.scoring == ROUTE_SOFTMAX;
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    if (softmax && v[q] != v[q]) v[q] = -INFINITY;
    m = larger(m, v[q]);
  }
  m = row_top(m);
  bool open = m == INFINITY;  // left to route_exact
  if (m == -INFINITY) m = 0.0f;
  // scores (what cannot be chosen: NaN), also where the weights need their sum
  float total = 1.0f, eps = 0x1p-22f;
  if (BIASED || pairs || (!p.renormalise && softmax)) {
    float e[PER];
    if (softmax) {
#pragma unroll
      for (int q = 0; q < PER; ++q) e[q] = expf(v[q] - m);
      total = row_sum(lane_sum(e));
      const float inverse = 1.0f / total;
      eps = inverse * 0x1p-18f;
#pragma unroll
      for (int q = 0; q < PER; ++q) e[q] *= inverse;
    } else {
#pragma unroll
      for (int q = 0; q < PER; ++q)
        e[q] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v[q] * -1.44269504f));
    }
#pragma unroll
    for (int q = 0; q < PER; ++q)  // v 0 is NaN for a v of -inf
      c[q] = BIASED ? __builtin_fmaf(v[q], 0.0f, e[q] + c[q]) : __builtin_fmaf(v[q], 0.0f, e[q]);
  }
  uint32_t key[PER], near = 0;  // values within `near` of each other are not told apart
  if (exact) {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const uint32_t u = ordered(v[q] + 0.0f) & 0xFFFF0000u;  // -0 is 0
      key[q] = v[q] > -INFINITY ? u | (uint32_t)(0xFFFF - base - q) : 0;
    }
  } else {
    float hi = -INFINITY;
#pragma unroll
    for (int q = 0; q < PER; ++q) hi = larger(hi, BIASED ? c[q] : v[q]);
    hi = row_top(hi);
    const float lo = hi - G::window;
    open = open || (hi > -INFINITY && !(fabsf(hi) < 65536.0f));
    const float size = fminf(fmaxf(fabsf(hi), fabsf(lo)), 65536.0f);  // of c in the window
    near = 6 + (BIASED ? (uint32_t)(2.0f * G::steps * (fminf(eps, 1.0f) + size * 0x1p-24f)) : 0);
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const float x = BIASED ? c[q] : v[q];
      const uint32_t value = (uint32_t)__builtin_amdgcn_fmed3f((x - lo) * G::steps, 0.0f, G::top);
      key[q] = (value << G::index_bits) + (G::most - (uint32_t)(base + q));
    }
  }
  const uint32_t shift = exact ? 16 : G::index_bits;
  if constexpr (GROUPED) {
    // a group's value, as an unsigned number: the largest key, or the sum of the
    // two largest scores in FP32 (off by the two errors and one rounding)
    uint32_t value = 0;
    float off = 0.0f;
    if (pairs) {
      float a = -INFINITY, b = -INFINITY;  // a >= b
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const float x = c[q] > -INFINITY ? c[q] : -INFINITY;  // no NaN into the median
        b = __builtin_amdgcn_fmed3f(a, b, x);
        a = larger(a, x);
      }
      const auto meet = [&](float oa, float ob) {
        b = larger(__builtin_amdgcn_fmed3f(a, b, oa), ob);  // the second of the two firsts, or a second
        a = larger(a, oa);
      };
      if (p.lanes >= 2) meet(dpp<0xB1>(a), dpp<0xB1>(b));
      if (p.lanes >= 4) meet(dpp<0x4E>(a), dpp<0x4E>(b));
      if (p.lanes >= 8) meet(dpp<0x141>(a), dpp<0x141>(b));
      if (!(b > -INFINITY)) b = 0.0f;
      if (a > -INFINITY) value = ordered(a + b + 0.0f);
      // two sums of two scores with their bias, each sum rounded
      const float size = row_top(a > -INFINITY ? larger(fabsf(a), fabsf(b)) : 0.0f);
      off = 4.0f * eps + size * (BIASED ? 8 * 0x1p-24f : 4 * 0x1p-24f);
    } else {
#pragma unroll
      for (int q = 0; q < PER; ++q) value = max(value, key[q]);
      if (p.lanes >= 2) value = max(value, dpp<0xB1>(value));
      if (p.lanes >= 4) value = max(value, dpp<0x4E>(value));
      if (p.lanes >= 8) value = max(value, dpp<0x141>(value));
    }
    int ahead = 0, level = 0;  // of the other groups, by rotating the 16 lanes
    static_for<15>([&](auto R) {
      constexpr int r = decltype(R)::value + 1;
      if ((r & (p.lanes - 1)) == 0) {
        const uint32_t o = dpp<0x120 + r>(value);
        ahead += o > value;
        level += o >= value;
      }
    });
    const bool stays = ahead < p.top_groups;
    open = open || (stays && value > 0 && level >= p.top_groups);  // equal sums
    // the smallest that stays against the largest that does not
    const uint32_t in = ~row_top(stays ? ~value : 0u), out = row_top(stays ? 0u : value);
    if (out > 0) {
      if (pairs) {
        open = open || !(from_ordered(in) - from_ordered(out) > off);
      } else {
        open = open || (!exact && (in >> shift) - (out >> shift) <= near);
      }
    }
#pragma unroll
    for (int q = 0; q < PER; ++q) key[q] = stays ? key[q] : 0;
  }
  // k rounds of the largest key below the last one: key - last wraps round to
  // the top of the range for these and stays below them for keys taken before
  uint32_t mine = 0, after = 0, last = 0;
  const auto take = [&](int j) {  // lane j gets the largest of what is left
    if (lane16 == j) mine = last;
    uint32_t d = 0u - last;  // no key: 0
#pragma unroll
    for (int q = 0; q < PER; ++q) d = max(d, key[q] - last);
    const uint32_t next = last + row_top(d);
    last = last > 0 ? next : 0;
    if (lane16 == j) after = last;
  };
#pragma unroll
  for (int q = 0; q < PER; ++q) last = max(last, key[q]);
  last = row_top(last);
  for (int j = 0; j < p.k; ++j) take(j);
  const auto id_of = [&](uint32_t k) {
    return k >> shift == 0 ? -1 : (int)((exact ? 0xFFFFu : G::most) - (k & ((1u << shift) - 1)));
  };
  bool chosen = lane16 < p.k, doubt = false;
  if (!exact) {
    open = open || (chosen && mine >> shift == 0);
    doubt = chosen && (mine >> shift) - (after >> shift) <= near;
    if (BIASED && softmax) open = open || doubt;
  }
  int slot = lane16, id = id_of(mine);
  float l = chosen && id >= 0 ? load_logit(p, t * p.ldl + id) : -INFINITY;
  if (__ballot(doubt && !open)) {
    for (int j = p.k; j < 16; ++j) take(j);
    const uint32_t kth = (uint32_t)__shfl((int)mine, (lane & 48) + p.k - 1, 64) >> shift;
    const auto close = [&](uint32_t k) { return k >> shift != 0 && kth - (k >> shift) <= near; };
    open = open || close(last);  // a seventeenth
    chosen = chosen || close(mine);
    id = chosen ? id_of(mine) : -1;
    l = id >= 0 ? load_logit(p, t * p.ldl + id) : -INFINITY;
    double x = l;
    if (BIASED && id >= 0) x = 1.0 / (1.0 + exp(-x)) + (double)p.bias[id];
    slot = 0;
    static_for<15>([&](auto R) {
      constexpr int r = decltype(R)::value + 1;
      const double o = dpp<0x120 + r>(x);
      const int oid = (int)dpp<0x120 + r>((uint32_t)id);
      slot += oid >= 0 && (o > x || (o == x && oid < id));
    });
    chosen = chosen && slot < p.k;
    if (!chosen) l = -INFINITY;
  }
  const uint64_t left = __ballot(open && t0 + (lane >> 4) < p.T);
  const bool some = chosen && id >= 0;
  float w = 0.0f;
  if (p.renormalise) {
    const float top = row_top(l);
    const float r = some ? relative_score(l, top, p.scoring) : 0.0f;
    w = p.scale * r / row_sum(r);
  } else if (softmax) {
    w = p.scale * (expf(l - m) / total);
  } else {
    w = p.scale * sigmoid(l);
  }
  if (chosen && t0 + (lane >> 4) < p.T && !(left >> (lane & 48) & 0xFFFF)) {
    p.ids[t * p.k + slot] = id;
    p.weights[t * p.k + slot] = some ? w : 0.0f;
  }
  if (left == 0) return;
  for (int r = 0; r < 4; ++r)
    if (left >> (16 * r) & 0xFFFF)
      route_exact<EXACT, BIASED, GROUPED>(p, t0 + r, lane, s_value[ROOM ? wave : 0]);
}

// The gradient: LANES lanes a token (16 or 64), PER consecutive experts each.
template <int LANES, int PER>
__global__ void __launch_bounds__(64 * kRouteWaves) route_backward_kernel(RouteArgs p) {
  constexpr int TOKENS = 64 / LANES;
  const int lane = threadIdx.x & 63, at = lane & (LANES - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * TOKENS;
  if (t0 >= p.T) return;
  const bool real = t0 + lane / LANES < p.T;
  const int64_t t = real ? t0 + lane / LANES : p.T - 1;
  const auto top_of = [](float x) { return LANES == 16 ? row_top(x) : wave_top(x); };
  const auto sum_of = [](float x) { return LANES == 16 ? row_sum(x) : wave_sum(x); };
  // lane j has slot j; a slot without an expert, or one of an expert that
  // cannot be chosen, gives and gets nothing
  int id = at < p.k ? p.ids[t * p.k + at] : -1;
  if (id >= p.E) id = -1;
  float l = id >= 0 ? load_logit(p, t * p.ldl + id) : -INFINITY;
  if (!(l > -INFINITY)) id = -1, l = -INFINITY;
  const float g = id >= 0 ? p.scale * p.dweights[t * p.k + at] : 0.0f;
  // slot: what is added to the logit of the slot's expert
  float slot = 0.0f, d[PER];
#pragma unroll
  for (int q = 0; q < PER; ++q) d[q] = 0.0f;
  if (p.renormalise) {
    const float top = top_of(l);
    const float r = id >= 0 ? relative_score(l, top, p.scoring) : 0.0f;
    const float sum = sum_of(r);
    const float q = sum == 0.0f ? 0.0f : r / sum;  // NaN with +inf among the chosen
    slot = q * (g - sum_of(g * q));
    if (p.scoring == ROUTE_SIGMOID) slot *= sigmoid(-l);
  } else if (p.scoring == ROUTE_SOFTMAX) {
    // every logit: minus the sum of the slots' parts times its score
    float v[PER], m = -INFINITY;
    load_logits<PER>(p.logits, p.bf16, t * p.ldl + at * PER, p.E - at * PER, v);
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      if (v[q] != v[q]) v[q] = -INFINITY;
      m = larger(m, v[q]);
    }
    m = top_of(m);
    if (!(m > -INFINITY)) m = 0.0f;
#pragma unroll
    for (int q = 0; q < PER; ++q) d[q] = expf(v[q] - m);
    const float sum = sum_of(lane_sum(d));
    const float inverse = sum == 0.0f ? 0.0f : 1.0f / sum;
    slot = id >= 0 ? g * (expf(l - m) * inverse) : 0.0f;
    const float all = -sum_of(slot) * inverse;
#pragma unroll
    for (int q = 0; q < PER; ++q) d[q] *= all;
  } else {
    slot = g * sigmoid(l) * sigmoid(-l);
  }
  if (id < 0) slot = 0.0f;
  const int e0 = at * PER;
  const auto add = [&](int e, float s) {
#pragma unroll
    for (int q = 0; q < PER; ++q) d[q] += e - e0 == q ? s : 0.0f;
  };
  static_while<kMoeMaxSlots>([&](auto J) {
    constexpr int j = decltype(J)::value;
    if (j >= p.k) return false;
    if constexpr (LANES == 16) add((int)dpp<0x150 + j>((uint32_t)id), dpp<0x150 + j>(slot));
    else add(__builtin_amdgcn_readlane(id, j), lane_of(slot, j));
    return true;
  });
  if (!real || e0 >= p.E) return;
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

template <int PER, bool WIDE>
void launch_forward(const RouteArgs& p, hipStream_t stream) {
  const int64_t tokens = kRouteWaves * (WIDE ? 1 : 4);  // a workgroup
  const dim3 grid((unsigned)((p.T + tokens - 1) / tokens)), block(64 * kRouteWaves);
  const auto go = [&](auto biased, auto grouped) {
    constexpr bool B = decltype(biased)::value, G = decltype(grouped)::value;
    if constexpr (WIDE && PER <= 8 && !G) return;  // 16 lanes always do
    else if constexpr (WIDE) hipLaunchKernelGGL((route_wide_kernel<PER, B, G>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((route_kernel<PER, B, G>), grid, block, 0, stream, p);
  };
  if (p.top_groups < p.groups) p.bias ? go(IntTag<1>{}, IntTag<1>{}) : go(IntTag<0>{}, IntTag<1>{});
  else p.bias ? go(IntTag<1>{}, IntTag<0>{}) : go(IntTag<0>{}, IntTag<0>{});
}

template <int LANES, int PER>
void launch_backward(const RouteArgs& p, hipStream_t stream) {
  constexpr int64_t tokens = kRouteWaves * 64 / LANES;
  hipLaunchKernelGGL((route_backward_kernel<LANES, PER>), dim3((unsigned)((p.T + tokens - 1) / tokens)),
                     dim3(64 * kRouteWaves), 0, stream, p);
}

}  // namespace

hipError_t launch_route(RouteArgs p, hipStream_t stream) {
  const bool grouped = p.top_groups < p.groups;
  const auto lanes_of = [&](int lanes) {  // the power of two that gives every group as many
    int n = 1;
    while (2 * n * p.groups <= lanes) n *= 2;
    return n;
  };
  p.wide_lanes = lanes_of(64);
  p.lanes = grouped ? lanes_of(16) : 16;
  // experts a lane, where 16 lanes take a token
  const int per = grouped ? (p.E / p.groups + p.lanes - 1) / p.lanes : (p.E + 15) / 16;
  if (p.E > 512 || per > 32 || (grouped && p.groups > 16)) {
    if (p.E <= 256) launch_forward<4, true>(p, stream);
    else if (p.E <= 512) launch_forward<8, true>(p, stream);
    else launch_forward<16, true>(p, stream);
  } else if (per <= 4) {
    launch_forward<4, false>(p, stream);
  } else if (per <= 8) {
    launch_forward<8, false>(p, stream);
  } else if (per <= 16) {
    launch_forward<16, false>(p, stream);
  } else {
    launch_forward<32, false>(p, stream);
  }
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteArgs& p, hipStream_t stream) {
  if (p.E <= 64) launch_backward<16, 4>(p, stream);
  else if (p.E <= 128) launch_backward<16, 8>(p, stream);
  else if (p.E <= 256) launch_backward<16, 16>(p, stream);
  else if (p.E <= 512) launch_backward<64, 8>(p, stream);
  else launch_backward<64, 16>(p, stream);
  return hipGetLastError();
}

}  // namespace dg
