// A whole mixture-of-experts layer for a few tokens (T <= 64), gfx950:
//   ids, p  = the k largest router logits of a token (ties: the lowest index)
//             and their softmax or sigmoid scores, normalised to sum 1
//   h[t,j]  = p[t,j] silu(x[t] . Wg^T) (x[t] . Wu^T)      Wg, Wu of expert ids[t,j]
//   y[t]    = sum_j h[t,j] . W2^T                         W2 of expert ids[t,j]
// with the expert weights in E4M3 (128 x 128 FP32 scales) or MXFP4 and the
// activations in BF16.
//
// The time is the stream of the weights of the experts that some token chose,
// each read once.  Three launches: the router (one workgroup: top-k, and per
// expert the list of its (token, slot) pairs), gate/up with the SwiGLU and the
// routing weight in its epilogue, and down, whose last workgroup per column
// tile adds the k slots of each token in slot order.
#include "mxfp4_device.hpp"
#include <stdlib.h>

namespace dg {
namespace {

constexpr int kWaves = 4;
constexpr int kRouterThreads = 1024;

// Routing tables in the workspace: counts [E], then per expert a list of
// pairs t * k + j (ascending), offsets [E] into one array of T k entries.
struct MoeTables {
  int* active;    // workgroups of the down launch that have work, per column tile
  int* counts;    // [E]
  int* offsets;   // [E]
  int* pairs;     // [T k]
};

struct MoeArgs {
  uint16_t* y;
  const uint16_t* x;
  const uint8_t* w13;
  const uint8_t* w2;
  const void* s13;
  const void* s2;
  int32_t* ids;
  float* weights;
  const float* logits;
  int scoring;
  int T, E, k;
  int64_t H, I;
  MoeTables tb;
  int* counters;   // per column tile of the down launch (zero between calls)
  uint16_t* h;     // [T k][I] BF16
  float* part;     // [T k][H]
};

// max over the wave, with the lowest index among equal values
__device__ __forceinline__ void wave_argmax(float& v, int& i) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const float ov = __shfl_xor(v, off, 64);
    const int oi = __shfl_xor(i, off, 64);
    if (ov > v || (ov == v && oi < i)) {
      v = ov;
      i = oi;
    }
  }
}

// Score of v relative to the largest chosen logit m: softmax e^(v - m),
// sigmoid sig(v) / sig(m), formed without overflow or underflow of either:
// sig(v) = e^min(v,0) / (1 + e^-|v|).
__device__ __forceinline__ float relative_score(float v, float m, int scoring) {
  if (scoring == MOE_SOFTMAX) return expf(v - m);
  return expf(fminf(v, 0.0f) - fminf(m, 0.0f)) * ((1.0f + expf(-fabsf(m))) / (1.0f + expf(-fabsf(v))));
}

// One workgroup.  A wave takes a token: k rounds of argmax over its logits
// (16 per lane at most, kMoeMaxExperts = 1024).  A logit of -inf or NaN is an
// expert that cannot be chosen; slots left over get id -1 and weight 0.
template <int PER>
__device__ __forceinline__ void route_token(const MoeArgs& p, int t, int lane, int* s_ids) {
  float v[PER];
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int e = lane + 64 * q;
    v[q] = e < p.E ? p.logits[(int64_t)t * p.E + e] : -INFINITY;
    if (v[q] != v[q]) v[q] = -INFINITY;
  }
  float m = 0.0f, sum = 0.0f, mine = 0.0f;
  int my_id = -1;
  for (int j = 0; j < p.k; ++j) {
    float b = -INFINITY;
    int bi = 0x7FFFFFFF;
#pragma unroll
    for (int q = 0; q < PER; ++q)
      if (v[q] > b) {
        b = v[q];
        bi = lane + 64 * q;
      }
    wave_argmax(b, bi);
    if (b == -INFINITY) break;  // wave-uniform
    if (j == 0) m = b;
    const float r = relative_score(b, m, p.scoring);
    sum += r;
    if (lane == j) {
      mine = r;
      my_id = bi;
    }
#pragma unroll
    for (int q = 0; q < PER; ++q)
      if (bi == lane + 64 * q) v[q] = -INFINITY;
  }
  if (lane < p.k) {
    s_ids[t * p.k + lane] = my_id;
    p.ids[t * p.k + lane] = my_id;
    p.weights[t * p.k + lane] = my_id < 0 ? 0.0f : mine / sum;
  }
}

__global__ void __launch_bounds__(kRouterThreads) moe_router_kernel(MoeArgs p) {
  __shared__ int s_ids[kMoeMaxPairs];
  __shared__ int s_cnt[kMoeMaxExperts], s_active;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = p.T * p.k;
  if (p.logits) {
    for (int t = wave; t < p.T; t += kRouterThreads / 64) {
      if (p.E <= 64) route_token<1>(p, t, lane, s_ids);
      else if (p.E <= 256) route_token<4>(p, t, lane, s_ids);
      else route_token<16>(p, t, lane, s_ids);
    }
  } else {
    for (int q = tid; q < n; q += kRouterThreads) {
      const int id = p.ids[q];  // the caller's: an id outside [0, E) is no expert
      s_ids[q] = id >= 0 && id < p.E ? id : -1;
    }
  }
  if (tid == 0) s_active = 0;
  __syncthreads();
  if (tid < p.E) {
    int c = 0;
    for (int q = 0; q < n; ++q) c += s_ids[q] == tid;
    s_cnt[tid] = c;
    if (c) atomicAdd(&s_active, 1);
  }
  __syncthreads();
  if (tid < p.E) {
    int off = 0;
    for (int e = 0; e < tid; ++e) off += s_cnt[e];
    p.tb.counts[tid] = s_cnt[tid];
    p.tb.offsets[tid] = off;
    for (int q = 0; q < n; ++q)
      if (s_ids[q] == tid) p.tb.pairs[off++] = q;
  }
  if (tid == 0) *p.tb.active = s_active;
}

// f(IntTag<NI>) for the 16-row fragments that `rows` rows need, at most MAXNI
template <int MAXNI, int NI = 1, class F>
__device__ __forceinline__ void with_fragments(int rows, F&& f) {
  if constexpr (NI == MAXNI) {
    f(IntTag<NI>{});
  } else {
    if (rows <= 16 * NI) f(IntTag<NI>{});
    else with_fragments<MAXNI, NI + 1>(rows, f);
  }
}

// Sums over the four waves of one tile of 16 NF weight rows by 16 NI
// activation rows; finish(f, i, quad) is called for every fragment by the
// wave that owns it.
template <int BF, int NI, int NF, int U, class Rows, class Finish>
__device__ __forceinline__ void expert_tile(const uint8_t* w, const void* scales, int64_t N,
                                            int64_t K, int64_t n0, const void* act,
                                            int64_t act_bytes, Rows&& row_of, v4f* red,
                                            Finish&& finish) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15;
  const int nkb = (int)((K + 127) / 128);
  const int64_t ldb = BF == FMT_FP8 ? K : K / 2;
  const int rows_b = (int)(N - n0 < 16 * NF ? N - n0 : 16 * NF);
  StreamOperands o;
  o.b = buffer_of(w + n0 * ldb, rows_b * ldb);
  if (BF == FMT_FP8) {
    const int64_t nb = (N + 127) / 128;
    o.sb = buffer_of(static_cast<const float*>(scales) + n0 / 128, (nkb * nb - n0 / 128) * 4);
    o.sb_step = (uint32_t)nb * 4;
  } else {
    o.sb = buffer_of(static_cast<const uint32_t*>(scales) + n0, (nkb * N - n0) * 4);
    o.sb_step = (uint32_t)N * 4;
  }
  o.a = buffer_of(act, act_bytes);
  Stream<ACT_BF16, BF, NI, NF, U> s;
  s.g = lane >> 4;
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int r = 16 * f + fr;
    s.vb[f] = r < rows_b ? (uint32_t)(r * ldb + (BF == FMT_FP8 ? 32 : 16) * s.g) : kOob;
    s.vsb[f] = r < rows_b ? (uint32_t)(4 * r) : kOob;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = row_of(16 * i + fr);  // row of the activations, -1: none
    s.va[i] = r >= 0 ? (uint32_t)(r * (K * 2) + 64 * s.g) : kOob;
  }
  const int kb0 = wave * nkb / kWaves, kb1 = (wave + 1) * nkb / kWaves;
  const int kmax = kb1 * 128 < K ? kb1 * 128 : (int)K;
  v4f acc[NF][NI];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[f][i] = v4f{0.f, 0.f, 0.f, 0.f};
  s.run(o, kb0, kb1, kmax, acc);
  constexpr int Q = NF * NI;
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < NI; ++i) red[(wave * Q + f * NI + i) * 64 + lane] = acc[f][i];
  __syncthreads();
  for (int q = wave; q < Q; q += kWaves) {
    v4f t = red[q * 64 + lane];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) t += red[(v * Q + q) * 64 + lane];
    finish(q / NI, q % NI, t);
  }
  __syncthreads();  // red is free again
}

// gate/up: rows 2i and 2i + 1 of W13 give gate and up of hidden unit i
template <int BF, int MAXNI, int NF, int U>
__global__ void __launch_bounds__(64 * kWaves) moe_up_kernel(MoeArgs p) {
  __shared__ v4f red[kWaves * NF * MAXNI * 64];
  const int e = blockIdx.y;
  const int count = p.tb.counts[e];
  if (count == 0) return;
  const int lane = threadIdx.x & 63, fr = lane & 15;
  const int64_t N = 2 * p.I, K = p.H, n0 = (int64_t)blockIdx.x * (16 * NF);
  const int* list = p.tb.pairs + p.tb.offsets[e];
  const int64_t sstep = BF == FMT_FP8 ? (K / 128) * ((N + 127) / 128) : ((K + 127) / 128) * N;
  const uint8_t* w = p.w13 + (int64_t)e * N * (BF == FMT_FP8 ? K : K / 2);
  const void* sc = static_cast<const uint32_t*>(p.s13) + e * sstep;
  for (int c0 = 0; c0 < count; c0 += 16 * MAXNI) {
    const int rows = count - c0 < 16 * MAXNI ? count - c0 : 16 * MAXNI;
    with_fragments<MAXNI>(rows, [&](auto ni) {
      expert_tile<BF, decltype(ni)::value, NF, U>(
          w, sc, N, K, n0, p.x, p.T * K * 2,
          [&](int r) { return r < rows ? list[c0 + r] / p.k : -1; }, red,
          [&](int f, int i, v4f t) {
            const int r = 16 * i + fr;
            if (r >= rows) return;
            const int pair = list[c0 + r];
            const float wt = p.weights[pair];
            const int64_t u = (n0 + 16 * f + 4 * (lane >> 4)) / 2;  // units u, u + 1 (I is even)
            if (u >= p.I) return;
            *reinterpret_cast<uint32_t*>(p.h + pair * p.I + u) =
                bf16x2_rne(silu_f(t[0]) * t[1] * wt, silu_f(t[2]) * t[3] * wt);
          });
    });
  }
}

template <int BF, int MAXNI, int NF, int U>
__global__ void __launch_bounds__(64 * kWaves) moe_down_kernel(MoeArgs p) {
  __shared__ v4f red[kWaves * NF * MAXNI * 64];
  __shared__ int s_last;
  const int e = blockIdx.y;
  const int count = p.tb.counts[e];
  const int active = *p.tb.active;
  const int lane = threadIdx.x & 63, fr = lane & 15;
  const int64_t N = p.H, K = p.I, n0 = (int64_t)blockIdx.x * (16 * NF);
  if (active == 0) {  // no token chose anything: y = 0
    if (e == 0)
      for (int q = threadIdx.x; q < p.T * 16 * NF; q += 64 * kWaves)
        if (n0 + q % (16 * NF) < N) p.y[q / (16 * NF) * N + n0 + q % (16 * NF)] = 0;
    return;
  }
  if (count == 0) return;
  const int* list = p.tb.pairs + p.tb.offsets[e];
  const int64_t sstep = BF == FMT_FP8 ? (K / 128) * ((N + 127) / 128) : ((K + 127) / 128) * N;
  const uint8_t* w = p.w2 + (int64_t)e * N * (BF == FMT_FP8 ? K : K / 2);
  const void* sc = static_cast<const uint32_t*>(p.s2) + e * sstep;
  for (int c0 = 0; c0 < count; c0 += 16 * MAXNI) {
    const int rows = count - c0 < 16 * MAXNI ? count - c0 : 16 * MAXNI;
    with_fragments<MAXNI>(rows, [&](auto ni) {
      expert_tile<BF, decltype(ni)::value, NF, U>(
          w, sc, N, K, n0, p.h, (int64_t)p.T * p.k * K * 2,
          [&](int r) { return r < rows ? list[c0 + r] : -1; }, red,
          [&](int f, int i, v4f t) {
            const int r = 16 * i + fr;
            const int64_t n = n0 + 16 * f + 4 * (lane >> 4);
            if (r < rows && n < N) publish4(p.part + list[c0 + r] * N + n, t);
          });
    });
  }
  if (!arrive_last(&p.counters[blockIdx.x], active, &s_last)) return;
  for (int q = threadIdx.x; q < p.T * 4 * NF; q += 64 * kWaves) {
    const int t = q / (4 * NF);
    const int64_t n = n0 + 4 * (q % (4 * NF));
    if (n >= N) continue;
    v4f s = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < p.k; ++j) {
      const int id = p.ids[t * p.k + j];
      if (id >= 0 && id < p.E) s += collect4(p.part + (int64_t)(t * p.k + j) * N + n);
    }
    *reinterpret_cast<uint2*>(p.y + t * N + n) =
        make_uint2(bf16x2_rne(s[0], s[1]), bf16x2_rne(s[2], s[3]));
  }
  if (threadIdx.x == 0)
    __hip_atomic_store(&p.counters[blockIdx.x], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

struct MoeLayout {
  size_t tables, h, part, total;
};
MoeLayout moe_layout(int T, int E, int k, int64_t H, int64_t I) {
  MoeLayout l;
  l.tables = kSplitkCounterBytes;
  l.h = l.tables + up16((size_t)(4 + 2 * E + T * k) * 4);
  l.part = l.h + up16((size_t)T * k * I * 2);
  l.total = l.part + (size_t)T * k * H * 4;
  return l;
}

int envi(const char* n, int d) { const char* e = getenv(n); return e ? atoi(e) : d; }

template <int BF, int MAXNI, int NF, int U>
hipError_t launch_up(const MoeArgs& p, hipStream_t stream) {
  hipLaunchKernelGGL((moe_up_kernel<BF, MAXNI, NF, U>),
                     dim3((unsigned)((2 * p.I + 16 * NF - 1) / (16 * NF)), (unsigned)p.E),
                     dim3(64 * kWaves), 0, stream, p);
  return hipGetLastError();
}
template <int BF, int MAXNI, int NF, int U>
hipError_t launch_down(const MoeArgs& p, hipStream_t stream) {
  hipLaunchKernelGGL((moe_down_kernel<BF, MAXNI, NF, U>),
                     dim3((unsigned)((p.H + 16 * NF - 1) / (16 * NF)), (unsigned)p.E),
                     dim3(64 * kWaves), 0, stream, p);
  return hipGetLastError();
}

template <int BF, int MAXNI>
hipError_t launch_experts(const MoeArgs& p, hipStream_t stream) {
  hipError_t e;
  const int a = envi("DG_UP", 11), b = envi("DG_DN", 11);
#define X(A, FN) switch (A) { case 11: e = FN<BF, MAXNI, 1, 1>(p, stream); break; \
  case 12: e = FN<BF, MAXNI, 1, 2>(p, stream); break; case 14: e = FN<BF, MAXNI, 1, 4>(p, stream); break;\
  case 21: e = FN<BF, MAXNI, 2, 1>(p, stream); break; case 22: e = FN<BF, MAXNI, 2, 2>(p, stream); break; \
  case 41: e = FN<BF, MAXNI, 4, 1>(p, stream); break; default: e = FN<BF, MAXNI, 4, 2>(p, stream); }
  X(a, launch_up)
  if (e != hipSuccess) return e;
  X(b, launch_down)
  return e;
}

}  // namespace

size_t moe_workspace_bytes(int T, int E, int k, int64_t H, int64_t I) {
  return moe_layout(T, E, k, H, I).total;
}

hipError_t launch_moe_layer(const MoeProblem& q, void* workspace, hipStream_t stream) {
  const MoeLayout l = moe_layout(q.T, q.E, q.k, q.H, q.I);
  char* ws = static_cast<char*>(workspace);
  MoeArgs p;
  p.y = q.y;
  p.x = q.x;
  p.w13 = q.w13;
  p.w2 = q.w2;
  p.s13 = q.s13;
  p.s2 = q.s2;
  p.ids = q.ids;
  p.weights = q.weights;
  p.logits = q.logits;
  p.scoring = q.scoring;
  p.T = q.T;
  p.E = q.E;
  p.k = q.k;
  p.H = q.H;
  p.I = q.I;
  p.counters = reinterpret_cast<int*>(ws);
  p.tb.active = reinterpret_cast<int*>(ws + l.tables);
  p.tb.counts = p.tb.active + 4;
  p.tb.offsets = p.tb.counts + q.E;
  p.tb.pairs = p.tb.offsets + q.E;
  p.h = reinterpret_cast<uint16_t*>(ws + l.h);
  p.part = reinterpret_cast<float*>(ws + l.part);
  hipLaunchKernelGGL(moe_router_kernel, dim3(1), dim3(kRouterThreads), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (q.T <= 16)
    return q.format == FMT_FP8 ? launch_experts<FMT_FP8, 1>(p, stream)
                               : launch_experts<FMT_MXFP4, 1>(p, stream);
  return q.format == FMT_FP8 ? launch_experts<FMT_FP8, 4>(p, stream)
                             : launch_experts<FMT_MXFP4, 4>(p, stream);
}

}  // namespace dg
