// A whole mixture-of-experts layer for a few tokens (T <= 64), gfx950:
//   ids, p  = the k largest router logits of a token (ties: the lowest index)
//             and their softmax or sigmoid scores, normalised to sum 1
//   h[t,j]  = p[t,j] silu(x[t] . Wg^T) (x[t] . Wu^T)      Wg, Wu of expert ids[t,j]
//             (held in FP32's 24 bits, as the sum of three BF16 numbers)
//   y[t]    = sum_j h[t,j] . W2^T                         W2 of expert ids[t,j]
// with the expert weights in E4M3 (128 x 128 FP32 scales) or MXFP4 and the
// activations in BF16.
//
// The time is the stream of the weights of the experts that some token chose,
// each read once.  Three launches: the router (one workgroup: top-k, and per
// expert the list of its (token, slot) pairs), gate/up with the SwiGLU and the
// routing weight in its epilogue, and down, whose last workgroup per column
// tile adds the k slots of each token in slot order.  Where the hidden values of
// all pairs would take more than kMaxHidden, gate/up and down take the hidden
// units in chunks, down adding to what it has.
//
// MI355X, kernels alone (router, up, down): 1 token on 8 experts of 4096 x
// 11008 in E4M3 4.7 + 37 + 23 us at best (180 MB at 4.9 TB/s, 90 MB at 4.0); 64 tokens
// on the same experts in MXFP4 9 + 98 + 80 us (383 MB at 3.9 TB/s, 191 MB at
// 2.4: 256 workgroups of 128 weight rows, one a CU, whose LDS reads and products
// for 20 pairs, 60 rows, no longer hide behind the weights; 65 us when h had two
// parts and a pair two rows).
#include "mxfp4_device.hpp"

namespace dg {
namespace {

constexpr int kWaves = 4;
constexpr int kRouterThreads = 1024;
constexpr int kParts = 3;  // BF16 numbers that hold a hidden value

// Routing tables in the workspace: counts [E], offsets [E] into one array of T k
// entries, and there each expert's list of pairs t * k + j, in any order.
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
  uint16_t* h;     // [T k][3][chunk] BF16: the value's three parts
  float* part;     // [T k][H]
  int64_t u0, chunk;  // the hidden units of this launch: u0 .. u0 + chunk - 1
};

// Largest value of the wave, in every lane (no NaN among them).
__device__ __forceinline__ float wave_top(float v) {
  auto join = [](float x, int y) { return fmaxf(x, __int_as_float(y)); };
  const auto dpp = [](float x, auto ctrl) {
    return __builtin_amdgcn_mov_dpp(__float_as_int(x), decltype(ctrl)::value, 0xF, 0xF, false);
  };
  v = join(v, dpp(v, IntTag<0xB1>{}));   // within 4 lanes
  v = join(v, dpp(v, IntTag<0x4E>{}));
  v = join(v, dpp(v, IntTag<0x124>{}));  // within 16
  v = join(v, dpp(v, IntTag<0x128>{}));
  const int b = __float_as_int(v);
  const float lo = join(__int_as_float(__builtin_amdgcn_readlane(b, 0)), __builtin_amdgcn_readlane(b, 16));
  const float hi = join(__int_as_float(__builtin_amdgcn_readlane(b, 32)), __builtin_amdgcn_readlane(b, 48));
  return fmaxf(lo, hi);
}

// Score of v relative to the largest chosen logit m: softmax e^(v - m),
// sigmoid sig(v) / sig(m), formed without overflow or underflow of either:
// sig(v) = e^min(v,0) / (1 + e^-|v|).
__device__ __forceinline__ float relative_score(float v, float m, int scoring) {
  if (scoring == MOE_SOFTMAX) return expf(v - m);
  return expf(fminf(v, 0.0f) - fminf(m, 0.0f)) * ((1.0f + expf(-fabsf(m))) / (1.0f + expf(-fabsf(v))));
}

// One wave, one token: k rounds of the largest logit, PER consecutive experts
// a lane, so that the lowest lane of the lanes that hold it has the lowest
// index.  A logit of -inf or NaN is an expert that cannot be chosen; slots left
// over get id -1 and weight 0.
template <int PER>
__device__ __forceinline__ void route_token(const MoeArgs& p, int t, int lane, int* s_ids) {
  float v[PER];
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int e = lane * PER + q;
    v[q] = e < p.E ? p.logits[(int64_t)t * p.E + e] : -INFINITY;
    if (v[q] != v[q]) v[q] = -INFINITY;
  }
  float m = 0.0f, sum = 0.0f, mine = 0.0f;
  int my_id = -1;
  for (int j = 0; j < p.k; ++j) {
    float b = v[0];
    int bi = 0;
#pragma unroll
    for (int q = 1; q < PER; ++q)
      if (v[q] > b) {
        b = v[q];
        bi = q;
      }
    const float top = wave_top(b);
    if (top == -INFINITY) break;  // wave-uniform
    const int owner = __ffsll((unsigned long long)__ballot(b == top)) - 1;
    const int id = owner * PER + __builtin_amdgcn_readlane(bi, owner);
    if (j == 0) m = top;
    const float r = relative_score(top, m, p.scoring);
    sum += r;
    if (lane == j) {
      mine = r;
      my_id = id;
    }
#pragma unroll
    for (int q = 0; q < PER; ++q)
      if (id == lane * PER + q) v[q] = -INFINITY;
  }
  if (lane < p.k) {
    s_ids[t * p.k + lane] = my_id;
    p.ids[t * p.k + lane] = my_id;
    p.weights[t * p.k + lane] = my_id < 0 ? 0.0f : mine / sum;
  }
}

// One workgroup: a wave takes a token at a time, then every expert gets its
// list of pairs.  The order within a list is the order of arrival at a counter
// in LDS; it decides which row of a tile a pair takes, not its result.
__global__ void __launch_bounds__(kRouterThreads) moe_router_kernel(MoeArgs p) {
  constexpr int W = kRouterThreads / 64;
  static_assert(kRouterThreads >= kMoeMaxExperts && kRouterThreads >= kMoeMaxPairs, "one each");
  __shared__ int s_ids[kMoeMaxPairs];
  __shared__ int s_cnt[kRouterThreads], s_off[kRouterThreads], s_sum[W], s_active[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = p.T * p.k;
  s_cnt[tid] = 0;
  if (p.logits) {
    for (int t = wave; t < p.T; t += W) {
      if (p.E <= 64) route_token<1>(p, t, lane, s_ids);
      else if (p.E <= 256) route_token<4>(p, t, lane, s_ids);
      else route_token<16>(p, t, lane, s_ids);
    }
  } else if (tid < n) {
    const int id = p.ids[tid];  // the caller's: an id outside [0, E) is no expert
    s_ids[tid] = id >= 0 && id < p.E ? id : -1;
  }
  __syncthreads();
  const int id = tid < n ? s_ids[tid] : -1;
  const int rank = id >= 0 ? atomicAdd(&s_cnt[id], 1) : 0;
  __syncthreads();
  // offsets: running sum of the counts over the wave, then over the waves
  const int count = s_cnt[tid];
  int sum = count;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(sum, d, 64);
    if (lane >= d) sum += o;
  }
  const int used = __popcll(__ballot(count > 0));
  if (lane == 63) {
    s_sum[wave] = sum;
    s_active[wave] = used;
  }
  __syncthreads();
  int before = 0, active = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < wave) before += s_sum[w];
    active += s_active[w];
  }
  const int offset = before + sum - count;
  s_off[tid] = offset;
  if (tid < p.E) {
    p.tb.counts[tid] = count;
    p.tb.offsets[tid] = offset;
  }
  if (tid == 0) *p.tb.active = active;
  __syncthreads();
  if (id >= 0) p.tb.pairs[s_off[id] + rank] = tid;
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

// Operands of weight rows n0 .. n0 + rows_b - 1 of one expert's [N][ld] matrix,
// its columns k0 .. k0 + K - 1 (k0 a multiple of 128), with activations in BF16.
template <int BF>
__device__ __forceinline__ StreamOperands expert_operands(const uint8_t* w, const void* scales,
                                                          int64_t N, int64_t ld, int64_t k0,
                                                          int64_t K, int64_t n0, int rows_b,
                                                          const void* act, int64_t act_bytes) {
  const int nkb = (int)((K + 127) / 128);
  const int64_t ldb = BF == FMT_FP8 ? ld : ld / 2, off = BF == FMT_FP8 ? k0 : k0 / 2;
  StreamOperands o;
  o.b = buffer_of(w + n0 * ldb + off, rows_b * ldb - off);
  if (BF == FMT_FP8) {
    const int64_t nb = (N + 127) / 128;
    o.sb = buffer_of(static_cast<const float*>(scales) + k0 / 128 * nb + n0 / 128,
                     (nkb * nb - n0 / 128) * 4);
    o.sb_step = (uint32_t)nb * 4;
  } else {
    o.sb = buffer_of(static_cast<const uint32_t*>(scales) + k0 / 128 * N + n0, (nkb * N - n0) * 4);
    o.sb_step = (uint32_t)N * 4;
  }
  o.a = buffer_of(act, act_bytes);
  o.last = nkb - 1;
  return o;
}

// One tile of weight rows (ldb bytes apart) by 16 NI activation rows:
// finish(f, quads) is called for every 16 weight rows with the NI quads of their
// outputs, by one wave.
//
// Few rows: four waves with a quarter of K each and the same 16 NF weight rows,
// activations straight into fragments.
template <int BF, int NF_, int MAXNI>
struct StreamEngine {
  static constexpr int NF = NF_, ROWS_B = 16 * NF, THREADS = 64 * kWaves, WAVES = 1;
  template <int NI, class Rows, class Finish>
  static __device__ __forceinline__ void tile(const StreamOperands& o, int64_t K, int64_t ldb,
                                              int rows_b, Rows&& row_of,
                                              uint8_t* const (&slots)[kSharedMaxDepth],
                                              Finish&& finish) {
    v4f* red = reinterpret_cast<v4f*>(slots[0]);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15;
    const int nkb = o.last + 1;
    Stream<ACT_BF16, BF, NI, NF, 1> s;
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
    const int kb0 = run_begin(wave, nkb, kWaves), kb1 = run_begin(wave + 1, nkb, kWaves);
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
    for (int f = wave; f < NF; f += kWaves) {
      v4f t[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        t[i] = red[(f * NI + i) * 64 + lane];
#pragma unroll
        for (int v = 1; v < kWaves; ++v) t[i] += red[(v * Q + f * NI + i) * 64 + lane];
      }
      finish(f, t);
    }
    __syncthreads();  // red is free again
  }
  static constexpr int R = 1, SLOT = 16, SLOT0 = kWaves * NF * MAXNI * 1024;
};

// More rows: activations in LDS (Shared, mxfp4_device.hpp).
template <int BF, int MAXNI, int R_ = shared_depth(BF, MAXNI)>
struct SharedEngine {
  static constexpr int R = R_;
  typedef Shared<BF, MAXNI, R> Largest;
  static constexpr int ROWS_B = Largest::ROWS_B, NF = ROWS_B / 16, THREADS = kSharedThreads;
  static constexpr int SLOT0 = Largest::SLOT0, SLOT = Largest::SLOT;
  static constexpr int WAVES = Largest::WAVES;
  template <int NI, class Rows, class Finish>
  static __device__ __forceinline__ void tile(const StreamOperands& o, int64_t K, int64_t ldb,
                                              int rows_b, Rows&& row_of,
                                              uint8_t* const (&slots)[kSharedMaxDepth],
                                              Finish&& finish) {
    Shared<BF, NI, R> s;
    s.init(ldb, rows_b, K * 2, row_of);
    s.run(o, K, 0, s.WK, slots, finish);
  }
};

// gate/up: rows 2i and 2i + 1 of W13 give gate and up of hidden unit i
template <int BF, int MAXNI, class Engine>
__global__ void __launch_bounds__(Engine::THREADS, Engine::WAVES) moe_up_kernel(MoeArgs p) {
  constexpr int NF = Engine::NF;
  DG_SHARED_SLOTS(Engine);
  const int e = blockIdx.y;
  const int count = p.tb.counts[e];
  if (count == 0) return;
  const int lane = threadIdx.x & 63, fr = lane & 15;
  const int64_t N = 2 * p.I, K = p.H, n0 = 2 * p.u0 + (int64_t)blockIdx.x * (16 * NF);
  const int64_t end = 2 * (p.u0 + p.chunk), ldb = BF == FMT_FP8 ? K : K / 2;
  const int* list = p.tb.pairs + p.tb.offsets[e];
  const int64_t sstep = BF == FMT_FP8 ? (K / 128) * ((N + 127) / 128) : ((K + 127) / 128) * N;
  const uint8_t* w = p.w13 + e * N * ldb;
  const void* sc = static_cast<const uint32_t*>(p.s13) + e * sstep;
  const int rows_b = (int)(end - n0 < 16 * NF ? end - n0 : 16 * NF);
  const StreamOperands o = expert_operands<BF>(w, sc, N, K, 0, K, n0, rows_b, p.x, p.T * K * 2);
  for (int c0 = 0; c0 < count; c0 += 16 * MAXNI) {
    const int rows = count - c0 < 16 * MAXNI ? count - c0 : 16 * MAXNI;
    with_fragments<MAXNI>(rows, [&](auto ni) {
      constexpr int NI = decltype(ni)::value;
      Engine::template tile<NI>(
          o, K, ldb, rows_b, [&](int r) { return r < rows ? list[c0 + r] / p.k : -1; }, slots,
          [&](int f, const v4f (&t)[NI]) {
            // units u, u + 1 (the chunk is even)
            const int64_t u = (n0 + 16 * f + 4 * (lane >> 4)) / 2 - p.u0;
            if (u >= p.chunk) return;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              const int r = 16 * i + fr;
              if (r >= rows) continue;
              const int pair = list[c0 + r];
              const float wt = p.weights[pair];
              // Three parts, each the leading BF16 of what is left (exact, so they
              // hold FP32's 24 bits).  With two, 16 bits, the rounding of h was all
              // of y's error before its own: 2.4e-6 of rms, the sums' 1e-7 to 3e-7.
              float h0 = silu_f(t[i][0]) * t[i][1] * wt, h1 = silu_f(t[i][2]) * t[i][3] * wt;
              uint16_t* d = p.h + pair * kParts * p.chunk + u;
#pragma unroll
              for (int part = 0; part < kParts; ++part) {
                const uint32_t v = bf16x2_rne(h0, h1);
                *reinterpret_cast<uint32_t*>(d + part * p.chunk) = v;
                h0 -= __uint_as_float(v << 16);
                h1 -= __uint_as_float(v & 0xFFFF0000u);
                // infinite and NaN values are their first part
                h0 = fabsf(h0) < INFINITY ? h0 : 0.0f;
                h1 = fabsf(h1) < INFINITY ? h1 : 0.0f;
              }
            }
          });
    });
  }
}

// v of the lane D after this one among 16, of `next` where that is past the 16th
template <int D>
__device__ __forceinline__ float after(float v, float next, int fr) {
  const int a = __builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + 16 - D, 0xF, 0xF, false);
  const int b = __builtin_amdgcn_mov_dpp(__float_as_int(next), 0x120 + 16 - D, 0xF, 0xF, false);
  return __int_as_float(fr + D < 16 ? a : b);
}

template <int BF, int MAXNI, class Engine>
__global__ void __launch_bounds__(Engine::THREADS, Engine::WAVES) moe_down_kernel(MoeArgs p) {
  constexpr int NF = Engine::NF;
  DG_SHARED_SLOTS(Engine);
  __shared__ int s_last;
  const int e = blockIdx.y;
  const int count = p.tb.counts[e];
  const int active = *p.tb.active;
  const int lane = threadIdx.x & 63, fr = lane & 15;
  const int64_t N = p.H, K = p.chunk, n0 = (int64_t)blockIdx.x * (16 * NF);
  const int64_t ldb = BF == FMT_FP8 ? p.I : p.I / 2;
  if (active == 0) {  // no token chose anything: y = 0 (in every chunk's launch)
    if (e == 0)
      for (int q = threadIdx.x; q < p.T * 16 * NF; q += Engine::THREADS)
        if (n0 + q % (16 * NF) < N) p.y[q / (16 * NF) * N + n0 + q % (16 * NF)] = 0;
    return;
  }
  if (count == 0) return;
  const int* list = p.tb.pairs + p.tb.offsets[e];
  const int64_t sstep = (p.I + 127) / 128 * (BF == FMT_FP8 ? (N + 127) / 128 : N);
  const uint8_t* w = p.w2 + e * N * ldb;
  const void* sc = static_cast<const uint32_t*>(p.s2) + e * sstep;
  const int rows_b = (int)(N - n0 < 16 * NF ? N - n0 : 16 * NF);
  const StreamOperands o = expert_operands<BF>(w, sc, N, p.I, p.u0, K, n0, rows_b, p.h,
                                               (int64_t)p.T * p.k * kParts * K * 2);
  // a pair takes three neighbouring rows, its h's parts, without gaps between
  // pairs; their sums are added before they leave
  constexpr int kPairs = 16 * MAXNI / kParts;
  for (int c0 = 0; c0 < count; c0 += kPairs) {
    const int rows = kParts * (count - c0 < kPairs ? count - c0 : kPairs);
    with_fragments<MAXNI>(rows, [&](auto ni) {
      constexpr int NI = decltype(ni)::value;
      Engine::template tile<NI>(
          o, K, ldb, rows_b,
          [&](int r) { return r < rows ? kParts * list[c0 + r / kParts] + r % kParts : -1; }, slots,
          [&](int f, const v4f (&t)[NI]) {
            const int64_t n = n0 + 16 * f + 4 * (lane >> 4);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              const int r = 16 * i + fr;
              const v4f next = t[i + 1 < NI ? i + 1 : i];
              v4f s = t[i];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                s[q] += after<1>(t[i][q], next[q], fr) + after<2>(t[i][q], next[q], fr);
              if (r % kParts != 0 || r >= rows || n >= N) continue;
              float* d = p.part + (int64_t)list[c0 + r / kParts] * N + n;
              if (p.u0 > 0) s += *reinterpret_cast<const v4f*>(d);  // of the launch before
              publish4(d, s);
            }
          });
    });
  }
  if (p.u0 + K < p.I) return;
  if (!arrive_last(&p.counters[blockIdx.x], active, &s_last)) return;
  for (int q = threadIdx.x; q < p.T * 4 * NF; q += Engine::THREADS) {
    const int t = q / (4 * NF);
    const int64_t n = n0 + 4 * (q % (4 * NF));
    if (n >= N) continue;
    v4f s = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < p.k; j += 4) {  // four slots in flight: they come from beyond the L2
      v4f v[4];
      bool on[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int slot = t * p.k + (j + u < p.k ? j + u : j);
        const int id = p.ids[slot];
        on[u] = j + u < p.k && id >= 0 && id < p.E;
        v[u] = collect4(p.part + (int64_t)slot * N + n);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (on[u]) s += v[u];
    }
    *reinterpret_cast<uint2*>(p.y + t * N + n) =
        make_uint2(bf16x2_rne(s[0], s[1]), bf16x2_rne(s[2], s[3]));
  }
  if (threadIdx.x == 0)
    __hip_atomic_store(&p.counters[blockIdx.x], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// Bytes of hidden values at a time: with the down product's sums they stay in
// the L2s (32 MiB together), and the workspace of 512 pairs of 4096 x 11008
// stays below 32 MiB.  A chunk then has thousands of units, beside whose weights
// two more launches are little.
constexpr int64_t kMaxHidden = 20 << 20;

struct MoeLayout {
  int64_t chunk;  // hidden units at a time: all, or whole K blocks
  size_t tables, h, part, total;
};
MoeLayout moe_layout(int T, int E, int k, int64_t H, int64_t I) {
  MoeLayout l;
  const int64_t pairs = (int64_t)T * k, bytes = pairs * I * kParts * 2;
  const int64_t chunks = (bytes + kMaxHidden - 1) / kMaxHidden;
  l.chunk = chunks == 1 ? I : ((I + chunks - 1) / chunks + 127) / 128 * 128;
  l.tables = kSplitkCounterBytes;
  l.h = l.tables + up16((size_t)(4 + 2 * E + pairs) * 4);
  l.part = l.h + up16((size_t)pairs * l.chunk * kParts * 2);
  l.total = l.part + (size_t)pairs * H * 4;
  return l;
}

template <int BF, int MAXNI, class Engine>
hipError_t launch_up(const MoeArgs& p, hipStream_t stream) {
  hipLaunchKernelGGL((moe_up_kernel<BF, MAXNI, Engine>),
                     dim3((unsigned)((2 * p.chunk + Engine::ROWS_B - 1) / Engine::ROWS_B), (unsigned)p.E),
                     dim3(Engine::THREADS), 0, stream, p);
  return hipGetLastError();
}
template <int BF, int MAXNI, class Engine>
hipError_t launch_down(const MoeArgs& p, hipStream_t stream) {
  hipLaunchKernelGGL((moe_down_kernel<BF, MAXNI, Engine>),
                     dim3((unsigned)((p.H + Engine::ROWS_B - 1) / Engine::ROWS_B), (unsigned)p.E),
                     dim3(Engine::THREADS), 0, stream, p);
  return hipGetLastError();
}

// Measured on an MI355X, us a layer with the weights from HBM (E4M3, then MXFP4;
// experts as number of H x I), every alternative of a launch with the best of the
// other one.
//
// gate/up: a row a pair.
//  * up to four tokens 32 weight rows a workgroup, up to 16 tokens 64, whose waves
//    read their activations half as often: 125 against 128 (two tokens, 8 of
//    4096 x 11008, E4M3), 77.9 / 77.6 (13 tokens, 60 of 2048 x 1408);
//  * more tokens: activations in LDS, 260 / 273 and 179 / 198 (64 tokens, 8 of
//    4096 x 11008) against two fragments straight from memory; with many small
//    experts that is no loss to speak of (132 / 134, 64 tokens on 60);
//  * 32 rows at a time leave two workgroups a CU (260 / 263, 179 / 187, same
//    layer), but an expert with more rows reads its weights again: 64 at a time
//    where the mean is above 20 rows (260 / 279, 223 / 227 with 64 rows).
//
// down: three rows a pair.
//  * one or two tokens: 32 weight rows a workgroup (68 / 94 and 51 / 69 for one
//    token on 8 of 4096 x 11008); with three or four there are experts enough for
//    128 rows a workgroup, one a CU: 189 / 192 and 131 / 137, 57 / 61 and 44 / 49
//    (four tokens, 32 of 2048 x 2816);
//  * up to six pairs an expert in the mean: 10 at a time, two workgroups a CU or
//    more: 80 / 85 and 60 / 63 (13 tokens, 60 of 2048 x 1408), 160 / 173 and 120 /
//    134 (64 tokens, top 8 of 128 of 2048 x 768), 224 / 224 and 152 / 151 (16
//    tokens, 8 of 4096 x 11008);
//  * more: 32 at a time, 254 / 311 and 166 / 189 (48 tokens, 8 of 4096 x 11008);
//    in MXFP4 up to ten in the mean 16 at a time, which still leaves two
//    workgroups a CU: 99 / 104 (64 tokens, top 4 of 32 of 2048 x 2816), but 200 /
//    179 with 16 in the mean (64 tokens, 8 of 4096 x 11008).
template <int BF>
hipError_t launch_experts(const MoeArgs& p, hipStream_t stream) {
  const int pairs = p.T * p.k;
  hipError_t e;
  if (p.T <= 4)
    e = launch_up<BF, 1, StreamEngine<BF, 2, 1>>(p, stream);
  else if (p.T <= 16)
    e = launch_up<BF, 1, StreamEngine<BF, 4, 1>>(p, stream);
  else if (p.T <= 32 || pairs <= 20 * p.E)
    e = launch_up<BF, 2, SharedEngine<BF, 2>>(p, stream);
  else
    e = launch_up<BF, 4, SharedEngine<BF, 4>>(p, stream);
  if (e != hipSuccess) return e;
  if (p.T <= 2) return launch_down<BF, 1, StreamEngine<BF, 2, 1>>(p, stream);
  if (p.T > 4 && pairs <= 6 * p.E) return launch_down<BF, 2, SharedEngine<BF, 2>>(p, stream);
  if constexpr (BF == FMT_MXFP4)
    if (p.T > 4 && pairs <= 10 * p.E) return launch_down<BF, 3, SharedEngine<BF, 3, 3>>(p, stream);
  return launch_down<BF, 6, SharedEngine<BF, 6>>(p, stream);
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
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  for (p.u0 = 0; p.u0 < p.I; p.u0 += l.chunk) {
    p.chunk = p.I - p.u0 < l.chunk ? p.I - p.u0 : l.chunk;
    e = q.format == FMT_FP8 ? launch_experts<FMT_FP8>(p, stream)
                            : launch_experts<FMT_MXFP4>(p, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace dg
