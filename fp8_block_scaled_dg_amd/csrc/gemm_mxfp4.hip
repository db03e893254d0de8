// MXFP4 NT products for gfx950:
//   C[m][n] = bf16( sum_k A[m][k] B[n][k] ),
// B in MXFP4 (mxfp4_device.hpp), A in MXFP4 or in BF16.
//
// Three kernels for up to 64 rows of A, whose time is the stream of B from HBM
// (1 x 7168 x 16384 in 12.9 us: 4.8 TB/s with the launch in it); larger M goes
// to gemm_mxfp4_tiled.hip.
//
// gemm_mxfp4_stream_kernel: a workgroup's four waves take the same 16 NF rows
// of B and 16 NI rows of A and a quarter each of a run of K; their FP32 sums
// meet in LDS and are added in wave order.  With S > 1 the run is the S-th
// part of K: each part's sums go to the workspace and the last workgroup to
// arrive adds the parts in order, so the result does not depend on which one
// that is.
#include "mxfp4_device.hpp"

namespace dg {
namespace {

constexpr int kWaves = 4;

struct Mxfp4Args {
  uint16_t* c;
  const uint8_t* a;
  const uint8_t* b;
  const uint32_t* sfa;
  const uint32_t* sfb;
  int64_t M, N, K;
  float* partials;  // [tile][S][NF NI][64] quads, when S > 1
  int* counters;
  int S;
};

// Four consecutive outputs of row m from column n (n % 4 == 0), as far as the
// row goes.  A row of C starts at any element, so the wide store is not aligned
// to its size (the memory path takes that).
__device__ __forceinline__ void store_quad(uint16_t* c, int64_t m, int64_t n, int64_t N, v4f t) {
  const uint32_t v[2] = {bf16x2_rne(t[0], t[1]), bf16x2_rne(t[2], t[3])};
  uint16_t* d = c + m * N + n;
  if (n + 4 <= N) {
    __builtin_memcpy(__builtin_assume_aligned(d, 2), v, 8);
    return;
  }
  if (n < N) d[0] = (uint16_t)v[0];
  if (n + 1 < N) d[1] = (uint16_t)(v[0] >> 16);
  if (n + 2 < N) d[2] = (uint16_t)v[1];
}

template <int AF, int NI, int NF, int U>
__global__ void __launch_bounds__(64 * kWaves) gemm_mxfp4_stream_kernel(Mxfp4Args p) {
  constexpr int Q = NF * NI;
  __shared__ v4f red[kWaves][Q][64];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15;
  const int tile_n = (int)(blockIdx.x / (unsigned)p.S);
  const int split = blockIdx.x - tile_n * p.S;
  const int64_t n0 = (int64_t)tile_n * (16 * NF);
  const int rows_b = (int)(p.N - n0 < 16 * NF ? p.N - n0 : 16 * NF);
  const int rows_a = (int)p.M;  // <= 16 NI
  const int64_t ldb = p.K / 2, lda = AF == ACT_BF16 ? p.K * 2 : p.K / 2;
  const int nkb = (int)((p.K + 127) / 128);

  StreamOperands o;
  o.b = buffer_of(p.b + n0 * ldb, rows_b * ldb);
  o.sb = buffer_of(p.sfb + n0, (nkb * p.N - n0) * 4);
  o.sb_step = (uint32_t)p.N * 4;
  o.last = nkb - 1;
  o.a = buffer_of(p.a, rows_a * lda);
  if (AF == ACT_MXFP4) {
    o.sa = buffer_of(p.sfa, nkb * p.M * 4);
    o.sa_step = (uint32_t)p.M * 4;
  }
  Stream<AF, FMT_MXFP4, NI, NF, U> s;
  s.g = lane >> 4;
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int r = 16 * f + fr;
    s.vb[f] = r < rows_b ? (uint32_t)(r * ldb + 16 * s.g) : kOob;
    s.vsb[f] = r < rows_b ? (uint32_t)(4 * r) : kOob;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = 16 * i + fr;
    s.va[i] = r < rows_a ? (uint32_t)(r * lda + (AF == ACT_BF16 ? 64 : 16) * s.g) : kOob;
    s.vsa[i] = r < rows_a ? (uint32_t)(4 * r) : kOob;
  }
  const int parts = p.S * kWaves, part = split * kWaves + wave;
  const int kb0 = run_begin(part, nkb, parts), kb1 = run_begin(part + 1, nkb, parts);
  const int kmax = kb1 * 128 < p.K ? kb1 * 128 : (int)p.K;

  v4f acc[NF][NI];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[f][i] = v4f{0.f, 0.f, 0.f, 0.f};
  s.run(o, kb0, kb1, kmax, acc);

#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < NI; ++i) red[wave][f * NI + i][lane] = acc[f][i];
  __syncthreads();

  const int tile = tile_n;
  auto sum_waves = [&](int q) {
    v4f t = red[0][q][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) t += red[w][q][lane];
    return t;
  };
  auto store = [&](int q, v4f t) {
    const int f = q / NI, i = q - f * NI;
    const int64_t m = 16 * i + fr;
    if (m < p.M) store_quad(p.c, m, n0 + 16 * f + 4 * s.g, p.N, t);
  };
  if (p.S == 1) {
    for (int q = wave; q < Q; q += kWaves) store(q, sum_waves(q));
    return;
  }
  float* part0 = p.partials + (int64_t)tile * p.S * (Q * 256);
  for (int q = wave; q < Q; q += kWaves)
    publish4(part0 + split * (Q * 256) + (q * 64 + lane) * 4, sum_waves(q));
  if (!arrive_last(&p.counters[tile], p.S, &s_last)) return;
  v4f t[(Q + kWaves - 1) / kWaves];
#pragma unroll
  for (int u = 0; u < (Q + kWaves - 1) / kWaves; ++u) {
    const int q = wave + u * kWaves;
    if (q < Q) t[u] = collect_sum(part0 + (q * 64 + lane) * 4, Q * 256, p.S);
  }
#pragma unroll
  for (int u = 0; u < (Q + kWaves - 1) / kWaves; ++u) {
    const int q = wave + u * kWaves;
    if (q < Q) store(q, t[u]);
  }
  if (threadIdx.x == 0)  // zero again for the next call
    __hip_atomic_store(&p.counters[tile], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// MXFP4 activations, both operands through LDS: four waves with the same 32
// rows of B and 16 NI rows of A and a quarter of K each, every wave with a ring
// of its own (R stages of 256 K values, R - 1 in flight), so no barrier sits in
// the loop.  The DMA reads whole 128-byte lines of eight rows an instruction;
// loads straight into fragments touch 16 rows 16 bytes at a time, four times
// as many accesses, which is what bounds them from 17 rows of A on.
template <int NI>
struct Ring {
  static constexpr int R = NI <= 2 ? 4 : 3, NF = 2;
  static constexpr int ROWS = 16 * (NF + NI);           // of B, then of A
  static constexpr int SCALES = ROWS * 128;             // words [2][32] of B, [2][64] of A
  static constexpr int SLOT = SCALES + 256 + 512;       // bytes of a wave's stage
  static constexpr int DMAS = ROWS / 8, LOADS = DMAS + 3;
  static_assert((R - 1) * LOADS <= 63, "range of the counter");
};

template <int NI>
__global__ void __launch_bounds__(64 * kWaves) gemm_mxfp4_ring_kernel(Mxfp4Args p) {
  typedef Ring<NI> S;
  constexpr int R = S::R, NF = S::NF, Q = NF * NI;
  // variables of their own: a read of one is not taken to depend on a transfer
  // into another
  __shared__ __attribute__((aligned(1024))) uint8_t slot0[kWaves * S::SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t slot1[kWaves * S::SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t slot2[kWaves * S::SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t slot3[R > 3 ? kWaves * S::SLOT : 16];
  uint8_t* const slots[4] = {slot0, slot1, slot2, slot3};
  static_assert(Q * 1024 <= S::SLOT, "the waves' sums meet in slot 0");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NF);
  const int rows_b = (int)(p.N - n0 < 16 * NF ? p.N - n0 : 16 * NF), rows_a = (int)p.M;
  const int64_t ld = p.K / 2;
  const int nkb = (int)((p.K + 127) / 128), nk = (int)((p.K + 255) / 256);
  const __amdgpu_buffer_rsrc_t rb = buffer_of(p.b + n0 * ld, rows_b * ld);
  const __amdgpu_buffer_rsrc_t ra = buffer_of(p.a, rows_a * ld);
  const __amdgpu_buffer_rsrc_t rsb = buffer_of(p.sfb + n0, (nkb * p.N - n0) * 4);
  const __amdgpu_buffer_rsrc_t rsa = buffer_of(p.sfa, nkb * p.M * 4);
  const uint32_t step_b = (uint32_t)p.N * 4, step_a = (uint32_t)p.M * 4;
  const int kb0 = run_begin(wave, nk, kWaves), kb1 = run_begin(wave + 1, nk, kWaves);
  const int kmax = kb1 * 256 < p.K ? kb1 * 256 : (int)p.K;

  // 16-byte chunk c of LDS row r sits at c ^ swz(r): with chunk 4h + g read by
  // lane 16g + r, each group of 16 lanes that a 16-byte read serves at a time
  // (0-3, 12-15, 20-27, ...) has 16 different slots of a sweep of the banks
  auto swz = [](int r) { return (r & 2) | ((r >> 1) & 4); };
  uint32_t off[S::DMAS];
  int chunk_k[2];  // first K value of this lane's chunk, rows 0-7 and 8-15 of 16
#pragma unroll
  for (int e = 0; e < 2; ++e) chunk_k[e] = 32 * ((lane & 7) ^ swz(8 * e + (lane >> 3)));
#pragma unroll
  for (int j = 0; j < S::DMAS; ++j) {
    const int r = 8 * j + (lane >> 3) - (j < 2 * NF ? 0 : 16 * NF);
    off[j] = r < (j < 2 * NF ? rows_b : rows_a) ? (uint32_t)(r * ld + chunk_k[j & 1] / 2) : kOob;
  }
  // scale words: B's two K blocks of 32 rows in one instruction, A's in two of 64
  const uint32_t osb = (lane & 31) < rows_b ? (uint32_t)(4 * (lane & 31)) : kOob;
  const uint32_t osa = lane < rows_a ? (uint32_t)(4 * lane) : kOob;

  auto load = [&](uint8_t* slot, int kb) {
    uint8_t* st = slot + wave * S::SLOT;
    const int soff = kb < kb1 ? kb * 128 : 0;  // no scalar offset past a resource
    const bool in[2] = {kb * 256 + chunk_k[0] < kmax, kb * 256 + chunk_k[1] < kmax};
    auto dma4 = [&](__amdgpu_buffer_rsrc_t r, int at, uint32_t v, uint32_t s) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          r, (__attribute__((address_space(3))) void*)(st + at), 4, (int)v, (int)s, 0, 0);
    };
#pragma unroll
    for (int j = 0; j < S::DMAS; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          j < 2 * NF ? rb : ra, (__attribute__((address_space(3))) void*)(st + j * 1024), 16,
          (int)(in[j & 1] ? off[j] : kOob), soff, 0, 0);
    const int w0 = 2 * kb, w1 = 2 * kb + 1;
    const bool on0 = kb < kb1 && w0 < nkb, on1 = kb < kb1 && w1 < nkb;
    // the second K block's words of B lie step_b further
    const bool onb = lane < 32 ? on0 : on1;
    dma4(rsb, S::SCALES, onb && osb != kOob ? osb + (lane < 32 ? 0u : step_b) : kOob,
        on0 ? w0 * step_b : 0u);
    dma4(rsa, S::SCALES + 256, on0 ? osa : kOob, on0 ? w0 * step_a : 0u);
    dma4(rsa, S::SCALES + 512, on1 ? osa : kOob, on1 ? w1 * step_a : 0u);
  };

  v4f acc[NF][NI];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[f][i] = v4f{0.f, 0.f, 0.f, 0.f};
  static_for<R - 1>([&](auto j) {
    load(slots[decltype(j)::value], kb0 + decltype(j)::value);
    __builtin_amdgcn_sched_barrier(0);
  });
  auto stage = [&](auto jc, int kb) {
    constexpr int j = decltype(jc)::value, nx = (j + R - 1) % R;
    __builtin_amdgcn_sched_barrier(0);
    // all but the R - 2 newest stages have landed; the slot to fill has been read
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((R - 2) * S::LOADS) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    load(slots[nx], kb + R - 1);
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* st = slots[j] + wave * S::SLOT;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // exponent bytes of this lane's 32-block; 0 past K, where the codes are 0
      const int width = kb * 256 + h * 128 + 32 * g < kmax ? 8 : 0;
      auto frag = [&](int row) {
        const v4i q = *reinterpret_cast<const v4i*>(st + (row + fr) * 128 + 16 * ((4 * h + g) ^ swz(fr)));
        return v8i{q[0], q[1], q[2], q[3], 0, 0, 0, 0};
      };
      auto exponent = [&](int at) {
        return (int)__builtin_amdgcn_ubfe(*reinterpret_cast<const uint32_t*>(st + S::SCALES + at + 4 * fr),
                                          8 * g, width);
      };
      v8i bq[NF];
      int eb[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        bq[f] = frag(16 * f);
        eb[f] = exponent(128 * h + 64 * f);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const v8i aq = frag(16 * (NF + i));
        const int ea = exponent(256 + 256 * h + 64 * i);
#pragma unroll
        for (int f = 0; f < NF; ++f)
          acc[f][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bq[f], aq, acc[f][i], 4, 4, 0,
                                                                       eb[f], 0, ea);
      }
    }
  };
  int kb = kb0;
  for (; kb + R <= kb1; kb += R)
    static_for<R>([&](auto j) { stage(j, kb + decltype(j)::value); });
  static_for<R - 1>([&](auto j) {
    if (kb + decltype(j)::value < kb1) stage(j, kb + decltype(j)::value);
  });
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __syncthreads();
  v4f* red = reinterpret_cast<v4f*>(slot0);
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < NI; ++i) red[(wave * Q + f * NI + i) * 64 + lane] = acc[f][i];
  __syncthreads();
  for (int q = wave; q < Q; q += kWaves) {
    v4f t = red[q * 64 + lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) t += red[(w * Q + q) * 64 + lane];
    const int64_t m = 16 * (q % NI) + fr;
    if (m < p.M) store_quad(p.c, m, n0 + 16 * (q / NI) + 4 * g, p.N, t);
  }
}

// BF16 activations in LDS (Shared, mxfp4_device.hpp): 128 rows of B a
// workgroup, eight waves.
template <int NI>
using SharedProduct = Shared<FMT_MXFP4, NI, shared_depth(FMT_MXFP4, NI)>;

template <int NI>
__global__ void __launch_bounds__(kSharedThreads, (SharedProduct<NI>::WAVES))
gemm_mxfp4_shared_kernel(Mxfp4Args p) {
  typedef SharedProduct<NI> S;
  constexpr int QT = S::ROWS_B / 16 * NI;
  DG_SHARED_SLOTS(S);
  __shared__ int s_last;
  const int tile = (int)(blockIdx.x / (unsigned)p.S);
  const int split = blockIdx.x - tile * p.S;
  const int64_t n0 = (int64_t)tile * S::ROWS_B;
  const int rows_b = (int)(p.N - n0 < S::ROWS_B ? p.N - n0 : S::ROWS_B);
  const int rows_a = (int)p.M;
  const int64_t ldb = p.K / 2, lda = p.K * 2;
  const int nkb = (int)((p.K + 127) / 128);
  StreamOperands o;
  o.b = buffer_of(p.b + n0 * ldb, rows_b * ldb);
  o.sb = buffer_of(p.sfb + n0, (nkb * p.N - n0) * 4);
  o.sb_step = (uint32_t)p.N * 4;
  o.last = nkb - 1;
  o.a = buffer_of(p.a, rows_a * lda);
  S s;
  s.init(ldb, rows_b, lda, [&](int r) { return r < rows_a ? r : -1; });
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto store = [&](int f, int i, v4f t) {
    const int64_t m = 16 * i + (lane & 15);
    if (m < p.M) store_quad(p.c, m, n0 + 16 * f + 4 * (lane >> 4), p.N, t);
  };
  float* part0 = p.partials + (int64_t)tile * p.S * (QT * 256);
  s.run(o, p.K, split * S::WK, p.S * S::WK, slots, [&](int f, const v4f (&t)[NI]) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (p.S == 1) store(f, i, t[i]);
      else publish4(part0 + split * (QT * 256) + ((f * NI + i) * 64 + lane) * 4, t[i]);
  });
  if (p.S == 1) return;
  if (!arrive_last(&p.counters[tile], p.S, &s_last)) return;
  // this wave's quads of all parts, four parts in flight
  v4f t[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) t[i] = v4f{0.f, 0.f, 0.f, 0.f};
  const float* mine = part0 + (wave * NI * 64 + lane) * 4;
  for (int sp = 0; sp < p.S; sp += 4) {
    v4f v[4][NI];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < NI; ++i)
        v[u][i] = collect4(mine + (sp + u < p.S ? sp + u : sp) * (QT * 256) + i * 256);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (sp + u < p.S) t[i] += v[u][i];
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) store(wave, i, t[i]);
  if (threadIdx.x == 0)
    __hip_atomic_store(&p.counters[tile], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Kernel, rows of A and B per workgroup and K parts for a shape.
enum Kernel { STREAM, SHARED, RING };
struct StreamPlan {
  Kernel kernel;
  int ni, nf, S, u;  // S parts of K
  int64_t tiles_n;
};

// Measured on an MI355X, us, every call with weights of its own, 1.2 GB in all
// (M x N x K):
//  * MXFP4 activations, K from 16 stages of 256 on and 100 workgroups: rings in
//    LDS, 12.9 against 15.9 (1 x 7168 x 16384), 17.8 / 24.6 (33) and 22.0 / 31
//    (64), 11.1 / 13.8 (64 x 4096 x 8192); shorter runs do not pay for one
//    workgroup a CU: 7.6 / 6.1 (40 x 16384 x 1024), 3.4 / 3.2 (4 x 2048 x
//    2048), nor do few columns: 8.4 / 7.0 (64 x 512 x 8192, which splits K).
//  * BF16 activations in LDS from 17 rows on, where N gives workgroups enough:
//    27 against 73 (33 x 7168 x 16384), 9.7 / 13.4 (20 x 24576 x 1536), 13.6 /
//    43 (64 x 24576 x 1536); up to 16 rows straight into fragments: 18.7 / 22
//    (1 x 7168 x 16384), 5.9 / 7.8 (16 x 7168 x 2048), and for few columns
//    9.9 / 15.8 (64 x 512 x 8192).
//  * 32 rows of B a workgroup where that leaves 192 workgroups, else 16: 5.9 /
//    7.5 (16 x 7168 x 2048, BF16), but 7.1 / 6.2 (8 x 4096 x 4096, BF16).
//  * BF16, two K blocks a buffer for long runs of few rows: 18.7 / 19.6 (1 x
//    7168 x 16384); 8.9 / 8.3 on short ones (1 x 24576 x 1536).
//  * K parts cost about 4 us, so they have to save more: 7.0 / 11.6 in four
//    (64 x 512 x 8192, MXFP4); with LDS 27 / 61 in four (33 x 7168 x 16384),
//    but 26.5 / 13.6 in two (64 x 24576 x 1536: 192 workgroups already).
StreamPlan stream_plan(int64_t M, int64_t N, int64_t K, bool bf16_a) {
  StreamPlan s;
  const int64_t nkb = (K + 127) / 128;
  s.ni = (int)((M + 15) / 16);
  s.kernel = STREAM;
  s.S = 1;
  s.u = 1;
  if (bf16_a && M > 16 && N >= 2048) {
    s.kernel = SHARED;
    s.nf = 8;
    s.tiles_n = (N + 127) / 128;
    while (s.tiles_n * 2 * s.S <= 256 && nkb / (4 * s.S) >= 4 && s.S < 16) s.S *= 2;
    return s;
  }
  if (!bf16_a && nkb >= 32 && (N + 31) / 32 >= 100) {
    s.kernel = RING;
    s.nf = 2;
    s.tiles_n = (N + 31) / 32;
    return s;
  }
  s.nf = (N + 31) / 32 >= 192 ? 2 : 1;
  if (bf16_a && s.nf == 2 && s.ni == 1 && nkb >= 64) s.u = 2;
  s.tiles_n = (N + 16 * s.nf - 1) / (16 * s.nf);
  while (s.tiles_n * s.S < 256 && nkb / (kWaves * s.S) >= 8 && s.S < 16) s.S *= 2;
  return s;
}

template <int AF, int NI, int NF, int U>
hipError_t launch_stream(const Mxfp4Args& p, const StreamPlan& s, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_mxfp4_stream_kernel<AF, NI, NF, U>), dim3((unsigned)(s.tiles_n * p.S)),
                     dim3(64 * kWaves), 0, stream, p);
  return hipGetLastError();
}
template <int NI>
hipError_t launch_shared(const Mxfp4Args& p, const StreamPlan& s, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_mxfp4_shared_kernel<NI>), dim3((unsigned)(s.tiles_n * p.S)),
                     dim3(kSharedThreads), 0, stream, p);
  return hipGetLastError();
}
template <int NI>
hipError_t launch_ring(const Mxfp4Args& p, const StreamPlan& s, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_mxfp4_ring_kernel<NI>), dim3((unsigned)s.tiles_n), dim3(64 * kWaves), 0,
                     stream, p);
  return hipGetLastError();
}
template <int AF, int NI>
hipError_t launch_rows(const Mxfp4Args& p, const StreamPlan& s, hipStream_t stream) {
  if constexpr (AF == ACT_BF16 && NI > 1) {
    if (s.kernel == SHARED) return launch_shared<NI>(p, s, stream);
    return launch_stream<AF, NI, 1, 1>(p, s, stream);
  } else {
    if constexpr (AF == ACT_MXFP4)
      if (s.kernel == RING) return launch_ring<NI>(p, s, stream);
    if constexpr (AF == ACT_BF16)
      if (s.u == 2) return launch_stream<AF, NI, 2, 2>(p, s, stream);
    if (s.nf == 2) return launch_stream<AF, NI, 2, 1>(p, s, stream);
    return launch_stream<AF, NI, 1, 1>(p, s, stream);
  }
}
template <int AF>
hipError_t launch_ni(const Mxfp4Args& p, const StreamPlan& s, hipStream_t stream) {
  if (s.ni == 1) return launch_rows<AF, 1>(p, s, stream);
  if (s.ni == 2) return launch_rows<AF, 2>(p, s, stream);
  if (s.ni == 3) return launch_rows<AF, 3>(p, s, stream);
  return launch_rows<AF, 4>(p, s, stream);
}

size_t plan_bytes(const StreamPlan& s) {
  if (s.S == 1) return 0;
  return kSplitkCounterBytes + (size_t)s.tiles_n * s.S * s.ni * s.nf * 1024;
}

}  // namespace

size_t mxfp4_workspace_bytes(int64_t M, int64_t N, int64_t K, bool bf16_a) {
  if (M > 64) return bf16_a ? 0 : mxfp4_tiled_workspace_bytes(M, N, K);
  return plan_bytes(stream_plan(M, N, K, bf16_a));
}

hipError_t launch_gemm_mxfp4(const Mxfp4Problem& q, void* workspace, size_t workspace_bytes,
                             hipStream_t stream) {
  if (q.M > 64) return launch_gemm_mxfp4_tiled(q, workspace, workspace_bytes, stream);
  Mxfp4Args p;
  p.c = q.c;
  p.a = static_cast<const uint8_t*>(q.a);
  p.b = q.b;
  p.sfa = q.sfa;
  p.sfb = q.sfb;
  p.M = q.M;
  p.N = q.N;
  p.K = q.K;
  StreamPlan s = stream_plan(q.M, q.N, q.K, q.sfa == nullptr);
  if (workspace_bytes < plan_bytes(s)) s.S = 1;
  p.S = s.S;
  p.counters = static_cast<int*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + kSplitkCounterBytes);
  return q.sfa ? launch_ni<ACT_MXFP4>(p, s, stream) : launch_ni<ACT_BF16>(p, s, stream);
}

}  // namespace dg
