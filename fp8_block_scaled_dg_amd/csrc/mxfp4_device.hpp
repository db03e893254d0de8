// Device-side helpers shared by the MXFP4 and mixture-of-experts kernels.
//
// MXFP4 as stored here: E2M1 codes (magnitudes 0 .5 1 1.5 2 3 4 6, bit 3 the
// sign), element k of a row in nibble k % 2 of byte k / 2, and one E8M0
// exponent byte per 32 elements of a row (value 2^(byte - 127), 255 = NaN),
// four bytes in an int32, K-block-major: sf[ceil(K / 128)][rows].
#pragma once

#include "dg_device.hpp"

namespace dg {

typedef __bf16 dg_bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t v4u32 __attribute__((ext_vector_type(4)));

enum { FMT_MXFP4 = 0, FMT_FP8 = 1 };  // weight formats
enum { ACT_MXFP4 = 0, ACT_BF16 = 1 };  // activation formats

// Buffer resource over [base, base + bytes): loads past the end return zero
// and touch no memory.  kOob is an offset past every resource made here
// (their sizes stay below 2^31), so a masked lane or row costs one select.
constexpr uint32_t kOob = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, (int)soff, 0));
}
__device__ __forceinline__ uint32_t load4(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, (int)voff, (int)soff, 0);
}

// 32 E2M1 codes (16 bytes) times 2^(e - 127), e the low byte of `e`, as 4 x 8
// BF16: exact (at most two significant bits) down to BF16's subnormals; e =
// 255 gives NaN.  The conversion reads only the exponent field of its scale
// operand, so the E8M0 byte goes there as it is (checked on an MI355X for all
// 256 code pairs at scales 2^-127, 2^-126, 1, 2^127 and NaN).
__device__ __forceinline__ void widen_mxfp4(v4i q, uint32_t e, dg_bf16x8 (&out)[4]) {
  const float s = __uint_as_float((e & 0xFFu) << 23);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = (uint32_t)q[j];
    const dg_bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    const dg_bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    const dg_bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    const dg_bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    out[j] = dg_bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
  }
}

// 32 E4M3 codes (32 bytes) as 4 x 8 BF16: exact (four significant bits).
__device__ __forceinline__ void widen_fp8(v4i lo, v4i hi, dg_bf16x8 (&out)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w0 = (uint32_t)(j < 2 ? lo[2 * j] : hi[2 * j - 4]);
    const uint32_t w1 = (uint32_t)(j < 2 ? lo[2 * j + 1] : hi[2 * j - 3]);
    const dg_bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
    const dg_bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
    const dg_bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
    const dg_bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
    out[j] = dg_bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
  }
}

// FP32 quads published to, and read from, the level that all XCDs share (each
// has its own L2): relaxed device-scope atomics are written through without a
// write-back of the whole L2.
__device__ __forceinline__ void publish4(float* d, v4f v) {
  uint64_t* p = reinterpret_cast<uint64_t*>(d);
  const uint64_t lo = (uint64_t)__float_as_uint(v[0]) | ((uint64_t)__float_as_uint(v[1]) << 32);
  const uint64_t hi = (uint64_t)__float_as_uint(v[2]) | ((uint64_t)__float_as_uint(v[3]) << 32);
  __hip_atomic_store(p, lo, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(p + 1, hi, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ v4f collect4(const float* s) {
  uint64_t* p = reinterpret_cast<uint64_t*>(const_cast<float*>(s));
  const uint64_t lo = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint64_t hi = __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return v4f{__uint_as_float((uint32_t)lo), __uint_as_float((uint32_t)(lo >> 32)),
             __uint_as_float((uint32_t)hi), __uint_as_float((uint32_t)(hi >> 32))};
}

// True in the workgroup that arrives last of `count` at *counter (zero before
// the first arrival; the caller resets it).  Every wave's stores are complete
// before its workgroup arrives.
__device__ __forceinline__ bool arrive_last(int* counter, int count, int* s_last) {
  __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xF << 8));  // vmcnt(0)
  __syncthreads();
  if (threadIdx.x == 0)
    *s_last = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
              count - 1;
  __syncthreads();
  return *s_last != 0;
}

// What one wave multiplies: 16 NF rows of a weight matrix with 16 NI rows of
// activations over a run of 128-wide K blocks.  Rows of the weight start at
// resource b (row stride b_ld bytes), its scales at sb.
struct StreamOperands {
  __amdgpu_buffer_rsrc_t b, sb, a, sa;
  uint32_t sb_step;  // bytes between the scales of one K block and the next
  uint32_t sa_step;
};

// Both operands go from memory straight into the matrix instruction's layout
// (lane l: row l % 16, the 32 K values of group l / 16), so no LDS or barrier
// sits in the loop; U K blocks are in flight while U others are multiplied.
// Weight rows drive the instruction's first operand, so a lane ends with four
// consecutive outputs n = 16f + 4 (l / 16) + r of activation row 16i + l % 16.
//
// A 32-wide block whose first column is at kmax or past it (the end of K, or
// of this wave's run) is read as zero codes with a zero scale byte, whatever
// the bytes behind it hold.
template <int AF, int BF, int NI, int NF, int U>
struct Stream {
  static constexpr int BV = BF == FMT_FP8 ? 2 : 1;
  static constexpr int AV = AF == ACT_BF16 ? 4 : 1;
  struct Buf {
    v4i b[U][NF][BV];
    uint32_t sb[U][BF == FMT_FP8 ? 1 : NF];
    v4i a[U][NI][AV];
    uint32_t sa[U][AF == ACT_BF16 ? 1 : NI];
  };
  uint32_t vb[NF], vsb[NF], va[NI], vsa[NI];  // lane offsets (kOob: no such row)
  int g;                                      // 32-wide block of the K block

  __device__ __forceinline__ void load(const StreamOperands& o, Buf& x, int kb, int kmax) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = (kb + u) * 128 + 32 * g < kmax;
      const uint32_t k = (uint32_t)(kb + u);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const uint32_t v = in ? vb[f] : kOob;
#pragma unroll
        for (int h = 0; h < BV; ++h) x.b[u][f][h] = load16(o.b, v + 16 * h, k * (64 * BV));
        if (BF == FMT_MXFP4) x.sb[u][f] = load4(o.sb, in ? vsb[f] : kOob, k * o.sb_step);
      }
      if (BF == FMT_FP8) x.sb[u][0] = load4(o.sb, in ? 0u : kOob, k * o.sb_step);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint32_t v = in ? va[i] : kOob;
#pragma unroll
        for (int h = 0; h < AV; ++h) x.a[u][i][h] = load16(o.a, v + 16 * h, k * (64 * AV));
        if (AF == ACT_MXFP4) x.sa[u][i] = load4(o.sa, in ? vsa[i] : kOob, k * o.sa_step);
      }
    }
  }

  __device__ __forceinline__ void multiply(const Buf& x, v4f (&acc)[NF][NI]) const {
    const int sh = 8 * g;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (AF == ACT_MXFP4) {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const v4i q = x.b[u][f][0];
          const v8i bq = {q[0], q[1], q[2], q[3], 0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const v4i p = x.a[u][i][0];
            const v8i aq = {p[0], p[1], p[2], p[3], 0, 0, 0, 0};
            acc[f][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                bq, aq, acc[f][i], 4, 4, 0, (int)(x.sb[u][f] >> sh), 0, (int)(x.sa[u][i] >> sh));
          }
        }
      } else {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          dg_bf16x8 bw[4];
          if constexpr (BF == FMT_FP8)
            widen_fp8(x.b[u][f][0], x.b[u][f][1], bw);
          else
            widen_mxfp4(x.b[u][f][0], x.sb[u][f] >> sh, bw);
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            v4f t = BF == FMT_FP8 ? v4f{0.f, 0.f, 0.f, 0.f} : acc[f][i];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  bw[j], __builtin_bit_cast(dg_bf16x8, x.a[u][i][j]), t, 0, 0, 0);
            if constexpr (BF == FMT_FP8)
              acc[f][i] += t * __uint_as_float(x.sb[u][0]);  // the block's FP32 scale
            else
              acc[f][i] = t;
          }
        }
      }
    }
  }

  __device__ __forceinline__ void run(const StreamOperands& o, int kb0, int kb1, int kmax,
                                      v4f (&acc)[NF][NI]) const {
    Buf x0, x1;
    load(o, x0, kb0, kmax);
    for (int kb = kb0; kb < kb1; kb += 2 * U) {
      // the fences keep every load of a buffer ahead of the products of the
      // other one; left to itself the scheduler sinks the loads among the
      // products and the loop waits for memory with nothing in flight
      load(o, x1, kb + U, kmax);
      __builtin_amdgcn_sched_barrier(0);
      multiply(x0, acc);
      __builtin_amdgcn_sched_barrier(0);
      load(o, x0, kb + 2 * U, kmax);
      __builtin_amdgcn_sched_barrier(0);
      multiply(x1, acc);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// Row r of the activations, 16-byte chunk c of its 256 (BF16) or 128 (MXFP4)
// bytes in LDS: the slot that keeps both the fragment reads (lane 16g + r
// reads chunk 4g + j, or 4h + g, of row r; served in the groups of lanes that
// a 16-byte read has) and the row-wise writes off each other's banks.
template <int AF>
__device__ __forceinline__ int act_slot(int r, int c) {
  if (AF == ACT_BF16) return c ^ ((r & 3) | ((r & 8) ? 12 : 0));
  return c ^ ((r & 2) | ((r >> 1) & 4));
}

// The same product with the activations staged in LDS, for more than a few of
// their rows: read straight into fragments they cost, per K block, NI / NF
// times the weight's bytes and more requests than bytes (a fragment's 16 rows
// are 16 pieces of 64 bytes).  Eight waves: WK = 4 runs of K, and in each run
// two waves with 16 NF weight rows each, which share the run's activations.
// A stage is KS K blocks.  Activations go memory -> registers -> LDS one stage
// ahead of their use (full rows, 256 or 128 bytes each), weights straight into
// registers one stage ahead.
constexpr int kSharedThreads = 512;
template <int AF, int BF, int NI, int NF, int KS>
struct Shared {
  static constexpr int WK = 4, WN = 2, BV = BF == FMT_FP8 ? 2 : 1;
  static constexpr int MP = 16 * NI;
  static constexpr int ROW = AF == ACT_BF16 ? 256 : 128;        // bytes of an LDS row
  static constexpr int TILES = AF == ACT_BF16 ? KS : KS / 2;    // LDS tiles of MP rows a stage
  static constexpr int LPR = ROW / 16;                          // lanes per row
  static constexpr int RPI = 64 * WN / LPR;                     // rows per load of the two waves
  static constexpr int IT = (MP + RPI - 1) / RPI;
  static constexpr int STAGE = TILES * MP * ROW;                // bytes of a run's stage
  static constexpr int LDS = 2 * WK * STAGE > 8 * NF * NI * 1024 ? 2 * WK * STAGE
                                                                  : 8 * NF * NI * 1024;
  static_assert(AF == ACT_BF16 || KS % 2 == 0, "MXFP4 stages are pairs of K blocks");
  struct B {
    v4i b[KS][NF][BV];
    uint32_t sb[KS][BF == FMT_FP8 ? 1 : NF];
    uint32_t sa[KS][AF == ACT_BF16 ? 1 : NI];
  };
  struct A {
    v4i v[TILES][IT];
  };
  uint32_t vb[NF], vsb[NF], vsa[NI], va[IT];
  int lane, wave, wk, wn, g;

  // row_of(r): activation row of the tile's row r, or -1
  template <class Rows>
  __device__ __forceinline__ void init(int64_t ldb, int rows_b, int64_t lda, Rows&& row_of) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wn = wave & 1;
    wk = wave >> 1;
    g = lane >> 4;
    const int fr = lane & 15;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int r = 16 * (NF * wn + f) + fr;
      vb[f] = r < rows_b ? (uint32_t)(r * ldb + 16 * BV * g) : kOob;
      vsb[f] = r < rows_b ? (uint32_t)(4 * r) : kOob;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = row_of(16 * i + fr);
      vsa[i] = r >= 0 ? (uint32_t)(4 * r) : kOob;
    }
    const int t = wn * 64 + lane;
#pragma unroll
    for (int j = 0; j < IT; ++j) {
      const int r = j * RPI + t / LPR;
      const int a = r < MP ? row_of(r) : -1;
      va[j] = a >= 0 ? (uint32_t)(a * lda + 16 * (t % LPR)) : kOob;
    }
  }

  __device__ __forceinline__ void load_b(const StreamOperands& o, B& x, int kb, int kmax) const {
#pragma unroll
    for (int u = 0; u < KS; ++u) {
      const bool in = (kb + u) * 128 + 32 * g < kmax;
      const uint32_t k = (uint32_t)(kb + u);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const uint32_t v = in ? vb[f] : kOob;
#pragma unroll
        for (int h = 0; h < BV; ++h) x.b[u][f][h] = load16(o.b, v + 16 * h, k * (64 * BV));
        if (BF == FMT_MXFP4) x.sb[u][f] = load4(o.sb, in ? vsb[f] : kOob, k * o.sb_step);
      }
      if (BF == FMT_FP8) x.sb[u][0] = load4(o.sb, in ? 0u : kOob, k * o.sb_step);
      if (AF == ACT_MXFP4) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
          x.sa[u][i] = load4(o.sa, in ? vsa[i] : kOob, k * o.sa_step);
      }
    }
  }
  __device__ __forceinline__ void load_a(const StreamOperands& o, A& x, int kb, int kmax) const {
    const int c = (wn * 64 + lane) % LPR;
    constexpr int TK = AF == ACT_BF16 ? 128 : 256, CK = TK / LPR;  // K of a tile, of a chunk
#pragma unroll
    for (int u = 0; u < TILES; ++u) {
      const bool in = kb * 128 + u * TK + c * CK < kmax;
#pragma unroll
      for (int j = 0; j < IT; ++j)
        x.v[u][j] = load16(o.a, in ? va[j] : kOob,
                           (uint32_t)kb * (AF == ACT_BF16 ? 256 : 64) + u * ROW);
    }
  }
  __device__ __forceinline__ void store_a(const A& x, uint8_t* st) const {
    const int t = wn * 64 + lane, c = t % LPR;
#pragma unroll
    for (int u = 0; u < TILES; ++u)
#pragma unroll
      for (int j = 0; j < IT; ++j) {
        const int r = j * RPI + t / LPR;
        if (MP % RPI == 0 || r < MP)
          *reinterpret_cast<v4i*>(st + (u * MP + r) * ROW + 16 * act_slot<AF>(r, c)) = x.v[u][j];
      }
  }
  __device__ __forceinline__ v4i frag(const uint8_t* st, int tile, int i, int c) const {
    const int fr = lane & 15;
    return *reinterpret_cast<const v4i*>(st + (tile * MP + 16 * i + fr) * ROW +
                                         16 * act_slot<AF>(fr, c));
  }
  __device__ __forceinline__ void multiply(const B& x, const uint8_t* st,
                                           v4f (&acc)[NF][NI]) const {
    const int sh = 8 * g;
#pragma unroll
    for (int u = 0; u < KS; ++u) {
      if constexpr (AF == ACT_MXFP4) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const v4i q = frag(st, u >> 1, i, 4 * (u & 1) + g);
          const v8i aq = {q[0], q[1], q[2], q[3], 0, 0, 0, 0};
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            const v4i p = x.b[u][f][0];
            const v8i bq = {p[0], p[1], p[2], p[3], 0, 0, 0, 0};
            acc[f][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                bq, aq, acc[f][i], 4, 4, 0, (int)(x.sb[u][f] >> sh), 0, (int)(x.sa[u][i] >> sh));
          }
        }
      } else {
        dg_bf16x8 bw[NF][4];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          if constexpr (BF == FMT_FP8)
            widen_fp8(x.b[u][f][0], x.b[u][f][1], bw[f]);
          else
            widen_mxfp4(x.b[u][f][0], x.sb[u][f] >> sh, bw[f]);
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          dg_bf16x8 aw[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            aw[j] = __builtin_bit_cast(dg_bf16x8, frag(st, u, i, 4 * g + j));
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            v4f t = BF == FMT_FP8 ? v4f{0.f, 0.f, 0.f, 0.f} : acc[f][i];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bw[f][j], aw[j], t, 0, 0, 0);
            if constexpr (BF == FMT_FP8)
              acc[f][i] += t * __uint_as_float(x.sb[u][0]);
            else
              acc[f][i] = t;
          }
        }
      }
    }
  }

  // K blocks of part wk of `parts` runs; every wave of the workgroup makes the
  // same number of stages (the barriers), past its run on zeros.
  // finish(f, i, quad): f in [0, WN NF), each fragment by the wave that owns it.
  template <class Finish>
  __device__ __forceinline__ void run(const StreamOperands& o, int64_t K, int part0, int parts,
                                      uint8_t* lds, Finish&& finish) {
    const int nkb = (int)((K + 127) / 128);
    const int part = part0 + wk;
    const int kb0 = (int)((int64_t)part * nkb / parts);
    const int kb1 = (int)((int64_t)(part + 1) * nkb / parts);
    const int kmax = kb1 * 128 < K ? kb1 * 128 : (int)K;
    const int stages = ((nkb + parts - 1) / parts + KS - 1) / KS;  // of the longest run
    uint8_t* s0 = lds + wk * (2 * STAGE);
    uint8_t* s1 = s0 + STAGE;
    v4f acc[NF][NI];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[f][i] = v4f{0.f, 0.f, 0.f, 0.f};
    A a;
    B b0, b1;
    load_a(o, a, kb0, kmax);
    load_b(o, b0, kb0, kmax);
    store_a(a, s0);
    load_a(o, a, kb0 + KS, kmax);
    __syncthreads();
    auto stage = [&](const B& cur, B& nxt, const uint8_t* rd, uint8_t* wr, int kb) {
      load_b(o, nxt, kb + KS, kmax);
      __builtin_amdgcn_sched_barrier(0);
      multiply(cur, rd, acc);
      __builtin_amdgcn_sched_barrier(0);
      store_a(a, wr);
      load_a(o, a, kb + 2 * KS, kmax);
      __builtin_amdgcn_sched_barrier(0);
      // the stage's LDS writes are visible before any wave reads them; loads
      // in flight stay in flight
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    for (int s = 0; s < stages; s += 2) {
      stage(b0, b1, s0, s1, kb0 + s * KS);
      if (s + 1 < stages) stage(b1, b0, s1, s0, kb0 + (s + 1) * KS);
    }
    __syncthreads();  // the stages' room becomes the sums'
    v4f* red = reinterpret_cast<v4f*>(lds);
    constexpr int Q = NF * NI;
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < NI; ++i) red[((wk * WN + wn) * Q + f * NI + i) * 64 + lane] = acc[f][i];
    __syncthreads();
    for (int q = wave; q < WN * Q; q += WN * WK) {
      v4f t = red[q * 64 + lane];
#pragma unroll
      for (int v = 1; v < WK; ++v) t += red[(v * WN * Q + q) * 64 + lane];
      finish(q / NI, q % NI, t);  // q / Q is the wave's half: fragment rows follow on
    }
    __syncthreads();
  }
};

}  // namespace dg
