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

// Eight E2M1 codes times 2^(e - 127), e the low byte of `e`, as BF16: exact
// (at most two significant bits) down to BF16's subnormals; e = 255 gives NaN.
// The conversion reads only the exponent field of its scale operand, so the
// E8M0 byte goes there as it is (checked on an MI355X for all 256 code pairs
// at scales 2^-127, 2^-126, 1, 2^127 and NaN).
__device__ __forceinline__ dg_bf16x8 widen8_mxfp4(uint32_t w, uint32_t e) {
  const float s = __uint_as_float((e & 0xFFu) << 23);
  const dg_bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  const dg_bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  const dg_bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  const dg_bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return dg_bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// Eight E4M3 codes as BF16: exact (four significant bits).
__device__ __forceinline__ dg_bf16x8 widen8_fp8(uint32_t w0, uint32_t w1) {
  const dg_bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const dg_bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const dg_bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const dg_bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
  return dg_bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
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

// Sum of the quads at s, s + step, ... (S of them), in that order.  They come
// from beyond the L2, so four are asked for at a time.
__device__ __forceinline__ v4f collect_sum(const float* s, int64_t step, int S) {
  v4f t = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < S; p += 4) {
    v4f v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = collect4(s + (p + u < S ? p + u : p) * step);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (p + u < S) t += v[u];
  }
  return t;
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

// First K block of part `part` of `parts` (nkb <= 2^16, parts <= 2^8).
__device__ __forceinline__ int run_begin(int part, int nkb, int parts) {
  return (int)((uint32_t)part * (uint32_t)nkb / (uint32_t)parts);
}

// What one wave multiplies: 16 NF rows of a weight matrix with 16 NI rows of
// activations over a run of 128-wide K blocks.  Rows of the weight start at
// resource b (row stride b_ld bytes), its scales at sb.
struct StreamOperands {
  __amdgpu_buffer_rsrc_t b, sb, a, sa;
  uint32_t sb_step;  // bytes between the scales of one K block and the next
  uint32_t sa_step;
  int last;          // the last K block: blocks past it are addressed as it, with
                     // every lane masked, so no scalar offset passes a resource
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
      const uint32_t k = (uint32_t)min(kb + u, o.last);
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
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (BF == FMT_FP8)
              bw[j] = widen8_fp8((uint32_t)x.b[u][f][j >> 1][2 * (j & 1)],
                                 (uint32_t)x.b[u][f][j >> 1][2 * (j & 1) + 1]);
            else
              bw[j] = widen8_mxfp4((uint32_t)x.b[u][f][0][j], x.sb[u][f] >> sh);
          }
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

// The same product with BF16 activations in LDS, for more than a few of their
// rows.  A fragment load that goes straight to registers makes neighbouring
// lanes read different rows, and activations in BF16 are 4 NI / NF times (E4M3
// weights: 2 NI / NF) the weights' bytes.  By LDS DMA they come in full rows of
// 256 bytes, once for the four waves that multiply them with 32 weight rows
// each.
//
// Eight waves: WK = 2 runs of K, four waves of 16 NF weight rows in each.  A
// stage is one K block of each run.  Stages are R deep, the weights' in
// registers, the activations' in R LDS slots, so R - 1 are in flight while one
// is multiplied; one barrier a stage tells that every wave's DMA of it has
// landed and that the slot of the stage before is free.
// MI355X: BF16 A 33 x 7168 x 16384 27 us with the weights from HBM, of which
// about 6 are the K parts meeting in memory; the layer's gate/up 98 us for 383 MB.
constexpr int kSharedThreads = 512;
constexpr int kSharedMaxDepth = 6;

// Depth for NI fragments of activation rows: what the slots leave room for in
// LDS (two workgroups a CU up to NI = 2, else one) and in registers.  Weight bytes in flight a stage and workgroup: 16 KB in 4 bits,
// 32 KB in 8.
constexpr int shared_depth(int bf, int ni) {
  if (bf == FMT_FP8 || ni > 4) return 3;
  return ni == 1 ? 5 : (ni == 3 ? 6 : 4);
}

// LDS of a workgroup: every slot is a variable of its own, so that a read of
// one is not taken to depend on a transfer into another.
#define DG_SHARED_SLOTS(S)                                                              \
  __shared__ __attribute__((aligned(1024))) uint8_t slot0[S::SLOT0];                    \
  __shared__ __attribute__((aligned(1024))) uint8_t slot1[S::R > 1 ? S::SLOT : 16];     \
  __shared__ __attribute__((aligned(1024))) uint8_t slot2[S::R > 2 ? S::SLOT : 16];     \
  __shared__ __attribute__((aligned(1024))) uint8_t slot3[S::R > 3 ? S::SLOT : 16];     \
  __shared__ __attribute__((aligned(1024))) uint8_t slot4[S::R > 4 ? S::SLOT : 16];     \
  __shared__ __attribute__((aligned(1024))) uint8_t slot5[S::R > 5 ? S::SLOT : 16];     \
  uint8_t* const slots[kSharedMaxDepth] = {slot0, slot1, slot2, slot3, slot4, slot5}

template <int BF, int NI, int R_>
struct Shared {
  static constexpr int R = R_;
  static constexpr int WN = 4, WK = 2, NF = 2, BV = BF == FMT_FP8 ? 2 : 1;
  static constexpr int ROWS_B = 16 * NF * WN;     // weight rows of a workgroup
  static constexpr int ROW = 256;                 // bytes of an LDS row: a K block in BF16
  static constexpr int IT = NI;                   // DMA instructions a wave and stage, 4 rows each
  static constexpr int RUN = IT * WN * 1024;      // bytes of a run's stage
  static constexpr int SLOT = WK * RUN, SLOT0 = SLOT;
  static constexpr int SUMS = WK * WN * NI * 1024;  // the runs' sums meet in slot 0
  static_assert(SUMS <= SLOT, "room for the sums");
  static constexpr int WAVES = R * SLOT <= 79 << 10 ? 4 : 2;  // a SIMD's, as the LDS allows
  static constexpr int LOADS = IT + NF * BV + (BF == FMT_FP8 ? 1 : NF);  // a wave's of a stage
  struct W {
    v4i b[NF][BV];
    uint32_t sb[BF == FMT_FP8 ? 1 : NF];
  };
  uint32_t vb[NF], vsb[NF], va[IT];
  int lane, wave, wk, wn, g, ck;

  // A 16-byte LDS read is served 16 lanes at a time: lanes 0-3, 12-15 and
  // 20-27, then the other 16 of the half wave.  These put the 16 rows of each
  // such group on the 16 different 16-byte slots of a row, which is one sweep
  // of the banks, when lane 16g + r reads chunk 4g + j (MXFP4 weights) or
  // 8h + 2g + j (E4M3) of row r.
  static __device__ __forceinline__ int swz(int r) {
    if (BF == FMT_FP8) return r & 15;
    return (r & 3) | ((r & 8) ? 12 : 0);
  }

  // row_of(r): activation row of the tile's row r, or -1
  template <class Rows>
  __device__ __forceinline__ void init(int64_t ldb, int rows_b, int64_t lda, Rows&& row_of) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wn = wave % WN;
    wk = wave / WN;
    g = lane >> 4;
    const int fr = lane & 15;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int r = 16 * (NF * wn + f) + fr;
      vb[f] = r < rows_b ? (uint32_t)(r * ldb + 16 * g) : kOob;
      vsb[f] = r < rows_b ? (uint32_t)(4 * r) : kOob;
    }
    // DMA: 1 KB of consecutive LDS rows an instruction, the lane's chunk chosen
    // by the row (rows of a wave's instructions agree modulo 16)
    const int r0 = wn * 4 + (lane >> 4);
    ck = (lane & 15) ^ swz(r0);
#pragma unroll
    for (int j = 0; j < IT; ++j) {
      const int a = row_of(16 * j + r0);
      va[j] = a >= 0 ? (uint32_t)(a * lda + 16 * ck) : kOob;
    }
  }

  __device__ __forceinline__ void load(const StreamOperands& o, uint8_t* slot, W& x, int kb,
                                       int kmax) const {
    const uint32_t k = (uint32_t)min(kb, o.last);
    const bool in_a = kb * 128 + ck * 8 < kmax;
#pragma unroll
    for (int j = 0; j < IT; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          o.a, (__attribute__((address_space(3))) void*)(slot + wk * RUN + (j * WN + wn) * 1024), 16,
          (int)(in_a ? va[j] : kOob), (int)(k * ROW), 0, 0);
    // E4M3: a lane's two pieces of 16 are 64 apart, so that an instruction
    // reads 64 bytes of each row
    const bool in = kb * 128 + (BF == FMT_FP8 ? 16 : 32) * g < kmax;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
#pragma unroll
      for (int h = 0; h < BV; ++h)
        x.b[f][h] = load16(o.b, (in ? vb[f] : kOob) + 64 * h, k * (64 * BV));
      if (BF == FMT_MXFP4) x.sb[f] = load4(o.sb, in ? vsb[f] : kOob, k * o.sb_step);
    }
    if (BF == FMT_FP8) x.sb[0] = load4(o.sb, in ? 0u : kOob, k * o.sb_step);
  }

  __device__ __forceinline__ v4i frag(const uint8_t* st, int i, int c) const {
    const int fr = lane & 15;
    return *reinterpret_cast<const v4i*>(st + (16 * i + fr) * ROW + 16 * (c ^ swz(fr)));
  }
  __device__ __forceinline__ void multiply(const W& x, const uint8_t* slot,
                                           v4f (&acc)[NF][NI]) const {
    const uint8_t* st = slot + wk * RUN;
    const int sh = 8 * g;
    // eight K values of a lane at a time, so that few widened weights and
    // activations are live; E4M3 sums a block before its scale is applied
    v4f t[NF][NI];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < NI; ++i) t[f][i] = BF == FMT_FP8 ? v4f{0.f, 0.f, 0.f, 0.f} : acc[f][i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      dg_bf16x8 bw[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        if constexpr (BF == FMT_FP8)
          bw[f] = widen8_fp8((uint32_t)x.b[f][j >> 1][2 * (j & 1)],
                             (uint32_t)x.b[f][j >> 1][2 * (j & 1) + 1]);
        else
          bw[f] = widen8_mxfp4((uint32_t)x.b[f][0][j], x.sb[f] >> sh);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const dg_bf16x8 aw = __builtin_bit_cast(
            dg_bf16x8,
            frag(st, i, BF == FMT_FP8 ? 8 * (j >> 1) + 2 * g + (j & 1) : 4 * g + j));
#pragma unroll
        for (int f = 0; f < NF; ++f)
          t[f][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bw[f], aw, t[f][i], 0, 0, 0);
      }
    }
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if constexpr (BF == FMT_FP8)
          acc[f][i] += t[f][i] * __uint_as_float(x.sb[0]);
        else
          acc[f][i] = t[f][i];
      }
  }

  // Parts part0 + wk of `parts` of K; every wave of the workgroup makes the
  // same number of stages (the barriers), past its run on zeros.
  // finish(f, quads): f in [0, WN NF), the NI quads of its rows, by one wave.
  template <class Finish>
  __device__ __forceinline__ void run(const StreamOperands& o, int64_t K, int part0, int parts,
                                      uint8_t* const (&slots)[kSharedMaxDepth], Finish&& finish) {
    const int nkb = o.last + 1;
    const int part = part0 + wk;
    const int kb0 = run_begin(part, nkb, parts), kb1 = run_begin(part + 1, nkb, parts);
    const int kmax = kb1 * 128 < K ? kb1 * 128 : (int)K;
    const int stages = (nkb + parts - 1) / parts;  // of the longest run
    v4f acc[NF][NI];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[f][i] = v4f{0.f, 0.f, 0.f, 0.f};
    W w[R];
    static_for<R - 1>([&](auto j) {
      load(o, slots[decltype(j)::value], w[decltype(j)::value], kb0 + decltype(j)::value, kmax);
      __builtin_amdgcn_sched_barrier(0);
    });
    static_assert((R - 1) * LOADS <= 63, "range of the counter");
    // This wave's transfers of the stage to multiply have landed, all but the
    // loads of the `newer` stages issued after it; the barrier tells so of every
    // wave's, and that the slot of the stage before is free.  The count stands
    // for what was issued, so every load of a newer stage has to be one that the
    // compiler keeps: the loop's are multiplied by a later pass or by the tail,
    // and the tail, whose loads nothing would read, makes none.
    auto landed = [&](auto newer) {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier ; stage of %1 transfers" ::"n"(
                       decltype(newer)::value * LOADS),
                   "n"(IT)
                   : "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    int s = 0;
    for (; s + R <= stages; s += R)
      static_for<R>([&](auto jc) {
        constexpr int j = decltype(jc)::value, nx = (j + R - 1) % R;
        landed(IntTag<R - 2>{});
        load(o, slots[nx], w[nx], kb0 + s + j + R - 1, kmax);
        __builtin_amdgcn_sched_barrier(0);
        multiply(w[j], slots[j], acc);
      });
    static_while<R - 1>([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      if (s + j >= stages) return false;
      landed(IntTag<R - 2 - j>{});
      multiply(w[j], slots[j], acc);
      return true;
    });
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier ; end of stages" ::: "memory");
    v4f* red = reinterpret_cast<v4f*>(slots[0]);
    // run wk keeps fragment f = wk of its waves and hands over the other
    static_assert(WK == 2 && NF == 2, "each run finishes one fragment row");
#pragma unroll
    for (int i = 0; i < NI; ++i) red[(wave * NI + i) * 64 + lane] = wk ? acc[0][i] : acc[1][i];
    __syncthreads();
    v4f t[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const v4f other = red[((wave ^ 4) * NI + i) * 64 + lane];
      t[i] = wk ? other + acc[1][i] : acc[0][i] + other;
    }
    finish(NF * wn + wk, t);
    __syncthreads();
  }
};

}  // namespace dg
