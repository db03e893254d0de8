// Tiled MXFP4 x MXFP4 NT product for gfx950 (many rows of A).
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 128 K values of a 16 x 16
// sub-tile with both operands' E8M0 scales applied per 32 values, so the FP32
// accumulators chain through K.  FP4 operands take half the cycles of FP8
// ones (16 instead of 32 per instruction), so a stage of K = 256 costs what
// one of K = 128 costs in FP8: the same bytes and the same matrix cycles.
//
//  * Stages: 256 K values (128 bytes) of every row of the A and B tile, two
//    of them in LDS, filled by LDS DMA (buffer loads: rows past the operand
//    and 32-blocks past K read as zeros, without memory traffic).  The 16-byte
//    chunk c of LDS row r sits at chunk c ^ lds_swz(r), which the fragment
//    reads (16 rows, one chunk per 16 lanes) hit without bank conflicts.
//  * LDS row 16 i + f of a group of 64 holds row 4 f + i of the operand.  So
//    the scale words of a lane's four fragments are neighbours in memory (one
//    16-byte load per 64 rows and K block, straight into registers), and a
//    lane ends with 16 consecutive columns of each of its rows: the store
//    needs no staging.
//  * Workgroup ids are dealt round-robin to the 8 XCDs; they are remapped so
//    that each XCD gets a contiguous run of tiles in groups of 4 tile rows
//    swept along N, whose A and B panels its L2 holds.
#include "mxfp4_device.hpp"

namespace dg {
namespace {

struct TileArgs {
  uint16_t* c;
  const uint8_t* a;
  const uint8_t* b;
  const uint32_t* sfa;
  const uint32_t* sfb;
  int64_t M, N;
  int K, tiles_m, tiles_n;
};

constexpr int kGroupM = 4;  // tile rows swept together

// A 16-byte LDS read is served 16 lanes at a time: lanes 0-3, 12-15, 20-23 and
// 24-27, then 4-11, 16-19 and 28-31 (and the same of the upper half).  With
// chunk 4h + g read by lane 16g + r of row r, and two rows to a sweep of the
// banks, this puts each such group on 16 different 16-byte slots.
__device__ __forceinline__ int lds_swz(int r) { return (r & 2) | ((r >> 1) & 4); }

__device__ __forceinline__ void map_tile(const TileArgs& p, int& tm, int& tn) {
  const int total = p.tiles_m * p.tiles_n, bid = blockIdx.x;
  const int x = bid & 7, per = total >> 3, extra = total & 7;
  const int L = x * per + min(x, extra) + (bid >> 3);
  const int per_group = kGroupM * p.tiles_n;
  const int group = L / per_group, rem = L - group * per_group;
  const int gsz = min(p.tiles_m - group * kGroupM, kGroupM);
  tm = group * kGroupM + rem % gsz;
  tn = rem / gsz;
}

// Row of the operand that LDS row r of a tile holds.
__device__ __forceinline__ int tile_row(int r) {
  return (r & ~63) + 4 * (r & 15) + ((r >> 4) & 3);
}

// One operand's tile: ROWS rows, staged by NW waves.
template <int ROWS, int NW>
struct Panel {
  static constexpr int ITERS = ROWS / 8 / NW;
  __amdgpu_buffer_rsrc_t r;
  uint32_t off[ITERS];

  __device__ __forceinline__ void init(const uint8_t* base, int64_t row0, int64_t rows, int K,
                                       int wave, int lane) {
    const int64_t ld = K / 2;
    const int64_t n = rows - row0 < ROWS ? rows - row0 : ROWS;
    r = buffer_of(base + row0 * ld, n * ld);
#pragma unroll
    for (int j = 0; j < ITERS; ++j) {
      const int lr = (j * NW + wave) * 8 + (lane >> 3);
      const int row = tile_row(lr);
      off[j] = row < n ? (uint32_t)(row * ld + (((lane & 7) ^ lds_swz(lr)) * 16)) : kOob;
    }
  }
  __device__ __forceinline__ void issue(uint8_t* lds, int wave, int j, int soff, bool in) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, (__attribute__((address_space(3))) void*)(lds + (j * NW + wave) * 1024), 16,
        (int)(in ? off[j] : kOob), soff, 0, 0);
  }
};

template <int WM, int WN, int NJ>
__global__ void __launch_bounds__(64 * WM * WN) gemm_mxfp4_tile_kernel(TileArgs p) {
  constexpr int NW = WM * WN, BM = 64 * WM, BN = 16 * NJ * WN, NG = NJ / 4;
  constexpr int A_BYTES = BM * 128, STAGE = A_BYTES + BN * 128;
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int fr = lane & 15, g = lane >> 4;
  int tm, tn;
  map_tile(p, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int nkb = (p.K + 127) / 128, nk = (p.K + 255) / 256;

  Panel<BM, NW> pa;
  Panel<BN, NW> pb;
  pa.init(p.a, m0, p.M, p.K, wave, lane);
  pb.init(p.b, n0, p.N, p.K, wave, lane);
  // the 32-block of a stage that this lane's DMA chunks hold (one per lane:
  // lds_swz repeats every 16 rows, a wave's pieces are 8 NW rows apart)
  static_assert(NW % 2 == 0, "rows of a wave's pieces agree modulo 16");
  const int chunk_k = 32 * ((lane & 7) ^ lds_swz(8 * wave + (lane >> 3)));

  // scale words: rows 64 wm + 4 fr .. + 3 of A; 64-row groups of B alike
  const __amdgpu_buffer_rsrc_t rsa = buffer_of(p.sfa + m0, (nkb * p.M - m0) * 4);
  const __amdgpu_buffer_rsrc_t rsb = buffer_of(p.sfb + n0, (nkb * p.N - n0) * 4);
  const uint32_t osa = (uint32_t)(64 * wm + 4 * fr) * 4;
  const uint32_t osb = (uint32_t)(16 * NJ * wn + 4 * fr) * 4;
  const uint32_t step_a = (uint32_t)p.M * 4, step_b = (uint32_t)p.N * 4;
  struct Scales {
    v4i a[2], b[2][NG];
  };
  auto load_scales = [&](Scales& s, int kb) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int w = 2 * kb + h;
      const bool in = w < nkb;
      s.a[h] = load16(rsa, in ? osa : kOob, in ? w * step_a : 0);
#pragma unroll
      for (int q = 0; q < NG; ++q)
        s.b[h][q] = load16(rsb, in ? osb + 256 * q : kOob, in ? w * step_b : 0);
    }
  };

  v4f acc[4][NJ];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  constexpr int IA = Panel<BM, NW>::ITERS, IB = Panel<BN, NW>::ITERS;
  const int swz = lds_swz(fr);
  const int off_h[2] = {fr * 128 + ((g ^ swz) * 16), fr * 128 + (((4 + g) ^ swz) * 16)};
  auto frag = [&](const uint8_t* base, int row, int h) {
    const v4i q = *reinterpret_cast<const v4i*>(base + row * 128 + off_h[h]);
    return v8i{q[0], q[1], q[2], q[3], 0, 0, 0, 0};
  };

  Scales sc, sn;
  {
    const bool in = chunk_k < p.K;
#pragma unroll
    for (int j = 0; j < IA; ++j) pa.issue(lds0, wave, j, 0, in);
#pragma unroll
    for (int j = 0; j < IB; ++j) pb.issue(lds0 + A_BYTES, wave, j, 0, in);
    load_scales(sc, 0);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  }

  auto step = [&](const uint8_t* cur, uint8_t* nxt, int kb) {
    const int kn = kb + 1;
    const bool in = kn * 256 + chunk_k < p.K;
    load_scales(sn, kn);
    const int ko = kn < nk ? kn * 128 : 0;  // no scalar offset past a resource
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // exponent bytes of this lane's 32-block; 0 past K, where the codes are 0
      const int width = kb * 256 + h * 128 + 32 * g < p.K ? 8 : 0;
      int ea[4], eb[NJ];
#pragma unroll
      for (int i = 0; i < 4; ++i) ea[i] = __builtin_amdgcn_ubfe(sc.a[h][i], 8 * g, width);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        eb[j] = __builtin_amdgcn_ubfe(sc.b[h][j >> 2][j & 3], 8 * g, width);
      v8i af[4], bf[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) af[i] = frag(cur, wm * 64 + 16 * i, h);
      bf[0] = frag(cur + A_BYTES, wn * 16 * NJ, h);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < 4 * NJ; ++t) {
        const int j = t >> 2, i = t & 3;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            bf[j & 1], af[i], acc[i][j], 4, 4, 0, eb[j], 0, ea[i]);
        __builtin_amdgcn_sched_barrier(0);
        if (i == 0 && j + 1 < NJ) {
          bf[(j + 1) & 1] = frag(cur + A_BYTES, wn * 16 * NJ + 16 * (j + 1), h);
          __builtin_amdgcn_sched_barrier(0);
        }
        // the next stage's transfers, one per two instructions of the first half
        if (h == 0 && (t & 1) == 1 && (t >> 1) < IA + IB) {
          const int q = t >> 1;
          if (q < IA)
            pa.issue(nxt, wave, q, ko, in);
          else
            pb.issue(nxt + A_BYTES, wave, q - IA, ko, in);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    static_assert(2 * (IA + IB) <= 4 * NJ, "transfer slots");
    sc = sn;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  };

  for (int kb = 0; kb < nk; kb += 2) {
    step(lds0, lds1, kb);
    if (kb + 1 < nk) step(lds1, lds0, kb + 1);
  }

  // lane: rows 4 fr + i, columns 64 q + 16 g + 4 r + jj of the wave's part
  const bool wide = (p.N & 7) == 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + 64 * wm + 4 * fr + i;
    if (m >= p.M) continue;
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      const int64_t n = n0 + 16 * NJ * wn + 64 * q + 16 * g;
      uint32_t v[8];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[2 * r] = bf16x2_rne(acc[i][4 * q][r], acc[i][4 * q + 1][r]);
        v[2 * r + 1] = bf16x2_rne(acc[i][4 * q + 2][r], acc[i][4 * q + 3][r]);
      }
      uint16_t* d = p.c + m * p.N + n;
      if (wide) {
        if (n < p.N) *reinterpret_cast<uint4*>(d) = make_uint4(v[0], v[1], v[2], v[3]);
        if (n + 8 < p.N) *reinterpret_cast<uint4*>(d + 8) = make_uint4(v[4], v[5], v[6], v[7]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (n + e < p.N) d[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

template <int WM, int WN, int NJ>
hipError_t launch(TileArgs p, hipStream_t stream) {
  p.tiles_m = (int)((p.M + 64 * WM - 1) / (64 * WM));
  p.tiles_n = (int)((p.N + 16 * NJ * WN - 1) / (16 * NJ * WN));
  hipLaunchKernelGGL((gemm_mxfp4_tile_kernel<WM, WN, NJ>), dim3((unsigned)(p.tiles_m * p.tiles_n)),
                     dim3(64 * WM * WN), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_mxfp4_tiled(const Mxfp4Problem& q, hipStream_t stream) {
  TileArgs p;
  p.c = q.c;
  p.a = static_cast<const uint8_t*>(q.a);
  p.b = q.b;
  p.sfa = q.sfa;
  p.sfb = q.sfb;
  p.M = q.M;
  p.N = q.N;
  p.K = (int)q.K;
  const int64_t big = ((q.M + 255) / 256) * ((q.N + 255) / 256);
  if (big >= 200) return launch<4, 2, 8>(p, stream);
  return launch<2, 2, 4>(p, stream);
}

}  // namespace dg
