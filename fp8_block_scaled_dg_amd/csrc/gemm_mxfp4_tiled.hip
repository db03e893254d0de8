// Tiled MXFP4 x MXFP4 NT product for gfx950 (many rows of A).
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 128 K values of a 16 x 16
// sub-tile with both operands' E8M0 scales applied per 32 values, so the FP32
// accumulators chain through K.  FP4 operands take half the cycles of FP8
// ones (16 instead of 32 per instruction).
//
//  * Stages: 256 K values (128 bytes, so the L2 is asked for full lines) of
//    every row of the A and B tile, two of them in LDS, filled by LDS DMA
//    (buffer loads: rows past the operand and 32-blocks past K read as zeros,
//    without memory traffic).  One barrier a stage, two columns of products
//    before its end: the next stage has landed, so its first fragments are
//    read under the last products, and this one has been read, so the
//    transfers of the stage after the next go into its room at once.
//  * The 16-byte chunk c of LDS row r sits at chunk c ^ lds_swz(r), which the
//    fragment reads (16 rows, one chunk per 16 lanes) hit without bank
//    conflicts.
//  * LDS row 16 i + f of a group of 64 holds row 4 f + i of the operand.  So
//    the scale words of a lane's four fragments are neighbours in memory (one
//    16-byte load per 64 rows and K block, straight into registers), and a
//    lane ends with 16 consecutive columns of each of its rows: the store
//    needs no staging.
//  * Workgroup ids are dealt round-robin to the 8 XCDs; they are remapped so
//    that each XCD gets a contiguous run of tiles in groups of 4 tile rows
//    swept along N, whose A and B panels its L2 holds.
//
// MI355X: 8192^3 261 us (4.2 PFLOP/s), 4096 x 7168 x 2048 41 us.  A loop of
// nothing but these instructions on random codes reaches 7.1 PFLOP/s (9.7 on
// zeros: the clock gives way to power).  What holds the 8192^3 product is LDS: a
// CU reads 96 KB of fragments and takes in 32 KB per 128 K values, 1024 cycles at
// 128 bytes each, as many as its matrix instructions last; the two overlap in
// part, and the matrix cores are busy 52 % of the cycles, at 1.9 GHz.  L2 requests fell
// by half with 128-byte rows (34 to 18 million, 298 to 273 us); deeper rings of
// 64-byte rows, smaller tiles side by side and four waves of 128 x 128 (512
// registers, spilling) were slower.
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
  int S;            // parts of K
  float* partials;  // [tile][S][wave][4 NJ][64] quads, when S > 1
  int* counters;
};

constexpr int kGroupM = 4;  // tile rows swept together

// A 16-byte LDS read is served 16 lanes at a time: lanes 0-3, 12-15, 20-23 and
// 24-27, then 4-11, 16-19 and 28-31 (and the same of the upper half).  With
// chunk 4h + g read by lane 16g + r of row r, and two rows to a sweep of the
// banks, this puts each such group on 16 different 16-byte slots.
__device__ __forceinline__ int lds_swz(int r) { return (r & 2) | ((r >> 1) & 4); }

__device__ __forceinline__ void map_tile(const TileArgs& p, int bid, int& tm, int& tn) {
  const int total = p.tiles_m * p.tiles_n;
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

// One operand's tile: ROWS rows, staged by NW waves, eight rows an instruction.
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

template <int WM, int WN, int NJ, bool SPLIT>
__global__ void __launch_bounds__(64 * WM * WN, 2) gemm_mxfp4_tile_kernel(TileArgs p) {
  constexpr int NW = WM * WN, BM = 64 * WM, BN = 16 * NJ * WN, NG = NJ / 4;
  constexpr int A_BYTES = BM * 128, STAGE = A_BYTES + BN * 128;
  // variables of their own: a read of one stage is not taken to depend on a
  // transfer into the other
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int fr = lane & 15, g = lane >> 4;
  const int tile = (int)(blockIdx.x / (unsigned)p.S), split = (int)blockIdx.x - tile * p.S;
  int tm, tn;
  map_tile(p, tile, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int nkb = (p.K + 127) / 128, nk = (p.K + 255) / 256;
  // this part's stages [kb0, kb1); what is transferred ends with them
  const int kb0 = run_begin(split, nk, p.S), kb1 = run_begin(split + 1, nk, p.S);
  const int kmax = min(kb1 * 256, p.K);

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
  struct Scales {  // of a K block
    v4i a, b[NG];
  };
  auto load_scales = [&](Scales& s, int w) {
    const bool in = w < nkb;
    s.a = load16(rsa, in ? osa : kOob, in ? w * step_a : 0);
#pragma unroll
    for (int q = 0; q < NG; ++q)
      s.b[q] = load16(rsb, in ? osb + 256 * q : kOob, in ? w * step_b : 0);
  };

  v4f acc[4][NJ];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  constexpr int IA = Panel<BM, NW>::ITERS, IB = Panel<BN, NW>::ITERS;
  constexpr int PIECES = IA + IB, EARLY = 4;  // transfers a wave; those right after the barrier
  constexpr int H = 4 * NJ, LAST = 2 * H - 8;  // products of a K block; the first after the barrier
  const int swz = lds_swz(fr);
  const int off_h[2] = {fr * 128 + ((g ^ swz) * 16), fr * 128 + (((4 + g) ^ swz) * 16)};
  auto frag = [&](const uint8_t* base, int row, int h) {
    const v4i q = *reinterpret_cast<const v4i*>(base + row * 128 + off_h[h]);
    return v8i{q[0], q[1], q[2], q[3], 0, 0, 0, 0};
  };
  auto frag_a = [&](const uint8_t* st, int i, int h) { return frag(st, wm * 64 + 16 * i, h); };
  auto frag_b = [&](const uint8_t* st, int c) {  // column c of 2 NJ: NJ of each K block
    return frag(st + A_BYTES, wn * 16 * NJ + 16 * (c % NJ), c / NJ);
  };
  auto piece = [&](uint8_t* st, int q, int kb) {  // the q-th transfer of stage kb
    const bool in = kb * 256 + chunk_k < kmax;
    const int soff = kb < kb1 ? kb * 128 : 0;  // no scalar offset past a resource
    if (q < IA)
      pa.issue(st, wave, q, soff, in);
    else
      pb.issue(st + A_BYTES, wave, q - IA, soff, in);
  };

  Scales sc[2];  // of the stage's two K blocks
  v8i af[2][4], bf[4];
#pragma unroll
  for (int q = 0; q < PIECES; ++q) piece(lds0, q, kb0);
  __builtin_amdgcn_sched_barrier(0);
  load_scales(sc[0], 2 * kb0);
  load_scales(sc[1], 2 * kb0 + 1);
#pragma unroll
  for (int q = 0; q < EARLY; ++q) piece(lds1, q, kb0 + 1);
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(2 * (1 + NG) + EARLY) : "memory");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < 4; ++i) af[0][i] = frag_a(lds0, i, 0);
  bf[0] = frag_b(lds0, 0);
  bf[1] = frag_b(lds0, 1);

  auto step = [&](uint8_t* st, uint8_t* next, int kb) {
    int ea[4], eb[NJ];
    __builtin_amdgcn_sched_barrier(0);
    static_for<2 * H>([&](auto t) {
      constexpr int m = decltype(t)::value, c = m >> 2, i = m & 3, h = m / H, j = c % NJ;
      if constexpr (m == 0 || m == H) {
        // exponent bytes of this lane's 32-block; 0 past K, where the codes are
        // 0; the registers then take the next stage's words
        const int width = kb * 256 + h * 128 + 32 * g < p.K ? 8 : 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) ea[q] = __builtin_amdgcn_ubfe(sc[h].a[q], 8 * g, width);
#pragma unroll
        for (int q = 0; q < NJ; ++q)
          eb[q] = __builtin_amdgcn_ubfe(sc[h].b[q >> 2][q & 3], 8 * g, width);
        __builtin_amdgcn_sched_barrier(0);
        load_scales(sc[h], 2 * kb + 2 + h);
        __builtin_amdgcn_sched_barrier(0);
      }
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          bf[c & 3], af[h][i], acc[i][j], 4, 4, 0, eb[j], 0, ea[i]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (i == 0 && c + 2 < 2 * NJ) bf[(c + 2) & 3] = frag_b(st, c + 2);
      if constexpr (m >= H - 8 && m < H - 4) af[1][m - (H - 8)] = frag_a(st, m - (H - 8), 1);
      // the other transfers of the next stage, one per two instructions
      if constexpr ((m & 1) == 1 && (m >> 1) < PIECES - EARLY) piece(next, EARLY + (m >> 1), kb + 1);
      if constexpr (m == LAST - 1) {
        __builtin_amdgcn_sched_barrier(0);
        // all but the second K block's scales, issued after the next stage's
        // transfers; this stage's LDS reads done
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(1 + NG) : "memory");
      }
      if constexpr (m >= LAST) {
        constexpr int q = m - LAST;
        if constexpr (q == 0) bf[0] = frag_b(next, 0);
        if constexpr (q >= 1 && q < 5) af[0][q - 1] = frag_a(next, q - 1, 0);
        if constexpr (q == 5) bf[1] = frag_b(next, 1);
        if constexpr ((q & 1) == 1) piece(st, q >> 1, kb + 2);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    static_assert(2 * (PIECES - EARLY) <= H && EARLY == 4, "transfers before the scales");
  };
  int kb = kb0;
  for (; kb + 2 <= kb1; kb += 2) {
    step(lds0, lds1, kb);
    step(lds1, lds0, kb + 1);
  }
  if (kb < kb1) step(lds0, lds1, kb);

  // the (masked) transfers past the end land before this workgroup's LDS is freed
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  if constexpr (SPLIT) {
    if (p.S > 1) {
      // parts meet in the workspace; the last workgroup to arrive adds them in
      // order, a whole part in flight at a time
      __shared__ int s_last;
      constexpr int QT = NW * 4 * NJ;
      float* mine = p.partials + ((int64_t)tile * p.S * QT + wave * (4 * NJ)) * 256 + lane * 4;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) publish4(mine + (split * QT + 4 * j + i) * 256, acc[i][j]);
      if (!arrive_last(&p.counters[tile], p.S, &s_last)) return;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
      for (int sp = 0; sp < p.S; ++sp) {
        v4f v[4][NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i][j] = collect4(mine + (sp * QT + 4 * j + i) * 256);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i][j] += v[i][j];
      }
      if (threadIdx.x == 0)  // zero again for the next call
        __hip_atomic_store(&p.counters[tile], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }

  // lane: rows 4 fr + i, columns 64 q + 16 g + 4 r + jj of the wave's part
  // (a row of C starts at any element, so the wide stores are not aligned to
  // their size: the memory path takes that)
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
      if (n + 16 <= p.N) {
        __builtin_memcpy(__builtin_assume_aligned(d, 2), v, 16);
        __builtin_memcpy(__builtin_assume_aligned(d + 8, 2), v + 4, 16);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (n + e < p.N) d[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

template <int WM, int WN, int NJ, bool SPLIT>
hipError_t launch(TileArgs p, hipStream_t stream) {
  p.tiles_m = (int)((p.M + 64 * WM - 1) / (64 * WM));
  p.tiles_n = (int)((p.N + 16 * NJ * WN - 1) / (16 * NJ * WN));
  hipLaunchKernelGGL((gemm_mxfp4_tile_kernel<WM, WN, NJ, SPLIT>),
                     dim3((unsigned)(p.tiles_m * p.tiles_n * p.S)), dim3(64 * WM * WN), 0, stream, p);
  return hipGetLastError();
}

// One 256 x 256 tile a CU or two of 128 x 128.  The large one moves half as
// much per product, but needs tiles enough for whole rounds of the 256 CUs:
// 263 against 326 us (8192^3), 26 / 30.5 (4096 x 4096 x 2016: one round), 43 /
// 44 (4096 x 7168 x 2048: 1.75 rounds), but 28.4 / 26.1 (3000 x 8192 x 1024:
// 1.5) and 32 / 26 (2001 x 4096 x 4096: half a round).
bool large_tiles(int64_t M, int64_t N) {
  const int64_t t = ((M + 255) / 256) * ((N + 255) / 256), rounds = (t + 255) / 256;
  return 5 * t >= 4 * 256 * rounds;
}

// Parts of K for few small tiles.  A 256-wide stage takes 0.7 us here, meeting
// in the workspace 6 to 8 us, so a part keeps 12 stages: 35 against 64 us (128
// x 7168 x 16384 in four; 31 / 49 with the operands in the 256 MB cache, as a
// quantiser leaves them), 23 / 31 (19.5 / 24.4) (128 x 1024 x 8192 in two).  Of
// 8 stages: 16.8 / 18.4, but 15.1 / 14.3 from the cache (65 x 4096 x 4096 in two).
int tile_split(int64_t M, int64_t N, int64_t K) {
  if (large_tiles(M, N)) return 1;
  const int64_t t = ((M + 127) / 128) * ((N + 127) / 128), nk = (K + 255) / 256;
  int S = 1;
  while (2 * S * t <= 384 && nk / (2 * S) >= 12 && S < 16) S *= 2;
  return S;
}

}  // namespace

size_t mxfp4_tiled_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const int S = tile_split(M, N, K);
  if (S == 1) return 0;
  return kSplitkCounterBytes + (size_t)(((M + 127) / 128) * ((N + 127) / 128)) * S * 65536;
}

hipError_t launch_gemm_mxfp4_tiled(const Mxfp4Problem& q, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
  TileArgs p;
  p.c = q.c;
  p.a = static_cast<const uint8_t*>(q.a);
  p.b = q.b;
  p.sfa = q.sfa;
  p.sfb = q.sfb;
  p.M = q.M;
  p.N = q.N;
  p.K = (int)q.K;
  p.S = workspace_bytes < mxfp4_tiled_workspace_bytes(q.M, q.N, q.K) ? 1
                                                                     : tile_split(q.M, q.N, q.K);
  p.counters = static_cast<int*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + kSplitkCounterBytes);
  if (large_tiles(q.M, q.N)) return launch<4, 2, 8, false>(p, stream);
  return launch<2, 2, 4, true>(p, stream);
}

}  // namespace dg
