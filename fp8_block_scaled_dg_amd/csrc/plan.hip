// The layout of the grouped products (experts contiguous along M, each one's
// rows filled up to a multiple of 128) from the experts of all tokens, gfx950.
//
// A stable counting sort of the n = T k pairs (token, slot) by expert: the row
// of a pair is its expert's offset plus the number of earlier pairs of that
// expert.  The pairs are cut into chunks, one workgroup each; a workgroup needs
// each expert's total and its count in the chunks before its own.  Few pairs:
// every workgroup counts all of them itself (one launch).  Many: a first launch
// leaves each chunk's counts in the workspace.
//
// MI355X, a call of many in a graph: 128 pairs 3.8 us, 8004 of 60 experts 5.3, 16384 of
// 256 8.1, 65536 9.7, 262144 14.7.  One launch / two, with chunks of 1024: 8004 6.3 /
// 7.8, 16384 of 256 8.3 / 8.9, of 8 (whose counters collide) 10.2 / 8.3, 65536 15.6 / 9.7.
// Reading and writing take 0.2 us at most; the rest is launches and a chain of four
// steps, each a memory latency or a barrier.
//
// Nothing depends on the order in which workgroups or waves run: the counters
// in LDS are sums, and a wave ranks its 64 pairs by which lanes hold the same
// expert (one ballot a bit of the expert's id).
#include "dg_device.hpp"
#include "dg_internal.hpp"

namespace dg {
namespace {

constexpr int kPlanWaves = 8, kPlanThreads = 64 * kPlanWaves;
constexpr int kPlanMaxChunks = 256;
constexpr int64_t kPlanSelfPairs = 8192;  // up to here workgroups count all pairs
static_assert(2 * kPlanThreads >= kMoeMaxExperts, "two experts a thread");

__device__ __forceinline__ int expert_of(const PlanArgs& p, int64_t i) {
  const int id = p.ids[i];
  return (unsigned)id < (unsigned)p.E ? id : -1;
}

// f(expert, pair) for the pairs begin .. end - 1 that have one, four neighbours a
// thread and turn, two turns' loads on their way at once.
template <class F>
__device__ __forceinline__ void for_pairs(const PlanArgs& p, int64_t begin, int64_t end, F&& f) {
  constexpr int64_t step = 4 * kPlanThreads;
  for (int64_t i = begin + 4 * threadIdx.x; i < end; i += 2 * step) {
    int id[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t at = i + u * step;
#pragma unroll
      for (int j = 0; j < 4; ++j) id[u][j] = -1;
      if (at + 4 <= end) {
        __builtin_memcpy(id[u], __builtin_assume_aligned(p.ids + at, 4), 16);
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (at + j < end) id[u][j] = p.ids[at + j];
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((unsigned)id[u][j] < (unsigned)p.E) f(id[u][j], i + u * step + j);
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(PlanArgs p) {
  __shared__ int s_count[kMoeMaxExperts];
  for (int e = threadIdx.x; e < p.E; e += kPlanThreads) s_count[e] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * p.chunk, end = begin + p.chunk < p.n ? begin + p.chunk : p.n;
  for_pairs(p, begin, end, [&](int e, int64_t) { atomicAdd(&s_count[e], 1); });
  __syncthreads();
  const int pitch = (p.E + 3) & ~3;
  for (int e = threadIdx.x; e < pitch; e += kPlanThreads)
    p.chunk_counts[(int64_t)blockIdx.x * pitch + e] = e < p.E ? s_count[e] : 0;
}

template <bool SELF>
__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(PlanArgs p) {
  __shared__ int s_next[kPlanWaves][kMoeMaxExperts];  // a wave's next row of each expert
  __shared__ int s_total[kMoeMaxExperts], s_before[kMoeMaxExperts];
  __shared__ int s_offset[kMoeMaxExperts + 1], s_sum[kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t begin = blockIdx.x * p.chunk, end = begin + p.chunk < p.n ? begin + p.chunk : p.n;
  for (int e = tid; e < p.E; e += kPlanThreads) {
    s_total[e] = 0;
    s_before[e] = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) s_next[w][e] = 0;
  }
  __syncthreads();
  // this wave's part of the chunk, a multiple of 64 pairs
  const int64_t part = (p.chunk + kPlanThreads - 1) / kPlanThreads * 64;
  const int64_t w0 = begin + wave * part < end ? begin + wave * part : end;
  const int64_t w1 = w0 + part < end ? w0 + part : end;
  for (int64_t i = w0 + lane; i < w1; i += 64) {
    const int e = expert_of(p, i);
    if (e >= 0) atomicAdd(&s_next[wave][e], 1);
  }
  if constexpr (SELF) {
    for_pairs(p, 0, p.n, [&](int e, int64_t i) {
      atomicAdd(&s_total[e], 1);
      if (i < begin) atomicAdd(&s_before[e], 1);
    });
  } else {
    // four experts a thread, the chunks shared out over the threads that have
    // the same four
    const int quads = (p.E + 3) / 4, q = tid % quads, first = tid / quads, step = kPlanThreads / quads;
    const int4* counts = reinterpret_cast<const int4*>(p.chunk_counts);
    if (first < step) {
      int4 t = make_int4(0, 0, 0, 0), b = t;
#pragma unroll 8
      for (int c = first; c < p.chunks; c += step) {
        const int4 n = counts[(int64_t)c * quads + q];
        t.x += n.x; t.y += n.y; t.z += n.z; t.w += n.w;
        if (c < (int)blockIdx.x) { b.x += n.x; b.y += n.y; b.z += n.z; b.w += n.w; }
      }
      const int tt[4] = {t.x, t.y, t.z, t.w}, bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * q + i < p.E) {
          atomicAdd(&s_total[4 * q + i], tt[i]);
          atomicAdd(&s_before[4 * q + i], bb[i]);
        }
    }
  }
  __syncthreads();
  // experts 2 tid and 2 tid + 1
  int total[2] = {0, 0}, before[2] = {0, 0}, padded[2], own = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = 2 * tid + h;
    if (e < p.E) {
      total[h] = s_total[e];
      before[h] = s_before[e];
    }
    padded[h] = (total[h] + 127) & ~127;
    own += padded[h];
  }
  int sum = own;  // running sum over the wave, then over the waves
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(sum, d, 64);
    if (lane >= d) sum += o;
  }
  if (lane == 63) s_sum[wave] = sum;
  __syncthreads();
  int offset = sum - own;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w)
    if (w < wave) offset += s_sum[w];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = 2 * tid + h;
    if (e < p.E) {
      s_offset[e] = offset;
      int next = offset + before[h];
#pragma unroll
      for (int w = 0; w < kPlanWaves; ++w) {
        const int n = s_next[w][e];
        s_next[w][e] = next;
        next += n;
      }
      if (blockIdx.x == 0) {
        p.offsets[e] = offset;
        p.counts[e] = total[h];
      }
      offset += padded[h];
      if (e == p.E - 1) {
        s_offset[p.E] = offset;
        if (blockIdx.x == 0) p.offsets[p.E] = offset;
      }
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz((unsigned)p.E);
  for (int64_t i0 = w0; i0 < w1; i0 += 64) {
    const int64_t i = i0 + lane;
    const int e = i < w1 ? expert_of(p, i) : -1;
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(e >> b & 1);
      same &= e >> b & 1 ? set : ~set;
    }
    const int first = __ffsll((unsigned long long)same) - 1;
    int row = 0;
    if (e >= 0 && lane == first) row = atomicAdd(&s_next[wave][e], (int)__popcll(same));
    row = __shfl(row, first < 0 ? 0 : first, 64) + __popcll(same & ((1ull << lane) - 1));
    if (i < w1) p.rows[i] = e >= 0 ? row : -1;
    if (e >= 0) {
      p.pairs[row] = (int)i;
      p.m_indices[row] = e;
    }
  }
  // rows that no pair has: the ends of the experts' blocks (128 threads an
  // expert) and what is behind the last expert
  for (int e = (int)blockIdx.x * (kPlanThreads / 128) + (tid >> 7); e < p.E;
       e += p.chunks * (kPlanThreads / 128)) {
    const int r = s_offset[e] + s_total[e] + (tid & 127);
    if (r < s_offset[e + 1]) {
      p.pairs[r] = -1;
      p.m_indices[r] = -1;
    }
  }
  for (int64_t r = s_offset[p.E] + (int64_t)blockIdx.x * kPlanThreads + tid; r < p.M;
       r += (int64_t)p.chunks * kPlanThreads) {
    p.pairs[r] = -1;
    p.m_indices[r] = -1;
  }
}

// Chunks of 512 pairs (a round of 64 a wave), more where the rows to fill are many
// next to the pairs, at most 256.  8004 pairs 5.3 us, with chunks of 1024 6.3, of 2048
// 8.2; 65536 9.7, 9.7 and 11.7.
int plan_chunks(int64_t n, int64_t M) {
  int64_t c = (n + 511) / 512;
  const int64_t fill = (M + 8191) / 8192;
  if (c < fill) c = fill;
  const int64_t most = (n + 63) / 64;  // not more than there is work for
  if (c > most) c = most;
  return (int)(c < 1 ? 1 : c > kPlanMaxChunks ? kPlanMaxChunks : c);
}

}  // namespace

int64_t plan_rows(int64_t T, int E, int k) {
  const int64_t n = T * k, used = n < E ? n : E;
  return 128 * (used + (n - used) / 128);
}

size_t plan_workspace_bytes(int64_t T, int E, int k) {
  const int64_t n = T * k;
  return n <= kPlanSelfPairs ? 0 : (size_t)kPlanMaxChunks * ((E + 3) / 4) * sizeof(int4);
}

hipError_t launch_plan(PlanArgs p, void* workspace, hipStream_t stream) {
  p.chunks = plan_chunks(p.n, p.M);
  p.chunk = (p.n + p.chunks - 1) / p.chunks;
  p.chunk_counts = static_cast<int*>(workspace);
  const dim3 grid((unsigned)p.chunks), block(kPlanThreads);
  if (p.n <= kPlanSelfPairs) {
    hipLaunchKernelGGL(plan_place_kernel<true>, grid, block, 0, stream, p);
  } else {
    hipLaunchKernelGGL(plan_count_kernel, grid, block, 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(plan_place_kernel<false>, grid, block, 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace dg
