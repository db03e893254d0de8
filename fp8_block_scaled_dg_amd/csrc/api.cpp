// C ABI of libdg (declared in include/dg.h): host-side validation and
// dispatch to the gfx950 kernels.  Validation happens before any HIP call, so
// a rejected call enqueues nothing.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include "../../include/dg.h"
#include "dg_internal.hpp"

namespace {

static_assert(DG_WORKSPACE_COUNTER_BYTES == dg::kSplitkCounterBytes,
              "counter region of dg.h and of the kernels");

constexpr int64_t kMaxGridY = 65535;
constexpr int64_t kU32 = 4294967295LL;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int from_hip(hipError_t e) { return e == hipSuccess ? DG_OK : DG_ERR_HIP; }

// Checks shared by the dense and grouped GEMMs.
int check_gemm(const uint16_t* c, const uint8_t* a, const uint8_t* b, const float* sa,
               const float* sb, int a_block_rows, int64_t M, int64_t N, int64_t K) {
  if (!c || !a || !b || !sa || !sb) return DG_ERR_NULL;
  if (a_block_rows != 1 && a_block_rows != 128) return DG_ERR_UNSUPPORTED;
  if (M < 1 || N < 8 || K < 128) return DG_ERR_SHAPE;
  if (N % 8 != 0 || K % 128 != 0) return DG_ERR_SHAPE;
  // 32-bit tile offsets inside the kernels
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return DG_ERR_SHAPE;
  if (M * K > kU32 || N * K > kU32) return DG_ERR_SHAPE;
  if (!aligned(c, 16) || !aligned(a, 16) || !aligned(b, 16)) return DG_ERR_ALIGN;
  if (!aligned(sa, 4) || !aligned(sb, 4)) return DG_ERR_ALIGN;
  return DG_OK;
}

// A split-K workspace, when given, must hold what the small-M plan for this
// shape uses and be 16-byte aligned; a NULL pointer or a zero size means none.
int check_workspace(int64_t M, int64_t N, int64_t K, void** workspace, size_t* workspace_bytes) {
  if (*workspace != nullptr && *workspace_bytes > 0) {
    const size_t need = dg::skinny_applies(M, N, K) ? dg::skinny_workspace_bytes(M, N, K) : 0;
    if (*workspace_bytes < need) return DG_ERR_WORKSPACE;
    if (!aligned(*workspace, 16)) return DG_ERR_ALIGN;
  } else {
    *workspace = nullptr;  // one of the two missing: treat as "no workspace"
    *workspace_bytes = 0;
  }
  return DG_OK;
}

size_t align16(int64_t n) { return (size_t)((n + 15) / 16 * 16); }

// Workspace bytes for the operands a layout has to transpose.
size_t transpose_bytes(int64_t M, int64_t N, int64_t K, int layout) {
  const bool a_t = layout == DG_LAYOUT_TN || layout == DG_LAYOUT_TT;
  const bool b_n = layout == DG_LAYOUT_TN || layout == DG_LAYOUT_NN;
  return (a_t ? align16(M * K) : 0) + (b_n ? align16(N * K) : 0);
}

}  // namespace

extern "C" {

int dg_abi_version(void) { return DG_ABI_VERSION; }

const char* dg_status_string(int status) {
  switch (status) {
    case DG_OK: return "ok";
    case DG_ERR_NULL: return "a required pointer is NULL";
    case DG_ERR_SHAPE: return "invalid or unsupported shape";
    case DG_ERR_UNSUPPORTED: return "unsupported block_rows, group count or epilogue";
    case DG_ERR_ALIGN: return "pointer not suitably aligned";
    case DG_ERR_WORKSPACE: return "workspace smaller than required";
    case DG_ERR_HIP: return "HIP runtime error";
    case DG_ERR_SCRATCH: return "shape needs more split-K scratch than the static array holds";
    default: return "unknown status";
  }
}

int dg_get_mk_alignment_for_contiguous_layout(void) { return 128; }

int dg_quantize_fp8_block(uint8_t* q, float* scales, const float* x, int64_t rows, int64_t cols,
                          int block_rows, void* stream) {
  if (!q || !scales || !x) return DG_ERR_NULL;
  if (block_rows != 1 && block_rows != 128) return DG_ERR_UNSUPPORTED;
  if (rows < 1 || cols < 1 || cols % 16 != 0) return DG_ERR_SHAPE;
  const int64_t n_kb = (cols + 127) / 128;
  const int64_t grid_y = block_rows == 128 ? (rows + 127) / 128 : (rows + 31) / 32;
  if (grid_y > kMaxGridY || n_kb > INT32_MAX) return DG_ERR_SHAPE;
  if (rows > INT64_MAX / cols) return DG_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 4)) return DG_ERR_ALIGN;
  return from_hip(dg::launch_quantize(q, scales, x, rows, cols, block_rows,
                                      static_cast<hipStream_t>(stream)));
}

int dg_quantize_fp8_block_ue8m0(uint8_t* q, int32_t* sf, const float* x, int64_t rows,
                                int64_t cols, int block_rows, void* stream) {
  if (!q || !sf || !x) return DG_ERR_NULL;
  if (block_rows != 1 && block_rows != 128) return DG_ERR_UNSUPPORTED;
  if (rows < 1 || cols < 1 || cols % 16 != 0) return DG_ERR_SHAPE;
  const int64_t n_kb = (cols + 127) / 128;
  const int64_t grid_y = block_rows == 128 ? (rows + 127) / 128 : (rows + 31) / 32;
  if (grid_y > kMaxGridY || n_kb > INT32_MAX) return DG_ERR_SHAPE;
  if (rows > INT64_MAX / cols) return DG_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 4)) return DG_ERR_ALIGN;
  return from_hip(dg::launch_quantize_ue8m0(q, reinterpret_cast<uint32_t*>(sf), x, rows, cols,
                                            block_rows, static_cast<hipStream_t>(stream)));
}

size_t dg_fp8_gemm_nt_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 1) return 0;
  return dg::skinny_applies(M, N, K) ? dg::skinny_workspace_bytes(M, N, K) : 0;
}

int dg_fp8_gemm_nt(uint16_t* c, const uint8_t* a, const uint8_t* b, const float* sa,
                   const float* sb, int a_block_rows, int64_t M, int64_t N, int64_t K,
                   void* workspace, size_t workspace_bytes, void* stream) {
  return dg_fp8_gemm_nt_epilogue(c, a, b, sa, sb, a_block_rows, M, N, K, DG_EPI_NONE, nullptr,
                                 workspace, workspace_bytes, stream);
}

int dg_fp8_gemm_nt_epilogue(uint16_t* c, const uint8_t* a, const uint8_t* b, const float* sa,
                            const float* sb, int a_block_rows, int64_t M, int64_t N, int64_t K,
                            int act, const uint16_t* residual, void* workspace,
                            size_t workspace_bytes, void* stream) {
  int st = check_gemm(c, a, b, sa, sb, a_block_rows, M, N, K);
  if (st != DG_OK) return st;
  if (act < DG_EPI_NONE || act > DG_EPI_SWIGLU) return DG_ERR_UNSUPPORTED;
  if (residual && !aligned(residual, 16)) return DG_ERR_ALIGN;
  const bool skinny = dg::skinny_applies(M, N, K);
  st = check_workspace(M, N, K, &workspace, &workspace_bytes);
  if (st != DG_OK) return st;
  dg::GemmProblem p{c, a, b, sa, sb, nullptr, 1, a_block_rows, M, N, K};
  p.epi.act = act;
  p.epi.res = residual;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (skinny) {
    if (dg::stream_preferred(M, N, K)) return from_hip(dg::launch_gemm_stream(p, s));
    return from_hip(dg::launch_gemm_skinny(p, workspace, workspace_bytes, s));
  }
  const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
  if (tiles > INT32_MAX) return DG_ERR_SHAPE;
  return from_hip(dg::launch_gemm_tiled(p, false, s));
}

int dg_fp8_gemm_nt_ue8m0(uint16_t* c, const uint8_t* a, const uint8_t* b, const int32_t* sfa,
                         const int32_t* sfb, int a_block_rows, int64_t M, int64_t N, int64_t K,
                         void* workspace, size_t workspace_bytes, void* stream) {
  // the FP32-scale checks apply unchanged (the scale pointers only need
  // 4-byte alignment in both forms)
  int st = check_gemm(c, a, b, reinterpret_cast<const float*>(sfa),
                      reinterpret_cast<const float*>(sfb), a_block_rows, M, N, K);
  if (st != DG_OK) return st;
  st = check_workspace(M, N, K, &workspace, &workspace_bytes);
  if (st != DG_OK) return st;
  dg::GemmProblem p{c, a, b, nullptr, nullptr, nullptr, 1, a_block_rows, M, N, K};
  p.sfa = reinterpret_cast<const uint32_t*>(sfa);
  p.sfb = reinterpret_cast<const uint32_t*>(sfb);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dg::skinny_applies(M, N, K)) {
    if (dg::stream_preferred(M, N, K)) return from_hip(dg::launch_gemm_stream(p, s));
    return from_hip(dg::launch_gemm_skinny(p, workspace, workspace_bytes, s));
  }
  const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
  if (tiles > INT32_MAX) return DG_ERR_SHAPE;
  return from_hip(dg::launch_gemm_tiled_ue8m0(p, s));
}

namespace {
int fused_a(uint16_t* c, const void* a, bool bf16, const uint8_t* b, const float* sb, int64_t M,
            int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  if (!c || !a || !b || !sb) return DG_ERR_NULL;
  if (M < 1 || M > DG_FUSED_A_MAX_M || N < 8 || K < 128) return DG_ERR_SHAPE;
  if (N % 8 != 0 || K % 128 != 0) return DG_ERR_SHAPE;
  if (N > INT32_MAX || K > INT32_MAX || N * K > kU32) return DG_ERR_SHAPE;
  if (!dg::skinny_applies(M, N, K)) return DG_ERR_SHAPE;
  if (!aligned(c, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(sb, 4))
    return DG_ERR_ALIGN;
  const int st = check_workspace(M, N, K, &workspace, &workspace_bytes);
  if (st != DG_OK) return st;
  dg::GemmProblem p{c, nullptr, b, nullptr, sb, nullptr, 1, 1, M, N, K};
  return from_hip(dg::launch_gemm_skinny_fused_a(p, a, bf16, workspace, workspace_bytes,
                                                 static_cast<hipStream_t>(stream)));
}
}  // namespace

int dg_fp8_gemm_nt_fused_a(uint16_t* c, const float* a, const uint8_t* b, const float* sb,
                           int64_t M, int64_t N, int64_t K, void* workspace,
                           size_t workspace_bytes, void* stream) {
  return fused_a(c, a, false, b, sb, M, N, K, workspace, workspace_bytes, stream);
}

int dg_fp8_gemm_nt_fused_a_bf16(uint16_t* c, const uint16_t* a, const uint8_t* b, const float* sb,
                                int64_t M, int64_t N, int64_t K, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return fused_a(c, a, true, b, sb, M, N, K, workspace, workspace_bytes, stream);
}

int dg_transpose_fp8(uint8_t* out, const uint8_t* in, int64_t rows, int64_t cols, void* stream) {
  if (!out || !in) return DG_ERR_NULL;
  if (rows < 16 || cols < 16 || rows % 16 != 0 || cols % 16 != 0) return DG_ERR_SHAPE;
  if ((rows + 127) / 128 > kMaxGridY || (cols + 127) / 128 > INT32_MAX) return DG_ERR_SHAPE;
  if (rows > INT64_MAX / cols) return DG_ERR_SHAPE;
  if (!aligned(out, 16) || !aligned(in, 16)) return DG_ERR_ALIGN;
  const uint8_t* o = out;
  if (o < in + rows * cols && in < o + rows * cols) return DG_ERR_UNSUPPORTED;  // overlap
  return from_hip(dg::launch_transpose_u8(out, in, rows, cols, static_cast<hipStream_t>(stream)));
}

size_t dg_fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int layout) {
  if (M < 1 || N < 1 || K < 1 || layout < DG_LAYOUT_NT || layout > DG_LAYOUT_TT) return 0;
  const size_t nt = dg_fp8_gemm_nt_workspace_bytes(M, N, K);
  if (layout == DG_LAYOUT_NT) return nt;
  // split-K region (at least the counter region, which the transposes never
  // touch) first, then the transposed copies
  return (nt > DG_WORKSPACE_COUNTER_BYTES ? nt : DG_WORKSPACE_COUNTER_BYTES) +
         transpose_bytes(M, N, K, layout);
}

int dg_fp8_gemm(uint16_t* c, const uint8_t* a, const uint8_t* b, const float* sa, const float* sb,
                int a_block_rows, int64_t M, int64_t N, int64_t K, int layout, void* workspace,
                size_t workspace_bytes, void* stream) {
  if (layout < DG_LAYOUT_NT || layout > DG_LAYOUT_TT) return DG_ERR_UNSUPPORTED;
  if (layout == DG_LAYOUT_NT)
    return dg_fp8_gemm_nt(c, a, b, sa, sb, a_block_rows, M, N, K, workspace, workspace_bytes,
                          stream);
  // every check, the NT GEMM's included, before the first launch
  int st = check_gemm(c, a, b, sa, sb, a_block_rows, M, N, K);
  if (st != DG_OK) return st;
  const bool a_t = layout == DG_LAYOUT_TN || layout == DG_LAYOUT_TT;  // A given [K][M]
  const bool b_n = layout == DG_LAYOUT_TN || layout == DG_LAYOUT_NN;  // B given [K][N]
  if ((a_t && M % 16 != 0) || (b_n && N % 16 != 0)) return DG_ERR_SHAPE;
  if ((a_t && (K + 127) / 128 > kMaxGridY) || (b_n && (K + 127) / 128 > kMaxGridY))
    return DG_ERR_SHAPE;
  const bool skinny = dg::skinny_applies(M, N, K);
  if (!skinny && ((M + 255) / 256) * ((N + 255) / 256) > INT32_MAX) return DG_ERR_SHAPE;
  const size_t tb = transpose_bytes(M, N, K, layout);
  if (!workspace || workspace_bytes < DG_WORKSPACE_COUNTER_BYTES + tb) return DG_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return DG_ERR_ALIGN;
  // split-K when the workspace also holds the plan's partials after the
  // copies; otherwise the copies follow the (untouched) counter region
  const size_t split = skinny ? dg::skinny_workspace_bytes(M, N, K) : 0;
  const bool use_split = split > 0 && workspace_bytes >= split + tb;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  size_t used = use_split ? split : DG_WORKSPACE_COUNTER_BYTES;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const uint8_t* ak = a;
  const uint8_t* bk = b;
  if (a_t) {
    st = from_hip(dg::launch_transpose_u8(ws + used, a, K, M, s));  // [K][M] -> [M][K]
    if (st != DG_OK) return st;
    ak = ws + used;
    used += align16(M * K);
  }
  if (b_n) {
    st = from_hip(dg::launch_transpose_u8(ws + used, b, K, N, s));  // [K][N] -> [N][K]
    if (st != DG_OK) return st;
    bk = ws + used;
    used += align16(N * K);
  }
  return dg_fp8_gemm_nt(c, ak, bk, sa, sb, a_block_rows, M, N, K, use_split ? workspace : nullptr,
                        use_split ? split : 0, stream);
}

int dg_fp8_grouped_gemm_k(uint16_t* c, const uint8_t* a, const uint8_t* b, const float* sa,
                          const float* sb, int a_block_rows, const int64_t* k_offsets,
                          int num_groups, int64_t M, int64_t N, int64_t K, void* stream) {
  int st = check_gemm(c, a, b, sa, sb, a_block_rows, M, N, K);
  if (st != DG_OK) return st;
  if (!k_offsets) return DG_ERR_NULL;
  if (!aligned(k_offsets, 8)) return DG_ERR_ALIGN;
  if (num_groups < 1) return DG_ERR_UNSUPPORTED;
  const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
  if (tiles * num_groups > INT32_MAX) return DG_ERR_SHAPE;
  if (M * N > INT64_MAX / num_groups) return DG_ERR_SHAPE;
  dg::GemmProblem p{c, a, b, sa, sb, nullptr, num_groups, a_block_rows, M, N, K};
  p.k_offsets = k_offsets;
  return from_hip(dg::launch_gemm_tiled_kgrouped(p, static_cast<hipStream_t>(stream)));
}

int dg_fp8_grouped_gemm_contig(uint16_t* c, const uint8_t* a, const uint8_t* b, const float* sa,
                               const float* sb, int a_block_rows, const int32_t* m_indices,
                               int num_groups, int64_t M, int64_t N, int64_t K, void* stream) {
  return dg_fp8_grouped_gemm_contig_epilogue(c, a, b, sa, sb, a_block_rows, m_indices, num_groups,
                                             M, N, K, DG_EPI_NONE, nullptr, stream);
}

int dg_fp8_grouped_gemm_contig_epilogue(uint16_t* c, const uint8_t* a, const uint8_t* b,
                                        const float* sa, const float* sb, int a_block_rows,
                                        const int32_t* m_indices, int num_groups, int64_t M,
                                        int64_t N, int64_t K, int act, const uint16_t* residual,
                                        void* stream) {
  return dg_fp8_grouped_gemm_contig_balanced(c, a, b, sa, sb, a_block_rows, m_indices, num_groups,
                                             M, N, K, act, residual, nullptr, 0, stream);
}

size_t dg_fp8_grouped_gemm_contig_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 128 || M % 128 != 0 || N < 8 || K < 128 || K % 128 != 0) return 0;
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return 0;
  return dg::grouped_balanced_workspace_bytes(M, N, K);
}

int dg_fp8_grouped_gemm_contig_balanced(uint16_t* c, const uint8_t* a, const uint8_t* b,
                                        const float* sa, const float* sb, int a_block_rows,
                                        const int32_t* m_indices, int num_groups, int64_t M,
                                        int64_t N, int64_t K, int act, const uint16_t* residual,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_gemm(c, a, b, sa, sb, a_block_rows, M, N, K);
  if (st != DG_OK) return st;
  if (!m_indices) return DG_ERR_NULL;
  if (!aligned(m_indices, 4)) return DG_ERR_ALIGN;
  if (num_groups < 1) return DG_ERR_UNSUPPORTED;
  if (act < DG_EPI_NONE || act > DG_EPI_SWIGLU) return DG_ERR_UNSUPPORTED;
  if (residual && !aligned(residual, 16)) return DG_ERR_ALIGN;
  if (M % 128 != 0) return DG_ERR_SHAPE;
  if ((int64_t)num_groups * N * K / num_groups != N * K) return DG_ERR_SHAPE;
  if (workspace != nullptr && workspace_bytes > 0) {
    if (workspace_bytes < dg::grouped_balanced_workspace_bytes(M, N, K)) return DG_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return DG_ERR_ALIGN;
  } else {
    workspace = nullptr;  // one of the two missing: one workgroup per tile
    workspace_bytes = 0;
  }
  dg::GemmProblem p{c, a, b, sa, sb, m_indices, num_groups, a_block_rows, M, N, K};
  p.epi.act = act;
  p.epi.res = residual;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!workspace) return from_hip(dg::launch_gemm_tiled(p, true, s));
  return from_hip(dg::launch_gemm_grouped_balanced(p, workspace, workspace_bytes, s));
}

int dg_fp8_grouped_gemm_contig_ue8m0(uint16_t* c, const uint8_t* a, const uint8_t* b,
                                     const int32_t* sfa, const int32_t* sfb, int a_block_rows,
                                     const int32_t* m_indices, int num_groups, int64_t M,
                                     int64_t N, int64_t K, void* stream) {
  int st = check_gemm(c, a, b, reinterpret_cast<const float*>(sfa),
                      reinterpret_cast<const float*>(sfb), a_block_rows, M, N, K);
  if (st != DG_OK) return st;
  if (!m_indices) return DG_ERR_NULL;
  if (!aligned(m_indices, 4)) return DG_ERR_ALIGN;
  if (num_groups < 1) return DG_ERR_UNSUPPORTED;
  if (M % 128 != 0) return DG_ERR_SHAPE;
  if ((int64_t)num_groups * N * K / num_groups != N * K) return DG_ERR_SHAPE;
  dg::GemmProblem p{c, a, b, nullptr, nullptr, m_indices, num_groups, a_block_rows, M, N, K};
  p.sfa = reinterpret_cast<const uint32_t*>(sfa);
  p.sfb = reinterpret_cast<const uint32_t*>(sfb);
  return from_hip(dg::launch_gemm_tiled_grouped_ue8m0(p, static_cast<hipStream_t>(stream)));
}

int dg_fp8_grouped_gemm_masked_ue8m0(uint16_t* c, const uint8_t* a, const uint8_t* b,
                                     const int32_t* sfa, const int32_t* sfb, int a_block_rows,
                                     const int32_t* masked_m, int num_groups, int64_t max_m,
                                     int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  int st = check_gemm(c, a, b, reinterpret_cast<const float*>(sfa),
                      reinterpret_cast<const float*>(sfb), a_block_rows, max_m, N, K);
  if (st != DG_OK) return st;
  if (!masked_m) return DG_ERR_NULL;
  if (!aligned(masked_m, 4)) return DG_ERR_ALIGN;
  if (num_groups < 1) return DG_ERR_UNSUPPORTED;
  if (max_m > INT64_MAX / K / num_groups || max_m > INT64_MAX / N / num_groups)
    return DG_ERR_SHAPE;
  if (dg::skinny_masked_grid(num_groups, max_m, N, K) > INT32_MAX) return DG_ERR_SHAPE;
  if (workspace != nullptr && workspace_bytes > 0) {
    if (workspace_bytes < dg::skinny_masked_workspace_bytes(num_groups, max_m, N, K))
      return DG_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return DG_ERR_ALIGN;
  } else {
    workspace = nullptr;
    workspace_bytes = 0;
  }
  dg::GemmProblem p{c, a, b, nullptr, nullptr, nullptr, num_groups, a_block_rows, max_m, N, K};
  p.sfa = reinterpret_cast<const uint32_t*>(sfa);
  p.sfb = reinterpret_cast<const uint32_t*>(sfb);
  return from_hip(dg::launch_gemm_skinny_masked(p, masked_m, max_m, workspace, workspace_bytes,
                                                static_cast<hipStream_t>(stream)));
}

size_t dg_fp8_grouped_gemm_masked_workspace_bytes(int num_groups, int64_t max_m, int64_t N,
                                                  int64_t K) {
  if (num_groups < 1 || max_m < 1 || N < 1 || K < 1) return 0;
  return dg::skinny_masked_workspace_bytes(num_groups, max_m, N, K);
}

int dg_fp8_grouped_gemm_masked(uint16_t* c, const uint8_t* a, const uint8_t* b, const float* sa,
                               const float* sb, int a_block_rows, const int32_t* masked_m,
                               int num_groups, int64_t max_m, int64_t N, int64_t K,
                               void* workspace, size_t workspace_bytes, void* stream) {
  return dg_fp8_grouped_gemm_masked_epilogue(c, a, b, sa, sb, a_block_rows, masked_m, num_groups,
                                             max_m, N, K, DG_EPI_NONE, nullptr, workspace,
                                             workspace_bytes, stream);
}

int dg_fp8_grouped_gemm_masked_epilogue(uint16_t* c, const uint8_t* a, const uint8_t* b,
                                        const float* sa, const float* sb, int a_block_rows,
                                        const int32_t* masked_m, int num_groups, int64_t max_m,
                                        int64_t N, int64_t K, int act, const uint16_t* residual,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_gemm(c, a, b, sa, sb, a_block_rows, max_m, N, K);
  if (st != DG_OK) return st;
  if (!masked_m) return DG_ERR_NULL;
  if (!aligned(masked_m, 4)) return DG_ERR_ALIGN;
  if (num_groups < 1) return DG_ERR_UNSUPPORTED;
  if (act < DG_EPI_NONE || act > DG_EPI_SWIGLU) return DG_ERR_UNSUPPORTED;
  if (residual && !aligned(residual, 16)) return DG_ERR_ALIGN;
  if (max_m > INT64_MAX / K / num_groups || max_m > INT64_MAX / N / num_groups)
    return DG_ERR_SHAPE;
  if (dg::skinny_masked_grid(num_groups, max_m, N, K) > INT32_MAX) return DG_ERR_SHAPE;
  if (workspace != nullptr && workspace_bytes > 0) {
    if (workspace_bytes < dg::skinny_masked_workspace_bytes(num_groups, max_m, N, K))
      return DG_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return DG_ERR_ALIGN;
  } else {
    workspace = nullptr;
    workspace_bytes = 0;
  }
  dg::GemmProblem p{c, a, b, sa, sb, nullptr, num_groups, a_block_rows, max_m, N, K};
  p.epi.act = act;
  p.epi.res = residual;
  return from_hip(dg::launch_gemm_skinny_masked(p, masked_m, max_m, workspace, workspace_bytes,
                                                static_cast<hipStream_t>(stream)));
}

int dg_fp8_gemm_nt_noalloc(uint16_t* c, const uint8_t* a, const uint8_t* b, const float* sa,
                           const float* sb, int a_block_rows, int64_t M, int64_t N, int64_t K,
                           void* stream) {
  const int st = check_gemm(c, a, b, sa, sb, a_block_rows, M, N, K);
  if (st != DG_OK) return st;
  // plans that split K: the LDS-ring small-M kernel with a non-zero workspace
  const bool split = dg::skinny_applies(M, N, K) && !dg::stream_preferred(M, N, K) &&
                     dg::skinny_workspace_bytes(M, N, K) > 0;
  if (!split) return dg_fp8_gemm_nt(c, a, b, sa, sb, a_block_rows, M, N, K, nullptr, 0, stream);
  const size_t need = dg::skinny_workspace_bytes(M, N, K);
  if (need > DG_NOALLOC_SCRATCH_BYTES) return DG_ERR_SCRATCH;
  hipStream_t s = static_cast<hipStream_t>(stream);
  int cur = 0;
  if (hipGetDevice(&cur) != hipSuccess) return DG_ERR_HIP;
  if (s) {  // the scratch address is the current device's
    int sdev = 0;
    if (hipStreamGetDevice(s, &sdev) != hipSuccess) return DG_ERR_HIP;
    if (sdev != cur) return DG_ERR_UNSUPPORTED;
  }
  void* ws = nullptr;
  if (dg::noalloc_scratch(&ws) != hipSuccess) return DG_ERR_HIP;
  const int zs = from_hip(dg::launch_zero_counters(ws, s));
  if (zs != DG_OK) return zs;
  return dg_fp8_gemm_nt(c, a, b, sa, sb, a_block_rows, M, N, K, ws, need, stream);
}

// ---- MXFP4 and the mixture-of-experts layer ----

namespace {

constexpr int64_t kMaxScaleWords = int64_t(1) << 29;  // scale arrays below 2^31 bytes

bool scale_words_ok(int64_t rows, int64_t cols) {
  return rows < kMaxScaleWords && cols < kMaxScaleWords &&
         (cols + 127) / 128 <= (kMaxScaleWords - 1) / rows;
}

int check_mxfp4(const void* c, const void* a, const void* b, const void* sfb, int64_t M, int64_t N,
                int64_t K) {
  if (!c || !a || !b || !sfb) return DG_ERR_NULL;
  if (M < 1 || N < 1 || K < 32 || K % 32 != 0 || K > (int64_t(1) << 23)) return DG_ERR_SHAPE;
  if (!scale_words_ok(M, K) || !scale_words_ok(N, K) || M > (int64_t(1) << 44) / N)
    return DG_ERR_SHAPE;
  if (!aligned(c, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(sfb, 4))
    return DG_ERR_ALIGN;
  return DG_OK;
}

int run_mxfp4(const dg::Mxfp4Problem& p, void* workspace, size_t workspace_bytes, void* stream) {
  if (workspace != nullptr && workspace_bytes > 0) {
    if (workspace_bytes < dg::mxfp4_workspace_bytes(p.M, p.N, p.K, p.sfa == nullptr))
      return DG_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return DG_ERR_ALIGN;
  } else {
    workspace = nullptr;
    workspace_bytes = 0;
  }
  return from_hip(dg::launch_gemm_mxfp4(p, workspace, workspace_bytes,
                                        static_cast<hipStream_t>(stream)));
}

}  // namespace

int dg_quantize_mxfp4(uint8_t* q, int32_t* sf, uint8_t* qt, int32_t* sft, const void* x, int dtype,
                      int64_t rows, int64_t cols, int64_t ldx, void* stream) {
  if (!x || (!q && !qt) || !q != !sf || !qt != !sft) return DG_ERR_NULL;
  if (dtype != DG_DTYPE_F32 && dtype != DG_DTYPE_BF16) return DG_ERR_UNSUPPORTED;
  if (rows < 1 || rows > (1 << 22) || cols < 1 || ldx < cols || ldx > INT64_MAX / 4 / rows) return DG_ERR_SHAPE;
  if (!scale_words_ok(rows, cols) || !scale_words_ok(cols, rows)) return DG_ERR_SHAPE;
  if (!aligned(x, dtype == DG_DTYPE_BF16 ? 2 : 4) || !aligned(q, 16) || !aligned(qt, 16) ||
      !aligned(sf, 4) || !aligned(sft, 4))
    return DG_ERR_ALIGN;
  return from_hip(dg::launch_quantize_mxfp4(q, reinterpret_cast<uint32_t*>(sf), qt,
                                            reinterpret_cast<uint32_t*>(sft), x,
                                            dtype == DG_DTYPE_BF16, rows, cols, ldx,
                                            static_cast<hipStream_t>(stream)));
}

int dg_dequantize_mxfp4(void* out, int dtype, const uint8_t* q, const int32_t* sf, int64_t rows,
                        int64_t cols, void* stream) {
  if (!out || !q || !sf) return DG_ERR_NULL;
  if (dtype != DG_DTYPE_F32 && dtype != DG_DTYPE_BF16) return DG_ERR_UNSUPPORTED;
  if (rows < 1 || cols < 1 || !scale_words_ok(rows, cols)) return DG_ERR_SHAPE;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(sf, 4)) return DG_ERR_ALIGN;
  return from_hip(dg::launch_dequantize_mxfp4(out, dtype == DG_DTYPE_BF16, q,
                                              reinterpret_cast<const uint32_t*>(sf), rows, cols,
                                              static_cast<hipStream_t>(stream)));
}

size_t dg_mxfp4_gemm_nt_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 1) return 0;
  return dg::mxfp4_workspace_bytes(M, N, K, false);
}

int dg_mxfp4_gemm_nt(uint16_t* c, const uint8_t* a, const uint8_t* b, const int32_t* sfa,
                     const int32_t* sfb, int64_t M, int64_t N, int64_t K, void* workspace,
                     size_t workspace_bytes, void* stream) {
  const int st = check_mxfp4(c, a, b, sfb, M, N, K);
  if (st != DG_OK) return st;
  if (!sfa) return DG_ERR_NULL;
  if (!aligned(sfa, 4)) return DG_ERR_ALIGN;
  const dg::Mxfp4Problem p{c, a, b, reinterpret_cast<const uint32_t*>(sfa),
                           reinterpret_cast<const uint32_t*>(sfb), M, N, K};
  return run_mxfp4(p, workspace, workspace_bytes, stream);
}

size_t dg_mxfp4_gemm_nt_bf16a_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 1) return 0;
  return dg::mxfp4_workspace_bytes(M, N, K, true);
}

int dg_mxfp4_gemm_nt_bf16a(uint16_t* c, const uint16_t* a, const uint8_t* b, const int32_t* sfb,
                           int64_t M, int64_t N, int64_t K, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const int st = check_mxfp4(c, a, b, sfb, M, N, K);
  if (st != DG_OK) return st;
  if (M > DG_MXFP4_BF16A_MAX_M) return DG_ERR_SHAPE;
  const dg::Mxfp4Problem p{c, a, b, nullptr, reinterpret_cast<const uint32_t*>(sfb), M, N, K};
  return run_mxfp4(p, workspace, workspace_bytes, stream);
}

namespace {

// H / 16 column tiles each have an arrival counter in the workspace
static_assert(131072 / 16 * 4 <= DG_WORKSPACE_COUNTER_BYTES, "counters of the layer");

bool moe_shape_ok(int T, int E, int k, int64_t H, int64_t I) {
  return T >= 1 && T <= DG_MOE_MAX_TOKENS && E >= 1 && E <= DG_MOE_MAX_EXPERTS && k >= 1 &&
         k <= E && k <= DG_MOE_MAX_SLOTS && H >= 32 && H <= 131072 && I >= 32 &&
         I <= (int64_t(1) << 20) && int64_t(T) * k * I < (int64_t(1) << 29) &&  // as dg.h says
         scale_words_ok(2 * I, H) && scale_words_ok(H, I);
}

}  // namespace

size_t dg_moe_layer_workspace_bytes(int T, int E, int k, int64_t H, int64_t I) {
  return moe_shape_ok(T, E, k, H, I) ? dg::moe_workspace_bytes(T, E, k, H, I) : 0;
}

int dg_moe_layer(uint16_t* y, const uint16_t* x, const uint8_t* w13, const uint8_t* w2,
                 const void* s13, const void* s2, int format, int32_t* ids, float* weights,
                 const float* logits, int scoring, int T, int E, int k, int64_t H, int64_t I,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!y || !x || !w13 || !w2 || !s13 || !s2 || !ids || !weights) return DG_ERR_NULL;
  if (format != DG_MOE_MXFP4 && format != DG_MOE_FP8) return DG_ERR_UNSUPPORTED;
  if (logits && scoring != DG_MOE_SOFTMAX && scoring != DG_MOE_SIGMOID) return DG_ERR_UNSUPPORTED;
  const int64_t step = format == DG_MOE_FP8 ? 128 : 32;
  if (!moe_shape_ok(T, E, k, H, I) || H % step != 0 || I % step != 0) return DG_ERR_SHAPE;
  if (!workspace || workspace_bytes < dg::moe_workspace_bytes(T, E, k, H, I))
    return DG_ERR_WORKSPACE;
  if (!aligned(y, 16) || !aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16) ||
      !aligned(workspace, 16) || !aligned(s13, 4) || !aligned(s2, 4) || !aligned(ids, 4) ||
      !aligned(weights, 4) || !aligned(logits, 4))
    return DG_ERR_ALIGN;
  dg::MoeProblem p{y, x, w13, w2, s13, s2, ids, weights, logits, scoring, format, T, E, k, H, I};
  return from_hip(dg::launch_moe_layer(p, workspace, static_cast<hipStream_t>(stream)));
}

// ---- around the grouped products ----

namespace {

bool dtype_ok(int dtype) { return dtype == DG_DTYPE_F32 || dtype == DG_DTYPE_BF16; }
size_t dtype_size(int dtype) { return dtype == DG_DTYPE_BF16 ? 2 : 4; }

static_assert(DG_MOE_SOFTMAX == dg::ROUTE_SOFTMAX && DG_MOE_SIGMOID == dg::ROUTE_SIGMOID &&
              DG_MOE_MAX_SLOTS == dg::kMoeMaxSlots && DG_MOE_MAX_EXPERTS == dg::kMoeMaxExperts,
              "constants of dg.h and of the kernels");

// Tokens, experts and slots.
bool experts_ok(int64_t T, int E, int k, int64_t most) {
  return T >= 1 && T <= most && E >= 1 && E <= DG_MOE_MAX_EXPERTS && k >= 1 && k <= E &&
         k <= DG_MOE_MAX_SLOTS;
}
bool plan_ok(int64_t T, int E, int k) {
  return experts_ok(T, E, k, int64_t(1) << 27) && T * k <= (int64_t(1) << 27);
}

int check_route(const void* ids, const void* weights, const void* logits, int dtype, int64_t ldl,
                int scoring, int64_t T, int E, int k) {
  if (!ids || !weights || !logits) return DG_ERR_NULL;
  if (!dtype_ok(dtype) || (scoring != DG_MOE_SOFTMAX && scoring != DG_MOE_SIGMOID))
    return DG_ERR_UNSUPPORTED;
  if (!experts_ok(T, E, k, int64_t(1) << 25) || ldl < E || ldl > INT64_MAX / 4 / T)
    return DG_ERR_SHAPE;
  if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(logits, dtype_size(dtype)))
    return DG_ERR_ALIGN;
  return DG_OK;
}

// Tokens and rows of `cols` columns in the layout (multiples of `step`).
bool layout_ok(int64_t T, int k, int64_t M, int64_t cols, int64_t step) {
  if (T < 1 || k < 1 || k > DG_MOE_MAX_SLOTS || M < 128 || M % 128 != 0 || cols < step ||
      cols % step != 0 || cols > (int64_t(1) << 34))
    return false;
  const int64_t parts = (cols + 511) / 512;
  // launches of 256 threads have fewer than 2^24 workgroups
  return T <= (int64_t(1) << 23) && T <= (int64_t(1) << 25) / parts && M <= (int64_t(1) << 27) / parts;
}

int check_swiglu(const int32_t* m_indices, int64_t M, int64_t I) {
  // a workgroup takes 4 to 16 rows by 512 units: fewer than 2^24 of them for one row too
  if (M < 1 || I < 128 || I % 128 != 0 || I > (int64_t(1) << 32)) return DG_ERR_SHAPE;
  if (M > (int64_t(1) << 25) / ((I + 511) / 512)) return DG_ERR_SHAPE;
  if (m_indices && M % 128 != 0) return DG_ERR_SHAPE;
  return aligned(m_indices, 4) ? DG_OK : DG_ERR_ALIGN;
}

}  // namespace

int dg_moe_route(int32_t* ids, float* weights, const void* logits, int dtype, int64_t ldl,
                 const float* bias, int scoring, int groups, int top_groups, int group_best,
                 int renormalise, float scale, int64_t T, int E, int k, void* stream) {
  const int st = check_route(ids, weights, logits, dtype, ldl, scoring, T, E, k);
  if (st != DG_OK) return st;
  if (group_best != 1 && group_best != 2) return DG_ERR_UNSUPPORTED;
  if (groups < 1 || groups > DG_ROUTE_MAX_GROUPS || E % groups != 0 || top_groups < 1 ||
      top_groups > groups || E / groups < group_best)
    return DG_ERR_SHAPE;
  if (!aligned(bias, 4)) return DG_ERR_ALIGN;
  dg::RouteArgs p{};
  p.ids = ids;
  p.weights = weights;
  p.logits = logits;
  p.bias = bias;
  p.bf16 = dtype == DG_DTYPE_BF16;
  p.renormalise = renormalise != 0;
  p.scoring = scoring;
  p.groups = groups;
  p.top_groups = top_groups;
  p.best = group_best;
  p.scale = scale;
  p.T = T;
  p.ldl = ldl;
  p.E = E;
  p.k = k;
  return from_hip(dg::launch_route(p, static_cast<hipStream_t>(stream)));
}

int dg_moe_route_backward(void* dlogits, int64_t ldd, const float* dweights, const int32_t* ids,
                          const void* logits, int dtype, int64_t ldl, int scoring,
                          int renormalise, float scale, int64_t T, int E, int k, void* stream) {
  if (!dlogits) return DG_ERR_NULL;
  const int st = check_route(ids, dweights, logits, dtype, ldl, scoring, T, E, k);
  if (st != DG_OK) return st;
  if (ldd < E || ldd > INT64_MAX / 4 / T) return DG_ERR_SHAPE;
  if (!aligned(dlogits, dtype_size(dtype))) return DG_ERR_ALIGN;
  dg::RouteArgs p{};
  p.ids = const_cast<int32_t*>(ids);
  p.dlogits = dlogits;
  p.dweights = dweights;
  p.logits = logits;
  p.bf16 = dtype == DG_DTYPE_BF16;
  p.renormalise = renormalise != 0;
  p.scoring = scoring;
  p.scale = scale;
  p.T = T;
  p.ldl = ldl;
  p.ldd = ldd;
  p.E = E;
  p.k = k;
  return from_hip(dg::launch_route_backward(p, static_cast<hipStream_t>(stream)));
}

int64_t dg_moe_plan_rows(int64_t T, int E, int k) {
  return plan_ok(T, E, k) ? dg::plan_rows(T, E, k) : 0;
}

size_t dg_moe_plan_workspace_bytes(int64_t T, int E, int k) {
  return plan_ok(T, E, k) ? dg::plan_workspace_bytes(T, E, k) : 0;
}

int dg_moe_plan(int32_t* rows, int32_t* pairs, int32_t* m_indices, int64_t* offsets,
                int32_t* counts, const int32_t* ids, int64_t T, int E, int k, int64_t M,
                void* workspace, size_t workspace_bytes, void* stream) {
  if (!rows || !pairs || !m_indices || !offsets || !counts || !ids) return DG_ERR_NULL;
  if (!plan_ok(T, E, k) || M % 128 != 0 || M < dg::plan_rows(T, E, k) || M > (int64_t(1) << 30))
    return DG_ERR_SHAPE;
  const size_t need = dg::plan_workspace_bytes(T, E, k);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DG_ERR_WORKSPACE;
  if (!aligned(rows, 4) || !aligned(pairs, 4) || !aligned(m_indices, 4) || !aligned(offsets, 8) ||
      !aligned(counts, 4) || !aligned(ids, 4) || !aligned(workspace, 16))
    return DG_ERR_ALIGN;
  dg::PlanArgs p{rows, pairs, m_indices, offsets, counts, ids, T * k, M, E, 0, 0, nullptr};
  return from_hip(dg::launch_plan(p, workspace, static_cast<hipStream_t>(stream)));
}

namespace {

// A workspace for the scales is optional; one that is given has to hold them.
int check_scales(const dg::DispatchArgs& p, void** workspace, size_t workspace_bytes) {
  const size_t need = dg::dispatch_workspace_bytes(p.T, p.k, p.H, p.weights != nullptr);
  if (*workspace == nullptr || workspace_bytes == 0 || need == 0) *workspace = nullptr;
  else if (workspace_bytes < need) return DG_ERR_WORKSPACE;
  return aligned(*workspace, 16) ? DG_OK : DG_ERR_ALIGN;
}

}  // namespace

size_t dg_moe_dispatch_fp8_workspace_bytes(int64_t T, int k, int64_t H, int weighted) {
  return layout_ok(T, k, 128, H, 128) ? dg::dispatch_workspace_bytes(T, k, H, weighted != 0) : 0;
}

int dg_moe_dispatch_fp8(uint8_t* a, float* sa, const void* x, int dtype, int64_t ldx,
                        const int32_t* rows, const int32_t* pairs, const float* weights,
                        int64_t T, int k, int64_t M, int64_t H, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!a || !sa || !x || !rows || !pairs) return DG_ERR_NULL;
  if (!dtype_ok(dtype)) return DG_ERR_UNSUPPORTED;
  if (!layout_ok(T, k, M, H, 128) || ldx < H || ldx > INT64_MAX / 4 / T) return DG_ERR_SHAPE;
  if (!aligned(a, 16) || !aligned(sa, 4) || !aligned(x, dtype_size(dtype)) || !aligned(rows, 4) ||
      !aligned(pairs, 4) || !aligned(weights, 4))
    return DG_ERR_ALIGN;
  const dg::DispatchArgs p{a, sa, x, dtype == DG_DTYPE_BF16, rows, pairs, weights, T, ldx, M, H, k,
                           0, nullptr};
  const int st = check_scales(p, &workspace, workspace_bytes);
  return st != DG_OK ? st : from_hip(dg::launch_dispatch(p, workspace, static_cast<hipStream_t>(stream)));
}

int dg_moe_combine(uint16_t* y, const uint16_t* c, const int32_t* rows, const float* weights,
                   const uint16_t* residual, int64_t T, int k, int64_t M, int64_t H,
                   void* stream) {
  if (!y || !c || !rows) return DG_ERR_NULL;
  if (!layout_ok(T, k, M, H, 8)) return DG_ERR_SHAPE;
  if (!aligned(y, 16) || !aligned(c, 16) || !aligned(residual, 16) || !aligned(rows, 4) ||
      !aligned(weights, 4))
    return DG_ERR_ALIGN;
  const dg::CombineArgs p{y, c, rows, weights, residual, nullptr, nullptr, T, M, H, 0, k};
  return from_hip(dg::launch_combine(p, static_cast<hipStream_t>(stream)));
}

int dg_moe_combine_backward(uint8_t* dc, float* sdc, float* dweights, const uint16_t* dy,
                            int64_t lddy, const uint16_t* c, const int32_t* rows,
                            const int32_t* pairs, const float* weights, int64_t T, int k,
                            int64_t M, int64_t H, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (!dy || !rows || (!dc && !dweights) || !dc != !sdc || (dc && !pairs) || (dweights && !c))
    return DG_ERR_NULL;
  if (!layout_ok(T, k, M, H, 128) || lddy < H || lddy > INT64_MAX / 4 / T) return DG_ERR_SHAPE;
  if (!aligned(dc, 16) || !aligned(c, 16) || !aligned(dy, 2) || !aligned(sdc, 4) ||
      !aligned(dweights, 4) || !aligned(rows, 4) || !aligned(pairs, 4) || !aligned(weights, 4))
    return DG_ERR_ALIGN;
  hipStream_t q = static_cast<hipStream_t>(stream);
  const dg::DispatchArgs d{dc, sdc, dy, true, rows, pairs, weights, T, lddy, M, H, k, 0, nullptr};
  if (dc) {
    const int st = check_scales(d, &workspace, workspace_bytes);
    if (st != DG_OK) return st;
    if (!dweights) return from_hip(dg::launch_dispatch(d, workspace, q));
  }
  const dg::CombineArgs p{nullptr, c, rows, weights, nullptr, dweights, dy, T, M, H, lddy, k};
  return from_hip(dg::launch_combine_backward(p, d, workspace, q));
}

int dg_swiglu_fp8(uint8_t* h, float* sh, uint8_t* kept, float* skept, const uint16_t* gu,
                  const int32_t* m_indices, int64_t M, int64_t I, void* stream) {
  if (!h || !sh || !gu || !kept != !skept) return DG_ERR_NULL;
  const int st = check_swiglu(m_indices, M, I);
  if (st != DG_OK) return st;
  if (!aligned(h, 16) || !aligned(kept, 16) || !aligned(gu, 16) || !aligned(sh, 4) ||
      !aligned(skept, 4))
    return DG_ERR_ALIGN;
  const dg::SwigluArgs p{h, sh, kept, skept, gu, nullptr, nullptr, nullptr, m_indices, M, I, 0};
  return from_hip(dg::launch_swiglu(p, false, static_cast<hipStream_t>(stream)));
}

int dg_swiglu_fp8_backward(uint8_t* dgu, float* sdgu, uint8_t* h, float* sh, const uint16_t* dh,
                           const uint8_t* kept, const float* skept, const int32_t* m_indices,
                           int64_t M, int64_t I, void* stream) {
  if (!dgu || !sdgu || !dh || !kept || !skept || !h != !sh) return DG_ERR_NULL;
  const int st = check_swiglu(m_indices, M, I);
  if (st != DG_OK) return st;
  if (!aligned(dgu, 16) || !aligned(h, 16) || !aligned(dh, 16) || !aligned(kept, 16) ||
      !aligned(sdgu, 4) || !aligned(sh, 4) || !aligned(skept, 4))
    return DG_ERR_ALIGN;
  const dg::SwigluArgs p{h, sh, const_cast<uint8_t*>(kept), const_cast<float*>(skept),
                         nullptr, dh, dgu, sdgu, m_indices, M, I, 0};
  return from_hip(dg::launch_swiglu(p, true, static_cast<hipStream_t>(stream)));
}

int dg_transpose_fp8_blocks(uint8_t* qt, float* st, int block_rows, const uint8_t* q,
                            const float* s, const int32_t* m_indices, int64_t M, int64_t C,
                            void* stream) {
  if (!qt || !st || !q || !s) return DG_ERR_NULL;
  if (block_rows != 1 && block_rows != 128) return DG_ERR_UNSUPPORTED;
  if (M < 128 || C < 128 || M % 128 != 0 || C % 128 != 0) return DG_ERR_SHAPE;
  if (M / 128 > (int64_t(1) << 23) / (C / 128)) return DG_ERR_SHAPE;
  if (!aligned(qt, 16) || !aligned(q, 16) || !aligned(st, 4) || !aligned(s, 4) ||
      !aligned(m_indices, 4))
    return DG_ERR_ALIGN;
  const uintptr_t a = reinterpret_cast<uintptr_t>(q), b = reinterpret_cast<uintptr_t>(qt);
  const uintptr_t n = (uintptr_t)(M * C);
  if (a < b + n && b < a + n) return DG_ERR_UNSUPPORTED;
  const dg::TransposeArgs p{qt, st, q, s, m_indices, M, C};
  return from_hip(dg::launch_transpose_blocks(p, block_rows == 1, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
