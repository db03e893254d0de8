// Probe of fp8_rows.hpp, not part of the library's C ABI: what reciprocal_rn and
// row_scale give for a list of numbers, for a test that compares them with the host's
// divisions.  Built into libdg_probe.so.
#include "../fp8_rows.hpp"

namespace {

__global__ void __launch_bounds__(256) row_scale_list(const float* x, float* reciprocal, float* scale,
                                                      float* divisor, float* inverse, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v[4] = {x[i], 0.0f, 0.0f, 0.0f};
  reciprocal[i] = dg::reciprocal_rn(x[i]);
  const dg::RowScale b = dg::row_scale(v, x[i]);
  scale[i] = b.scale;
  divisor[i] = b.s;
  inverse[i] = b.r;
}

}  // namespace

extern "C" {

// For each of the n positive numbers x (at most 2^31 - 256 of them): RN(1 / x), and the
// scale, divisor and RN(1 / divisor) of a block with the largest magnitude x.  Returns
// 0, or the HIP error of the launch.
int dgp_row_scale(const float* x, float* reciprocal, float* scale, float* divisor, float* inverse,
                       int64_t n, void* stream) {
  if (!x || !reciprocal || !scale || !divisor || !inverse || n < 1 || n > INT32_MAX - 255) return -1;
  hipLaunchKernelGGL(row_scale_list, dim3((unsigned)((n + 255) / 256)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), x, reciprocal, scale, divisor, inverse, n);
  return (int)hipGetLastError();
}

}  // extern "C"
