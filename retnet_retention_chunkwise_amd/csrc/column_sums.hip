// Sums over rows of [P, n] fp32 partial sums, the second stage of parameter
// gradients.  A fixed order of additions, so the same call gives the same
// bits: a workgroup owns 64 columns, its waves each add every sixteenth row,
// and their sums are added in wave order.
#include "kernels.h"

#include <hip/hip_runtime.h>

namespace ret {
namespace {

constexpr int kWaves = 16;

__global__ __launch_bounds__(64 * kWaves) void column_sums_kernel(ColumnSums a) {
  __shared__ float part[kWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  float* out = a.out[blockIdx.y];
  if (out == nullptr) return;  // the whole workgroup
  const float* p = a.partial + static_cast<long>(blockIdx.y) * a.rows * a.n;
  const long c = static_cast<long>(blockIdx.x) * 64 + lane;
  float s = 0.0f;
  if (c < a.n) {
#pragma unroll 8
    for (int r = w; r < a.rows; r += kWaves) s += p[r * a.n + c];
  }
  part[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < a.n) {
#pragma unroll
    for (int i = 1; i < kWaves; ++i) s += part[i][lane];
    out[c] = s;
  }
}

}  // namespace

hipError_t launch_column_sums(const ColumnSums& a, hipStream_t s) {
  hipLaunchKernelGGL(column_sums_kernel, dim3(static_cast<unsigned>((a.n + 63) / 64), 3), dim3(64 * kWaves), 0, s, a);
  return hipGetLastError();
}

}  // namespace ret
