// stepq_layer_sum.hip -- partial sums of parameter gradients, added up column by column in row order.
#include "stepq_layer.h"

namespace stepq {
namespace {

// 64 columns a workgroup; its 16 waves take every 16th row each and are joined in wave order.
__global__ __launch_bounds__(1024) void k_sum(SumArgs A) {
  __shared__ float sum[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long m = (long long)blockIdx.x * 64 + lane;
  float acc = 0;
  if (m < A.M) {
#pragma unroll 8
    for (int p = wave; p < A.P; p += 16) acc += A.part[p * A.M + m];
  }
  sum[wave][lane] = acc;
  __syncthreads();
  if (wave || m >= A.M) return;
  for (int w = 1; w < 16; w++) acc += sum[w][lane];
  if (m < A.m0) {
    if (A.out0) A.out0[m] = acc;
  } else if (m < A.m0 + A.m1) {
    if (A.out1) A.out1[m - A.m0] = acc;
  } else if (A.out2) {
    A.out2[m - A.m0 - A.m1] = acc;
  }
}

}  // namespace

hipError_t launch_sum(const SumArgs& a, hipStream_t s) {
  if (a.M <= 0) return hipSuccess;
  hipLaunchKernelGGL(k_sum, dim3((unsigned)((a.M + 63) / 64)), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace stepq
