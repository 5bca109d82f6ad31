// stepq_delta_step.hip -- the delta rule token by token on binary32 states: one token of each request
// (decode of layers that keep FP32 states), a few (drafted tokens), or any length and gate kind.
//
// Columns of S are independent given k, q and the gates, so a wave owns 32 columns of one
// (sequence, head) tile from its first token to its last and nothing is exchanged between waves:
//   lane l: columns 4 (l & 7) .. + 3, key rows R (l >> 3) .. + R - 1 with R = d / 8
// (R x 4 state entries in registers; a row's 8 lanes read 128 contiguous bytes, and a lane's key rows
// are contiguous, so k, q and row gates come as plain vector loads).  u = S^T k and o = S^T q are sums
// over a lane's rows and then over the 8 row groups.
//
// Bound by HBM: a single token reads and writes every state once and computes 6 operations an entry.  70 x 48
// states of 128 x 128 (440 MB) take 62 us where a part of them is in the memory-side cache (the same states call
// after call) and 87 us where six pools take turns (5.0 TB/s; a copy reaches 5.2); 64 x 32 states and four tokens
// with row gates 58 and 71 us; one request's 48 states 5.3 us.  32 columns a wave, not 64: one request then still has 192 waves on as many SIMDs.
#include "stepq_delta.h"

namespace stepq {
namespace {

using namespace dlt;

// Sum over the 8 row groups (lanes that differ in bits 3, 4 and 5).
__device__ __forceinline__ float sum_groups(float x) {
  x += __shfl_xor(x, 8);
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}

template <int D, int DT, int KDA>
__global__ __launch_bounds__(256) void k_recurrent(SeqArgs A) {
  constexpr int R = D / 8, NS = D / 32;
  const int lane = threadIdx.x & 63;
  const long long unit = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long long tile = unit / NS;
  if (tile >= (long long)A.N * A.H) return;
  const int sl = (int)(unit - tile * NS);
  const int s = (int)(tile / A.H), h = (int)(tile - (long long)s * A.H);
  int t0, t1;
  const bool valid = seq_range(A, s, t0, t1);
  const int slot = seq_slot(A, s, valid, h == 0 && sl == 0 && lane == 0);
  if (slot < 0 || (A.split && t1 - t0 >= A.split)) return;
  if (t0 == t1 && (!A.S_out || A.S_out == A.S_in)) return;
  const int col = 32 * sl + 4 * (lane & 7), row = R * (lane >> 3);
  const long long so = (((long long)slot * A.H + h) * D + row) * D + col;
  f4 S[R];
#pragma unroll
  for (int n = 0; n < R; n++) S[n] = A.S_in ? *(const f4*)(A.S_in + so + (long long)n * D) : f4{0, 0, 0, 0};
  const int hq = h / A.grp;
  for (int t = t0; t < t1; t++) {
    float k[R], q[R], a[R];
#pragma unroll
    for (int n = 0; n < R; n += 8) {
      load8<DT>(A.k, t * A.ks + (long long)hq * D + row + n, k + n);
      load8<DT>(A.q, t * A.qs + (long long)hq * D + row + n, q + n);
    }
    const f4 v = load4<DT>(A.v, t * A.vs + (long long)h * D + col);
    const long long th = (long long)t * A.H + h;
    const float beta = A.beta[th];
    if constexpr (KDA) {
#pragma unroll
      for (int n = 0; n < R; n += 8) load8<kF32>(A.alpha, th * D + row + n, a + n);
    } else {
      a[0] = A.alpha[th];
    }
    f4 u = {0, 0, 0, 0}, o = {0, 0, 0, 0};
#pragma unroll
    for (int n = 0; n < R; n++) {
      const float w = KDA && A.order ? a[n] * k[n] : k[n];
#pragma unroll
      for (int c = 0; c < 4; c++) u[c] = fmaf(w, S[n][c], u[c]);
    }
#pragma unroll
    for (int c = 0; c < 4; c++) u[c] = sum_groups(u[c]);
    if constexpr (!KDA) {
#pragma unroll
      for (int c = 0; c < 4; c++) u[c] = fmaf(-a[0], u[c], v[c]);  // the error e_j
    } else if (A.order) {
#pragma unroll
      for (int c = 0; c < 4; c++) u[c] = v[c] - u[c];
    }
#pragma unroll
    for (int n = 0; n < R; n++) {
      const float bk = beta * k[n], an = KDA ? a[n] : a[0];
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const float e = KDA && !A.order ? fmaf(-an, u[c], v[c]) : u[c];
        S[n][c] = fmaf(an, S[n][c], bk * e);
        o[c] = fmaf(q[n], S[n][c], o[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < 4; c++) o[c] = sum_groups(o[c]);
    if (lane < 8) store4<DT>(A.out, t * A.os + (long long)h * D + col, o);
  }
  if (A.S_out) {
#pragma unroll
    for (int n = 0; n < R; n++) *(f4*)(A.S_out + so + (long long)n * D) = S[n];
  }
}

template <int D, int DT>
hipError_t launch(const SeqArgs& a, hipStream_t s) {
  const long long units = (long long)a.N * a.H * (D / 32);
  const dim3 grid((unsigned)((units + 3) / 4)), block(256);
  if (a.kind) hipLaunchKernelGGL((k_recurrent<D, DT, 1>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_recurrent<D, DT, 0>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_recurrent(const SeqArgs& a, hipStream_t s) {
  if (a.N <= 0) return hipSuccess;
  if (a.D == 64)
    return a.dtype == kF32 ? launch<64, kF32>(a, s)
                           : a.dtype == kBF16 ? launch<64, kBF16>(a, s) : launch<64, kF16>(a, s);
  return a.dtype == kF32 ? launch<128, kF32>(a, s)
                         : a.dtype == kBF16 ? launch<128, kBF16>(a, s) : launch<128, kF16>(a, s);
}

}  // namespace stepq
