// stepq_scan.hip -- selective state space scan, token by token:
//   h_t = exp(D_t A) h_{t-1} + D_t B_t x_t,  out_t = (C_t . h_t + D x_t) z sigmoid(z)
// A wave owns 256 / n channels of one group of a sequence: n / 4 neighbouring lanes a channel, four states a lane,
// so that states are read and written 16 bytes a lane side by side.
#include "stepq_scan_block.h"

namespace stepq {
namespace {

using namespace lay;

template <int DT, int LN>
__global__ __launch_bounds__(256) void k_scan_tokens(ScanArgs A, int tiles) {
  constexpr int GW = 64 / LN, n = 4 * LN;
  const int lane = threadIdx.x & 63;
  const long long unit = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long long per = (long long)tiles * A.G;
  if (unit >= per * A.N) return;
  const int s = (int)(unit / per), tg = (int)(unit - s * per), g = tg / tiles, tile = tg - g * tiles;
  int t0, t1;
  const bool valid = seq_range(A, s, t0, t1);
  const int slot = seq_slot(A, s, valid, tg == 0 && lane == 0);
  if (slot < 0) return;
  if (t0 == t1 && (!A.S_out || A.S_out == A.S_in)) return;
  const int cg = tile * GW + lane / LN, part = lane % LN;
  const bool live = cg < A.Cg;
  const int c = g * A.Cg + (live ? cg : A.Cg - 1);  // lanes past the group's end repeat its last channel
  const long long so = ((long long)slot * A.C + c) * n + 4 * part;
  f4 h = A.S_in ? *(const f4*)(A.S_in + so) : f4{0, 0, 0, 0};
  f4 a2 = *(const f4*)(A.A + (long long)c * n + 4 * part);
#pragma unroll
  for (int i = 0; i < 4; i++) a2[i] *= kLog2e;
  const float skip = A.D ? A.D[c] : 0.0f, bias = A.bias ? A.bias[c] : 0.0f;
  for (int t = t0; t < t1; t++) {
    float x, raw, z, slope;
    loadn<DT, 1>(A.x, t * A.xs + c, &x);
    loadn<DT, 1>(A.dt, t * A.dts + c, &raw);
    const f4 B = load4<DT>(A.B, t * A.bs + g * n + 4 * part), Cm = load4<DT>(A.Cm, t * A.cs + g * n + 4 * part);
    const float D = step_of(A.softplus, raw + bias, slope), dx = D * x;
    float y = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      h[i] = fmaf(decay(D, a2[i]), h[i], dx * B[i]);
      y = fmaf(Cm[i], h[i], y);
    }
#pragma unroll
    for (int m = 1; m < LN; m *= 2) y += __shfl_xor(y, m);
    if (A.D) y = fmaf(skip, x, y);
    if (A.z) {
      loadn<DT, 1>(A.z, t * A.zs + c, &z);
      y *= z * sigmoid(z);
    }
    if (live && part == 0) storen<DT, 1>(A.out, t * A.os + c, &y);
  }
  if (A.S_out && live) *(f4*)(A.S_out + so) = h;
}

// Blocks pay from 16 tokens a sequence on.
bool in_blocks(const ScanArgs& a) { return a.N > 0 && (long long)a.T >= 16LL * a.N; }

template <int DT, int LN>
hipError_t tokens(const ScanArgs& a, hipStream_t s) {
  const int tiles = (a.Cg + 64 / LN - 1) / (64 / LN);
  const long long units = (long long)tiles * a.G * a.N;
  hipLaunchKernelGGL((k_scan_tokens<DT, LN>), dim3((unsigned)((units + 3) / 4)), dim3(256), 0, s, a, tiles);
  return hipGetLastError();
}

template <int DT, int NS, int NW>
hipError_t blocks(const ScanArgs& a, hipStream_t s) {
  char* end;
  const int sh = segments_of(a, kLeastForward);
  const Segments q = lay_segments(a, sh, a.ws, &end);
  const long long per = (long long)q.tiles * a.G;
  if (!sh) {
    hipLaunchKernelGGL((k_scan_run<DT, NS, 32, NW, 0>), dim3((unsigned)(per * a.N)), dim3(64 * NW), 0, s, a, q);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(per * pieces(a, sh)));
  hipLaunchKernelGGL((k_scan_run<DT, NS, 32, NW, 1>), grid, dim3(64 * NW), 0, s, a, q);
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL((k_scan_run<DT, NS, 32, NW, 2>), grid, dim3(64 * NW), 0, s, a, q);
  return hipGetLastError();
}

template <int DT>
hipError_t by_states(const ScanArgs& a, hipStream_t s) {
  if (!in_blocks(a)) {
    return a.n == 8 ? tokens<DT, 2>(a, s)
                    : a.n == 16 ? tokens<DT, 4>(a, s) : a.n == 32 ? tokens<DT, 8>(a, s) : tokens<DT, 16>(a, s);
  }
  return a.n == 8    ? blocks<DT, 2, 2>(a, s)
         : a.n == 16 ? blocks<DT, 2, 4>(a, s)
         : a.n == 32 ? blocks<DT, 4, 4>(a, s)
                     : blocks<DT, 8, 4>(a, s);
}

}  // namespace

size_t scan_forward_bytes(const ScanArgs& a) {
  if (!in_blocks(a)) return 0;
  char* end;
  lay_segments(a, segments_of(a, kLeastForward), nullptr, &end);
  return (size_t)end;
}

hipError_t launch_scan(const ScanArgs& a, hipStream_t s) {
  if (a.N <= 0) return hipSuccess;
  return a.dtype == kF32 ? by_states<kF32>(a, s) : a.dtype == kBF16 ? by_states<kBF16>(a, s) : by_states<kF16>(a, s);
}

}  // namespace stepq
