// stepq_scan.hip -- selective state space scan, token by token, and the choice between that and blocks of tokens
// (stepq_scan_block.h):
//   h_t = exp(D_t A) h_{t-1} + D_t B_t x_t,  out_t = (C_t . h_t + D x_t) z sigmoid(z)
// A wave owns two tiles of 256 / n channels of one group of a sequence: n / 4 neighbouring lanes a channel, four states a
// lane, so that states are read and written 16 bytes a lane side by side.  Bound by HBM: 70 single tokens x 6,144 channels of
// 16 states, bf16, 12.4 us for 59 MB, 4.8 TB/s (one tile a wave 15.8 us, four 14.6).
#include "stepq_scan_block.h"

namespace stepq {
namespace {

using namespace lay;

constexpr int kTiles = 2;  // of 64 / LN channels, in a wave

template <int DT, int LN>
__global__ __launch_bounds__(256) void k_scan_tokens(ScanArgs A, int tiles) {
  constexpr int GW = 64 / LN, n = 4 * LN, K = kTiles;
  const int lane = threadIdx.x & 63;
  const long long unit = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long long per = (long long)tiles * A.G;
  if (unit >= per * A.N) return;
  const int s = (int)(unit / per), tg = (int)(unit - s * per), g = tg / tiles, tile = tg - g * tiles;
  int t0, t1;
  const bool valid = seq_range(A, s, t0, t1);
  const int slot = seq_slot(A, s, valid, tg == 0 && lane == 0);
  if (slot < 0 || (A.split && t1 - t0 >= A.split)) return;
  if (t0 == t1 && (!A.S_out || A.S_out == A.S_in)) return;
  const int part = lane % LN;
  int c[K];
  bool live[K];
  f4 h[K], a2[K];
  float skip[K], bias[K];
#pragma unroll
  for (int k = 0; k < K; k++) {
    const int cg = (tile * K + k) * GW + lane / LN;
    live[k] = cg < A.Cg;
    c[k] = g * A.Cg + (live[k] ? cg : A.Cg - 1);  // lanes past the group's end repeat its last channel
    const long long so = ((long long)slot * A.C + c[k]) * n + 4 * part;
    h[k] = A.S_in ? *(const f4*)(A.S_in + so) : f4{0, 0, 0, 0};
    a2[k] = *(const f4*)(A.A + (long long)c[k] * n + 4 * part);
    skip[k] = A.D ? A.D[c[k]] : 0.0f;
    bias[k] = A.bias ? A.bias[c[k]] : 0.0f;
  }
#pragma unroll
  for (int k = 0; k < K; k++) {
#pragma unroll
    for (int i = 0; i < 4; i++) a2[k][i] *= kLog2e;
  }
  const void* zp = A.z ? A.z : A.x;  // without a gate its loads repeat x's
  const long long zs = A.z ? A.zs : A.xs;
  for (int t = t0; t < t1; t++) {
    Raw<DT, 1> rx[K], rd[K], rz[K];
    constexpr int size = DT == kF32 ? 4 : 2;
#pragma unroll
    for (int k = 0; k < K; k++) {
      rx[k].load(A.x, (t * A.xs + c[k]) * size);
      rd[k].load(A.dt, (t * A.dts + c[k]) * size);
      rz[k].load(zp, (t * zs + c[k]) * size);
    }
    const f4 B = load4<DT>(A.B, t * A.bs + g * n + 4 * part), Cm = load4<DT>(A.Cm, t * A.cs + g * n + 4 * part);
#pragma unroll
    for (int k = 0; k < K; k++) {
      const float x = rx[k][0], z = rz[k][0];
      const float D = step_of<DT>(A.softplus, rd[k][0] + bias[k]), dx = D * x;
      float y = 0;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        h[k][i] = fmaf(decay(D, a2[k][i]), h[k][i], dx * B[i]);
        y = fmaf(Cm[i], h[k][i], y);
      }
#pragma unroll
      for (int m = 1; m < LN; m *= 2) y += __shfl_xor(y, m);
      if (A.D) y = fmaf(skip[k], x, y);
      if (A.z) y *= z * sigmoid<DT>(z);
      if (live[k] && part == 0) storen<DT, 1>(A.out, t * A.os + c[k], &y);
    }
  }
  if (!A.S_out) return;
#pragma unroll
  for (int k = 0; k < K; k++) {
    if (live[k]) *(f4*)(A.S_out + ((long long)slot * A.C + c[k]) * n + 4 * part) = h[k];
  }
}

// Blocks pay from about 16 tokens a sequence on in large batches, earlier in small ones (us, token by token against
// blocks at 4 / 8 / 16 / 32 tokens of 4,096 channels, 16 states, bf16: 70 sequences 15 / 24 / 42 / 84 against 28 / 32 / 35 /
// 52, one 5.4 / 7.5 / 12 / 20 against 3.9 / 4.2 / 4.2 / 5.3).  Lengths are on the device: where they are shorter on
// average but one may be long, both kernels are launched and each takes its sequences (MIXED).
constexpr int kShort = 16, kMaybeLong = 128;
bool in_blocks(const ScanArgs& a) {
  return a.N > 0 && ((long long)a.T >= (long long)kShort * a.N || (a.cu && a.T - a.N >= kMaybeLong));
}
bool in_tokens(const ScanArgs& a) { return (long long)a.T < (long long)kShort * a.N; }

template <int DT, int LN>
hipError_t tokens(const ScanArgs& a, hipStream_t s) {
  const int wide = kTiles * 64 / LN, tiles = (a.Cg + wide - 1) / wide;
  const long long units = (long long)tiles * a.G * a.N;
  hipLaunchKernelGGL((k_scan_tokens<DT, LN>), dim3((unsigned)((units + 3) / 4)), dim3(256), 0, s, a, tiles);
  return hipGetLastError();
}

template <int DT, int NS, int NW>
hipError_t blocks(const ScanArgs& a, hipStream_t s) {
  char* end;
  const Segments q = lay_segments(a, segments_of(a, kLeastForward), a.ws, &end);
  const long long per = (long long)q.tiles * a.G;
  if (!q.sh) {
    hipLaunchKernelGGL((k_scan_run<DT, NS, 32, NW, 0>), dim3((unsigned)(per * a.N)), dim3(64 * NW), 0, s, a, q);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(per * pieces(a, q.sh)));
  hipLaunchKernelGGL((k_scan_run<DT, NS, 32, NW, 1>), grid, dim3(64 * NW), 0, s, a, q);
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL((k_scan_run<DT, NS, 32, NW, 2>), grid, dim3(64 * NW), 0, s, a, q);
  return hipGetLastError();
}

template <int DT>
hipError_t by_states(const ScanArgs& given, hipStream_t s) {
  ScanArgs a = given;
  if (in_tokens(a)) {
    if (in_blocks(a)) a.split = kShort;
    const hipError_t e = a.n == 8    ? tokens<DT, 2>(a, s)
                         : a.n == 16 ? tokens<DT, 4>(a, s)
                         : a.n == 32 ? tokens<DT, 8>(a, s)
                                     : tokens<DT, 16>(a, s);
    if (e || !in_blocks(a)) return e;
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
