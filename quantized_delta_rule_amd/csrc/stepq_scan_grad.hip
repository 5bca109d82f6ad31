// stepq_scan_grad.hip -- gradient of the selective scan.  With e_t = dout_t z sigmoid(z), a_t = exp(D_t A) and
// g_t the gradient of h_t:
//   g_t = C_t e_t + a_{t+1} g_{t+1} (behind the last token: the last state's gradient)
//   dC_t = sum_c e_t h_t;  dB_t = sum_c g_t D_t x_t;  dx_t = D_t sum_n g_t B_t + D e_t
//   dD_t = sum_n g_t (A a_t h_{t-1} + B_t x_t), ddt_t = dD_t sigmoid(dt + bias);  dA = sum_t D_t g_t a_t h_{t-1}
//   dz_t = dout_t (C_t . h_t + D x_t) (z sigmoid(z))';  dD = sum_t e_t x_t;  dS_in = a_1 g_1
#include "stepq_scan.h"

namespace stepq {
namespace {

using namespace lay;

constexpr size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace: every token's state, partial dB and dC of every tile, partial dA, dD and dbias of every sequence.
struct Space {
  int tiles;
  long long row;  // dA | dD | dbias
  size_t h, bc, par, all;
};
Space space(const ScanArgs& a) {
  Space w;
  const int gw = 256 / a.n;
  w.tiles = (a.Cg + gw - 1) / gw;
  w.row = (long long)a.C * a.n + 2 * a.C;
  w.h = 0;
  w.bc = w.h + up((size_t)a.T * a.C * a.n * 4);
  w.par = w.bc + up((size_t)w.tiles * a.T * a.G * a.n * 8);
  w.all = w.par + up((size_t)a.N * w.row * 4);
  return w;
}

template <int DT, int LN>
__global__ __launch_bounds__(256) void k_scan_grad(ScanArgs A, Space W) {
  constexpr int GW = 64 / LN, n = 4 * LN;
  const int lane = threadIdx.x & 63;
  const long long unit = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long long per = (long long)W.tiles * A.G;
  if (unit >= per * A.N) return;
  const int s = (int)(unit / per), tg = (int)(unit - s * per), g = tg / W.tiles, tile = tg - g * W.tiles;
  int t0, t1;
  const bool valid = seq_range(A, s, t0, t1);
  seq_slot(A, s, valid, tg == 0 && lane == 0);
  const int cg = tile * GW + lane / LN, part = lane % LN;
  const bool live = cg < A.Cg;
  const int c = g * A.Cg + (live ? cg : A.Cg - 1);
  const long long so = ((long long)s * A.C + c) * n + 4 * part;
  float* H = (float*)(A.ws + W.h);
  float* bc = (float*)(A.ws + W.bc);
  float* par = (float*)(A.ws + W.par) + s * W.row;
  f4 h = valid && A.S_in ? *(const f4*)(A.S_in + so) : f4{0, 0, 0, 0};
  const f4 a = *(const f4*)(A.A + (long long)c * n + 4 * part);
  const float skip = A.D ? A.D[c] : 0.0f, bias = A.bias ? A.bias[c] : 0.0f;
  for (int t = t0; t < t1; t++) {
    float x, raw, slope;
    loadn<DT, 1>(A.x, t * A.xs + c, &x);
    loadn<DT, 1>(A.dt, t * A.dts + c, &raw);
    const f4 B = load4<DT>(A.B, t * A.bs + g * n + 4 * part);
    const float D = step_of(A.softplus, raw + bias, slope);
    if (live) *(f4*)(H + ((long long)t * A.C + c) * n + 4 * part) = h;  // h_{t-1}
#pragma unroll
    for (int i = 0; i < 4; i++) h[i] = fmaf(decay(D, a[i] * kLog2e), h[i], D * x * B[i]);
  }
  f4 G = valid && A.dS_out ? *(const f4*)(A.dS_out + so) : f4{0, 0, 0, 0}, dA = {0, 0, 0, 0};
  float dD = 0, dbias = 0;
  for (int t = t1 - 1; t >= t0; t--) {
    float x, raw, slope, up, z = 0;
    loadn<DT, 1>(A.x, t * A.xs + c, &x);
    loadn<DT, 1>(A.dt, t * A.dts + c, &raw);
    loadn<DT, 1>(A.d_out, t * A.os + c, &up);
    const f4 B = load4<DT>(A.B, t * A.bs + g * n + 4 * part), Cm = load4<DT>(A.Cm, t * A.cs + g * n + 4 * part);
    const f4 was = *(const f4*)(H + ((long long)t * A.C + c) * n + 4 * part);
    const float D = step_of(A.softplus, raw + bias, slope);
    float e = up;
    if (A.z) {
      loadn<DT, 1>(A.z, t * A.zs + c, &z);
      e *= z * sigmoid(z);
    }
    float y = 0, gB = 0, gA = 0;
    f4 pB, pC;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float al = decay(D, a[i] * kLog2e);
      const float now = fmaf(al, was[i], D * x * B[i]);
      y = fmaf(Cm[i], now, y);
      G[i] = fmaf(Cm[i], e, G[i]);
      pC[i] = live ? e * now : 0.0f;
      pB[i] = live ? G[i] * (D * x) : 0.0f;
      gB = fmaf(G[i], B[i], gB);
      G[i] *= al;
      const float w = G[i] * was[i];
      gA = fmaf(a[i], w, gA);
      dA[i] = fmaf(D, w, dA[i]);
    }
#pragma unroll
    for (int m = 1; m < LN; m *= 2) {
      y += __shfl_xor(y, m);
      gB += __shfl_xor(gB, m);
      gA += __shfl_xor(gA, m);
    }
#pragma unroll
    for (int m = LN; m < 64; m *= 2) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        pB[i] += __shfl_xor(pB[i], m);
        pC[i] += __shfl_xor(pC[i], m);
      }
    }
    if (lane < LN) {
      float* o = bc + (((long long)tile * A.T + t) * A.G + g) * 2 * n + 4 * part;
      *(f4*)o = pB;
      *(f4*)(o + n) = pC;
    }
    const float step = fmaf(x, gB, gA) * slope, dx = fmaf(D, gB, skip * e);
    dD = fmaf(e, x, dD);
    dbias += step;
    if (live && part == 0) {
      const long long o = (long long)t * A.C + c;
      storen<DT, 1>(A.dx, o, &dx);
      storen<DT, 1>(A.ddt, o, &step);
      if (A.z) {
        const float sg = sigmoid(z), dz = up * fmaf(skip, x, y) * fmaf(z * sg, 1.0f - sg, sg);
        storen<DT, 1>(A.dz, o, &dz);
      }
    }
  }
  if (!live) return;
  if (valid && A.dS_in) *(f4*)(A.dS_in + so) = G;
  *(f4*)(par + (long long)c * n + 4 * part) = dA;
  if (part == 0) {
    par[(long long)A.C * n + c] = dD;
    par[(long long)A.C * n + A.C + c] = dbias;
  }
}

// dB and dC of every token of a sequence: the tiles' partial sums in order.
template <int DT>
__global__ __launch_bounds__(256) void k_scan_bc(ScanArgs A, Space W) {
  const long long row = 2LL * A.G * A.n, i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= row * A.T) return;
  const int t = (int)(i / row), k = (int)(i % row), g = k / (2 * A.n), m = k % (2 * A.n);
  if (A.cu) {  // rows of no sequence are left alone: the last sequence that begins at or before t holds it, or none does
    int lo = 0, hi = A.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (A.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    int t0, t1;
    if (!seq_range(A, lo, t0, t1) || t < t0 || t >= t1) return;
  }
  const float* p = (const float*)(A.ws + W.bc) + i;
  float acc = 0;
  for (int q = 0; q < W.tiles; q++) acc += p[q * row * A.T];
  const long long o = ((long long)t * A.G + g) * A.n + (m < A.n ? m : m - A.n);
  storen<DT, 1>(m < A.n ? A.dB : A.dC, o, &acc);
}

template <int DT, int LN>
hipError_t launch(const ScanArgs& a, const Space& w, hipStream_t s) {
  const long long units = (long long)w.tiles * a.G * a.N;
  hipLaunchKernelGGL((k_scan_grad<DT, LN>), dim3((unsigned)((units + 3) / 4)), dim3(256), 0, s, a, w);
  if (hipError_t e = hipGetLastError()) return e;
  const long long all = 2LL * a.G * a.n * a.T;
  if (all) hipLaunchKernelGGL((k_scan_bc<DT>), dim3((unsigned)((all + 255) / 256)), dim3(256), 0, s, a, w);
  return hipGetLastError();
}

template <int DT>
hipError_t by_states(const ScanArgs& a, const Space& w, hipStream_t s) {
  return a.n == 8 ? launch<DT, 2>(a, w, s)
                  : a.n == 16 ? launch<DT, 4>(a, w, s) : a.n == 32 ? launch<DT, 8>(a, w, s) : launch<DT, 16>(a, w, s);
}

}  // namespace

size_t scan_backward_bytes(const ScanArgs& a) { return space(a).all; }

hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s) {
  const Space w = space(a);
  if (a.N > 0) {
    const hipError_t e = a.dtype == kF32    ? by_states<kF32>(a, w, s)
                         : a.dtype == kBF16 ? by_states<kBF16>(a, w, s)
                                            : by_states<kF16>(a, w, s);
    if (e) return e;
  }
  SumArgs m{(const float*)(a.ws + w.par), a.N, w.row, (long long)a.C * a.n, a.C, a.dA, a.dD, a.dbias};
  return launch_sum(m, s);
}

}  // namespace stepq
