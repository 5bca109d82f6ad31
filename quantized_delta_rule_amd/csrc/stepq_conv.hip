// stepq_conv.hip -- short causal convolution of each channel over its own tokens, and its gradient:
//   u_t = b + sum_{j < W} w_j x_{t - (W - 1) + j},  y = u or u sigmoid(u)
//   du = dy act'(u);  dx_t = sum_j w_j du_{t + (W - 1) - j};  dw_j = sum_t du_t x_{t - (W - 1) + j};  db = sum_t du_t
// A lane owns a few neighbouring channels of one piece of a sequence and goes down its tokens with the last W - 1
// inputs (and, backwards, derivatives) in registers, so every row is read once but for W - 1 rows at a piece's ends.
// Bound by HBM: 2 W + 5 operations an element against 4 bytes of a 16-bit type.  16,381 tokens x 10,240 channels, bf16: 138 us,
// 4.9 TB/s (a copy reaches 5.05); the gradient of 8,192 x 8,192 89 us for its 403 MB, 4.5 TB/s, and 5 for the last sums; 70
// single tokens x 10,240 7.5 us.  Eight channels a lane forward (16 bytes), four backward, where five sums and two windows
// a channel are held.  Four rows in flight, not one: 158 -> 138 us and 112 -> 107.  Pieces of 32 tokens forward and 64
// backward there (64 / 128: 152 and 99 us; backward 32: 107): shorter ones read more rows twice, longer ones fill fewer CUs.
#include "stepq_layer.h"

namespace stepq {
namespace {

using namespace lay;

constexpr int kAhead = 4;  // rows read at once
template <int DT>
constexpr int kSize = DT == kF32 ? 4 : 2;

// The part of a sequence that a wave works on.
struct Part {
  int s, slot;
  long long t0, len, p, end;  // first row and length of the sequence, the piece's positions p .. end - 1 in it
  bool first;
};

// False where the wave has nothing to do.  One lane a sequence raises the flags.
__device__ __forceinline__ bool part_of(const ConvArgs& A, long long j, bool report, int lane, Part& P) {
  int a, b;
  if (report && j < A.N) {
    const bool ok = seq_range(A, (int)j, a, b);
    seq_slot(A, (int)j, ok, lane == 0);
  }
  long long idx;
  if (!piece(A, A.sh, j, lane, P.s, idx)) return false;
  const bool ok = seq_range(A, P.s, a, b);
  P.slot = seq_slot(A, P.s, ok, false);
  P.t0 = a;
  P.len = b - a;
  P.p = idx << A.sh;
  P.end = P.p + (1 << A.sh) < P.len ? P.p + (1 << A.sh) : P.len;
  P.first = idx == 0;
  return P.slot >= 0 && (P.p < P.len || P.first);
}

// Weights of V channels, [j][channel], and their bias.
template <int W, int V>
__device__ __forceinline__ void weights(const ConvArgs& A, int c, float (&w)[W][V], float (&b)[V]) {
  float raw[W * V];
#pragma unroll
  for (int i = 0; i < W * V; i += 4) load4_any(A.pdtype, A.w, (long long)c * W + i, raw + i);
#pragma unroll
  for (int v = 0; v < V; v++) {
    b[v] = 0;
#pragma unroll
    for (int j = 0; j < W; j++) w[j][v] = raw[v * W + j];
  }
  if (A.b) {
#pragma unroll
    for (int v = 0; v < V; v += 4) load4_any(A.pdtype, A.b, c + v, b + v);
  }
}

template <int DT, int W, int V>
__global__ __launch_bounds__(256) void k_conv(ConvArgs A, int blocks) {
  const int lane = threadIdx.x & 63;
  const int cb = blockIdx.x % blocks;
  const long long j = (long long)(blockIdx.x / blocks) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Part P;
  if (!part_of(A, j, cb == 0, lane, P)) return;
  const int c = (cb * 64 + lane) * V;
  if (c >= A.C) return;
  float w[W][V], b[V], x[W][V];  // x: the last W inputs
  weights<W, V>(A, c, w, b);
  const long long so = (long long)P.slot * (W - 1) * A.C + c;
#pragma unroll
  for (int i = 0; i < W - 1; i++) {
    const long long at = P.p - (W - 1) + i;
    if (at >= 0) loadv<DT, V>(A.x, (P.t0 + at) * A.xs + c, x[i]);
    else if (A.S_in) loadv<DT, V>(A.S_in, so + (at + W - 1) * A.C, x[i]);
    else {
#pragma unroll
      for (int v = 0; v < V; v++) x[i][v] = 0;
    }
  }
  if (P.first && A.S_out) {  // the piece that read the old state is the one that writes the new one
    float last[W - 1][V];
#pragma unroll
    for (int i = 0; i < W - 1; i++) {
      const long long at = P.len - (W - 1) + i;
      if (at >= 0) loadv<DT, V>(A.x, (P.t0 + at) * A.xs + c, last[i]);
      else {  // row at + W - 1 of the old one
#pragma unroll
        for (int v = 0; v < V; v++) {
          float o = 0;
#pragma unroll
          for (int k = 0; k < W - 1; k++) o = at + W - 1 == k ? x[k][v] : o;
          last[i][v] = o;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < W - 1; i++) storev<DT, V>(A.S_out, so + (long long)i * A.C, last[i]);
  }
  // rows are read kAhead at a time, the next ones while these are worked on
  const int n = (int)(P.end - P.p);
  const char* px = (const char*)A.x + ((P.t0 + P.p) * A.xs + c) * kSize<DT>;
  char* po = (char*)A.out + ((P.t0 + P.p) * A.os + c) * kSize<DT>;
  const long long ax = A.xs * kSize<DT>, ao = A.os * kSize<DT>;
  Raw<DT, V> next[kAhead];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kAhead; i++) next[i].load(px + (t0 + i < n ? t0 + i : n - 1) * ax);
  };
  if (n > 0) fetch(0);
  for (int t0 = 0; t0 < n; t0 += kAhead) {
    Raw<DT, V> now[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; i++) now[i] = next[i];
    if (t0 + kAhead < n) fetch(t0 + kAhead);
#pragma unroll
    for (int r = 0; r < kAhead; r++) {
      if (t0 + r >= n) break;
      float y[V];
#pragma unroll
      for (int v = 0; v < V; v++) {
        x[W - 1][v] = now[r][v];
        float u = b[v];
#pragma unroll
        for (int i = 0; i < W; i++) u = fmaf(w[i][v], x[i][v], u);
        y[v] = act_of<DT>(A.act, u);
      }
      storev<DT, V>(po + (t0 + r) * ao, 0, y);
#pragma unroll
      for (int i = 0; i < W - 1; i++) {
#pragma unroll
        for (int v = 0; v < V; v++) x[i][v] = x[i + 1][v];
      }
    }
  }
}

// A piece's wave goes from its first token to W - 1 tokens behind its last: with du of the last W tokens it
// settles dx of the token W - 1 back.  Positions before the sequence are the state's rows, so the first piece
// begins W - 1 tokens earlier, where du is zero.  Sums of dw and db are over the piece's own tokens.
template <int DT, int W, int V>
__global__ __launch_bounds__(256) void k_conv_grad(ConvArgs A, int blocks) {
  __shared__ float sum[4][(W + 1) * V][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cb = blockIdx.x % blocks;
  const long long j = (long long)(blockIdx.x / blocks) * 4 + wave;
  const int c = (cb * 64 + lane) * V;
  float dw[W][V], db[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    db[v] = 0;
#pragma unroll
    for (int i = 0; i < W; i++) dw[i][v] = 0;
  }
  Part P;
  if (part_of(A, j, cb == 0, lane, P) && c < A.C) {
    float w[W][V], b[V], x[W][V], du[W][V];
    weights<W, V>(A, c, w, b);
    const long long so = (long long)P.s * (W - 1) * A.C + c;
#pragma unroll
    for (int i = 0; i < W - 1; i++) {
      const long long at = P.p - (W - 1) + i;
      if (at >= 0) loadv<DT, V>(A.x, (P.t0 + at) * A.xs + c, x[i]);
      else if (A.S_in) loadv<DT, V>(A.S_in, so + (at + W - 1) * A.C, x[i]);
      else {
#pragma unroll
        for (int v = 0; v < V; v++) x[i][v] = 0;
      }
    }
#pragma unroll
    for (int i = 0; i < W; i++) {
#pragma unroll
      for (int v = 0; v < V; v++) du[i][v] = 0;
    }
    // positions settled: p .. end - 1, from -(W - 1) in the first piece
    const long long from = P.first ? -(long long)(W - 1) : P.p;
    const char* px = (const char*)A.x + (P.t0 * A.xs + c) * kSize<DT>;
    const char* pu = (const char*)A.d_out + (P.t0 * A.os + c) * kSize<DT>;
    const long long ax = A.xs * kSize<DT>, au = A.os * kSize<DT>, most = P.len - 1;
    Raw<DT, V> nx[kAhead], nu[kAhead], rx[kAhead], ru[kAhead];
    auto fetch = [&](long long q) {
#pragma unroll
      for (int i = 0; i < kAhead; i++) {
        const long long t = q + i < P.len ? q + i : most;
        nx[i].load(px + t * ax);
        nu[i].load(pu + t * au);
      }
    };
    if (P.p < P.len) fetch(P.p);
    for (long long q0 = P.p; q0 < P.end + W - 1; q0 += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; i++) rx[i] = nx[i], ru[i] = nu[i];
      if (q0 + kAhead < P.end + W - 1 && q0 + kAhead < P.len) fetch(q0 + kAhead);
#pragma unroll
      for (int r = 0; r < kAhead; r++) {
      const long long q = q0 + r;
      if (q >= P.end + W - 1) break;
      const bool in = q < P.len;
#pragma unroll
      for (int v = 0; v < V; v++) du[W - 1][v] = 0;
      if (in) {
        float dy[V];
#pragma unroll
        for (int v = 0; v < V; v++) x[W - 1][v] = rx[r][v], dy[v] = ru[r][v];
#pragma unroll
        for (int v = 0; v < V; v++) {
          float u = b[v];
#pragma unroll
          for (int i = 0; i < W; i++) u = fmaf(w[i][v], x[i][v], u);
          float d = dy[v];
          if (A.act == kSilu) {
            const float s = sigmoid<DT>(u);
            d *= fmaf(u * s, 1.0f - s, s);
          }
          du[W - 1][v] = d;
          if (q < P.end) {
            db[v] += d;
#pragma unroll
            for (int i = 0; i < W; i++) dw[i][v] = fmaf(d, x[i][v], dw[i][v]);
          }
        }
      }
      const long long o = q - (W - 1);
      if (o >= from && o < P.end) {
        float g[V];
#pragma unroll
        for (int v = 0; v < V; v++) {
          g[v] = 0;
#pragma unroll
          for (int i = 0; i < W; i++) g[v] = fmaf(w[W - 1 - i][v], du[i][v], g[v]);
        }
        const long long r = o - P.len + W - 1;  // the last rows are the state that the sequence leaves
        if (r >= 0 && A.dS_out) {
          float more[V];
          loadv<DT, V>(A.dS_out, so + r * A.C, more);
#pragma unroll
          for (int v = 0; v < V; v++) g[v] += more[v];
        }
        if (o >= 0) storev<DT, V>(A.dx, (P.t0 + o) * A.C + c, g);
        else if (A.dS_in) storev<DT, V>(A.dS_in, so + (o + W - 1) * A.C, g);
      }
#pragma unroll
      for (int i = 0; i < W - 1; i++) {
#pragma unroll
        for (int v = 0; v < V; v++) {
          x[i][v] = x[i + 1][v];
          du[i][v] = du[i + 1][v];
        }
      }
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; v++) {
#pragma unroll
    for (int i = 0; i < W; i++) sum[wave][v * W + i][lane] = dw[i][v];
    sum[wave][W * V + v][lane] = db[v];
  }
  __syncthreads();
  // row of the partial sums: dw as [C, W], then db
  float* part = A.ws + (long long)(blockIdx.x / blocks) * A.C * (W + 1);
  for (int i = threadIdx.x; i < W * V * 64; i += 256) {
    const int l = i / (W * V), e = i % (W * V);
    const long long m = (long long)cb * 64 * V * W + i;
    if (m < (long long)A.C * W) part[m] = sum[0][e][l] + sum[1][e][l] + sum[2][e][l] + sum[3][e][l];
  }
  for (int i = threadIdx.x; i < V * 64; i += 256) {
    const int l = i / V, e = W * V + i % V;
    const long long m = (long long)cb * 64 * V + i;
    if (m < A.C) part[(long long)A.C * W + m] = sum[0][e][l] + sum[1][e][l] + sum[2][e][l] + sum[3][e][l];
  }
}

constexpr int kFwdV = 8, kBwdV = 4;

long long channel_blocks(const ConvArgs& a, bool back) {
  const int wide = 64 * (back ? kBwdV : kFwdV);
  return (a.C + wide - 1) / wide;
}

// Tokens of a piece (2^n): long pieces where they are waves enough, short ones where a call would be a few long chains.  us of
// calls, long against short pieces: gradient 2,657 tokens x 120 channels 42 and 18, 2,933 x 4,752 (1,400 waves) 50 and 30,
// 8,192 x 2,048 (1,100) 49 and 35, 8,192 x 8,192 (4,100) 97 and 104; forward 14 and 7, 22 and 18, 22 and 19, 53 and 55.
constexpr long long kWaves = 2048;
int piece_of(const ConvArgs& a, bool back) {
  const int big = back ? 6 : 5, small = back ? 4 : 3;
  return pieces(a, big) * channel_blocks(a, back) >= kWaves ? big : small;
}

template <int DT, int W>
hipError_t launch(const ConvArgs& given, bool back, hipStream_t s) {
  ConvArgs a = given;
  a.sh = piece_of(a, back);
  const int blocks = (int)channel_blocks(a, back);
  const long long groups = (pieces(a, a.sh) + 3) / 4;
  const dim3 grid((unsigned)(groups * blocks)), block(256);
  if (back) hipLaunchKernelGGL((k_conv_grad<DT, W, kBwdV>), grid, block, 0, s, a, blocks);
  else hipLaunchKernelGGL((k_conv<DT, W, kFwdV>), grid, block, 0, s, a, blocks);
  return hipGetLastError();
}

template <int DT>
hipError_t by_width(const ConvArgs& a, bool back, hipStream_t s) {
  return a.W == 2 ? launch<DT, 2>(a, back, s) : a.W == 3 ? launch<DT, 3>(a, back, s) : launch<DT, 4>(a, back, s);
}

hipError_t by_type(const ConvArgs& a, bool back, hipStream_t s) {
  return a.dtype == kF32 ? by_width<kF32>(a, back, s)
                         : a.dtype == kBF16 ? by_width<kBF16>(a, back, s) : by_width<kF16>(a, back, s);
}

}  // namespace

hipError_t launch_conv(const ConvArgs& a, hipStream_t s) { return a.N <= 0 ? hipSuccess : by_type(a, false, s); }

size_t conv_backward_bytes(const ConvArgs& a) {
  return (size_t)((pieces(a, piece_of(a, true)) + 3) / 4) * a.C * (a.W + 1) * sizeof(float);
}

hipError_t launch_conv_backward(const ConvArgs& a, hipStream_t s) {
  SumArgs m{a.ws, (int)((pieces(a, piece_of(a, true)) + 3) / 4), (long long)a.C * (a.W + 1), (long long)a.C * a.W, a.C, a.dw,
            a.db, nullptr};
  if (a.N > 0) {
    if (hipError_t e = by_type(a, true, s)) return e;
  }
  return launch_sum(m, s);  // without a sequence: sums of nothing
}

}  // namespace stepq
