// stepq_delta_grad.hip -- gradient of the chunked gated delta rule (see stepq_chunk.h for the forward
// mathematics and the operands).  With dO the outputs' gradient and dS1 that of the states behind a
// chunk (D = diag(L[C,.]), G = diag(G_t)):
//   dW = P^T dO + D K dS1,   Y = T^T dW,   dV = diag(beta) Y
//   dS0 = G_C dS1 + Q^T G dO - K^T G diag(beta) Y
//   N = lower(L o dO W^T),   X = Y W^T,   Z = -strict-lower(L o diag(beta) X)
//   dQ = G dO S0^T + N K
//   dK = -G diag(beta) Y S0^T + D W dS1^T + (Z + Z^T) K + N^T Q
//   dbeta_t = Y_t.V_t - G_t k_t.(Y S0^T)_t - sum_s X[t,s] L[t,s] (k_t.k_s)
//   dalpha_r = sum over the pairs (t >= r > s) of L[t,r] x[t,s] L[r-1,s], where x is the pair's value
//     without its gates: dO_t.W_s (q_t.k_s) - beta_t X[t,s] (k_t.k_s); the state before the chunk counts
//     as s = -1 (x = q_t.(dO S0^T)_t - beta_t k_t.(Y S0^T)_t), the state behind it as t = C
//     (x = k_s.(W dS1^T)_s, and <S0, dS1> for both).  Products of the other gates only: a gate of zero
//     has its gradient like any other.
// Four launches: local matrices (k_chunk_prep), states before every chunk (k_chunk_state), their gradients
// in reverse order (k_chunk_reverse), and every chunk's gradients at once (k_chunk_grad).
#include "stepq_chunk_kernels.h"

namespace stepq {
namespace {

using namespace dlt;

struct Keep {  // per chunk slot and value head, binary32
  float* S;    // [D][D] state before the chunk
  float* G;    // [D][D] gradient of the state behind it
  float* W;    // [64][D]
  float* Y;    // [64][D]
};

// The reverse pass: like k_chunk_state a wave owns 16 CT columns of one state's gradient for the whole
// sequence.
template <int D, int DT, int CT, int NW>
__global__ __launch_bounds__(64 * NW) void k_chunk_reverse(GradArgs B, Keep keep) {
  using L = LayB<D, DT>;
  constexpr int KS = D / 32, NPI = L::NPI, NB = D / 32;
  constexpr int keyN = L::offKK, triN = 4 * kTri * kFrag;  // K, K^T, Q^T; T^T, P^T
  constexpr int offTt = keyN, offP = keyN + 2 * kTri * kFrag, offTab = keyN + triN;
  const SeqArgs& A = B.f;
  __shared__ __attribute__((aligned(16))) char lds[offTab + 2048];
  const long long tile = blockIdx.x;
  const int s = (int)(tile / A.H), h = (int)(tile - (long long)s * A.H);
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  int t0, t1;
  const bool valid = seq_range(A, s, t0, t1);
  if (seq_slot(A, s, valid, h == 0 && blockIdx.y == 0 && tid == 0) < 0) return;
  const int col = 16 * CT * ((int)blockIdx.y * NW + w) + CT * c16;
  const long long so = ((long long)s * A.H + h) * D * D + col;
  auto state_row = [&](int rt, int i) { return 32 * (rt >> 1) + 8 * g + 4 * (rt & 1) + i; };
  f4 G[CT][2 * NB];
#pragma unroll
  for (int rt = 0; rt < 2 * NB; rt++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      float x[CT] = {};
      if (B.dS_out) loadn<kF32, CT>(B.dS_out, so + (long long)state_row(rt, i) * D, x);
#pragma unroll
      for (int ct = 0; ct < CT; ct++) G[ct][rt][i] = x[ct];
    }
  auto store_G = [&](float* dst) {
#pragma unroll
    for (int rt = 0; rt < 2 * NB; rt++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float x[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ct++) x[ct] = G[ct][rt][i];
        storen<kF32, CT>(dst, (long long)state_row(rt, i) * D, x);
      }
  };
  const long long j0 = first_slot(A, s);
  const char* const heads = A.ws + key_bytes<L>(A);
  const int hq = h / A.grp;
  for (int c = (t1 - t0 + kChunk - 1) / kChunk - 1; c >= 0; c--) {
    const char* const key = A.ws + ((j0 + c) * A.Hq + hq) * L::key;
    const char* const head = heads + ((j0 + c) * A.H + h) * L::head;
    __syncthreads();
    for (int i = tid * 16; i < keyN; i += 64 * NW * 16) *(f4*)(lds + i) = *(const f4*)(key + i);
    for (int i = tid * 16; i < triN; i += 64 * NW * 16) *(f4*)(lds + offTt + i) = *(const f4*)(head + L::offTt + i);
    for (int i = tid * 16; i < 2048; i += 64 * NW * 16) *(f4*)(lds + offTab + i) = *(const f4*)(head + L::offTab + i);
    store_G(keep.G + ((j0 + c) * A.H + h) * D * D + col);
    const int tc = t0 + c * kChunk, len = t1 - tc < kChunk ? t1 - tc : kChunk;
    f4 dO[CT][4];  // accumulator order, zero behind the end
#pragma unroll
    for (int rt = 0; rt < 4; rt++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int t = state_row(rt, i);
        float x[CT] = {};
        if (t < len) loadn<DT, CT>(B.d_out, (tc + (long long)t) * A.os + (long long)h * D + col, x);
#pragma unroll
        for (int ct = 0; ct < CT; ct++) dO[ct][rt][i] = x[ct];
      }
    __syncthreads();
    const float* const tab = (const float*)(lds + offTab);
    auto frag = [&](int off, int n, int p, int f) { return *(const h8*)(lds + off + (p * n + f) * kFrag + lane * 16); };
    auto rows = [&](int t, int rt) { return *(const f4*)(tab + t + 32 * (rt >> 1) + 8 * g + 4 * (rt & 1)); };
    // dW = P^T dO + D K dS1
    h8 Gh[CT][NB], Gl[CT][NB], xh[CT][2], xl[CT][2];
    float iG[CT], ix[CT];
    f4 Y[CT][4];
#pragma unroll
    for (int ct = 0; ct < CT; ct++) {
      iG[ct] = to_operand<NB, 2>(G[ct], Gh[ct], Gl[ct]);
      ix[ct] = to_operand<2, NPI>(dO[ct], xh[ct], xl[ct]);
    }
#pragma unroll
    for (int rt = 0; rt < 4; rt++) {
      f4 u[CT] = {}, y[CT] = {};
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        const h8 a = frag(L::offK, L::NF, 0, rt * KS + ks);
#pragma unroll
        for (int ct = 0; ct < CT; ct++) u[ct] = mfma(a, Gl[ct][ks], mfma(a, Gh[ct][ks], u[ct]));
        if constexpr (NPI == 2) {
          const h8 al = frag(L::offK, L::NF, 1, rt * KS + ks);
#pragma unroll
          for (int ct = 0; ct < CT; ct++) u[ct] = mfma(al, Gh[ct][ks], u[ct]);
        }
      }
#pragma unroll
      for (int ks = rt >> 1; ks < 2; ks++) {
        const h8 a = frag(offP, kTri, 0, up_frag(rt, ks)), al = frag(offP, kTri, 1, up_frag(rt, ks));
#pragma unroll
        for (int ct = 0; ct < CT; ct++) {
          y[ct] = mfma(al, xh[ct][ks], mfma(a, xh[ct][ks], y[ct]));
          if constexpr (NPI == 2) y[ct] = mfma(a, xl[ct][ks], y[ct]);
        }
      }
      const f4 cd = rows(kTabD, rt), ip = rows(kTabP, rt);
#pragma unroll
      for (int ct = 0; ct < CT; ct++)
#pragma unroll
        for (int i = 0; i < 4; i++) Y[ct][rt][i] = fmaf(cd[i] * iG[ct], u[ct][i], (ip[i] * ix[ct]) * y[ct][i]);
    }
    // Y = T^T dW
#pragma unroll
    for (int ct = 0; ct < CT; ct++) ix[ct] = to_operand<2, 2>(Y[ct], xh[ct], xl[ct]);
    float* const dstY = keep.Y + ((j0 + c) * A.H + h) * 64 * D + col;
#pragma unroll
    for (int rt = 0; rt < 4; rt++) {
      f4 y[CT] = {};
#pragma unroll
      for (int ks = rt >> 1; ks < 2; ks++) {
        const h8 a = frag(offTt, kTri, 0, up_frag(rt, ks)), al = frag(offTt, kTri, 1, up_frag(rt, ks));
#pragma unroll
        for (int ct = 0; ct < CT; ct++) y[ct] = mfma(al, xh[ct][ks], mfma(a, xl[ct][ks], mfma(a, xh[ct][ks], y[ct])));
      }
      const f4 it = rows(kTabTt, rt), be = rows(kTabB, rt);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int t = state_row(rt, i);
        float x[CT], v[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ct++) {
          Y[ct][rt][i] = x[ct] = y[ct][i] * (it[i] * ix[ct]);
          v[ct] = be[i] * x[ct];
        }
        storen<kF32, CT>(dstY, (long long)t * D, x);
        if (t < len) storen<DT, CT>(B.dv, ((tc + (long long)t) * A.H + h) * D + col, v);
      }
    }
    // dS0 = G_C dS1 + Q^T G dO - K^T G diag(beta) Y
    h8 qh[CT][2], ql[CT][2];
    float iq[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ct++) {
#pragma unroll
      for (int rt = 0; rt < 4; rt++) {
        dO[ct][rt] *= rows(kTabQ, rt);
        Y[ct][rt] *= -rows(kTabU, rt);
      }
      iq[ct] = to_operand<2, 2>(dO[ct], qh[ct], ql[ct]);
      ix[ct] = to_operand<2, 2>(Y[ct], xh[ct], xl[ct]);
    }
    const float GC = tab[kTabG + 63];
#pragma unroll
    for (int rt = 0; rt < 2 * NB; rt++) {
      f4 y[CT] = {}, z[CT] = {};
#pragma unroll
      for (int ks = 0; ks < 2; ks++) {
        const h8 a = frag(L::offKT, L::NF, 0, 2 * rt + ks), b = frag(L::offQ, L::NF, 0, 2 * rt + ks);
#pragma unroll
        for (int ct = 0; ct < CT; ct++) {
          y[ct] = mfma(a, xl[ct][ks], mfma(a, xh[ct][ks], y[ct]));
          z[ct] = mfma(b, ql[ct][ks], mfma(b, qh[ct][ks], z[ct]));
        }
        if constexpr (NPI == 2) {
          const h8 al = frag(L::offKT, L::NF, 1, 2 * rt + ks), bl = frag(L::offQ, L::NF, 1, 2 * rt + ks);
#pragma unroll
          for (int ct = 0; ct < CT; ct++) {
            y[ct] = mfma(al, xh[ct][ks], y[ct]);
            z[ct] = mfma(bl, qh[ct][ks], z[ct]);
          }
        }
      }
#pragma unroll
      for (int ct = 0; ct < CT; ct++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          G[ct][rt][i] = fmaf(GC, G[ct][rt][i], fmaf(ix[ct], y[ct][i], iq[ct] * z[ct][i]));
    }
  }
  if (B.dS_in) store_G(B.dS_in + so);
}

// ---------------------------------------------------------------------------------------------
// every chunk's gradients
// ---------------------------------------------------------------------------------------------

// Sum over the 16 lanes of a row.
__device__ __forceinline__ float sum16(float x) {
  x += __shfl_xor(x, 1);
  x += __shfl_xor(x, 2);
  x += __shfl_xor(x, 4);
  x += __shfl_xor(x, 8);
  return x;
}

template <int D, int DT>
struct GradSmem {
  static constexpr int NPI = kInPlanes<DT>, NW = D / 16;
  union {
    struct {
      _Float16 O[NPI][64][D + 8], Y[2][64][D + 8], W[2][64][D + 8];
    } in;
    struct {  // N, N^T and Z + Z^T with K's or Q's scales folded into their columns; xT[s][t] the pairs
      float L[64][kPitch], N[64][kPitch], Nt[64][kPitch], Z[64][kPitch], xT[64][kPitch];
    } m;
    float out[64][D + 4];
  };
  char fr[20 * 2 * kFrag];  // fragments of N (6), N^T (6) and Z (8)
  float isO[64], isY[64], isW[64], sN[3][64], iN[3][64];
  float al[64], be[64], yv[64], rowx[2][64], dot[3][NW][64], corner[NW], z[64], y[64], extra[64];
};

// Rows of a 64-row operand as planes, TPR threads a row; zero from row `len` on.  vrow: adds the row's
// product with a row of v (the strengths' gradient).
template <int D, int DT, int ET, int NP, int TPR>
__device__ __forceinline__ void rows_in(const void* src, long long at, bool live, _Float16 (*dst)[64][D + 8],
                                        float* is, const void* vsrc, long long vat, float* dot) {
  constexpr int E = D / TPR;
  const int row = threadIdx.x / TPR, part = threadIdx.x % TPR;
  float x[E], m = 0.0f, p = 0.0f;
#pragma unroll
  for (int i = 0; i < E; i += 8) {
#pragma unroll
    for (int e = 0; e < 8; e++) x[i + e] = 0.0f;
    if (live) load8<ET>(src, at + part * E + i, x + i);
#pragma unroll
    for (int e = 0; e < 8; e++) m = fmaxf(m, fabsf(x[i + e]));
    if (dot && live) {
      float v[8];
      load8<DT>(vsrc, vat + part * E + i, v);
#pragma unroll
      for (int e = 0; e < 8; e++) p = fmaf(x[i + e], v[e], p);
    }
  }
#pragma unroll
  for (int o = 1; o < TPR; o <<= 1) {
    m = fmaxf(m, __shfl_xor(m, o));
    if (dot) p += __shfl_xor(p, o);
  }
  float inv;
  const float s = scale_of(m, inv);
  if (part == 0) {
    is[row] = inv;
    if (dot) dot[row] = p;
  }
#pragma unroll
  for (int i = 0; i < E; i += 8) {
    h8 hi, lo;
    split8<NP>(x + i, s, hi, lo);
    *(h8*)&dst[0][row][part * E + i] = hi;
    if constexpr (NP == 2) *(h8*)&dst[1][row][part * E + i] = lo;
  }
}

// One workgroup of D / 16 waves per (chunk, key head); the value heads that share the key head one after
// another, dQ and dK summed in registers.  Wave w owns the 16 key dimensions 32 (w >> 1) + perm(., w & 1).
template <int D, int DT>
__global__ __launch_bounds__(4 * D) void k_chunk_grad(GradArgs B, Keep keep) {
  using Y = LayB<D, DT>;
  constexpr int KS = D / 32, NPI = Y::NPI, NW = D / 16, NT = 4 * D, TPR = NT / 64;
  __shared__ GradSmem<D, DT> sm;
  const SeqArgs& A = B.f;
  const long long j = blockIdx.x;
  const int hq = blockIdx.y;
  ChunkAt at;
  if (!chunk_at(A, j, at)) return;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  const int dk = 32 * (w >> 1) + perm_row(c16, w & 1);
  const char* const key = A.ws + (j * A.Hq + hq) * Y::key;
  const float* const KK = (const float*)(key + Y::offKK);
  const float* const QK = (const float*)(key + Y::offQK);
  const int row = tid / TPR;
  const f4 zero = {0, 0, 0, 0};
  f4 dQ[4] = {zero, zero, zero, zero}, dK[4] = {zero, zero, zero, zero};
  for (int hh = 0; hh < A.grp; hh++) {
    const int h = hq * A.grp + hh;
    const float* const tab = (const float*)(A.ws + key_bytes<Y>(A) + (j * A.H + h) * Y::head + Y::offTab);
    const long long jh = j * A.H + h;
    __syncthreads();
    if (tid < 64) {
      const long long th = (at.t0 + (long long)(tid < at.len ? tid : 0)) * A.H + h;
      sm.al[tid] = tid < at.len ? A.alpha[th] : 1.0f;
      sm.be[tid] = tid < at.len ? A.beta[th] : 0.0f;
    }
    const long long tok = at.t0 + (long long)row;
    rows_in<D, DT, DT, NPI, TPR>(B.d_out, tok * A.os + (long long)h * D, row < at.len, sm.in.O, sm.isO, nullptr, 0, nullptr);
    rows_in<D, DT, kF32, 2, TPR>(keep.Y, (jh * 64 + row) * D, row < at.len, sm.in.Y, sm.isY, A.v, tok * A.vs + (long long)h * D, sm.yv);
    rows_in<D, DT, kF32, 2, TPR>(keep.W, (jh * 64 + row) * D, row < at.len, sm.in.W, sm.isW, nullptr, 0, nullptr);
    __syncthreads();
    // products with the states: this wave's 16 rows of S0 and dS1 as column operands
    {
      h8 Sh[KS], Sl[KS], Gh[KS], Gl[KS];
      float iS, iG;
      {
        float x[KS][8], y[KS][8], m = 0.0f, n = 0.0f, cn = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
          load8<kF32>(keep.S, (jh * D + dk) * D + 32 * ks + 8 * g, x[ks]);
          load8<kF32>(keep.G, (jh * D + dk) * D + 32 * ks + 8 * g, y[ks]);
#pragma unroll
          for (int e = 0; e < 8; e++) {
            m = fmaxf(m, fabsf(x[ks][e]));
            n = fmaxf(n, fabsf(y[ks][e]));
            cn = fmaf(x[ks][e], y[ks][e], cn);
          }
        }
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        n = fmaxf(n, __shfl_xor(n, 16));
        n = fmaxf(n, __shfl_xor(n, 32));
        cn = sum16(cn);
        cn += __shfl_xor(cn, 16);
        cn += __shfl_xor(cn, 32);
        if (lane == 0) sm.corner[w] = cn;
        const float s = scale_of(m, iS), r = scale_of(n, iG);
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
          split8<2>(x[ks], s, Sh[ks], Sl[ks]);
          split8<2>(y[ks], r, Gh[ks], Gl[ks]);
        }
      }
#pragma unroll
      for (int rt = 0; rt < 4; rt++) {
        f4 e1 = zero, e2 = zero, e3 = zero;
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
          const int r = 16 * rt + c16, k = 32 * ks + 8 * g;
          const h8 o = *(const h8*)&sm.in.O[0][r][k];
          e1 = mfma(o, Sl[ks], mfma(o, Sh[ks], e1));
          if constexpr (NPI == 2) e1 = mfma(*(const h8*)&sm.in.O[1][r][k], Sh[ks], e1);
          const h8 yh = *(const h8*)&sm.in.Y[0][r][k], yl = *(const h8*)&sm.in.Y[1][r][k];
          e2 = mfma(yl, Sh[ks], mfma(yh, Sl[ks], mfma(yh, Sh[ks], e2)));
          const h8 wh = *(const h8*)&sm.in.W[0][r][k], wl = *(const h8*)&sm.in.W[1][r][k];
          e3 = mfma(wl, Gh[ks], mfma(wh, Gl[ks], mfma(wh, Gh[ks], e3)));
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int t = 16 * rt + 4 * g + i;
          const float a = e1[i] * (sm.isO[t] * iS), b = e2[i] * (sm.isY[t] * iS), c = e3[i] * (sm.isW[t] * iG);
          const float G = tab[kTabG + t];
          dQ[rt][i] = fmaf(G, a, dQ[rt][i]);
          dK[rt][i] = fmaf(-G * sm.be[t], b, fmaf(tab[kTabL + t], c, dK[rt][i]));
          float q = 0.0f, k = 0.0f;
          if (t < at.len) {
            loadn<DT, 1>(A.q, (at.t0 + (long long)t) * A.qs + (long long)hq * D + dk, &q);
            loadn<DT, 1>(A.k, (at.t0 + (long long)t) * A.ks + (long long)hq * D + dk, &k);
          }
          const float zq = sum16(q * a), zk = sum16(k * b), yk = sum16(k * c);
          if (c16 == 0) {
            sm.dot[0][w][t] = zq;
            sm.dot[1][w][t] = zk;
            sm.dot[2][w][t] = yk;
          }
        }
      }
    }
    // dO W^T and Y W^T: lower tiles, row tile rt with the columns of one parity (D = 128), or all (64)
    constexpr int NC = NW == 8 ? 2 : 4, step = NW == 8 ? 2 : 1;
    const int rt = NW == 8 ? w >> 1 : w, c0 = NW == 8 ? w & 1 : 0;
    f4 dp[NC], dx[NC];
#pragma unroll
    for (int n = 0; n < NC; n++) {
      dp[n] = dx[n] = zero;
      const int c = c0 + step * n;
      if (c > rt) continue;
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        const int r = 16 * rt + c16, q = 16 * c + c16, k = 32 * ks + 8 * g;
        const h8 wh = *(const h8*)&sm.in.W[0][q][k], wl = *(const h8*)&sm.in.W[1][q][k];
        const h8 o = *(const h8*)&sm.in.O[0][r][k];
        dp[n] = mfma(o, wl, mfma(o, wh, dp[n]));
        if constexpr (NPI == 2) dp[n] = mfma(*(const h8*)&sm.in.O[1][r][k], wh, dp[n]);
        const h8 yh = *(const h8*)&sm.in.Y[0][r][k], yl = *(const h8*)&sm.in.Y[1][r][k];
        dx[n] = mfma(yl, wh, mfma(yh, wl, mfma(yh, wh, dx[n])));
      }
    }
    __syncthreads();  // the planes are free: matrices in their place
    {
      constexpr int RW = 64 / NW;  // rows of L a wave
      int ln = lane;
      asm("" : "+v"(ln));
      float l = 1.0f;
      for (int t = 0; t < RW * w; t++) l = t > ln ? l * sm.al[t] : 1.0f;
#pragma unroll
      for (int i = 0; i < RW; i++) {
        const int t = RW * w + i;
        l = t > ln ? l * sm.al[t] : 1.0f;
        sm.m.L[t][ln] = t >= ln ? l : 0.0f;
      }
      if (tid < 64) {
        float zq = 0.0f, zk = 0.0f, yk = 0.0f;
#pragma unroll
        for (int v = 0; v < NW; v++) zq += sm.dot[0][v][tid], zk += sm.dot[1][v][tid], yk += sm.dot[2][v][tid];
        sm.z[tid] = fmaf(-sm.be[tid], zk, zq);
        sm.y[tid] = yk;
        sm.yv[tid] = fmaf(-tab[kTabG + tid], zk, sm.yv[tid]);
      }
    }
    __syncthreads();
    {
      float rx[4] = {};
#pragma unroll
      for (int n = 0; n < NC; n++) {
        const int c = c0 + step * n, s = 16 * c + c16;
        const float ik = tab[kTabIK + s];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int t = 16 * rt + 4 * g + i;
          if (c > rt) {
            sm.m.N[t][s] = 0.0f;
            sm.m.Nt[s][t] = 0.0f;
            continue;
          }
          float nv = 0.0f, zv = 0.0f, x = 0.0f;
          if (s <= t) {
            const float l = sm.m.L[t][s], p = dp[n][i] * (sm.isO[t] * sm.isW[s]);
            nv = p * l;
            x = p * QK[s * 64 + t];
            if (s < t) {
              const float y = dx[n][i] * (sm.isY[t] * sm.isW[s]), kk = KK[t * 64 + s], b = sm.be[t] * y;
              zv = -b * l;
              x = fmaf(-b, kk, x);
              rx[i] = fmaf(y, l * kk, rx[i]);
            }
          }
          sm.m.N[t][s] = nv * ik;
          sm.m.Nt[s][t] = nv * tab[kTabIQ + t];
          if (s <= t) {
            sm.m.Z[t][s] = zv * ik;
            sm.m.Z[s][t] = zv * tab[kTabIK + t];
          }
          sm.m.xT[s][t] = x;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float v = sum16(rx[i]);
        if (c16 == 0) sm.rowx[NW == 8 ? w & 1 : 0][16 * rt + 4 * g + i] = v;
      }
    }
    __syncthreads();
    // row scales of N, N^T and Z
    {
      constexpr int E = 64 / TPR;
      const int part = tid % TPR;
      float m[3] = {};
#pragma unroll
      for (int i = 0; i < E; i++) {
        m[0] = fmaxf(m[0], fabsf(sm.m.N[row][part * E + i]));
        m[1] = fmaxf(m[1], fabsf(sm.m.Nt[row][part * E + i]));
        m[2] = fmaxf(m[2], fabsf(sm.m.Z[row][part * E + i]));
      }
#pragma unroll
      for (int v = 0; v < 3; v++) {
#pragma unroll
        for (int o = 1; o < TPR; o <<= 1) m[v] = fmaxf(m[v], __shfl_xor(m[v], o));
        if (part == 0) {
          float inv;
          sm.sN[v][row] = scale_of(m[v], inv);
          sm.iN[v][row] = inv;
        }
      }
    }
    __syncthreads();
    // fragments: N row tile rt, k-steps ks <= rt / 2; N^T ks >= rt / 2; Z all
    for (int f = w; f < 20; f += NW) {
      const int v = f < 6 ? 0 : f < 12 ? 1 : 2, e = f - 6 * v;
      const int r = v == 0 ? (e < 2 ? e : 2 + ((e - 2) >> 1)) : v == 1 ? (e < 4 ? e >> 1 : e - 2) : e >> 1;
      const int ks = v == 0 ? (e < 2 ? 0 : (e - 2) & 1) : v == 1 ? (e < 4 ? e & 1 : 1) : e & 1;
      const float* src = v == 0 ? &sm.m.N[16 * r + c16][32 * ks + 8 * g]
                                : v == 1 ? &sm.m.Nt[16 * r + c16][32 * ks + 8 * g] : &sm.m.Z[16 * r + c16][32 * ks + 8 * g];
      const f4 x0 = *(const f4*)src, x1 = *(const f4*)(src + 4);
      const float x[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
      h8 hi, lo;
      split8<2>(x, sm.sN[v][16 * r + c16], hi, lo);
      *(h8*)(sm.fr + 2 * f * kFrag + lane * 16) = hi;
      *(h8*)(sm.fr + (2 * f + 1) * kFrag + lane * 16) = lo;
    }
    // gates: lane t follows F_r = sum over s < r of x[t,s] L[r-1,s]; xT[r][t] becomes L[t,r] F_r
    if (w == NW - 1) {
      float F = sm.z[lane], C = 0.0f, mine = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; v++) C += sm.corner[v];
#pragma unroll 8
      for (int r = 0; r < 64; r++) {
        const float x = sm.m.xT[r][lane], a = sm.al[r];
        sm.m.xT[r][lane] = lane >= r ? sm.m.L[lane][r] * F : 0.0f;
        mine = lane == r ? C : mine;
        F = fmaf(a, F, x);
        C = fmaf(a, C, sm.y[r]);
      }
      sm.extra[lane] = sm.m.L[63][lane] * mine;
    }
    __syncthreads();
    {
      f4 n[4] = {zero, zero, zero, zero}, t[4] = {zero, zero, zero, zero}, z[4] = {zero, zero, zero, zero};
      auto fr = [&](int f, int p) { return *(const h8*)(sm.fr + (2 * f + p) * kFrag + lane * 16); };
#pragma unroll
      for (int ks = 0; ks < 2; ks++) {
        const h8 k = *(const h8*)(key + Y::offKT + (2 * w + ks) * kFrag + lane * 16);
        const h8 q = *(const h8*)(key + Y::offQ + (2 * w + ks) * kFrag + lane * 16);
        h8 kl, ql;
        if constexpr (NPI == 2) {
          kl = *(const h8*)(key + Y::offKT + (Y::NF + 2 * w + ks) * kFrag + lane * 16);
          ql = *(const h8*)(key + Y::offQ + (Y::NF + 2 * w + ks) * kFrag + lane * 16);
        }
#pragma unroll
        for (int r = 0; r < 4; r++) {
          if (ks <= r >> 1) {
            const h8 a = fr(tri_frag(r, ks), 0);
            n[r] = mfma(fr(tri_frag(r, ks), 1), k, mfma(a, k, n[r]));
            if constexpr (NPI == 2) n[r] = mfma(a, kl, n[r]);
          }
          if (ks >= r >> 1) {
            const h8 a = fr(6 + up_frag(r, ks), 0);
            t[r] = mfma(fr(6 + up_frag(r, ks), 1), q, mfma(a, q, t[r]));
            if constexpr (NPI == 2) t[r] = mfma(a, ql, t[r]);
          }
          const h8 a = fr(12 + 2 * r + ks, 0);
          z[r] = mfma(fr(12 + 2 * r + ks, 1), k, mfma(a, k, z[r]));
          if constexpr (NPI == 2) z[r] = mfma(a, kl, z[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; r++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int tt = 16 * r + 4 * g + i;
          dQ[r][i] = fmaf(sm.iN[0][tt], n[r][i], dQ[r][i]);
          dK[r][i] = fmaf(sm.iN[1][tt], t[r][i], fmaf(sm.iN[2][tt], z[r][i], dK[r][i]));
        }
    }
    {
      constexpr int E = 64 / TPR;
      const int part = tid % TPR;
      float a = 0.0f;
#pragma unroll
      for (int i = 0; i < E; i++) a += sm.m.xT[row][part * E + i];
#pragma unroll
      for (int o = 1; o < TPR; o <<= 1) a += __shfl_xor(a, o);
      if (part == 0 && row < at.len) {
        const long long th = (at.t0 + (long long)row) * A.H + h;
        B.dalpha[th] = a + sm.extra[row];
        B.dbeta[th] = sm.yv[row] - (sm.rowx[0][row] + (NW == 8 ? sm.rowx[1][row] : 0.0f));
      }
    }
  }
  // dQ and dK to rows through LDS
#pragma unroll
  for (int which = 0; which < 2; which++) {
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
      for (int i = 0; i < 4; i++) sm.out[16 * r + 4 * g + i][dk] = which ? dK[r][i] : dQ[r][i];
    __syncthreads();
    constexpr int E = D / TPR;
    if (row < at.len) {
      const long long o = ((at.t0 + (long long)row) * A.Hq + hq) * D + (tid % TPR) * E;
#pragma unroll
      for (int i = 0; i < E; i += 8) store8<DT>(which ? B.dk : B.dq, o + i, &sm.out[row][(tid % TPR) * E + i]);
    }
  }
}

template <int D, int DT>
size_t fixed_bytes(const SeqArgs& a) {
  return (size_t)(key_bytes<LayB<D, DT>>(a) + head_bytes<LayB<D, DT>>(a));
}

template <int D, int DT>
size_t bytes(const SeqArgs& a) {
  return fixed_bytes<D, DT>(a) + (size_t)chunk_slots(a.T, a.N) * a.H * (2 * D * D + 2 * 64 * D) * sizeof(float);
}

template <int D, int DT>
hipError_t launch(GradArgs b, hipStream_t s) {
  SeqArgs& a = b.f;
  const size_t n = (size_t)chunk_slots(a.T, a.N) * a.H;
  Keep keep;
  keep.S = (float*)(a.ws + fixed_bytes<D, DT>(a));
  keep.G = keep.S + n * D * D;
  keep.W = keep.G + n * D * D;
  keep.Y = keep.W + n * 64 * D;
  constexpr int CT = D == 128 ? 2 : 1;
  const dim3 slots((unsigned)chunk_slots(a.T, a.N), a.Hq), tiles((unsigned)((long long)a.N * a.H), D / (64 * CT));
  unsigned* const status = a.status;
  a.status = nullptr;  // reported once, by the reverse pass
  if (a.T > 0) {
    hipLaunchKernelGGL((k_chunk_prep<D, DT, LayB<D, DT>>), slots, dim3(256), 0, s, a);
    hipLaunchKernelGGL((k_chunk_state<D, DT, D / 16, LayB<D, DT>>), dim3(tiles.x, 1), dim3(4 * D), 0, s, a, keep.S, keep.W);
  }
  a.status = status;
  hipLaunchKernelGGL((k_chunk_reverse<D, DT, CT, 4>), tiles, dim3(256), 0, s, b, keep);
  if (a.T > 0) hipLaunchKernelGGL((k_chunk_grad<D, DT>), slots, dim3(4 * D), 0, s, b, keep);
  return hipGetLastError();
}

}  // namespace

size_t chunk_backward_bytes(const SeqArgs& a) {
  if (a.N <= 0) return 0;
  if (a.D == 64)
    return a.dtype == kF32 ? bytes<64, kF32>(a) : a.dtype == kBF16 ? bytes<64, kBF16>(a) : bytes<64, kF16>(a);
  return a.dtype == kF32 ? bytes<128, kF32>(a) : a.dtype == kBF16 ? bytes<128, kBF16>(a) : bytes<128, kF16>(a);
}

hipError_t launch_chunk_backward(const GradArgs& b, hipStream_t s) {
  const SeqArgs& a = b.f;
  if (a.N <= 0) return hipSuccess;
  if (a.D == 64)
    return a.dtype == kF32 ? launch<64, kF32>(b, s) : a.dtype == kBF16 ? launch<64, kBF16>(b, s) : launch<64, kF16>(b, s);
  return a.dtype == kF32 ? launch<128, kF32>(b, s) : a.dtype == kBF16 ? launch<128, kBF16>(b, s) : launch<128, kF16>(b, s);
}

}  // namespace stepq
