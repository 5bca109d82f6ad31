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

// The reverse pass: like k_chunk_state a wave owns 16 columns of one state's gradient for the whole sequence
// and holds it in units of a power of two per column.
template <int D, int DT, int NW>
__global__ __launch_bounds__(64 * NW) void k_chunk_reverse(GradArgs B, Keep keep) {
  using L = LayB<D, DT>;
  constexpr int KS = D / 32, NPI = L::NPI, NB = D / 32;
  constexpr int keyN = L::offKK, triN = 4 * kTri * kFrag;  // K, K^T, Q^T; T^T, P^T
  constexpr int offTt = keyN, offP = keyN + 2 * kTri * kFrag, offTab = keyN + triN;
  constexpr int part = offTab + 2048;
  constexpr int NBUF = 2 * part <= 160 * 1024 ? 2 : 1;
  const SeqArgs& A = B.f;
  __shared__ __attribute__((aligned(16))) char buf[NBUF * part];
  const long long tile = blockIdx.x;
  const int s = (int)(tile / A.H), h = (int)(tile - (long long)s * A.H);
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  int t0, t1;
  const bool valid = seq_range(A, s, t0, t1);
  if (seq_slot(A, s, valid, h == 0 && blockIdx.y == 0 && tid == 0) < 0) return;
  const int col = 16 * ((int)blockIdx.y * NW + w) + c16;
  const long long so = ((long long)s * A.H + h) * D * D + col;
  auto state_row = [&](int rt, int i) { return 32 * (rt >> 1) + 8 * g + 4 * (rt & 1) + i; };
  f4 Gt[2 * NB];
#pragma unroll
  for (int rt = 0; rt < 2 * NB; rt++)
#pragma unroll
    for (int i = 0; i < 4; i++) Gt[rt][i] = B.dS_out ? B.dS_out[so + (long long)state_row(rt, i) * D] : 0.0f;
  float unit = 0x1p-10f;
  auto rescale = [&](float m) {
    float inv;
    const float f = m > 0.0f ? scale_of(m, inv) : (inv = 1.0f);
    unit *= inv;
#pragma unroll
    for (int rt = 0; rt < 2 * NB; rt++) Gt[rt] *= f;
  };
  {
    const float m = tiles_max<2 * NB>(Gt);
    if (m > 0.0f) unit = 1.0f;
    rescale(m);
  }
  auto store_G = [&](float* dst) {
#pragma unroll
    for (int rt = 0; rt < 2 * NB; rt++)
#pragma unroll
      for (int i = 0; i < 4; i++) dst[(long long)state_row(rt, i) * D] = Gt[rt][i] * unit;
  };
  const long long j0 = first_slot(A, s);
  const char* const heads = A.ws + key_bytes<L>(A);
  const int hq = h / A.grp;
  const int nc = (t1 - t0 + kChunk - 1) / kChunk;
  const unsigned lds0 = lds_offset(buf), lane16 = 16 * lane;
  auto fetch = [&](int c) {
    const char* const key = A.ws + ((j0 + c) * A.Hq + hq) * L::key;
    const char* const head = heads + ((j0 + c) * A.H + h) * L::head;
    const unsigned at = lds0 + (NBUF == 2 ? (c & 1) * part : 0);
    copy_block<NW>(key, at, keyN, w, lane16);
    copy_block<NW>(head + L::offTt, at + offTt, triN, w, lane16);
    copy_block<NW>(head + L::offTab, at + offTab, 2048, w, lane16);
  };
  const Rows<DT> orows(A.os, col, g), vrows((long long)A.H * D, col, g);
  unsigned o[4][4];
  auto fetch_o = [&](int c) {
    const int tc = t0 + c * kChunk;
    orows.load(orows.at(B.d_out, tc, A.os, h * D, D, t1 - tc < kChunk ? t1 - tc : kChunk), o);
  };
  if (nc) {
    fetch(nc - 1);
    fetch_o(nc - 1);
  }
  const f4 zero = {0, 0, 0, 0};
  for (int c = nc - 1; c >= 0; c--) {
    const char* const lds = buf + (NBUF == 2 ? (c & 1) * part : 0);
    const int tc = t0 + c * kChunk, len = t1 - tc < kChunk ? t1 - tc : kChunk;
    wait_copies();
    __syncthreads();
    f4 dO[4];
#pragma unroll
    for (int rt = 0; rt < 4; rt++)
#pragma unroll
      for (int i = 0; i < 4; i++) dO[rt][i] = orows.value(o[rt][i]);
    if (c) {
      if (NBUF == 2) fetch(c - 1);
      fetch_o(c - 1);
    }
    const float* const tab = (const float*)(lds + offTab);
    auto frag = [&](int off, int n, int p, int f) { return *(const h8*)(lds + off + (p * n + f) * kFrag + lane16); };
    auto rows = [&](int t, int rt) { return *(const f4*)(tab + t + 32 * (rt >> 1) + 8 * g + 4 * (rt & 1)); };
    h8 f[L::NF], fl[NPI == 2 ? L::NF : 1];
    auto read = [&](int off) {
#pragma unroll
      for (int n = 0; n < L::NF; n++) {
        f[n] = frag(off, L::NF, 0, n);
        if constexpr (NPI == 2) fl[n] = frag(off, L::NF, 1, n);
      }
    };
    h8 ft[2][kTri];
    auto read_tri = [&](int off) {
#pragma unroll
      for (int n = 0; n < kTri; n++) {
        ft[0][n] = frag(off, kTri, 0, n);
        ft[1][n] = frag(off, kTri, 1, n);
      }
    };
    read(L::offK);
    ahead();
    {
      const float m = tiles_max<2 * NB>(Gt);
      if (__any(m > 0x1p14f || (m < 1.0f && m > 0.0f))) rescale(m);
    }
    store_G(keep.G + ((j0 + c) * A.H + h) * D * D + col);
    h8 xh[2], xl[2];
    f4 z[4], y[4];
    {  // z = K dS1
      h8 Gh[NB], Gl[NB];
      to_planes<NB, 2, true>(Gt, 1.0f, Gh, Gl);
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int rt = 0; rt < 4; rt++) z[rt] = mfma(f[rt * KS + ks], Gh[ks], ks ? z[rt] : zero);
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int rt = 0; rt < 4; rt++) z[rt] = mfma(f[rt * KS + ks], Gl[ks], z[rt]);
      if constexpr (NPI == 2)
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
          for (int rt = 0; rt < 4; rt++) z[rt] = mfma(fl[rt * KS + ks], Gh[ks], z[rt]);
    }
    ahead();
    read_tri(offP);
    ahead();
    auto tri = [&](int p, const h8* b, bool first) {
#pragma unroll
      for (int ks = 1; ks >= 0; ks--)
#pragma unroll
        for (int rt = 0; rt < 4; rt++)
          if (ks >= rt >> 1) y[rt] = mfma(ft[p][up_frag(rt, ks)], b[ks], first && ks ? zero : y[rt]);
    };
    float ix = to_operand<2, NPI>(dO, xh, xl);
    tri(0, xh, true);
    tri(1, xh, false);
    if constexpr (NPI == 2) tri(0, xl, false);
    ahead();
    read_tri(offTt);
    ahead();
    // dW = P^T dO + D K dS1, then Y = T^T dW
    f4 Y[4];
#pragma unroll
    for (int rt = 0; rt < 4; rt++) {
      const f4 cd = rows(kTabD, rt), ip = rows(kTabP, rt);
#pragma unroll
      for (int i = 0; i < 4; i++) Y[rt][i] = fmaf(cd[i] * unit, z[rt][i], (ip[i] * ix) * y[rt][i]);
    }
    ix = to_operand<2, 2>(Y, xh, xl);
    tri(0, xh, true);
    tri(0, xl, false);
    tri(1, xh, false);
    ahead();
    read(L::offQ);
    ahead();
    {
      float* const dst = keep.Y + ((j0 + c) * A.H + h) * 64 * D + col;
      const __amdgpu_buffer_rsrc_t dv = vrows.at(B.dv, tc, (long long)A.H * D, h * D, D, len);
#pragma unroll
      for (int rt = 0; rt < 4; rt++) {
        const f4 it = rows(kTabTt, rt), be = rows(kTabB, rt);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          Y[rt][i] = y[rt][i] * (it[i] * ix);
          dst[(long long)state_row(rt, i) * D] = Y[rt][i];
          vrows.store(dv, rt, i, be[i] * Y[rt][i]);
        }
      }
    }
    // dS0 = G_C dS1 + Q^T G dO - K^T G diag(beta) Y, in the gradient's units
#pragma unroll
    for (int rt = 0; rt < 4; rt++) {
      dO[rt] *= rows(kTabQ, rt);
      Y[rt] *= -rows(kTabU, rt);
    }
    {
      const float m = fmaxf(tiles_max<4>(dO), tiles_max<4>(Y));
      if (__any(m > unit * 0x1p14f)) {
        float inv, to = unit;
        if (m > unit * 0x1p14f) {
          (void)scale_of(m, inv);
          to = inv;
        }
        const float r = unit / to;
#pragma unroll
        for (int rt = 0; rt < 2 * NB; rt++) Gt[rt] *= r;
        unit = to;
      }
    }
    const float GC = tab[kTabG + 63], iu = 1.0f / unit;
#pragma unroll
    for (int rt = 0; rt < 2 * NB; rt++) Gt[rt] *= GC;
    auto update = [&]() {
#pragma unroll
      for (int ks = 0; ks < 2; ks++) {
#pragma unroll
        for (int rt = 0; rt < 2 * NB; rt++) Gt[rt] = mfma(f[2 * rt + ks], xh[ks], Gt[rt]);
#pragma unroll
        for (int rt = 0; rt < 2 * NB; rt++) Gt[rt] = mfma(f[2 * rt + ks], xl[ks], Gt[rt]);
        if constexpr (NPI == 2)
#pragma unroll
          for (int rt = 0; rt < 2 * NB; rt++) Gt[rt] = mfma(fl[2 * rt + ks], xh[ks], Gt[rt]);
      }
    };
    to_planes<2, 2>(dO, iu, xh, xl);
    update();
    ahead();
    read(L::offKT);
    ahead();
    to_planes<2, 2>(Y, iu, xh, xl);
    update();
    if (NBUF == 1 && c) {
      __syncthreads();
      fetch(c - 1);
    }
  }
  if (B.dS_in) store_G(B.dS_in + so);
}

// ---------------------------------------------------------------------------------------------
// every chunk's gradients
// ---------------------------------------------------------------------------------------------

// Sum over the 16 lanes of a row, without LDS.
template <int N>
__device__ __forceinline__ float add_ror(float x) {
  return x + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x120 + N, 0xf, 0xf, false));
}
__device__ __forceinline__ float sum16(float x) { return add_ror<1>(add_ror<2>(add_ror<4>(add_ror<8>(x)))); }
// Sum over the four rows of 16 lanes.
__device__ __forceinline__ float sum_rows(float x) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

template <int D, int DT>
struct GradSmem {
  static constexpr int NPI = kInPlanes<DT>, NW = D / 16;
  union {
    struct {
      _Float16 O[NPI][64][D + 8], Y[2][64][D + 8], W[2][64][D + 8];
    } in;
    struct {  // N, N^T and Z + Z^T with K's or Q's scales folded into their columns; xT[s][t] the pairs
      float L[64][kPitch], N[64][kPitch], Nt[64][kPitch], Z[64][kPitch], xT[64][kPitch];  // xT[s][t]
    } m;
    float out[64][D + 4];
  };
  char fr[20 * 2 * kFrag];  // fragments of N (6), N^T (6) and Z (8)
  float isO[64], isY[64], isW[64], sN[3][64], iN[3][64];
  float al[64], be[64], yv[64], rowx[2][64], dot[3][NW][64], corner[NW], z[64], y[64], da[64];
};

// Rows of a 64-row operand as planes, TPR threads a row; zero from row `len` on.  vrow: adds the row's
// product with a row of v (the strengths' gradient).
template <int D, int DT, int ET, int NP, int TPR>
__device__ __forceinline__ void rows_in(int tid, const void* src, long long at, bool live, _Float16 (*dst)[64][D + 8],
                                        float* is, const void* vsrc, long long vat, float* dot) {
  constexpr int E = D / TPR;
  const int row = tid / TPR, part = tid % TPR;
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
  int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  int c16 = lane & 15, g = lane >> 4;
  const int dk = 32 * (w >> 1) + perm_row(c16, w & 1);
  const char* const key = A.ws + (j * A.Hq + hq) * Y::key;
  // dO W^T and Y W^T: lower tiles, row tile rt with the columns of one parity (D = 128), or all (64)
  constexpr int NC = NW == 8 ? 2 : 4, step = NW == 8 ? 2 : 1;
  const int rt = NW == 8 ? w >> 1 : w, c0 = NW == 8 ? w & 1 : 0;
  // what all heads share: k_t.k_s and q_t.k_s of this wave's pairs, this lane's column of Q and K
  f4 kk[NC], qk[NC];
#pragma unroll
  for (int n = 0; n < NC; n++) {
    const int c = min(c0 + step * n, rt), s = 16 * c + c16;
#pragma unroll
    for (int i = 0; i < 4; i++) kk[n][i] = ((const float*)(key + Y::offKK))[(16 * rt + 4 * g + i) * 64 + s];
    qk[n] = *(const f4*)((const float*)(key + Y::offQK) + s * 64 + 16 * rt + 4 * g);
  }
  float qv[4][4], kv[4][4];
#pragma unroll
  for (int r = 0; r < 4; r++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const long long t = at.t0 + (long long)min(16 * r + 4 * g + i, at.len - 1);
      loadn<DT, 1>(A.q, t * A.qs + (long long)hq * D + dk, &qv[r][i]);
      loadn<DT, 1>(A.k, t * A.ks + (long long)hq * D + dk, &kv[r][i]);
    }
  int row = tid / TPR;
  const f4 zero = {0, 0, 0, 0};
  f4 dQ[4] = {zero, zero, zero, zero}, dK[4] = {zero, zero, zero, zero};
  for (int hh = 0; hh < A.grp; hh++) {
    const int h = hq * A.grp + hh;
    const float* const tab = (const float*)(A.ws + key_bytes<Y>(A) + (j * A.H + h) * Y::head + Y::offTab);
    const long long jh = j * A.H + h;
    // opaque per head: the addresses and predicates made from them are not kept across heads, where
    // they would spill
    asm("" : "+v"(tid));
    lane = tid & 63;
    c16 = lane & 15;
    g = lane >> 4;
    row = tid / TPR;
    __syncthreads();
    if (tid < 64) {
      const long long th = (at.t0 + (long long)(tid < at.len ? tid : 0)) * A.H + h;
      sm.al[tid] = tid < at.len ? A.alpha[th] : 1.0f;
      sm.be[tid] = tid < at.len ? A.beta[th] : 0.0f;
    }
    const long long tok = at.t0 + (long long)row;
    rows_in<D, DT, DT, NPI, TPR>(tid, B.d_out, tok * A.os + (long long)h * D, row < at.len, sm.in.O, sm.isO, nullptr, 0, nullptr);
    rows_in<D, DT, kF32, 2, TPR>(tid, keep.Y, (jh * 64 + row) * D, row < at.len, sm.in.Y, sm.isY, A.v, tok * A.vs + (long long)h * D, sm.yv);
    rows_in<D, DT, kF32, 2, TPR>(tid, keep.W, (jh * 64 + row) * D, row < at.len, sm.in.W, sm.isW, nullptr, 0, nullptr);
    ahead();
    __syncthreads();
    // products with the states: this wave's 16 rows of S0, then of dS1, as column operands
    {
      h8 Sh[KS], Sl[KS], Gh[KS], Gl[KS];
      float iS, iG;
      {
        float x[KS][8], m = 0.0f, cn = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ks++) load8<kF32>(keep.S, (jh * D + dk) * D + 32 * ks + 8 * g, x[ks]);
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
          for (int e = 0; e < 8; e++) m = fmaxf(m, fabsf(x[ks][e]));
        float s = scale_of(col_max(m), iS);
#pragma unroll
        for (int ks = 0; ks < KS; ks++) split8<2>(x[ks], s, Sh[ks], Sl[ks]);
        ahead();
#pragma unroll
        for (int ks = 0; ks < KS; ks++) load8<kF32>(keep.G, (jh * D + dk) * D + 32 * ks + 8 * g, x[ks]);
        m = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
          for (int e = 0; e < 8; e++) {
            m = fmaxf(m, fabsf(x[ks][e]));
            cn = fmaf(x[ks][e], (float)Sh[ks][e] + (float)Sl[ks][e], cn);
          }
        cn = sum_rows(sum16(cn * iS));
        if (lane == 0) sm.corner[w] = cn;
        s = scale_of(col_max(m), iG);
#pragma unroll
        for (int ks = 0; ks < KS; ks++) split8<2>(x[ks], s, Gh[ks], Gl[ks]);
      }
      ahead();
#pragma unroll
      for (int rt = 0; rt < 4; rt++) {
        f4 e1 = zero, e2 = zero, e3 = zero;
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
          const int r = 16 * rt + c16, k = 32 * ks + 8 * g;
          const h8 o = *(const h8*)&sm.in.O[0][r][k];
          const h8 yh = *(const h8*)&sm.in.Y[0][r][k], yl = *(const h8*)&sm.in.Y[1][r][k];
          const h8 wh = *(const h8*)&sm.in.W[0][r][k], wl = *(const h8*)&sm.in.W[1][r][k];
          e1 = mfma(o, Sh[ks], e1);
          e2 = mfma(yh, Sh[ks], e2);
          e3 = mfma(wh, Gh[ks], e3);
          e1 = mfma(o, Sl[ks], e1);
          e2 = mfma(yh, Sl[ks], e2);
          e3 = mfma(wh, Gl[ks], e3);
          if constexpr (NPI == 2) e1 = mfma(*(const h8*)&sm.in.O[1][r][k], Sh[ks], e1);
          e2 = mfma(yl, Sh[ks], e2);
          e3 = mfma(wl, Gh[ks], e3);
        }
        const int t0 = 16 * rt + 4 * g;
        const f4 io = *(const f4*)&sm.isO[t0], iy = *(const f4*)&sm.isY[t0], iw = *(const f4*)&sm.isW[t0];
        const f4 G = *(const f4*)&tab[kTabG + t0], lc = *(const f4*)&tab[kTabL + t0], be = *(const f4*)&sm.be[t0];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float a = e1[i] * (io[i] * iS), b = e2[i] * (iy[i] * iS), c = e3[i] * (iw[i] * iG);
          dQ[rt][i] = fmaf(G[i], a, dQ[rt][i]);
          dK[rt][i] = fmaf(-G[i] * be[i], b, fmaf(lc[i], c, dK[rt][i]));
          const float zq = sum16(qv[rt][i] * a), zk = sum16(kv[rt][i] * b), yk = sum16(kv[rt][i] * c);
          if (c16 == 0) {
            sm.dot[0][w][t0 + i] = zq;
            sm.dot[1][w][t0 + i] = zk;
            sm.dot[2][w][t0 + i] = yk;
          }
        }
        ahead();
      }
    }
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
            x = p * qk[n][i];
            if (s < t) {
              const float y = dx[n][i] * (sm.isY[t] * sm.isW[s]), b = sm.be[t] * y;
              zv = -b * l;
              x = fmaf(-b, kk[n][i], x);
              rx[i] = fmaf(y, l * kk[n][i], rx[i]);
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
    // gates: dalpha_r = sum over t >= r of L[t,r] F_r[t] with F_r[t] = sum over s < r of x[t,s] L[r-1,s]
    // (the state before the chunk as s = -1, the state behind it as one more t).  Lane t; a wave takes
    // 64 / NW gates: F at its first by a sum, then F_{r+1} = a_r F_r + x[t,r].
    {
      constexpr int RW = 64 / NW;
      const int r0 = RW * w;
      float F = sm.z[lane], C = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; v++) C += sm.corner[v];
      if (w) {
        const float* const lr = sm.m.L[r0 - 1];
        const float G = sm.al[0] * lr[0];
        const float y = lane < r0 ? sm.y[lane] * lr[lane] : 0.0f;
        C = fmaf(C, G, sum_rows(sum16(y)));
        float f0 = F * G, f1 = 0.0f;
#pragma unroll 8
        for (int s = 0; s < r0; s += 2) {
          f0 = fmaf(lr[s], sm.m.xT[s][lane], f0);
          f1 = fmaf(lr[s + 1], sm.m.xT[s + 1][lane], f1);
        }
        F = f0 + f1;
      }
#pragma unroll
      for (int i = 0; i < RW; i++) {
        const int r = r0 + i;
        const float v = sum_rows(sum16(lane >= r ? sm.m.L[lane][r] * F : 0.0f));
        if (lane == 0) sm.da[r] = fmaf(sm.m.L[63][r], C, v);
        F = fmaf(sm.al[r], F, sm.m.xT[r][lane]);
        C = fmaf(sm.al[r], C, sm.y[r]);
      }
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
    if (tid < at.len) {
      const long long th = (at.t0 + (long long)tid) * A.H + h;
      B.dalpha[th] = sm.da[tid];
      B.dbeta[th] = sm.yv[tid] - (sm.rowx[0][tid] + (NW == 8 ? sm.rowx[1][tid] : 0.0f));
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
  const dim3 slots((unsigned)chunk_slots(a.T, a.N), a.Hq), tiles((unsigned)((long long)a.N * a.H));
  unsigned* const status = a.status;
  a.status = nullptr;  // reported once, by the reverse pass
  if (a.T > 0) {
    hipLaunchKernelGGL((k_chunk_prep<D, DT, LayB<D, DT>>), slots, dim3(256), 0, s, a);
    hipLaunchKernelGGL((k_chunk_state<D, DT, D / 16, LayB<D, DT>>), tiles, dim3(4 * D), 0, s, a, keep.S, keep.W);
  }
  a.status = status;
  hipLaunchKernelGGL((k_chunk_reverse<D, DT, D / 16>), tiles, dim3(4 * D), 0, s, b, keep);
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
