// stepq_chunk_kernels.h -- kernels that the chunked forward pass and its gradient share: the chunks'
// local matrices (k_chunk_prep) and the pass over the chunks (k_chunk_state).
#pragma once
#include "stepq_chunk.h"

namespace stepq {
namespace dlt {

constexpr int kPitch = 68;  // floats of a row of the 64 x 64 matrices in LDS

// ---------------------------------------------------------------------------------------------
// local matrices
// ---------------------------------------------------------------------------------------------

template <int D, int DT>
struct PrepSmem {
  static constexpr int NPI = kInPlanes<DT>, KP = D + 8;  // 16-byte aligned rows, 4 banks apart
  union {
    struct {
      _Float16 K[NPI][64][KP], Q[NPI][64][KP];
    } in;
    struct {
      float L[64][kPitch], A[64][kPitch], P[64][kPitch];  // L becomes T once A and P are formed
    } m;
  };
  float isk[64], isq[64], al[64], be[64], sT[64], sP[64], sU[64];
};

// Rows of q or k (tokens behind the end repeat the last one: their W is zero) as scaled planes.
template <int D, int DT>
__device__ __forceinline__ void load_rows(const void* src, long long stride, long long head, int t0,
                                          int len, _Float16 (*dst)[64][D + 8], float* is) {
  constexpr int E = D / 4;
  const int row = threadIdx.x >> 2, part = threadIdx.x & 3;
  const long long at = (t0 + (long long)(row < len ? row : len - 1)) * stride + head + part * E;
  float x[E];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < E; i += 8) {
    load8<DT>(src, at + i, x + i);
#pragma unroll
    for (int j = 0; j < 8; j++) m = fmaxf(m, fabsf(x[i + j]));
  }
  m = fmaxf(m, __shfl_xor(m, 1));
  m = fmaxf(m, __shfl_xor(m, 2));
  float inv;
  const float s = scale_of(m, inv);
  if (part == 0) is[row] = inv;
#pragma unroll
  for (int i = 0; i < E; i += 8) {
    h8 hi, lo;
    split8<kInPlanes<DT>>(x + i, s, hi, lo);
    *(h8*)&dst[0][row][part * E + i] = hi;
    if constexpr (kInPlanes<DT> == 2) *(h8*)&dst[1][row][part * E + i] = lo;
  }
}

// T = (I + A)^-1 in place of X: 16 x 16 diagonal blocks by forward substitution (a wave each, a column a
// lane), then X21 = -X22 (A21 X11) for 16- and 32-row halves on binary32 matrix instructions.
__device__ __forceinline__ void invert(const float (*A)[kPitch], float (*X)[kPitch], int w, int lane) {
  const int c = lane & 15, g = lane >> 4;
  if (lane < 16) {
    float x[16];
#pragma unroll
    for (int t = 0; t < 16; t++) {
      float acc = t == c ? 1.0f : 0.0f;
#pragma unroll
      for (int s = 0; s < t; s++) acc = fmaf(-A[16 * w + t][16 * w + s], x[s], acc);
      x[t] = acc;
    }
#pragma unroll
    for (int t = 0; t < 16; t++) X[16 * w + t][16 * w + c] = x[t];
  } else if (lane < 32 && !(w & 1)) {  // the block right of an even diagonal block
#pragma unroll
    for (int t = 0; t < 16; t++) X[16 * w + t][16 * w + 16 + c] = 0.0f;
  }
  __syncthreads();
  auto dot = [&](const float (*M)[kPitch], int r, int m, const float (*B)[kPitch], int cb, f4 y) {
#pragma unroll
    for (int kk = 0; kk < 4; kk++)
      y = __builtin_amdgcn_mfma_f32_16x16x4f32(M[16 * r + c][16 * m + 4 * kk + g],
                                               B[16 * m + 4 * kk + g][16 * cb + c], y, 0, 0, 0);
    return y;
  };
  auto dot_acc = [&](int r, int m, f4 y, f4 x) {  // x += X[r][m] y, y an accumulator tile
#pragma unroll
    for (int kk = 0; kk < 4; kk++)
      x = __builtin_amdgcn_mfma_f32_16x16x4f32(X[16 * r + c][16 * m + 4 * g + kk], y[kk], x, 0, 0, 0);
    return x;
  };
  const f4 zero = {0, 0, 0, 0};
  if (w < 2) {
    const int r = 2 * w + 1;
    const f4 y = dot(A, r, r - 1, X, r - 1, zero);
    const f4 x = dot_acc(r, r, y, zero);
#pragma unroll
    for (int i = 0; i < 4; i++) X[16 * r + 4 * g + i][16 * (r - 1) + c] = -x[i];
  }
  __syncthreads();
  {
    const int cb = w & 1, r = 2 + (w >> 1);
    auto half = [&](int row) {
      f4 y = zero;
      for (int m = cb; m < 2; m++) y = dot(A, row, m, X, cb, y);
      return y;
    };
    f4 x = dot_acc(r, 2, half(2), zero);
    if (r == 3) x = dot_acc(3, 3, half(3), x);
#pragma unroll
    for (int i = 0; i < 4; i++) X[16 * r + 4 * g + i][16 * cb + c] = -x[i];
  }
  __syncthreads();
}

// Y: the workspace's layout (LayF, or LayB: with the gradient's extra pieces).
template <int D, int DT, class Y>
__global__ __launch_bounds__(256) void k_chunk_prep(SeqArgs A) {
  constexpr int KS = D / 32, NPI = Y::NPI, NPO = Y::NPO;
  __shared__ PrepSmem<D, DT> sm;
  const long long j = blockIdx.x;
  const int hq = blockIdx.y;
  ChunkAt at;
  if (!chunk_at(A, j, at)) return;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  load_rows<D, DT>(A.k, A.ks, (long long)hq * D, at.t0, at.len, sm.in.K, sm.isk);
  load_rows<D, DT>(A.q, A.qs, (long long)hq * D, at.t0, at.len, sm.in.Q, sm.isq);
  __syncthreads();
  // fragments of K, Q (rows = tokens) and K^T (rows = key dimensions)
  char* const key = A.ws + (j * A.Hq + hq) * Y::key;
  for (int f = w; f < Y::NF; f += 4) {
    const int rt = f / KS, ks = f - rt * KS;
    const int row = 32 * (rt >> 1) + perm_row(c16, rt & 1), col = 32 * ks + 8 * g;
    const int kr = 32 * (f >> 2) + perm_row(c16, (f >> 1) & 1), kc = 32 * (f & 1) + 8 * g;
#pragma unroll
    for (int p = 0; p < NPI; p++) {
      const int o = (p * Y::NF + f) * kFrag + lane * 16;
      *(h8*)(key + Y::offK + o) = *(const h8*)&sm.in.K[p][row][col];
      h8 t;
#pragma unroll
      for (int i = 0; i < 8; i++) t[i] = sm.in.K[p][kc + i][kr];
      *(h8*)(key + Y::offKT + o) = t;
      if constexpr (Y::grad) {
#pragma unroll
        for (int i = 0; i < 8; i++) t[i] = sm.in.Q[p][kc + i][kr];
        *(h8*)(key + Y::offQ + o) = t;
      } else {
        *(h8*)(key + Y::offQ + o) = *(const h8*)&sm.in.Q[p][row][col];
      }
    }
  }
  // K K^T and Q K^T, row tile w (plain row order), lower tiles only
  f4 kk[4], qk[4];
#pragma unroll
  for (int c = 0; c < 4; c++) {
    kk[c] = qk[c] = f4{0, 0, 0, 0};
    if (c > w) continue;
#pragma unroll
    for (int ks = 0; ks < KS; ks++) {
      h8 a[NPI], q[NPI], b[NPI];
#pragma unroll
      for (int p = 0; p < NPI; p++) {
        a[p] = *(const h8*)&sm.in.K[p][16 * w + c16][32 * ks + 8 * g];
        q[p] = *(const h8*)&sm.in.Q[p][16 * w + c16][32 * ks + 8 * g];
        b[p] = *(const h8*)&sm.in.K[p][16 * c + c16][32 * ks + 8 * g];
      }
      kk[c] = mfma(a[0], b[0], kk[c]);
      qk[c] = mfma(q[0], b[0], qk[c]);
      if constexpr (NPI == 2) {
        kk[c] = mfma(a[0], b[1], mfma(a[1], b[0], kk[c]));
        qk[c] = mfma(q[0], b[1], mfma(q[1], b[0], qk[c]));
      }
    }
  }
  if constexpr (Y::grad) {
#pragma unroll
    for (int c = 0; c < 4; c++) {
      if (c > w) continue;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int t = 16 * w + 4 * g + i, s = 16 * c + c16;
        ((float*)(key + Y::offKK))[t * 64 + s] = kk[c][i] * (sm.isk[t] * sm.isk[s]);
        ((float*)(key + Y::offQK))[t * 64 + s] = qk[c][i] * (sm.isq[t] * sm.isk[s]);
      }
    }
  }
  for (int hh = 0; hh < A.grp; hh++) {
    const int h = hq * A.grp + hh;
    char* const head = A.ws + key_bytes<Y>(A) + (j * A.H + h) * Y::head;
    float* const tab = (float*)(head + Y::offTab);
    __syncthreads();  // the operand planes (first head) or the last head's matrices are free
    if (tid < 64) {
      const long long th = (at.t0 + (long long)(tid < at.len ? tid : 0)) * A.H + h;
      sm.al[tid] = tid < at.len ? A.alpha[th] : 1.0f;
      sm.be[tid] = tid < at.len ? A.beta[th] : 0.0f;
    }
    __syncthreads();
    // L[t][s], rows 16 w .. 16 w + 15, column s = lane: a running product down the column
    {
      int ln = lane;  // opaque: the 64 comparisons are not kept in scalar registers across heads
      asm("" : "+v"(ln));
      float l = 1.0f;
      for (int t = 0; t < 16 * w; t++) l = t > ln ? l * sm.al[t] : 1.0f;
#pragma unroll
      for (int i = 0; i < 16; i++) {
        const int t = 16 * w + i;
        l = t > ln ? l * sm.al[t] : 1.0f;
        sm.m.L[t][ln] = t >= ln ? l : 0.0f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; c++) {
      const int s = 16 * c + c16;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int t = 16 * w + 4 * g + i;
        float a = 0.0f, p = 0.0f;
        if (s <= t) {
          const float l = sm.m.L[t][s] * sm.isk[s];
          p = qk[c][i] * sm.isq[t] * l;
          if (s < t) a = sm.be[t] * (kk[c][i] * sm.isk[t] * l);
        }
        sm.m.A[t][s] = a;
        sm.m.P[t][s] = p;
      }
    }
    if (tid < 64) {
      const float G = sm.al[0] * sm.m.L[tid][0];
      tab[kTabU + tid] = sm.be[tid] * G * sm.isk[tid];
      tab[kTabB + tid] = sm.be[tid];
      tab[kTabQ + tid] = G * sm.isq[tid];
      tab[kTabD + tid] = sm.m.L[63][tid] * sm.isk[tid];
      tab[kTabG + tid] = G;
      if constexpr (Y::grad) {
        tab[kTabL + tid] = sm.m.L[63][tid];
        tab[kTabIK + tid] = sm.isk[tid];
        tab[kTabIQ + tid] = sm.isq[tid];
      }
    }
    __syncthreads();
    float(*const X)[kPitch] = sm.m.L;
    invert(sm.m.A, X, w, lane);
    // row scales of T and P (gradient: of T, and of the columns of T and P)
    {
      const int row = tid >> 2, part = tid & 3;
      float mt = 0.0f, mp = 0.0f, mu = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        if (row >= 32 || part < 2) {
          const f4 x = *(const f4*)&X[row][16 * part + i], p = *(const f4*)&sm.m.P[row][16 * part + i];
#pragma unroll
          for (int e = 0; e < 4; e++) mt = fmaxf(mt, fabsf(x[e])), mp = fmaxf(mp, fabsf(p[e]));
        }
      }
      if constexpr (Y::grad) {
        mp = 0.0f;
        if (row < 32 || part >= 2)
#pragma unroll
          for (int i = 0; i < 16; i++) {
            mu = fmaxf(mu, fabsf(X[16 * part + i][row]));
            mp = fmaxf(mp, fabsf(sm.m.P[16 * part + i][row]));
          }
        mu = fmaxf(mu, __shfl_xor(mu, 1));
        mu = fmaxf(mu, __shfl_xor(mu, 2));
      }
      mt = fmaxf(mt, __shfl_xor(mt, 1));
      mt = fmaxf(mt, __shfl_xor(mt, 2));
      mp = fmaxf(mp, __shfl_xor(mp, 1));
      mp = fmaxf(mp, __shfl_xor(mp, 2));
      if (part == 0) {
        float it, ip;
        sm.sT[row] = scale_of(mt, it);
        sm.sP[row] = scale_of(mp, ip);
        tab[kTabT + row] = it;
        tab[kTabP + row] = ip;
        if constexpr (Y::grad) {
          sm.sU[row] = scale_of(mu, it);
          tab[kTabTt + row] = it;
        }
      }
    }
    __syncthreads();
    // 6 fragments each of T and P: three a wave; gradient: T, T^T and P^T, 18 over the waves
    if constexpr (!Y::grad) {
#pragma unroll
      for (int n = 0; n < 3; n++) {
        const int f = 3 * (w & 1) + n;
        const int rt = f < 2 ? f : 2 + ((f - 2) >> 1), ks = f < 2 ? 0 : (f - 2) & 1;
        const int row = 32 * (rt >> 1) + perm_row(c16, rt & 1), col = 32 * ks + 8 * g;
        const float* src = w < 2 ? &X[row][col] : &sm.m.P[row][col];
        const f4 x0 = *(const f4*)src, x1 = *(const f4*)(src + 4);
        const float x[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
        h8 hi, lo;
        split8<2>(x, w < 2 ? sm.sT[row] : sm.sP[row], hi, lo);
        char* const dst = head + (w < 2 ? Y::offT : Y::offP) + f * kFrag + lane * 16;
        *(h8*)dst = hi;
        if (w < 2 || NPO == 2) *(h8*)(dst + kTri * kFrag) = lo;
      }
    } else {
      for (int n = w; n < 18; n += 4) {
        const int m = n / 6, f = n - 6 * m;  // 0 T, 1 T^T, 2 P^T
        const int rt = m ? (f < 4 ? f >> 1 : f - 2) : (f < 2 ? f : 2 + ((f - 2) >> 1));
        const int ks = m ? (f < 4 ? f & 1 : 1) : (f < 2 ? 0 : (f - 2) & 1);
        const int row = 32 * (rt >> 1) + perm_row(c16, rt & 1), col = 32 * ks + 8 * g;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = m == 0 ? X[row][col + i] : m == 1 ? X[col + i][row] : sm.m.P[col + i][row];
        h8 hi, lo;
        split8<2>(x, m == 0 ? sm.sT[row] : m == 1 ? sm.sU[row] : sm.sP[row], hi, lo);
        char* const dst = head + (2 * m * kTri + f) * kFrag + lane * 16;
        *(h8*)dst = hi;
        *(h8*)(dst + kTri * kFrag) = lo;
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// the pass over the chunks
// ---------------------------------------------------------------------------------------------

// A wave owns 16 CT columns of one (sequence, head) state for the whole sequence: lane l holds columns
// CT (l & 15) .. + CT - 1 (column tile ct = column CT (l & 15) + ct), rows in accumulator order.  All
// waves of a workgroup read the same fragments, staged in LDS once a chunk.
// For the gradient (LayB) nothing is read out: the states before every chunk and W are kept.
template <int D, int DT, int CT, int NW, class Y>
__global__ __launch_bounds__(64 * NW) void k_chunk_state(SeqArgs A, float* keepS, float* keepW) {
  constexpr int KS = D / 32, NPI = Y::NPI, NPO = Y::NPO, NB = D / 32;
  // staged: K, K^T (and Q), then T (and P), then the tables
  constexpr int keyN = Y::grad ? Y::offQ : Y::key, triN = Y::grad ? Y::offTt : Y::offTab;
  constexpr int offT = keyN, offP = keyN + Y::offP, offTab = keyN + triN;
  constexpr int part = offTab + 2048;
  constexpr int NBUF = 2 * part <= 160 * 1024 ? 2 : 1;  // binary32 inputs have room for one
  __shared__ __attribute__((aligned(16))) char buf[NBUF * part];
  const long long tile = blockIdx.x;
  const int s = (int)(tile / A.H), h = (int)(tile - (long long)s * A.H);
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  int t0, t1;
  const bool valid = seq_range(A, s, t0, t1);
  const int slot = seq_slot(A, s, valid, h == 0 && blockIdx.y == 0 && tid == 0);
  if (slot < 0) return;
  if (t0 == t1 && (Y::grad || !A.S_out || A.S_out == A.S_in)) return;
  const int col = 16 * CT * ((int)blockIdx.y * NW + w) + CT * c16;
  const long long so = ((long long)slot * A.H + h) * D * D + col;
  f4 S[CT][2 * NB];
#pragma unroll
  for (int rt = 0; rt < 2 * NB; rt++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      float x[CT] = {};
      if (A.S_in) loadn<kF32, CT>(A.S_in, so + (long long)(32 * (rt >> 1) + 8 * g + 4 * (rt & 1) + i) * D, x);
#pragma unroll
      for (int ct = 0; ct < CT; ct++) S[ct][rt][i] = x[ct];
    }
  const long long j0 = first_slot(A, s);
  const char* const heads = A.ws + key_bytes<Y>(A);
  const int hq = h / A.grp;
  const int nc = (t1 - t0 + kChunk - 1) / kChunk;
  // chunk c's pieces on their way into LDS, 1 KiB a wave at a time
  const unsigned lds0 = lds_offset(buf), lane16 = 16 * lane;
  auto fetch = [&](int c) {
    const char* const key = A.ws + ((j0 + c) * A.Hq + hq) * Y::key;
    const char* const head = heads + ((j0 + c) * A.H + h) * Y::head;
    const unsigned at = lds0 + (NBUF == 2 ? (c & 1) * part : 0);
    copy_block<NW>(key, at, keyN, w, lane16);
    if constexpr (Y::grad) {
      copy_block<NW>(head, at + offT, triN, w, lane16);
      copy_block<NW>(head + Y::offTab, at + offTab, 2048, w, lane16);
    } else {
      copy_block<NW>(head, at + offT, Y::head, w, lane16);
    }
  };
  // V of chunk c in accumulator order
  Raw<DT, CT> v[4][4];
  auto fetch_v = [&](int c) {
    const int tc = t0 + c * kChunk;
    rows_acc<DT, CT>((const char*)A.v + (tc * A.vs + (long long)h * D) * (DT == kF32 ? 4 : 2), (int)A.vs, t1 - tc, col, g, v);
  };
  if (nc) {
    fetch(0);
    fetch_v(0);
  }
  for (int c = 0; c < nc; c++) {
    const char* const lds = buf + (NBUF == 2 ? (c & 1) * part : 0);
    const int tc = t0 + c * kChunk, len = t1 - tc < kChunk ? t1 - tc : kChunk;
    wait_copies();
    __syncthreads();  // chunk c is there, and every wave is done with chunk c - 1
    f4 R[CT][4];
#pragma unroll
    for (int rt = 0; rt < 4; rt++)
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int ct = 0; ct < CT; ct++)
          R[ct][rt][i] = 32 * (rt >> 1) + 8 * g + 4 * (rt & 1) + i < len ? raw_value<DT, CT>(v[rt][i], ct) : 0.0f;
    if (c + 1 < nc) {
      if (NBUF == 2) fetch(c + 1);
      fetch_v(c + 1);
    }
    if constexpr (Y::grad) {
      float* const dst = keepS + ((j0 + c) * A.H + h) * D * D + col;
#pragma unroll
      for (int rt = 0; rt < 2 * NB; rt++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          float x[CT];
#pragma unroll
          for (int ct = 0; ct < CT; ct++) x[ct] = S[ct][rt][i];
          storen<kF32, CT>(dst, (long long)(32 * (rt >> 1) + 8 * g + 4 * (rt & 1) + i) * D, x);
        }
    }
    const float* const tab = (const float*)(lds + offTab);
    auto frag = [&](int off, int n, int p, int f) { return *(const h8*)(lds + off + (p * n + f) * kFrag + lane * 16); };
    auto rows = [&](int t, int rt) { return *(const f4*)(tab + t + 32 * (rt >> 1) + 8 * g + 4 * (rt & 1)); };
    // Every product's fragments are read while its other operand is formed.
    h8 f[Y::NF], fl[NPI == 2 ? Y::NF : 1];
    auto read = [&](int off) {
#pragma unroll
      for (int n = 0; n < Y::NF; n++) {
        f[n] = frag(off, Y::NF, 0, n);
        if constexpr (NPI == 2) fl[n] = frag(off, Y::NF, 1, n);
      }
    };
    h8 Sh[CT][NB], Sl[CT][NB], xh[CT][2], xl[CT][2];
    float iS[CT], ix[CT];
    read(Y::offK);
    ahead();
#pragma unroll
    for (int ct = 0; ct < CT; ct++) iS[ct] = to_operand<NB, 2>(S[ct], Sh[ct], Sl[ct]);
    // R = beta V - beta G K S0
    f4 z[CT][2 * NB > 4 ? 2 * NB : 4];
    auto times_state = [&](bool low) {
#pragma unroll
      for (int rt = 0; rt < 4; rt++) {
#pragma unroll
        for (int ct = 0; ct < CT; ct++) z[ct][rt] = f4{0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
          for (int ct = 0; ct < CT; ct++) {
            z[ct][rt] = mfma(f[rt * KS + ks], Sh[ct][ks], z[ct][rt]);
            if (low) z[ct][rt] = mfma(f[rt * KS + ks], Sl[ct][ks], z[ct][rt]);
            if constexpr (NPI == 2) z[ct][rt] = mfma(fl[rt * KS + ks], Sh[ct][ks], z[ct][rt]);
          }
      }
    };
    times_state(true);
    ahead();
    h8 ft[2][kTri];
#pragma unroll
    for (int n = 0; n < kTri; n++) {
      ft[0][n] = frag(offT, kTri, 0, n);
      ft[1][n] = frag(offT, kTri, 1, n);
    }
    ahead();
#pragma unroll
    for (int ct = 0; ct < CT; ct++) {
#pragma unroll
      for (int rt = 0; rt < 4; rt++) {
        const f4 cu = rows(kTabU, rt), be = rows(kTabB, rt);
#pragma unroll
        for (int i = 0; i < 4; i++) R[ct][rt][i] = fmaf(-cu[i] * iS[ct], z[ct][rt][i], be[i] * R[ct][rt][i]);
      }
      ix[ct] = to_operand<2, 2>(R[ct], xh[ct], xl[ct]);
    }
    // W = T R (in R's place)
#pragma unroll
    for (int rt = 0; rt < 4; rt++)
#pragma unroll
      for (int ct = 0; ct < CT; ct++) {
        z[ct][rt] = f4{0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks <= rt >> 1; ks++) {
          const int n = tri_frag(rt, ks);
          z[ct][rt] = mfma(ft[1][n], xh[ct][ks], mfma(ft[0][n], xl[ct][ks], mfma(ft[0][n], xh[ct][ks], z[ct][rt])));
        }
      }
    ahead();
    if constexpr (!Y::grad) read(Y::offQ);
    else read(Y::offKT);
    ahead();
#pragma unroll
    for (int rt = 0; rt < 4; rt++) {
      const f4 it = rows(kTabT, rt);
#pragma unroll
      for (int ct = 0; ct < CT; ct++)
#pragma unroll
        for (int i = 0; i < 4; i++) R[ct][rt][i] = z[ct][rt][i] * (it[i] * ix[ct]);
    }
    if constexpr (Y::grad) {
      float* const dst = keepW + ((j0 + c) * A.H + h) * 64 * D + col;
#pragma unroll
      for (int rt = 0; rt < 4; rt++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          float x[CT];
#pragma unroll
          for (int ct = 0; ct < CT; ct++) x[ct] = R[ct][rt][i];
          storen<kF32, CT>(dst, (long long)(32 * (rt >> 1) + 8 * g + 4 * (rt & 1) + i) * D, x);
        }
    } else {
      // O = G Q S0 + P W
#pragma unroll
      for (int ct = 0; ct < CT; ct++) ix[ct] = to_operand<2, NPO>(R[ct], xh[ct], xl[ct]);
      times_state(NPO == 2);
      ahead();
      h8 fp[NPO][kTri];
#pragma unroll
      for (int p = 0; p < NPO; p++)
#pragma unroll
        for (int n = 0; n < kTri; n++) fp[p][n] = frag(offP, kTri, p, n);
      ahead();
      float o[4][4][CT];
#pragma unroll
      for (int rt = 0; rt < 4; rt++) {
        f4 y[CT] = {};
#pragma unroll
        for (int ks = 0; ks <= rt >> 1; ks++) {
          const int n = tri_frag(rt, ks);
#pragma unroll
          for (int ct = 0; ct < CT; ct++) {
            y[ct] = mfma(fp[0][n], xh[ct][ks], y[ct]);
            if constexpr (NPO == 2) y[ct] = mfma(fp[NPO - 1][n], xh[ct][ks], mfma(fp[0][n], xl[ct][ks], y[ct]));
          }
        }
        const f4 cq = rows(kTabQ, rt), ip = rows(kTabP, rt);
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int ct = 0; ct < CT; ct++) o[rt][i][ct] = fmaf(cq[i] * iS[ct], z[ct][rt][i], (ip[i] * ix[ct]) * y[ct][i]);
      }
      ahead();
      read(Y::offKT);
      ahead();
      rows_store<DT, CT>((char*)A.out + (tc * A.os + (long long)h * D) * (DT == kF32 ? 4 : 2), (int)A.os, len, col, g, o);
    }
    // S1 = G_C S0 + K^T diag(L[C, .]) W
#pragma unroll
    for (int ct = 0; ct < CT; ct++) {
#pragma unroll
      for (int rt = 0; rt < 4; rt++) R[ct][rt] *= rows(kTabD, rt);
      ix[ct] = to_operand<2, 2>(R[ct], xh[ct], xl[ct]);
    }
    const float G = tab[kTabG + 63];
#pragma unroll
    for (int rt = 0; rt < 2 * NB; rt++)
#pragma unroll
      for (int ct = 0; ct < CT; ct++) {
        f4 y = {0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < 2; ks++) {
          y = mfma(f[2 * rt + ks], xl[ct][ks], mfma(f[2 * rt + ks], xh[ct][ks], y));
          if constexpr (NPI == 2) y = mfma(fl[2 * rt + ks], xh[ct][ks], y);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) S[ct][rt][i] = fmaf(G, S[ct][rt][i], ix[ct] * y[i]);
      }
    if (NBUF == 1 && c + 1 < nc) {
      __syncthreads();
      fetch(c + 1);
    }
  }
  if (!Y::grad && A.S_out) {
#pragma unroll
    for (int rt = 0; rt < 2 * NB; rt++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float x[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ct++) x[ct] = S[ct][rt][i];
        storen<kF32, CT>(A.S_out, so + (long long)(32 * (rt >> 1) + 8 * g + 4 * (rt & 1) + i) * D, x);
      }
  }
}

}  // namespace dlt
}  // namespace stepq
