// stepq_chunk_kernels.h -- kernels that the chunked forward pass and its gradient share: the chunks'
// local matrices (k_chunk_prep) and the pass over the chunks (k_chunk_state).
#pragma once
#include <type_traits>

#include "stepq_chunk.h"

namespace stepq {
namespace dlt {

// 64 rows of N elements in LDS, 16 bytes and, from row to row of 16, 64 bytes apart: the rows of an operand
// (perm_row) and of K^T's columns are on different banks.
template <class T, int N>
struct LdsRows {
  static constexpr int pad = 16 / (int)sizeof(T), pitch = N + pad;
  T x[64 * pitch + 3 * 4 * pad];
  __device__ T* operator[](int r) { return x + r * pitch + (r >> 4) * 4 * pad; }
};
using Square = LdsRows<float, 64>;

// ---------------------------------------------------------------------------------------------
// local matrices
// ---------------------------------------------------------------------------------------------

// One workgroup per (chunk, key head): K and Q once, then the value heads that share them.  Wave w owns the 16
// tokens of row tile w (32 (w >> 1) + perm(lane & 15, w & 1)) as columns of K K^T and K Q^T: with K's row
// tiles as the A side the accumulators of a pair hold 8 consecutive tokens s of a lane's token t, which is
// P's fragment as it is and two 16-byte stores of A.  (The gradient wants P^T: Q on the A side, s as columns.)
//
// 16,381 tokens x 48 heads on 16 key heads (d = 128 bf16): 163 us for 105 MB read and 446 MB written, 3.4 TB/s of the
// 5.2 that a copy reaches; 8,192 tokens x 32 heads on 16 for the gradient 100 us.  Three workgroups a CU wait for
// each other's memory most of the time (56% of wave cycles); the vector ALUs are busy 40%, LDS 35%.
// A fourth workgroup would spill (188 us).
//
// Products of gates between two tokens come from running products inside groups of 8 and blocks of 32:
//   L[t,s] = pre32[t] suf32[s] across blocks, pre8[t] mid suf8[s] across groups of a block,
// pre = from the group's start to t, suf = behind s to the group's end; inside a group one by one.
template <int D, int DT, bool QT>
struct alignas(16) PrepSmem {
  static constexpr int NPI = kInPlanes<DT>;
  union {
    struct {
      LdsRows<_Float16, D> K[NPI], Q[QT ? NPI : 1];
    };
    struct {               // of two heads
      Square X[2];         // A, then T but for its lower left quarter
      float Z[2][32][36];  // T's lower left quarter
    };
  };
  float gate[2][5][64];  // a, pre8, suf8, pre32, suf32; every wave writes the same values for itself
  float isk[64], isq[64], be[2][64], most[2][6];
};

// The wave's 16 rows of q or k as scaled planes (a lane: row `row`, elements 32 ks + 8 g ..); returns the
// inverse scale.
template <int D, int DT>
__device__ __forceinline__ float load_rows(const void* src, long long at, int g, h8 (*f)[kInPlanes<DT>]) {
  constexpr int KS = D / 32, NPI = kInPlanes<DT>;
  float x[KS][8], m = 0.0f;
#pragma unroll
  for (int ks = 0; ks < KS; ks++) load8<DT>(src, at + 32 * ks + 8 * g, x[ks]);
#pragma unroll
  for (int ks = 0; ks < KS; ks++)
#pragma unroll
    for (int e = 0; e < 8; e++) m = fmaxf(m, fabsf(x[ks][e]));
  float inv;
  const float s = scale_of(col_max(m), inv);
#pragma unroll
  for (int ks = 0; ks < KS; ks++) {
    h8 lo;
    split8<NPI>(x[ks], s, f[ks][0], lo);
    if constexpr (NPI == 2) f[ks][1] = lo;
  }
  return inv;
}

// Inverses of the two 32 x 32 diagonal blocks I + A (strictly lower A in X), one wave each: the 16 x 16
// blocks by forward substitution (a column a lane, both blocks at once), then X10 = -X11 (A10 X00) on
// binary32 matrix instructions.  Substitution, not a power series: keys that repeat make A's powers large.
// Returns the largest magnitude written, columns times be.
__device__ __forceinline__ float invert_block(Square& X, const float* be, int r0, int lane) {
  const int c = lane & 15, g = lane >> 4;
  float m = 0.0f;
  if (lane < 32) {
    const int b = r0 + 16 * g;
    float x[16];
#pragma unroll
    for (int t = 0; t < 16; t++) {
      float acc = t == c ? 1.0f : 0.0f;
#pragma unroll
      for (int s = 0; s < t; s += 4) {
        const f4 a = *(const f4*)&X[b + t][b + s];
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (s + i < t) acc = fmaf(-a[i], x[s + i], acc);
      }
      x[t] = acc;
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int t = 0; t < 16; t++) {
      X[b + t][b + c] = x[t];
      m = fmaxf(m, fabsf(x[t]));
    }
    m *= fabsf(be[b + c]);
  } else if (lane < 48) {
#pragma unroll
    for (int t = 0; t < 16; t++) X[r0 + t][r0 + 16 + c] = 0.0f;
  }
  __builtin_amdgcn_wave_barrier();
  f4 y = {0, 0, 0, 0}, x = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < 4; k++)
    y = __builtin_amdgcn_mfma_f32_16x16x4f32(X[r0 + 16 + c][r0 + 4 * k + g], X[r0 + 4 * k + g][r0 + c], y, 0, 0, 0);
#pragma unroll
  for (int k = 0; k < 4; k++)
    x = __builtin_amdgcn_mfma_f32_16x16x4f32(X[r0 + 16 + c][r0 + 16 + 4 * g + k], y[k], x, 0, 0, 0);
  __builtin_amdgcn_wave_barrier();
  float n = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    X[r0 + 16 + 4 * g + i][r0 + c] = -x[i];
    n = fmaxf(n, fabsf(x[i]));
  }
  return fmaxf(m, n * fabsf(be[r0 + c]));
}

// T's lower left 32 x 32 quarter, -X11 (A10 X00) with 32 x 32 blocks, one 16 x 16 tile a wave, into Z.
__device__ __forceinline__ float invert_corner(Square& X, float (*Z)[36], const float* be, int w, int lane) {
  const int c = lane & 15, g = lane >> 4, cb = w & 1, r = 2 + (w >> 1);
  auto half = [&](int row) {
    f4 y = {0, 0, 0, 0};
    for (int m = cb; m < 2; m++)
#pragma unroll
      for (int k = 0; k < 4; k++)
        y = __builtin_amdgcn_mfma_f32_16x16x4f32(X[16 * row + c][16 * m + 4 * k + g], X[16 * m + 4 * k + g][16 * cb + c], y, 0, 0, 0);
    return y;
  };
  auto add = [&](int m, f4 y, f4 x) {
#pragma unroll
    for (int k = 0; k < 4; k++)
      x = __builtin_amdgcn_mfma_f32_16x16x4f32(X[16 * r + c][16 * m + 4 * g + k], y[k], x, 0, 0, 0);
    return x;
  };
  f4 x = add(2, half(2), f4{0, 0, 0, 0});
  if (r == 3) x = add(3, half(3), x);
  float n = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    Z[16 * (r - 2) + 4 * g + i][16 * cb + c] = -x[i];
    n = fmaxf(n, fabsf(x[i]));
  }
  return n * fabsf(be[16 * cb + c]);
}

// Y: the workspace's layout (LayF, or LayB: with the gradient's extra pieces).
template <int D, int DT, class Y>
__global__ __launch_bounds__(256, Y::grad ? 2 : 3) void k_chunk_prep(SeqArgs A) {
  constexpr int KS = D / 32, NPI = Y::NPI, NPO = Y::NPO;
  __shared__ PrepSmem<D, DT, Y::grad> sm;
  const long long j = blockIdx.x;
  const int hq = blockIdx.y;
  ChunkAt at;
  if (!chunk_at(A, j, at)) return;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, g = lane >> 4, wb = w >> 1, wp = w & 1;
  const int own = 32 * wb + perm_row(c16, wp);  // the lane's token
  char* const key = A.ws + (j * A.Hq + hq) * Y::key;
  float* const KK = (float*)(key + (Y::grad ? Y::offKK : 0));
  float* const QK = (float*)(key + (Y::grad ? Y::offQK : 0));
  // K and Q: fragments of row tile w, K (gradient: and Q) into LDS.  Tokens behind the end repeat the
  // last one: their W is zero.
  h8 kf[KS][NPI], qf[KS][NPI];
  float ik, iq;
  {
    const long long t = at.t0 + (long long)min(own, at.len - 1);
    ik = load_rows<D, DT>(A.k, t * A.ks + (long long)hq * D, g, kf);
    iq = load_rows<D, DT>(A.q, t * A.qs + (long long)hq * D, g, qf);
    if (g == 0) {
      sm.isk[own] = ik;
      sm.isq[own] = iq;
    }
#pragma unroll
    for (int ks = 0; ks < KS; ks++)
#pragma unroll
      for (int p = 0; p < NPI; p++) {
        const int o = (p * Y::NF + w * KS + ks) * kFrag + lane * 16;
        *(h8*)(key + Y::offK + o) = kf[ks][p];
        *(h8*)&sm.K[p][own][32 * ks + 8 * g] = kf[ks][p];
        if constexpr (Y::grad) *(h8*)&sm.Q[p][own][32 * ks + 8 * g] = qf[ks][p];
        else *(h8*)(key + Y::offQ + o) = qf[ks][p];
      }
  }
  __syncthreads();
  // K K^T, columns = this wave's tokens, rows up to their block; K Q^T likewise (gradient: Q K^T, rows from
  // their block on).  Block nb of both runs over tiles 2 nb, 2 nb + 1.
  float kk[2][8], qk[2][8];
#pragma unroll
  for (int nb = 0; nb < 2; nb++) {
    const bool kk_on = nb <= wb, qk_on = Y::grad ? nb >= wb : nb <= wb;
    f4 a[2], b[2];
#pragma unroll
    for (int p = 0; p < 2; p++) {
      a[p] = b[p] = f4{0, 0, 0, 0};
      const int row = 32 * nb + perm_row(c16, p);
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        h8 fk[NPI], fq[NPI];
#pragma unroll
        for (int n = 0; n < NPI; n++) {
          if (kk_on) fk[n] = *(const h8*)&sm.K[n][row][32 * ks + 8 * g];
          if (Y::grad && qk_on) fq[n] = *(const h8*)&sm.Q[Y::grad ? n : 0][row][32 * ks + 8 * g];
        }
        if (kk_on) {
          a[p] = mfma(fk[0], kf[ks][0], a[p]);
          if constexpr (NPI == 2) a[p] = mfma(fk[0], kf[ks][1], mfma(fk[1], kf[ks][0], a[p]));
        }
        if (qk_on) {
          if constexpr (Y::grad) {
            b[p] = mfma(fq[0], kf[ks][0], b[p]);
            if constexpr (NPI == 2) b[p] = mfma(fq[0], kf[ks][1], mfma(fq[1], kf[ks][0], b[p]));
          } else {
            b[p] = mfma(fk[0], qf[ks][0], b[p]);
            if constexpr (NPI == 2) b[p] = mfma(fk[0], qf[ks][1], mfma(fk[1], qf[ks][0], b[p]));
          }
        }
      }
    }
    const float* const isr = Y::grad ? sm.isq : sm.isk;
    const float io = Y::grad ? ik : iq;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const int r = 32 * nb + 8 * g + e;
      kk[nb][e] = kk_on ? a[e >> 2][e & 3] * (sm.isk[r] * ik) : 0.0f;
      qk[nb][e] = qk_on ? b[e >> 2][e & 3] * (isr[r] * io) : 0.0f;
    }
    if constexpr (Y::grad) {
      if (kk_on) store8<kF32>(KK, own * 64 + 32 * nb + 8 * g, kk[nb]);  // [t][s], t own
      if (qk_on) store8<kF32>(QK, own * 64 + 32 * nb + 8 * g, qk[nb]);  // [s][t], s own
    }
  }
  // K^T (and Q^T): rows = key dimensions
#pragma unroll
  for (int f = w; f < Y::NF; f += 4) {
    const int kr = 32 * (f >> 2) + perm_row(c16, (f >> 1) & 1), kc = 32 * (f & 1) + 8 * g;
#pragma unroll
    for (int p = 0; p < NPI; p++) {
      const int o = (p * Y::NF + f) * kFrag + lane * 16;
      h8 t;
#pragma unroll
      for (int i = 0; i < 8; i++) t[i] = sm.K[p][kc + i][kr];
      *(h8*)(key + Y::offKT + o) = t;
      if constexpr (Y::grad) {
#pragma unroll
        for (int i = 0; i < 8; i++) t[i] = sm.Q[p][kc + i][kr];
        *(h8*)(key + Y::offQ + o) = t;
      }
    }
  }
  float al_next = 1.0f, be_next = 0.0f;  // gates of the next head, token `lane`
  auto gates = [&](int hh) {
    if (lane < at.len) {
      const long long th = (at.t0 + (long long)lane) * A.H + hq * A.grp + hh;
      al_next = A.alpha[th];
      be_next = A.beta[th];
    }
  };
  gates(0);
  char* const heads = A.ws + key_bytes<Y>(A) + (j * A.H + hq * A.grp) * Y::head;
  // Two heads at a time: the four diagonal blocks of their A keep all waves busy
  for (int h0 = 0; h0 < A.grp; h0 += 2) {
    const int nh = min(2, A.grp - h0);
    __syncthreads();  // the last heads' T has been read (the first heads: K and Q)
    for (int u = 0; u < nh; u++) {
      char* const head = heads + (h0 + u) * Y::head;
      float* const tab = (float*)(head + Y::offTab);
      const float al = al_next, be = be_next;
      if (h0 + u + 1 < A.grp) gates(h0 + u + 1);
      // running products, token = lane
      float(*const gt)[64] = sm.gate[u];
      float p8 = al, s8 = 1.0f;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        const float x = __shfl_up(p8, o);
        if ((lane & 7) >= o) p8 *= x;
      }
      {
        float x = __shfl_down(al, 1);
        s8 = (lane & 7) < 7 ? x : 1.0f;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          x = __shfl_down(s8, o);
          if ((lane & 7) + o < 8) s8 *= x;
        }
      }
      float B[8];  // whole groups of 8
#pragma unroll
      for (int n = 0; n < 8; n++) B[n] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(p8), 8 * n + 7));
      float p32 = p8, s32 = s8;
      {
        const int n = (lane >> 3) & 3;
        const bool up = lane >= 32;
        const float b0 = up ? B[4] : B[0], b1 = up ? B[5] : B[1], b2 = up ? B[6] : B[2], b3 = up ? B[7] : B[3];
        if (n > 0) p32 *= b0;
        if (n > 1) p32 *= b1;
        if (n > 2) p32 *= b2;
        if (n < 3) s32 *= b3;
        if (n < 2) s32 *= b2;
        if (n < 1) s32 *= b1;
      }
      gt[0][lane] = al;
      gt[1][lane] = p8;
      gt[2][lane] = s8;
      gt[3][lane] = p32;
      gt[4][lane] = s32;
      __builtin_amdgcn_wave_barrier();
      const float BL = B[0] * B[1] * B[2] * B[3], BU = B[4] * B[5] * B[6] * B[7];
      if (w == 0) {
        const float G = lane < 32 ? p32 : BL * p32, L63 = lane < 32 ? s32 * BU : s32;
        const float ik0 = sm.isk[lane], iq0 = sm.isq[lane];
        tab[kTabU + lane] = (Y::grad ? be * G : G) * ik0;
        tab[kTabQ + lane] = G * iq0;
        tab[kTabD + lane] = L63 * ik0;
        if (lane == 63) tab[kTabG + 63] = G;
        if constexpr (Y::grad) {
          tab[kTabB + lane] = be;
          tab[kTabL + lane] = L63;
          tab[kTabIK + lane] = ik0;
          tab[kTabIQ + lane] = iq0;
        }
      }
      const float be_own = __shfl(be, own);
      // own token: place in its block, group, place in that; opaque: the predicates made from them are not
      // kept in scalar registers across heads
      int po = own & 31, pg = g;
      asm("" : "+v"(po), "+v"(pg));
      const int og = po >> 3, oi = po & 7;
      // L between `own` and the 8 tokens 8 g + e of its own block: down: own is the later one
      float Lo[8];
      auto in_block = [&](bool down) {
        const float *a = &gt[0][32 * wb + 8 * g], *pre = &gt[1][32 * wb + 8 * g], *suf = &gt[2][32 * wb + 8 * g];
        const int lo = down ? pg : og, hi = down ? og : pg;  // earlier and later group
        const float b1 = wb ? B[5] : B[1], b2 = wb ? B[6] : B[2];
        float mid = gt[down ? 1 : 2][own];
        if (lo == 0 && hi > 1) mid *= b1;
        if (lo <= 1 && hi == 3) mid *= b2;
        float c = 1.0f;
        if (down) {
#pragma unroll
          for (int e = 7; e >= 0; e--) {
            const float l = pg < og ? mid * suf[e] : c;
            Lo[e] = 8 * pg + e <= po ? l : 0.0f;
            if (e <= oi) c *= a[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; e++) {
            if (e > oi) c *= a[e];
            const float l = pg > og ? mid * pre[e] : c;
            Lo[e] = 8 * pg + e >= po ? l : 0.0f;
          }
        }
      };
      in_block(true);
      float pv[2][8];
      if (w == 0) sm.be[u][lane] = be;
#pragma unroll
      for (int nb = 0; nb < 2; nb++) {
        if (nb > wb) continue;
        float av[8];
        const float pre = gt[3][own];
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const float l = nb == wb ? Lo[e] : pre * gt[4][8 * g + e];
          const bool strict = nb < wb || 8 * pg + e < po;
          av[e] = strict ? be_own * (kk[nb][e] * l) : 0.0f;
          if constexpr (!Y::grad) pv[nb][e] = qk[nb][e] * l;
        }
        store8<kF32>(&sm.X[u][own][0], 32 * nb + 8 * g, av);
      }
      if constexpr (Y::grad) {
        in_block(false);
#pragma unroll
        for (int nb = 0; nb < 2; nb++) {
          if (nb < wb) continue;
          const float suf = gt[4][own];
#pragma unroll
          for (int e = 0; e < 8; e++) pv[nb][e] = qk[nb][e] * (nb == wb ? Lo[e] : suf * gt[3][32 + 8 * g + e]);
        }
      }
      // P's (gradient: P^T's) fragments
      {
        float mp = 0.0f;
#pragma unroll
        for (int nb = 0; nb < 2; nb++)
          if (Y::grad ? nb >= wb : nb <= wb)
#pragma unroll
            for (int e = 0; e < 8; e++) mp = fmaxf(mp, fabsf(pv[nb][e]));
        float ip;
        const float sp = scale_of(col_max(mp), ip);
        if (g == 0) tab[kTabP + own] = ip;
#pragma unroll
        for (int nb = 0; nb < 2; nb++)
          if (Y::grad ? nb >= wb : nb <= wb) {
            h8 hi, lo;
            split8<2>(pv[nb], sp, hi, lo);
            char* const dst = head + Y::offP + (Y::grad ? up_frag(w, nb) : tri_frag(w, nb)) * kFrag + lane * 16;
            *(h8*)dst = hi;
            if constexpr (NPO == 2) *(h8*)(dst + kTri * kFrag) = lo;
          }
      }
    }
    __syncthreads();
    auto most = [&](float m, int u, int n) {
      m = fmaxf(m, __shfl_xor(m, 1));
      m = fmaxf(m, __shfl_xor(m, 2));
      m = fmaxf(m, __shfl_xor(m, 4));
      m = fmaxf(m, __shfl_xor(m, 8));
      m = col_max(m);
      if (lane == 0) sm.most[u][n] = m;
    };
    if (wb < nh) most(invert_block(sm.X[wb], sm.be[wb], 32 * wp, lane), wb, wp);
    __syncthreads();
    for (int u = 0; u < nh; u++) most(invert_corner(sm.X[u], sm.Z[u], sm.be[u], w, lane), u, 2 + w);
    __syncthreads();
    for (int u = 0; u < nh; u++) {
      char* const head = heads + (h0 + u) * Y::head;
      float* const tab = (float*)(head + Y::offTab);
      // T's fragments of row tile w
      auto T_row = [&](int ks, float* x) {
        const float* src = wb && !ks ? &sm.Z[u][own - 32][8 * g] : &sm.X[u][own][32 * ks + 8 * g];
        const f4 x0 = *(const f4*)src, x1 = *(const f4*)(src + 4);
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = x0[e], x[4 + e] = x1[e];
      };
      if constexpr (!Y::grad) {
        float iT;
        float m = 0.0f;
#pragma unroll
        for (int n = 0; n < 6; n++) m = fmaxf(m, sm.most[u][n]);
        const float sT = scale_of(m, iT);
        if (tid == 0) tab[kTabG + 62] = iT;
#pragma unroll
        for (int ks = 0; ks < 2; ks++) {
          if (ks > wb) continue;
          float x[8];
          T_row(ks, x);
#pragma unroll
          for (int e = 0; e < 8; e++) x[e] *= sm.be[u][32 * ks + 8 * g + e];
          h8 hi, lo;
          split8<2>(x, sT, hi, lo);
          char* const dst = head + Y::offT + tri_frag(w, ks) * kFrag + lane * 16;
          *(h8*)dst = hi;
          *(h8*)(dst + kTri * kFrag) = lo;
        }
      } else {
        // T and T^T, rows scaled
        float x[2][8], y[2][8], mt = 0.0f, mu = 0.0f;
#pragma unroll
        for (int ks = 0; ks < 2; ks++) {
          if (ks <= wb) {
            T_row(ks, x[ks]);
#pragma unroll
            for (int e = 0; e < 8; e++) mt = fmaxf(mt, fabsf(x[ks][e]));
          }
          if (ks >= wb) {
#pragma unroll
            for (int e = 0; e < 8; e++) {
              y[ks][e] = !wb && ks ? sm.Z[u][8 * g + e][own] : sm.X[u][32 * ks + 8 * g + e][own];
              mu = fmaxf(mu, fabsf(y[ks][e]));
            }
          }
        }
        float it, iu;
        const float st = scale_of(col_max(mt), it), su = scale_of(col_max(mu), iu);
        if (g == 0) {
          tab[kTabT + own] = it;
          tab[kTabTt + own] = iu;
        }
#pragma unroll
        for (int ks = 0; ks < 2; ks++) {
          h8 hi, lo;
          if (ks <= wb) {
            split8<2>(x[ks], st, hi, lo);
            char* const dst = head + Y::offT + tri_frag(w, ks) * kFrag + lane * 16;
            *(h8*)dst = hi;
            *(h8*)(dst + kTri * kFrag) = lo;
          }
          if (ks >= wb) {
            split8<2>(y[ks], su, hi, lo);
            char* const dst = head + Y::offTt + up_frag(w, ks) * kFrag + lane * 16;
            *(h8*)dst = hi;
            *(h8*)(dst + kTri * kFrag) = lo;
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// the pass over the chunks
// ---------------------------------------------------------------------------------------------

// A wave owns 16 columns of one (sequence, head) state for the whole sequence (lane l: column l & 15, rows in
// accumulator order) and never needs another wave's: all waves of a workgroup read the same fragments,
// staged in LDS one chunk ahead.  The state is held in units of a power of two per column (S = unit * St,
// St within binary16's range, checked every chunk), so that it turns into an operand without a product and
// the update accumulates on it directly.
//
// 8 sequences of 0 .. 3,698 tokens x 48 states (d = 128 bf16): 331 us (median of calls; 319 .. 350), of it about 5.5 a
// chunk of the longest sequence; 541 MB read, 226 written.  A chunk is one chain of products and roundings to operands (K S, T R, P W,
// K^T W), and two waves a SIMD fill its gaps only in part: the vector ALUs are busy 48%, the matrix cores 29%,
// 30% of the wave cycles wait.  Four waves a SIMD do not fit: a state column with its operands takes 190
// registers.  The chain of a column does not shorten with more CUs, hence the segments below.
//
// kForward: the whole sequence, read out.  kKeep (gradient, LayB): no readout, the states before every chunk
// and W are kept.  Where there are few (sequence, head) pairs and many chunks, the chunks of a sequence are
// cut into segs.P segments (blockIdx.y): the state behind a segment is M S + N, so kSegment runs every
// segment twice, from the unit matrix without V (M, blockIdx.z = 1) and from zero with V (N);
// k_chunk_join then walks over the segments, and kReadout runs them all at once from their first states.
struct Segs {
  int P;            // segments of a sequence
  float *MN, *S;    // [2][tiles][P][D][D] (N, then M), [tiles][P][D][D] first states
};
// The sequence of a workgroup: where there are more states than CUs, the longest sequences first, so that
// the last ones to finish are short (8 sequences of 0 .. 3,698 tokens x 48 states: 394 -> 346 us).  A wave ranks
// up to 64 lengths for that; more sequences even out by themselves over many rounds of workgroups, and
// with short ones the ranking costs more than it gives (16 x 48 states of two chunks: 60 -> 66 us).
__device__ __forceinline__ int seq_in_order(const SeqArgs& A, int r) {
  if (!A.cu || A.N > 64 || A.T < 256 * A.N || (long long)A.N * A.H <= 256) return r;
  const int lane = threadIdx.x & 63;
  int t0 = 0, t1 = -1;
  if (lane < A.N) seq_range(A, lane, t0, t1);
  const int len = t1 - t0;
  int before = 0;
  for (int j = 0; j < A.N; j++) {
    const int l = __builtin_amdgcn_readlane(len, j);
    before += l > len || (l == len && j < lane);
  }
  return __builtin_ctzll(__ballot(lane < A.N && before == r));
}

// HV workgroups of NW waves share a state's columns.  They are 8 apart, on one XCD and its L2.
template <int HV> __device__ __forceinline__ long long state_of(unsigned x) { return HV == 1 ? x : x / (8 * HV) * 8 + x % 8; }
template <int HV> __device__ __forceinline__ int columns_of(unsigned x) { return HV == 1 ? 0 : x / 8 % HV; }
template <int NW> unsigned workgroups(const SeqArgs& a, int D) {
  const long long n = (long long)a.N * a.H, hv = D / (16 * NW);
  return (unsigned)(hv == 1 ? n : (n + 7) / 8 * 8 * hv);
}
// Calls f with a workgroup's waves (an integral constant), for P passes over every state at once.
// D = 128, 16-bit types: a state's columns go to two workgroups of four waves where the states leave CUs
// idle (at most 128 passes; 128 states x 32 chunks: 225 -> 177 us kept, 308 -> 243 in reverse) and where
// sequences are short (under 256 tokens: 70 x 48 states of two chunks 299 -> 285 us), because two such
// workgroups share a CU and one's first and last states move while the other computes.  Elsewhere all
// eight waves share one copy of the operands (384 states x 43 chunks: 394 us against 440).
template <int D, int DT, class F>
hipError_t with_state_waves(const SeqArgs& a, int P, F&& f) {
  if constexpr (D == 64) return f(std::integral_constant<int, 4>{});
  else if constexpr (DT == kF32) return f(std::integral_constant<int, 8>{});
  else if ((long long)a.N * a.H * P > 128 && a.T >= 256LL * a.N) return f(std::integral_constant<int, 8>{});
  else return f(std::integral_constant<int, 4>{});
}
enum StateMode { kForward, kKeep, kSegment, kReadout };
__device__ __forceinline__ int seg_chunks(int nc, int P) { return (nc + P - 1) / P; }

template <int D, int DT, int NW, class Y, int MODE>
__global__ __launch_bounds__(64 * NW, D == 64 && DT != kF32 ? 3 : 2) void k_chunk_state(SeqArgs A, float* keepS, float* keepW, Segs segs) {
  constexpr int KS = D / 32, NPI = Y::NPI, NPO = Y::NPO, NB = D / 32;
  constexpr bool out_on = MODE == kForward || MODE == kReadout, cut = MODE == kSegment || MODE == kReadout;
  // staged: K, K^T (and Q), then T (and P), then the tables of two chunks
  constexpr int keyN = out_on ? Y::key : Y::offQ, HV = D / (16 * NW);
  constexpr int offT = keyN, offP = keyN + Y::offP, offTab = offT + (out_on ? Y::offTab : 2 * kTri * kFrag);
  constexpr int part = offTab + 2 * Y::tab;
  using Tr = Slice<DT>;
  using TrF = Slice<kF32>;
  constexpr int trN = Tr::bytes;
  __shared__ __attribute__((aligned(16))) char buf[part + NW * trN];
  const long long tile = state_of<HV>(blockIdx.x);
  const int part0 = columns_of<HV>(blockIdx.x);
  if (HV > 1 && tile >= (long long)A.N * A.H) return;
  const int rank = (int)(tile / A.H), h = (int)(tile - (long long)rank * A.H), s = seq_in_order(A, rank);
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  int t0, t1;
  const bool valid = seq_range(A, s, t0, t1);
  const int slot = seq_slot(A, s, valid, h == 0 && !cut && part0 == 0 && tid == 0);
  if (slot < 0 || t1 - t0 < A.split) return;
  if (t0 == t1 && MODE == kKeep) return;
  if (t0 == t1 && MODE == kForward && (!A.S_out || A.S_out == A.S_in)) return;
  const int col0 = 16 * (part0 * NW + w), col = col0 + c16;
  const long long so = ((long long)slot * A.H + h) * D * D;
  const int nc = (t1 - t0 + kChunk - 1) / kChunk;
  int c_first = 0, c_end = nc;
  long long seg = 0;
  if (cut) {
    const int n = seg_chunks(nc, segs.P);
    c_first = min((int)blockIdx.y * n, nc);
    c_end = min(c_first + n, nc);
    seg = (((long long)s * A.H + h) * segs.P + blockIdx.y) * D * D;
  }
  const bool unit_start = MODE == kSegment && blockIdx.z;
  char* const piece = buf + part + w * trN;
  const Tr vrows(piece, A.vs, col0, lane), orows(piece, A.os, col0, lane);
  const TrF krows(piece, D, col0, lane);
  const long long j0 = first_slot(A, s);
  const char* const heads = A.ws + key_bytes<Y>(A);
  const int hq = h / A.grp;
  // chunk c's pieces on their way into LDS, 1 KiB a wave at a time, each as soon as every wave holds the last
  // chunk's in registers: K, Q and T (early), then P, K^T and the tables (late)
  const unsigned lds0 = lds_offset(buf), lane16 = 16 * lane;
  auto fetch = [&](int c, bool early) {
    const char* const key = A.ws + ((j0 + c) * A.Hq + hq) * Y::key;
    const char* const head = heads + ((j0 + c) * A.H + h) * Y::head;
    if (early) {
      copy_block<NW>(key, lds0, 0, Y::offKT, w, lane16);
      if constexpr (out_on) copy_block<NW>(key, lds0, Y::offQ, keyN, w, lane16);
      copy_block<NW>(head, lds0 + offT, 0, 2 * kTri * kFrag, w, lane16);
    } else {
      copy_block<NW>(key, lds0, Y::offKT, 2 * Y::offKT, w, lane16);
      if constexpr (out_on) copy_block<NW>(head, lds0 + offT, Y::offP, Y::offTab, w, lane16);
      const unsigned at = lds0 + offTab + (c & 1) * Y::tab;
      if (w == 0) copy_to_lds(head + Y::offTab, at, lane16);
      if (w == 1 && lane < (Y::tab - 1024) / 16) copy_to_lds(head + Y::offTab + 1024, at + 1024, lane16);
    }
  };
  typename Tr::u4 v[Tr::NL];  // V of the next chunk, as it lies in memory
  auto fetch_v = [&](int c) {
    const int tc = t0 + c * kChunk;
    // (M's segments: a descriptor without bytes, V = 0)
    vrows.load(rows_at<DT>(A.v, tc, A.vs, h * D, unit_start ? 0 : D, unit_start ? 1 : min(t1 - tc, kChunk)), v);
  };
  if (c_first < c_end) {
    fetch(c_first, true);
    fetch(c_first, false);
  }
  f4 St[2 * NB];
#pragma unroll
  for (int rt = 0; rt < 2 * NB; rt++)
#pragma unroll
    for (int i = 0; i < 4; i++) St[rt][i] = unit_start && 32 * (rt >> 1) + 8 * g + 4 * (rt & 1) + i == col ? 1.0f : 0.0f;
  if (const float* const first = MODE == kSegment ? nullptr : MODE == kReadout ? segs.S + seg : A.S_in ? A.S_in + so : nullptr)
    krows.template load_all<2 * NB>(first, St);
  if (c_first < c_end) fetch_v(c_first);
  float unit = 1.0f;
  const f4 zero = {0, 0, 0, 0};
  for (int c = c_first; c < c_end; c++) {
    const char* const lds = buf;
    const int tc = t0 + c * kChunk, len = t1 - tc < kChunk ? t1 - tc : kChunk;
    wait_copies();
    __syncthreads();  // chunk c is there, and every wave is done with chunk c - 1
    const bool more = c + 1 < c_end;
    const float* const tab = (const float*)(lds + offTab + (c & 1) * Y::tab);
    auto frag = [&](int off, int n, int p, int f) { return *(const h8*)(lds + off + (p * n + f) * kFrag + lane16); };
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
    h8 Sh[NB], Sl[NB], xh[2], xl[2];
    f4 z[2 * NB > 4 ? 2 * NB : 4];
    read(Y::offK);
    f4 R[4];
    vrows.to_acc(v, R);
    if (more) fetch_v(c + 1);
    ahead();
    float most = tiles_max<2 * NB>(St);
    fit<2 * NB>(St, unit, most);
    if constexpr (MODE == kKeep) krows.template store_all<2 * NB>(keepS + ((j0 + c) * A.H + h) * D * D, St, unit);
    to_planes<NB, 2, true>(St, 1.0f, Sh, Sl);
    auto times_state = [&](bool low) {
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int rt = 0; rt < 4; rt++) z[rt] = mfma(f[rt * KS + ks], Sh[ks], ks ? z[rt] : zero);
      if (low)
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
          for (int rt = 0; rt < 4; rt++) z[rt] = mfma(f[rt * KS + ks], Sl[ks], z[rt]);
      if constexpr (NPI == 2)
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
          for (int rt = 0; rt < 4; rt++) z[rt] = mfma(fl[rt * KS + ks], Sh[ks], z[rt]);
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
    // R = V - G K S0 (gradient: times beta)
    float ix, w1;
#pragma unroll
    for (int rt = 0; rt < 4; rt++) {
      const f4 cu = rows(kTabU, rt), be = Y::grad ? rows(kTabB, rt) : zero;
#pragma unroll
      for (int i = 0; i < 4; i++) R[rt][i] = fmaf(-cu[i] * unit, z[rt][i], Y::grad ? be[i] * R[rt][i] : R[rt][i]);
    }
    ix = to_operand<2, 2>(R, xh, xl);
    // W = w1 z, z = T R (gradient: T's rows have scales of their own)
    w1 = (Y::grad ? 1.0f : tab[kTabG + 62]) * ix;
    auto tri = [&](auto&& a, int p, const h8* b, bool first) {
#pragma unroll
      for (int ks = 0; ks < 2; ks++)
#pragma unroll
        for (int rt = 0; rt < 4; rt++)
          if (ks <= rt >> 1) z[rt] = mfma(a[p][tri_frag(rt, ks)], b[ks], first && !ks ? zero : z[rt]);
    };
    tri(ft, 0, xh, true);
    tri(ft, 0, xl, false);
    tri(ft, 1, xh, false);
    ahead();
    if constexpr (out_on) read(Y::offQ);
    else read(Y::offKT);
    __syncthreads();
    if (more) fetch(c + 1, true);
    if (more && !out_on) fetch(c + 1, false);
    ahead();
#pragma unroll
    for (int rt = 0; rt < 4; rt++) R[rt] = Y::grad ? z[rt] * rows(kTabT, rt) : z[rt];
    if constexpr (MODE == kKeep) {
      krows.template store_all<4>(keepW + ((j0 + c) * A.H + h) * 64 * D, R, w1);
    } else if constexpr (out_on) {
      // O = G Q S0 + P W
      const float iw = to_operand<2, NPO>(R, xh, xl) * w1;
      times_state(NPO == 2);
      ahead();
      h8 fp[NPO][kTri];
#pragma unroll
      for (int p = 0; p < NPO; p++)
#pragma unroll
        for (int n = 0; n < kTri; n++) fp[p][n] = frag(offP, kTri, p, n);
      ahead();
      f4 y[4];
#pragma unroll
      for (int rt = 0; rt < 4; rt++) y[rt] = z[rt];
      tri(fp, 0, xh, true);
      if constexpr (NPO == 2) {
        tri(fp, 0, xl, false);
        tri(fp, 1, xh, false);
      }
      ahead();
      read(Y::offKT);
      __syncthreads();
      if (more) fetch(c + 1, false);
      ahead();
#pragma unroll
      for (int rt = 0; rt < 4; rt++) {
        const f4 cq = rows(kTabQ, rt), ip = rows(kTabP, rt);
#pragma unroll
        for (int i = 0; i < 4; i++) y[rt][i] = fmaf(cq[i] * unit, y[rt][i], (ip[i] * iw) * z[rt][i]);
      }
      orows.store(rows_at<DT>(A.out, tc, A.os, h * D, D, len), y);
    }
    // S1 = G_C S0 + K^T diag(L[C, .]) W, in the state's units
#pragma unroll
    for (int rt = 0; rt < 4; rt++) R[rt] *= rows(kTabD, rt);
    fit_sum<2 * NB>(St, unit, most, tab[kTabG + 63], tiles_max<4>(R) * w1);
    // unit is a power of two: its inverse by the exponent
    to_planes<2, 2>(R, w1 * __uint_as_float(0x7f000000u - __float_as_uint(unit)), xh, xl);
#pragma unroll
    for (int ks = 0; ks < 2; ks++) {
#pragma unroll
      for (int rt = 0; rt < 2 * NB; rt++) St[rt] = mfma(f[2 * rt + ks], xh[ks], St[rt]);
#pragma unroll
      for (int rt = 0; rt < 2 * NB; rt++) St[rt] = mfma(f[2 * rt + ks], xl[ks], St[rt]);
      if constexpr (NPI == 2)
#pragma unroll
        for (int rt = 0; rt < 2 * NB; rt++) St[rt] = mfma(fl[2 * rt + ks], xh[ks], St[rt]);
    }
  }
  float* dst = nullptr;
  if (MODE == kForward || (MODE == kReadout && c_end == nc && (c_first < nc || (nc == 0 && blockIdx.y == 0))))
    dst = A.S_out ? A.S_out + so : nullptr;
  if (MODE == kSegment) dst = segs.MN + (unit_start ? (long long)A.N * A.H * segs.P * D * D : 0LL) + seg;
  if (dst) krows.template store_all<2 * NB>(dst, St, unit);
}

// First states of the segments: S_0 = S_in, S_{p+1} = M_p S_p + N_p.  A wave owns 16 columns, as in the pass,
// and the waves of a state are spread over the card, two a workgroup: there is nothing they share but M,
// whose rows are on their way one row tile ahead.  32 states x 8 segments of 128 x 128: 50 us, the latency of 8
// steps of a 128 x 128 by 128 x 16 product with M from HBM (eight waves a workgroup: 146 us).
template <int D>
__global__ __launch_bounds__(128) void k_chunk_join(SeqArgs A, Segs segs) {
  constexpr int KS = D / 32, NB = D / 32;
  __shared__ __attribute__((aligned(16))) char buf[2 * Slice<kF32>::bytes];
  const long long tile = blockIdx.x;
  const int s = (int)(tile / A.H), h = (int)(tile - (long long)s * A.H);
  const int lane = threadIdx.x & 63, v = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = 2 * blockIdx.y + v;
  const int c16 = lane & 15, g = lane >> 4;
  int t0, t1;
  const bool valid = seq_range(A, s, t0, t1);
  const int slot = seq_slot(A, s, valid, h == 0 && blockIdx.y == 0 && threadIdx.x == 0);
  if (slot < 0) return;
  const int col = 16 * w + c16;
  const Slice<kF32> rows(buf + v * Slice<kF32>::bytes, D, 16 * w, lane);
  auto at = [&](int rt, int i) { return (long long)(32 * (rt >> 1) + 8 * g + 4 * (rt & 1) + i) * D + col; };
  f4 S[2 * NB];
#pragma unroll
  for (int rt = 0; rt < 2 * NB; rt++)
#pragma unroll
    for (int i = 0; i < 4; i++) S[rt][i] = A.S_in ? A.S_in[((long long)slot * A.H + h) * D * D + at(rt, i)] : 0.0f;
  const int nc = (t1 - t0 + kChunk - 1) / kChunk, per = seg_chunks(nc, segs.P);
  for (int p = 0;; p++) {
    const long long seg = (tile * segs.P + p) * D * D;
    const bool last = (p + 1) * per >= nc;  // of the segments that have chunks
    const float *N = segs.MN + seg, *M = N + (long long)gridDim.x * segs.P * D * D;
    float x[2][KS][8];
    f4 n[2];
    auto fetch = [&](int rt) {
      const int row = 32 * (rt >> 1) + perm_row(c16, rt & 1);
#pragma unroll
      for (int ks = 0; ks < KS; ks++) load8<kF32>(M, row * D + 32 * ks + 8 * g, x[rt & 1][ks]);
#pragma unroll
      for (int i = 0; i < 4; i++) n[rt & 1][i] = N[at(rt, i)];
    };
    if (!last) fetch(0);
    rows.template store_all<2 * NB>(segs.S + seg, S, 1.0f);
    if (last) return;
    h8 Sh[NB], Sl[NB];
    const float iS = to_operand<NB, 2>(S, Sh, Sl);
#pragma unroll
    for (int rt = 0; rt < 2 * NB; rt++) {
      if (rt + 1 < 2 * NB) fetch(rt + 1);
      ahead();
      float m = 0.0f, inv;
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int e = 0; e < 8; e++) m = fmaxf(m, fabsf(x[rt & 1][ks][e]));
      const float sc = scale_of(col_max(m), inv);
      f4 z = {0, 0, 0, 0};
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        h8 hi, lo;
        split8<2>(x[rt & 1][ks], sc, hi, lo);
        z = mfma(lo, Sh[ks], mfma(hi, Sl[ks], mfma(hi, Sh[ks], z)));
      }
#pragma unroll
      for (int i = 0; i < 4; i++) S[rt][i] = fmaf(z[i], __shfl(inv, 4 * g + i) * iS, n[rt & 1][i]);
      ahead();
    }
  }
}

}  // namespace dlt
}  // namespace stepq
