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
// and holds it in units of a power of two per column.  4 sequences of 2,048 tokens x 32 states (d = 128
// bf16): 245 us (median of calls; 237 .. 255), 7.6 a chunk, 189 MB read and 470 written (the state's gradient behind every chunk among them): two
// operands' roundings more a chunk than forward, and one wave a SIMD.
template <int D, int DT, int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_chunk_reverse(GradArgs B, Keep keep) {
  using L = LayB<D, DT>;
  constexpr int KS = D / 32, NPI = L::NPI, NB = D / 32;
  constexpr int keyN = L::offKK, triN = 4 * kTri * kFrag;  // K, K^T, Q^T; T^T, P^T
  constexpr int offTt = keyN, offP = keyN + 2 * kTri * kFrag, offTab = keyN + triN;
  constexpr int part = offTab + 2 * L::tab, HV = D / (16 * NW);
  const SeqArgs& A = B.f;
  using Tr = Slice<DT>;
  using TrF = Slice<kF32>;
  constexpr int trN = TrF::bytes;
  static_assert(part + NW * trN <= 160 * 1024);
  __shared__ __attribute__((aligned(16))) char buf[part + NW * trN];
  const long long tile = state_of<HV>(blockIdx.x);
  const int part0 = columns_of<HV>(blockIdx.x);
  if (HV > 1 && tile >= (long long)A.N * A.H) return;
  const int rank = (int)(tile / A.H), h = (int)(tile - (long long)rank * A.H), s = seq_in_order(A, rank);
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  int t0, t1;
  const bool valid = seq_range(A, s, t0, t1);
  if (seq_slot(A, s, valid, h == 0 && part0 == 0 && tid == 0) < 0) return;
  const int col0 = 16 * (part0 * NW + w);
  char* const piece = buf + part + w * trN;
  const Tr orows(piece, A.os, col0, lane), vrows(piece, (long long)A.H * D, col0, lane);
  const TrF krows(piece, D, col0, lane);
  const long long so = ((long long)s * A.H + h) * D * D;
  const long long j0 = first_slot(A, s);
  const char* const heads = A.ws + key_bytes<L>(A);
  const int hq = h / A.grp;
  const int nc = (t1 - t0 + kChunk - 1) / kChunk;
  const unsigned lds0 = lds_offset(buf), lane16 = 16 * lane;
  auto fetch = [&](int c, bool early) {
    const char* const key = A.ws + ((j0 + c) * A.Hq + hq) * L::key;
    const char* const head = heads + ((j0 + c) * A.H + h) * L::head;
    if (early) {
      copy_block<NW>(key, lds0, 0, L::offKT, w, lane16);
      copy_block<NW>(key, lds0, L::offQ, keyN, w, lane16);
      copy_block<NW>(head + L::offTt, lds0 + offTt, 0, triN, w, lane16);
    } else {
      copy_block<NW>(key, lds0, L::offKT, L::offQ, w, lane16);
      copy_block<NW>(head + L::offTab, lds0 + offTab + (c & 1) * L::tab, 0, L::tab, w, lane16);
    }
  };
  typename Tr::u4 o[Tr::NL];
  auto fetch_o = [&](int c) {
    const int tc = t0 + c * kChunk;
    orows.load(rows_at<DT>(B.d_out, tc, A.os, h * D, D, t1 - tc < kChunk ? t1 - tc : kChunk), o);
  };
  if (nc) {
    fetch(nc - 1, true);
    fetch(nc - 1, false);
  }
  f4 Gt[2 * NB];
#pragma unroll
  for (int rt = 0; rt < 2 * NB; rt++) Gt[rt] = f4{0, 0, 0, 0};
  if (B.dS_out) krows.template load_all<2 * NB>(B.dS_out + so, Gt);
  if (nc) fetch_o(nc - 1);
  float unit = 1.0f;
  const f4 zero = {0, 0, 0, 0};
  for (int c = nc - 1; c >= 0; c--) {
    const char* const lds = buf;
    const int tc = t0 + c * kChunk, len = t1 - tc < kChunk ? t1 - tc : kChunk;
    wait_copies();
    __syncthreads();
    const float* const tab = (const float*)(lds + offTab + (c & 1) * L::tab);
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
    f4 dO[4];
    orows.to_acc(o, dO);
    if (c) fetch_o(c - 1);
    ahead();
    float most = tiles_max<2 * NB>(Gt);
    fit<2 * NB>(Gt, unit, most);
    krows.template store_all<2 * NB>(keep.G + ((j0 + c) * A.H + h) * D * D, Gt, unit);
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
    __syncthreads();
    if (c) fetch(c - 1, true);
    ahead();
    {
      f4 dv[4];
#pragma unroll
      for (int rt = 0; rt < 4; rt++) {
        Y[rt] = y[rt] * (rows(kTabTt, rt) * ix);
        dv[rt] = rows(kTabB, rt) * Y[rt];
      }
      krows.template store_all<4>(keep.Y + ((j0 + c) * A.H + h) * 64 * D, Y, 1.0f);
      vrows.store(rows_at<DT>(B.dv, tc, (long long)A.H * D, h * D, D, len), dv);
    }
    // dS0 = G_C dS1 + Q^T G dO - K^T G diag(beta) Y, in the gradient's units
#pragma unroll
    for (int rt = 0; rt < 4; rt++) {
      dO[rt] *= rows(kTabQ, rt);
      Y[rt] *= -rows(kTabU, rt);
    }
    fit_sum<2 * NB>(Gt, unit, most, tab[kTabG + 63], fmaxf(tiles_max<4>(dO), tiles_max<4>(Y)));
    const float iu = 1.0f / unit;
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
    __syncthreads();
    if (c) fetch(c - 1, false);
    ahead();
    to_planes<2, 2>(Y, iu, xh, xl);
    update();
  }
  if (B.dS_in) krows.template store_all<2 * NB>(B.dS_in + so, Gt, unit);
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

// Aligned, so that 8 neighbouring floats are read as two 16-byte pieces: as pairs of 4 bytes they took 40% of
// the LDS time in conflicts (593 us -> 540).
template <int D, int DT>
struct alignas(16) GradSmem {
  static constexpr int NPI = kInPlanes<DT>, NW = D / 16;
  // What the value heads share, every wave's as it reads it back: k_t.k_s and q_t.k_s of the down pairs, and
  // (where there is room) its rows of K^T and Q^T.
  static constexpr bool keep_kq = D == 64 || DT != kF32;
  char pairs[4][8 * kFrag], kq[keep_kq ? NW : 1][keep_kq ? 4 * NPI * kFrag : 16];
  union {
    struct {  // fragments: row tiles in accumulator order, D / 32 steps each
      char O[NPI][4 * (D / 32) * kFrag], Y[2][4 * (D / 32) * kFrag], W[2][4 * (D / 32) * kFrag];
    } in;
    struct {
      char fr[24 * 2 * kFrag];  // fragments of N, Zd (lower, 6 each), N^T, Zu (upper)
      float xT[64][66];         // xT[s][t]: the pairs' values without their gates
      float iF[4][64];          // inverse row scales of the four
    } m;
    float out[64][D + 4];
  };
  float isO[64], isY[64], isW[64], isk[64], isq[64];
  float gate[7][64];            // a, pre8, suf8, pre32, suf32, G, L[C,.]
  float be[64], yv[64], rowx[64], dot[3][NW][64], corner[NW], z[64], y[64], da[64];
};

// 8 elements as they lie in memory.
template <int DT>
struct Raw8 {
  static constexpr int N = DT == kF32 ? 2 : 1;
  typedef unsigned u4 __attribute__((ext_vector_type(4)));
  u4 a[N];
  __device__ void load(const void* p, long long at) {
#pragma unroll
    for (int n = 0; n < N; n++) a[n] = ((const u4*)((const char*)p + at * (16 * N / 8)))[n];
  }
  __device__ void get(float* x) const {
#pragma unroll
    for (int e = 0; e < 8; e++) {
      if constexpr (DT == kF32) x[e] = __uint_as_float(a[e >> 2][e & 3]);
      else x[e] = e_f<DT>((unsigned short)(e & 1 ? a[0][e >> 1] >> 16 : a[0][e >> 1]));
    }
  }
};

// Row tile rt of a 64-row operand as fragments, from the lane's pieces of its row; zero where not `live`.
template <int D, int NP>
__device__ __forceinline__ void rows_put(float (*x)[8], bool live, int rt, int lane, int row,
                                         char (*dst)[4 * (D / 32) * kFrag], float* is) {
  constexpr int KS = D / 32;
  float m = 0.0f;
#pragma unroll
  for (int ks = 0; ks < KS; ks++)
#pragma unroll
    for (int e = 0; e < 8; e++) {
      x[ks][e] = live ? x[ks][e] : 0.0f;
      m = fmaxf(m, fabsf(x[ks][e]));
    }
  float inv;
  const float s = scale_of(col_max(m), inv);
  if (lane < 16) is[row] = inv;
#pragma unroll
  for (int ks = 0; ks < KS; ks++) {
    h8 hi, lo;
    split8<NP>(x[ks], s, hi, lo);
    char* const o = &dst[0][(rt * KS + ks) * kFrag + lane * 16];
    *(h8*)o = hi;
    if constexpr (NP == 2) *(h8*)(o + 4 * KS * kFrag) = lo;
  }
}

// One workgroup of D / 16 waves per (chunk, key head); the value heads that share the key head one after
// another, dQ and dK summed in registers.  Wave w owns the 16 key dimensions 32 (w >> 1) + perm(., w & 1) of
// all products with the states and of dQ and dK.  The pairs of tokens are formed twice, with the later
// token and with the earlier one as the lane's own (a wave each where there are eight): a lane then holds 8
// consecutive partners (their row tiles permuted), which is the fragment of N, N^T and either half of Z + Z^T as it is.
//
// 8,192 tokens x 32 heads on 16 key heads (d = 128 bf16): 480 .. 550 us, 32 a head and workgroup, 0.6 GB read.  One
// workgroup a CU (operands of 64 x 128 in two planes fill LDS, 256 registers a lane), so a head's phases --
// rows in, products with the states, pairs, gates -- follow each other with barriers between and half of
// the wave cycles wait; the vector ALUs are busy 38%, the matrix cores 11%, LDS 18%.
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
  // pairs: row tile pt, own token; down: own is the later token
  const int pt = w & 3, pb = pt >> 1;
  const bool down = NW == 4 || w < 4, up = NW == 4 || w >= 4;
  // this lane's column of Q and K, rows in accumulator order (zero behind the end)
  const Rows<DT> qrows(A.qs, dk, g), krows(A.ks, dk, g);
  constexpr int NV = DT == kF32 ? 4 : 2;  // 16-bit types: two rows a register
  unsigned qv[4][NV], kv[4][NV];
  {
    unsigned q[4][4], k[4][4];
    qrows.load(rows_at<DT>(A.q, at.t0, A.qs, hq * D, D, at.len), q);
    krows.load(rows_at<DT>(A.k, at.t0, A.ks, hq * D, D, at.len), k);
#pragma unroll
    for (int rt = 0; rt < 4; rt++)
#pragma unroll
      for (int i = 0; i < NV; i++) {
        qv[rt][i] = NV == 4 ? q[rt][i] : q[rt][2 * i & 3] | q[rt][(2 * i + 1) & 3] << 16;
        kv[rt][i] = NV == 4 ? k[rt][i] : k[rt][2 * i & 3] | k[rt][(2 * i + 1) & 3] << 16;
      }
  }
  auto column = [&](unsigned (*v)[NV], int rt, int i) {
    if constexpr (NV == 4) return raw_value<DT>(v[rt][i]);
    else return raw_value<DT>(i & 1 ? v[rt][i >> 1] >> 16 : v[rt][i >> 1]);
  };
  if (tid < 64) {
    const float* const tab = (const float*)(A.ws + key_bytes<Y>(A) + (j * A.H + hq * A.grp) * Y::head + Y::offTab);
    sm.isk[tid] = tab[kTabIK + tid];
    sm.isq[tid] = tab[kTabIQ + tid];
  }
  int row = tid / TPR, own = 32 * pb + perm_row(c16, pt & 1);
  // what the value heads share
  auto kq_at = [&](int n, int ks, int p) {  // fragments of this wave's rows of K^T (n = 0) and Q^T
    return *(const h8*)(key + (n ? Y::offQ : Y::offKT) + (p * Y::NF + 2 * w + ks) * kFrag + lane * 16);
  };
  if (down)
#pragma unroll
    for (int nb = 0; nb < 2; nb++) {
      if (nb > pb) continue;
      float x[8];
      load8<kF32>(key + Y::offKK, own * 64 + 32 * nb + 8 * g, x);
      store8<kF32>(sm.pairs[pt], (4 * nb * kFrag + lane * 32) / 4, x);
#pragma unroll
      for (int e = 0; e < 8; e++) x[e] = ((const float*)(key + Y::offQK))[(32 * nb + 8 * g + e) * 64 + own];
      store8<kF32>(sm.pairs[pt], ((4 * nb + 2) * kFrag + lane * 32) / 4, x);
    }
  if constexpr (GradSmem<D, DT>::keep_kq)
#pragma unroll
    for (int n = 0; n < 4 * NPI; n++) *(h8*)(sm.kq[w] + n * kFrag + lane * 16) = kq_at(n / (2 * NPI), n / NPI % 2, n % NPI);
  // What a wave brings in of a head: row tile pt of Y and V or of W and dO (four waves: of both), 16 rows of S0.
  // Not one head ahead: the registers that this takes cost more in spills than it hides (a kernel of 600 us
  // took 676 with S0 alone ahead; with Y and W ahead in LDS 742 instead of 713).
  constexpr int NR = NW == 4 ? 2 : 1;
  float xs[KS][8], xr[NR][KS][8];
  Raw8<DT> xe[NR][KS];
  auto load_head = [&](int hh) {
    const int h = hq * A.grp + hh;
    const long long jh = j * A.H + h, tok = at.t0 + (long long)min(own, at.len - 1);
#pragma unroll
    for (int n = 0; n < NR; n++) {
      const bool y = NR == 2 ? n == 0 : down;
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        load8<kF32>(y ? keep.Y : keep.W, (jh * 64 + own) * D + 32 * ks + 8 * g, xr[n][ks]);
        xe[n][ks].load(y ? A.v : B.d_out, tok * (y ? A.vs : A.os) + (long long)h * D + 32 * ks + 8 * g);
      }
    }
#pragma unroll
    for (int ks = 0; ks < KS; ks++) load8<kF32>(keep.S, (jh * D + dk) * D + 32 * ks + 8 * g, xs[ks]);
  };
  const f4 zero = {0, 0, 0, 0};
  f4 dQ[4] = {zero, zero, zero, zero}, dK[4] = {zero, zero, zero, zero};
  // the sums are taken where they stand: left to the end they would hold every term in registers
  auto settle = [](f4& x) { asm volatile("" : "+v"(x)); };
  for (int hh = 0; hh < A.grp; hh++) {
    const int h = hq * A.grp + hh;
    const long long jh = j * A.H + h;
    // opaque again at every phase: addresses and predicates made from the lane are not kept across phases
    // and heads, where they would spill
    auto rd = [&](const char* plane, int rt, int ks) { return *(const h8*)(plane + (rt * KS + ks) * kFrag + lane * 16); };
    auto fresh = [&]() {
      asm("" : "+v"(tid));
      lane = tid & 63;
      c16 = lane & 15;
      g = lane >> 4;
      row = tid / TPR;
      own = 32 * pb + perm_row(c16, pt & 1);
    };
    fresh();
#pragma unroll
    for (int rt = 0; rt < 4; rt++)
#pragma unroll
      for (int i = 0; i < NV; i++) asm volatile("" : "+v"(qv[rt][i]), "+v"(kv[rt][i]));  // stay as they are packed
    load_head(hh);
    const long long sat = (jh * D + dk) * D + 8 * g;
    float al = 1.0f, be = 0.0f;
    if (w == NW - 1 && lane < at.len) {
      const long long th = (at.t0 + (long long)lane) * A.H + h;
      al = A.alpha[th];
      be = A.beta[th];
    }
    ahead();
    __syncthreads();  // the last head's fragments have been read
    const bool live = own < at.len;
    if (down) {  // Y (with V)
      float p = 0.0f;
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        float v[8];
        xe[0][ks].get(v);
#pragma unroll
        for (int e = 0; e < 8; e++) p = fmaf(xr[0][ks][e], v[e], p);
      }
      p = sum_rows(p);
      if (g == 0) sm.yv[own] = p;
      rows_put<D, 2>(xr[0], live, pt, lane, own, sm.in.Y, sm.isY);
    }
    if (up) {  // W and dO
      rows_put<D, 2>(xr[NR - 1], live, pt, lane, own, sm.in.W, sm.isW);
      float x[KS][8];
#pragma unroll
      for (int ks = 0; ks < KS; ks++) xe[NR - 1][ks].get(x[ks]);
      rows_put<D, NPI>(x, live, pt, lane, own, sm.in.O, sm.isO);
    }
    if (w == NW - 1) {
      float p8 = al, s8 = __shfl_down(al, 1);
      s8 = (lane & 7) < 7 ? s8 : 1.0f;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        const float u = __shfl_up(p8, o), d = __shfl_down(s8, o);
        if ((lane & 7) >= o) p8 *= u;
        if ((lane & 7) + o < 8) s8 *= d;
      }
      float p32 = p8, s32 = s8, G = 1.0f, lc = 1.0f;
#pragma unroll
      for (int n = 0; n < 8; n++) {
        const float b = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(p8), 8 * n + 7));
        const int m = lane >> 3;
        if (n < m) G *= b;
        if (n > m) lc *= b;
        if (n < m && (n >> 2) == (m >> 2)) p32 *= b;
        if (n > m && (n >> 2) == (m >> 2)) s32 *= b;
      }
      sm.gate[0][lane] = al;
      sm.gate[1][lane] = p8;
      sm.gate[2][lane] = s8;
      sm.gate[3][lane] = p32;
      sm.gate[4][lane] = s32;
      sm.gate[5][lane] = G * p8;
      sm.gate[6][lane] = lc * s8;
      sm.be[lane] = be;
    }
    // this wave's 16 rows of S0 as column operands
    h8 Sh[KS], Sl[KS];
    float iS;
    {
      float m = 0.0f;
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int e = 0; e < 8; e++) m = fmaxf(m, fabsf(xs[ks][e]));
      const float s = scale_of(col_max(m), iS);
#pragma unroll
      for (int ks = 0; ks < KS; ks++) split8<2>(xs[ks], s, Sh[ks], Sl[ks]);
    }
    ahead();
    float x[KS][8];  // dS1's rows
#pragma unroll
    for (int ks = 0; ks < KS; ks++) load8<kF32>(keep.G, sat + 32 * ks, x[ks]);
    ahead();
    __syncthreads();
    fresh();
    // dQ += G dO S0^T, dK -= G beta Y S0^T; and their products with q_t and k_t
#pragma unroll
    for (int rt = 0; rt < 4; rt++) {
      f4 e1 = zero, e2 = zero;
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        const h8 o = rd(sm.in.O[0], rt, ks), yh = rd(sm.in.Y[0], rt, ks), yl = rd(sm.in.Y[1], rt, ks);
        e1 = mfma(o, Sh[ks], e1);
        e2 = mfma(yh, Sh[ks], e2);
        e1 = mfma(o, Sl[ks], e1);
        e2 = mfma(yh, Sl[ks], e2);
        if constexpr (NPI == 2) e1 = mfma(rd(sm.in.O[NPI - 1], rt, ks), Sh[ks], e1);
        e2 = mfma(yl, Sh[ks], e2);
      }
      const int t0 = 32 * (rt >> 1) + 8 * g + 4 * (rt & 1);
      const f4 io = *(const f4*)&sm.isO[t0] * iS, iy = *(const f4*)&sm.isY[t0] * iS;
      const f4 G = *(const f4*)&sm.gate[5][t0], be4 = *(const f4*)&sm.be[t0];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float a = e1[i] * io[i], b = e2[i] * iy[i];
        dQ[rt][i] = fmaf(G[i], a, dQ[rt][i]);
        dK[rt][i] = fmaf(-G[i] * be4[i], b, dK[rt][i]);
        const float zq = sum16(column(qv, rt, i) * a), zk = sum16(column(kv, rt, i) * b);
        if (c16 == 0) {
          sm.dot[0][w][t0 + i] = zq;
          sm.dot[1][w][t0 + i] = zk;
        }
      }
      settle(dQ[rt]);
      settle(dK[rt]);
      ahead();
    }
    fresh();
    // dK += D W dS1^T; <S0, dS1>
    {
      h8 Gh[KS], Gl[KS];
      float m = 0.0f, cn = 0.0f, iG;
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int e = 0; e < 8; e++) {
          m = fmaxf(m, fabsf(x[ks][e]));
          cn = fmaf(x[ks][e], (float)Sh[ks][e] + (float)Sl[ks][e], cn);
        }
      cn = sum_rows(sum16(cn * iS));
      if (lane == 0) sm.corner[w] = cn;
      const float s = scale_of(col_max(m), iG);
#pragma unroll
      for (int ks = 0; ks < KS; ks++) split8<2>(x[ks], s, Gh[ks], Gl[ks]);
      ahead();
#pragma unroll
      for (int rt = 0; rt < 4; rt++) {
        f4 e3 = zero;
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
          const h8 wh = rd(sm.in.W[0], rt, ks), wl = rd(sm.in.W[1], rt, ks);
          e3 = mfma(wl, Gh[ks], mfma(wh, Gl[ks], mfma(wh, Gh[ks], e3)));
        }
        const int t0 = 32 * (rt >> 1) + 8 * g + 4 * (rt & 1);
        const f4 iw = *(const f4*)&sm.isW[t0] * iG, lc = *(const f4*)&sm.gate[6][t0];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float c = e3[i] * iw[i];
          dK[rt][i] = fmaf(lc[i], c, dK[rt][i]);
          const float yk = sum16(column(kv, rt, i) * c);
          if (c16 == 0) sm.dot[2][w][t0 + i] = yk;
        }
        settle(dK[rt]);
      }
      ahead();
    }
    fresh();
    // pairs: dO W^T and Y W^T (down: [own t][8 s], up: [own s][8 t])
    float pd[2][8], xd[2][8], p1[NW == 4 ? 2 : 1][8], x1[NW == 4 ? 2 : 1][8];
    float(*const pu)[8] = NW == 4 ? p1 : pd;
    float(*const xu)[8] = NW == 4 ? x1 : xd;
    if (down) {
      h8 o[KS][NPI], yh[KS], yl[KS];
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
#pragma unroll
        for (int p = 0; p < NPI; p++) o[ks][p] = rd(sm.in.O[p], pt, ks);
        yh[ks] = rd(sm.in.Y[0], pt, ks);
        yl[ks] = rd(sm.in.Y[1], pt, ks);
      }
      const float io = sm.isO[own], iy = sm.isY[own];
#pragma unroll
      for (int nb = 0; nb < 2; nb++) {
        if (nb > pb) continue;
        f4 a[2] = {zero, zero}, b[2] = {zero, zero};
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
          for (int p = 0; p < 2; p++) {
            const h8 wh = rd(sm.in.W[0], 2 * nb + p, ks), wl = rd(sm.in.W[1], 2 * nb + p, ks);
            a[p] = mfma(wl, o[ks][0], mfma(wh, o[ks][0], a[p]));
            if constexpr (NPI == 2) a[p] = mfma(wh, o[ks][NPI - 1], a[p]);
            b[p] = mfma(wl, yh[ks], mfma(wh, yl[ks], mfma(wh, yh[ks], b[p])));
          }
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const float iw = sm.isW[32 * nb + 8 * g + e];
          pd[nb][e] = a[e >> 2][e & 3] * (iw * io);
          xd[nb][e] = b[e >> 2][e & 3] * (iw * iy);
        }
      }
    }
    if (up) {
      h8 wh[KS], wl[KS];
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        wh[ks] = rd(sm.in.W[0], pt, ks);
        wl[ks] = rd(sm.in.W[1], pt, ks);
      }
      const float iw = sm.isW[own];
#pragma unroll
      for (int nb = 0; nb < 2; nb++) {
        if (nb < pb) continue;
        f4 a[2] = {zero, zero}, b[2] = {zero, zero};
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
          for (int p = 0; p < 2; p++) {
            const h8 o = rd(sm.in.O[0], 2 * nb + p, ks);
            const h8 yh = rd(sm.in.Y[0], 2 * nb + p, ks), yl = rd(sm.in.Y[1], 2 * nb + p, ks);
            a[p] = mfma(o, wl[ks], mfma(o, wh[ks], a[p]));
            if constexpr (NPI == 2) a[p] = mfma(rd(sm.in.O[NPI - 1], 2 * nb + p, ks), wh[ks], a[p]);
            b[p] = mfma(yl, wh[ks], mfma(yh, wl[ks], mfma(yh, wh[ks], b[p])));
          }
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int t = 32 * nb + 8 * g + e;
          pu[nb][e] = a[e >> 2][e & 3] * (sm.isO[t] * iw);
          xu[nb][e] = b[e >> 2][e & 3] * (sm.isY[t] * iw);
        }
      }
    }
    ahead();
    h8 fk[2][NPI], fq[2][NPI];  // this wave's rows of K^T and Q^T, for the products after the next barrier
    if constexpr (!GradSmem<D, DT>::keep_kq)
#pragma unroll
      for (int n = 0; n < 2 * NPI; n++) {
        fk[n / NPI][n % NPI] = kq_at(0, n / NPI, n % NPI);
        fq[n / NPI][n % NPI] = kq_at(1, n / NPI, n % NPI);
      }
    ahead();
    __syncthreads();  // the planes are free: fragments and pairs in their place
    fresh();
    {
      const int po = own & 31, og = po >> 3, oi = po & 7;  // own token: place in its block, group, place in that
      const float* const ga = &sm.gate[0][32 * pb + 8 * g];
      auto mid = [&](bool dn) {
        const int lo = dn ? g : og, hi = dn ? og : g;
        float m = sm.gate[dn ? 1 : 2][own];
        if (lo == 0 && hi > 1) m *= sm.gate[1][32 * pb + 15];
        if (lo <= 1 && hi == 3) m *= sm.gate[1][32 * pb + 23];
        return m;
      };
      // a fragment pair and its rows' scale
      auto put = [&](float (*v)[8], int which, bool lower) {
        float m = 0.0f, inv;
#pragma unroll
        for (int nb = 0; nb < 2; nb++)
          if (lower ? nb <= pb : nb >= pb)
#pragma unroll
            for (int e = 0; e < 8; e++) m = fmaxf(m, fabsf(v[nb][e]));
        const float s = scale_of(col_max(m), inv);
        if (g == 0) sm.m.iF[which][own] = inv;
#pragma unroll
        for (int nb = 0; nb < 2; nb++)
          if (lower ? nb <= pb : nb >= pb) {
            h8 hi, lo;
            split8<2>(v[nb], s, hi, lo);
            char* const dst = sm.m.fr + 2 * (6 * which + (lower ? tri_frag(pt, nb) : up_frag(pt, nb))) * kFrag + lane * 16;
            *(h8*)dst = hi;
            *(h8*)(dst + kFrag) = lo;
          }
      };
      if (down) {
        const float be_own = sm.be[own], m = mid(true), pre = sm.gate[3][own];
        float rx = 0.0f;
#pragma unroll
        for (int nb = 0; nb < 2; nb++) {
          if (nb > pb) continue;
          float kk[8], qk[8];  // k_t.k_s and q_t.k_s
          load8<kF32>(sm.pairs[pt], (4 * nb * kFrag + lane * 32) / 4, kk);
          load8<kF32>(sm.pairs[pt], ((4 * nb + 2) * kFrag + lane * 32) / 4, qk);
          float c = 1.0f;
#pragma unroll
          for (int e = 7; e >= 0; e--) {
            const int s = 32 * nb + 8 * g + e;
            float l;
            bool on = true, strict = true;  // s <= t, s < t
            if (nb < pb) {
              l = pre * sm.gate[4][s];
            } else {
              on = 8 * g + e <= po;
              strict = 8 * g + e < po;
              l = g < og ? m * sm.gate[2][s] : c;
              if (e <= oi) c *= ga[e];
            }
            const float p = on ? pd[nb][e] : 0.0f, y = strict ? xd[nb][e] : 0.0f, ik = sm.isk[s];
            l = on ? l : 0.0f;
            const float by = be_own * y;
            sm.m.xT[s][own] = fmaf(p, qk[e], -by * kk[e]);
            rx = fmaf(y, l * kk[e], rx);
            pd[nb][e] = p * l * ik;
            xd[nb][e] = -by * l * ik;
          }
        }
        rx = sum_rows(rx);
        if (g == 0) sm.rowx[own] = rx;
        put(pd, 0, true);
        put(xd, 1, true);
      }
      if (up) {
        const float m = mid(false), suf = sm.gate[4][own];
#pragma unroll
        for (int nb = 0; nb < 2; nb++) {
          if (nb < pb) continue;
          float c = 1.0f;
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const int t = 32 * nb + 8 * g + e;
            float l;
            bool on = true, strict = true;  // t >= s, t > s
            if (nb > pb) {
              l = suf * sm.gate[3][t];
            } else {
              on = 8 * g + e >= po;
              strict = 8 * g + e > po;
              if (e > oi) c *= ga[e];
              l = g > og ? m * sm.gate[1][t] : c;
            }
            l = on ? l : 0.0f;
            const float p = on ? pu[nb][e] : 0.0f, y = strict ? xu[nb][e] : 0.0f;
            pu[nb][e] = p * l * sm.isq[t];
            xu[nb][e] = -sm.be[t] * y * l * sm.isk[t];
          }
        }
        put(pu, 2, false);
        put(xu, 3, false);
      }
      if (w == 0) {
        float zq = 0.0f, zk = 0.0f, yk = 0.0f;
#pragma unroll
        for (int v = 0; v < NW; v++) zq += sm.dot[0][v][lane], zk += sm.dot[1][v][lane], yk += sm.dot[2][v][lane];
        sm.z[lane] = fmaf(-sm.be[lane], zk, zq);
        sm.y[lane] = yk;
        sm.yv[lane] = fmaf(-sm.gate[5][lane], zk, sm.yv[lane]);
      }
    }
    __syncthreads();
    fresh();
    // dQ += N K, dK += (Zd + Zu) K + N^T Q
    {
      if constexpr (GradSmem<D, DT>::keep_kq)
#pragma unroll
        for (int i = 0; i < 2 * NPI; i++) {
          fk[i / NPI][i % NPI] = *(const h8*)(sm.kq[w] + i * kFrag + lane * 16);
          fq[i / NPI][i % NPI] = *(const h8*)(sm.kq[w] + (2 * NPI + i) * kFrag + lane * 16);
        }
      f4 n[4], d[4], t[4], u[4];
#pragma unroll
      for (int r = 0; r < 4; r++) n[r] = d[r] = t[r] = u[r] = zero;
      auto fr = [&](int which, int f, int p) { return *(const h8*)(sm.m.fr + (2 * (6 * which + f) + p) * kFrag + lane * 16); };
#pragma unroll
      for (int ks = 0; ks < 2; ks++) {
        const h8 *k = fk[ks], *q = fq[ks];
#pragma unroll
        for (int r = 0; r < 4; r++) {
          if (ks <= r >> 1) {
            const int f = tri_frag(r, ks);
            const h8 a = fr(0, f, 0), b = fr(1, f, 0);
            n[r] = mfma(fr(0, f, 1), k[0], mfma(a, k[0], n[r]));
            d[r] = mfma(fr(1, f, 1), k[0], mfma(b, k[0], d[r]));
            if constexpr (NPI == 2) {
              n[r] = mfma(a, k[NPI - 1], n[r]);
              d[r] = mfma(b, k[NPI - 1], d[r]);
            }
          }
          if (ks >= r >> 1) {
            const int f = up_frag(r, ks);
            const h8 a = fr(2, f, 0), b = fr(3, f, 0);
            t[r] = mfma(fr(2, f, 1), q[0], mfma(a, q[0], t[r]));
            u[r] = mfma(fr(3, f, 1), k[0], mfma(b, k[0], u[r]));
            if constexpr (NPI == 2) {
              t[r] = mfma(a, q[NPI - 1], t[r]);
              u[r] = mfma(b, k[NPI - 1], u[r]);
            }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const int t0 = 32 * (r >> 1) + 8 * g + 4 * (r & 1);
        const f4 i0 = *(const f4*)&sm.m.iF[0][t0], i1 = *(const f4*)&sm.m.iF[1][t0];
        const f4 i2 = *(const f4*)&sm.m.iF[2][t0], i3 = *(const f4*)&sm.m.iF[3][t0];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          dQ[r][i] = fmaf(i0[i], n[r][i], dQ[r][i]);
          dK[r][i] = fmaf(i1[i], d[r][i], fmaf(i3[i], u[r][i], fmaf(i2[i], t[r][i], dK[r][i])));
        }
        settle(dQ[r]);
        settle(dK[r]);
      }
    }
    fresh();
    // gates: dalpha_r = sum over t >= r of L[t,r] F_r[t] with F_r[t] = sum over s < r of x[t,s] L[r-1,s]
    // (the state before the chunk as s = -1, the state behind it as one more t).  Lane t; a wave takes groups
    // of 8 gates: F at a group's first by a sum, then F_{r+1} = a_r F_r + x[t,r].
    {
      const int tg = lane >> 3;
      float corner = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; v++) corner += sm.corner[v];
      const float zl = sm.z[lane], yl = sm.y[lane], p8 = sm.gate[1][lane], s8 = sm.gate[2][lane];
#pragma unroll
      for (int q = 0; q < 8 / NW; q++) {
        const int n = (8 / NW) * w + q, r0 = 8 * n;
        float v = lane < r0 ? s8 : 0.0f, u = tg > n ? p8 : 0.0f;  // L[r0 - 1, s] and L[t, r0 + 7]
#pragma unroll
        for (int m = 1; m < 7; m++) {
          const float b = sm.gate[1][8 * m + 7];
          if (m > tg && m < n) v *= b;
          if (m > n && m < tg) u *= b;
        }
        const float G = n ? sm.gate[5][n ? r0 - 1 : 0] : 1.0f;
        float C = fmaf(corner, G, sum_rows(sum16(lane < r0 ? yl * v : 0.0f)));
        float f0 = zl * G, f1 = 0.0f;
#pragma unroll 4
        for (int s = 0; s < r0; s += 2) {
          f0 = fmaf(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), s)), sm.m.xT[s][lane], f0);
          f1 = fmaf(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), s + 1)), sm.m.xT[s + 1][lane], f1);
        }
        float F = f0 + f1;
        float l[8], c = 1.0f;  // L[lane, r0 + e]
#pragma unroll
        for (int e = 7; e >= 0; e--) {
          const bool in = tg == n && e <= (lane & 7);
          l[e] = tg > n ? u * sm.gate[2][r0 + e] : in ? c : 0.0f;
          if (in) c *= sm.gate[0][r0 + e];
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int r = r0 + e;
          const float a = sm.gate[0][r];
          const float d = sum_rows(sum16(lane >= r ? l[e] * F : 0.0f));
          if (lane == 0) sm.da[r] = fmaf(sm.gate[6][r], C, d);
          F = fmaf(a, F, sm.m.xT[r][lane]);
          C = fmaf(a, C, sm.y[r]);
        }
      }
    }
    __syncthreads();
    if (tid < at.len) {
      const long long th = (at.t0 + (long long)tid) * A.H + h;
      B.dalpha[th] = sm.da[tid];
      B.dbeta[th] = sm.yv[tid] - sm.rowx[tid];
    }
  }
  // dQ and dK to rows through LDS
  row = tid / TPR;
#pragma unroll
  for (int which = 0; which < 2; which++) {
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
      for (int i = 0; i < 4; i++) sm.out[32 * (r >> 1) + 8 * g + 4 * (r & 1) + i][dk] = which ? dK[r][i] : dQ[r][i];
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
hipError_t launch(const GradArgs& b, hipStream_t s) {
  const SeqArgs& a = b.f;
  const size_t n = (size_t)chunk_slots(a.T, a.N) * a.H;
  Keep keep;
  keep.S = (float*)(a.ws + fixed_bytes<D, DT>(a));
  keep.G = keep.S + n * D * D;
  keep.W = keep.G + n * D * D;
  keep.Y = keep.W + n * 64 * D;
  const dim3 slots((unsigned)chunk_slots(a.T, a.N), a.Hq);
  if (a.T > 0) {
    hipLaunchKernelGGL((k_chunk_prep<D, DT, LayB<D, DT>>), slots, dim3(256), 0, s, a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  const hipError_t rc = with_state_waves<D, DT>(a, 1, [&](auto nw) {
    constexpr int NW = nw.value;
    const dim3 tiles(workgroups<NW>(a, D));
    if (a.T > 0) {
      SeqArgs quiet = a;
      quiet.status = nullptr;  // flags are raised once, by the reverse pass
      hipLaunchKernelGGL((k_chunk_state<D, DT, NW, LayB<D, DT>, kKeep>), tiles, dim3(64 * NW), 0, s, quiet, keep.S, keep.W, Segs{});
      if (hipError_t e = hipGetLastError()) return e;
    }
    hipLaunchKernelGGL((k_chunk_reverse<D, DT, NW>), tiles, dim3(64 * NW), 0, s, b, keep);
    return hipGetLastError();
  });
  if (rc != hipSuccess || a.T == 0) return rc;
  hipLaunchKernelGGL((k_chunk_grad<D, DT>), slots, dim3(4 * D), 0, s, b, keep);
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
