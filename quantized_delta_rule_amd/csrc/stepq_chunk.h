// stepq_chunk.h -- device pieces of the chunked delta rule (forward and gradient): matrix-core operands
// in binary16 planes, the chunk's local matrices, and the workspace's layout.
//
// Mathematics of a chunk of C = 64 tokens (GDN; a_t gates, L[t,s] = prod_{s<r<=t} a_r, G_t = L[t,-1]):
//   A = strict-lower(diag(beta) (L o K K^T)),  T = (I + A)^-1,  P = lower(L o Q K^T)
//   R = diag(beta) (V - diag(G) K S0),  W = T R        (W_t = beta_t e_t, the weighted errors)
//   O = diag(G) Q S0 + P W,             S1 = G_C S0 + K^T diag(L[C,.]) W
// L is formed by running products, never by quotients or logarithms, so a gate may be zero, negative
// or above one.
//
// Operands: v_mfma_f32_16x16x32_f16 with binary32 accumulation.  An operand row (A side) or column (B
// side) is scaled by a power of two that puts its largest magnitude into [2^11, 2^12), then written as
// x = hi + lo with hi, lo binary16: 22 bits of the largest element.  bfloat16 and binary16 inputs need hi
// alone (an element keeps all its bits down to 2^-26 of its row's largest).  A product of two pairs
// takes hi hi + hi lo + lo hi; the dropped lo lo is 2^-22 of the product.  Scales are undone exactly on
// the accumulators, whose rows and columns they belong to.
//
// Layouts of the 16x16x32 instruction (lane l, g = l >> 4): A row l & 15, k = 8 g + i; B column l & 15,
// k = 8 g + i; C/D column l & 15, row 4 g + i.  Row tiles are permuted in pairs: tile p of rows
// 32 b .. 32 b + 31 has operand row r at 32 b + 8 (r >> 2) + 4 p + (r & 3).  Then the two accumulators of
// a pair hold, in lane group g, rows 32 b + 8 g .. + 7 of their column: exactly the B operand of the next
// product over those rows.  W = T R, K^T W and the next chunk's K S run from registers to registers.
#pragma once
#include "stepq_delta.h"

namespace stepq {
namespace dlt {

__device__ __forceinline__ int perm_row(int r, int p) { return 8 * (r >> 2) + 4 * p + (r & 3); }

// Fragment of a 64 x 64 lower-triangular matrix: row tile rt = 2 b + p, k-step ks <= b.
__host__ __device__ constexpr int tri_frag(int rt, int ks) { return rt < 2 ? rt : 2 + 2 * (rt - 2) + ks; }
constexpr int kTri = 6;
constexpr int kFrag = 1024;  // bytes of one fragment plane: 64 lanes x 8 binary16

template <int DT> constexpr int kInPlanes = DT == kF32 ? 2 : 1;   // q, k, v, d_out as operands
template <int DT> constexpr int kOutPlanes = DT == kBF16 ? 1 : 2; // operands of 16-bit outputs only

// Workspace of the forward pass.  Key block (chunk slot, key head): K, K^T and Q fragments.  Head block
// (chunk slot, value head): T and P fragments and the row tables.
template <int D, int DT> struct LayF {
  static constexpr bool grad = false;
  static constexpr int NF = D / 8;                       // fragments of K, K^T or Q (one plane)
  static constexpr int NPI = kInPlanes<DT>, NPO = kOutPlanes<DT>;
  static constexpr int offK = 0, offKT = NPI * NF * kFrag, offQ = 2 * NPI * NF * kFrag;
  static constexpr int key = 3 * NPI * NF * kFrag;
  static constexpr int offT = 0, offP = 2 * kTri * kFrag, offTab = offP + NPO * kTri * kFrag;
  static constexpr int offTt = offTab;  // none
  static constexpr int head = offTab + 2048;
};
// Workspace of the gradient.  Q^T in Q's place, K K^T and Q K^T (binary32, row-major, lower tiles) behind
// the fragments; T, T^T, P^T (two planes each).  Then, per chunk slot and value head in binary32: the
// states before and the states' gradients behind every chunk, W and Y.
template <int D, int DT> struct LayB {
  static constexpr bool grad = true;
  static constexpr int NF = D / 8, NPI = kInPlanes<DT>, NPO = 2;
  static constexpr int offK = 0, offKT = NPI * NF * kFrag, offQ = 2 * NPI * NF * kFrag;
  static constexpr int offKK = 3 * NPI * NF * kFrag, offQK = offKK + 64 * 64 * 4;
  static constexpr int key = offQK + 64 * 64 * 4;
  static constexpr int offT = 0, offTt = 2 * kTri * kFrag, offP = 4 * kTri * kFrag, offTab = 6 * kTri * kFrag;
  static constexpr int head = offTab + 4096;
};
// Row tables (64 floats each); inverse operand scales are folded in.
constexpr int kTabU = 0;     // beta G / scale of K's row
constexpr int kTabB = 64;    // beta (0 behind the sequence's end)
constexpr int kTabT = 128;   // 1 / scale of T's row
constexpr int kTabQ = 192;   // G / scale of Q's row
constexpr int kTabP = 256;   // 1 / scale of P's (gradient: P^T's) row
constexpr int kTabD = 320;   // L[C, s] / scale of K's row (K^T's column)
constexpr int kTabG = 384;   // G; [63] = G_C
constexpr int kTabTt = 448;  // 1 / scale of T^T's row            (gradient from here on)
constexpr int kTabL = 512;   // L[C, s]
constexpr int kTabIK = 576;  // 1 / scale of K's row
constexpr int kTabIQ = 640;  // 1 / scale of Q's row

// Fragment of a 64 x 64 upper-triangular matrix: row tile rt = 2 b + p, k-step ks >= b.
__host__ __device__ constexpr int up_frag(int rt, int ks) { return rt < 2 ? 2 * rt + ks : 2 + rt; }

template <class Y>
__host__ __device__ inline long long key_bytes(const SeqArgs& a) {
  return chunk_slots(a.T, a.N) * a.Hq * Y::key;
}
template <class Y>
__host__ __device__ inline long long head_bytes(const SeqArgs& a) {
  return chunk_slots(a.T, a.N) * a.H * Y::head;
}

// Power of two that brings magnitude m into [2^11, 2^12), and its inverse.  Zero, subnormal and
// non-finite m get the nearest scale whose inverse is normal too.
__device__ __forceinline__ float scale_of(float m, float& inv) {
  int e = 265 - (int)((__float_as_uint(m) >> 23) & 255u);
  e = e > 253 ? 253 : e;
  inv = __uint_as_float((unsigned)(254 - e) << 23);
  return __uint_as_float((unsigned)e << 23);
}

__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// 8 binary32 values times s as hi (and lo) planes.
template <int NP>
__device__ __forceinline__ void split8(const float* x, float s, h8& hi, h8& lo) {
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float y = x[i] * s;
    hi[i] = (_Float16)y;
    if constexpr (NP == 2) lo[i] = (_Float16)(y - (float)hi[i]);
  }
}

// Accumulator row tiles x[0 .. 2 NB - 1] (16 rows each, one column a lane) -> B operands of NB 32-row
// steps, with the column's scale; returns the inverse scale.
template <int NB, int NP>
__device__ __forceinline__ float to_operand(const f4* x, h8* hi, h8* lo) {
  float m = 0.0f;
#pragma unroll
  for (int t = 0; t < 2 * NB; t++)
#pragma unroll
    for (int i = 0; i < 4; i++) m = fmaxf(m, fabsf(x[t][i]));
  m = fmaxf(m, __shfl_xor(m, 16));
  m = fmaxf(m, __shfl_xor(m, 32));
  float inv;
  const float s = scale_of(m, inv);
#pragma unroll
  for (int b = 0; b < NB; b++) {
    const float y[8] = {x[2 * b][0], x[2 * b][1], x[2 * b][2], x[2 * b][3],
                        x[2 * b + 1][0], x[2 * b + 1][1], x[2 * b + 1][2], x[2 * b + 1][3]};
    split8<NP>(y, s, hi[b], lo[b]);
  }
  return inv;
}

// Copies 1 KiB (16 bytes a lane) from memory straight into LDS, without registers and without a wait: the
// reader waits for vmcnt 0 and then for a barrier.  In assembly because the compiler would otherwise wait
// before the next LDS read of any buffer; there is no output register that could be reused too early.
// src and at (an LDS byte offset) are uniform, lane16 = 16 * lane.
__device__ __forceinline__ void copy_to_lds(const char* src, unsigned at, unsigned lane16) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(lane16), "s"(src) : "memory", "m0");
}
__device__ __forceinline__ unsigned lds_offset(const void* p) {
  return __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)(__attribute__((address_space(3))) const char*)p);
}
// `bytes` (a multiple of 1 KiB) from src to LDS offset `at`, the pieces over NW waves.
template <int NW>
__device__ __forceinline__ void copy_block(const char* src, unsigned at, int bytes, int w, unsigned lane16) {
  src += w * kFrag;
  at += w * kFrag;
#pragma unroll
  for (int i = 0; i < bytes; i += NW * kFrag)
    if (i + NW * kFrag <= bytes || i + w * kFrag < bytes) copy_to_lds(src + i, at + i, lane16);
}
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// Keeps the LDS reads above it above the arithmetic below it: fragments are read one product ahead.
__device__ __forceinline__ void ahead() { __builtin_amdgcn_sched_barrier(0); }

// Rows of a chunk in accumulator order: x[rt][i] = row 32 (rt >> 1) + 8 g + 4 (rt & 1) + i of `base` (the
// chunk's first row, this head's first column), this lane's CT columns as they lie in memory.  Rows
// behind the end (len <= r) read the last row instead and are dropped by the caller: no load sits in a
// branch of its own, and none is converted before it is used, so all are in flight at once.
template <int DT, int CT> struct Raw;
template <> struct Raw<kF32, 1> { float x; };
template <> struct Raw<kF32, 2> { f2 x; };
template <> struct Raw<kBF16, 1> { unsigned x; };  // a register each: pairs would be packed on arrival
template <> struct Raw<kBF16, 2> { us2 x; };
template <> struct Raw<kF16, 1> { unsigned x; };  // a register each: pairs would be packed on arrival
template <> struct Raw<kF16, 2> { us2 x; };
template <int DT, int CT>
__device__ __forceinline__ float raw_value(const Raw<DT, CT>& r, int ct) {
  if constexpr (DT == kF32 && CT == 1) return r.x;
  else if constexpr (DT == kF32) return r.x[ct];
  else if constexpr (CT == 1) return e_f<DT>((unsigned short)r.x);
  else return e_f<DT>(r.x[ct]);
}
template <int DT, int CT>
__device__ __forceinline__ void rows_acc(const char* base, int stride, int len, int col, int g, Raw<DT, CT> (*x)[4]) {
  constexpr int es = DT == kF32 ? 4 : 2;
#pragma unroll
  for (int rt = 0; rt < 4; rt++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int r = min(32 * (rt >> 1) + 8 * g + 4 * (rt & 1) + i, len - 1);
      const char* const p = base + (__umul24(r, stride) + col) * es;
      if constexpr (DT != kF32 && CT == 1) x[rt][i].x = *(const unsigned short*)p;
      else x[rt][i] = *(const Raw<DT, CT>*)p;
    }
}
template <int DT, int CT>
__device__ __forceinline__ void rows_store(char* base, int stride, int len, int col, int g, const float (*x)[4][CT]) {
  constexpr int es = DT == kF32 ? 4 : 2;
  const unsigned lane_off = (unsigned)(8 * g * stride + col) * es;
#pragma unroll
  for (int rt = 0; rt < 4; rt++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int r = 32 * (rt >> 1) + 4 * (rt & 1) + i;
      if (len >= kChunk || r + 8 * g < len)
        storen<DT, CT>(base + (long long)r * stride * es + lane_off, 0, x[rt][i]);
    }
}

// The chunk of chunk slot j: sequence, first token, tokens (<= 64).  False: the slot is empty.
struct ChunkAt {
  int s, t0, len, c;
  long long slot0;  // the sequence's first slot
};
__device__ __forceinline__ long long first_slot(const SeqArgs& A, int s) {
  return A.cu ? (long long)(A.cu[s] >> 6) + s : (long long)s * (A.T / A.N) / kChunk + s;
}
__device__ __forceinline__ bool chunk_at(const SeqArgs& A, long long j, ChunkAt& at) {
  int lo = 0, hi = A.N - 1;  // the last sequence whose first slot is not behind j
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_slot(A, mid) <= j) lo = mid;
    else hi = mid - 1;
  }
  at.s = lo;
  at.slot0 = first_slot(A, lo);
  if (j < at.slot0) return false;
  int t0, t1;
  seq_range(A, lo, t0, t1);
  const long long c = j - at.slot0;
  if (c * kChunk >= t1 - t0) return false;
  at.c = (int)c;
  at.t0 = t0 + (int)c * kChunk;
  at.len = t1 - at.t0 < kChunk ? t1 - at.t0 : kChunk;
  return true;
}

}  // namespace dlt
}  // namespace stepq
