// stepq_chunk.h -- device pieces of the chunked delta rule (forward and gradient): matrix-core operands
// in binary16 planes, the chunk's local matrices, and the workspace's layout.
//
// Mathematics of a chunk of C = 64 tokens (GDN; a_t gates, L[t,s] = prod_{s<r<=t} a_r, G_t = L[t,-1]):
//   A = strict-lower(diag(beta) (L o K K^T)),  T = (I + A)^-1,  P = lower(L o Q K^T)
//   R = V - diag(G) K S0,  W = T diag(beta) R            (W_t = beta_t e_t, the weighted errors)
//   O = diag(G) Q S0 + P W,             S1 = G_C S0 + K^T diag(L[C,.]) W
// L is formed by running products, never by quotients or logarithms, so a gate may be zero, negative
// or above one.
//
// Operands: v_mfma_f32_16x16x32_f16 with binary32 accumulation.  An operand row (A side) or column (B
// side) is scaled by a power of two that puts its largest magnitude into [2^11, 2^12), then written as
// x = hi + lo with hi, lo binary16: 22 bits of the largest element.  (The state, and what is added to it, have
// the units of the state's column instead: see `fit`.)  bfloat16 and binary16 inputs need hi
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
// The readout's operands (the state, P and W) are single planes for a bfloat16 output, 11 bits of every term
// against the 8 that the output keeps: 8 ragged prompts of 16,381 tokens x 48 heads 445 us a call, with two planes
// 479.  An output's error grows from 1.652e-3 (its rounding alone) to 1.678e-3 (relative 2-norms, 704 tokens),
// 12% of the values are the next one up or down; one that cancels to a tenth of its terms has twice its error.
template <int DT> constexpr int kOutPlanes = DT == kBF16 ? 1 : 2;

// Workspace of the forward pass.  Key block (chunk slot, key head): K, K^T and Q fragments.  Head block
// (chunk slot, value head): T diag(beta) and P fragments and the row tables.
template <int D, int DT> struct LayF {
  static constexpr bool grad = false;
  static constexpr int NF = D / 8;                       // fragments of K, K^T or Q (one plane)
  static constexpr int NPI = kInPlanes<DT>, NPO = kOutPlanes<DT>;
  static constexpr int offK = 0, offKT = NPI * NF * kFrag, offQ = 2 * NPI * NF * kFrag;
  static constexpr int key = 3 * NPI * NF * kFrag, offKK = 0, offQK = 0;  // none
  static constexpr int offT = 0, offP = 2 * kTri * kFrag, offTab = offP + NPO * kTri * kFrag;
  static constexpr int offTt = offTab;  // none
  static constexpr int tab = 1280, head = offTab + tab;  // bytes of the tables that the pass reads
};
// Workspace of the gradient.  Q^T in Q's place, K K^T [t][s] and Q K^T [s][t] (binary32, t >= s within 32-row
// blocks) behind the fragments; T, T^T, P^T (two planes each).  Then, per chunk slot and value head in binary32: the
// states before and the states' gradients behind every chunk, W and Y.
template <int D, int DT> struct LayB {
  static constexpr bool grad = true;
  static constexpr int NF = D / 8, NPI = kInPlanes<DT>, NPO = 2;
  static constexpr int offK = 0, offKT = NPI * NF * kFrag, offQ = 2 * NPI * NF * kFrag;
  static constexpr int offKK = 3 * NPI * NF * kFrag, offQK = offKK + 64 * 64 * 4;
  static constexpr int key = offQK + 64 * 64 * 4;
  static constexpr int offT = 0, offTt = 2 * kTri * kFrag, offP = 4 * kTri * kFrag, offTab = 6 * kTri * kFrag;
  static constexpr int head = offTab + 4096, tab = 2048;
};
// Row tables (64 floats each); inverse operand scales are folded in.
constexpr int kTabU = 0;     // G / scale of K's row (gradient: times beta)
constexpr int kTabQ = 64;    // G / scale of Q's row
constexpr int kTabP = 128;   // 1 / scale of P's (gradient: P^T's) row
constexpr int kTabD = 192;   // L[C, s] / scale of K's row (K^T's column)
constexpr int kTabG = 256;   // [62] = 1 / scale of T (forward), [63] = G_C
constexpr int kTabT = 320;   // 1 / scale of T's row              (gradient from here on)
constexpr int kTabB = 384;   // beta (0 behind the sequence's end)
constexpr int kTabTt = 448;  // 1 / scale of T^T's row
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

// Maximum over the four lanes of a column (lanes that differ in bits 4 and 5), without LDS.
__device__ __forceinline__ float col_max(float x) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// 8 binary32 values times s as hi (and lo) planes.
template <int NP>
__device__ __forceinline__ void split8(const float* x, float s, h8& hi, h8& lo) {
#pragma unroll
  for (int i = 0; i < 8; i++) {
    hi[i] = (_Float16)(x[i] * s);
    if constexpr (NP == 2) lo[i] = (_Float16)fmaf(x[i], s, -(float)hi[i]);  // one mixed-precision fma
  }
}

// Largest magnitude of a column's accumulator tiles.
template <int NT>
__device__ __forceinline__ float tiles_max(const f4* x) {
  float m = 0.0f;
#pragma unroll
  for (int t = 0; t < NT; t++)
#pragma unroll
    for (int i = 0; i < 4; i++) m = fmaxf(m, fabsf(x[t][i]));
  return col_max(m);
}
// Accumulator row tiles x[0 .. 2 NB - 1] (16 rows each, one column a lane) times s -> B operands of NB
// 32-row steps.  SCALED: s is 1.
template <int NB, int NP, bool SCALED = false>
__device__ __forceinline__ void to_planes(const f4* x, float s, h8* hi, h8* lo) {
#pragma unroll
  for (int b = 0; b < NB; b++) {
    if (SCALED) asm("" : "+v"(s));  // an opaque 1: keeps the fma below, which rounds to binary16 by itself
    const float y[8] = {x[2 * b][0], x[2 * b][1], x[2 * b][2], x[2 * b][3],
                        x[2 * b + 1][0], x[2 * b + 1][1], x[2 * b + 1][2], x[2 * b + 1][3]};
#pragma unroll
    for (int i = 0; i < 8; i++) {
      hi[b][i] = (_Float16)(SCALED ? y[i] : y[i] * s);
      if constexpr (NP == 2) lo[b][i] = (_Float16)fmaf(y[i], s, -(float)hi[b][i]);
    }
  }
}
// The same with the column's own scale; returns the inverse scale.
template <int NB, int NP>
__device__ __forceinline__ float to_operand(const f4* x, h8* hi, h8* lo) {
  float inv;
  const float s = scale_of(tiles_max<2 * NB>(x), inv);
  to_planes<NB, NP>(x, s, hi, lo);
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
// Bytes [from, to) (multiples of 1 KiB) of src to LDS offset `at` + from, the pieces over NW waves.
template <int NW>
__device__ __forceinline__ void copy_block(const char* src, unsigned at, int from, int to, int w, unsigned lane16) {
  src += from + w * kFrag;
  at += from + w * kFrag;
#pragma unroll
  for (int i = 0; i < to - from; i += NW * kFrag)
    if (i + NW * kFrag <= to - from || i + w * kFrag < to - from) copy_to_lds(src + i, at + i, lane16);
}
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// The units of a column's tiles x (the column is unit * x): its largest magnitude m (in units) in [2^13, 2^14)
// after `fit`, in [2^12, 2^15] while it is left alone.  Above 2^16 it would not be a binary16; far below, the
// update would be coarse: y of the update K^T y is written in these units as two binary16 planes, off by
// max(2^-22 |y|, 2^-25), and K's planes (below 2^12) raise that to 2^-13 units a token -- 2^-25 of a column's
// largest.  (Left alone down to 1, states of size one kept 12 bits.)
// A column of zeros has the least unit, so that whatever is added first sets it.  Columns below 2^-98 (3e-30) stay at
// the least unit and lose bits as they shrink.
constexpr float kLeastUnit = 0x1p-110f;
template <int NT>
__device__ __forceinline__ void fit(f4* x, float& unit, float& m) {
  if (!__any(m > 0x1p15f || (m < 0x1p12f && unit > kLeastUnit))) return;
  float inv, f = 1.0f, to = kLeastUnit;
  if (m > 0.0f) {
    (void)scale_of(m, inv);
    to = fmaxf(unit * (0.25f * inv), kLeastUnit);
    f = unit / to;  // both powers of two
  }
#pragma unroll
  for (int t = 0; t < NT; t++) x[t] *= f;
  m *= f;
  unit = to;
}
// The column becomes G x + K^T y, with y's largest magnitude my (not in units): x times G, and in units that suit
// the larger of the two, where K's planes make K^T y about 2^11 my.  It may be far below what x was before G.
// Left alone down to 2^10 units (2^-23 a token; 64 that err independently, on K's mean instead of its largest
// elements, 2^-22.4): at 2^12 an ordinary chunk's gates moved the units every time, for no measurable bit
// (8 ragged prompts of 16,381 tokens x 48 heads: 460 us a call against 450).
template <int NT>
__device__ __forceinline__ void fit_sum(f4* x, float& unit, float m, float G, float my) {
#pragma unroll
  for (int t = 0; t < NT; t++) x[t] *= G;
  const float top = fmaxf(0x1p11f * my, fabsf(G) * m * unit);
  const bool off = my > unit * 0x1p14f || (top < unit * 0x1p10f && top > 0.0f && unit > kLeastUnit);
  if (!__any(off)) return;
  float inv, to = unit;
  if (off) {
    (void)scale_of(top, inv);
    to = fmaxf(fmaxf(0.25f * inv, kLeastUnit), unit * 0x1p-100f);
  }
  const float f = unit / to;
#pragma unroll
  for (int t = 0; t < NT; t++) x[t] *= f;
  unit = to;
}
// Keeps the LDS reads above it above the arithmetic below it: fragments are read one product ahead.
__device__ __forceinline__ void ahead() { __builtin_amdgcn_sched_barrier(0); }

// Rows of a chunk in accumulator order: x[rt][i] = row 32 (rt >> 1) + 8 g + 4 (rt & 1) + i, this lane's
// column.  Through a buffer descriptor that ends behind the chunk's last token: rows behind it read as
// zero and are not written, without a branch or a comparison, and nothing is converted before it is used,
// so all loads are in flight at once.
template <int DT>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const void* p, long long row, long long stride, int head_col, int D, int len) {
  constexpr int es = DT == kF32 ? 4 : 2;
  return __builtin_amdgcn_make_buffer_rsrc((char*)p + (row * stride + head_col) * es, 0,
                                           (int)((unsigned)(len - 1) * (unsigned)stride * es + D * es), 0x00020000);
}
template <int DT>
__device__ __forceinline__ float raw_value(unsigned x) {
  if constexpr (DT == kF32) return __uint_as_float(x);
  else return e_f<DT>((unsigned short)x);
}
template <int DT>
struct Rows {
  static constexpr int es = DT == kF32 ? 4 : 2;
  unsigned first;  // byte offset of row 8 g
  int step;        // bytes from row to row
  __device__ Rows(long long stride, int col, int g) : first((unsigned)((8 * g * (int)stride + col) * es)), step((int)stride * es) {}
  __device__ unsigned off(int rt, int i) const { return first + (unsigned)((32 * (rt >> 1) + 4 * (rt & 1) + i) * step); }
  __device__ void load(__amdgpu_buffer_rsrc_t r, unsigned (*x)[4]) const {
#pragma unroll
    for (int rt = 0; rt < 4; rt++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        if constexpr (DT == kF32) x[rt][i] = __builtin_amdgcn_raw_buffer_load_b32(r, off(rt, i), 0, 0);
        else x[rt][i] = (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, off(rt, i), 0, 0);
      }
  }
};

// The same for a wave's 16 neighbouring columns, 16 bytes a lane: memory instructions that move 2 bytes a
// lane keep the address unit busy for as long as ones that move 16 (16 loads of V and 16 stores of O a chunk
// took 3,000 of the chunk pass's 11,600 cycles).  Rows and lanes change places through a piece of LDS of
// the wave's own, a pass of 32 rows (16-bit types) or one 16-row tile (binary32) at a time; pitches keep the
// four lane groups on different banks.
template <int DT>
struct Slice {
  static constexpr bool F = DT == kF32;
  static constexpr int es = F ? 4 : 2, NL = F ? 4 : 2, lr = F ? 4 : 2;  // passes of 64 rows, lanes a row
  static constexpr int pitch = F ? 80 : 40, bytes = 1280, TP = F ? 1 : 2;  // tiles a pass
  typedef unsigned u4 __attribute__((ext_vector_type(4)));
  typedef unsigned u2 __attribute__((ext_vector_type(2)));
  unsigned first;   // byte offset of the lane's place in a pass
  int row;          // bytes of a row
  char *put, *get;  // the lane's places in the piece: 16 bytes of a row; its column in its first row
  // col0: the wave's first column
  __device__ Slice(char* piece, long long stride, int col0, int lane)
      : first((unsigned)(((F ? perm_row(lane / lr, 0) : lane / lr) * (int)stride + col0) * es + (lane % lr) * 16)),
        row((int)stride * es),
        put(piece + (lane / lr) * pitch + (lane % lr) * 16),
        get(piece + (F ? 4 : 8) * (lane >> 4) * pitch + (lane & 15) * es) {}
  __device__ unsigned off(int n) const { return first + (unsigned)((F ? 32 * (n >> 1) + 4 * (n & 1) : 32 * n) * row); }
  __device__ void load(__amdgpu_buffer_rsrc_t r, u4* x) const {
#pragma unroll
    for (int n = 0; n < NL; n++) x[n] = __builtin_amdgcn_raw_buffer_load_b128(r, off(n), 0, 0);
  }
  __device__ void to_acc(const u4* x, f4* y) const {
#pragma unroll
    for (int n = 0; n < NL; n++) {
      *(u2*)put = u2{x[n][0], x[n][1]};
      *(u2*)(put + 8) = u2{x[n][2], x[n][3]};
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int p = 0; p < TP; p++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          if constexpr (F) y[n][i] = *(const float*)(get + i * pitch);
          else y[TP * n + p][i] = e_f<DT>(*(const unsigned short*)(get + (4 * p + i) * pitch));
        }
      __builtin_amdgcn_wave_barrier();
    }
  }
  // a pass: TP tiles into the piece, then 16 bytes a lane
  __device__ u4 gather(const f4* y) const {
#pragma unroll
    for (int p = 0; p < TP; p++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        if constexpr (F) *(float*)(get + i * pitch) = y[p][i];
        else *(unsigned short*)(get + (4 * p + i) * pitch) = f_e<DT>(y[p][i]);
      }
    __builtin_amdgcn_wave_barrier();
    const u2 a = *(const u2*)put, b = *(const u2*)(put + 8);
    __builtin_amdgcn_wave_barrier();
    return u4{a[0], a[1], b[0], b[1]};
  }
  __device__ void store(__amdgpu_buffer_rsrc_t r, const f4* y) const {  // 64 rows
#pragma unroll
    for (int n = 0; n < NL; n++) __builtin_amdgcn_raw_buffer_store_b128(gather(y + TP * n), r, off(n), 0, 0);
  }
  // NT row tiles of a packed binary32 matrix (this slice made with its stride), all rows
  template <int NT>
  __device__ void load_all(const float* src, f4* y) const {
    static_assert(F);
    u4 x[NT];
#pragma unroll
    for (int n = 0; n < NT; n++) x[n] = *(const u4*)((const char*)src + off(n));
#pragma unroll
    for (int n = 0; n < NT; n += NL) to_acc(x + n, y + n);
  }
  // NT row tiles times s to the rows of a packed binary32 matrix (this slice made with its stride), all rows
  template <int NT>
  __device__ void store_all(float* dst, const f4* y, float s) const {
    static_assert(F);
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const f4 z = y[n] * s;
      *(u4*)((char*)dst + off(n)) = gather(&z);
    }
  }
};

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
  if (c * kChunk >= t1 - t0 || t1 - t0 < A.split) return false;
  at.c = (int)c;
  at.t0 = t0 + (int)c * kChunk;
  at.len = t1 - at.t0 < kChunk ? t1 - at.t0 : kChunk;
  return true;
}

}  // namespace dlt
}  // namespace stepq
