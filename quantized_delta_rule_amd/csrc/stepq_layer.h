// stepq_layer.h -- the operators around the recurrence: short causal convolution (stepq_conv.hip), selective
// state space scan (stepq_scan.hip, stepq_scan_grad.hip), root-mean-square norm (stepq_norm.hip); arguments and
// what their kernels share.  Not part of the public ABI.
#pragma once
#include <type_traits>

#include "stepq_delta.h"

namespace stepq {

constexpr int kE4M3 = 3, kI8 = 4;             // STEPQ_DTYPE_*, the norm's output only
constexpr int kNone = 0, kSilu = 1, kSigmoid = 2;  // STEPQ_ACT_*

struct ConvArgs {
  int dtype, pdtype, C, W, act;
  int N, T;                 // sequences, token rows
  const int* cu;            // [N + 1] token offsets, or nullptr: N sequences of T / N tokens
  int n_slots;
  const int* slots;         // [N] or nullptr
  unsigned* status;
  long long xs, os;         // elements between tokens of x, and of out / d_out
  int sh;                   // tokens of a piece: 2^sh (set by the launch)
  const void* x;
  const void* w;            // [C, W] pdtype
  const void* b;            // [C] or nullptr
  const void* S_in;         // [.., W - 1, C] or nullptr
  void* S_out;
  void* out;
  // gradient
  const void* d_out;
  const void* dS_out;
  void* dx;                 // [T, C] packed
  float* dw;                // [C, W]
  float* db;                // [C] or nullptr
  void* dS_in;
  float* ws;
};
hipError_t launch_conv(const ConvArgs& a, hipStream_t s);
size_t conv_backward_bytes(const ConvArgs& a);
hipError_t launch_conv_backward(const ConvArgs& a, hipStream_t s);

struct ScanArgs {
  int dtype, C, G, Cg, n, softplus;  // channels, groups, channels of a group, states of a channel
  int N, T;
  const int* cu;
  int n_slots;
  const int* slots;
  unsigned* status;
  long long xs, dts, zs, os, bs, cs;
  const void* x;
  const void* dt;
  const float* A;           // [C, n]
  const void* B;            // [T, G, n]
  const void* Cm;
  const float* D;           // [C] or nullptr
  const float* bias;        // [C] or nullptr
  const void* z;            // or nullptr
  const float* S_in;        // [.., C, n] or nullptr
  float* S_out;
  void* out;
  char* ws;
  int split;                // not 0: sequences of fewer tokens go token by token, the others in blocks
  // gradient
  const void* d_out;
  const float* dS_out;
  void* dx;
  void* ddt;
  void* dz;
  void* dB;
  void* dC;
  float* dA;
  float* dD;
  float* dbias;
  float* dS_in;
};
size_t scan_forward_bytes(const ScanArgs& a);
hipError_t launch_scan(const ScanArgs& a, hipStream_t s);
size_t scan_backward_bytes(const ScanArgs& a);
hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s);

struct NormArgs {
  int dtype, pdtype, odtype, H, D, gate, group;
  long long R;              // head rows: rows * H
  float eps;
  long long xs, rs, zs, os; // elements between rows of x, residual, z, out / d_out
  const void* x;
  const void* w;            // [D] or nullptr
  const void* res;
  const void* z;
  void* out;
  float* scale;
  void* res_out;
  // gradient (res: the residual's gradient)
  const void* d_out;
  void* dx;
  void* dz;
  float* dw;
  float* ws;
};
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
// Threads of that launch, which have to stay below 2^32: 8 to 64 a row of up to 512 columns, in workgroups of 256.
constexpr long long norm_threads(long long rows, int D) {
  const int wide = D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : D <= 512 ? 64 : D <= 8192 ? 256 : 1024;
  return wide < 256 ? (rows * wide + 255) / 256 * 256 : rows * wide;
}
size_t norm_backward_bytes(const NormArgs& a);
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s);

// Sums over P rows of `part` [P, M], each column in row order: into up to three arrays that lie behind each other in
// a row, of m0, m1 and M - m0 - m1 columns (nullptr: not wanted).  stepq_layer_sum.hip.
struct SumArgs {
  const float* part;
  int P;
  long long M, m0, m1;
  float* out0;
  float* out1;
  float* out2;
};
hipError_t launch_sum(const SumArgs& a, hipStream_t s);

#ifdef __HIPCC__
namespace lay {

using namespace dlt;

constexpr float kLog2e = 1.44269504f;

// exp(-a) for a >= 0, for rows of type DT.  The argument t = -a log2(e) of the hardware's exponential is rounded, which by
// itself makes the result wrong by up to 1.3 a U (U = 2^-24); for 16-bit rows, whose values are rounded to 2^13 U and more,
// it stays so.  For binary32 r is what the rounding took, right to 1.9e-9 t (ln 2 is rounded), and 3 U + 0.05 a U are left.
// The bounds on r (it is below 1e-5 where the result is not zero) are for a = inf, where it is NaN; NaN passes by t.  Corrected
// for all types, 16,381 tokens x 10,240 channels of the convolution would take 145 us, not 140, the scan of 16,381 x 4,096 340,
// not 332, and the scan's gradient of 3,001 x 1,536 of 32 states 310, not 232 (its registers would no longer allow two waves a
// SIMD).  Binary32 rows: the convolution and both gradients take 1% more for it, the scan of 8,000 x 4,096 175 us, not 170.
template <int DT>
__device__ __forceinline__ float exp_minus(float a) {
  const float t = a * -kLog2e, e = __builtin_amdgcn_exp2f(t);
  if constexpr (DT != kF32) return e;
  return fmaf(e, __builtin_amdgcn_fmed3f(fmaf(t, -0.693147181f, -a), -1e-3f, 1e-3f), e);
}

// sigmoid(v), one and zero at the ends.  Binary32 rows: from e = exp(-|v|) as 1 / (1 + e) or e / (1 + e), right to
// (7 + 0.05 |v|) U; 16-bit ones: from exp(-v), to (6 + 1.3 |v|) U.
template <int DT>
__device__ __forceinline__ float sigmoid(float v) {
  if constexpr (DT != kF32) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -kLog2e));
  const float e = exp_minus<DT>(fabsf(v)), i = __builtin_amdgcn_rcpf(1.0f + e);
  return v >= 0 ? i : e * i;
}
template <int DT>
__device__ __forceinline__ float act_of(int act, float v) {
  if (act == kNone) return v;
  const float s = sigmoid<DT>(v);
  return act == kSilu ? v * s : s;
}

// V (1, 2, 4 or 8) consecutive elements.
template <int DT, int V>
__device__ __forceinline__ void loadv(const void* p, long long i, float* x) {
  if constexpr (V == 8) load8<DT>(p, i, x);
  else loadn<DT, V>(p, i, x);
}
template <int DT, int V>
__device__ __forceinline__ void storev(void* p, long long i, const float* x) {
  if constexpr (V == 8) store8<DT>(p, i, x);
  else storen<DT, V>(p, i, x);
}

// E neighbouring elements as they lie in memory: kept until they are used, so that their load is not waited for before.
// Rows are 16-byte aligned, so a read of 32 bytes may assume no more than that.
template <int DT, int E>
struct Raw {
  typedef typename std::conditional<DT == kF32, float, unsigned short>::type T;
  typedef T V __attribute__((ext_vector_type(E)));
  typedef typename std::conditional<E == 1, T, V>::type Held;
  typedef Held InMemory __attribute__((aligned(E * sizeof(T) < 16 ? E * sizeof(T) : 16)));
  static_assert(alignof(InMemory) <= 16);
  Held v;
  __device__ __forceinline__ void load(const void* p, long long at = 0) { v = *(const InMemory*)((const char*)p + at); }
  __device__ __forceinline__ float operator[](int i) const {
    T x;
    if constexpr (E == 1) x = v;
    else x = v[i];
    if constexpr (DT == kF32) return x;
    else return e_f<DT>(x);
  }
};

// 8 consecutive parameters whose type is known at run time.
__device__ __forceinline__ void load8_any(int dt, const void* p, long long i, float* x) {
  if (dt == kF32) load8<kF32>(p, i, x);
  else if (dt == kBF16) load8<kBF16>(p, i, x);
  else load8<kF16>(p, i, x);
}
__device__ __forceinline__ void load4_any(int dt, const void* p, long long i, float* x) {
  const f4 a = dt == kF32 ? load4<kF32>(p, i) : dt == kBF16 ? load4<kBF16>(p, i) : load4<kF16>(p, i);
#pragma unroll
  for (int j = 0; j < 4; j++) x[j] = a[j];
}

// Pieces of 2^SH tokens that no two sequences share: sequence s owns pieces (cu[s] >> SH) + s .. of T / 2^SH + N
// (a sequence of any length has at least one, so an empty one can hand its state on), or, where lengths are
// equal, `per` pieces each.
template <class Args>
__host__ __device__ inline long long pieces(const Args& A, int sh) {
  if (A.cu) return ((long long)A.T >> sh) + A.N;
  const long long L = A.N ? A.T / A.N : 0, per = (L + (1LL << sh) - 1) >> sh;
  return (per > 1 ? per : 1) * A.N;
}

// Sequence s of piece j, and which of its pieces it is; false for a piece of no sequence.  The whole wave asks for
// one j: 64 sequences are looked at at once, one round for up to 64 of them, two up to 4,096.  What
// broken offsets give is a sequence of the call and a piece that may lie outside it; callers check.
template <class Args>
__device__ __forceinline__ bool piece(const Args& A, int sh, long long j, int lane, int& s, long long& idx) {
  if (!A.cu) {
    const long long L = A.T / A.N, p = (L + (1LL << sh) - 1) >> sh, per = p > 1 ? p : 1;
    s = (int)(j / per);
    idx = j - s * per;
    return s < A.N;
  }
  long long lo = 0, n = A.N;
  do {
    const long long step = (n + 63) >> 6, at = lo + lane * step;
    const bool in = lane * step < n && (long long)(A.cu[at] >> sh) + at <= j;
    const int k = __popcll(__ballot(in));
    if (k == 0) return false;
    lo += (k - 1) * step;
    n = n - (k - 1) * step < step ? n - (k - 1) * step : step;
  } while (n > 1);
  s = __builtin_amdgcn_readfirstlane((int)lo);
  idx = j - ((long long)(A.cu[s] >> sh) + s);
  return idx >= 0;
}

}  // namespace lay
#endif

}  // namespace stepq
