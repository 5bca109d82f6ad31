// stepq_delta.h -- the gated delta rule over sequences: arguments and device helpers shared by the
// recurrent kernel (stepq_delta_step.hip), the chunked forward pass (stepq_delta_chunk.hip) and its
// gradient (stepq_delta_grad.hip).  Not part of the public ABI.
//
// Per value head, S [d, d] with key rows and value columns:
//   e_t = v_t - (Diag(a_t) S_{t-1})^T k_t,  S_t = Diag(a_t) S_{t-1} + beta_t k_t e_t^T,  o_t = S_t^T q_t
// (KDA's delta-first order: S_t = Diag(a_t)(I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace stepq {

constexpr int kF32 = 0, kBF16 = 1, kF16 = 2;  // STEPQ_DTYPE_*
constexpr int kChunk = 64;                    // tokens of a chunk

// Everything the sequence kernels read; built by the host entry points after their checks.
struct SeqArgs {
  int kind, order, dtype, D;
  int Hq, H, grp;           // key heads, value heads, value heads per key head
  int N, T;                 // sequences, token rows
  const int* cu;            // [N + 1] token offsets, or nullptr: N sequences of T / N tokens
  long long qs, ks, vs, os; // elements between tokens of q, k, v and out / d_out
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;       // [T, H] (GDN) or [T, H, D] (KDA)
  const float* beta;        // [T, H]
  const float* S_in;        // [n_slots, H, D, D] or nullptr: zero
  float* S_out;             // the same shape, or nullptr: not kept; may be S_in
  int n_slots;
  const int* slots;         // [N] or nullptr: sequence s uses state s
  void* out;
  unsigned* status;         // may be nullptr
  char* ws;                 // chunked passes: workspace
  int split;                // not 0: sequences of fewer tokens go token by token, the others in chunks
};

// Gradient of the chunked pass.
struct GradArgs {
  SeqArgs f;
  const void* d_out;        // [T, H, D], token stride f.os
  const float* dS_out;      // [N, H, D, D] or nullptr: zero
  void* dq;                 // [T, Hq, D] packed
  void* dk;
  void* dv;                 // [T, H, D] packed
  float* dalpha;            // [T, H]
  float* dbeta;
  float* dS_in;             // [N, H, D, D] or nullptr: not wanted
};

// Chunk slots: sequence s owns slots cu[s]/64 + s .. of a range of T/64 + N, which needs no scan over
// the sequences (ceil(len/64) <= (cu[s]+len)/64 - cu[s]/64 + 1, so ranges never meet).
__host__ __device__ inline long long chunk_slots(long long T, long long N) { return T / kChunk + N; }

// Host checks shared by the sequence entry points (stepq_delta_api.cpp); each returns STEPQ_OK or an
// error with its message.  `stepq_delta_desc` is the C struct of stepq.h.
int seq_args(const void* desc, SeqArgs* a);
int seq_inputs(SeqArgs* a, const void* q, const void* k, const void* v, const float* alpha,
               const float* beta, void* out);
int seq_workspace(const void* ws, size_t have, size_t need);
size_t forward_bytes(const SeqArgs& a);                    // workspace of launch_forward
hipError_t launch_forward(const SeqArgs& a, hipStream_t s);  // all sequences, by the paths that suit them

size_t chunk_forward_bytes(const SeqArgs& a);
size_t chunk_backward_bytes(const SeqArgs& a);
hipError_t launch_recurrent(const SeqArgs& a, hipStream_t s);
hipError_t launch_chunk_forward(const SeqArgs& a, hipStream_t s);
hipError_t launch_chunk_backward(const GradArgs& a, hipStream_t s);

// Values of packed states by slot (stepq_read.hip); seq, slot_out and row_out: for a prompt pass.
struct DevPlan;
hipError_t launch_read(const DevPlan& P, const uint8_t* pool, int n_slots, const int* slots, int B,
                       void* S, int dtype, const SeqArgs* seq, int* slot_out, int* row_out,
                       hipStream_t s);

#ifdef __HIPCC__
namespace dlt {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef unsigned short us8 __attribute__((ext_vector_type(8)));
typedef unsigned short us4 __attribute__((ext_vector_type(4)));
typedef unsigned short us2 __attribute__((ext_vector_type(2)));

constexpr unsigned kFlagBadSlotSeq = 8u, kFlagBadSeq = 16u;

__device__ __forceinline__ float bf_f(unsigned short x) { return __uint_as_float((unsigned)x << 16); }
// binary32 -> bfloat16, round half to even; NaN stays NaN
__device__ __forceinline__ unsigned short f_bf(float x) {
  const __bf16 y = (__bf16)x;
  return __builtin_bit_cast(unsigned short, y);
}
__device__ __forceinline__ unsigned short f_h(float x) {
  return __builtin_bit_cast(unsigned short, (_Float16)x);
}
__device__ __forceinline__ float h_f(unsigned short x) {
  return (float)__builtin_bit_cast(_Float16, x);
}
template <int DT>
__device__ __forceinline__ float e_f(unsigned short x) {
  return DT == kBF16 ? bf_f(x) : h_f(x);
}
template <int DT>
__device__ __forceinline__ unsigned short f_e(float x) {
  return DT == kBF16 ? f_bf(x) : f_h(x);
}

// 8 consecutive elements (16 bytes of a 16-bit type, 32 of binary32) as binary32.
template <int DT>
__device__ __forceinline__ void load8(const void* p, long long i, float* x) {
  if constexpr (DT == kF32) {
    const f4 a = *(const f4*)((const float*)p + i), b = *(const f4*)((const float*)p + i + 4);
#pragma unroll
    for (int j = 0; j < 4; j++) x[j] = a[j], x[4 + j] = b[j];
  } else {
    const us8 a = *(const us8*)((const unsigned short*)p + i);
#pragma unroll
    for (int j = 0; j < 8; j++) x[j] = e_f<DT>(a[j]);
  }
}
template <int DT>
__device__ __forceinline__ void store8(void* p, long long i, const float* x) {
  if constexpr (DT == kF32) {
    *(f4*)((float*)p + i) = f4{x[0], x[1], x[2], x[3]};
    *(f4*)((float*)p + i + 4) = f4{x[4], x[5], x[6], x[7]};
  } else {
    us8 a;
#pragma unroll
    for (int j = 0; j < 8; j++) a[j] = f_e<DT>(x[j]);
    *(us8*)((unsigned short*)p + i) = a;
  }
}
template <int DT>
__device__ __forceinline__ f4 load4(const void* p, long long i) {
  if constexpr (DT == kF32) return *(const f4*)((const float*)p + i);
  const us4 a = *(const us4*)((const unsigned short*)p + i);
  return f4{e_f<DT>(a[0]), e_f<DT>(a[1]), e_f<DT>(a[2]), e_f<DT>(a[3])};
}
template <int DT>
__device__ __forceinline__ void store4(void* p, long long i, f4 x) {
  if constexpr (DT == kF32) {
    *(f4*)((float*)p + i) = x;
  } else {
    *(us4*)((unsigned short*)p + i) = us4{f_e<DT>(x[0]), f_e<DT>(x[1]), f_e<DT>(x[2]), f_e<DT>(x[3])};
  }
}
// NC (1, 2 or 4) consecutive elements.
template <int DT, int NC>
__device__ __forceinline__ void loadn(const void* p, long long i, float* x) {
  if constexpr (NC == 4) {
    const f4 a = load4<DT>(p, i);
#pragma unroll
    for (int j = 0; j < 4; j++) x[j] = a[j];
  } else if constexpr (NC == 2) {
    if constexpr (DT == kF32) {
      const f2 a = *(const f2*)((const float*)p + i);
      x[0] = a[0], x[1] = a[1];
    } else {
      const us2 a = *(const us2*)((const unsigned short*)p + i);
      x[0] = e_f<DT>(a[0]), x[1] = e_f<DT>(a[1]);
    }
  } else {
    if constexpr (DT == kF32) x[0] = ((const float*)p)[i];
    else x[0] = e_f<DT>(((const unsigned short*)p)[i]);
  }
}
template <int DT, int NC>
__device__ __forceinline__ void storen(void* p, long long i, const float* x) {
  if constexpr (NC == 4) {
    store4<DT>(p, i, f4{x[0], x[1], x[2], x[3]});
  } else if constexpr (NC == 2) {
    if constexpr (DT == kF32) *(f2*)((float*)p + i) = f2{x[0], x[1]};
    else *(us2*)((unsigned short*)p + i) = us2{f_e<DT>(x[0]), f_e<DT>(x[1])};
  } else {
    if constexpr (DT == kF32) ((float*)p)[i] = x[0];
    else ((unsigned short*)p)[i] = f_e<DT>(x[0]);
  }
}

// Token range [t0, t1) of sequence s; false (and an empty range) where the offsets are not
// 0 <= cu[s] <= cu[s + 1] <= T, so that no caller reads or writes outside the T rows.
__device__ __forceinline__ bool seq_range(const SeqArgs& A, int s, int& t0, int& t1) {
  if (!A.cu) {
    const int L = A.T / A.N;
    t0 = s * L;
    t1 = t0 + L;
    return true;
  }
  t0 = A.cu[s];
  t1 = A.cu[s + 1];
  if (t0 >= 0 && t0 <= t1 && t1 <= A.T) return true;
  t0 = t1 = 0;
  return false;
}

// State index of sequence s (itself, or its slot); -1: skip the sequence.  `report`: one thread of the
// launch per sequence, which raises the flags.
__device__ __forceinline__ int seq_slot(const SeqArgs& A, int s, bool valid, bool report) {
  int slot = s;
  unsigned flag = valid ? 0u : kFlagBadSeq;
  if (A.slots) {
    slot = A.slots[s];
    if (slot < 0 || slot >= A.n_slots) {
      if (slot != -1) flag |= kFlagBadSlotSeq;
      slot = -1;
    }
  }
  if (report && flag && A.status) atomicOr(A.status, flag);
  return valid ? slot : -1;
}

}  // namespace dlt
#endif

}  // namespace stepq
