// stepq_read.hip -- read packed states back (page: "STEPQuant" paper digest, Method 3:
// X_hat[i,j] = r_i c_j z[i,j], FP16 pivot rows as stored), by slot, as binary32, bfloat16 or binary16.
//
// One workgroup per (request, head), a quarter of the rows a wave.  A row's codes sit at one bit offset in
// all 64 lane streams, so its width, shift and factor are wave-uniform and a lane reads one or two words.
// r c z is formed as r (c z): c z is exact in binary32 (11 + 8 bits), so the value is the exact product
// rounded once, and once more where the output type is narrower.
//
// Bound by HBM, written side: 16 x 48 states of 6 bits to binary32 (50 MB out, 10 in) take 12 us, 5.0 TB/s; to
// bfloat16 10 us.  Eight rows' words are in flight at once: one row at a time waited for each (28 us
// against 8 for 4 x 48 states of 8 bits).
#include "stepq_delta.h"
#include "stepq_internal.h"

namespace stepq {
namespace {

using namespace dlt;

// Also resolves the slots for a prompt pass over the pool: slot_out[b] / row_out[b] = the slot / b, or
// -1 where the row is skipped (padding, a bad slot, or `seq` without tokens or with bad offsets).
template <int D, int DT>
__global__ __launch_bounds__(256) void k_read(DevPlan P, const uint8_t* pool, int n_slots,
                                              const int* slots, void* S, SeqArgs seq, int* slot_out,
                                              int* row_out) {
  constexpr int G = D / 64;
  const int b = blockIdx.x, h = blockIdx.y;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int slot = slots ? slots[b] : b;
  unsigned flag = 0;
  if (slot < 0 || slot >= n_slots) {
    if (slot != -1) flag = kFlagBadSlotSeq;
    slot = -1;
  }
  if (slot_out) {
    int t0, t1;
    if (!seq_range(seq, b, t0, t1)) flag |= kFlagBadSeq;
    if (t0 == t1) slot = -1;
  }
  if (h == 0 && threadIdx.x == 0) {
    if (slot_out) {
      slot_out[b] = slot;
      row_out[b] = slot < 0 ? -1 : b;
    }
    if (flag) atomicOr(P.status, flag);
  }
  if (slot < 0) return;
  const uint8_t* seg = pool + (long long)slot * P.bpr + P.head_off[h];
  const uint32_t* words = (const uint32_t*)seg + lane;
  const int nw = P.words[h];
  const uint16_t* rb = (const uint16_t*)(seg + P.off_r[h]);
  const uint16_t* pb = (const uint16_t*)(seg + P.off_piv[h]);
  const long long out = ((long long)b * P.H + h) * D * D + G * lane;
  constexpr int R = D / 4;  // rows of a wave, R w ..
  // the wave's row words and factors, one a lane; a row's are broadcast from there
  const int mine = R * w + (lane < R ? lane : R - 1);
  const unsigned meta = (unsigned)P.rowmeta[h * D + mine];
  auto values = [&](unsigned m, uint32_t lo, uint32_t hi, float r, const float* c, float* x) {
    const int bits = (m >> 16) & 15;
    const uint32_t y = __builtin_amdgcn_alignbit(hi, lo, m & 31);
#pragma unroll
    for (int g = 0; g < G; g++) {
      x[g] = r * (c[g] * (float)(int)__builtin_amdgcn_sbfe((int)y, g * bits, bits));
      // keeps the rounding to binary32: the product and a narrowing to binary16 would be fused
      if constexpr (DT == kF16) asm("" : "+v"(x[g]));
    }
  };
  float c[G];
  unsigned short fac = 0;
  if (nw) {
    const uint16_t* cb = (const uint16_t*)(seg + P.off_c[h]);
#pragma unroll
    for (int g = 0; g < G; g++) c[g] = h_f(cb[G * lane + g]);
    fac = rb[mine];
  }
  const bool piv = (meta & 0x80000000u) != 0;
  if (__any(piv)) {  // FP16 pivot rows among them: a row at a time
    for (int i = 0; i < R; i++) {
      const unsigned m = __builtin_amdgcn_readlane(meta, i);
      float x[G];
      if (m & 0x80000000u) {
#pragma unroll
        for (int g = 0; g < G; g++) x[g] = h_f(pb[(m & 0x7fffffffu) * D + G * lane + g]);
      } else {
        const int wi = (m >> 8) & 255;
        values(m, words[wi * 64], (m >> 20) & 1 ? words[(wi + 1) * 64] : 0u, h_f(__builtin_amdgcn_readlane(fac, i)), c, x);
      }
      storen<DT, G>(S, out + (long long)(R * w + i) * D, x);
    }
    return;
  }
  // all rows quantized: 8 rows' words in flight at once (a row whose codes end in one word reads it twice)
#pragma unroll
  for (int i0 = 0; i0 < R; i0 += 8) {
    uint32_t lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const unsigned m = __builtin_amdgcn_readlane(meta, i0 + i);
      const int wi = (m >> 8) & 255;
      lo[i] = words[wi * 64];
      hi[i] = words[(wi + ((m >> 20) & 1)) * 64];
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const unsigned m = __builtin_amdgcn_readlane(meta, i0 + i);
      float x[G];
      values(m, lo[i], hi[i], h_f((unsigned short)__builtin_amdgcn_readlane(fac, i0 + i)), c, x);
      storen<DT, G>(S, out + (long long)(R * w + i0 + i) * D, x);
    }
  }
}

template <int D>
hipError_t launch(const DevPlan& P, const uint8_t* pool, int n_slots, const int* slots, int B, void* S,
                  int dtype, const SeqArgs& seq, int* slot_out, int* row_out, hipStream_t s) {
  const dim3 grid(B, P.H), block(256);
  if (dtype == kF32)
    hipLaunchKernelGGL((k_read<D, kF32>), grid, block, 0, s, P, pool, n_slots, slots, S, seq, slot_out, row_out);
  else if (dtype == kBF16)
    hipLaunchKernelGGL((k_read<D, kBF16>), grid, block, 0, s, P, pool, n_slots, slots, S, seq, slot_out, row_out);
  else
    hipLaunchKernelGGL((k_read<D, kF16>), grid, block, 0, s, P, pool, n_slots, slots, S, seq, slot_out, row_out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_read(const DevPlan& P, const uint8_t* pool, int n_slots, const int* slots, int B,
                       void* S, int dtype, const SeqArgs* seq, int* slot_out, int* row_out,
                       hipStream_t s) {
  if (B <= 0) return hipSuccess;
  const SeqArgs none{};
  return P.D == 64 ? launch<64>(P, pool, n_slots, slots, B, S, dtype, seq ? *seq : none, slot_out, row_out, s)
                   : launch<128>(P, pool, n_slots, slots, B, S, dtype, seq ? *seq : none, slot_out, row_out, s);
}

}  // namespace stepq
