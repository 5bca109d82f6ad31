// stepq_delta_chunk.hip -- the gated delta rule in chunks of 64 tokens, forward (see stepq_chunk.h for
// the mathematics and the operands).  Two launches: the chunks' local matrices, all chunks at once
// (k_chunk_prep), then one pass over the chunks of every sequence in order (k_chunk_state).
#include "stepq_chunk_kernels.h"

namespace stepq {
namespace {

using namespace dlt;

template <int D, int DT>
size_t bytes(const SeqArgs& a) {
  return (size_t)(key_bytes<LayF<D, DT>>(a) + head_bytes<LayF<D, DT>>(a));
}

template <int D, int DT>
hipError_t launch(const SeqArgs& a, hipStream_t s) {
  if (a.T > 0) {
    hipLaunchKernelGGL((k_chunk_prep<D, DT, LayF<D, DT>>), dim3((unsigned)chunk_slots(a.T, a.N), a.Hq), dim3(256), 0, s, a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  constexpr int NW = D / 16;
  hipLaunchKernelGGL((k_chunk_state<D, DT, NW, LayF<D, DT>>), dim3((unsigned)((long long)a.N * a.H), 1), dim3(64 * NW), 0, s,
                     a, nullptr, nullptr);
  return hipGetLastError();
}

}  // namespace

size_t chunk_forward_bytes(const SeqArgs& a) {
  if (a.D == 64)
    return a.dtype == kF32 ? bytes<64, kF32>(a) : a.dtype == kBF16 ? bytes<64, kBF16>(a) : bytes<64, kF16>(a);
  return a.dtype == kF32 ? bytes<128, kF32>(a) : a.dtype == kBF16 ? bytes<128, kBF16>(a) : bytes<128, kF16>(a);
}

hipError_t launch_chunk_forward(const SeqArgs& a, hipStream_t s) {
  if (a.N <= 0) return hipSuccess;
  if (a.D == 64)
    return a.dtype == kF32 ? launch<64, kF32>(a, s) : a.dtype == kBF16 ? launch<64, kBF16>(a, s) : launch<64, kF16>(a, s);
  return a.dtype == kF32 ? launch<128, kF32>(a, s) : a.dtype == kBF16 ? launch<128, kBF16>(a, s) : launch<128, kF16>(a, s);
}

}  // namespace stepq
