// stepq_delta_chunk.hip -- the gated delta rule in chunks of 64 tokens, forward (see stepq_chunk.h for
// the mathematics and the operands).  Two launches: the chunks' local matrices, all chunks at once
// (k_chunk_prep), then one pass over the chunks of every sequence in order (k_chunk_state); four where a
// few long sequences are cut into segments.
#include "stepq_chunk_kernels.h"

namespace stepq {
namespace {

using namespace dlt;

// Segments of a sequence: with at most 32 (sequence, head) pairs and 40 chunks a sequence or more on
// average, 256 / pairs segments (at most 16, of at least four chunks) run at once.  Every chunk is then run
// three times, so it takes many idle CUs and long segments to gain (us, d = 128 bf16, cut against whole:
// 1 x 32 heads of 1,024 / 2,048 / 4,096 / 16,384 tokens 80 / 137 / 204 / 676 against 73 / 131 / 254 / 984;
// 1 x 4 heads of 1,024 / 4,096 tokens 61 / 140 against 65 / 219; 64 heads of 8,192 tokens 655 against 608).
int segments(const SeqArgs& a) {
  const long long tiles = (long long)a.N * a.H, chunks = (long long)a.T / ((long long)a.N * kChunk);
  if (tiles > 32 || chunks < 40) return 1;
  long long P = 256 / tiles;
  P = P > 16 ? 16 : P;
  return (int)(P > chunks / 4 ? chunks / 4 : P);
}

template <int D, int DT>
size_t fixed_bytes(const SeqArgs& a) {
  return (size_t)(key_bytes<LayF<D, DT>>(a) + head_bytes<LayF<D, DT>>(a));
}
template <int D, int DT>
size_t bytes(const SeqArgs& a) {
  const int P = segments(a);
  return fixed_bytes<D, DT>(a) + (P > 1 ? (size_t)3 * a.N * a.H * P * D * D * sizeof(float) : 0);
}

template <int D, int DT>
hipError_t launch(const SeqArgs& a, hipStream_t s) {
  using Y = LayF<D, DT>;
  if (a.T > 0) {
    hipLaunchKernelGGL((k_chunk_prep<D, DT, Y>), dim3((unsigned)chunk_slots(a.T, a.N), a.Hq), dim3(256), 0, s, a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  Segs g{segments(a), nullptr, nullptr};
  const long long states = (long long)a.N * a.H;
  return with_state_waves<D, DT>(a, g.P, [&](auto nw) {
    constexpr int NW = nw.value;
    const unsigned tiles = workgroups<NW>(a, D);
    if (g.P == 1) {
      hipLaunchKernelGGL((k_chunk_state<D, DT, NW, Y, kForward>), dim3(tiles), dim3(64 * NW), 0, s, a, nullptr, nullptr, g);
      return hipGetLastError();
    }
    g.MN = (float*)(a.ws + fixed_bytes<D, DT>(a));
    g.S = g.MN + (size_t)2 * states * g.P * D * D;
    hipLaunchKernelGGL((k_chunk_state<D, DT, NW, Y, kSegment>), dim3(tiles, g.P, 2), dim3(64 * NW), 0, s, a, nullptr, nullptr, g);
    if (hipError_t e = hipGetLastError()) return e;
    hipLaunchKernelGGL((k_chunk_join<D>), dim3((unsigned)states, D / 32), dim3(128), 0, s, a, g);
    if (hipError_t e = hipGetLastError()) return e;
    hipLaunchKernelGGL((k_chunk_state<D, DT, NW, Y, kReadout>), dim3(tiles, g.P), dim3(64 * NW), 0, s, a, nullptr, nullptr, g);
    return hipGetLastError();
  });
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
