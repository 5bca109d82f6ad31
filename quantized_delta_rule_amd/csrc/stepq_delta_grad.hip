// stepq_delta_grad.hip -- gradient of the chunked delta rule (not built yet: the call is refused).
#include "stepq_chunk.h"

namespace stepq {

size_t chunk_backward_bytes(const SeqArgs&) { return 0; }
hipError_t launch_chunk_backward(const GradArgs&, hipStream_t) { return hipErrorNotSupported; }

}  // namespace stepq
