// seq_sm100.cu -- tensor-core family of sequence attention: not in yet, every
// description runs on the portable kernels.
#include "seq.h"

namespace swin {

bool seq_fast_supported(int, int) { return false; }
cudaError_t seq_fast_forward(const SeqParams&, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t seq_fast_backward(const SeqParams&, cudaStream_t) { return cudaErrorNotSupported; }

}  // namespace swin
