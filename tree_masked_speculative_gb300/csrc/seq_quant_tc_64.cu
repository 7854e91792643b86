// Tensor-core attention over 4-bit pages, head dimension 64.
#include "seq_tc.cuh"

namespace ta {
cudaError_t launch_seq_quant_tc64(const SeqQuantArgs &a, const SeqTcPlan &pl, cudaStream_t s) {
    return seqtc::launch_quant_dim<64>(a, pl, s);
}
}  // namespace ta
