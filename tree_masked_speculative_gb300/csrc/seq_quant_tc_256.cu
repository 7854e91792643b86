// Tensor-core attention over 4-bit pages, head dimension 256.
#include "seq_tc.cuh"

namespace ta {
cudaError_t launch_seq_quant_tc256(const SeqQuantArgs &a, const SeqTcPlan &pl, cudaStream_t s) {
    return seqtc::launch_quant_dim<256>(a, pl, s);
}
}  // namespace ta
