// Tensor-core attention of ragged rows, head dimension 64.
#include "seq_tc.cuh"

namespace ta {
cudaError_t launch_seq_tc64(const SeqArgs &a, const SeqTcPlan &pl, cudaStream_t s) {
    return seqtc::launch_dim<64>(a, pl, s);
}
}  // namespace ta
