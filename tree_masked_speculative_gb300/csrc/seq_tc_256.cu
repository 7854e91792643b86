// Tensor-core attention of ragged rows, head dimension 256.
#include "seq_tc.cuh"

namespace ta {
cudaError_t launch_seq_tc256(const SeqArgs &a, const SeqTcPlan &pl, cudaStream_t s) {
    return seqtc::launch_dim<256>(a, pl, s);
}
}  // namespace ta
