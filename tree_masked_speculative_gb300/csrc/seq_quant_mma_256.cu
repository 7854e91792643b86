// Warp-MMA attention over 4-bit pages, head dimension 256.
#include "seq_quant_mma.cuh"

namespace ta {
cudaError_t launch_seq_quant_mma256(const SeqQuantArgs &a, void *ws, int sms, cudaStream_t s) { return qm_launch_dim<256>(a, ws, sms, s); }
unsigned long long seq_quant_mma_workspace256(int rows, int sms) { return qm_workspace<256>(rows, sms); }
}  // namespace ta
