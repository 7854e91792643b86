// Warp-MMA attention over 4-bit pages, head dimension 128.
#include "seq_quant_mma.cuh"

namespace ta {
cudaError_t launch_seq_quant_mma128(const SeqQuantArgs &a, void *ws, int sms, cudaStream_t s) { return qm_launch_dim<128>(a, ws, sms, s); }
unsigned long long seq_quant_mma_workspace128(int rows, int sms) { return qm_workspace<128>(rows, sms); }
}  // namespace ta
