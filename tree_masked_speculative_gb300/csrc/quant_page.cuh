// 4-bit pages and the rotation of new rows: internal declarations (not installed).
//
// A row of a KV head is D / 8 words: 16-bit quads (4 neighbouring elements, lowest nibble
// first), quad g of 32-element block j at place g * (D / 32) + j.  Scale and bias of a group
// stand side by side, so that one load brings both.
#pragma once

#include "seq_internal.cuh"

namespace ta {

struct QuantCache {
    uint32_t *kc, *vc;                // codes
    void *ka, *va;                    // scale, bias pairs
    // strides in bytes, of the codes and of the affine: below 2^32, so that an offset is one 32 x 32 -> 64 bit product
    uint32_t c_sp, c_sh, c_st;
    uint32_t a_sp, a_sh, a_st;
};
// base + i * stride
template <typename T>
__device__ __forceinline__ T *at_bytes(T *base, uint32_t i, uint32_t stride) {
    return reinterpret_cast<T *>(reinterpret_cast<uintptr_t>(base) + static_cast<uint64_t>(i) * stride);
}

// New rows: q turned to q_out, k_new turned and v_new to the cache.  Row strides in 16-byte
// vectors.
struct RotaryArgs {
    const void *q, *k_new, *v_new;
    void *q_out;
    const int64_t *slot;
    const int32_t *pos;               // nullptr: nothing is turned
    const float *table;               // [max_pos][R]: cos, sin
    int T, H, Hk, D, R, max_pos, interleaved;
    int page_shift, n_pages, bf16;
    long long q_st, q_sh, qo_st, qo_sh, k_st, k_sh, v_st, v_sh;
};
struct RotaryAppendArgs {
    RotaryArgs r;
    void *k, *v;
    long long c_sp, c_sh, c_st;       // of the 16-bit cache, vectors
};
cudaError_t launch_rotary_append(const RotaryAppendArgs &a, cudaStream_t s);

struct QuantAppendArgs {
    RotaryArgs r;
    QuantCache c;
    int group;
};
cudaError_t launch_quant_append(const QuantAppendArgs &a, cudaStream_t s);

struct QuantReadArgs {
    QuantCache c;
    const int64_t *slot;
    void *k, *v;
    int T, Hk, D, group, page_shift, n_pages, bf16;
    long long k_st, k_sh, v_st, v_sh;   // elements
};
cudaError_t launch_quant_read(const QuantReadArgs &a, cudaStream_t s);

// Attention of ragged rows over 4-bit pages: SeqArgs (whose k, v and their strides are not used)
// and the cache.
struct SeqQuantArgs {
    SeqArgs s;
    QuantCache c;
    int group;
};
cudaError_t launch_seq_quant_fma(const SeqQuantArgs &a, cudaStream_t s);

// Warp-MMA kernel for few rows (max_q_len * heads per KV head); its workspace and launch.  More rows would be
// products it has no registers for, or keys widened twice.  Replayed graphs, us, warp MMA / tcgen05 (bf16, 32 / 8
// heads; D = 256 with half the requests):
//                                      4 rows       8 rows      16 rows     32 rows
//   64 of 900 to 16384 keys, D 128 G 64  162 / 539  164 / 537   262 / 537   - / 542
//                            D 128 G 32  196 / 527  198 / 525   326 / 530   - / 527
//                            D  64 G 32  126 / 419  126 / 421   189 / 419   - / 421
//                            D 256 G 64  158 / 322  159 / 328    -  / 327   - / 329
//                            D 256 G 32  187 / 329  192 / 332    -  / 333   - / 332
//   16 of 300 to 9000 keys,  D 128 G 64   32 / 86    33 / 87     49 / 89    - / 89
//   1 of 4000 keys,          D 128 G 64   12 / 28    14 / 28     18 / 28    - / 29
//   200 of 300 keys,         D 128 G 64   48 / 99    49 / 100    70 / 100   - / 104
//                            D 256 G 32   96 / 117  105 / 118    -  / 117   - / 120
// An earlier state of the kernel had four row tiles (32 rows: 483 / 484 for the first line, 1027 / 480 for the second, 358 /
// 382 for the third, 95 / 70 for 16 requests) and two at D = 256 (16 rows, half as many KV heads: 149 / 179 with groups of
// 64, 307 / 185 with groups of 32, 98 / 38 for 200 of 300 keys, but 22 / 41 for one request of 4000): neither is compiled.
constexpr int quant_mma_rows(int d) { return d == 256 ? 8 : 16; }
unsigned long long seq_quant_mma_workspace64(int rows, int sms);
unsigned long long seq_quant_mma_workspace128(int rows, int sms);
unsigned long long seq_quant_mma_workspace256(int rows, int sms);
cudaError_t launch_seq_quant_mma64(const SeqQuantArgs &a, void *ws, int sms, cudaStream_t s);
cudaError_t launch_seq_quant_mma128(const SeqQuantArgs &a, void *ws, int sms, cudaStream_t s);
cudaError_t launch_seq_quant_mma256(const SeqQuantArgs &a, void *ws, int sms, cudaStream_t s);

// Tensor-core kernel (the plan's maps of K and V are not used).
cudaError_t launch_seq_quant_tc64(const SeqQuantArgs &a, const SeqTcPlan &pl, cudaStream_t s);
cudaError_t launch_seq_quant_tc128(const SeqQuantArgs &a, const SeqTcPlan &pl, cudaStream_t s);
cudaError_t launch_seq_quant_tc256(const SeqQuantArgs &a, const SeqTcPlan &pl, cudaStream_t s);

}  // namespace ta
