// Internal declarations of the batched serving operators (not installed):
// step planning, cache append and attention over a paged K/V cache or over
// packed prompts.
#pragma once

#include "ta_internal.cuh"

namespace ta {

// Bits of the status word that the serving operators OR into.
enum SeqStatus : int {
    kSeqTimeout = 1,     // a bounded wait of the tensor-core kernel gave up
    kSeqBadPage = 2,     // a block-table cell outside [0, n_pages) was attended
    kSeqBadLength = 4,   // a length or row offset outside its range
};
enum PlanStatus : int {
    kPlanNoPages = 1,    // the free stack holds fewer pages than the step needs
    kPlanBadLength = 2,  // a negative length, or more tokens / pages than a table row holds
    kPlanTokens = 4,     // more new tokens than max_tokens
    kPlanStack = 8,      // released pages would not fit the stack, or its count is out of range
};

// Attention of ragged rows.  Row (token t, head h) of request b is token
// i = t - cu[b] of the request's q_len = cu[b+1] - cu[b] new tokens, at
// position kv_len - q_len + i of its kv_len keys.
struct SeqArgs {
    const void *q, *k, *v;
    void *out;
    const int32_t *cu;        // [B + 1]
    const int32_t *kv_lens;   // [B]; nullptr: packed prompts (kv_len = q_len, K/V rows at cu[b])
    const int32_t *table;     // [B, max_pages] (paged)
    const int32_t *parents;   // [T] or nullptr
    int32_t *status;          // ORed into
    int B, H, Hk, g, D, T;
    int max_q;                // most new tokens of a request (paged; T for prompts)
    int window;               // 0: none
    int page_shift, n_pages, max_pages;
    int bf16;
    long long q_st, q_sh, o_st, o_sh;      // token and head strides, elements
    long long k_sp, k_st, k_sh, v_st, v_sh;  // K/V: page (paged), token and head strides
    float scale;
};

// Rows, tokens and keys of request b, made safe against inconsistent inputs:
// every row index stays inside [0, T) and every key inside the table row.
struct SeqReq {
    int q0, qn, kv;
    bool bad;
};
__device__ __forceinline__ SeqReq seq_request(const SeqArgs &a, int b) {
    SeqReq r;
    const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
    r.q0 = min(max(c0, 0), a.T);
    const int q1 = min(max(c1, r.q0), a.T);
    r.qn = min(q1 - r.q0, a.max_q);
    r.bad = r.q0 != c0 || r.q0 + r.qn != c1;
    if (a.kv_lens) {
        const int n = __ldg(a.kv_lens + b);
        const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
        r.kv = static_cast<int>(min(static_cast<long long>(max(n, 0)), cap));
        r.bad |= r.kv != n;
    } else {
        r.kv = r.qn;
    }
    return r;
}

cudaError_t launch_seq_fma(const SeqArgs &a, cudaStream_t s);

// Polls (about 1 us each) after which a wait of the tensor-core kernel gives up.
constexpr uint32_t kSeqWaitPolls = 1u << 21;
// Tensor-core kernel: grid size, workspace and the tensor maps of K and V.
struct SeqTcPlan {
    int G;
    uint32_t polls;     // bound of its waits (kSeqWaitPolls but for a test)
    void *ws;
    CUtensorMap q, k, v;
};
// Keys per key tile, tiles' worth of time of a unit's start and end, and rows per row
// tile of the tensor-core kernel.
constexpr int kSeqTcTileKeys = 64, kSeqTcUnitCost = 5;
constexpr int seq_tc_rows(int d) { return d == 256 ? 128 : 256; }
// Its workspace on a grid of G CTAs: status, records, (m, l) and O of 2 G partial
// slots, and the marks of columns that are not finite (8 pieces a CTA).
constexpr unsigned long long seq_tc_workspace(int d, int G) {
    return 256ull + (G * 16ull + 255) / 256 * 256 + 2ull * G * seq_tc_rows(d) * (8ull + 4ull * d) +
           8ull * G * seq_tc_rows(d) * (d / 8);
}
cudaError_t launch_seq_tc64(const SeqArgs &a, const SeqTcPlan &pl, cudaStream_t s);
cudaError_t launch_seq_tc128(const SeqArgs &a, const SeqTcPlan &pl, cudaStream_t s);
cudaError_t launch_seq_tc256(const SeqArgs &a, const SeqTcPlan &pl, cudaStream_t s);

// Warp-MMA kernel for few rows per KV head (paged): which rows it takes, with how many
// (request, KV head) pairs it is the faster one, its workspace and launch.
bool seq_mma_takes(int d, long long rows);
bool seq_mma_best(int d, long long units);
unsigned long long seq_mma_workspace(int d, int rows, int sms);
cudaError_t launch_seq_mma(const SeqArgs &a, void *ws, int sms, cudaStream_t s);

// ---------------------------------------------------------------- planning
struct PlanArgs {
    const int32_t *keep, *fresh, *held;
    int32_t *table, *stack;
    const int32_t *n_free;
    int32_t *held_out, *n_free_out, *cu, *lens;
    int64_t *slot;
    int32_t *pos, *status;
    int B, max_pages, capacity, max_tokens, page_shift;
};
constexpr int kPlanMaxBatch = 16384;
cudaError_t launch_paged_plan(const PlanArgs &a, cudaStream_t s);

// ------------------------------------------------------------------ append
struct AppendArgs {
    const void *k_new, *v_new;
    void *k, *v;
    const int64_t *slot;
    int T, Hk, D, page_shift, n_pages;
    long long kn_st, kn_sh, vn_st, vn_sh, c_sp, c_st, c_sh;
};
cudaError_t launch_paged_append(const AppendArgs &a, cudaStream_t s);

}  // namespace ta
