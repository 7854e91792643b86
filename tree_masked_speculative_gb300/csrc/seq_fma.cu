// Attention of ragged rows on CUDA cores: one warp per (token, head) row, the
// keys one after the other, an online softmax in f32.  It reads K and V once
// per row, so it is bound by L2 bandwidth (rows x keys x 4 D bytes); it holds P
// in f32 and serves as the selectable cross-check of the other families.
#include "seq_internal.cuh"

namespace ta {
namespace {

constexpr int kWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) seq_fma_kernel(const SeqArgs a) {
    constexpr int E = D / 32;                     // dimensions per lane: lane * E ..
    pdl_wait();
    const int lane = threadIdx.x & 31;
    // every request is checked, those without rows too
    for (long long b = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; b < a.B; b += static_cast<long long>(gridDim.x) * blockDim.x)
        if (seq_request(a, static_cast<int>(b)).bad) atomicOr(a.status, kSeqBadLength);
    const long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(a.T) * a.H) return;
    const int t = static_cast<int>(row / a.H), h = static_cast<int>(row % a.H), kh = h / a.g;
    // the last request that starts at or before t
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu + mid) <= t) lo = mid; else hi = mid;
    }
    const SeqReq r = seq_request(a, lo);
    const int i = t - r.q0;
    if (i < 0 || i >= r.qn) return;               // behind the last sequence: left as it was

    const T *q = static_cast<const T *>(a.q) + t * a.q_st + h * a.q_sh + lane * E;
    float qf[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) { qf[e] = to_f32(q[e]) * a.scale; o[e] = 0.0f; }
    const int prefix = r.kv - r.qn, pos = prefix + i;
    uint32_t anc[kMaxTreeBitsNodes / 32] = {};
    int last = min(pos, r.kv - 1), first = 0;
    if (a.parents) {
        last = r.kv - 1;
        for (int n = i;;) {                       // the chain i, parents[i], ...
            anc[n >> 5] |= 1u << (n & 31);
            const int p = __ldg(a.parents + r.q0 + n);
            if (p < 0 || p >= n) break;
            n = p;
        }
    } else if (a.window) {
        first = max(0, pos - a.window + 1);
    }
    float m = -INFINITY, l = 0.0f;
    for (int j = first; j <= last; ++j) {
        if (a.parents && j >= prefix && !((anc[(j - prefix) >> 5] >> ((j - prefix) & 31)) & 1u)) continue;
        long long ko, vo;
        if (a.kv_lens) {
            const int page = __ldg(a.table + static_cast<long long>(lo) * a.max_pages + (j >> a.page_shift));
            if (page < 0 || page >= a.n_pages) {
                if (lane == 0) atomicOr(a.status, kSeqBadPage);
                continue;
            }
            ko = vo = page * a.k_sp + (j & ((1 << a.page_shift) - 1)) * a.k_st + kh * a.k_sh;
        } else {
            ko = (static_cast<long long>(r.q0) + j) * a.k_st + kh * a.k_sh;
            vo = (static_cast<long long>(r.q0) + j) * a.v_st + kh * a.v_sh;
        }
        const T *k = static_cast<const T *>(a.k) + ko + lane * E;
        const T *v = static_cast<const T *>(a.v) + vo + lane * E;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(qf[e], to_f32(k[e]), s);
        s = warp_sum(s);
        // relative to a finite max, so that a NaN logit is kept (fmaxf drops it) wherever it stands
        const float mn = fmaxf(m, s), mu = mn == -INFINITY ? 0.0f : mn;
        const float c = expf(m - mu), p = expf(s - mu);
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * to_f32(v[e]);
        m = mn;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T *out = static_cast<T *>(a.out) + t * a.o_st + h * a.o_sh + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = static_cast<T>(o[e] * inv);
}

template <typename T>
cudaError_t launch(const SeqArgs &a, cudaStream_t s) {
    const long long rows = static_cast<long long>(a.T) * a.H;
    const dim3 grid(static_cast<unsigned>((rows + kWarps - 1) / kWarps));
    if (a.D == 64) return launch_pdl(seq_fma_kernel<T, 64>, grid, dim3(kWarps * 32), 0, s, a);
    if (a.D == 128) return launch_pdl(seq_fma_kernel<T, 128>, grid, dim3(kWarps * 32), 0, s, a);
    return launch_pdl(seq_fma_kernel<T, 256>, grid, dim3(kWarps * 32), 0, s, a);
}

}  // namespace

cudaError_t launch_seq_fma(const SeqArgs &a, cudaStream_t s) {
    const cudaError_t e = a.bf16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
    count_launch();
    return e;
}

}  // namespace ta
