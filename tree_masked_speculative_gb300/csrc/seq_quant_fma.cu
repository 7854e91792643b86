// Attention of ragged rows over 4-bit pages on CUDA cores: one warp per (token, head) row,
// the keys one after the other, an online softmax in f32, each element widened on its way
// (scale * code + bias in f32).  Every row reads all its keys, so L2 and the decoding bound
// it; it serves as the selectable cross-check of the other families and takes negative scales.
#include "quant_page.cuh"

namespace ta {
namespace {

constexpr int kWarps = 4;

// A lane's E = D / 32 codes of a row, from the lowest nibble on.
template <int E>
__device__ __forceinline__ uint32_t lane_codes(const uint32_t *row, int lane) {
    if constexpr (E == 2) return reinterpret_cast<const uint8_t *>(row)[lane];
    else if constexpr (E == 4) return reinterpret_cast<const uint16_t *>(row)[lane];
    else return row[lane];
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) seq_quant_fma_kernel(const SeqQuantArgs ar) {
    constexpr int E = D / 32;                     // elements per lane
    const SeqArgs &a = ar.s;
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

    // the lane's codes are nibbles n of quad g of block j: elements d0 .. d0 + E - 1 (E = 8: two
    // quads, of blocks j and j + 1, 32 elements apart)
    const int quad = lane * E / 4, j = quad % (D / 32), g = quad / (D / 32), n = lane * E % 4;
    const int d0 = 32 * j + 4 * g + n;
    auto element = [&](int e) { return E == 8 && e >= 4 ? d0 + 28 + e : d0 + e; };
    const T *q = static_cast<const T *>(a.q) + t * a.q_st + h * a.q_sh;
    float qf[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) { qf[e] = to_f32(q[element(e)]) * a.scale; o[e] = 0.0f; }
    const int prefix = r.kv - r.qn, pos = prefix + i;
    uint32_t anc[kMaxTreeBitsNodes / 32] = {};
    int last = min(pos, r.kv - 1), first = 0;
    if (a.parents) {
        last = r.kv - 1;
        for (int m = i;;) {                       // the chain i, parents[i], ...
            anc[m >> 5] |= 1u << (m & 31);
            const int p = __ldg(a.parents + r.q0 + m);
            if (p < 0 || p >= m) break;
            m = p;
        }
    } else if (a.window) {
        first = max(0, pos - a.window + 1);
    }
    float m = -INFINITY, l = 0.0f;
    for (int key = first; key <= last; ++key) {
        if (a.parents && key >= prefix && !((anc[(key - prefix) >> 5] >> ((key - prefix) & 31)) & 1u)) continue;
        const int page = __ldg(a.table + static_cast<long long>(lo) * a.max_pages + (key >> a.page_shift));
        if (page < 0 || page >= a.n_pages) {
            if (lane == 0) atomicOr(a.status, kSeqBadPage);
            continue;
        }
        const int in = key & ((1 << a.page_shift) - 1);
        auto codes = [&](const uint32_t *c) { return lane_codes<E>(at_bytes(at_bytes(at_bytes(c, page, ar.c.c_sp), kh, ar.c.c_sh), in, ar.c.c_st), lane); };
        auto affine = [&](const void *f) { return at_bytes(at_bytes(at_bytes(static_cast<const T *>(f), page, ar.c.a_sp), kh, ar.c.a_sh), in, ar.c.a_st); };
        const uint32_t kw = codes(ar.c.kc), vw = codes(ar.c.vc);
        const T *ka = affine(ar.c.ka), *va = affine(ar.c.va);
        float s = 0.0f, v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int gr = 2 * (element(e) / ar.group);
            s = fmaf(qf[e], fmaf(to_f32(ka[gr]), static_cast<float>((kw >> (4 * e)) & 15u), to_f32(ka[gr + 1])), s);
            v[e] = fmaf(to_f32(va[gr]), static_cast<float>((vw >> (4 * e)) & 15u), to_f32(va[gr + 1]));
        }
        s = warp_sum(s);
        // relative to a finite max, so that a NaN logit is kept (fmaxf drops it) wherever it stands
        const float mn = fmaxf(m, s), mu = mn == -INFINITY ? 0.0f : mn;
        const float c = expf(m - mu), p = expf(s - mu);
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * v[e];
        m = mn;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T *out = static_cast<T *>(a.out) + t * a.o_st + h * a.o_sh;
#pragma unroll
    for (int e = 0; e < E; ++e) out[element(e)] = static_cast<T>(o[e] * inv);
}

template <typename T>
cudaError_t launch(const SeqQuantArgs &a, cudaStream_t s) {
    const long long rows = static_cast<long long>(a.s.T) * a.s.H;
    const dim3 grid(static_cast<unsigned>((rows + kWarps - 1) / kWarps));
    if (a.s.D == 64) return launch_pdl(seq_quant_fma_kernel<T, 64>, grid, dim3(kWarps * 32), 0, s, a);
    if (a.s.D == 128) return launch_pdl(seq_quant_fma_kernel<T, 128>, grid, dim3(kWarps * 32), 0, s, a);
    return launch_pdl(seq_quant_fma_kernel<T, 256>, grid, dim3(kWarps * 32), 0, s, a);
}

}  // namespace

cudaError_t launch_seq_quant_fma(const SeqQuantArgs &a, cudaStream_t s) {
    const cudaError_t e = a.s.bf16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
    count_launch();
    return e;
}

}  // namespace ta
