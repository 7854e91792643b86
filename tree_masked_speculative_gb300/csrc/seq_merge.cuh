// What the warp-MMA kernels over 16-bit and 4-bit pages share: small helpers and the merge of cut
// units' pieces.
#pragma once

#include "seq_sched.cuh"

namespace ta {
namespace {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// K and V are read once: past L1.
__device__ __forceinline__ uint4 load_once(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}
// out = sum_p O_p 2^(m_p - m*) / sum_p l_p 2^(m_p - m*) over the pieces of the cut unit
// that starts in CTA blockIdx.x.  A few units are cut into many pieces when the
// batch is small, so a block's threads share the pieces as well as the columns
// (one thread a column through all of 22 pieces took 14 us).
constexpr int kMergeThreads = 256;
// CAP: rows of a partial slot.  COLS: columns a block takes (blockIdx.y), fewer than D where a few units of many pieces
// would leave the work to a few blocks.
template <int D, int CAP, bool BF16, int COLS = D>
__global__ void __launch_bounds__(kMergeThreads) seq_mma_merge_kernel(const SeqArgs a, const SeqRec *recs, const float2 *ml, const float *o) {
    __shared__ float s_m[CAP], s_inv[CAP];
    __shared__ float4 s_part[kMergeThreads];
    pdl_wait();
    const int c = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const SeqRec rec = recs[c];
    if (rec.parts == 0) return;
    auto slot = [&](int p) { return static_cast<size_t>(p == 0 ? 2 * c + 1 : 2 * (c + p)); };
    for (int row = warp; row < rec.rows; row += kMergeThreads / 32) {
        float m = -INFINITY, l = 0.0f;
#pragma unroll 2
        for (int p = lane; p < rec.parts; p += 32) {
            const float2 w = ml[slot(p) * CAP + row];
            const float mn = fmaxf(m, w.x), mu = mn == -INFINITY ? 0.0f : mn;
            l = l * ex2(m - mu) + w.y * ex2(w.x - mu);
            m = mn;
        }
        const float mr = warp_max(m), mu = mr == -INFINITY ? 0.0f : mr;
        l = warp_sum(l * ex2(m - mu));
        if (lane == 0) {
            s_m[row] = mu;
            s_inv[row] = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
        }
    }
    __syncthreads();
    // items: 4 columns of a row; `share` threads take the pieces of one item in turn
    const int items = rec.rows * (COLS / 4);
    int share = 1;
    while (2 * share * items <= kMergeThreads) share *= 2;
    const int per = kMergeThreads / share;              // items at a time
    for (int i0 = 0; i0 < items; i0 += per) {
        const int k = tid / per, i = i0 + tid - k * per;
        float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int row = i / (COLS / 4), d = blockIdx.y * COLS + (i - row * (COLS / 4)) * 4;
        if (i < items) {
            const float mu = s_m[row];
#pragma unroll 4
            for (int p = k; p < rec.parts; p += share) {
                const float f = ex2(ml[slot(p) * CAP + row].x - mu);
                const float4 y = *reinterpret_cast<const float4 *>(o + (slot(p) * CAP + row) * D + d);
                r.x += f * y.x; r.y += f * y.y; r.z += f * y.z; r.w += f * y.w;
            }
        }
        s_part[tid] = r;
        __syncthreads();
        if (k == 0 && i < items) {
            for (int j = 1; j < share; ++j) {
                const float4 y = s_part[tid + j * per];
                r.x += y.x; r.y += y.y; r.z += y.z; r.w += y.w;
            }
            const float inv = s_inv[row];
            const int tk = row / a.g;
            uint16_t *out = static_cast<uint16_t *>(a.out) + static_cast<long long>(rec.token + tk) * a.o_st +
                            static_cast<long long>(rec.kh * a.g + row - tk * a.g) * a.o_sh + d;
            *reinterpret_cast<uint2 *>(out) = make_uint2(pack16<BF16>(r.x * inv, r.y * inv), pack16<BF16>(r.z * inv, r.w * inv));
        }
        __syncthreads();
    }
}

}  // namespace
}  // namespace ta
