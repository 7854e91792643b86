// New rows turned by their positions: queries to q_out, keys and values to 16-bit pages, one
// launch.  A pair (x1, x2) of row t becomes (x1 c - x2 s, x2 c + x1 s), c and s from the row
// of the table that belongs to its position.
//
// It moves 4 D bytes a query head and 8 D a KV head and token, so HBM bounds it; a thread takes
// the two vectors of a column that belong together, of up to HB heads, so that a cosine and sine
// (4 bytes each against 2 of an element) are loaded once for them and 2 HB loads are in flight.
// Measured: 16381 tokens, 24 / 4 heads of 256, half of each turned (545 MB): 80 us, 6.8 TB/s; 64 tokens, 32 / 8 heads of
// 128: 2.2 us.
#include "rotary.cuh"

namespace ta {
namespace {

// Blocks [0, nq) turn queries, [nq, nq + nk) keys, the others copy values.
template <bool BF16, int HB>
__global__ void __launch_bounds__(kRotThreads) rotary_append_kernel(const RotaryAppendArgs ar, unsigned nq, unsigned nk) {
    pdl_wait();
    const RotaryArgs &a = ar.r;
    if (blockIdx.x < nq) {
        turn_queries<BF16, HB>(a, static_cast<long long>(blockIdx.x) * kRotThreads + threadIdx.x);
        return;
    }
    const bool is_v = blockIdx.x >= nq + nk;
    const long long x = static_cast<long long>(blockIdx.x - (is_v ? nq + nk : nq)) * kRotThreads + threadIdx.x;
    const unsigned cols = static_cast<unsigned>(a.D) >> 4, blocks = (static_cast<unsigned>(a.Hk) + HB - 1) / HB;
    const long long t = item_token(x, cols * blocks);
    if (t >= a.T) return;
    const unsigned r = static_cast<unsigned>(x - t * (cols * blocks)), hb = r / cols, c = r - hb * cols;
    const float *row = rot_row(a, static_cast<int>(t));
    const long long slot = a.slot[t];
    if (row == nullptr || slot < 0 || slot >= static_cast<long long>(a.n_pages) << a.page_shift) return;
    const int h = static_cast<int>(hb) * HB, heads = min(HB, a.Hk - h);
    const long long at = (slot >> a.page_shift) * ar.c_sp + (slot & ((1ll << a.page_shift) - 1)) * ar.c_st + h * ar.c_sh;
    if (!is_v) {
        turn_rows<BF16, HB>(a, row, static_cast<int>(c), heads, static_cast<const uint4 *>(a.k_new) + t * a.k_st + h * a.k_sh, a.k_sh,
                            static_cast<uint4 *>(ar.k) + at, ar.c_sh);
        return;
    }
    const uint4 *src = static_cast<const uint4 *>(a.v_new) + t * a.v_st + h * a.v_sh + c;
    uint4 *dst = static_cast<uint4 *>(ar.v) + at + c, y[HB][2];
#pragma unroll
    for (int i = 0; i < HB; ++i)
        if (i < heads) {
            y[i][0] = src[i * a.v_sh];
            y[i][1] = src[i * a.v_sh + cols];
        }
#pragma unroll
    for (int i = 0; i < HB; ++i)
        if (i < heads) {
            dst[i * ar.c_sh] = y[i][0];
            dst[i * ar.c_sh + cols] = y[i][1];
        }
}

template <bool BF16, int HB>
cudaError_t launch(const RotaryAppendArgs &a, cudaStream_t s) {
    const long long nq = a.r.H ? rot_blocks(a.r.T, a.r.H, HB, a.r.D / 16) : 0, nk = rot_blocks(a.r.T, a.r.Hk, HB, a.r.D / 16);
    if (nq + 2 * nk > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_pdl(rotary_append_kernel<BF16, HB>, dim3(static_cast<unsigned>(nq + 2 * nk)), dim3(kRotThreads), 0, s, a,
                                     static_cast<unsigned>(nq), static_cast<unsigned>(nk));
    count_launch();
    return e;
}

}  // namespace

cudaError_t launch_rotary_append(const RotaryAppendArgs &a, cudaStream_t s) {
    // one head a thread while that leaves the GPU's thread slots unfilled (more loads of the table, but all of them at once)
    const bool few = static_cast<long long>(a.r.T) * (a.r.H + 2 * a.r.Hk) * (a.r.D / 16) <= 152ll * 2048;
    if (a.r.bf16) return few ? launch<true, 1>(a, s) : launch<true, 4>(a, s);
    return few ? launch<false, 1>(a, s) : launch<false, 4>(a, s);
}

}  // namespace ta
