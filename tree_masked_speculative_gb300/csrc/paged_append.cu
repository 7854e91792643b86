// New K/V rows to their pages.  Row t of k_new / v_new ([T, Hk, D]) goes to
// page slot / page_size, token slot % page_size of the cache; a slot outside
// [0, n_pages * page_size) (in particular -1) stores nothing.
//
// A copy: 4 T Hk D bytes each way and 8 T bytes of slots, bound by HBM.  A
// thread moves one 16-byte vector of K and the matching one of V per step, so
// every row is read and written in whole 128-byte lines.  32749 tokens of 4 heads x
// 256: 42.5 us, 6.3 TB/s (93 % of a plain copy's rate); 64 tokens of 8 x 128: 1.9 us
// of the GPU.
#include "seq_internal.cuh"

namespace ta {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendArgs a) {
    pdl_wait();
    const unsigned vec = static_cast<unsigned>(a.D) / 8, per_token = vec * a.Hk;
    const long long n = static_cast<long long>(a.T) * per_token;
    const long long slots = static_cast<long long>(a.n_pages) << a.page_shift;
    const uint4 *kn = static_cast<const uint4 *>(a.k_new), *vn = static_cast<const uint4 *>(a.v_new);
    uint4 *kc = static_cast<uint4 *>(a.k), *vc = static_cast<uint4 *>(a.v);
    for (long long x = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; x < n;
         x += static_cast<long long>(gridDim.x) * kThreads) {
        const long long t = x / per_token;
        const unsigned r = static_cast<unsigned>(x - t * per_token), h = r / vec, c = r % vec;
        const long long slot = a.slot[t];
        if (slot < 0 || slot >= slots) continue;
        const long long dst = (slot >> a.page_shift) * a.c_sp + (slot & ((1ll << a.page_shift) - 1)) * a.c_st + h * a.c_sh + c;
        kc[dst] = kn[t * a.kn_st + h * a.kn_sh + c];
        vc[dst] = vn[t * a.vn_st + h * a.vn_sh + c];
    }
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs &a, cudaStream_t s) {
    const long long n = static_cast<long long>(a.T) * a.Hk * (a.D / 8);
    const long long blocks = (n + kThreads - 1) / kThreads;
    const cudaError_t e = launch_pdl(paged_append_kernel, dim3(static_cast<unsigned>(blocks < 152 * 8 ? blocks : 152 * 8)),
                                     dim3(kThreads), 0, s, a);
    count_launch();
    return e;
}

}  // namespace ta
