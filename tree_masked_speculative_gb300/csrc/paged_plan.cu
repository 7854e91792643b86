// Step planning on the device: from the lengths of a batch of requests, which
// pages they give back or take, their block tables, and every new token's
// cache slot.
//
//   need[b]  = ceil((keep[b] + fresh[b]) / page_size)
//   released : cells need <= j < held of each row are pushed on the free stack,
//              in (row, cell) order
//   taken    : cells held <= j < need are popped off its top, in (row, cell) order
//   cu       = exclusive prefix sum of fresh;  lens = keep + fresh
//   slot[t]  = table[b, pos / page_size] * page_size + pos % page_size with
//              pos = keep[b] + t - cu[b]; -1 for t >= cu[B]
//
// The work is a few prefix sums over the batch and 12 bytes a token, so a
// launch's latency bounds it, not bandwidth.  One cluster does all of it in one
// launch: every CTA scans the whole batch (cheaper than exchanging results) and
// takes its share of rows and tokens; cluster barriers separate the phases that
// hand pages over through memory (pushes before pops, pops before slots).
#include "seq_internal.cuh"
#include "sm100_ptx.cuh"

namespace ta {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct Sums {
    int back, grow;
    long long fresh;
};

// Inclusive sums over the block of one (back, grow, fresh) per thread, and the
// block's totals.
__device__ Sums block_scan(Sums x, Sums *warp_tot, Sums *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int b = __shfl_up_sync(0xffffffffu, x.back, o), g = __shfl_up_sync(0xffffffffu, x.grow, o);
        const long long f = __shfl_up_sync(0xffffffffu, x.fresh, o);
        if (lane >= o) { x.back += b; x.grow += g; x.fresh += f; }
    }
    if (lane == 31) warp_tot[warp] = x;
    __syncthreads();
    Sums all = {0, 0, 0};
    for (int w = 0; w < kWarps; ++w) {
        const Sums y = warp_tot[w];
        if (w < warp) { x.back += y.back; x.grow += y.grow; x.fresh += y.fresh; }
        all.back += y.back; all.grow += y.grow; all.fresh += y.fresh;
    }
    *total = all;
    __syncthreads();
    return x;
}

__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const PlanArgs a) {
    // per row: exclusive sums of pages given back, of pages taken, of tokens
    extern __shared__ int rows[];
    int *s_back = rows, *s_grow = rows + a.B + 1, *s_cu = rows + 2 * (a.B + 1);
    __shared__ Sums warp_tot[kWarps];
    __shared__ int s_bad;
    pdl_wait();
    const int tid = threadIdx.x, rank = static_cast<int>(sm100::cluster_ctarank()), nr = static_cast<int>(sm100::cluster_nctarank());
    const int ps = 1 << a.page_shift;
    const long long room = static_cast<long long>(a.max_pages) << a.page_shift;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    const int n_free = *a.n_free;
    Sums run = {0, 0, 0};
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        Sums x = {0, 0, 0};
        if (b < a.B) {
            const int keep = a.keep[b], fresh = a.fresh[b], held = a.held[b];
            const long long len = static_cast<long long>(keep) + fresh;
            if (keep < 0 || fresh < 0 || held < 0 || held > a.max_pages || len > room) {
                s_bad = 1;
            } else {
                const int need = static_cast<int>((len + ps - 1) >> a.page_shift);
                x.back = max(held - need, 0);
                x.grow = max(need - held, 0);
                x.fresh = fresh;
            }
        }
        Sums tot;
        const Sums inc = block_scan(x, warp_tot, &tot);
        if (b < a.B) {
            s_back[b] = run.back + inc.back - x.back;
            s_grow[b] = run.grow + inc.grow - x.grow;
            s_cu[b] = static_cast<int>(min(run.fresh + inc.fresh - x.fresh, 0x7fffffffll));
        }
        run.back += tot.back; run.grow += tot.grow; run.fresh += tot.fresh;
    }
    int bad = s_bad ? kPlanBadLength : 0;
    if (n_free < 0 || n_free > a.capacity || static_cast<long long>(n_free) + run.back > a.capacity) bad |= kPlanStack;
    else if (static_cast<long long>(n_free) + run.back < run.grow) bad |= kPlanNoPages;
    if (run.fresh > a.max_tokens) bad |= kPlanTokens;
    if (tid == 0) {
        s_back[a.B] = run.back;
        s_grow[a.B] = run.grow;
        s_cu[a.B] = bad ? 0 : static_cast<int>(run.fresh);
    }
    // every CTA has read held and n_free: the outputs may be the inputs' memory
    sm100::cluster_sync();
    const int top = n_free + run.back;
    const int warp = (tid >> 5) * nr + rank, lane = tid & 31, nw = kWarps * nr;
    if (!bad && run.back > 0) {
        for (int b = warp; b < a.B; b += nw) {
            const int n = s_back[b + 1] - s_back[b];
            if (n == 0) continue;
            const int need = static_cast<int>((static_cast<long long>(a.keep[b]) + a.fresh[b] + ps - 1) >> a.page_shift);
            for (int j = lane; j < n; j += 32)
                a.stack[n_free + s_back[b] + j] = a.table[static_cast<long long>(b) * a.max_pages + need + j];
        }
        sm100::cluster_sync();
    }
    if (!bad) {
        for (int b = warp; b < a.B; b += nw) {
            const int n = s_grow[b + 1] - s_grow[b];
            if (n == 0) continue;
            const int need = static_cast<int>((static_cast<long long>(a.keep[b]) + a.fresh[b] + ps - 1) >> a.page_shift);
            for (int j = lane; j < n; j += 32)
                a.table[static_cast<long long>(b) * a.max_pages + need - n + j] = a.stack[top - 1 - s_grow[b] - j];
        }
    }
    sm100::cluster_sync();
    // row outputs, now that nobody reads the inputs of other rows' pages any more
    for (int b = rank * kThreads + tid; b < a.B; b += nr * kThreads) {
        const int keep = a.keep[b], fresh = a.fresh[b];
        if (!bad) a.held_out[b] = static_cast<int>((static_cast<long long>(keep) + fresh + ps - 1) >> a.page_shift);
        else if (a.held_out != a.held) a.held_out[b] = a.held[b];
        a.lens[b] = bad ? 0 : keep + fresh;
        a.cu[b] = bad ? 0 : s_cu[b];
    }
    if (rank == 0 && tid == 0) {
        a.cu[a.B] = s_cu[a.B];
        *a.n_free_out = bad ? n_free : top - run.grow;
        if (bad) atomicOr(a.status, bad);
    }
    const int total = s_cu[a.B];
    for (int t = rank * kThreads + tid; t < a.max_tokens; t += nr * kThreads) {
        long long slot = -1;
        int pos = -1;
        if (t < total) {
            int lo = 0, hi = a.B;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_cu[mid] <= t) lo = mid; else hi = mid;
            }
            pos = a.keep[lo] + t - s_cu[lo];
            slot = (static_cast<long long>(a.table[static_cast<long long>(lo) * a.max_pages + (pos >> a.page_shift)])
                    << a.page_shift) + (pos & (ps - 1));
        }
        a.slot[t] = slot;
        a.pos[t] = pos;
    }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs &a, cudaStream_t s) {
    static unsigned long long done = 0;
    const size_t smem = 3 * (static_cast<size_t>(a.B) + 1) * sizeof(int);
    if (smem > 40 * 1024) {
        const cudaError_t e = set_smem_limit_once(paged_plan_kernel, 3 * (kPlanMaxBatch + 1) * sizeof(int), &done);
        if (e != cudaSuccess) return e;
    }
    // one CTA where it holds the batch and the tokens in one sweep; else 8
    const unsigned ctas = a.B <= kThreads && a.max_tokens <= kThreads ? 1 : 8;
    const cudaError_t e = launch_pdl_cluster(paged_plan_kernel, dim3(ctas), dim3(kThreads), smem, s, ctas, 1u, a);
    count_launch();
    return e;
}

}  // namespace ta
