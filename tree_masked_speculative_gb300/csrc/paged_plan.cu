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
// The work is a few prefix sums over the batch and 12 bytes a token, so latency
// bounds it, not bandwidth.  One cluster does the batch in one launch: every CTA scans
// all of it (cheaper than exchanging results) and takes its share of pages, a
// (row, cell) pair a thread; cluster barriers separate the phases that hand pages over
// through memory (pushes before pops, pops before slots).  Few tokens get their slots
// in the same launch; many in a second one over the whole GPU (131k tokens by the 8
// CTAs of the cluster: 32 us in all, with one warp a row and one token a thread).
#include "seq_internal.cuh"
#include "sm100_ptx.cuh"

namespace ta {
namespace {

constexpr int kThreads = 512;
constexpr int kTokensHere = 4096;       // up to this many tokens get their slots in the planning launch
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
    const int me = rank * kThreads + tid, all = nr * kThreads;
    // the last row whose exclusive sum is at most k: the row of page (or token) k
    auto row_of = [&](const int *sums, int k) {
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sums[mid] <= k) lo = mid; else hi = mid;
        }
        return lo;
    };
    auto need_of = [&](int b) { return static_cast<int>((static_cast<long long>(a.keep[b]) + a.fresh[b] + ps - 1) >> a.page_shift); };
    if (!bad && run.back > 0) {
#pragma unroll 4
        for (int k = me; k < run.back; k += all) {
            const int b = row_of(s_back, k);
            a.stack[n_free + k] = a.table[static_cast<long long>(b) * a.max_pages + need_of(b) + k - s_back[b]];
        }
        sm100::cluster_sync();
    }
    if (!bad) {
#pragma unroll 4
        for (int k = me; k < run.grow; k += all) {
            const int b = row_of(s_grow, k);
            a.table[static_cast<long long>(b) * a.max_pages + need_of(b) - (s_grow[b + 1] - k)] = a.stack[top - 1 - k];
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
    if (a.max_tokens > kTokensHere) return;             // the slots are the next launch's
    const int total = s_cu[a.B];
    for (int t = me; t < a.max_tokens; t += all) {
        long long slot = -1;
        int pos = -1;
        if (t < total) {
            const int b = row_of(s_cu, t);
            pos = a.keep[b] + t - s_cu[b];
            slot = (static_cast<long long>(a.table[static_cast<long long>(b) * a.max_pages + (pos >> a.page_shift)])
                    << a.page_shift) + (pos & (ps - 1));
        }
        a.slot[t] = slot;
        a.pos[t] = pos;
    }
}

// Slots and positions of 4 consecutive tokens a thread, from the row offsets and
// tables that the first kernel has written.
constexpr int kSlotThreads = 256, kSlotTokens = 4, kSlotRows = 2048;
__global__ void __launch_bounds__(kSlotThreads) paged_slots_kernel(const PlanArgs a) {
    __shared__ int s_cu[kSlotRows + 1];
    pdl_wait();
    const bool here = a.B <= kSlotRows;
    if (here) {
        for (int i = threadIdx.x; i <= a.B; i += kSlotThreads) s_cu[i] = a.cu[i];
        __syncthreads();
    }
    const int *cu = here ? s_cu : a.cu;
    const int t0 = (blockIdx.x * kSlotThreads + threadIdx.x) * kSlotTokens;
    if (t0 >= a.max_tokens) return;
    const int total = cu[a.B], mask = (1 << a.page_shift) - 1;
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t0) lo = mid; else hi = mid;
    }
    long long slot[kSlotTokens];
    int pos[kSlotTokens];
    int row = -1, cell = -1, page = 0, keep = 0, first = 0, end = cu[lo + 1];
#pragma unroll
    for (int i = 0; i < kSlotTokens; ++i) {
        const int t = t0 + i;
        slot[i] = -1;
        pos[i] = -1;
        if (t >= total) continue;
        while (t >= end) end = cu[++lo + 1];            // ends: t < total = cu[B]
        if (lo != row) {
            row = lo;
            keep = a.keep[row];
            first = cu[row];
            cell = -1;
        }
        pos[i] = keep + t - first;
        if ((pos[i] >> a.page_shift) != cell) {
            cell = pos[i] >> a.page_shift;
            page = a.table[static_cast<long long>(row) * a.max_pages + cell];
        }
        slot[i] = (static_cast<long long>(page) << a.page_shift) + (pos[i] & mask);
    }
    const bool wide = t0 + kSlotTokens <= a.max_tokens && ((reinterpret_cast<uintptr_t>(a.slot) | reinterpret_cast<uintptr_t>(a.pos)) & 15) == 0;
    if (wide) {
        *reinterpret_cast<longlong2 *>(a.slot + t0) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2 *>(a.slot + t0 + 2) = make_longlong2(slot[2], slot[3]);
        *reinterpret_cast<int4 *>(a.pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kSlotTokens; ++i)
            if (t0 + i < a.max_tokens) {
                a.slot[t0 + i] = slot[i];
                a.pos[t0 + i] = pos[i];
            }
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
    const unsigned ctas = a.B <= kThreads / 2 && a.max_tokens <= kThreads ? 1 : 8;
    cudaError_t e = launch_pdl_cluster(paged_plan_kernel, dim3(ctas), dim3(kThreads), smem, s, ctas, 1u, a);
    count_launch();
    if (e != cudaSuccess || a.max_tokens <= kTokensHere) return e;
    const unsigned blocks = (static_cast<unsigned>(a.max_tokens) + kSlotThreads * kSlotTokens - 1) / (kSlotThreads * kSlotTokens);
    e = launch_pdl(paged_slots_kernel, dim3(blocks), dim3(kSlotThreads), 0, s, a);
    count_launch();
    return e;
}

}  // namespace ta
