// Work schedule of the ragged attention kernels, computed by every CTA from the
// lengths on the device.
//
// A unit is (request, KV head, row tile): `tpt` tokens x g query heads.  Its
// work is the run of key tiles (1 << TKS keys each) some of its rows see, at
// least one, and UC tiles' worth of time before the first (its rows of Q, its
// epilogue).  All units' work, one behind the other (request, then KV head, then row
// tile), is cut into G equal runs (fewer where there is less), one per CTA: the batch
// is balanced whatever its lengths are (LEAST: tiles a run has at least), a unit is cut only where a run ends, and a CTA
// has at most two pieces of cut units (its first and its last), so 2 G partial
// slots hold every cut piece.  (With UC = 0, of the time of a causal prompt of 4096
// tokens a CTA worked 72 % on average: those with the short units ended last.)
#pragma once

#include "seq_internal.cuh"

namespace ta {

// First key tile of a unit and how many it has.
template <int TKS>
__device__ __forceinline__ int seq_unit_tiles(const SeqArgs &a, int qn, int kv, int qt, int tpt, int *first) {
    int lo = 0, hi = kv;
    if (a.parents == nullptr) {
        const int i0 = qt * tpt, i1 = min(qn, i0 + tpt) - 1;
        hi = min(kv, kv - qn + i1 + 1);
        if (a.window) lo = max(0, kv - qn + i0 - a.window + 1);
    }
    const int t0 = lo >> TKS, t1 = (max(hi, 0) + (1 << TKS) - 1) >> TKS;
    *first = t0;
    return max(1, t1 - t0);
}

// Work of one KV head of each lane's request (qn, kv), in key tiles; warp-collective.
// Long requests (more than 4 row tiles) are summed by the whole warp.
template <int TKS, int UC>
__device__ __forceinline__ int seq_head_tiles(const SeqArgs &a, int qn, int kv, int tpt) {
    const int lane = threadIdx.x & 31, nqt = (qn + tpt - 1) / tpt;
    int c = 0, f;
    if (nqt <= 4)
        for (int qt = 0; qt < nqt; ++qt) c += UC + seq_unit_tiles<TKS>(a, qn, kv, qt, tpt, &f);
    for (uint32_t big = __ballot_sync(0xffffffffu, nqt > 4); big; big &= big - 1) {
        const int src = __ffs(big) - 1;
        const int qn_s = __shfl_sync(0xffffffffu, qn, src), kv_s = __shfl_sync(0xffffffffu, kv, src);
        const int n = (qn_s + tpt - 1) / tpt;
        int s = 0;
        for (int qt = lane; qt < n; qt += 32) s += UC + seq_unit_tiles<TKS>(a, qn_s, kv_s, qt, tpt, &f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == src) c = s;
    }
    return c;
}

struct SeqRec {
    int parts;      // pieces of the cut unit that starts in this CTA (0: none)
    int token;      // its first row of q / out
    int kh, rows;
};

// Cut of W tiles of work into G runs whose lengths differ by one at most: CTA c
// starts at c * base + min(c, extra).
struct SeqRun {
    long long W, P0, P1;
    long long base;
    int G, extra;       // G: CTAs with a run, one tile of work at least for each
    __device__ __forceinline__ long long start(int c) const { return c * base + min(c, extra); }
    // CTA whose run holds position P
    __device__ __forceinline__ int cta_of(long long P) const {
        const long long big = extra * (base + 1);
        const long long x = P < big ? P : P - big, d = P < big ? base + 1 : base;
        const int q = W <= 0x7fffffffll ? static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(d)) : static_cast<int>(x / d);
        return P < big ? q : extra + q;
    }
};

struct SeqScratch {
    long long warp_tot[32];
    long long off;      // start inside the first request
    SeqReq r;           // the first request
    int b, per_head;    // its index; its work of one KV head
};

// This CTA's run [P0, P1) of the W tiles of work and where it starts (in *s, valid when
// P0 < P1).  Block-collective.
template <int NT, int TKS, int UC, int LEAST>
__device__ SeqRun seq_schedule(const SeqArgs &a, int tpt, int cta, int G, SeqScratch *s) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    SeqReq r;
    int per_head;
    auto tiles_of = [&](int b) -> long long {      // warp-collective
        r = {0, 0, 0, false};
        if (b < a.B) r = seq_request(a, b);
        if (r.bad && cta == 0) atomicOr(a.status, kSeqBadLength);
        per_head = seq_head_tiles<TKS, UC>(a, r.qn, r.kv, tpt);
        return static_cast<long long>(per_head) * a.Hk;
    };
    // inclusive sum over the block's threads; *total of all
    auto scan = [&](long long x, long long *total) -> long long {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) s->warp_tot[warp] = x;
        __syncthreads();
        long long all = 0;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            const long long y = s->warp_tot[w];
            if (w < warp) x += y;
            all += y;
        }
        *total = all;
        return x;
    };
    SeqRun run;
    long long mine = tiles_of(tid), tot;
    long long inc = scan(mine, &tot);
    run.W = tot;
#pragma unroll 1
    for (int b0 = NT; b0 < a.B; b0 += NT) {
        long long t;
        scan(tiles_of(b0 + tid), &t);
        run.W += t;
    }
    run.G = static_cast<int>(min(static_cast<long long>(G), max(1ll, run.W / LEAST)));
    if (run.W == 0) run.G = 0;
    if (run.W <= 0x7fffffffll) {
        const uint32_t g = max(run.G, 1), w = static_cast<uint32_t>(run.W), q = w / g;
        run.base = q;
        run.extra = static_cast<int>(w - q * g);
    } else {
        run.base = run.W / run.G;
        run.extra = static_cast<int>(run.W - run.base * run.G);
    }
    run.P0 = cta < run.G ? run.start(cta) : run.W;
    run.P1 = cta < run.G ? run.start(cta + 1) : run.W;
    long long before = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        if (b0 > 0 || a.B > NT) {
            mine = tiles_of(b0 + tid);
            inc = scan(mine, &tot);
        }
        if (run.P0 < run.P1 && run.P0 >= before + inc - mine && run.P0 < before + inc) {
            s->b = b0 + tid;
            s->r = r;
            s->per_head = per_head;
            s->off = run.P0 - (before + inc - mine);
        }
        before += tot;
        if (before > run.P0) break;
    }
    __syncthreads();
    return run;
}

// One piece of a unit: a run of its key tiles worked on by one CTA.
struct SeqPiece {
    int valid;
    int b, kh;
    int q0, i0;          // the request's first row; the unit's first token in it
    int rows;            // rows of the unit (tokens x g)
    int kv, prefix;      // keys; position of the request's token 0 (kv - q_len)
    int t0, nt;          // first key tile, key tiles
    int full_lo, full_hi;  // every row sees the keys in [full_lo, full_hi)
    int slot;            // partial slot, or -1: the whole unit
    long long pos;       // position of its first tile among all
    int rest;            // key tiles of the unit after this piece, counted in a cut unit's first piece (else 0)
};

// Walks this CTA's pieces.  Warp-collective; all lanes hold the same state.
template <int TKS, int UC>
struct SeqWalk {
    long long left, pos;
    int b, u, off, nqt, cta;
    SeqReq r;

    __device__ void enter(const SeqArgs &a, int tpt) {
        r = seq_request(a, b);
        nqt = (r.qn + tpt - 1) / tpt;
    }
    __device__ void init(const SeqArgs &a, int tpt, const SeqRun &run, const SeqScratch *s, int cta_) {
        left = run.P1 - run.P0;
        pos = run.P0;
        cta = cta_;
        if (left <= 0) return;
        b = s->b;
        r = s->r;
        nqt = (r.qn + tpt - 1) / tpt;
        const long long o = s->off;
        const int c = s->per_head;
        const int kh = o <= 0x7fffffffll ? static_cast<int>(static_cast<uint32_t>(o) / static_cast<uint32_t>(c)) : static_cast<int>(o / c);
        off = static_cast<int>(o - static_cast<long long>(kh) * c);
        if (nqt == 1) {
            u = kh;
            return;
        }
        int qt = 0;
        // the row tile that holds tile `off` of this KV head, 32 row tiles a step
        for (;; qt += 32) {
            const int lane = threadIdx.x & 31;
            int f, x = qt + lane < nqt ? UC + seq_unit_tiles<TKS>(a, r.qn, r.kv, qt + lane, tpt, &f) : 0;
            const int n = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, off < x);
            if (hit) {
                const int l = __ffs(hit) - 1;
                off -= __shfl_sync(0xffffffffu, x - n, l);
                qt += l;
                break;
            }
            off -= __shfl_sync(0xffffffffu, x, 31);
            if (qt + 32 >= nqt) { qt = nqt - 1; off = 0; break; }    // not reached
        }
        u = kh * nqt + qt;
    }
    __device__ bool next(const SeqArgs &a, int tpt, const SeqRun &run, SeqPiece *p) {
        if (left <= 0) return false;
        int first;
        const int kh = nqt == 1 ? u : u / nqt, qt = u - kh * nqt, n = seq_unit_tiles<TKS>(a, r.qn, r.kv, qt, tpt, &first);
        // the run may begin or end in the time before a unit's first tile
        const int before = max(0, UC - off), t = max(0, off - UC);
        if (left <= before) {
            left = 0;
            return false;
        }
        p->valid = 1;
        p->b = b;
        p->kh = kh;
        p->q0 = r.q0;
        p->i0 = qt * tpt;
        const int nt_tok = min(tpt, r.qn - p->i0);
        p->rows = nt_tok * a.g;
        p->kv = r.kv;
        p->prefix = r.kv - r.qn;
        p->t0 = first + t;
        p->nt = static_cast<int>(min(static_cast<long long>(n - t), left - before));
        p->full_hi = a.parents ? p->prefix : p->prefix + p->i0 + 1;
        p->full_lo = a.parents || !a.window ? 0 : max(0, p->prefix + p->i0 + nt_tok - a.window);
        const bool starts = t == 0, ends = t + p->nt == n;
        p->slot = starts && ends ? -1 : starts ? 2 * cta + 1 : 2 * cta;
        p->rest = starts && !ends ? n - p->nt : 0;
        p->pos = pos + before;
        pos += before + p->nt;
        left -= before + p->nt;
        off = 0;
        ++u;
        if (left > 0 && u == a.Hk * nqt) {
            do {
                if (++b >= a.B) { left = 0; break; }
                enter(a, tpt);
            } while (r.qn == 0);
            u = 0;
        }
        return true;
    }
};

// Record of a cut unit's first piece, for the merge.
__device__ __forceinline__ SeqRec seq_record(const SeqRun &run, int cta, const SeqPiece &p) {
    return {run.cta_of(p.pos + p.nt + p.rest - 1) - cta + 1, p.q0 + p.i0, p.kh, p.rows};
}

// Bit e of word w: does row `i` (token of its request) of a piece see key
// k0 + 32 w + e.  `anc`: the token's ancestor bits (trees).
template <int NW>
__device__ __forceinline__ void seq_visible(const SeqArgs &a, int prefix, int kv, int i, const uint32_t *anc, int k0,
                                            uint32_t (&m)[NW]) {
    int lo = 0, hi = min(kv, prefix + i + 1);
    if (a.parents) hi = min(kv, prefix);
    else if (a.window) lo = max(0, prefix + i - a.window + 1);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const int k = k0 + 32 * w;
        const int x = hi - k, y = lo - k;                     // bits [y, x)
        uint32_t v = x <= 0 ? 0u : x >= 32 ? 0xffffffffu : (1u << x) - 1u;
        v &= y <= 0 ? 0xffffffffu : y >= 32 ? 0u : ~((1u << y) - 1u);
        if (a.parents) {
            // tree positions prefix + n for the set bits n of anc: 32 of them from
            // bit k - prefix on
            const int n = k - prefix, wi = n >> 5, sh = n & 31;
            const uint32_t l = wi >= 0 && wi < kMaxTreeBitsNodes / 32 ? anc[wi] : 0u;
            const uint32_t h = wi + 1 >= 0 && wi + 1 < kMaxTreeBitsNodes / 32 ? anc[wi + 1] : 0u;
            uint32_t t = sh ? (l >> sh) | (h << (32 - sh)) : l;
            // keys before position 0 or past the last key do not exist
            const int past = kv - k;
            t &= past <= 0 ? 0u : past >= 32 ? 0xffffffffu : (1u << past) - 1u;
            v |= t;
        }
        m[w] = v;
    }
}

// Ancestor bits of token i: the chain i, parents[i], ... (row q0 holds token 0).
__device__ __forceinline__ void seq_ancestors(const int32_t *parents, int i, uint32_t (&anc)[kMaxTreeBitsNodes / 32]) {
#pragma unroll
    for (int w = 0; w < kMaxTreeBitsNodes / 32; ++w) anc[w] = 0u;
    for (int n = i;;) {
        anc[n >> 5] |= 1u << (n & 31);
        const int p = parents[n];
        if (p < 0 || p >= n) break;
        n = p;
    }
}

// Workspace of the scheduled kernels: [status word, 256 B][records][(m, l) of
// the partial slots][O of the partial slots].
struct SeqWs {
    SeqRec *rec;       // [G]
    float2 *ml;        // [2 G][rows]: running max in log2 units, sum
    float *o;          // [2 G][D / 4][rows][4]
};

}  // namespace ta
