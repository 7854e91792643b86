// Attention of ragged rows on the 5th-generation tensor core (tcgen05): paged
// K/V (PAGED) or packed prompts, f16 / bf16, head dimension 64, 128 or 256.
//
// Rows of a unit are (token, query head) pairs of one KV head, so grouped heads
// share every K/V tile.  For D <= 128 a unit has 256 rows in two streams of 128, for
// D = 256 it has 128 rows in one.  S = Q K^T of a 64-key tile is taken from TMEM into
// registers by one thread a row, which frees it at once: Q K^T of the next tile runs
// while the softmax warps work on this one.  P goes to TMEM columns of its own, as one
// 16-bit term (off by half a step of a weight, as the 16-bit output is of its value: the error
// against 64 bits is 1.1 to 1.4 times that of an f32 form rounded once; a second term would
// double the P V products), and P V accumulates in f32.  (With P over S in two buffers of S, Q K^T waited for the P V two tiles back:
// 1820 cycles a tile against 1280 of products; with 128-key tiles and one buffer, 4200
// against 2048.)
//
//   warp 0      schedule and TMA producer: Q of a unit, K tiles through a ring
//   warp 6      TMA producer of V tiles (one producer for both held K back until V's
//               slot was free: Q K^T could not run ahead)
//   warps 1, 2  issue Q K^T and P V of stream 0; warps 4, 5 of stream 1.  Four issuing
//               threads: the tensor core's queue is short, so it idles while a thread
//               that has just issued its products waits on barriers and commits (two
//               threads for both streams: 2240 cycles a tile, of them 1280 of products)
//   warps 3, 7  V guard: before a V tile that not every row sees in full is used,
//               rows past the last key are zeroed and elements that are not finite
//               are taken out (0 x NaN would reach rows that do not see them); the
//               rows that do see such an element get NaN in its column at the end
//   4 warps per stream  softmax and epilogue, one row a thread
// The running max moves only when a row's max exceeds it by more than 2^8
// (P <= 2^15 fits f16, see kRaise; the sum stays in f32), so O in TMEM is rarely rescaled.
// Bound: one key tile of both streams is 1280 cycles of products at D = 128 (1024 at the
// rate of wider products) and about as many issue slots of softmax; a prompt of 8192 tokens with 32 / 8
// heads of 128 takes 431 us on inputs out of L2, 1276 TFLOP/s (68 % of the cuBLAS rate).
// Every wait is bounded; a wait that gives up sets the status word, and the CTA
// drains its copies and MMAs, frees TMEM and exits.
#pragma once

#include "seq_sched.cuh"
#include "sm100_ptx.cuh"

namespace ta {
namespace seqtc {

using namespace sm100;

template <int D>
struct Cfg {
    static constexpr int TKS = 6;
    static constexpr int TK = 1 << TKS;                 // keys per tile
    static constexpr int NSTR = D == 256 ? 1 : 2;       // row streams
    static constexpr int ROWS = 128 * NSTR;
    // TMEM, 512 columns: per stream NS buffers of S (64 columns), NP of P (32), and O
    static constexpr int NS = D == 128 ? 1 : 2, NP = 2;
    static constexpr int CS = 64 * NS + 32 * NP;        // S and P columns of a stream
    static constexpr int CO = NSTR * CS;                // first column of O
    static_assert(CO + NSTR * D <= 512, "TMEM");
    // Who waits for a P buffer to be read: the issuer of Q K^T (S then means the buffer is
    // free) or the softmax warps.  D = 64, whose softmax sets the pace: 189 against 206 us
    // for a prompt of 8192 tokens, 16 heads; D = 256, whose products do: 230 against 208 us
    // (4096 tokens, 24 / 4 heads); D = 128 the same.
    static constexpr bool kQkWaitsP = D == 64;
    static constexpr int SW = 8;                        // first softmax warp
    static constexpr int THREADS = 32 * SW + 128 * NSTR;
    static constexpr int SLABS = D / 64;                // 64-column slabs of a tile
    static constexpr int SLAB = TK * 128;               // bytes of a K / V slab
    static constexpr int QSLAB = ROWS * 128;            // bytes of a Q slab
    static constexpr int STAGE = SLABS * SLAB;
    static constexpr int NK = D == 256 ? 2 : 4, NV = D == 256 ? 2 : 4;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + SLABS * QSLAB;
    static constexpr int OFF_V = OFF_K + NK * STAGE;
    static constexpr int OFF_OUT = OFF_V + NV * STAGE;   // 2 KB a softmax warp: 32 rows x 32 columns of the output
    static constexpr int OFF_MISC = OFF_OUT + NSTR * 8192;
};

constexpr int kPieces = 4;
constexpr int kUnitCost = kSeqTcUnitCost;      // of the schedule: a unit's start and end take as long as 5 key tiles
// The guard is at most kPieces + 2 pieces ahead of an epilogue (a piece is published
// once every reader has fetched the one kPieces before it, and an epilogue runs
// right after the next fetch), so a ring of 8 marks is never overrun.
constexpr int kPoison = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;
// P and l of f16 rows are held 2^7 higher (P <= 2^15): a weight is subnormal only below 2^-21 of
// the running max's, and off by 2^-32 of it at most (at 2^0 weights up to 2^-25 were lost).
template <bool BF16>
constexpr float kRaise = BF16 ? 0.0f : 7.0f;

struct Misc {
    uint64_t k_full[4], k_empty[4], v_full[4], v_ready[4], v_empty[4];
    uint64_t q_full, q_empty, s_full[2][2], s_free[2][2], p_full[2][2], o_done[2][2], o_free[2];   // stream, S or P buffer
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    uint64_t drain[4], guard;         // guard: both guard warps have looked at a masked tile
    int found[2][2];                  // masked tile parity, guard warp
    SeqPiece piece[kPieces];
    SeqScratch sched;
    uint32_t tmem_base;
    int poisoned[kPoison];            // piece n % kPoison: some row has a poisoned column
};
constexpr int kMiscBytes = 3000;
static_assert(sizeof(Misc) <= kMiscBytes, "barrier area");
template <int D>
constexpr int kSmem = Cfg<D>::OFF_MISC + kMiscBytes;
static_assert(kSmem<64> <= 232448 && kSmem<128> <= 232448 && kSmem<256> <= 232448, "shared memory budget");

struct Args {
    SeqArgs a;
    SeqWs ws;
    uint32_t *poison;     // [G][kPoison][ROWS][D / 32]
    int tpt, G;
    uint32_t polls;       // of every wait, see wait_bar
    uint32_t g_inv;       // ceil(2^16 / g): row / g = row * g_inv >> 16, exact for rows < 256 and g <= 128
};
struct Maps {
    CUtensorMap q;        // {D, H, T}, box {64, g, tokens of a unit}: rows (token, head) as they stand in a unit
    // {64, tokens, D / 64, Hk, pages} (packed: no last axis), 128-byte swizzle.  A box is
    // a whole 64-key tile where a page holds one; of smaller pages V comes a page at a
    // time and K a page and 64 columns at a time.  (A box costs about 0.15 us of the copy
    // engine whatever its size: eight 8 KB boxes a tile held D = 256 at 3200 cycles a tile.)
    CUtensorMap k, v;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
// Two f32 at a time.
__device__ __forceinline__ uint64_t pack64(float x, float y) {
    return static_cast<uint64_t>(__float_as_uint(x)) | (static_cast<uint64_t>(__float_as_uint(y)) << 32);
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ float lo64(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float hi64(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }

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
// Bits 15 and 31: does the low / high 16-bit value hold an infinity or a NaN.  One
// added to an exponent field carries into the (cleared) sign place only from all ones.
template <bool BF16>
__device__ __forceinline__ uint32_t odd16(uint32_t w) {
    return BF16 ? (w & 0x7f807f80u) + 0x00800080u : (w & 0x7c007c00u) + 0x04000400u;
}

// Wait for a phase, `polls` polls of about 1 us at most; false: given up.  Six instructions and no call:
// the instruction cache holds the loops of all roles only while they are small (the
// same kernel with 100 bytes more a wait took 1.25 times as long), and a call would
// spill what the softmax warps hold.  The lanes of a warp may see a phase end at different
// polls, so the branches are not uniform.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, uint32_t polls) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, 0;\n\t"
        "L:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
        "@p bra D;\n\t"
        "add.u32 n, n, 1;\n\t"
        "setp.lt.u32 q, n, %3;\n\t"
        "@q bra L;\n\t"
        "D:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity & 1u), "r"(polls)
        : "memory");
    return ok != 0;
}
// Has the phase completed.
__device__ __forceinline__ bool poll_bar(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity & 1u) : "memory");
    return ok != 0;
}
// Registers of this warpgroup's threads from here on (the block's sum stays what
// it was launched with).
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// MMAs with descriptors as (low word with the address, constant high word).
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 a, {%1, %2};\n\t"
        "mov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, q;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, q;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z, int w, int v) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
        : "memory");
}

// Byte offset of (64-column slab, key row) of a V tile: `bk` rows a box, the slabs of a
// box one behind the other.
template <int D>
__device__ __forceinline__ int v_offset(int bk, int slab, int row) {
    return (row & ~(bk - 1)) * (Cfg<D>::SLABS * 128) + slab * bk * 128 + (row & (bk - 1)) * 128;
}

// One warp: mark the rows that see an element of this V tile that is not finite
// (bit d of a row's marks), and take the element out.
template <int D, bool BF16>
__device__ __noinline__ void mark_odd(const SeqArgs &a, const SeqPiece &p, int k0, int live, int bk, unsigned char *v,
                                      uint32_t *poison, bool clear) {
    using C = Cfg<D>;
    const int lane = threadIdx.x & 31;
    if (clear)
        for (int i = lane; i < C::ROWS * (D / 32); i += 32) poison[i] = 0u;
    __syncwarp();
#pragma unroll 1
    for (int r = 0; r < live; ++r)
#pragma unroll 1
        for (int c = lane; c < D / 2; c += 32) {
            // column pair c of key row r, at its swizzled place
            const int s = c >> 5, ch = (c & 31) >> 2;
            uint32_t *x = reinterpret_cast<uint32_t *>(v + v_offset<D>(bk, s, r) + ((ch ^ (r & 7)) << 4)) + (c & 3);
            const uint32_t odd = odd16<BF16>(*x) & 0x80008000u;
            if (odd == 0u) continue;
            const uint32_t bits = ((odd >> 15) & 1u) << ((2 * c) & 31) | (odd >> 31) << ((2 * c + 1) & 31);
#pragma unroll 1
            for (int row = 0; row < p.rows; ++row) {
                const int i = p.i0 + row / a.g;
                uint32_t anc[kMaxTreeBitsNodes / 32] = {}, m[1];
                if (a.parents) seq_ancestors(a.parents + p.q0, i, anc);
                seq_visible<1>(a, p.prefix, p.kv, i, anc, k0 + r, m);
                if (m[0] & 1u) atomicOr(poison + row * (D / 32) + (2 * c) / 32, bits);
            }
            if (odd & 0x8000u) *x &= 0xffff0000u;
            if (odd >> 31) *x &= 0x0000ffffu;
        }
    __threadfence();
    __syncwarp();
}

// The larger magnitudes, NaN if either is one: a running check for values that are
// not finite, one instruction a pair.
template <bool BF16>
__device__ __forceinline__ uint32_t max_abs(uint32_t acc, uint32_t w) {
    uint32_t r;
    if constexpr (BF16) asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %2;\n\tmax.NaN.bf16x2 %0, %1, a;\n\t}" : "=r"(r) : "r"(acc), "r"(w));
    else asm("{\n\t.reg .b32 a;\n\tabs.f16x2 a, %2;\n\tmax.NaN.f16x2 %0, %1, a;\n\t}" : "=r"(r) : "r"(acc), "r"(w));
    return r;
}

template <int D, bool PAGED, bool BF16>
__global__ void __launch_bounds__(Cfg<D>::THREADS, 1) seq_tc_kernel(const Args ar, const __grid_constant__ Maps maps) {
    using C = Cfg<D>;
    constexpr int TK = C::TK, TKS = C::TKS, NSTR = C::NSTR, NK = C::NK, NV = C::NV, NS = C::NS, NP = C::NP, ROWS = C::ROWS;
    extern __shared__ __align__(1024) unsigned char sm[];
    const SeqArgs &a = ar.a;
    if ((smem_u32(sm) & 1023u) != 0) {                  // swizzled tiles need it; the same in every CTA
        pdl_wait();
        if (threadIdx.x == 0) {
            atomicOr(a.status, kSeqTimeout);
            ar.ws.rec[blockIdx.x] = {0, 0, 0, 0};       // nothing for the merge to read
        }
        return;
    }
    Misc *mi = reinterpret_cast<Misc *>(sm + C::OFF_MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    // arrivals on a piece's empty slot: issuers, guards, V producer, softmax warps
    constexpr int kReaders = 2 * NSTR + 3 + 4 * NSTR;
    if (tid == 0) {
        for (int i = 0; i < NK; ++i) { mbar_init(&mi->k_full[i], 1); mbar_init(&mi->k_empty[i], NSTR); }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&mi->v_full[i], 1);
            mbar_init(&mi->v_ready[i], 2);
            mbar_init(&mi->v_empty[i], NSTR);
        }
        mbar_init(&mi->q_full, 1);
        mbar_init(&mi->guard, 2);
        mbar_init(&mi->q_empty, NSTR);
        for (int i = 0; i < 2; ++i) {
            for (int j = 0; j < 2; ++j) {
                mbar_init(&mi->s_full[i][j], 1);
                mbar_init(&mi->s_free[i][j], 4);
                mbar_init(&mi->p_full[i][j], 4);
                mbar_init(&mi->o_done[i][j], 1);
            }
            mbar_init(&mi->o_free[i], 4);
            mbar_init(&mi->drain[2 * i], 1);
            mbar_init(&mi->drain[2 * i + 1], 1);
        }
        for (int i = 0; i < kPieces; ++i) { mbar_init(&mi->piece_full[i], 1); mbar_init(&mi->piece_empty[i], kReaders); }
        for (int i = 0; i < kPoison; ++i) mi->poisoned[i] = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&mi->tmem_base, 512);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
    }
    pdl_wait();
    const SeqRun run = seq_schedule<C::THREADS, TKS, kUnitCost, 1>(a, ar.tpt, cta, ar.G, &mi->sched);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = mi->tmem_base;
    const uint32_t tm_o0 = tmem + C::CO;

    // Boxes of bk keys; of a part tile K's are 64 columns wide: lanes 0 .. k_boxes - 1 issue
    // one each (V: lanes 0 .. per_slab - 1).
    const int bk = PAGED ? min(TK, 1 << a.page_shift) : TK, per_slab = TK / bk;          // 1, 2 or 4 boxes
    const int box = lane & (per_slab - 1), slab = bk == TK ? 0 : lane / per_slab, k_boxes = bk == TK ? 1 : per_slab * C::SLABS;
    // page of this lane's box of key tile t (n_pages: out of range, read as zeros)
    auto page_of = [&](const SeqPiece &p, int t) -> int {
        if constexpr (!PAGED) return 0;
        const int key = (t << TKS) + box * bk;
        if (key >= p.kv) return a.n_pages;
        const int g = __ldg(a.table + static_cast<long long>(p.b) * a.max_pages + (key >> a.page_shift));
        if (g >= 0 && g < a.n_pages) return g;
        // a page before every row's window may be gone
        if (lane < per_slab && !(a.window && key + bk <= p.prefix + p.i0 - a.window + 1)) atomicOr(a.status, kSeqBadPage);
        return a.n_pages;
    };

    // A whole warp's wait, one outcome.
    auto warp_wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_bar(bar, parity, ar.polls)) != 0; };
    // The next piece, in order; a reader's warp-wide copy.
    int piece_n = 0;
    bool failed = false;                                // a wait of this warp gave up
    auto fetch = [&](SeqPiece *p) -> bool {
        const int i = piece_n % kPieces;
        const bool ok = warp_wait(&mi->piece_full[i], piece_n / kPieces);
        ++piece_n;
        if (!ok) {                                      // gave up
            p->valid = 0;
            failed = true;
            return false;
        }
        *p = mi->piece[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(&mi->piece_empty[i]);
        return p->valid != 0;
    };
    // Does some row of the piece not see all of key tile t.
    auto is_masked = [&](const SeqPiece &p, int t) { return (t << TKS) < p.full_lo || ((t + 1) << TKS) > p.full_hi; };

    // D <= 128: 4 x 128 registers a thread at launch = 2 x 88 + 2 x 168.
    if (warp < C::SW) {
    if constexpr (NSTR == 2) regs_down<88>();
    if (warp == 0) {
        // ------------------------------------------------- schedule, TMA producer
        SeqWalk<TKS, kUnitCost> walk;
        walk.init(a, ar.tpt, run, &mi->sched, cta);
        int n = 0, kn = 0, qn = 0;                      // pieces, K tiles, Q tiles so far
        bool ok = true;
        if (lane == 0) ar.ws.rec[cta] = {0, 0, 0, 0};
#pragma unroll 1
        for (;; ++n) {
            SeqPiece p;
            p.valid = 0;
            const bool more = walk.next(a, ar.tpt, run, &p);
            const int i = n % kPieces;
            if (n >= kPieces)
                ok = warp_wait(&mi->piece_empty[i], n / kPieces - 1);
            if (!ok) break;
            if (lane == 0) {
                mi->piece[i] = p;
                mbar_arrive(&mi->piece_full[i]);
                // the unit's first piece leaves the record of how many there are
                if (more && p.rest > 0) ar.ws.rec[cta] = seq_record(run, cta, p);
            }
            __syncwarp();
            if (!more) break;
            int page = page_of(p, p.t0);
#pragma unroll 1
            for (int t = 0; t < p.nt; ++t) {
                const int next = t + 1 < p.nt ? page_of(p, p.t0 + t + 1) : 0;
                const int key = ((p.t0 + t) << TKS) + box * bk;
                const int st = kn % NK;
                ok = warp_wait(&mi->k_empty[st], (static_cast<uint32_t>(kn / NK) & 1u) ^ 1u);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&mi->k_full[st], C::STAGE);
                __syncwarp();
                if (lane < k_boxes) {
                    unsigned char *d = sm + C::OFF_K + st * C::STAGE + slab * C::SLAB + box * bk * 128;
                    if constexpr (PAGED) tma_load_5d(d, &maps.k, &mi->k_full[st], 0, key & ((1 << a.page_shift) - 1), slab, p.kh, page);
                    else tma_load_4d(d, &maps.k, &mi->k_full[st], 0, p.q0 + key, 0, p.kh);
                }
                ++kn;
                if (t == 0) {
                    // the unit's rows of Q, once the products of the piece before have read theirs
                    if (n > 0) ok = warp_wait(&mi->q_empty, n - 1);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&mi->q_full, C::SLABS * ar.tpt * a.g * 128);
                        for (int x = 0; x < C::SLABS; ++x)
                            tma_load_3d(sm + C::OFF_Q + x * C::QSLAB, &maps.q, &mi->q_full, x * 64, p.kh * a.g, p.q0 + p.i0);
                        ++qn;
                    }
                    __syncwarp();
                }
                page = next;
            }
            if (!ok) break;
        }
        failed = !ok;
        // every copy issued has landed before the CTA's memory goes
        if (lane == 0) {
            if (qn > 0 && !mbar_wait_sleep(&mi->q_full, static_cast<uint32_t>(qn - 1) & 1u, 1u << 21, 1000))
                atomicOr(a.status, kSeqTimeout);
            for (int i = max(0, kn - NK); i < kn; ++i)
                if (!mbar_wait_sleep(&mi->k_full[i % NK], static_cast<uint32_t>(i / NK) & 1u, 1u << 21, 1000))
                    atomicOr(a.status, kSeqTimeout);
        }
    } else if (warp == 6) {
        // ------------------------------------------------------------- V producer
        int vn = 0;
        bool ok = true;
        SeqPiece p;
#pragma unroll 1
        while (ok && fetch(&p)) {
            int page = page_of(p, p.t0);
#pragma unroll 1
            for (int t = 0; t < p.nt; ++t) {
                const int next = t + 1 < p.nt ? page_of(p, p.t0 + t + 1) : 0;
                const int key = ((p.t0 + t) << TKS) + box * bk;
                const int st = vn % NV;
                ok = warp_wait(&mi->v_empty[st], (static_cast<uint32_t>(vn / NV) & 1u) ^ 1u);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&mi->v_full[st], C::STAGE);
                __syncwarp();
                if (lane < per_slab) {
                    unsigned char *d = sm + C::OFF_V + st * C::STAGE + box * bk * (C::SLABS * 128);
                    if constexpr (PAGED) tma_load_5d(d, &maps.v, &mi->v_full[st], 0, key & ((1 << a.page_shift) - 1), 0, p.kh, page);
                    else tma_load_4d(d, &maps.v, &mi->v_full[st], 0, p.q0 + key, 0, p.kh);
                }
                ++vn;
                page = next;
            }
        }
        failed |= !ok;
        if (lane == 0)
            for (int i = max(0, vn - NV); i < vn; ++i)
                if (!mbar_wait_sleep(&mi->v_full[i % NV], static_cast<uint32_t>(i / NV) & 1u, 1u << 21, 1000))
                    atomicOr(a.status, kSeqTimeout);
    } else if (warp == 1 || warp == 2 || (NSTR == 2 && (warp == 4 || warp == 5))) {
        // ------------------------------------------------------------ MMA issuers
        const int x = warp >> 2, w = warp - (x ? 4 : 1);   // stream; 0: Q K^T, 1: P V
        const uint32_t q_addr = smem_u32(sm + C::OFF_Q), k_addr = smem_u32(sm + C::OFF_K), v_addr = smem_u32(sm + C::OFF_V);
        constexpr uint32_t id_qk = idesc_f16(128, TK, BF16 ? 1 : 0, 0, 0);
        constexpr uint32_t id_pv = idesc_f16(128, D, BF16 ? 1 : 0, 0, 1);
        constexpr uint64_t kHiQK = (uint64_t(16 >> 4) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
        constexpr uint64_t kHiV = (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
        constexpr uint32_t qk_lo = static_cast<uint32_t>(kHiQK), qk_hi = static_cast<uint32_t>(kHiQK >> 32);
        constexpr uint32_t v_hi = static_cast<uint32_t>(kHiV >> 32);
        const uint32_t v_lo = static_cast<uint32_t>(bk * 128 >> 4) << 16;    // slabs bk rows apart
        // shared addresses in a descriptor's 16-byte units
        const uint32_t q16 = (q_addr >> 4) | qk_lo, k16 = (k_addr >> 4) | qk_lo, v16 = (v_addr >> 4) | v_lo;
        auto qk = [&](uint32_t q, uint32_t k, uint32_t s) {
#pragma unroll
            for (int sl = 0; sl < C::SLABS; ++sl)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ss(s, q + sl * (C::QSLAB >> 4) + kk * 2, qk_hi, k + sl * (C::SLAB >> 4) + kk * 2, qk_hi, id_qk,
                           (sl | kk) != 0);
        };
        auto pv = [&](uint32_t p, uint32_t v, uint32_t o, uint32_t acc) {
#pragma unroll
            for (int kk = 0; kk < TK / 16; ++kk)
                mma_ts(o, p + 8 * kk, v + (v_offset<D>(bk, 0, 16 * kk) >> 4), v_hi, id_pv, kk != 0 ? 1u : acc);
        };
        bool ok = true;
        SeqPiece p;
        auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_bar(bar, parity, ar.polls); };
        // bn: tiles of the stream, in its S or P buffers in turn; pn: its pieces; cn: tiles of
        // the CTA; n: its pieces
        int bn = 0, pn = 0, cn = 0, n = 0;
        const uint32_t s0 = tmem + C::CS * x, o = tm_o0 + D * x, q = q16 + x * (16384 >> 4);
#pragma unroll 1
        while (ok && fetch(&p)) {
            if (lane == 0) {
                const bool act = NSTR == 1 || p.rows > 128 * x;
                if (w == 0) {
                    ok = wait(&mi->q_full, n);
#pragma unroll 1
                    for (int t = 0; t < p.nt && ok; ++t, ++cn) {
                        const int st = cn % NK, sb = bn % NS;
                        ok = wait(&mi->k_full[st], cn / NK);
                        if (!act) {                     // the other stream's alone: release it with that one
                            mbar_arrive(&mi->k_empty[st]);
                            continue;
                        }
                        // the softmax warps have taken the S that was here
                        if (ok && bn >= NS) ok = wait(&mi->s_free[x][sb], bn / NS - 1);
                        if (C::kQkWaitsP && ok && bn >= NP) ok = wait(&mi->o_done[x][bn % NP], bn / NP - 1);
                        if (!ok) break;
                        tc_fence_after();
                        qk(q, k16 + st * (C::STAGE >> 4), s0 + 64 * sb);
                        mma_commit(&mi->s_full[x][sb]);
                        mma_commit(&mi->k_empty[st]);
                        ++bn;
                    }
                    if (act) mma_commit(&mi->q_empty);
                    else mbar_arrive(&mi->q_empty);
                } else {
#pragma unroll 1
                    for (int t = 0; t < p.nt && ok; ++t, ++cn) {
                        const int st = cn % NV, sb = bn % NP;
                        ok = wait(&mi->v_ready[st], cn / NV);
                        if (!act) {
                            mbar_arrive(&mi->v_empty[st]);
                            continue;
                        }
                        if (ok) ok = wait(&mi->p_full[x][sb], bn / NP);
                        // O is rewritten: the piece before has been read out
                        if (ok && t == 0 && pn > 0) ok = wait(&mi->o_free[x], pn - 1);
                        if (!ok) break;
                        tc_fence_after();
                        pv(s0 + 64 * NS + 32 * sb, v16 + st * (C::STAGE >> 4), o, t != 0);
                        mma_commit(&mi->o_done[x][sb]);
                        mma_commit(&mi->v_empty[st]);
                        ++bn;
                    }
                    if (act) ++pn;
                }
                ++n;
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        failed |= !ok;
        if (lane == 0) {                                // every MMA issued has completed
            mma_commit(&mi->drain[2 * x + w]);
            if (!mbar_wait_sleep(&mi->drain[2 * x + w], 0, 1u << 21, 1000)) atomicOr(a.status, kSeqTimeout);
        }
        __syncwarp();
    } else if (warp == 3 || warp == 7) {
        // --------------------------------------------------------------- V guards
        // Two warps, every other 4 rows each; warp 3 does the marking.
        const int part = warp >> 2;
        int vn = 0, n = 0, gn = 0;                      // V tiles, pieces, masked tiles so far
        bool ok = true;
        SeqPiece p;
#pragma unroll 1
        for (; ok && fetch(&p); ++n) {
            bool marked = false;
            uint32_t *poison = ar.poison + (static_cast<size_t>(cta) * kPoison + n % kPoison) * ROWS * (D / 32);
            if (part == 0 && lane == 0) mi->poisoned[n % kPoison] = 0;
#pragma unroll 1
            for (int t = 0; t < p.nt && ok; ++t, ++vn) {
                const int st = vn % NV, k0 = (p.t0 + t) << TKS;
                ok = warp_wait(&mi->v_full[st], vn / NV);
                if (!ok) break;
                if (is_masked(p, p.t0 + t)) {
                    unsigned char *v = sm + C::OFF_V + st * C::STAGE;
                    const int live = min(max(p.kv - k0, 0), TK);
                    // slab rows are 128 bytes; lane l of guard `part` takes chunk l % 8 of rows
                    // l / 8 + 4 part, + 8, ...  Keys that every row of the unit sees need no look:
                    // left of full_lo and right of full_hi they are scanned, past the last key zeroed.
                    uint32_t acc[4] = {};
                    auto scan = [&](int r0, int r1) {              // r0 a multiple of 8
#pragma unroll 1
                        for (int s = 0; s < C::SLABS; ++s) {
                            uint4 y[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u) {
                                const int r = r0 + (lane >> 3) + 8 * u + 4 * part;
                                y[u] = r < r1 ? *reinterpret_cast<const uint4 *>(v + v_offset<D>(bk, s, r) + (lane & 7) * 16)
                                              : make_uint4(0, 0, 0, 0);
                            }
#pragma unroll
                            for (int u = 0; u < 8; ++u) {
                                acc[0] = max_abs<BF16>(acc[0], y[u].x);
                                acc[1] = max_abs<BF16>(acc[1], y[u].y);
                                acc[2] = max_abs<BF16>(acc[2], y[u].z);
                                acc[3] = max_abs<BF16>(acc[3], y[u].w);
                            }
                        }
                    };
                    const int right = min(max(p.full_hi - k0, 0), live) & ~7, left = min(p.full_lo - k0, right);
                    if (left > 0) scan(0, left);
                    if (right < live) scan(right, live);
#pragma unroll 1
                    for (int s = 0; s < C::SLABS; ++s)
#pragma unroll 1
                        for (int r = live + (lane >> 3) + 4 * part; r < TK; r += 8)
                            *reinterpret_cast<uint4 *>(v + v_offset<D>(bk, s, r) + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                    const bool found = ((odd16<BF16>(acc[0]) | odd16<BF16>(acc[1]) | odd16<BF16>(acc[2]) | odd16<BF16>(acc[3])) & 0x80008000u) != 0;
                    fence_proxy_async_smem();
                    const bool any = __any_sync(0xffffffffu, found);
                    if (lane == 0) {
                        mi->found[gn & 1][part] = any;
                        mbar_arrive(&mi->guard);
                    }
                    ok = warp_wait(&mi->guard, gn);
                    if (!ok) break;
                    const volatile int *f = mi->found[gn & 1];
                    ++gn;
                    if (f[0] | f[1]) {
                        if (part == 0) {
                            mark_odd<D, BF16>(a, p, k0, live, bk, v, poison, !marked);
                            if (lane == 0) mi->poisoned[n % kPoison] = 1;
                            fence_proxy_async_smem();
                        }
                        marked = true;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&mi->v_ready[st]);
            }
        }
        failed |= !ok;
    }
    } else {
        // ---------------------------------------------------- softmax and epilogue
        if constexpr (NSTR == 2) regs_up<168>();
        const int s = (warp - C::SW) >> 2;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;              // row within the stream
        const int urow = 128 * s + r;                   // row within the unit
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tm_s = tmem + lane_off + C::CS * s, tm_o = tm_o0 + lane_off + D * s;
        const float scale2 = fmaxf(a.scale * kLog2e, FLT_MIN);   // above 0: a masked -inf stays -inf
        const int tok_row = static_cast<int>((static_cast<uint32_t>(urow) * ar.g_inv) >> 16);
        int tn = 0, vn = 0;                             // tiles of this stream, tiles of the CTA
        bool ok = true;
        // (the lanes' outcomes are joined once a tile: a vote at every wait took 443 us for a
        // prompt of 8192 tokens against 423, on one set of inputs; the warp itself is joined here,
        // since the TMEM loads and stores behind a wait need all of it: 432 us against 427.  Polled
        // by one lane: 480)
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = wait_bar(bar, parity, ar.polls) && ok;
            __syncwarp();
        };
        SeqPiece p;
#pragma unroll 1
        for (int n = 0; ok && fetch(&p); ++n) {         // pieces of the CTA
            const bool act = NSTR == 1 || p.rows > 128 * s, live = urow < p.rows;
            float m_run = -INFINITY, l_run = 0.0f;
            if (act) {
                const int i = p.i0 + tok_row;
                uint32_t anc[kMaxTreeBitsNodes / 32];
                if (a.parents && live) seq_ancestors(a.parents + p.q0, i, anc);
                uint32_t v[TK];
                // S of tile tn of the stream, on its way into v
                auto take = [&](int n) {
                    wait(&mi->s_full[s][n % NS], n / NS);
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < TK / 32; ++c)
                        tmem_ld32(tm_s + 64 * (n % NS) + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&v[32 * c]));
                };
                // tiles [plain0, plain0 + plains) are seen by every row and are not the first: one
                // compare and branch a tile
                const int plain0 = max(1, ((p.full_lo + TK - 1) >> TKS) - p.t0), plains = max(0, (p.full_hi >> TKS) - p.t0 - plain0);
                take(tn);
#pragma unroll 1
                for (int t = 0; t < p.nt; ++t, ++tn) {
                    const int pb = tn % NP;
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&mi->s_free[s][tn % NS]);
                    ok = __all_sync(0xffffffffu, ok) != 0;
                    if (!ok) break;
                    bool masked = false;
                    if (__builtin_expect(static_cast<unsigned>(t - plain0) >= static_cast<unsigned>(plains), 0)) {
                        masked = is_masked(p, p.t0 + t);
                        if (masked) {
                            uint32_t m[TK / 32];
                            seq_visible<TK / 32>(a, p.prefix, live ? p.kv : 0, i, anc, (p.t0 + t) << TKS, m);
#pragma unroll
                            for (int e = 0; e < TK; ++e)
                                if (!((m[e >> 5] >> (e & 31)) & 1u)) v[e] = 0xff800000u;
                        }
                        if (t == 0) {
                            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                            for (int e = 0; e < TK / 2; ++e)
                                mx[e & 1] = max3(mx[e & 1], __uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                            m_run = fmaxf(mx[0], mx[1]) * scale2;
                        }
                    }
                    // P with the running max as it is, the tile's own max taken beside the
                    // exponentials (other pipes); only where some row's max rose by more than 2^8
                    // do O and l follow, and P is taken again
                    // has the P V that read this P buffer NP tiles ago finished (kQkWaitsP: S says so):
                    // asked here, where the answer arrives beside the exponentials (a wait in front of
                    // P's store: 420 us for a prompt of 8192 tokens against 402, on one set of inputs)
                    const bool o_done = C::kQkWaitsP || tn < NP || __all_sync(0xffffffffu, poll_bar(&mi->o_done[s][pb], tn / NP - 1));
                    uint32_t pk[TK / 2];
                    float l_tile;
#pragma unroll 1
                    for (;;) {
                        const float m_use = m_run == -INFINITY ? 0.0f : m_run - kRaise<BF16>;
                        const uint64_t sc = pack64(scale2, scale2), mm = pack64(-m_use, -m_use);
                        uint64_t sum[2] = {0, 0};
                        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < TK / 2; ++e) {
                            const float s0 = __uint_as_float(v[2 * e]), s1 = __uint_as_float(v[2 * e + 1]);
                            const uint64_t x = fma2(pack64(s0, s1), sc, mm);
                            const float p0 = ex2(lo64(x)), p1 = ex2(hi64(x));
                            sum[e & 1] = add2(sum[e & 1], pack64(p0, p1));
                            pk[e] = pack16<BF16>(p0, p1);
                            mx[e & 1] = max3(mx[e & 1], s0, s1);
                        }
                        const uint64_t all = add2(sum[0], sum[1]);
                        l_tile = lo64(all) + hi64(all);
                        const float top = fmaxf(mx[0], mx[1]) * scale2;
                        if (__builtin_expect(!__any_sync(0xffffffffu, top > m_run + kSlack), 1)) break;
                        float alpha = 1.0f;
                        if (top > m_run + kSlack) {
                            alpha = ex2(m_run - top);   // 0 from -inf
                            l_run *= alpha;
                            m_run = top;
                        }
                        // O must be at rest: the P V of the tile before is done (t > 0 here: the
                        // first tile's max is the running max)
                        wait(&mi->o_done[s][(tn - 1) % NP], (tn - 1) / NP);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(tm_o + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st16(tm_o + c, o);
                        }
                    }
                    l_run += l_tile;
                    if (__builtin_expect(!o_done, 0)) wait(&mi->o_done[s][pb], tn / NP - 1);
                    // the guard's marks of this V tile are in before its P V can be issued
                    if (masked) wait(&mi->v_ready[(vn + t) % NV], (vn + t) / NV);
                    tmem_st32(tm_s + 64 * NS + 32 * pb, pk);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&mi->p_full[s][pb]);
                    if (t + 1 < p.nt) take(tn + 1);     // (before P's store it held P V back)
                }
            }
            vn += p.nt;
            ok = __all_sync(0xffffffffu, ok) != 0;
            if (act && ok) {
                wait(&mi->o_done[s][(tn - 1) % NP], (tn - 1) / NP);
                ok = __all_sync(0xffffffffu, ok) != 0;
                if (!ok) break;
                tc_fence_after();
                const bool odd = *static_cast<volatile int *>(&mi->poisoned[n % kPoison]) != 0;
                const uint32_t *poison = ar.poison + ((static_cast<size_t>(cta) * kPoison + n % kPoison) * ROWS + urow) * (D / 32);
                const float inv = l_run > 0.0f ? 1.0f / l_run : (l_run == 0.0f ? 0.0f : l_run);
                const size_t slot = static_cast<size_t>(p.slot < 0 ? 0 : p.slot);
                float4 *part = reinterpret_cast<float4 *>(ar.ws.o) + slot * (D / 4) * ROWS + urow;
                unsigned char *stage = sm + C::OFF_OUT + (warp - C::SW) * 2048;
                // rows 8 u + lane / 4 of the warp, 16 bytes at 8 (lane % 4) columns
                uint16_t *dst[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int ur = 128 * s + 32 * quarter + 8 * u + (lane >> 2);
                    const int tok = static_cast<int>((static_cast<uint32_t>(ur) * ar.g_inv) >> 16), h = p.kh * a.g + ur - tok * a.g;
                    dst[u] = ur < p.rows ? static_cast<uint16_t *>(a.out) + static_cast<long long>(p.q0 + p.i0 + tok) * a.o_st +
                                               h * a.o_sh + (lane & 3) * 8
                                         : nullptr;
                }
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(tm_o + c, o);
                    tmem_wait_ld();
                    if (odd && live) {                  // poisoned columns of this row
                        const uint32_t bits = __ldcg(poison + c / 32);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if ((bits >> e) & 1u) o[e] = 0x7fffffffu;
                    }
                    if (p.slot < 0) {
                        // 32 columns of the warp's 32 rows through shared memory, so that a store
                        // covers 8 rows' 64 bytes (a row a lane took 32 cycles a store)
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint4 x;
                            x.x = pack16<BF16>(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                            x.y = pack16<BF16>(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                            x.z = pack16<BF16>(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                            x.w = pack16<BF16>(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
                            *reinterpret_cast<uint4 *>(stage + lane * 64 + (((e / 8) ^ ((lane >> 1) & 3)) << 4)) = x;
                        }
                        __syncwarp();
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int row = 8 * u + (lane >> 2);
                            const uint4 x = *reinterpret_cast<const uint4 *>(stage + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
                            if (dst[u]) *reinterpret_cast<uint4 *>(dst[u] + c) = x;
                        }
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            part[static_cast<size_t>((c + e) / 4) * ROWS] =
                                make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                            __uint_as_float(o[e + 3]));
                    }
                    __syncwarp();
                }
                if (live && p.slot >= 0) ar.ws.ml[slot * ROWS + urow] = make_float2(m_run, l_run);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&mi->o_free[s]);
            }
        }
        failed |= !ok;
    }
    if (failed && lane == 0) atomicOr(a.status, kSeqTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Merge of the pieces of the units that start in CTA blockIdx.x and are cut:
// out = sum_p O_p 2^(m_p - m*) / sum_p l_p 2^(m_p - m*).  16 columns a block, one
// row a thread; partials are laid out so that a warp reads whole lines.
template <int D, bool BF16>
__global__ void __launch_bounds__(Cfg<D>::ROWS) seq_merge_kernel(const SeqArgs a, const SeqWs ws) {
    constexpr int ROWS = Cfg<D>::ROWS;
    pdl_wait();
    const int c = blockIdx.x, r = threadIdx.x, d0 = blockIdx.y * 16;
    const SeqRec rec = ws.rec[c];
    if (r >= rec.rows || rec.parts == 0) return;
    // pieces: slot 2 c + 1, then the first slots of the CTAs after it
    auto slot = [&](int p) { return static_cast<size_t>(p == 0 ? 2 * c + 1 : 2 * (c + p)); };
    // the max first, then sums whose loads do not wait for one another
    float m = -INFINITY, l = 0.0f, o[16] = {};
#pragma unroll 4
    for (int p = 0; p < rec.parts; ++p) m = fmaxf(m, ws.ml[slot(p) * ROWS + r].x);
    const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll 4
    for (int p = 0; p < rec.parts; ++p) {
        const float2 x = ws.ml[slot(p) * ROWS + r];
        const float g = ex2(x.x - mu);
        l += x.y * g;
        const float4 *src = reinterpret_cast<const float4 *>(ws.o) + (slot(p) * (D / 4) + d0 / 4) * ROWS + r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 y = src[e * ROWS];
            o[4 * e] += y.x * g;
            o[4 * e + 1] += y.y * g;
            o[4 * e + 2] += y.z * g;
            o[4 * e + 3] += y.w * g;
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    const int tok = r / a.g, h = rec.kh * a.g + r - tok * a.g;
    uint16_t *out = static_cast<uint16_t *>(a.out) + static_cast<long long>(rec.token + tok) * a.o_st + h * a.o_sh + d0;
#pragma unroll
    for (int e = 0; e < 16; e += 8) {
        uint4 x;
        x.x = pack16<BF16>(o[e] * inv, o[e + 1] * inv);
        x.y = pack16<BF16>(o[e + 2] * inv, o[e + 3] * inv);
        x.z = pack16<BF16>(o[e + 4] * inv, o[e + 5] * inv);
        x.w = pack16<BF16>(o[e + 6] * inv, o[e + 7] * inv);
        *reinterpret_cast<uint4 *>(out + e) = x;
    }
}

template <int D, bool PAGED, bool BF16>
cudaError_t launch(const Args &ar, const Maps &maps, cudaStream_t s) {
    auto kern = seq_tc_kernel<D, PAGED, BF16>;
    static unsigned long long done = 0;
    cudaError_t e = set_smem_limit_once(kern, kSmem<D>, &done);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(ar.G), dim3(Cfg<D>::THREADS), kSmem<D>, s, ar, maps);
    count_launch();
    if (e != cudaSuccess) return e;
    e = launch_pdl(seq_merge_kernel<D, BF16>, dim3(ar.G, D / 16), dim3(Cfg<D>::ROWS), 0, s, ar.a, ar.ws);
    count_launch();
    return e;
}

template <int D>
cudaError_t launch_dim(const SeqArgs &a, const SeqTcPlan &pl, cudaStream_t s) {
    Args ar;
    ar.a = a;
    ar.G = pl.G;
    ar.polls = pl.polls;
    ar.tpt = Cfg<D>::ROWS / a.g;
    ar.g_inv = (65536u + a.g - 1) / a.g;
    char *ws = static_cast<char *>(pl.ws);
    ar.ws.rec = reinterpret_cast<SeqRec *>(ws + 256);
    const size_t slots = 2 * static_cast<size_t>(pl.G), rows = Cfg<D>::ROWS;
    size_t off = 256 + (pl.G * sizeof(SeqRec) + 255) / 256 * 256;
    ar.ws.ml = reinterpret_cast<float2 *>(ws + off);
    off += slots * rows * sizeof(float2);
    ar.ws.o = reinterpret_cast<float *>(ws + off);
    off += slots * rows * D * sizeof(float);
    ar.poison = reinterpret_cast<uint32_t *>(ws + off);
    Maps maps;
    maps.q = pl.q;
    maps.k = pl.k;
    maps.v = pl.v;
    if (a.kv_lens)
        return a.bf16 ? launch<D, true, true>(ar, maps, s) : launch<D, true, false>(ar, maps, s);
    return a.bf16 ? launch<D, false, true>(ar, maps, s) : launch<D, false, false>(ar, maps, s);
}

}  // namespace seqtc
}  // namespace ta
