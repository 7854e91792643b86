// Attention of few query rows per KV head over 4-bit pages with warp-level MMAs: single tokens
// and small drafts, max_q_len * (heads per KV head) <= 16 rows.
//
// The work is reading codes, scales and biases once, D + 8 D / G bytes a key and KV head; HBM
// bounds it, and next to it the instructions that widen the codes.  So codes are not
// turned into values: a nibble masked out of its word is the f16 subnormal c 2^-24 (or 16 c 2^-24,
// without a shift), which a matrix instruction takes as it is, and scales and biases are applied to
// sums.  With q' a row's group of G elements of Q times a power of two 2^e in f16
//   q . k = sum_g s_g 2^24 / 2^e_g (q'_g . c_g 2^-24) + sum_g b_g (sum of q in g)
//   sum_key P v = sum_key (P s_g) c + sum_key P b_g     (the second one number a row and group)
// The products are keys (16) x rows (8) x elements, and elements (16) x rows (8) x keys: keys and
// elements, not the few rows, fill the long side.  P s_g goes from the first product's layout to the
// second's by an 8 x 8 transpose (movmatrix), in f16, held within its range by a power of two per
// row and group that, like the running max, moves only when a block needs it (kQmTop).
// A lane's words: for K the quads 2 t and 2 t + 1 of every 32-element block of keys g and
// g + 8, for V quad g of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9 - one vector a key and
// product.  A warp takes every fourth block of 16 keys of its CTA's run, one or two blocks at a time, copied to
// shared memory two such sets ahead (cp.async; no barrier inside the key loop); the batch is cut evenly over the
// CTAs by the schedule of seq_sched.cuh.
// Measured: one token of 64 requests of 900 to 16384 keys, 32 / 8 heads of 128, groups of 64 (668 MB): 155 us, 4.3
// TB/s.  Batches of 16 to 128 requests of 8192 keys (45 to 270 us) lie on a line of 4.7 TB/s and 14 us of start, first
// copies, join and merge.  131001 keys of 4 heads of 256, groups of 32 (168 MB): 52 us; 96 requests with a window of
// 2000 keys, 16 / 16 heads of 64, groups of 32 (216 MB): 89 us, 2.4 TB/s, half of the products' rows empty.
// The same 64 requests took 253 us with codes straight from global memory into registers and a row an instruction, 198 with two
// rows an instruction, 179 through shared memory, 167 with 32-bit strides, 160 with copies without branches, 156 with two blocks
// at a time, 152 with the unit cost below, 155 since scales and queries of all sizes keep their weights (kQmTop, the careful
// loop).  Of a like batch that takes 162 us: 167 in the careful loop for the queries alone, 188 with 1 % of V's scales 0 (each
// asks for a second look), 700 where every block holds scales 2^10 and more apart.
#pragma once

#include <type_traits>

#include "quant_page.cuh"
#include "seq_merge.cuh"

namespace ta {
namespace {

constexpr int kQmWarps = 4, kQmThreads = kQmWarps * 32;
constexpr int kQmTks = 6;                           // schedule granularity: 64 keys, 16 a warp
constexpr int kQmLeast = 3;                         // tiles of a CTA's run at least
// A unit's start and end (Q, the first copies, the join) in tiles' worth of time.  0, 4, 6, 8 and 12: 160, 155, 155, 155 and
// 157 us for 64 requests of 900 to 16384 keys, 103, 89, 89, 89 and 89 us for 96 of up to 2000 keys with 16 KV heads.
constexpr int kQmUnitCost = 6;
constexpr float kQmLog2e = 1.4426950408889634f;
// The running max moves when a row's max exceeds it by more than 2^8; P and l are held 2^7 higher
// (P <= 2^15).
constexpr float kQmSlack = 8.0f, kQmRaise = 7.0f;
// P s as f16.  The power of two of a row and group, 2^110 at most, starts as that; a block whose largest P s leaves f16's
// range sets it so that this one becomes a quarter of the row's largest weight P, for which 2^7 is taken where it is less here
// (a weight may grow to 2^15 before the running max moves); where the running max moves it rises by what
// the older products lose.  So the largest of all products so far is 2^5 at least, as it counts now, and what f16 loses of
// another one is 2^-30 of that.  Elements whose code is 0 in that key would see the loss: blocks with a scale below 2^-12
// under the power of two (2^-10 or less of the one that counts) at a weight that is not far below all others (P > 2^-20) are
// taken in f32, a key at a time.
constexpr int kQmTop = 110;
constexpr float kQmFloor = 0x1p-12f, kQmFaint = 0x1p-20f, kQmPeak = 0x1p7f;

struct QmArgs {
    SeqQuantArgs q;
    SeqRec *rec;      // [G]
    float2 *ml;       // [2 G][8 NR]
    float *o;         // [2 G][8 NR][D]
    int G;
};

__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Two f32 at a time: the two query rows that a lane holds of a key.
__device__ __forceinline__ uint64_t two(float x, float y) {
    return static_cast<uint64_t>(__float_as_uint(x)) | (static_cast<uint64_t>(__float_as_uint(y)) << 32);
}
__device__ __forceinline__ float first(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float second(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ uint64_t fma_two(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t mul_two(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
// The larger of three, of the magnitudes where a NaN does not count.
__device__ __forceinline__ float max_abs3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(fabsf(y)), "f"(fabsf(z)));
    return r;
}
__device__ __forceinline__ float part(uint64_t x, int e) { return e ? second(x) : first(x); }
__device__ __forceinline__ float min_abs3(float x, float y, float z) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(fabsf(y)), "f"(fabsf(z)));
    return r;
}
// N words (1, 2, 4 or 8) of shared memory.
template <int N>
__device__ __forceinline__ void load_words(const unsigned char *p, uint32_t *w) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x; w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(p + 4 * i);
            w[i] = x.x; w[i + 1] = x.y; w[i + 2] = x.z; w[i + 3] = x.w;
        }
    }
}
// 16 bytes to shared memory, past L1; N words, or as many zeros, past L1 where the instruction takes 16 bytes.
__device__ __forceinline__ void copy_vector(uint32_t dst, const uint32_t *src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_words(uint32_t dst, const uint32_t *src, bool live) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst + 4 * i), "l"(src + i), "r"(live ? 16 : 0) : "memory");
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(4 * N), "r"(live ? 4 * N : 0) : "memory");
    }
}
// Scale and bias of a pair.
template <bool BF16>
__device__ __forceinline__ float scale_of(uint32_t sb) {
    if constexpr (BF16) return __uint_as_float(sb << 16);
    else return __half2float(__ushort_as_half(static_cast<unsigned short>(sb & 0xffffu)));
}
template <bool BF16>
__device__ __forceinline__ float bias_of(uint32_t sb) {
    if constexpr (BF16) return __uint_as_float(sb & 0xffff0000u);
    else return __half2float(__ushort_as_half(static_cast<unsigned short>(sb >> 16)));
}

// NR: tiles of 8 query rows.  CTAs an SM: as many as leave few registers in memory.  (Spilled, bytes a thread: D = 64 28 to 52
// with groups of 64 and 230 with groups of 32, with two row tiles 144 and 644; D = 128 none, with two row tiles 84 and 508;
// D = 256 none.)
template <int D, int NR>
constexpr int kQmCtas = D == 256 ? 2 : NR == 2 ? (D == 64 ? 4 : 3) : (D == 64 ? 5 : 3);
// Blocks of 16 keys that a warp takes at a time: two where registers allow, for work that does not wait for one another.
template <int D, int NR>
constexpr int kQmBlocks = D * NR <= 128 ? 2 : 1;
// Sets of blocks that a warp has on their way or in work, each block [K codes][V codes][K affine][V affine].
constexpr int kQmStages = 3;
template <int D, int G>
constexpr int kQmStage = 16 * D + 2 * 16 * (D / G) * 4;
// A warp's stages; its rows of O at the end of a piece stand in their place.
template <int D, int G, int NR>
constexpr int kQmWarpBytes = kQmStages * kQmBlocks<D, NR> * kQmStage<D, G> > 8 * NR * (D + 4) * 4 ? kQmStages * kQmBlocks<D, NR> * kQmStage<D, G>
                                                                                               : 8 * NR * (D + 4) * 4;
template <int D, int G, int NR>
constexpr size_t kQmSmem = kQmWarps * kQmWarpBytes<D, G, NR> + NR * (D / 32) * 512;

template <int D, int G, int NR, bool BF16>
__global__ void __launch_bounds__(kQmThreads, (kQmCtas<D, NR>)) seq_quant_mma_kernel(const QmArgs ar) {
    const SeqArgs &a = ar.q.s;
    const QuantCache &cc = ar.q.c;
    constexpr int RR = 8 * NR, NB = D / 32, NG = D / G, BPG = G / 32, VW = NB / 2, OS = D + 4;
    __shared__ SeqScratch sched;
    __shared__ float2 s_ml[kQmWarps][RR];
    __shared__ __align__(16) float s_qf[NR * NG][4][4];       // of rows 2 t and 2 t + 1: sums of Q in a group, factors of its products
    __shared__ float s_far[RR];
    extern __shared__ __align__(128) unsigned char s_mem[];   // the warps' stages (or rows of O: [RR][OS]), then Q's fragments
    constexpr int WB = kQmWarpBytes<D, G, NR>, STG = kQmStage<D, G>, BL = kQmBlocks<D, NR>, STEP = 16 * kQmWarps;
    uint4 *s_q = reinterpret_cast<uint4 *>(s_mem + kQmWarps * WB);      // [NR][NB][32]
    auto s_o = [&](int w) { return reinterpret_cast<float *>(s_mem + w * WB); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3, cta = blockIdx.x;
    pdl_wait();
    const SeqRun run = seq_schedule<kQmThreads, kQmTks, kQmUnitCost, kQmLeast>(a, a.max_q, cta, ar.G, &sched);
    pdl_launch_dependents();
    if (tid == 0) ar.rec[cta] = {0, 0, 0, 0};
    const float scale2 = fmaxf(a.scale * kQmLog2e, FLT_MIN);   // (a scale of 0 weighs all keys alike, infinite products too)
    SeqWalk<kQmTks, kQmUnitCost> walk;
    walk.init(a, a.max_q, run, &sched, cta);
    SeqPiece p;
    while (walk.next(a, a.max_q, run, &p)) {
        // Q fragments of each two products: with G = 32 of block j the elements 32 j + 8 t + {0, 4 | 1, 5 | 2, 6 | 3, 7};
        // with G = 64, whose two blocks' quads are the halves of a word as it is, of blocks j0 and j0 + 1 (j0 = j less its lowest
        // bit b) the elements 8 t + 4 b + {0 | 1 | 2 | 3} of both.  The second and fourth pair are over 16 (their codes come
        // as 16 c), all times 2^e: the row's largest in [2^13, 2^14); each group's where a group's largest is below 2^-10 of that
        // (what f16 loses of it could count beside keys of large scales).  Rows of very large queries are worked on as 2^-32 of
        // them, so that no factor or sum leaves f32's range before the logit does (s_far: 2^32 for such a row, 1 for another).
        // Both are for the careful loop.
        uint64_t fr[NR];
        bool careful = false;
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            const int row = g + 8 * x, tok = row / a.g;
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + static_cast<long long>(p.q0 + tok) * a.q_st +
                                                               static_cast<long long>(p.kh * a.g + row - tok * a.g) * a.q_sh) + t;
            uint4 raw[NB];
            float big = 0.0f;
#pragma unroll
            for (int j = 0; j < NB; ++j) raw[j] = row < p.rows ? src[4 * j] : make_uint4(0, 0, 0, 0);
            auto widen = [](uint32_t w, float *f) {
                f[0] = scale_of<BF16>(w);
                f[1] = bias_of<BF16>(w);
            };
            float sum[NG], most[NG];
#pragma unroll
            for (int n = 0; n < NG; ++n) sum[n] = most[n] = 0.0f;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                float f[8];
                widen(raw[j].x, f); widen(raw[j].y, f + 2); widen(raw[j].z, f + 4); widen(raw[j].w, f + 6);
#pragma unroll
                for (int e = 0; e < 8; ++e) most[j / BPG] = fmaxf(most[j / BPG], fabsf(f[e]));
                sum[j / BPG] += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
            }
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                most[n] = fmaxf(most[n], __shfl_xor_sync(0xffffffffu, most[n], 1));
                most[n] = fmaxf(most[n], __shfl_xor_sync(0xffffffffu, most[n], 2));
                big = fmaxf(big, most[n]);
            }
            const bool is_far = BF16 && !(big * fmaxf(scale2, 1.0f) < 0x1p90f);
            const float less = is_far ? 0x1p-32f : 1.0f;
            bool apart = false;
#pragma unroll
            for (int n = 0; n < NG; ++n) apart |= most[n] > 0.0f && most[n] < big * 0x1p-10f;
            careful |= __any_sync(0xffffffffu, is_far || apart) != 0;
            if (t == 0 && warp == 0) s_far[8 * x + g] = is_far ? 0x1p32f : 1.0f;
            if (BF16 && is_far) {                       // the sums again
#pragma unroll
                for (int n = 0; n < NG; ++n) sum[n] = 0.0f;
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    float f[8];
                    widen(raw[j].x, f); widen(raw[j].y, f + 2); widen(raw[j].z, f + 4); widen(raw[j].w, f + 6);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[j / BPG] = fmaf(f[e], less, sum[j / BPG]);
                }
            }
            // exponents as they stand in the bits: 2^(13 - floor(log2 of the largest))
            auto up = [&](int n) { return min(267 - static_cast<int>(__float_as_uint(apart ? most[n] : big) >> 23), 250); };
            auto back = [&](int n) { return __uint_as_float(static_cast<uint32_t>(254 - up(n)) << 23) * less * 0x1p24f * scale2; };
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                float f[8];
                if constexpr (G == 32) {
                    widen(raw[j].x, f); widen(raw[j].y, f + 2); widen(raw[j].z, f + 4); widen(raw[j].w, f + 6);
                } else {
                    const uint4 r0 = raw[j & ~1], r1 = raw[j | 1];
                    widen(j & 1 ? r0.z : r0.x, f); widen(j & 1 ? r0.w : r0.y, f + 2);
                    widen(j & 1 ? r1.z : r1.x, f + 4); widen(j & 1 ? r1.w : r1.y, f + 6);
                }
                const float mul = __uint_as_float(static_cast<uint32_t>(up(j / BPG)) << 23), mul16 = mul * 0.0625f;
                const uint4 y = make_uint4(pack16<false>(f[0] * mul, f[4] * mul), pack16<false>(f[1] * mul16, f[5] * mul16),
                                           pack16<false>(f[2] * mul, f[6] * mul), pack16<false>(f[3] * mul16, f[7] * mul16));
                if (warp == (j & 3)) s_q[(x * NB + j) * 32 + lane] = y;
            }
            // 2^24 / 2^e of row g, and its sums: to the lanes that hold the rows 2 t and 2 t + 1 of a product
            fr[x] = two(__shfl_sync(0xffffffffu, back(0), 8 * t), __shfl_sync(0xffffffffu, back(0), 8 * t + 4));
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                float y = sum[n];
                y += __shfl_xor_sync(0xffffffffu, y, 1);
                y += __shfl_xor_sync(0xffffffffu, y, 2);
                if (t == 0 && warp == 0) {
                    s_qf[x * NG + n][g >> 1][g & 1] = y * scale2;
                    s_qf[x * NG + n][g >> 1][2 + (g & 1)] = back(n);
                }
            }
        }
        __syncthreads();
        // Of rows 2 t + e of tile x: running max, sum, sums of P b (each lane its keys'), power of two of P s
        // (mu: the running max less the raise, 0 where there is none; up: what moves it)
        float o[NR][NB][2][4], up[NR][2], l[NR][2];
        uint64_t ab[NR][NG], sc[NR][NG];
        const float top = __uint_as_float(static_cast<uint32_t>(127 + kQmTop) << 23);
        const int key_end = min(p.kv, (p.t0 + p.nt) << kQmTks);
        const int32_t *table = a.table + static_cast<long long>(p.b) * a.max_pages;
        // page of the 16-key block at `key` (0 behind the last key; -1 where there is none: its scales and biases are 0, so that
        // what its codes are does not matter)
        auto page_of = [&](int key) -> int {
            if (key >= key_end) return 0;
            const int page = __ldg(table + (key >> a.page_shift));
            if (static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages)) return page;
            // a page before every row's window may be gone
            if (lane == 0 && !(a.window && key + 16 <= p.prefix - a.window + 1)) atomicOr(a.status, kSeqBadPage);
            return -1;
        };
        // Copies of a block: K's and V's rows of codes, a 16-byte vector a lane and instruction, then rows of scales and
        // biases, K's by lanes 0 .. 15, V's by the others.  The whole block is in its page, so keys past the last
        // one come too, and are masked like the others that a row does not see.  V's vectors stand swizzled, so that the
        // reads below, of rows 2 t, find all banks.
        constexpr int CPR = D / 32, ROWS = 32 / CPR;                        // vectors of a row, rows of an instruction
        constexpr int OV = 8 * D, OA = 16 * D;                              // of V's codes, of the affine in a stage
        auto swizzled = [](int row, int off) { return off ^ ((D == 64 ? (row >> 2) & 1 : (row >> 1) & 3) << 5); };
        unsigned char *mine = s_mem + warp * WB;
        constexpr int FG = NG >= 4 ? 2 : 1;                                 // groups that share a floor
        const int c_row = lane / CPR;
        const uint32_t *k_lane = at_bytes(at_bytes(cc.kc + lane % CPR * 4, p.kh, cc.c_sh), c_row, cc.c_st);
        const uint32_t *a_lane = at_bytes(at_bytes(static_cast<const uint32_t *>(lane < 16 ? cc.ka : cc.va), p.kh, cc.a_sh), lane & 15, cc.a_st);
        const long long v_off = cc.vc - cc.kc;
        // (as one group) of the blocks at `key` and, where BL = 2, 64 keys on
        auto copy_blocks = [&](int key, const int (&page)[BL], int st) {
#pragma unroll
            for (int b = 0; b < BL; ++b)
                if (key + b * STEP < key_end) {
                    const int in = (key + b * STEP) & ((1 << a.page_shift) - 1);
                    const int from = max(page[b], 0);
                    const uint32_t *c = at_bytes(at_bytes(k_lane, from, cc.c_sp), in, cc.c_st);
                    const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(mine + (st * BL + b) * STG));
#pragma unroll
                    for (int i = 0; i < CPR / 2; ++i) {
                        const uint32_t *ci = at_bytes(c, i * ROWS, cc.c_st);
                        copy_vector(dst + lane * 16 + 512 * i, ci);
                        copy_vector(dst + OV + swizzled(c_row + i * ROWS, lane * 16 + 512 * i), ci + v_off);
                    }
                    copy_words<NG>(dst + OA + lane * (NG * 4), at_bytes(at_bytes(a_lane, from, cc.a_sp), in, cc.a_st), page[b] >= 0);
                }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // All keys of this warp.  CAREFUL: factors of each row and group, the lift of very large queries, keys whose V scale is
        // far below others' in f32; without it, false where such a key is met.
        auto all_keys = [&](auto is_careful) -> bool {
        constexpr bool CAREFUL = decltype(is_careful)::value;
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                up[x][e] = -INFINITY;
                l[x][e] = 0.0f;
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    ab[x][n] = 0;
                    sc[x][n] = two(top, top);   // too large for most scales: the first block sets it
                }
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) o[x][j][h][e] = o[x][j][h][2 + e] = 0.0f;
            }
        float floors[NG / FG] = {};                                         // 0: nothing is below
        auto lift = [&](int x, int e) { return CAREFUL ? s_far[8 * x + 2 * t + e] : 1.0f; };
        int key = (p.t0 << kQmTks) + 16 * warp, ahead = key, st = 0, page[BL];
#pragma unroll
        for (int b = 0; b < BL; ++b) page[b] = page_of(key + b * STEP);
#pragma unroll 1
        for (int i = 0; i < kQmStages - 1; ++i) {
            int cell[BL];
#pragma unroll
            for (int b = 0; b < BL; ++b) cell[b] = page_of(ahead + (BL + b) * STEP);
            copy_blocks(ahead, page, i);
            ahead += BL * STEP;
#pragma unroll
            for (int b = 0; b < BL; ++b) page[b] = cell[b];
        }
#pragma unroll 1
        for (; key < key_end; key += BL * STEP) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kQmStages - 2) : "memory");
            __syncwarp();
            copy_blocks(ahead, page, (st + kQmStages - 1) % kQmStages);    // where the blocks before were
            ahead += BL * STEP;
#pragma unroll
            for (int b = 0; b < BL; ++b) page[b] = page_of(ahead + b * STEP);
            const unsigned char *blk = mine + st * BL * STG;
            st = (st + 1) % kQmStages;
            // logits in log2 units, before the lift: s[b][x][2 n + e] of key g + 8 n of block b, row 2 t + e of tile x
            float s[BL][NR][4];
#pragma unroll
            for (int b = 0; b < BL; ++b) {
                uint32_t kw[2][NB], ka[2][NG];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    load_words<NB>(blk + b * STG + (8 * n + g) * (D / 2) + t * (NB * 4), kw[n]);
                    load_words<NG>(blk + b * STG + OA + (8 * n + g) * (NG * 4), ka[n]);
                }
            uint64_t s2[NR][2], u2[NR][2];
#pragma unroll
            for (int x = 0; x < NR; ++x) s2[x][0] = s2[x][1] = u2[x][0] = u2[x][1] = 0;
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                float acc[NR][4];
#pragma unroll
                for (int x = 0; x < NR; ++x) acc[x][0] = acc[x][1] = acc[x][2] = acc[x][3] = 0.0f;
#pragma unroll
                for (int j = n * BPG; j < (n + 1) * BPG; ++j) {
                    const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                    const int i0 = j / 2 + (j & 1 ? NB / 2 : 0);
                    const uint32_t w0 = G == 64 ? kw[0][i0] : __byte_perm(kw[0][j / 2], kw[0][NB / 2 + j / 2], sel);
                    const uint32_t w1 = G == 64 ? kw[1][i0] : __byte_perm(kw[1][j / 2], kw[1][NB / 2 + j / 2], sel);
                    const uint32_t h0 = w0 >> 8, h1 = w1 >> 8;
#pragma unroll
                    for (int x = 0; x < NR; ++x) {
                        const uint4 b = s_q[(x * NB + j) * 32 + lane];
                        mma16(acc[x], w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u, b.x, b.y);
                        mma16(acc[x], h0 & 0x000f000fu, h1 & 0x000f000fu, h0 & 0x00f000f0u, h1 & 0x00f000f0u, b.z, b.w);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float sk = scale_of<BF16>(ka[i][n]), bk = bias_of<BF16>(ka[i][n]);
#pragma unroll
                    for (int x = 0; x < NR; ++x) {
                        const uint64_t *qf = reinterpret_cast<const uint64_t *>(s_qf[x * NG + n][t]);
                        const uint64_t y = two(acc[x][2 * i], acc[x][2 * i + 1]);
                        s2[x][i] = fma_two(two(sk, sk), CAREFUL ? mul_two(y, qf[1]) : y, s2[x][i]);
                        u2[x][i] = fma_two(two(bk, bk), qf[0], u2[x][i]);
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < NR; ++x)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint64_t y = fma_two(s2[x][i], CAREFUL ? two(1.0f, 1.0f) : fr[x], u2[x][i]);
                    s[b][x][2 * i] = first(y);
                    s[b][x][2 * i + 1] = second(y);
                }
            }
            // bit 2 n + e: is key g + 8 n of block b seen by row 2 t + e
            const int last = key + (BL - 1) * STEP;
            const bool masked = key < p.full_lo || last + 16 > p.full_hi || last >= key_end;
            uint32_t see[BL][NR];
#pragma unroll
            for (int b = 0; b < BL; ++b)
#pragma unroll
                for (int x = 0; x < NR; ++x) see[b][x] = 15u;
            if (masked) {
#pragma unroll
                for (int x = 0; x < NR; ++x) {
#pragma unroll
                    for (int b = 0; b < BL; ++b) see[b][x] = 0u;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 8 * x + 2 * t + e, tok = row / a.g;
                        const bool live = row < p.rows;
                        uint32_t anc[kMaxTreeBitsNodes / 32] = {}, w[1];
                        if (a.parents && live) seq_ancestors(a.parents + p.q0, tok, anc);
#pragma unroll
                        for (int b = 0; b < BL; ++b) {
                            seq_visible<1>(a, p.prefix, live && key + b * STEP < key_end ? p.kv : 0, tok, anc, key + b * STEP, w);
                            see[b][x] |= ((w[0] >> g) & 1u) << e | ((w[0] >> (g + 8)) & 1u) << (2 + e);
                        }
                    }
#pragma unroll
                    for (int b = 0; b < BL; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!((see[b][x] >> i) & 1u)) s[b][x][i] = -INFINITY;
                }
            }
            bool rise = false;
#pragma unroll
            for (int x = 0; x < NR; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(s[0][x][e], s[0][x][2 + e]);
                    if (BL == 2) mx = fmaxf(mx, fmaxf(s[BL - 1][x][e], s[BL - 1][x][2 + e]));
                    rise |= mx * lift(x, e) > up[x][e];
                }
            if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                for (int x = 0; x < NR; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(s[0][x][e], s[0][x][2 + e]);
                        if (BL == 2) mx = fmaxf(mx, fmaxf(s[BL - 1][x][e], s[BL - 1][x][2 + e]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)) * lift(x, e);
                        if (mx > up[x][e]) {
                            if (up[x][e] != -INFINITY) {
                                const float down = mx - (up[x][e] - kQmSlack), f = ex2(-down);
                                l[x][e] *= f;
#pragma unroll
                                for (int n = 0; n < NG; ++n) {
                                    ab[x][n] = mul_two(ab[x][n], e ? two(1.0f, f) : two(f, 1.0f));
                                    // what O holds of the scales keeps its size as far as its power of two can take the factor
                                    const uint32_t was = __float_as_uint(part(sc[x][n], e));
                                    const float raise = fminf(floorf(down), static_cast<float>(127 + kQmTop - static_cast<int>(was >> 23)));
                                    const float fo = ex2(raise - down), now = __uint_as_float(was + (static_cast<uint32_t>(raise) << 23));
                                    sc[x][n] = e ? two(first(sc[x][n]), now) : two(now, second(sc[x][n]));
#pragma unroll
                                    for (int j = n * BPG; j < (n + 1) * BPG; ++j)
#pragma unroll
                                        for (int h = 0; h < 2; ++h) {
                                            o[x][j][h][e] *= fo;
                                            o[x][j][h][2 + e] *= fo;
                                        }
                                }
                            }
                            up[x][e] = mx + kQmSlack;
                        }
                    }
            }
            uint64_t pr[BL][NR][2];
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                float mu[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) mu[e] = up[x][e] == -INFINITY ? 0.0f : up[x][e] - (kQmSlack + kQmRaise);
#pragma unroll
                for (int b = 0; b < BL; ++b) {
                    float y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = ex2(CAREFUL ? fmaf(s[b][x][i], lift(x, i & 1), -mu[i & 1]) : s[b][x][i] - mu[i & 1]);
                    l[x][0] += y[0] + y[2];
                    l[x][1] += y[1] + y[3];
                    pr[b][x][0] = two(y[0], y[1]);
                    pr[b][x][1] = two(y[2], y[3]);
                }
            }
            uint32_t va[BL][2][NG];
#pragma unroll
            for (int b = 0; b < BL; ++b)
#pragma unroll
                for (int n = 0; n < 2; ++n) load_words<NG>(blk + b * STG + OA + (16 + 8 * n + g) * (NG * 4), va[b][n]);
            // P s and the sums of P b; where a row does not see a key its scale and bias do not count
            uint64_t ps[BL][NR][NG][2];
            float most = 0.0f;
            if (!masked) {
#pragma unroll
                for (int b = 0; b < BL; ++b)
#pragma unroll
                    for (int n = 0; n < NG; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float sv = scale_of<BF16>(va[b][i][n]), bv = bias_of<BF16>(va[b][i][n]);
#pragma unroll
                            for (int x = 0; x < NR; ++x) {
                                ps[b][x][n][i] = mul_two(mul_two(pr[b][x][i], sc[x][n]), two(sv, sv));
                                ab[x][n] = fma_two(pr[b][x][i], two(bv, bv), ab[x][n]);
                                most = max_abs3(most, first(ps[b][x][n][i]), second(ps[b][x][n][i]));
                            }
                        }
            } else {
#pragma unroll
                for (int b = 0; b < BL; ++b)
#pragma unroll
                    for (int n = 0; n < NG; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int x = 0; x < NR; ++x) {
                                const uint32_t w0 = (see[b][x] >> (2 * i)) & 1u ? va[b][i][n] : 0u, w1 = (see[b][x] >> (2 * i + 1)) & 1u ? va[b][i][n] : 0u;
                                ps[b][x][n][i] = mul_two(mul_two(pr[b][x][i], sc[x][n]), two(scale_of<BF16>(w0), scale_of<BF16>(w1)));
                                ab[x][n] = fma_two(pr[b][x][i], two(bias_of<BF16>(w0), bias_of<BF16>(w1)), ab[x][n]);
                                most = max_abs3(most, first(ps[b][x][n][i]), second(ps[b][x][n][i]));
                            }
            }
            // is a scale of this lane's keys below its groups' floor (or 0)
            bool low = false;
#pragma unroll
            for (int f = 0; f < NG / FG; ++f) {
                float y = floors[f];
#pragma unroll
                for (int n = f * FG; n < (f + 1) * FG; ++n)
#pragma unroll
                    for (int b = 0; b < BL; ++b) y = min_abs3(y, scale_of<BF16>(va[b][0][n]), scale_of<BF16>(va[b][1][n]));
                low |= y < floors[f];
            }
            bool spread = false;                        // some scale is too far below the ones that count
            if (__any_sync(0xffffffffu, most > 40000.0f || low)) {
#pragma unroll
                for (int x = 0; x < NR; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float peak = kQmPeak;           // the row's largest weight here, if above the least one of a largest
#pragma unroll
                        for (int b = 0; b < BL; ++b) peak = fmaxf(peak, fmaxf(part(pr[b][x][0], e), part(pr[b][x][1], e)));
#pragma unroll
                        for (int k = 4; k < 32; k <<= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, k));
#pragma unroll
                        for (int n = 0; n < NG; ++n) {
                            float v[BL][2], hit = 0.0f; // hit: the largest P s, 2^-16 of it
#pragma unroll
                            for (int b = 0; b < BL; ++b)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    v[b][i] = (see[b][x] >> (2 * i + e)) & 1u ? scale_of<BF16>(va[b][i][n]) : 0.0f;
                                    hit = fmaxf(hit, fabsf(v[b][i]) <= FLT_MAX ? part(pr[b][x][i], e) * (fabsf(v[b][i]) * 0x1p-16f) : 0.0f);
                                }
#pragma unroll
                            for (int k = 4; k < 32; k <<= 1) hit = fmaxf(hit, __shfl_xor_sync(0xffffffffu, hit, k));
                            float now = part(sc[x][n], e);
                            if (hit * now > 40000.0f * 0x1p-16f) {
                                // out of f16's range: the power of two that brings it to a quarter of the peak
                                const float was = now;
                                const int to = 109 + static_cast<int>(__float_as_uint(peak) >> 23) - static_cast<int>(__float_as_uint(hit) >> 23);
                                now = fminf(__uint_as_float(static_cast<uint32_t>(max(to, 1)) << 23), was);
                                const float f = now / was;
                                sc[x][n] = e ? two(first(sc[x][n]), now) : two(now, second(sc[x][n]));
#pragma unroll
                                for (int j = n * BPG; j < (n + 1) * BPG; ++j)
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        o[x][j][h][e] *= f;
                                        o[x][j][h][2 + e] *= f;
                                    }
#pragma unroll
                                for (int b = 0; b < BL; ++b)
#pragma unroll
                                    for (int i = 0; i < 2; ++i) {
                                        const float y = part(pr[b][x][i], e) * now * v[b][i];
                                        ps[b][x][n][i] = e ? two(first(ps[b][x][n][i]), y) : two(y, second(ps[b][x][n][i]));
                                    }
                            }
#pragma unroll
                            for (int b = 0; b < BL; ++b)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const float y = fabsf(v[b][i]) * now;
                                    spread |= y > 0.0f && y < kQmFloor && part(pr[b][x][i], e) > kQmFaint;
                                }
                        }
                    }
                spread = __any_sync(0xffffffffu, spread);
                // the floors as scales, of the rows and groups that count them the highest
#pragma unroll
                for (int f = 0; f < NG / FG; ++f) {
                    float y = INFINITY;
#pragma unroll
                    for (int x = 0; x < NR; ++x)
#pragma unroll
                        for (int n = f * FG; n < (f + 1) * FG; ++n) y = min_abs3(y, first(sc[x][n]), second(sc[x][n]));
                    floors[f] = kQmFloor / y;
                }
            }
            if (!CAREFUL && spread) return false;
            if constexpr (CAREFUL)
            if (spread) {
                // in f32, a key at a time: O's places of the products below
#pragma unroll
                for (int b = 0; b < BL; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll 1
                        for (int r = 0; r < 8; ++r) {
                            const int row = r + 8 * i;
                            uint32_t w[VW];
                            load_words<VW>(blk + b * STG + OV + swizzled(row, row * (D / 2) + g * (VW * 4)), w);
#pragma unroll
                            for (int x = 0; x < NR; ++x)
#pragma unroll
                                for (int n = 0; n < NG; ++n) {
                                    const uint64_t y = mul_two(__shfl_sync(0xffffffffu, ps[b][x][n][i], 4 * r + t), two(0x1p-24f, 0x1p-24f));
#pragma unroll
                                    for (int j = n * BPG; j < (n + 1) * BPG; ++j)
#pragma unroll
                                        for (int h = 0; h < 2; ++h) {
                                            const uint32_t c = w[j / 2] >> (16 * (j & 1) + 8 * h);
                                            const float c0 = static_cast<float>(c & 15u), c1 = static_cast<float>(c & 240u);
                                            o[x][j][h][0] = fmaf(first(y), c0, o[x][j][h][0]);
                                            o[x][j][h][1] = fmaf(second(y), c0, o[x][j][h][1]);
                                            o[x][j][h][2] = fmaf(first(y), c1, o[x][j][h][2]);
                                            o[x][j][h][3] = fmaf(second(y), c1, o[x][j][h][3]);
                                        }
                                }
                        }
                continue;
            }
            // O += V^T (P s): elements 32 j + 4 g + 2 h (+ 1) of 16 rows of the product, 8 query rows
#pragma unroll
            for (int b = 0; b < BL; ++b) {
                uint32_t pb[NR][NG][2], vw[4][VW];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int row = 2 * t + (n & 1) + 8 * (n >> 1);
                    load_words<VW>(blk + b * STG + OV + swizzled(row, row * (D / 2) + g * (VW * 4)), vw[n]);
                }
#pragma unroll
                for (int x = 0; x < NR; ++x)
#pragma unroll
                    for (int n = 0; n < NG; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) pb[x][n][i] = transpose8(pack16<false>(first(ps[b][x][n][i]), second(ps[b][x][n][i])));
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                    const uint32_t w0 = __byte_perm(vw[0][j / 2], vw[1][j / 2], sel), w1 = __byte_perm(vw[2][j / 2], vw[3][j / 2], sel);
                    const uint32_t h0 = w0 >> 8, h1 = w1 >> 8;
#pragma unroll
                    for (int x = 0; x < NR; ++x) {
                        mma16(o[x][j][0], w0 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x000f000fu, w1 & 0x00f000f0u, pb[x][j / BPG][0], pb[x][j / BPG][1]);
                        mma16(o[x][j][1], h0 & 0x000f000fu, h0 & 0x00f000f0u, h1 & 0x000f000fu, h1 & 0x00f000f0u, pb[x][j / BPG][0], pb[x][j / BPG][1]);
                    }
                }
            }
        }
        return true;
        };
        if (careful || !all_keys(std::false_type{})) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
            all_keys(std::true_type{});
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();                                   // O's rows stand where the stages were
        if (tid == 0 && p.rest > 0) ar.rec[cta] = seq_record(run, cta, p);
        // ---- join the four warps
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * x + 2 * t + e;
                float y = l[x][e];
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) y += __shfl_xor_sync(0xffffffffu, y, k);
                if (g == 0) s_ml[warp][row] = make_float2(up[x][e] - kQmSlack, y);
                float *dst = s_o(warp) + row * OS + 4 * g;
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    float b = e ? second(ab[x][n]) : first(ab[x][n]);
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1) b += __shfl_xor_sync(0xffffffffu, b, k);
                    // (2^24 on O, not on f: that would be infinite for scales from 2^101 on)
                    const float f = 1.0f / part(sc[x][n], e), f16 = f * 0.0625f;
                    auto whole = [](float y) { return y * 0x1p24f; };
#pragma unroll
                    for (int j = n * BPG; j < (n + 1) * BPG; ++j)
                        *reinterpret_cast<float4 *>(dst + 32 * j) =
                            make_float4(fmaf(whole(o[x][j][0][e]), f, b), fmaf(whole(o[x][j][0][2 + e]), f16, b),
                                        fmaf(whole(o[x][j][1][e]), f, b), fmaf(whole(o[x][j][1][2 + e]), f16, b));
                }
            }
        __syncthreads();
        for (int i = tid; i < p.rows * (D / 8); i += kQmThreads) {
            const int row = i / (D / 8), d = (i - row * (D / 8)) * 8;
            float2 w[kQmWarps];
            float ms = -INFINITY, ls = 0.0f;
#pragma unroll
            for (int k = 0; k < kQmWarps; ++k) {
                w[k] = s_ml[k][row];
                ms = fmaxf(ms, w[k].x);
            }
            // a warp without a logit above -inf adds 0, or NaN where its logits were NaN
            const float mu = ms == -INFINITY ? 0.0f : ms;
            float r[8] = {};
#pragma unroll
            for (int k = 0; k < kQmWarps; ++k) {
                const float f = ex2(w[k].x - mu);
                ls += f * w[k].y;
                const float4 y = *reinterpret_cast<const float4 *>(s_o(k) + row * OS + d);
                const float4 z = *reinterpret_cast<const float4 *>(s_o(k) + row * OS + d + 4);
                r[0] += f * y.x; r[1] += f * y.y; r[2] += f * y.z; r[3] += f * y.w;
                r[4] += f * z.x; r[5] += f * z.y; r[6] += f * z.z; r[7] += f * z.w;
            }
            if (p.slot < 0) {
                const float inv = ls > 0.0f ? 1.0f / ls : (ls == 0.0f ? 0.0f : ls);
                const int tk = row / a.g;
                uint16_t *out = static_cast<uint16_t *>(a.out) + static_cast<long long>(p.q0 + tk) * a.o_st +
                                static_cast<long long>(p.kh * a.g + row - tk * a.g) * a.o_sh + d;
                uint4 y;
                y.x = pack16<BF16>(r[0] * inv, r[1] * inv);
                y.y = pack16<BF16>(r[2] * inv, r[3] * inv);
                y.z = pack16<BF16>(r[4] * inv, r[5] * inv);
                y.w = pack16<BF16>(r[6] * inv, r[7] * inv);
                *reinterpret_cast<uint4 *>(out) = y;
            } else {
                float *dst = ar.o + (static_cast<size_t>(p.slot) * RR + row) * D + d;
                *reinterpret_cast<float4 *>(dst) = make_float4(r[0], r[1], r[2], r[3]);
                *reinterpret_cast<float4 *>(dst + 4) = make_float4(r[4], r[5], r[6], r[7]);
                if (d == 0) ar.ml[static_cast<size_t>(p.slot) * RR + row] = make_float2(ms, ls);
            }
        }
        __syncthreads();
    }
}

template <int D, int G, int NR, bool BF16>
cudaError_t qm_launch(const SeqQuantArgs &a, void *ws, int sms, cudaStream_t s) {
    constexpr int RR = 8 * NR;
    QmArgs ar;
    ar.q = a;
    ar.G = sms * kQmCtas<D, NR>;
    char *w = static_cast<char *>(ws);
    ar.rec = reinterpret_cast<SeqRec *>(w + 256);
    w += 256 + (ar.G * sizeof(SeqRec) + 255) / 256 * 256;
    ar.ml = reinterpret_cast<float2 *>(w);
    ar.o = reinterpret_cast<float *>(w + sizeof(float2) * 2 * ar.G * RR);
    auto kern = seq_quant_mma_kernel<D, G, NR, BF16>;
    static unsigned long long done = 0;
    cudaError_t e = set_smem_limit_once(kern, kQmSmem<D, G, NR>, &done);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(ar.G), dim3(kQmThreads), kQmSmem<D, G, NR>, s, ar);
    count_launch();
    if (e != cudaSuccess) return e;
    e = launch_pdl(seq_mma_merge_kernel<D, RR, BF16, 32>, dim3(ar.G, D / 32), dim3(kMergeThreads), 0, s, a.s, ar.rec, ar.ml, ar.o);
    count_launch();
    return e;
}

template <int D, int G>
cudaError_t qm_launch_group(const SeqQuantArgs &a, void *ws, int sms, cudaStream_t s) {
    const int rows = a.s.max_q * a.s.g;
    if constexpr (D <= 128)
        if (rows > 8) return a.s.bf16 ? qm_launch<D, G, 2, true>(a, ws, sms, s) : qm_launch<D, G, 2, false>(a, ws, sms, s);
    return a.s.bf16 ? qm_launch<D, G, 1, true>(a, ws, sms, s) : qm_launch<D, G, 1, false>(a, ws, sms, s);
}
template <int D>
cudaError_t qm_launch_dim(const SeqQuantArgs &a, void *ws, int sms, cudaStream_t s) {
    return a.group == 32 ? qm_launch_group<D, 32>(a, ws, sms, s) : qm_launch_group<D, 64>(a, ws, sms, s);
}
template <int D>
unsigned long long qm_workspace(int rows, int sms) {
    const int nr = D <= 128 && rows > 8 ? 2 : 1;
    const unsigned long long G = static_cast<unsigned long long>(sms) * (nr == 2 ? kQmCtas<D, 2> : kQmCtas<D, 1>), cap = 8 * nr;
    return 256 + (G * sizeof(SeqRec) + 255) / 256 * 256 + 2 * G * cap * (sizeof(float2) + sizeof(float) * D);
}

}  // namespace
}  // namespace ta
