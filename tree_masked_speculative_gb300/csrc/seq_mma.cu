// Attention of few query rows per KV head over paged K/V (single tokens, small
// drafts) with warp-level MMAs: max_q_len * (heads per KV head) <= 16 rows (8 for
// head dimension 256), f16 / bf16.
//
// The work is reading K and V once, so HBM bounds it (4 D bytes a key and KV head;
// 16 query rows are far below the tensor rate).  Three requests of 200 to 2100 keys take
// 14 us, a chain of latencies: schedule, table, K and V, join, merge.  K and V go from global memory
// straight into MMA fragments, without shared memory: Q K^T contracts over d in any
// order, so a lane's 16-byte vector of K serves two m16n8k16 products as it is;
// for P V a lane holds the same 8 columns of keys 2t, 2t + 1, 2t + 8, 2t + 9 and
// pairs them by byte permutes.  A warp takes every fourth block of 16 keys of its
// CTA's run and keeps one block of K and V (8 KB at D = 128) in flight in registers;
// 12 warps an SM then cover HBM's latency.  No barrier inside the key loop; the four
// warps' (max, sum, O) are joined in shared memory at the end of a unit's piece.
// The batch is cut evenly over the CTAs by the schedule of seq_sched.cuh.
//
// Against the tcgen05 kernel, whose 128-row tiles hold these few rows (us, bf16, one token of 32
// heads on 8 KV heads where nothing else is said, graphs replayed on inputs out of L2):
//                                          D = 64       D = 128      D = 256
//   64 requests of 900 to 16384 keys      189 / 296    373 / 374   1064 / 694
//   32 of 4096 keys, 4 rows                53 /  80     96 / 101    270 / 177
//   32 of 4096 keys, 8 rows                54 /  82     97 / 101    274 / 177
//   32 of 4096 keys, 16 rows               59 /  82     99 / 102       -
//   200 of 300 keys                        37 /  73     62 /  82    154 / 111
//   1000 of 40 keys                        60 / 181     94 / 199    208 / 236
//   one of 4000 keys                       17 /  36     19 /  39     32 /  41
//   one of 4000 keys, 8 heads on one       14 /  52     18 /  52     25 /  54
// At D = 256 an SM holds only 8 warps of it, with 255 registers and 720 bytes of spills a thread: 4.4
// of 6.8 TB/s.  There it is chosen where (request, KV head) pairs are few, seq_mma_best().
// (Spills of the other instances: 316 bytes at D = 64, 232 with 16 rows; 360 at D = 128, none
// with 16 rows.)
#include "seq_sched.cuh"

namespace ta {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTks = 6;                             // schedule granularity: 64 keys, 16 a warp
// Tiles of a CTA's run at least: fewer CTAs than fit where the batch is small, for
// fewer pieces to join (three requests of 200 to 2100 keys: 15.6, 14.8, 14.0 and 16.0 us
// with 1, 2, 3 and 4).
constexpr int kLeast = 3;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;
// P and l of f16 rows are held 2^7 higher (P <= 2^15): a weight is subnormal only below 2^-21 of
// the running max's, and off by 2^-32 of it at most.  At 2^0 weights up to 2^-25 were lost: an
// output of 6000 such weights beside one large weight (whose value is 0) came out up to 43 % low.
template <bool BF16>
constexpr float kRaise = BF16 ? 0.0f : 7.0f;

struct MmaArgs {
    SeqArgs a;
    SeqRec *rec;      // [G]
    float2 *ml;       // [2 G][16]
    float *o;         // [2 G][16][D]
    int G;
};

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
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
// Bits 15 and 31: is the low / high value infinite or NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t odd16(uint32_t w) {
    return (BF16 ? (w & 0x7f807f80u) + 0x00800080u : (w & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
}

// RH: 8-row halves of the 16-row MMA tile in use.  Registers: 8 (K, V of a block: D / 4
// each) + Q and O (D / 8 and D / 4 a half); CTAs per SM follow.
template <int D, int RH>
constexpr int kCtasPerSm = D == 256 ? 2 : (RH == 2 ? (D == 64 ? 4 : 2) : (D == 64 ? 5 : 3));

template <int D, int RH, bool BF16>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<D, RH>) seq_mma_kernel(const MmaArgs ar) {
    const SeqArgs &a = ar.a;
    constexpr int RR = 8 * RH;                          // rows held
    constexpr int NQ = D / 64;                          // 64-column groups
    __shared__ SeqScratch sched;
    __shared__ float2 s_ml[kWarps][RR];
    __shared__ uint32_t s_odd[RR][D / 32];              // columns that are not finite for a row
    __shared__ int s_any_odd;
    extern __shared__ __align__(16) float s_o[];        // [kWarps][RR][D]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3, cta = blockIdx.x;
    pdl_wait();
    const SeqRun run = seq_schedule<kThreads, kTks, 0, kLeast>(a, a.max_q, cta, ar.G, &sched);
    pdl_launch_dependents();
    if (tid == 0) {
        ar.rec[cta] = {0, 0, 0, 0};
        s_any_odd = 0;
    }
    for (int i = tid; i < RR * (D / 32); i += kThreads) (&s_odd[0][0])[i] = 0u;
    __syncthreads();
    const float scale2 = fmaxf(a.scale * kLog2e, FLT_MIN);   // above 0: a masked -inf stays -inf
    const uint16_t *kc = static_cast<const uint16_t *>(a.k), *vc = static_cast<const uint16_t *>(a.v);
    SeqWalk<kTks, 0> walk;
    walk.init(a, a.max_q, run, &sched, cta);
    SeqPiece p;
    while (walk.next(a, a.max_q, run, &p)) {
        // Q fragments: columns 32 j + 8 t + 4 h + {0, 1 | 2, 3} of rows g, g + 8
        uint32_t qa[RH][D / 16][2];
        int tok[RH];
#pragma unroll
        for (int x = 0; x < RH; ++x) {
            const int row = g + 8 * x;
            tok[x] = row / a.g;
            const uint16_t *q = static_cast<const uint16_t *>(a.q) + static_cast<long long>(p.q0 + tok[x]) * a.q_st +
                                static_cast<long long>(p.kh * a.g + row - tok[x] * a.g) * a.q_sh + 8 * t;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                uint2 y = make_uint2(0, 0);
                if (row < p.rows) y = *reinterpret_cast<const uint2 *>(q + 32 * (j >> 1) + 4 * (j & 1));
                qa[x][j][0] = y.x;
                qa[x][j][1] = y.y;
            }
        }
        float o[NQ][8][RH][2];
        float m[RH], l[RH];
#pragma unroll
        for (int x = 0; x < RH; ++x) {
            m[x] = -INFINITY;
            l[x] = 0.0f;
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int j = 0; j < 8; ++j) o[q][j][x][0] = o[q][j][x][1] = 0.0f;
        }
        const int key_end = min(p.kv, (p.t0 + p.nt) << kTks);
        const int32_t *table = a.table + static_cast<long long>(p.b) * a.max_pages;
        const long long head = p.kh * a.k_sh;
        // element offset of key 0 of the 16-key block at `key` (its page holds all 16), -1: none
        auto block_of = [&](int key) -> long long {
            if (key >= key_end) return -1;
            const int page = __ldg(table + (key >> a.page_shift));
            if (page < 0 || page >= a.n_pages) {
                // a page before every row's window may be gone
                if (lane == 0 && !(a.window && key + 16 <= p.prefix - a.window + 1)) atomicOr(a.status, kSeqBadPage);
                return -1;
            }
            return page * a.k_sp + (key & ((1 << a.page_shift) - 1)) * a.k_st + head;
        };
        uint4 kb[2][D / 32], vb[4][NQ];
        auto load_k = [&](long long at, int key) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const bool in = at >= 0 && key + 8 * n + g < p.kv;
                const uint16_t *src = kc + at + (8 * n + g) * a.k_st + 8 * t;
#pragma unroll
                for (int j = 0; j < D / 32; ++j) kb[n][j] = in ? load_once(src + 32 * j) : make_uint4(0, 0, 0, 0);
            }
        };
        auto load_v = [&](long long at, int key) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int kk = 2 * t + (n & 1) + 8 * (n >> 1);
                const bool in = at >= 0 && key + kk < p.kv;
                const uint16_t *src = vc + at + kk * a.v_st + 8 * g;
#pragma unroll
                for (int q = 0; q < NQ; ++q) vb[n][q] = in ? load_once(src + 64 * q) : make_uint4(0, 0, 0, 0);
            }
        };
        int key = (p.t0 << kTks) + 16 * warp;
        long long at = block_of(key), next = block_of(key + 16 * kWarps);
        load_k(at, key);
        load_v(at, key);
#pragma unroll 1
        for (; key < key_end; key += 16 * kWarps) {
            // S = Q K^T of 16 keys
            float s[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const uint4 b = kb[n][j];
                    mma<BF16>(s[n], qa[0][2 * j][0], RH == 2 ? qa[RH - 1][2 * j][0] : 0u, qa[0][2 * j][1],
                              RH == 2 ? qa[RH - 1][2 * j][1] : 0u, b.x, b.y);
                    mma<BF16>(s[n], qa[0][2 * j + 1][0], RH == 2 ? qa[RH - 1][2 * j + 1][0] : 0u, qa[0][2 * j + 1][1],
                              RH == 2 ? qa[RH - 1][2 * j + 1][1] : 0u, b.z, b.w);
                }
            }
            const long long after = block_of(key + 32 * kWarps);
            load_k(next, key + 16 * kWarps);
            // mask: S element e of half x, block n is row g + 8 x, key + 8 n + 2 t + e
            const bool masked = key < p.full_lo || key + 16 > p.full_hi;
            uint32_t see[RH];
            if (masked) {
#pragma unroll
                for (int x = 0; x < RH; ++x) {
                    uint32_t anc[kMaxTreeBitsNodes / 32] = {}, w[1];
                    const bool live = g + 8 * x < p.rows;
                    if (a.parents && live) seq_ancestors(a.parents + p.q0, tok[x], anc);
                    seq_visible<1>(a, p.prefix, live ? p.kv : 0, tok[x], anc, key, w);
                    see[x] = w[0] & 0xffffu;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (!((see[x] >> (8 * n + 2 * t + e)) & 1u)) s[n][2 * x + e] = -INFINITY;
                }
            }
            uint32_t pa[RH][2];
            bool moved = false;
            float alpha[RH];
#pragma unroll
            for (int x = 0; x < RH; ++x) {
                float mx = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1])) * scale2;
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                alpha[x] = 1.0f;
                if (mx > m[x] + kSlack) {
                    alpha[x] = ex2(m[x] - mx);          // 0 from -inf
                    m[x] = mx;
                    l[x] *= alpha[x];
                    moved = true;
                }
                const float mu = m[x] == -INFINITY ? 0.0f : kRaise<BF16> - m[x];
                const float p0 = ex2(fmaf(s[0][2 * x], scale2, mu)), p1 = ex2(fmaf(s[0][2 * x + 1], scale2, mu));
                const float p2 = ex2(fmaf(s[1][2 * x], scale2, mu)), p3 = ex2(fmaf(s[1][2 * x + 1], scale2, mu));
                l[x] += (p0 + p1) + (p2 + p3);
                pa[x][0] = pack16<BF16>(p0, p1);
                pa[x][1] = pack16<BF16>(p2, p3);
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int q = 0; q < NQ; ++q)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int x = 0; x < RH; ++x) {
                            o[q][j][x][0] *= alpha[x];
                            o[q][j][x][1] *= alpha[x];
                        }
            }
            if (masked) {
                // an element of V that is not finite must not reach rows that do not see it (0 x NaN):
                // it is taken out, and the rows that see it are marked
                uint32_t odd = 0u;
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
                        odd |= odd16<BF16>(vb[n][q].x) | odd16<BF16>(vb[n][q].y) | odd16<BF16>(vb[n][q].z) | odd16<BF16>(vb[n][q].w);
                if (__any_sync(0xffffffffu, odd != 0u)) {
                    if (lane == 0) s_any_odd = 1;
#pragma unroll 1
                    for (int row = 0; row < p.rows; ++row) {
                        // row's visibility from the lanes that hold it
                        const uint32_t seen = __shfl_sync(0xffffffffu, RH == 2 && row >= 8 ? see[RH - 1] : see[0], (row & 7) * 4);
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            if (!((seen >> (2 * t + (n & 1) + 8 * (n >> 1))) & 1u)) continue;
#pragma unroll
                            for (int q = 0; q < NQ; ++q) {
                                const uint32_t w[4] = {vb[n][q].x, vb[n][q].y, vb[n][q].z, vb[n][q].w};
                                uint32_t bits = 0u;
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    const uint32_t f = odd16<BF16>(w[c]);
                                    bits |= ((f >> 15) & 1u) << (2 * c) | (f >> 31) << (2 * c + 1);
                                }
                                const int d = 64 * q + 8 * g;
                                if (bits) atomicOr(&s_odd[row][d >> 5], bits << (d & 31));
                            }
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int q = 0; q < NQ; ++q) {
                            auto fix = [](uint32_t w) {
                                const uint32_t f = odd16<BF16>(w);
                                return w & ~(((f >> 15) & 1u) * 0xffffu) & ~((f >> 31) * 0xffff0000u);
                            };
                            vb[n][q] = make_uint4(fix(vb[n][q].x), fix(vb[n][q].y), fix(vb[n][q].z), fix(vb[n][q].w));
                        }
                }
            }
            // O += P V, 8 columns 64 q + 8 n + j (n = 0 .. 7) a product
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const uint32_t v0[4] = {vb[0][q].x, vb[0][q].y, vb[0][q].z, vb[0][q].w}, v1[4] = {vb[1][q].x, vb[1][q].y, vb[1][q].z, vb[1][q].w};
                const uint32_t v2[4] = {vb[2][q].x, vb[2][q].y, vb[2][q].z, vb[2][q].w}, v3[4] = {vb[3][q].x, vb[3][q].y, vb[3][q].z, vb[3][q].w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                    const uint32_t b0 = __byte_perm(v0[j >> 1], v1[j >> 1], sel), b1 = __byte_perm(v2[j >> 1], v3[j >> 1], sel);
                    float c[4] = {o[q][j][0][0], o[q][j][0][1], RH == 2 ? o[q][j][RH - 1][0] : 0.0f, RH == 2 ? o[q][j][RH - 1][1] : 0.0f};
                    mma<BF16>(c, pa[0][0], RH == 2 ? pa[RH - 1][0] : 0u, pa[0][1], RH == 2 ? pa[RH - 1][1] : 0u, b0, b1);
                    o[q][j][0][0] = c[0];
                    o[q][j][0][1] = c[1];
                    if (RH == 2) {
                        o[q][j][RH - 1][0] = c[2];
                        o[q][j][RH - 1][1] = c[3];
                    }
                }
            }
            load_v(next, key + 16 * kWarps);
            next = after;
        }
        if (tid == 0 && p.rest > 0) ar.rec[cta] = seq_record(run, cta, p);
        // ---- join the four warps
#pragma unroll
        for (int x = 0; x < RH; ++x) {
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
            if (t == 0) s_ml[warp][g + 8 * x] = make_float2(m[x], l[x]);
            // columns 64 q + 16 t + {0 .. 7} (c0 of j = 0 .. 7), + 8 (c1)
            float *dst = s_o + (warp * RR + g + 8 * x) * D + 16 * t;
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < 8; j += 4)
                        *reinterpret_cast<float4 *>(dst + 64 * q + 8 * e + j) =
                            make_float4(o[q][j][x][e], o[q][j + 1][x][e], o[q][j + 2][x][e], o[q][j + 3][x][e]);
        }
        __syncthreads();
        const bool any_odd = s_any_odd != 0;
        for (int i = tid; i < p.rows * (D / 8); i += kThreads) {
            const int row = i / (D / 8), d = (i - row * (D / 8)) * 8;
            float2 w[kWarps];
            float ms = -INFINITY, ls = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                w[k] = s_ml[k][row];
                ms = fmaxf(ms, w[k].x);
            }
            // a warp without a logit above -inf adds 0, or NaN where its logits were NaN
            const float mu = ms == -INFINITY ? 0.0f : ms;
            float r[8] = {};
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float f = ex2(w[k].x - mu);
                ls += f * w[k].y;
                const float4 y = *reinterpret_cast<const float4 *>(s_o + (k * RR + row) * D + d);
                const float4 z = *reinterpret_cast<const float4 *>(s_o + (k * RR + row) * D + d + 4);
                r[0] += f * y.x; r[1] += f * y.y; r[2] += f * y.z; r[3] += f * y.w;
                r[4] += f * z.x; r[5] += f * z.y; r[6] += f * z.z; r[7] += f * z.w;
            }
            if (any_odd) {
                const uint32_t bits = s_odd[row][d >> 5] >> (d & 31);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if ((bits >> e) & 1u) r[e] = __int_as_float(0x7fffffff);
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
                float *dst = ar.o + (static_cast<size_t>(p.slot) * 16 + row) * D + d;
                *reinterpret_cast<float4 *>(dst) = make_float4(r[0], r[1], r[2], r[3]);
                *reinterpret_cast<float4 *>(dst + 4) = make_float4(r[4], r[5], r[6], r[7]);
                if (d == 0) ar.ml[static_cast<size_t>(p.slot) * 16 + row] = make_float2(ms, ls);
            }
        }
        __syncthreads();
        if (any_odd) {                                  // the next piece starts without marks
            for (int i = tid; i < RR * (D / 32); i += kThreads) (&s_odd[0][0])[i] = 0u;
            if (tid == 0) s_any_odd = 0;
            __syncthreads();
        }
    }
}

// out = sum_p O_p 2^(m_p - m*) / sum_p l_p 2^(m_p - m*) over the pieces of the cut unit
// that starts in CTA blockIdx.x.  A few units are cut into many pieces when the
// batch is small, so a block's threads share the pieces as well as the columns
// (one thread a column through all of 22 pieces took 14 us).
constexpr int kMergeThreads = 256;
template <int D, bool BF16>
__global__ void __launch_bounds__(kMergeThreads) seq_mma_merge_kernel(const MmaArgs ar) {
    const SeqArgs &a = ar.a;
    __shared__ float s_m[16], s_inv[16];
    __shared__ float4 s_part[kMergeThreads];
    pdl_wait();
    const int c = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const SeqRec rec = ar.rec[c];
    if (rec.parts == 0) return;
    auto slot = [&](int p) { return static_cast<size_t>(p == 0 ? 2 * c + 1 : 2 * (c + p)); };
    for (int row = warp; row < rec.rows; row += kMergeThreads / 32) {
        float m = -INFINITY, l = 0.0f;
#pragma unroll 2
        for (int p = lane; p < rec.parts; p += 32) {
            const float2 w = ar.ml[slot(p) * 16 + row];
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
    const int items = rec.rows * (D / 4);
    int share = 1;
    while (2 * share * items <= kMergeThreads) share *= 2;
    const int per = kMergeThreads / share;              // items at a time
    for (int i0 = 0; i0 < items; i0 += per) {
        const int k = tid / per, i = i0 + tid - k * per;
        float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int row = i / (D / 4), d = (i - row * (D / 4)) * 4;
        if (i < items) {
            const float mu = s_m[row];
#pragma unroll 4
            for (int p = k; p < rec.parts; p += share) {
                const float f = ex2(ar.ml[slot(p) * 16 + row].x - mu);
                const float4 y = *reinterpret_cast<const float4 *>(ar.o + (slot(p) * 16 + row) * D + d);
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

template <int D, int RH, bool BF16>
cudaError_t launch(const MmaArgs &ar, cudaStream_t s) {
    auto kern = seq_mma_kernel<D, RH, BF16>;
    const size_t smem = sizeof(float) * kWarps * 8 * RH * D;
    cudaError_t e = launch_pdl(kern, dim3(ar.G), dim3(kThreads), smem, s, ar);
    count_launch();
    if (e != cudaSuccess) return e;
    e = launch_pdl(seq_mma_merge_kernel<D, BF16>, dim3(ar.G), dim3(kMergeThreads), 0, s, ar);
    count_launch();
    return e;
}

int ctas_per_sm(int d, int rows) {
    const bool two = rows > 8;
    if (d == 64) return two ? kCtasPerSm<64, 2> : kCtasPerSm<64, 1>;
    if (d == 128) return two ? kCtasPerSm<128, 2> : kCtasPerSm<128, 1>;
    return kCtasPerSm<256, 1>;
}

}  // namespace

bool seq_mma_takes(int d, long long rows) { return rows <= (d == 256 ? 8 : 16); }
// Few units are cut into many pieces, and latency counts: one request of 4000 keys on 8 KV heads
// 32 us against 41, on one 25 against 54.  From 64 units on HBM does: 48 against 41 (2000 keys).
bool seq_mma_best(int d, long long units) { return d <= 128 || units <= 8; }

unsigned long long seq_mma_workspace(int d, int rows, int sms) {
    const unsigned long long G = static_cast<unsigned long long>(sms) * ctas_per_sm(d, rows);
    return 256 + (G * sizeof(SeqRec) + 255) / 256 * 256 + 2 * G * 16 * (sizeof(float2) + sizeof(float) * d);
}

cudaError_t launch_seq_mma(const SeqArgs &a, void *ws, int sms, cudaStream_t s) {
    const int rows = a.max_q * a.g;
    MmaArgs ar;
    ar.a = a;
    ar.G = sms * ctas_per_sm(a.D, rows);
    char *w = static_cast<char *>(ws);
    ar.rec = reinterpret_cast<SeqRec *>(w + 256);
    w += 256 + (ar.G * sizeof(SeqRec) + 255) / 256 * 256;
    ar.ml = reinterpret_cast<float2 *>(w);
    ar.o = reinterpret_cast<float *>(w + sizeof(float2) * 2 * ar.G * 16);
    const bool two = rows > 8;
    if (a.bf16) {
        if (a.D == 64) return two ? launch<64, 2, true>(ar, s) : launch<64, 1, true>(ar, s);
        if (a.D == 128) return two ? launch<128, 2, true>(ar, s) : launch<128, 1, true>(ar, s);
        return launch<256, 1, true>(ar, s);
    }
    if (a.D == 64) return two ? launch<64, 2, false>(ar, s) : launch<64, 1, false>(ar, s);
    if (a.D == 128) return two ? launch<128, 2, false>(ar, s) : launch<128, 1, false>(ar, s);
    return launch<256, 1, false>(ar, s);
}

}  // namespace ta
