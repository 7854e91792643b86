// New rows into 4-bit pages, keys turned by their positions on the way, and rows read back.
//
// A group of G elements x becomes scale = T((max - min) / 15), bias = T(min) and codes
// c = round((x - bias) / scale).  The codes are those of exact arithmetic, whatever the order
// of a sum: a turned element is held as f32 plus its rounding error (two products and a sum with
// their errors), a quotient next to a border between two codes is decided by the sign of
// x - bias - (c + 1/2) scale, which f32 gives exactly, and a scale next to a border of T is
// taken again in 64 bits.
//
// It reads 4 D and writes D + 8 D / G bytes a KV head and token (HBM); a lane takes 8
// neighbouring elements of up to HB heads, a group's 4 or 8 lanes reduce by shuffles.  Blocks run in order, so queries (HBM
// bounds them) and keys and values (latency of the loads and the instructions of exact codes) take their times one behind the
// other: half of the issue slots and half of HBM on average.  With four heads a thread 72 bytes are spilled and 140 read back.
// Measured: 16381 tokens, 32 / 8 heads of 128, f16, groups of 32: append 90 us (K and V alone 52 turned, 40 as they are, 50 in
// bf16), read 34 us, which together have 454 MB to move (68 us); 48 tokens: 3.0 and 1.7 us.
#include "rotary.cuh"

namespace ta {
namespace {

__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t bits16(float x) { return narrow2<BF16>(x, 0.0f) & 0xffffu; }
template <bool BF16>
__device__ __forceinline__ float round16(float x) {
    if constexpr (BF16) return __bfloat162float(__float2bfloat16_rn(x));
    else return __half2float(__float2half_rn(x));
}

// Two f32 at a time.
__device__ __forceinline__ uint64_t two(float x, float y) {
    return static_cast<uint64_t>(__float_as_uint(x)) | (static_cast<uint64_t>(__float_as_uint(y)) << 32);
}
__device__ __forceinline__ float first(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float second(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
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
// x - y
__device__ __forceinline__ uint64_t sub2(uint64_t x, uint64_t y) { return fma2(y, two(-1.0f, -1.0f), x); }

// x c + y s as hi + lo: hi the nearest f32, lo what is left (off by about 2^-48 of the larger product; where the two cancel
// so that this counts, nothing is off: products of a 16-bit and a 32-bit float of like size have 35 bits, and the errors'
// sums fit f32).
__device__ __forceinline__ void turn_exact(uint64_t x, uint64_t c, uint64_t y, uint64_t s, uint64_t *hi, uint64_t *lo) {
    const uint64_t minus = two(-1.0f, -1.0f);
    const uint64_t p = mul2(x, c), pe = fma2(mul2(x, minus), c, p);        // pe, qe: the products' errors, negated
    const uint64_t q = mul2(y, s), qe = fma2(mul2(y, minus), s, q);
    const uint64_t z = add2(p, q), b = sub2(z, p);
    const uint64_t e = add2(sub2(p, sub2(z, b)), sub2(q, b));
    const uint64_t l = sub2(e, add2(pe, qe));
    *hi = add2(z, l);
    *lo = sub2(l, sub2(*hi, z));
}

// A quotient next to k + 1/2: which of k and k + 1 is nearer to (hi + lo - bias) / scale.
// (`thr`: how far v may be from a code without asking; a small one says that v itself is of little use.)
__device__ __noinline__ float near_border(float hi, float lo, float bias, float scale, float v, float thr) {
    if (thr < 0.25f) {
        const double x = static_cast<double>(hi) + lo, d = __dadd_rn(x, -static_cast<double>(bias)), q = fmin(fmax(d / scale, -1.0), 16.0);
        const double k = floor(q);
        double left = 0.0;
        if (q - k == 0.5) {                             // what 64 bits dropped from the difference decides
            const double w = __dadd_rn(d, -x);
            left = __fma_rn(-(k + 0.5), static_cast<double>(scale), d) + (__dadd_rn(x, -__dadd_rn(d, -w)) - __dadd_rn(bias, w));
        }
        return static_cast<float>(left > 0.0 ? k + 1.0 : left < 0.0 ? k : rint(q));
    }
    const float k = floorf(v), d = __fadd_rn(hi, -bias), b = __fadd_rn(d, -hi);
    const float e = __fadd_rn(__fadd_rn(hi, -__fadd_rn(d, -b)), -__fadd_rn(bias, b));
    const float u = __fadd_rn(__fmaf_rn(-(k + 0.5f), scale, d), __fadd_rn(e, lo));
    return u > 0.0f ? k + 1.0f : u < 0.0f ? k : 2.0f * rintf(0.5f * (k + 0.5f));   // a tie: the even one
}

// Codes of a lane's 8 elements (4 bits each, lowest first) and their group's scale and bias as
// 16-bit halves of *affine.  The GL lanes of a group call it together, the warp's others too.
template <bool BF16, int GL, bool EXACT>
__device__ __forceinline__ uint32_t quantise(const uint64_t (&hi)[4], const uint64_t (&lo)[4], uint32_t *affine) {
    float mx = first(hi[0]), mn = mx;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        mx = max_nan(mx, max_nan(first(hi[e]), second(hi[e])));
        mn = min_nan(mn, min_nan(first(hi[e]), second(hi[e])));
    }
#pragma unroll
    for (int o = 1; o < GL; o <<= 1) {
        mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    }
    const float range = __fadd_rn(mx, -mn), r = __fmul_rn(range, 1.0f / 15.0f), big = fmaxf(fabsf(mx), fabsf(mn));
    // does a relative error of 2^-20 move the 16-bit scale (r is off by 2^-22, and by what is left of the
    // extremes, at most 2^-24 of each)
    const uint32_t both = narrow2<BF16>(r * (1.0f - 0x1p-20f), r * (1.0f + 0x1p-20f));
    uint32_t sb = both & 0xffffu;
    const bool unsure = sb != both >> 16 || !(range <= FLT_MAX) || (EXACT && big > 4.0f * range);
    if (__any_sync(0xffffffffu, unsure)) {
        float lx = -INFINITY, ln = INFINITY;            // what is left of the largest and the least
        if constexpr (EXACT) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (first(hi[e]) == mx) lx = fmaxf(lx, first(lo[e]));
                if (second(hi[e]) == mx) lx = fmaxf(lx, second(lo[e]));
                if (first(hi[e]) == mn) ln = fminf(ln, first(lo[e]));
                if (second(hi[e]) == mn) ln = fminf(ln, second(lo[e]));
            }
#pragma unroll
            for (int o = 1; o < GL; o <<= 1) {
                lx = fmaxf(lx, __shfl_xor_sync(0xffffffffu, lx, o));
                ln = fminf(ln, __shfl_xor_sync(0xffffffffu, ln, o));
            }
        } else {
            lx = ln = 0.0f;
        }
        if (unsure)
            sb = bits16<BF16>(static_cast<float>(((static_cast<double>(mx) + lx) - (static_cast<double>(mn) + ln)) / 15.0));
    }
    const uint32_t bb = bits16<BF16>(mn);
    const float bias = BF16 ? __uint_as_float(bb << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(bb)));
    const float scale = BF16 ? __uint_as_float(sb << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(sb)));
    // (a NaN fails every comparison)
    const bool bad = !(fabsf(mx) <= FLT_MAX && fabsf(mn) <= FLT_MAX && fabsf(bias) <= FLT_MAX && scale <= FLT_MAX);
    *affine = bad ? 0x7fff7fffu : sb | bb << 16;        // (NaN in either type)
    const float inv = scale > 0.0f && !bad ? __frcp_rn(scale) : 0.0f;
    // The quotients as x / scale - bias / scale, clamped, rounded by adding 1.5 2^23, packed by exact products.  They are
    // off by 2^-22 of the larger term and by lo / scale at most; where one is next to a border between two
    // codes, the 8 of them are looked at one by one.
    const float shift = -bias * inv;
    const uint64_t iv = two(inv, inv), sh = two(shift, shift), magic = two(12582912.0f, 12582912.0f), less = two(-12582912.0f, -12582912.0f);
    float dev = 0.0f, quad[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float n[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint64_t v = fma2(hi[2 * w + e], iv, sh);
            const uint64_t c = two(fminf(fmaxf(first(v), 0.0f), 15.0f), fminf(fmaxf(second(v), 0.0f), 15.0f));
            const uint64_t k = add2(add2(c, magic), less), d = sub2(c, k);
            asm("max.f32 %0, %0, %1, %2;" : "+f"(dev) : "f"(fabsf(first(d))), "f"(fabsf(second(d))));
            n[2 * e] = first(k);
            n[2 * e + 1] = second(k);
        }
        quad[w] = fmaf(fmaf(fmaf(n[3], 16.0f, n[2]), 16.0f, n[1]), 16.0f, n[0]);
    }
    uint32_t codes = static_cast<uint32_t>(quad[0]) | static_cast<uint32_t>(quad[1]) << 16;
    float thr = 0.5f - 4e-6f - big * inv * 0x1p-21f;
    if (scale < 0x1p-100f || !(range <= FLT_MAX)) thr = -1.0f;   // the reciprocal or a difference may be out of range
    if (!(dev <= thr)) {
        codes = 0u;
        if (scale > 0.0f && !bad) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = e & 1 ? second(hi[e >> 1]) : first(hi[e >> 1]), l = !EXACT ? 0.0f : e & 1 ? second(lo[e >> 1]) : first(lo[e >> 1]);
                const float v = __fmul_rn(__fadd_rn(h, -bias), inv);
                float k = rintf(v);
                if (!(fabsf(v - k) <= thr)) k = near_border(h, l, bias, scale, v, thr);
                codes |= static_cast<uint32_t>(fminf(fmaxf(k, 0.0f), 15.0f)) << (4 * e);
            }
        }
    }
    return bad ? 0u : codes;
}

// Blocks [0, nq) turn queries, [nq, nq + nk) take keys, the others values.  Three blocks an SM (90 us for the tokens above)
// leave more registers than four (105) and more warps than two (104); HB = 4 heads a thread: 1 and 2 took 135, 8 took 161.
template <bool BF16, int HB, int GL>
__global__ void __launch_bounds__(kRotThreads, 3) quant_append_kernel(const QuantAppendArgs ar, unsigned nq, unsigned nk) {
    pdl_wait();
    const RotaryArgs &a = ar.r;
    if (blockIdx.x < nq) {
        turn_queries<BF16, HB>(a, static_cast<long long>(blockIdx.x) * kRotThreads + threadIdx.x);
        return;
    }
    const bool is_v = blockIdx.x >= nq + nk;
    const long long x = static_cast<long long>(blockIdx.x - (is_v ? nq + nk : nq)) * kRotThreads + threadIdx.x;
    const unsigned cols = static_cast<unsigned>(a.D) >> 3, blocks = (static_cast<unsigned>(a.Hk) + HB - 1) / HB;
    const long long t = item_token(x, cols * blocks);
    const unsigned r = static_cast<unsigned>(x - t * (cols * blocks)), hb = r / cols, i = r - hb * cols;
    // all lanes stay for the shuffles; a row's lanes agree
    const float *row = nullptr;
    long long slot = -1;
    if (t < a.T) {
        slot = a.slot[t];
        if (a.pos) {
            row = rot_row(a, static_cast<int>(t));
            if (row == nullptr) slot = -1;
        }
    }
    const bool live = slot >= 0 && slot < static_cast<long long>(a.n_pages) << a.page_shift;
    const int h0 = static_cast<int>(hb) * HB, heads = live ? min(HB, a.Hk - h0) : 0;
    const uint32_t page = live ? static_cast<uint32_t>(slot >> a.page_shift) : 0u, in = live ? static_cast<uint32_t>(slot) & ((1u << a.page_shift) - 1) : 0u;
    // where the lane's word goes: quads g and g + 1 of block i / 4, two blocks' quads a word
    const unsigned j = i >> 2, nb = static_cast<unsigned>(a.D) >> 5, g = 2 * (i & 3) + (j & 1);
    uint32_t *codes = at_bytes(at_bytes(at_bytes((is_v ? ar.c.vc : ar.c.kc) + (g * nb + (j & ~1u)) / 2, page, ar.c.c_sp), in, ar.c.c_st), h0, ar.c.c_sh);
    uint32_t *affine = at_bytes(at_bytes(at_bytes(static_cast<uint32_t *>(is_v ? ar.c.va : ar.c.ka) + i / GL, page, ar.c.a_sp), in, ar.c.a_st), h0, ar.c.a_sh);
    const long long sh = is_v ? a.v_sh : a.k_sh;
    const uint4 *src = static_cast<const uint4 *>(is_v ? a.v_new : a.k_new) + (live ? t * (is_v ? a.v_st : a.k_st) + h0 * sh : 0);
    const unsigned half = static_cast<unsigned>(a.R) >> 4;          // vectors of half of the turned part
    const bool turned = !is_v && a.pos && i < 2 * half;
    const bool second_half = !a.interleaved && i >= half;
    const unsigned other = a.interleaved ? i : second_half ? i - half : i + half;
    uint4 u[HB], w[HB];
#pragma unroll
    for (int h = 0; h < HB; ++h) {
        u[h] = w[h] = make_uint4(0, 0, 0, 0);
        if (h < heads) {
            u[h] = src[h * sh + i];
            if (turned && !a.interleaved) w[h] = src[h * sh + other];
        }
    }
    uint64_t cs[4], sn[4];
    if (turned && live) {
        if (a.interleaved) {                            // 4 pairs
            const float4 c = __ldg(reinterpret_cast<const float4 *>(row) + i), s = __ldg(reinterpret_cast<const float4 *>(row + (a.R >> 1)) + i);
            const float c4[4] = {c.x, c.y, c.z, c.w}, s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                cs[e] = two(c4[e], c4[e]);
                sn[e] = two(-s4[e], s4[e]);
            }
        } else {
            const unsigned c = second_half ? i - half : i;
            float c8[8], s8[8];
            load8(row + 8 * c, c8);
            load8(row + (a.R >> 1) + 8 * c, s8);
            const float sign = second_half ? 1.0f : -1.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                cs[e] = two(c8[2 * e], c8[2 * e + 1]);
                sn[e] = two(sign * s8[2 * e], sign * s8[2 * e + 1]);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            cs[e] = two(1.0f, 1.0f);
            sn[e] = 0;
        }
    }
#pragma unroll
    for (int h = 0; h < HB; ++h) {
        float x8[8], y8[8];
        uint64_t hi[4], lo[4] = {};
        widen8<BF16>(u[h], x8);
#pragma unroll
        for (int e = 0; e < 4; ++e) hi[e] = two(x8[2 * e], x8[2 * e + 1]);
        uint32_t af, cd;
        if (is_v || !a.pos) {                           // uniform over the block
            cd = quantise<BF16, GL, false>(hi, lo, &af);
        } else {
            widen8<BF16>(w[h], y8);
            if (turned) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t y = a.interleaved ? two(x8[2 * e + 1], x8[2 * e]) : two(y8[2 * e], y8[2 * e + 1]);
                    turn_exact(hi[e], cs[e], y, sn[e], &hi[e], &lo[e]);
                }
            }
            cd = quantise<BF16, GL, true>(hi, lo, &af);
        }
        // blocks j and j + 1 (j even) swap quads, so that a lane holds a whole word
        const uint32_t send = j & 1 ? cd & 0xffffu : cd >> 16;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, send, 4);
        const uint32_t word = j & 1 ? got | (cd & 0xffff0000u) : (cd & 0xffffu) | got << 16;
        if (h < heads) {
            *at_bytes(codes, h, ar.c.c_sh) = word;
            if (i % GL == 0) *at_bytes(affine, h, ar.c.a_sh) = af;
        }
    }
}

// A thread: one word (8 codes) of K or V of a row.  Its index divisions by sizes that are known only at run time and its
// 8-byte stores keep it at 2.6 times the time of its bytes.
template <bool BF16>
__global__ void __launch_bounds__(kRotThreads) quant_read_kernel(const QuantReadArgs a) {
    pdl_wait();
    const unsigned words = static_cast<unsigned>(a.D) >> 3, per = 2 * words * a.Hk, nb = static_cast<unsigned>(a.D) >> 5;
    const long long n = static_cast<long long>(a.T) * per;
    for (long long x = static_cast<long long>(blockIdx.x) * kRotThreads + threadIdx.x; x < n; x += static_cast<long long>(gridDim.x) * kRotThreads) {
        const long long t = item_token(x, per);
        const unsigned r = static_cast<unsigned>(x - t * per), h2 = r / words, w = r - h2 * words, h = h2 >> 1;
        const bool is_v = h2 & 1;
        const long long slot = a.slot[t];
        uint16_t *out = static_cast<uint16_t *>(is_v ? a.v : a.k) + t * (is_v ? a.v_st : a.k_st) + h * (is_v ? a.v_sh : a.k_sh);
        const unsigned g = 2 * w / nb, j = 2 * w % nb;
        if (slot < 0 || slot >= static_cast<long long>(a.n_pages) << a.page_shift) {
            for (unsigned q = 0; q < 2; ++q) *reinterpret_cast<uint2 *>(out + 32 * (j + q) + 4 * g) = make_uint2(0, 0);
            continue;
        }
        const uint32_t page = static_cast<uint32_t>(slot >> a.page_shift), in = static_cast<uint32_t>(slot) & ((1u << a.page_shift) - 1);
        const uint32_t c = __ldg(at_bytes(at_bytes(at_bytes((is_v ? a.c.vc : a.c.kc) + w, page, a.c.c_sp), h, a.c.c_sh), in, a.c.c_st));
        const uint32_t *af = at_bytes(at_bytes(at_bytes(static_cast<const uint32_t *>(is_v ? a.c.va : a.c.ka), page, a.c.a_sp), h, a.c.a_sh), in, a.c.a_st);
#pragma unroll
        for (unsigned q = 0; q < 2; ++q) {
            const unsigned d = 32 * (j + q) + 4 * g;
            const uint32_t sb = __ldg(af + d / a.group);
            const float s = BF16 ? __uint_as_float(sb << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(sb & 0xffffu)));
            const float b = BF16 ? __uint_as_float(sb & 0xffff0000u) : __half2float(__ushort_as_half(static_cast<unsigned short>(sb >> 16)));
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = fmaf(s, static_cast<float>((c >> (16 * q + 4 * e)) & 15u), b);
            *reinterpret_cast<uint2 *>(out + d) = make_uint2(narrow2<BF16>(f[0], f[1]), narrow2<BF16>(f[2], f[3]));
        }
    }
}

template <bool BF16, int HB, int GL>
cudaError_t launch(const QuantAppendArgs &a, cudaStream_t s) {
    const long long nq = a.r.H ? rot_blocks(a.r.T, a.r.H, HB, a.r.D / 16) : 0, nk = rot_blocks(a.r.T, a.r.Hk, HB, a.r.D / 8);
    if (nq + 2 * nk > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_pdl(quant_append_kernel<BF16, HB, GL>, dim3(static_cast<unsigned>(nq + 2 * nk)), dim3(kRotThreads), 0, s, a,
                                     static_cast<unsigned>(nq), static_cast<unsigned>(nk));
    count_launch();
    return e;
}
template <bool BF16>
cudaError_t launch_type(const QuantAppendArgs &a, cudaStream_t s) {
    // one head a thread while that leaves the GPU's thread slots unfilled
    const bool few = static_cast<long long>(a.r.T) * (a.r.H + 4 * a.r.Hk) * (a.r.D / 16) <= 152ll * 2048;
    if (a.group == 32) return few ? launch<BF16, 1, 4>(a, s) : launch<BF16, 4, 4>(a, s);
    return few ? launch<BF16, 1, 8>(a, s) : launch<BF16, 4, 8>(a, s);
}

}  // namespace

cudaError_t launch_quant_append(const QuantAppendArgs &a, cudaStream_t s) {
    return a.r.bf16 ? launch_type<true>(a, s) : launch_type<false>(a, s);
}

cudaError_t launch_quant_read(const QuantReadArgs &a, cudaStream_t s) {
    const long long n = static_cast<long long>(a.T) * a.Hk * (a.D / 4), blocks = (n + kRotThreads - 1) / kRotThreads;
    const dim3 grid(static_cast<unsigned>(blocks < 152 * 8 ? blocks : 152 * 8));
    const cudaError_t e = a.bf16 ? launch_pdl(quant_read_kernel<true>, grid, dim3(kRotThreads), 0, s, a)
                                 : launch_pdl(quant_read_kernel<false>, grid, dim3(kRotThreads), 0, s, a);
    count_launch();
    return e;
}

}  // namespace ta
