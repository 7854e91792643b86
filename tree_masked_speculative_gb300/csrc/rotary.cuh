// Rotation of rows by their positions, shared by the appends: 16-byte vectors, the cosines and
// sines of a column kept over several heads.
#pragma once

#include "quant_page.cuh"

namespace ta {

constexpr int kRotThreads = 256;

template <bool BF16>
__device__ __forceinline__ void widen8(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 v;
        if constexpr (BF16) v = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        else v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}
template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}
template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
    return make_uint4(narrow2<BF16>(f[0], f[1]), narrow2<BF16>(f[2], f[3]), narrow2<BF16>(f[4], f[5]), narrow2<BF16>(f[6], f[7]));
}
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// x / per; most calls are small enough for a 32-bit quotient (a 64-bit one takes about a hundred instructions).
__device__ __forceinline__ long long item_token(long long x, unsigned per) {
    return x <= 0xffffffffll ? static_cast<long long>(static_cast<uint32_t>(x) / per) : x / per;
}

// Where row t goes: its table row (nullptr: position outside the table).
__device__ __forceinline__ const float *rot_row(const RotaryArgs &a, int t) {
    const int p = __ldg(a.pos + t);
    return p >= 0 && p < a.max_pos ? a.table + static_cast<long long>(p) * a.R : nullptr;
}

// A thread's part of HB heads' rows: column c of D / 16, two vectors of each row, turned where
// they are among the first R elements.  src and dst are the first head's rows, sh and dh head
// strides (vectors); `heads` of them.
template <bool BF16, int HB>
__device__ __forceinline__ void turn_rows(const RotaryArgs &a, const float *row, int c, int heads, const uint4 *src,
                                          long long sh, uint4 *dst, long long dh) {
    const int pairs = a.R >> 4;
    int v0, v1;
    if (c >= pairs) {                                   // behind the turned part: as it is
        v0 = (a.R >> 3) + c - pairs;
        v1 = v0 + ((a.D - a.R) >> 4);
    } else {
        v0 = a.interleaved ? 2 * c : c;
        v1 = a.interleaved ? v0 + 1 : c + pairs;
    }
    uint4 x[HB], y[HB];
#pragma unroll
    for (int h = 0; h < HB; ++h)
        if (h < heads) {
            x[h] = src[h * sh + v0];
            y[h] = src[h * sh + v1];
        }
    if (c < pairs) {
        float cs[8], sn[8];
        load8(row + 8 * c, cs);
        load8(row + (a.R >> 1) + 8 * c, sn);
#pragma unroll
        for (int h = 0; h < HB; ++h)
            if (h < heads) {
                float p[8], q[8];
                widen8<BF16>(x[h], p);
                widen8<BF16>(y[h], q);
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p0 = p[2 * e], p1 = p[2 * e + 1], q0 = q[2 * e], q1 = q[2 * e + 1];
                        p[2 * e] = fmaf(p0, cs[e], -(p1 * sn[e]));
                        p[2 * e + 1] = fmaf(p1, cs[e], p0 * sn[e]);
                        q[2 * e] = fmaf(q0, cs[4 + e], -(q1 * sn[4 + e]));
                        q[2 * e + 1] = fmaf(q1, cs[4 + e], q0 * sn[4 + e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float p0 = p[e], q0 = q[e];
                        p[e] = fmaf(p0, cs[e], -(q0 * sn[e]));
                        q[e] = fmaf(q0, cs[e], p0 * sn[e]);
                    }
                }
                x[h] = narrow8<BF16>(p);
                y[h] = narrow8<BF16>(q);
            }
    }
#pragma unroll
    for (int h = 0; h < HB; ++h)
        if (h < heads) {
            dst[h * dh + v0] = x[h];
            dst[h * dh + v1] = y[h];
        }
}

// Thread x of the query rows' part: items of (token, HB heads, column).
template <bool BF16, int HB>
__device__ __forceinline__ void turn_queries(const RotaryArgs &a, long long x) {
    const unsigned cols = static_cast<unsigned>(a.D) >> 4, blocks = (static_cast<unsigned>(a.H) + HB - 1) / HB;
    const long long t = item_token(x, cols * blocks);
    if (t >= a.T) return;
    const unsigned r = static_cast<unsigned>(x - t * (cols * blocks)), hb = r / cols, c = r - hb * cols;
    const float *row = rot_row(a, static_cast<int>(t));
    if (row == nullptr) return;
    const int h = static_cast<int>(hb) * HB;
    turn_rows<BF16, HB>(a, row, static_cast<int>(c), min(HB, a.H - h), static_cast<const uint4 *>(a.q) + t * a.q_st + h * a.q_sh,
                        a.q_sh, static_cast<uint4 *>(a.q_out) + t * a.qo_st + h * a.qo_sh, a.qo_sh);
}

// Blocks for items of `per` heads each.
inline long long rot_blocks(long long tokens, int heads, int per, int cols) {
    return (tokens * ((heads + per - 1) / per) * cols + kRotThreads - 1) / kRotThreads;
}

}  // namespace ta
