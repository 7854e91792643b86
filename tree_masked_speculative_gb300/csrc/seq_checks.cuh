// Argument checks shared by the serving entry points (seq_api.cu, quant_page_api.cu): all of
// them before any launch, overflow-checked.
#pragma once

#include <cudaTypedefs.h>

#include <atomic>
#include <climits>
#include <cmath>

#include "seq_internal.cuh"
#include "tree_attn.h"

namespace ta {
namespace {

#define SEQ_FAIL(st, ...)            \
    do {                             \
        set_last_error(__VA_ARGS__); \
        return st;                   \
    } while (0)
#define SEQ_TRY(x)                   \
    do {                             \
        const ta_status _s = (x);    \
        if (_s != TA_OK) return _s;  \
    } while (0)

constexpr ta_buf kNone = {nullptr, 0, TA_F32, 0};
bool is_absent(const ta_buf *b) { return b == nullptr || (b->ptr == nullptr && b->bytes == 0); }
const ta_buf &of(const ta_buf *b) { return b ? *b : kNone; }

const char *type_name(int t) {
    static const char *const names[] = {"F32", "F16", "BF16", "U32", "I32", "I64"};
    return t >= 0 && t <= TA_I64 ? names[t] : "unknown";
}

ta_status check(const char *op, const char *name, const ta_buf &b, int type, uint64_t need, size_t align) {
    if (b.reserved != 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: %s: reserved field must be 0", op, name);
    if (b.ptr == nullptr) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: %s: NULL pointer", op, name);
    if (b.dtype != type)
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: %s dtype must be %s, got %s", op, name, type_name(type), type_name(b.dtype));
    if (reinterpret_cast<uintptr_t>(b.ptr) % align != 0)
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: %s: pointer must be %zu-byte aligned", op, name, align);
    if (b.bytes < need)
        SEQ_FAIL(TA_ERR_BUFFER_TOO_SMALL, "%s: %s buffer too small: have %llu bytes, need >= %llu", op, name,
                 static_cast<unsigned long long>(b.bytes), static_cast<unsigned long long>(need));
    return TA_OK;
}

[[maybe_unused]] ta_status check_16bit(const char *op, const char *name, const ta_buf &b) {
    if (b.dtype != TA_F16 && b.dtype != TA_BF16)
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: %s dtype must be F16 or BF16, got %s", op, name, type_name(b.dtype));
    return TA_OK;
}

bool page_size_ok(uint32_t ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }
int log2_of(uint32_t ps) { return __builtin_ctz(ps); }

// Bytes of a strided 16-bit array: sum of (n_i - 1) * stride_i, plus the last
// axis's head_dim elements.  false on overflow.
struct Axis {
    uint64_t n, stride;
};
template <int N>
bool extent(const Axis (&ax)[N], uint64_t dim, uint64_t *bytes) {
    uint64_t e = dim;
    for (const Axis &x : ax) {
        uint64_t t;
        if (__builtin_mul_overflow(x.n - 1, x.stride, &t) || __builtin_add_overflow(e, t, &e)) return false;
    }
    return !__builtin_mul_overflow(e, uint64_t(2), bytes) && *bytes <= static_cast<uint64_t>(LLONG_MAX);
}

ta_status check_stride(const char *op, const char *name, uint64_t s) {
    if (s % 8 != 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: %s must be a multiple of 8 elements", op, name);
    // the range a tensor-map stride holds (2^40 bytes), and signed 64-bit offsets in the kernels
    if (s >= (uint64_t(1) << 38)) SEQ_FAIL(TA_ERR_UNSUPPORTED, "%s: %s exceeds 2^38 elements", op, name);
    return TA_OK;
}

// Rows of a call and keys of a request: positions, and positions less a window, stay
// within 32 bits.
constexpr uint32_t kMostKeys = 1u << 30;

ta_status check_heads(const char *op, uint32_t batch, uint32_t h, uint32_t hk, uint32_t d, uint32_t tokens, uint32_t kernel,
                      float scale) {
    if (batch == 0 || h == 0 || hk == 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: batch, n_heads and n_kv_heads must be > 0", op);
    if (h % hk != 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: n_heads (%u) must be divisible by n_kv_heads (%u)", op, h, hk);
    if (d != 64 && d != 128 && d != 256) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: head_dim must be 64, 128 or 256, got %u", op, d);
    if (h / hk > 128) SEQ_FAIL(TA_ERR_UNSUPPORTED, "%s: more than 128 query heads per KV head", op);
    if (batch > 65535 || hk > 65535 || tokens > kMostKeys || static_cast<uint64_t>(tokens) * h > static_cast<uint64_t>(INT_MAX))
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "%s: sizes exceed the kernels' index range", op);
    if (kernel > TA_KERNEL_WARP_MMA) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: kernel must be 0 (auto), 1, 2 or 3, got %u", op, kernel);
    if (!std::isfinite(scale)) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: scale is not finite", op);
    return TA_OK;
}

// Contiguous strides where the caller gave 0.
[[maybe_unused]] void row_strides(uint64_t h, uint64_t d, uint64_t *token, uint64_t *head) {
    if (*head == 0) *head = d;
    if (*token == 0) *token = h * d;
}
[[maybe_unused]] void cache_strides(uint64_t hk, uint64_t ps, uint64_t d, uint64_t *page, uint64_t *head, uint64_t *token) {
    if (*token == 0) *token = d;
    if (*head == 0) *head = ps * d;
    if (*page == 0) *page = hk * ps * d;
}

// SMs of the current device, asked once a device (0: none visible).
int device_sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
    else if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (dev < 0 || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// cuTensorMapEncodeTiled of the driver, looked up once; nullptr when it has none.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) == cudaSuccess &&
                        found == cudaDriverEntryPointSuccess;
        if (!ok) cudaGetLastError();
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn) : nullptr;
    }();
    return encode;
}

// The tensor-core kernel counts the key tiles of a request and KV head in 32 bits
// (`rows` tokens of it, `keys` a token sees on average; a part tile at either end).
[[maybe_unused]] ta_status check_work(const char *op, uint32_t g, uint32_t d, uint64_t rows, uint64_t keys) {
    const uint64_t tpt = static_cast<uint64_t>(seq_tc_rows(static_cast<int>(d))) / g;
    if ((rows / tpt + 1) * ((keys + tpt) / kSeqTcTileKeys + 2 + kSeqTcUnitCost) > static_cast<uint64_t>(INT_MAX))
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "%s: tokens x keys of a request exceed the kernel's index range", op);
    return TA_OK;
}

bool encode_16bit(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *m, const SeqArgs &a, const void *ptr, int rank,
                  const cuuint64_t *dims, const cuuint64_t *str, const cuuint32_t *box) {
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return encode(m, a.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                  const_cast<void *>(ptr), dims, str, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of Q: {D, H, T}, a unit's tokens x the g heads of a KV head at once.
bool q_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *m, const SeqArgs &a) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.D), static_cast<cuuint64_t>(a.H), static_cast<cuuint64_t>(a.T)};
    const cuuint64_t str[2] = {static_cast<cuuint64_t>(a.q_sh) * 2, static_cast<cuuint64_t>(a.q_st) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.g), static_cast<cuuint32_t>(seq_tc_rows(a.D) / a.g)};
    return encode_16bit(encode, m, a, a.q, 3, dims, str, box);
}

constexpr uint64_t kStatusBytes = 256;

}  // namespace
}  // namespace ta
