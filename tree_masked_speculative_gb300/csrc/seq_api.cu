// C ABI of the batched serving operators: argument checks (all before any
// launch, overflow-checked), workspace sizes and kernel choice.
#include <cudaTypedefs.h>

#include <atomic>
#include <climits>
#include <cmath>

#include "seq_internal.cuh"
#include "tree_attn.h"

#define TA_EXPORT extern "C" __attribute__((visibility("default")))

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

ta_status check_16bit(const char *op, const char *name, const ta_buf &b) {
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
void row_strides(uint64_t h, uint64_t d, uint64_t *token, uint64_t *head) {
    if (*head == 0) *head = d;
    if (*token == 0) *token = h * d;
}
void cache_strides(uint64_t hk, uint64_t ps, uint64_t d, uint64_t *page, uint64_t *head, uint64_t *token) {
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

constexpr uint64_t kStatusBytes = 256;

int seq_family(uint32_t d, uint32_t kernel, uint64_t rows, uint64_t units, float scale);
int paged_family(const ta_paged_params *p);

// The tensor-core kernel counts the key tiles of a request and KV head in 32 bits
// (`rows` tokens of it, `keys` a token sees on average; a part tile at either end).
ta_status check_work(const char *op, uint32_t g, uint32_t d, uint64_t rows, uint64_t keys) {
    const uint64_t tpt = static_cast<uint64_t>(seq_tc_rows(static_cast<int>(d))) / g;
    if ((rows / tpt + 1) * ((keys + tpt) / kSeqTcTileKeys + 2 + kSeqTcUnitCost) > static_cast<uint64_t>(INT_MAX))
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "%s: tokens x keys of a request exceed the kernel's index range", op);
    return TA_OK;
}

ta_status check_paged(const ta_paged_params *p) {
    if (p == nullptr) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_attn: params is NULL");
    SEQ_TRY(check_heads("paged_attn", p->batch, p->n_heads, p->n_kv_heads, p->head_dim, p->tokens, p->kernel, p->scale));
    if (p->max_q_len == 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_attn: max_q_len must be > 0");
    if (!page_size_ok(p->page_size))
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_attn: page_size must be 16, 32, 64, 128 or 256, got %u", p->page_size);
    if (p->n_pages == 0 || p->max_pages == 0)
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_attn: n_pages and max_pages must be > 0");
    if (p->window > static_cast<uint32_t>(INT_MAX) || p->max_q_len > static_cast<uint32_t>(INT_MAX) ||
        p->n_pages > static_cast<uint32_t>(INT_MAX) ||
        static_cast<uint64_t>(p->max_pages) * p->page_size > kMostKeys)
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "paged_attn: sizes exceed the kernels' index range");
    const uint64_t g = p->n_heads / p->n_kv_heads, keys = static_cast<uint64_t>(p->max_pages) * p->page_size;
    if (paged_family(p) == TA_KERNEL_TENSOR_CORES)
        SEQ_TRY(check_work("paged_attn", static_cast<uint32_t>(g), p->head_dim, p->max_q_len < p->tokens ? p->max_q_len : p->tokens,
                           p->window && p->window < keys ? p->window : keys));
    return TA_OK;
}

ta_status check_prompt(const ta_prompt_params *p) {
    if (p == nullptr) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "prompt_attn: params is NULL");
    SEQ_TRY(check_heads("prompt_attn", p->batch, p->n_heads, p->n_kv_heads, p->head_dim, p->tokens, p->kernel, p->scale));
    if (p->window > static_cast<uint32_t>(INT_MAX))
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "prompt_attn: sizes exceed the kernels' index range");
    const uint64_t keys = p->tokens / 2;               // causal: half of them on average
    if (seq_family(p->head_dim, p->kernel, 0, 0, p->scale) == TA_KERNEL_TENSOR_CORES)
        SEQ_TRY(check_work("prompt_attn", p->n_heads / p->n_kv_heads, p->head_dim, p->tokens,
                           p->window && p->window < keys ? p->window : keys));
    return TA_OK;
}

// Kernel family of a call (rows: most query rows of a request per KV head, 0 for
// prompts; units: requests x KV heads).  Few rows over pages go to the warp-MMA kernel,
// where it is the faster one, unless another family is asked for; the tensor-core kernel
// takes the largest product for the largest logit, so a negative scale goes to the CUDA
// cores, as it does for the warp-MMA one.
int seq_family(uint32_t d, uint32_t kernel, uint64_t rows, uint64_t units, float scale) {
    if (kernel == TA_KERNEL_CUDA_CORES || scale < 0.0f) return TA_KERNEL_CUDA_CORES;
    if (kernel != TA_KERNEL_TENSOR_CORES && rows > 0 && seq_mma_takes(static_cast<int>(d), static_cast<long long>(rows)) &&
        (kernel == TA_KERNEL_WARP_MMA || seq_mma_best(static_cast<int>(d), static_cast<long long>(units))))
        return TA_KERNEL_WARP_MMA;
    return TA_KERNEL_TENSOR_CORES;
}

// Workspace of a call; 0 when no device is visible to size the grid for.
uint64_t seq_workspace(uint32_t d, int family, uint64_t rows) {
    if (family == TA_KERNEL_CUDA_CORES) return kStatusBytes;
    const int sms = device_sm_count();
    if (sms <= 0) return 0;
    return family == TA_KERNEL_WARP_MMA ? seq_mma_workspace(static_cast<int>(d), static_cast<int>(rows), sms)
                                        : seq_tc_workspace(static_cast<int>(d), sms);
}
int paged_family(const ta_paged_params *p) {
    return seq_family(p->head_dim, p->kernel, static_cast<uint64_t>(p->max_q_len) * (p->n_heads / p->n_kv_heads),
                      static_cast<uint64_t>(p->batch) * p->n_kv_heads, p->scale);
}
uint64_t paged_workspace(const ta_paged_params *p) {
    return seq_workspace(p->head_dim, paged_family(p), static_cast<uint64_t>(p->max_q_len) * (p->n_heads / p->n_kv_heads));
}
uint64_t prompt_workspace(const ta_prompt_params *p) {
    return seq_workspace(p->head_dim, seq_family(p->head_dim, p->kernel, 0, 0, p->scale), 0);
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

// Tensor map of K or V: {64, page_size, D / 64, Hk, n_pages} (paged) or {64, T, D / 64, Hk};
// a box holds `slabs` 64-column slabs.
bool kv_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *m, const SeqArgs &a, const void *ptr, long long st,
            long long sh, bool is_v) {
    const bool paged = a.kv_lens != nullptr;
    const cuuint64_t rows = paged ? cuuint64_t(1) << a.page_shift : static_cast<cuuint64_t>(a.T);
    const cuuint64_t slabs = static_cast<cuuint64_t>(a.D) / 64;
    const cuuint64_t dims[5] = {64, rows, slabs, static_cast<cuuint64_t>(a.Hk), static_cast<cuuint64_t>(a.n_pages)};
    const cuuint64_t str[4] = {static_cast<cuuint64_t>(st) * 2, 128, static_cast<cuuint64_t>(sh) * 2, static_cast<cuuint64_t>(a.k_sp) * 2};
    const cuuint32_t box_rows = paged && rows < kSeqTcTileKeys ? static_cast<cuuint32_t>(rows) : kSeqTcTileKeys;
    const cuuint32_t box[5] = {64, box_rows, is_v || box_rows == kSeqTcTileKeys ? static_cast<cuuint32_t>(slabs) : 1, 1, 1};
    return encode_16bit(encode, m, a, ptr, paged ? 5 : 4, dims, str, box);
}

ta_status run_seq(const char *op, const SeqArgs &a, int family, void *ws, cudaStream_t s, uint32_t polls = kSeqWaitPolls) {
    cudaError_t e;
    if (family == TA_KERNEL_CUDA_CORES) {
        e = launch_seq_fma(a, s);
    } else if (family == TA_KERNEL_WARP_MMA) {
        e = launch_seq_mma(a, ws, device_sm_count(), s);
    } else {
        SeqTcPlan pl;
        pl.G = device_sm_count();
        pl.polls = polls;
        pl.ws = ws;
        const auto encode = tensor_map_encoder();
        if (encode == nullptr) SEQ_FAIL(TA_ERR_CUDA, "%s: cuTensorMapEncodeTiled is not available", op);
        if (!q_map(encode, &pl.q, a) || !kv_map(encode, &pl.k, a, a.k, a.k_st, a.k_sh, false) ||
            !kv_map(encode, &pl.v, a, a.v, a.v_st, a.v_sh, true))
            SEQ_FAIL(TA_ERR_CUDA, "%s: TMA descriptor encoding failed", op);
        e = a.D == 64 ? launch_seq_tc64(a, pl, s) : a.D == 128 ? launch_seq_tc128(a, pl, s) : launch_seq_tc256(a, pl, s);
    }
    if (e != cudaSuccess) SEQ_FAIL(TA_ERR_CUDA, "%s: launch: %s", op, cudaGetErrorString(e));
    return TA_OK;
}

}  // namespace
}  // namespace ta

using namespace ta;

TA_EXPORT ta_status paged_plan_build(const ta_plan_params *p, const ta_buf *keep, const ta_buf *fresh, const ta_buf *held,
                                     const ta_buf *table, const ta_buf *stack, const ta_buf *n_free,
                                     const ta_buf *held_out, const ta_buf *n_free_out, const ta_buf *cu,
                                     const ta_buf *kv_lens, const ta_buf *slot_map, const ta_buf *positions,
                                     const ta_buf *status, void *stream) {
    const char *op = "paged_plan";
    if (p == nullptr) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_plan: params is NULL");
    if (p->reserved != 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_plan: reserved must be 0");
    if (p->batch == 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_plan: batch must be > 0");
    if (!page_size_ok(p->page_size))
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_plan: page_size must be 16, 32, 64, 128 or 256, got %u", p->page_size);
    if (p->max_pages == 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_plan: max_pages must be > 0");
    if (p->batch > static_cast<uint32_t>(kPlanMaxBatch))
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "paged_plan: batch > %d is not implemented", kPlanMaxBatch);
    if (static_cast<uint64_t>(p->max_pages) * p->page_size > static_cast<uint64_t>(INT_MAX) ||
        static_cast<uint64_t>(p->batch) * p->max_pages > static_cast<uint64_t>(INT_MAX) / 2 ||
        p->capacity > static_cast<uint32_t>(INT_MAX) / 2 || p->max_tokens > static_cast<uint32_t>(INT_MAX) / 2)
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "paged_plan: sizes exceed the kernel's index range");
    const uint64_t b4 = static_cast<uint64_t>(p->batch) * 4;
    SEQ_TRY(check(op, "keep", of(keep), TA_I32, b4, 4));
    SEQ_TRY(check(op, "fresh", of(fresh), TA_I32, b4, 4));
    SEQ_TRY(check(op, "held", of(held), TA_I32, b4, 4));
    SEQ_TRY(check(op, "table", of(table), TA_I32, b4 * p->max_pages, 4));
    if (p->capacity > 0) SEQ_TRY(check(op, "stack", of(stack), TA_I32, static_cast<uint64_t>(p->capacity) * 4, 4));
    SEQ_TRY(check(op, "n_free", of(n_free), TA_I32, 4, 4));
    SEQ_TRY(check(op, "held_out", of(held_out), TA_I32, b4, 4));
    SEQ_TRY(check(op, "n_free_out", of(n_free_out), TA_I32, 4, 4));
    SEQ_TRY(check(op, "cu", of(cu), TA_I32, b4 + 4, 4));
    SEQ_TRY(check(op, "kv_lens", of(kv_lens), TA_I32, b4, 4));
    if (p->max_tokens > 0) {
        SEQ_TRY(check(op, "slot_map", of(slot_map), TA_I64, static_cast<uint64_t>(p->max_tokens) * 8, 8));
        SEQ_TRY(check(op, "positions", of(positions), TA_I32, static_cast<uint64_t>(p->max_tokens) * 4, 4));
    }
    SEQ_TRY(check(op, "status", of(status), TA_I32, 4, 4));
    PlanArgs a;
    a.keep = static_cast<const int32_t *>(keep->ptr);
    a.fresh = static_cast<const int32_t *>(fresh->ptr);
    a.held = static_cast<const int32_t *>(held->ptr);
    a.table = static_cast<int32_t *>(table->ptr);
    a.stack = static_cast<int32_t *>(of(stack).ptr);
    a.n_free = static_cast<const int32_t *>(n_free->ptr);
    a.held_out = static_cast<int32_t *>(held_out->ptr);
    a.n_free_out = static_cast<int32_t *>(n_free_out->ptr);
    a.cu = static_cast<int32_t *>(cu->ptr);
    a.lens = static_cast<int32_t *>(kv_lens->ptr);
    a.slot = static_cast<int64_t *>(of(slot_map).ptr);
    a.pos = static_cast<int32_t *>(of(positions).ptr);
    a.status = static_cast<int32_t *>(status->ptr);
    a.B = static_cast<int>(p->batch);
    a.max_pages = static_cast<int>(p->max_pages);
    a.capacity = static_cast<int>(p->capacity);
    a.max_tokens = static_cast<int>(p->max_tokens);
    a.page_shift = log2_of(p->page_size);
    const cudaError_t e = launch_paged_plan(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) SEQ_FAIL(TA_ERR_CUDA, "paged_plan: launch: %s", cudaGetErrorString(e));
    return TA_OK;
}

TA_EXPORT ta_status paged_kv_append(const ta_append_params *pp, const ta_buf *k_new, const ta_buf *v_new,
                                    const ta_buf *k_cache, const ta_buf *v_cache, const ta_buf *slot_map, void *stream) {
    const char *op = "paged_append";
    if (pp == nullptr) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_append: params is NULL");
    ta_append_params p = *pp;
    if (p.reserved != 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_append: reserved must be 0");
    if (p.n_kv_heads == 0 || p.n_pages == 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_append: n_kv_heads and n_pages must be > 0");
    if (p.head_dim != 64 && p.head_dim != 128 && p.head_dim != 256)
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_append: head_dim must be 64, 128 or 256, got %u", p.head_dim);
    if (!page_size_ok(p.page_size))
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_append: page_size must be 16, 32, 64, 128 or 256, got %u", p.page_size);
    if (p.n_kv_heads > 65535 || p.tokens > static_cast<uint32_t>(INT_MAX) || p.n_pages > static_cast<uint32_t>(INT_MAX))
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "paged_append: sizes exceed the kernel's index range");
    row_strides(p.n_kv_heads, p.head_dim, &p.k_token_stride, &p.k_head_stride);
    row_strides(p.n_kv_heads, p.head_dim, &p.v_token_stride, &p.v_head_stride);
    cache_strides(p.n_kv_heads, p.page_size, p.head_dim, &p.page_stride, &p.head_stride, &p.token_stride);
    SEQ_TRY(check_stride(op, "k_token_stride", p.k_token_stride));
    SEQ_TRY(check_stride(op, "k_head_stride", p.k_head_stride));
    SEQ_TRY(check_stride(op, "v_token_stride", p.v_token_stride));
    SEQ_TRY(check_stride(op, "v_head_stride", p.v_head_stride));
    SEQ_TRY(check_stride(op, "page_stride", p.page_stride));
    SEQ_TRY(check_stride(op, "head_stride", p.head_stride));
    SEQ_TRY(check_stride(op, "token_stride", p.token_stride));
    if (p.tokens == 0) return TA_OK;
    SEQ_TRY(check_16bit(op, "k_new", of(k_new)));
    const int type = k_new->dtype;
    uint64_t nk, nv, nc;
    const Axis kax[2] = {{p.tokens, p.k_token_stride}, {p.n_kv_heads, p.k_head_stride}};
    const Axis vax[2] = {{p.tokens, p.v_token_stride}, {p.n_kv_heads, p.v_head_stride}};
    const Axis cax[3] = {{p.n_pages, p.page_stride}, {p.n_kv_heads, p.head_stride}, {p.page_size, p.token_stride}};
    if (!extent(kax, p.head_dim, &nk) || !extent(vax, p.head_dim, &nv) || !extent(cax, p.head_dim, &nc))
        SEQ_FAIL(TA_ERR_OVERFLOW, "paged_append: sizes overflow");
    SEQ_TRY(check(op, "k_new", *k_new, type, nk, 16));
    SEQ_TRY(check(op, "v_new", of(v_new), type, nv, 16));
    SEQ_TRY(check(op, "k_cache", of(k_cache), type, nc, 16));
    SEQ_TRY(check(op, "v_cache", of(v_cache), type, nc, 16));
    SEQ_TRY(check(op, "slot_map", of(slot_map), TA_I64, static_cast<uint64_t>(p.tokens) * 8, 8));
    AppendArgs a;
    a.k_new = k_new->ptr;
    a.v_new = v_new->ptr;
    a.k = k_cache->ptr;
    a.v = v_cache->ptr;
    a.slot = static_cast<const int64_t *>(slot_map->ptr);
    a.T = static_cast<int>(p.tokens);
    a.Hk = static_cast<int>(p.n_kv_heads);
    a.D = static_cast<int>(p.head_dim);
    a.page_shift = log2_of(p.page_size);
    a.n_pages = static_cast<int>(p.n_pages);
    // the kernel counts in 16-byte vectors
    a.kn_st = static_cast<long long>(p.k_token_stride / 8);
    a.kn_sh = static_cast<long long>(p.k_head_stride / 8);
    a.vn_st = static_cast<long long>(p.v_token_stride / 8);
    a.vn_sh = static_cast<long long>(p.v_head_stride / 8);
    a.c_sp = static_cast<long long>(p.page_stride / 8);
    a.c_st = static_cast<long long>(p.token_stride / 8);
    a.c_sh = static_cast<long long>(p.head_stride / 8);
    const cudaError_t e = launch_paged_append(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) SEQ_FAIL(TA_ERR_CUDA, "paged_append: launch: %s", cudaGetErrorString(e));
    return TA_OK;
}

TA_EXPORT size_t paged_attn_workspace_bytes(const ta_paged_params *p) {
    if (check_paged(p) != TA_OK) return SIZE_MAX;
    uint64_t ws = paged_workspace(p);
    if (ws && paged_family(p) == TA_KERNEL_WARP_MMA && p->kernel == TA_KERNEL_AUTO) {
        // the same for every batch, also where a larger one takes the tensor-core kernel
        ta_paged_params most = *p;
        most.batch = 65535;
        const uint64_t other = paged_workspace(&most);
        ws = other > ws ? other : ws;
    }
    if (ws == 0) set_last_error("paged_attn: no CUDA device to size the workspace for");
    return ws ? ws : SIZE_MAX;
}

TA_EXPORT size_t prompt_attn_workspace_bytes(const ta_prompt_params *p) {
    if (check_prompt(p) != TA_OK) return SIZE_MAX;
    const uint64_t ws = prompt_workspace(p);
    if (ws == 0) set_last_error("prompt_attn: no CUDA device to size the workspace for");
    return ws ? ws : SIZE_MAX;
}

// paged_attn_fwd; `polls` bounds the tensor-core kernel's waits (hook: the test entry point, which
// takes that kernel alone).
static ta_status paged_fwd(const ta_paged_params *pp, const ta_buf *q, const ta_buf *k_cache, const ta_buf *v_cache,
                           const ta_buf *table, const ta_buf *cu, const ta_buf *kv_lens, const ta_buf *parents,
                           const ta_buf *tmp, const ta_buf *out, void *stream, uint32_t polls, bool hook) {
    const char *op = "paged_attn";
    SEQ_TRY(check_paged(pp));
    if (hook && paged_family(pp) != TA_KERNEL_TENSOR_CORES)
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "paged_attn: the wait-limit hook is for the tensor-core kernel only");
    ta_paged_params p = *pp;
    const bool tree = !is_absent(parents);
    if (tree && p.window != 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "paged_attn: window must be 0 with parents");
    if (tree && p.max_q_len > static_cast<uint32_t>(kMaxTreeBitsNodes))
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "paged_attn: parents take max_q_len <= %d (got %u)", kMaxTreeBitsNodes, p.max_q_len);
    row_strides(p.n_heads, p.head_dim, &p.q_token_stride, &p.q_head_stride);
    row_strides(p.n_heads, p.head_dim, &p.out_token_stride, &p.out_head_stride);
    cache_strides(p.n_kv_heads, p.page_size, p.head_dim, &p.page_stride, &p.head_stride, &p.token_stride);
    SEQ_TRY(check_stride(op, "q_token_stride", p.q_token_stride));
    SEQ_TRY(check_stride(op, "q_head_stride", p.q_head_stride));
    SEQ_TRY(check_stride(op, "out_token_stride", p.out_token_stride));
    SEQ_TRY(check_stride(op, "out_head_stride", p.out_head_stride));
    SEQ_TRY(check_stride(op, "page_stride", p.page_stride));
    SEQ_TRY(check_stride(op, "head_stride", p.head_stride));
    SEQ_TRY(check_stride(op, "token_stride", p.token_stride));
    if (p.tokens == 0) return TA_OK;
    SEQ_TRY(check_16bit(op, "q", of(q)));
    const int type = q->dtype;
    uint64_t nq, no, nc;
    const Axis qax[2] = {{p.tokens, p.q_token_stride}, {p.n_heads, p.q_head_stride}};
    const Axis oax[2] = {{p.tokens, p.out_token_stride}, {p.n_heads, p.out_head_stride}};
    const Axis cax[3] = {{p.n_pages, p.page_stride}, {p.n_kv_heads, p.head_stride}, {p.page_size, p.token_stride}};
    if (!extent(qax, p.head_dim, &nq) || !extent(oax, p.head_dim, &no) || !extent(cax, p.head_dim, &nc))
        SEQ_FAIL(TA_ERR_OVERFLOW, "paged_attn: sizes overflow");
    const uint64_t ws = paged_workspace(&p);
    SEQ_TRY(check(op, "q", *q, type, nq, 16));
    SEQ_TRY(check(op, "k_cache", of(k_cache), type, nc, 16));
    SEQ_TRY(check(op, "v_cache", of(v_cache), type, nc, 16));
    SEQ_TRY(check(op, "table", of(table), TA_I32, static_cast<uint64_t>(p.batch) * p.max_pages * 4, 4));
    SEQ_TRY(check(op, "cu", of(cu), TA_I32, (static_cast<uint64_t>(p.batch) + 1) * 4, 4));
    SEQ_TRY(check(op, "kv_lens", of(kv_lens), TA_I32, static_cast<uint64_t>(p.batch) * 4, 4));
    if (tree) SEQ_TRY(check(op, "parents", *parents, TA_I32, static_cast<uint64_t>(p.tokens) * 4, 4));
    SEQ_TRY(check(op, "tmp", of(tmp), TA_F32, ws ? ws : kStatusBytes, 16));
    SEQ_TRY(check(op, "out", of(out), type, no, 16));
    SeqArgs a = {};
    a.q = q->ptr;
    a.k = k_cache->ptr;
    a.v = v_cache->ptr;
    a.out = out->ptr;
    a.cu = static_cast<const int32_t *>(cu->ptr);
    a.kv_lens = static_cast<const int32_t *>(kv_lens->ptr);
    a.table = static_cast<const int32_t *>(table->ptr);
    a.parents = tree ? static_cast<const int32_t *>(parents->ptr) : nullptr;
    a.status = static_cast<int32_t *>(tmp->ptr);
    a.B = static_cast<int>(p.batch);
    a.H = static_cast<int>(p.n_heads);
    a.Hk = static_cast<int>(p.n_kv_heads);
    a.g = a.H / a.Hk;
    a.D = static_cast<int>(p.head_dim);
    a.T = static_cast<int>(p.tokens);
    a.max_q = static_cast<int>(p.max_q_len);
    a.window = static_cast<int>(p.window < kMostKeys ? p.window : kMostKeys);     // no request has more keys
    a.page_shift = log2_of(p.page_size);
    a.n_pages = static_cast<int>(p.n_pages);
    a.max_pages = static_cast<int>(p.max_pages);
    a.bf16 = type == TA_BF16;
    a.q_st = static_cast<long long>(p.q_token_stride);
    a.q_sh = static_cast<long long>(p.q_head_stride);
    a.o_st = static_cast<long long>(p.out_token_stride);
    a.o_sh = static_cast<long long>(p.out_head_stride);
    a.k_sp = static_cast<long long>(p.page_stride);
    a.k_st = a.v_st = static_cast<long long>(p.token_stride);
    a.k_sh = a.v_sh = static_cast<long long>(p.head_stride);
    a.scale = p.scale;
    if (ws == 0) SEQ_FAIL(TA_ERR_CUDA, "%s: no CUDA device", op);
    return run_seq(op, a, paged_family(&p), tmp->ptr, static_cast<cudaStream_t>(stream), polls);
}

TA_EXPORT ta_status paged_attn_fwd(const ta_paged_params *p, const ta_buf *q, const ta_buf *k_cache,
                                   const ta_buf *v_cache, const ta_buf *table, const ta_buf *cu, const ta_buf *kv_lens,
                                   const ta_buf *parents, const ta_buf *tmp, const ta_buf *out, void *stream) {
    return paged_fwd(p, q, k_cache, v_cache, table, cu, kv_lens, parents, tmp, out, stream, kSeqWaitPolls, false);
}

TA_EXPORT ta_status ta_test_paged_attn_fwd_wait_limit(uint32_t wait_polls, const ta_paged_params *p, const ta_buf *q,
                                                      const ta_buf *k_cache, const ta_buf *v_cache, const ta_buf *table,
                                                      const ta_buf *cu, const ta_buf *kv_lens, const ta_buf *parents,
                                                      const ta_buf *tmp, const ta_buf *out, void *stream) {
    return paged_fwd(p, q, k_cache, v_cache, table, cu, kv_lens, parents, tmp, out, stream, wait_polls, true);
}

TA_EXPORT ta_status prompt_attn_fwd(const ta_prompt_params *pp, const ta_buf *q, const ta_buf *k, const ta_buf *v,
                                    const ta_buf *cu, const ta_buf *tmp, const ta_buf *out, void *stream) {
    const char *op = "prompt_attn";
    SEQ_TRY(check_prompt(pp));
    ta_prompt_params p = *pp;
    row_strides(p.n_heads, p.head_dim, &p.q_token_stride, &p.q_head_stride);
    row_strides(p.n_heads, p.head_dim, &p.out_token_stride, &p.out_head_stride);
    row_strides(p.n_kv_heads, p.head_dim, &p.k_token_stride, &p.k_head_stride);
    row_strides(p.n_kv_heads, p.head_dim, &p.v_token_stride, &p.v_head_stride);
    SEQ_TRY(check_stride(op, "q_token_stride", p.q_token_stride));
    SEQ_TRY(check_stride(op, "q_head_stride", p.q_head_stride));
    SEQ_TRY(check_stride(op, "out_token_stride", p.out_token_stride));
    SEQ_TRY(check_stride(op, "out_head_stride", p.out_head_stride));
    SEQ_TRY(check_stride(op, "k_token_stride", p.k_token_stride));
    SEQ_TRY(check_stride(op, "k_head_stride", p.k_head_stride));
    SEQ_TRY(check_stride(op, "v_token_stride", p.v_token_stride));
    SEQ_TRY(check_stride(op, "v_head_stride", p.v_head_stride));
    if (p.tokens == 0) return TA_OK;
    SEQ_TRY(check_16bit(op, "q", of(q)));
    const int type = q->dtype;
    uint64_t nq, no, nk, nv;
    const Axis qax[2] = {{p.tokens, p.q_token_stride}, {p.n_heads, p.q_head_stride}};
    const Axis oax[2] = {{p.tokens, p.out_token_stride}, {p.n_heads, p.out_head_stride}};
    const Axis kax[2] = {{p.tokens, p.k_token_stride}, {p.n_kv_heads, p.k_head_stride}};
    const Axis vax[2] = {{p.tokens, p.v_token_stride}, {p.n_kv_heads, p.v_head_stride}};
    if (!extent(qax, p.head_dim, &nq) || !extent(oax, p.head_dim, &no) || !extent(kax, p.head_dim, &nk) ||
        !extent(vax, p.head_dim, &nv))
        SEQ_FAIL(TA_ERR_OVERFLOW, "prompt_attn: sizes overflow");
    const uint64_t ws = prompt_workspace(&p);
    SEQ_TRY(check(op, "q", *q, type, nq, 16));
    SEQ_TRY(check(op, "k", of(k), type, nk, 16));
    SEQ_TRY(check(op, "v", of(v), type, nv, 16));
    SEQ_TRY(check(op, "cu", of(cu), TA_I32, (static_cast<uint64_t>(p.batch) + 1) * 4, 4));
    SEQ_TRY(check(op, "tmp", of(tmp), TA_F32, ws ? ws : kStatusBytes, 16));
    SEQ_TRY(check(op, "out", of(out), type, no, 16));
    SeqArgs a = {};
    a.q = q->ptr;
    a.k = k->ptr;
    a.v = v->ptr;
    a.out = out->ptr;
    a.cu = static_cast<const int32_t *>(cu->ptr);
    a.status = static_cast<int32_t *>(tmp->ptr);
    a.B = static_cast<int>(p.batch);
    a.H = static_cast<int>(p.n_heads);
    a.Hk = static_cast<int>(p.n_kv_heads);
    a.g = a.H / a.Hk;
    a.D = static_cast<int>(p.head_dim);
    a.T = a.max_q = static_cast<int>(p.tokens);
    a.window = static_cast<int>(p.window < kMostKeys ? p.window : kMostKeys);     // no request has more keys
    a.bf16 = type == TA_BF16;
    a.q_st = static_cast<long long>(p.q_token_stride);
    a.q_sh = static_cast<long long>(p.q_head_stride);
    a.o_st = static_cast<long long>(p.out_token_stride);
    a.o_sh = static_cast<long long>(p.out_head_stride);
    a.k_st = static_cast<long long>(p.k_token_stride);
    a.k_sh = static_cast<long long>(p.k_head_stride);
    a.v_st = static_cast<long long>(p.v_token_stride);
    a.v_sh = static_cast<long long>(p.v_head_stride);
    a.scale = p.scale;
    if (ws == 0) SEQ_FAIL(TA_ERR_CUDA, "%s: no CUDA device", op);
    return run_seq(op, a, seq_family(p.head_dim, p.kernel, 0, 0, p.scale), tmp->ptr, static_cast<cudaStream_t>(stream));
}
