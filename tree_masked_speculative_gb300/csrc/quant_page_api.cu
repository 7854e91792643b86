// C ABI of the rotary append and of the 4-bit pages (append, read, attention): argument
// checks (all before any launch, overflow-checked), workspace sizes and kernel choice.
#include "quant_page.cuh"
#include "seq_checks.cuh"

#define TA_EXPORT extern "C" __attribute__((visibility("default")))

namespace ta {
namespace {

ta_status check_rows(const char *op, uint32_t tokens, uint32_t h, uint32_t hk, uint32_t d, uint32_t ps, uint32_t n_pages) {
    if (hk == 0 || n_pages == 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: n_kv_heads and n_pages must be > 0", op);
    if (d != 64 && d != 128 && d != 256) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: head_dim must be 64, 128 or 256, got %u", op, d);
    if (!page_size_ok(ps)) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: page_size must be 16, 32, 64, 128 or 256, got %u", op, ps);
    // (a launch takes a thread per 16 elements of at most one head)
    if (h > 65535 || hk > 65535 || tokens > kMostKeys || n_pages > static_cast<uint32_t>(INT_MAX) ||
        static_cast<uint64_t>(tokens) * (h + 2ull * hk) > static_cast<uint64_t>(INT_MAX))
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "%s: sizes exceed the kernels' index range", op);
    return TA_OK;
}

ta_status check_rotary(const char *op, uint32_t r, uint32_t d, uint32_t interleaved, uint32_t max_positions) {
    if (r % 16 != 0 || r > d) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: rotary_dim must be a multiple of 16 up to head_dim, got %u", op, r);
    if (interleaved > 1) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: interleaved must be 0 or 1, got %u", op, interleaved);
    if (max_positions > static_cast<uint32_t>(INT_MAX)) SEQ_FAIL(TA_ERR_UNSUPPORTED, "%s: max_positions exceeds the kernels' index range", op);
    return TA_OK;
}

// Strides of 4-bit pages: 0 replaced, codes in multiples of 16 bytes, affine in those of its loads.
struct PageStrides {
    uint64_t cp, ch, ct, ap, ah, at;
};
ta_status page_strides(const char *op, uint64_t hk, uint64_t ps, uint64_t d, uint64_t group, PageStrides *s) {
    if (group != 32 && group != 64)
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: group_size must be 32 or 64, got %llu", op, static_cast<unsigned long long>(group));
    cache_strides(hk, ps, d / 8, &s->cp, &s->ch, &s->ct);
    cache_strides(hk, ps, 2 * (d / group), &s->ap, &s->ah, &s->at);
    const uint64_t av = 2 * (d / group) < 8 ? 2 * (d / group) : 8;
    if (s->cp % 4 || s->ch % 4 || s->ct % 4)
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: strides of the codes must be multiples of 4 words", op);
    if (s->ap % av || s->ah % av || s->at % av)
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: strides of the affine must be multiples of %llu elements", op, static_cast<unsigned long long>(av));
    for (const uint64_t x : {s->cp, s->ch, s->ct, s->ap, s->ah, s->at})
        if (x >= (uint64_t(1) << 30)) SEQ_FAIL(TA_ERR_UNSUPPORTED, "%s: a cache stride exceeds 2^30 elements", op);
    return TA_OK;
}
// Buffers of 4-bit pages.
ta_status page_buffers(const char *op, const PageStrides &s, uint64_t n_pages, uint64_t hk, uint64_t ps, uint64_t d, uint64_t group, int type,
                       const ta_buf *kc, const ta_buf *ka, const ta_buf *vc, const ta_buf *va, QuantCache *c) {
    uint64_t nc, na;
    const Axis cax[3] = {{n_pages, s.cp}, {hk, s.ch}, {ps, s.ct}}, aax[3] = {{n_pages, s.ap}, {hk, s.ah}, {ps, s.at}};
    if (!extent(cax, d / 8, &nc) || __builtin_mul_overflow(nc, uint64_t(2), &nc) || nc > static_cast<uint64_t>(LLONG_MAX) ||
        !extent(aax, 2 * (d / group), &na))
        SEQ_FAIL(TA_ERR_OVERFLOW, "%s: sizes overflow", op);
    SEQ_TRY(check(op, "k_codes", of(kc), TA_U32, nc, 16));
    SEQ_TRY(check(op, "k_affine", of(ka), type, na, 16));
    SEQ_TRY(check(op, "v_codes", of(vc), TA_U32, nc, 16));
    SEQ_TRY(check(op, "v_affine", of(va), type, na, 16));
    c->kc = static_cast<uint32_t *>(kc->ptr);
    c->vc = static_cast<uint32_t *>(vc->ptr);
    c->ka = ka->ptr;
    c->va = va->ptr;
    c->c_sp = static_cast<uint32_t>(4 * s.cp);
    c->c_sh = static_cast<uint32_t>(4 * s.ch);
    c->c_st = static_cast<uint32_t>(4 * s.ct);
    c->a_sp = static_cast<uint32_t>(2 * s.ap);
    c->a_sh = static_cast<uint32_t>(2 * s.ah);
    c->a_st = static_cast<uint32_t>(2 * s.at);
    return TA_OK;
}

// What both appends share: checks of q, k_new, v_new, q_out, slots, positions and table, and their
// arguments (R = 0: nothing is turned).  `P`: either params struct.
template <typename P>
ta_status new_rows(const char *op, P *p, const ta_buf *q, const ta_buf *k_new, const ta_buf *v_new, const ta_buf *slot_map,
                   const ta_buf *positions, const ta_buf *table, const ta_buf *q_out, RotaryArgs *a) {
    row_strides(p->n_heads, p->head_dim, &p->q_token_stride, &p->q_head_stride);
    row_strides(p->n_heads, p->head_dim, &p->q_out_token_stride, &p->q_out_head_stride);
    row_strides(p->n_kv_heads, p->head_dim, &p->k_token_stride, &p->k_head_stride);
    row_strides(p->n_kv_heads, p->head_dim, &p->v_token_stride, &p->v_head_stride);
    SEQ_TRY(check_stride(op, "q_token_stride", p->q_token_stride));
    SEQ_TRY(check_stride(op, "q_head_stride", p->q_head_stride));
    SEQ_TRY(check_stride(op, "q_out_token_stride", p->q_out_token_stride));
    SEQ_TRY(check_stride(op, "q_out_head_stride", p->q_out_head_stride));
    SEQ_TRY(check_stride(op, "k_token_stride", p->k_token_stride));
    SEQ_TRY(check_stride(op, "k_head_stride", p->k_head_stride));
    SEQ_TRY(check_stride(op, "v_token_stride", p->v_token_stride));
    SEQ_TRY(check_stride(op, "v_head_stride", p->v_head_stride));
    if (p->tokens == 0) return TA_OK;
    SEQ_TRY(check_16bit(op, "k_new", of(k_new)));
    const int type = k_new->dtype;
    uint64_t nk, nv;
    const Axis kax[2] = {{p->tokens, p->k_token_stride}, {p->n_kv_heads, p->k_head_stride}};
    const Axis vax[2] = {{p->tokens, p->v_token_stride}, {p->n_kv_heads, p->v_head_stride}};
    if (!extent(kax, p->head_dim, &nk) || !extent(vax, p->head_dim, &nv)) SEQ_FAIL(TA_ERR_OVERFLOW, "%s: sizes overflow", op);
    if (p->n_heads > 0) {
        uint64_t nq, no;
        const Axis qax[2] = {{p->tokens, p->q_token_stride}, {p->n_heads, p->q_head_stride}};
        const Axis oax[2] = {{p->tokens, p->q_out_token_stride}, {p->n_heads, p->q_out_head_stride}};
        if (!extent(qax, p->head_dim, &nq) || !extent(oax, p->head_dim, &no)) SEQ_FAIL(TA_ERR_OVERFLOW, "%s: sizes overflow", op);
        SEQ_TRY(check(op, "q", of(q), type, nq, 16));
        SEQ_TRY(check(op, "q_out", of(q_out), type, no, 16));
        if (q->ptr == q_out->ptr && (p->q_token_stride != p->q_out_token_stride || p->q_head_stride != p->q_out_head_stride))
            SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: q_out in the place of q must have its strides", op);
    } else if (!is_absent(q) || !is_absent(q_out)) {
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: q and q_out must be absent with n_heads 0", op);
    }
    SEQ_TRY(check(op, "k_new", *k_new, type, nk, 16));
    SEQ_TRY(check(op, "v_new", of(v_new), type, nv, 16));
    SEQ_TRY(check(op, "slot_map", of(slot_map), TA_I64, static_cast<uint64_t>(p->tokens) * 8, 8));
    *a = {};
    if (p->rotary_dim > 0) {
        SEQ_TRY(check(op, "positions", of(positions), TA_I32, static_cast<uint64_t>(p->tokens) * 4, 4));
        if (p->max_positions > 0)
            SEQ_TRY(check(op, "table", of(table), TA_F32, static_cast<uint64_t>(p->max_positions) * p->rotary_dim * 4, 16));
        a->pos = static_cast<const int32_t *>(positions->ptr);
        a->table = static_cast<const float *>(of(table).ptr);
    }
    a->q = of(q).ptr;
    a->q_out = of(q_out).ptr;
    a->k_new = k_new->ptr;
    a->v_new = v_new->ptr;
    a->slot = static_cast<const int64_t *>(slot_map->ptr);
    a->T = static_cast<int>(p->tokens);
    a->H = static_cast<int>(p->n_heads);
    a->Hk = static_cast<int>(p->n_kv_heads);
    a->D = static_cast<int>(p->head_dim);
    a->R = static_cast<int>(p->rotary_dim);
    a->max_pos = static_cast<int>(p->max_positions);
    a->interleaved = static_cast<int>(p->interleaved);
    a->page_shift = log2_of(p->page_size);
    a->n_pages = static_cast<int>(p->n_pages);
    a->bf16 = type == TA_BF16;
    // the kernels count in 16-byte vectors
    a->q_st = static_cast<long long>(p->q_token_stride / 8);
    a->q_sh = static_cast<long long>(p->q_head_stride / 8);
    a->qo_st = static_cast<long long>(p->q_out_token_stride / 8);
    a->qo_sh = static_cast<long long>(p->q_out_head_stride / 8);
    a->k_st = static_cast<long long>(p->k_token_stride / 8);
    a->k_sh = static_cast<long long>(p->k_head_stride / 8);
    a->v_st = static_cast<long long>(p->v_token_stride / 8);
    a->v_sh = static_cast<long long>(p->v_head_stride / 8);
    return TA_OK;
}

uint64_t quant_rows(const ta_paged_quant_params *p) { return static_cast<uint64_t>(p->max_q_len) * (p->n_heads / p->n_kv_heads); }

// Kernel family of a call: few rows go to the warp-MMA kernel (measured at quant_mma_rows) unless the tensor-core kernel is
// asked for.  Both take the largest product for the largest logit, so a negative scale goes to the CUDA cores.
int quant_family(const ta_paged_quant_params *p) {
    if (p->kernel == TA_KERNEL_CUDA_CORES || p->scale < 0.0f) return TA_KERNEL_CUDA_CORES;
    return p->kernel != TA_KERNEL_TENSOR_CORES && quant_rows(p) <= static_cast<uint64_t>(quant_mma_rows(static_cast<int>(p->head_dim))) ? TA_KERNEL_WARP_MMA : TA_KERNEL_TENSOR_CORES;
}

// Workspace of a call; 0 when no device is visible to size the grid for.
uint64_t quant_workspace(const ta_paged_quant_params *p) {
    const int family = quant_family(p), rows = static_cast<int>(quant_rows(p));
    if (family == TA_KERNEL_CUDA_CORES) return kStatusBytes;
    const int sms = device_sm_count();
    if (sms <= 0) return 0;
    if (family == TA_KERNEL_TENSOR_CORES) return seq_tc_workspace(static_cast<int>(p->head_dim), sms);
    return p->head_dim == 64 ? seq_quant_mma_workspace64(rows, sms)
                             : p->head_dim == 128 ? seq_quant_mma_workspace128(rows, sms) : seq_quant_mma_workspace256(rows, sms);
}

ta_status run_quant(const char *op, const SeqQuantArgs &a, int family, void *ws, cudaStream_t s, uint32_t polls) {
    const int sms = device_sm_count();
    cudaError_t e;
    if (family == TA_KERNEL_CUDA_CORES) {
        e = launch_seq_quant_fma(a, s);
    } else if (family == TA_KERNEL_WARP_MMA) {
        e = a.s.D == 64 ? launch_seq_quant_mma64(a, ws, sms, s)
                        : a.s.D == 128 ? launch_seq_quant_mma128(a, ws, sms, s) : launch_seq_quant_mma256(a, ws, sms, s);
    } else {
        SeqTcPlan pl = {};
        pl.G = sms;
        pl.polls = polls;
        pl.ws = ws;
        const auto encode = tensor_map_encoder();
        if (encode == nullptr) SEQ_FAIL(TA_ERR_CUDA, "%s: cuTensorMapEncodeTiled is not available", op);
        if (!q_map(encode, &pl.q, a.s)) SEQ_FAIL(TA_ERR_CUDA, "%s: TMA descriptor encoding failed", op);
        e = a.s.D == 64 ? launch_seq_quant_tc64(a, pl, s) : a.s.D == 128 ? launch_seq_quant_tc128(a, pl, s) : launch_seq_quant_tc256(a, pl, s);
    }
    if (e != cudaSuccess) SEQ_FAIL(TA_ERR_CUDA, "%s: launch: %s", op, cudaGetErrorString(e));
    return TA_OK;
}

ta_status check_quant_attn(const ta_paged_quant_params *p) {
    const char *op = "paged_quant_attn";
    if (p == nullptr) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: params is NULL", op);
    if (p->reserved != 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: reserved must be 0", op);
    SEQ_TRY(check_heads(op, p->batch, p->n_heads, p->n_kv_heads, p->head_dim, p->tokens, p->kernel, p->scale));
    if (p->group_size != 32 && p->group_size != 64)
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: group_size must be 32 or 64, got %u", op, p->group_size);
    if (p->max_q_len == 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: max_q_len must be > 0", op);
    if (!page_size_ok(p->page_size))
        SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: page_size must be 16, 32, 64, 128 or 256, got %u", op, p->page_size);
    if (p->n_pages == 0 || p->max_pages == 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: n_pages and max_pages must be > 0", op);
    if (p->window > static_cast<uint32_t>(INT_MAX) || p->max_q_len > static_cast<uint32_t>(INT_MAX) ||
        p->n_pages > static_cast<uint32_t>(INT_MAX) || static_cast<uint64_t>(p->max_pages) * p->page_size > kMostKeys)
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "%s: sizes exceed the kernels' index range", op);
    const uint64_t keys = static_cast<uint64_t>(p->max_pages) * p->page_size;
    if (quant_family(p) == TA_KERNEL_TENSOR_CORES)
        SEQ_TRY(check_work(op, p->n_heads / p->n_kv_heads, p->head_dim, p->max_q_len < p->tokens ? p->max_q_len : p->tokens,
                           p->window && p->window < keys ? p->window : keys));
    return TA_OK;
}

}  // namespace
}  // namespace ta

using namespace ta;

TA_EXPORT ta_status paged_rotary_append(const ta_rotary_append_params *pp, const ta_buf *q, const ta_buf *k_new, const ta_buf *v_new,
                                        const ta_buf *slot_map, const ta_buf *positions, const ta_buf *table, const ta_buf *q_out,
                                        const ta_buf *k_cache, const ta_buf *v_cache, void *stream) {
    const char *op = "paged_rotary_append";
    if (pp == nullptr) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: params is NULL", op);
    ta_rotary_append_params p = *pp;
    if (p.reserved != 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: reserved must be 0", op);
    SEQ_TRY(check_rows(op, p.tokens, p.n_heads, p.n_kv_heads, p.head_dim, p.page_size, p.n_pages));
    if (p.rotary_dim == 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: rotary_dim must be > 0 (paged_kv_append turns nothing)", op);
    SEQ_TRY(check_rotary(op, p.rotary_dim, p.head_dim, p.interleaved, p.max_positions));
    cache_strides(p.n_kv_heads, p.page_size, p.head_dim, &p.page_stride, &p.head_stride, &p.token_stride);
    SEQ_TRY(check_stride(op, "page_stride", p.page_stride));
    SEQ_TRY(check_stride(op, "head_stride", p.head_stride));
    SEQ_TRY(check_stride(op, "token_stride", p.token_stride));
    RotaryAppendArgs a;
    SEQ_TRY(new_rows(op, &p, q, k_new, v_new, slot_map, positions, table, q_out, &a.r));
    if (p.tokens == 0) return TA_OK;
    uint64_t nc;
    const Axis cax[3] = {{p.n_pages, p.page_stride}, {p.n_kv_heads, p.head_stride}, {p.page_size, p.token_stride}};
    if (!extent(cax, p.head_dim, &nc)) SEQ_FAIL(TA_ERR_OVERFLOW, "%s: sizes overflow", op);
    SEQ_TRY(check(op, "k_cache", of(k_cache), k_new->dtype, nc, 16));
    SEQ_TRY(check(op, "v_cache", of(v_cache), k_new->dtype, nc, 16));
    a.k = k_cache->ptr;
    a.v = v_cache->ptr;
    a.c_sp = static_cast<long long>(p.page_stride / 8);
    a.c_sh = static_cast<long long>(p.head_stride / 8);
    a.c_st = static_cast<long long>(p.token_stride / 8);
    const cudaError_t e = launch_rotary_append(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) SEQ_FAIL(TA_ERR_CUDA, "%s: launch: %s", op, cudaGetErrorString(e));
    return TA_OK;
}

TA_EXPORT ta_status paged_quant_append(const ta_quant_append_params *pp, const ta_buf *q, const ta_buf *k_new, const ta_buf *v_new,
                                       const ta_buf *slot_map, const ta_buf *positions, const ta_buf *table, const ta_buf *q_out,
                                       const ta_buf *k_codes, const ta_buf *k_affine, const ta_buf *v_codes, const ta_buf *v_affine,
                                       void *stream) {
    const char *op = "paged_quant_append";
    if (pp == nullptr) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: params is NULL", op);
    ta_quant_append_params p = *pp;
    SEQ_TRY(check_rows(op, p.tokens, p.n_heads, p.n_kv_heads, p.head_dim, p.page_size, p.n_pages));
    SEQ_TRY(check_rotary(op, p.rotary_dim, p.head_dim, p.interleaved, p.max_positions));
    if (p.rotary_dim == 0 && p.n_heads > 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: q without a rotation (n_heads must be 0)", op);
    PageStrides st = {p.codes_page_stride, p.codes_head_stride, p.codes_token_stride, p.affine_page_stride, p.affine_head_stride, p.affine_token_stride};
    SEQ_TRY(page_strides(op, p.n_kv_heads, p.page_size, p.head_dim, p.group_size, &st));
    QuantAppendArgs a;
    SEQ_TRY(new_rows(op, &p, q, k_new, v_new, slot_map, positions, table, q_out, &a.r));
    if (p.tokens == 0) return TA_OK;
    SEQ_TRY(page_buffers(op, st, p.n_pages, p.n_kv_heads, p.page_size, p.head_dim, p.group_size, k_new->dtype, k_codes, k_affine, v_codes, v_affine, &a.c));
    a.group = static_cast<int>(p.group_size);
    const cudaError_t e = launch_quant_append(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) SEQ_FAIL(TA_ERR_CUDA, "%s: launch: %s", op, cudaGetErrorString(e));
    return TA_OK;
}

TA_EXPORT ta_status paged_quant_read(const ta_quant_append_params *pp, const ta_buf *slot_map, const ta_buf *k_codes,
                                     const ta_buf *k_affine, const ta_buf *v_codes, const ta_buf *v_affine, const ta_buf *k,
                                     const ta_buf *v, void *stream) {
    const char *op = "paged_quant_read";
    if (pp == nullptr) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: params is NULL", op);
    ta_quant_append_params p = *pp;
    SEQ_TRY(check_rows(op, p.tokens, p.n_heads, p.n_kv_heads, p.head_dim, p.page_size, p.n_pages));
    if (p.n_heads != 0 || p.rotary_dim != 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: n_heads and rotary_dim must be 0", op);
    PageStrides st = {p.codes_page_stride, p.codes_head_stride, p.codes_token_stride, p.affine_page_stride, p.affine_head_stride, p.affine_token_stride};
    SEQ_TRY(page_strides(op, p.n_kv_heads, p.page_size, p.head_dim, p.group_size, &st));
    row_strides(p.n_kv_heads, p.head_dim, &p.k_token_stride, &p.k_head_stride);
    row_strides(p.n_kv_heads, p.head_dim, &p.v_token_stride, &p.v_head_stride);
    SEQ_TRY(check_stride(op, "k_token_stride", p.k_token_stride));
    SEQ_TRY(check_stride(op, "k_head_stride", p.k_head_stride));
    SEQ_TRY(check_stride(op, "v_token_stride", p.v_token_stride));
    SEQ_TRY(check_stride(op, "v_head_stride", p.v_head_stride));
    if (p.tokens == 0) return TA_OK;
    SEQ_TRY(check_16bit(op, "k", of(k)));
    const int type = k->dtype;
    uint64_t nk, nv;
    const Axis kax[2] = {{p.tokens, p.k_token_stride}, {p.n_kv_heads, p.k_head_stride}};
    const Axis vax[2] = {{p.tokens, p.v_token_stride}, {p.n_kv_heads, p.v_head_stride}};
    if (!extent(kax, p.head_dim, &nk) || !extent(vax, p.head_dim, &nv)) SEQ_FAIL(TA_ERR_OVERFLOW, "%s: sizes overflow", op);
    QuantReadArgs a;
    SEQ_TRY(check(op, "slot_map", of(slot_map), TA_I64, static_cast<uint64_t>(p.tokens) * 8, 8));
    SEQ_TRY(page_buffers(op, st, p.n_pages, p.n_kv_heads, p.page_size, p.head_dim, p.group_size, type, k_codes, k_affine, v_codes, v_affine, &a.c));
    SEQ_TRY(check(op, "k", *k, type, nk, 16));
    SEQ_TRY(check(op, "v", of(v), type, nv, 16));
    a.slot = static_cast<const int64_t *>(slot_map->ptr);
    a.k = k->ptr;
    a.v = v->ptr;
    a.T = static_cast<int>(p.tokens);
    a.Hk = static_cast<int>(p.n_kv_heads);
    a.D = static_cast<int>(p.head_dim);
    a.group = static_cast<int>(p.group_size);
    a.page_shift = log2_of(p.page_size);
    a.n_pages = static_cast<int>(p.n_pages);
    a.bf16 = type == TA_BF16;
    a.k_st = static_cast<long long>(p.k_token_stride);
    a.k_sh = static_cast<long long>(p.k_head_stride);
    a.v_st = static_cast<long long>(p.v_token_stride);
    a.v_sh = static_cast<long long>(p.v_head_stride);
    const cudaError_t e = launch_quant_read(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) SEQ_FAIL(TA_ERR_CUDA, "%s: launch: %s", op, cudaGetErrorString(e));
    return TA_OK;
}

TA_EXPORT size_t paged_quant_attn_workspace_bytes(const ta_paged_quant_params *p) {
    if (check_quant_attn(p) != TA_OK) return SIZE_MAX;
    const uint64_t ws = quant_workspace(p);
    if (ws == 0) set_last_error("paged_quant_attn: no CUDA device to size the workspace for");
    return ws ? ws : SIZE_MAX;
}

static ta_status quant_attn_fwd(const ta_paged_quant_params *pp, const ta_buf *q, const ta_buf *k_codes, const ta_buf *k_affine,
                                const ta_buf *v_codes, const ta_buf *v_affine, const ta_buf *table, const ta_buf *cu,
                                const ta_buf *kv_lens, const ta_buf *parents, const ta_buf *tmp, const ta_buf *out, void *stream,
                                uint32_t polls, bool hook) {
    const char *op = "paged_quant_attn";
    SEQ_TRY(check_quant_attn(pp));
    if (hook && quant_family(pp) != TA_KERNEL_TENSOR_CORES)
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "%s: the wait-limit hook is for the tensor-core kernel only", op);
    ta_paged_quant_params p = *pp;
    const bool tree = !is_absent(parents);
    if (tree && p.window != 0) SEQ_FAIL(TA_ERR_INVALID_ARGUMENT, "%s: window must be 0 with parents", op);
    if (tree && p.max_q_len > static_cast<uint32_t>(kMaxTreeBitsNodes))
        SEQ_FAIL(TA_ERR_UNSUPPORTED, "%s: parents take max_q_len <= %d (got %u)", op, kMaxTreeBitsNodes, p.max_q_len);
    row_strides(p.n_heads, p.head_dim, &p.q_token_stride, &p.q_head_stride);
    row_strides(p.n_heads, p.head_dim, &p.out_token_stride, &p.out_head_stride);
    SEQ_TRY(check_stride(op, "q_token_stride", p.q_token_stride));
    SEQ_TRY(check_stride(op, "q_head_stride", p.q_head_stride));
    SEQ_TRY(check_stride(op, "out_token_stride", p.out_token_stride));
    SEQ_TRY(check_stride(op, "out_head_stride", p.out_head_stride));
    PageStrides st = {p.codes_page_stride, p.codes_head_stride, p.codes_token_stride, p.affine_page_stride, p.affine_head_stride, p.affine_token_stride};
    SEQ_TRY(page_strides(op, p.n_kv_heads, p.page_size, p.head_dim, p.group_size, &st));
    if (p.tokens == 0) return TA_OK;
    SEQ_TRY(check_16bit(op, "q", of(q)));
    const int type = q->dtype;
    uint64_t nq, no;
    const Axis qax[2] = {{p.tokens, p.q_token_stride}, {p.n_heads, p.q_head_stride}};
    const Axis oax[2] = {{p.tokens, p.out_token_stride}, {p.n_heads, p.out_head_stride}};
    if (!extent(qax, p.head_dim, &nq) || !extent(oax, p.head_dim, &no)) SEQ_FAIL(TA_ERR_OVERFLOW, "%s: sizes overflow", op);
    const uint64_t ws = quant_workspace(&p);
    SeqQuantArgs a = {};
    SEQ_TRY(check(op, "q", *q, type, nq, 16));
    SEQ_TRY(page_buffers(op, st, p.n_pages, p.n_kv_heads, p.page_size, p.head_dim, p.group_size, type, k_codes, k_affine, v_codes, v_affine, &a.c));
    SEQ_TRY(check(op, "table", of(table), TA_I32, static_cast<uint64_t>(p.batch) * p.max_pages * 4, 4));
    SEQ_TRY(check(op, "cu", of(cu), TA_I32, (static_cast<uint64_t>(p.batch) + 1) * 4, 4));
    SEQ_TRY(check(op, "kv_lens", of(kv_lens), TA_I32, static_cast<uint64_t>(p.batch) * 4, 4));
    if (tree) SEQ_TRY(check(op, "parents", *parents, TA_I32, static_cast<uint64_t>(p.tokens) * 4, 4));
    SEQ_TRY(check(op, "tmp", of(tmp), TA_F32, ws ? ws : kStatusBytes, 16));
    SEQ_TRY(check(op, "out", of(out), type, no, 16));
    SeqArgs &s = a.s;
    s.q = q->ptr;
    s.out = out->ptr;
    s.cu = static_cast<const int32_t *>(cu->ptr);
    s.kv_lens = static_cast<const int32_t *>(kv_lens->ptr);
    s.table = static_cast<const int32_t *>(table->ptr);
    s.parents = tree ? static_cast<const int32_t *>(parents->ptr) : nullptr;
    s.status = static_cast<int32_t *>(tmp->ptr);
    s.B = static_cast<int>(p.batch);
    s.H = static_cast<int>(p.n_heads);
    s.Hk = static_cast<int>(p.n_kv_heads);
    s.g = s.H / s.Hk;
    s.D = static_cast<int>(p.head_dim);
    s.T = static_cast<int>(p.tokens);
    s.max_q = static_cast<int>(p.max_q_len);
    s.window = static_cast<int>(p.window < kMostKeys ? p.window : kMostKeys);     // no request has more keys
    s.page_shift = log2_of(p.page_size);
    s.n_pages = static_cast<int>(p.n_pages);
    s.max_pages = static_cast<int>(p.max_pages);
    s.bf16 = type == TA_BF16;
    s.q_st = static_cast<long long>(p.q_token_stride);
    s.q_sh = static_cast<long long>(p.q_head_stride);
    s.o_st = static_cast<long long>(p.out_token_stride);
    s.o_sh = static_cast<long long>(p.out_head_stride);
    s.scale = p.scale;
    a.group = static_cast<int>(p.group_size);
    if (ws == 0) SEQ_FAIL(TA_ERR_CUDA, "%s: no CUDA device", op);
    return run_quant(op, a, quant_family(&p), tmp->ptr, static_cast<cudaStream_t>(stream), polls);
}

TA_EXPORT ta_status paged_quant_attn_fwd(const ta_paged_quant_params *p, const ta_buf *q, const ta_buf *k_codes, const ta_buf *k_affine,
                                         const ta_buf *v_codes, const ta_buf *v_affine, const ta_buf *table, const ta_buf *cu,
                                         const ta_buf *kv_lens, const ta_buf *parents, const ta_buf *tmp, const ta_buf *out, void *stream) {
    return quant_attn_fwd(p, q, k_codes, k_affine, v_codes, v_affine, table, cu, kv_lens, parents, tmp, out, stream, kSeqWaitPolls, false);
}

TA_EXPORT ta_status ta_test_paged_quant_attn_fwd_wait_limit(uint32_t wait_polls, const ta_paged_quant_params *p, const ta_buf *q,
                                                            const ta_buf *k_codes, const ta_buf *k_affine, const ta_buf *v_codes,
                                                            const ta_buf *v_affine, const ta_buf *table, const ta_buf *cu,
                                                            const ta_buf *kv_lens, const ta_buf *parents, const ta_buf *tmp,
                                                            const ta_buf *out, void *stream) {
    return quant_attn_fwd(p, q, k_codes, k_affine, v_codes, v_affine, table, cu, kv_lens, parents, tmp, out, stream, wait_polls, true);
}
