// C ABI of the paged 8-bit key/value cache: host-side checks, then the launches.
// Every check runs before the first, so an error return enqueues nothing.
#include "prox.h"
#include "prox_internal.hpp"
#include "prox_kv.hpp"

using namespace prox;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int kMaxTokens = 1 << 28;

prox_status check_cache(const prox_kv_cache* c) {
    if (!c) return fail(PROX_E_INVALID, "null cache");
    if (c->kind != PROX_KV_INT8 && c->kind != PROX_KV_FP8) return fail(PROX_E_INVALID, "unknown cache kind");
    if (c->n_pages < 1) return fail(PROX_E_INVALID, "n_pages must be >= 1");
    if (c->n_kv < 1) return fail(PROX_E_INVALID, "n_kv must be >= 1");
    if (c->n_kv > PROX_KV_MAX_HEADS) return fail(PROX_E_UNSUPPORTED, "n_kv above PROX_KV_MAX_HEADS");
    if (c->head_dim < 8 || c->head_dim % 8) return fail(PROX_E_INVALID, "head_dim must be a positive multiple of 8");
    if (c->head_dim > PROX_KV_MAX_HEAD_DIM) return fail(PROX_E_UNSUPPORTED, "head_dim above PROX_KV_MAX_HEAD_DIM");
    if (c->head_pad != prox_kv_head_pad(c->head_dim))
        return fail(PROX_E_MISMATCH, "head_pad is not prox_kv_head_pad(head_dim)");
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return fail(PROX_E_INVALID, "null cache buffer");
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return fail(PROX_E_INVALID, "misaligned cache buffer");
    return PROX_OK;
}

prox_status check_batch(const prox_kv_batch* b) {
    if (!b) return fail(PROX_E_INVALID, "null batch");
    if (b->n_seq < 1) return fail(PROX_E_INVALID, "n_seq must be >= 1");
    if (b->n_tokens < 0 || b->max_q < 0) return fail(PROX_E_INVALID, "n_tokens and max_q must be >= 0");
    if (b->n_tokens > kMaxTokens || b->n_seq > kMaxTokens) return fail(PROX_E_UNSUPPORTED, "more than 2^28 tokens");
    if (b->max_pages < 1) return fail(PROX_E_INVALID, "max_pages must be >= 1");
    if (b->max_pages > 0x7fffffff / PROX_KV_PAGE) return fail(PROX_E_UNSUPPORTED, "64 * max_pages above 2^31 - 1");
    if (!b->ctx_len || !b->block_table) return fail(PROX_E_INVALID, "null ctx_len or block_table");
    if (!aligned(b->ctx_len, 4) || !aligned(b->block_table, 4) || !aligned(b->q_start, 4))
        return fail(PROX_E_INVALID, "misaligned batch array");
    if (!b->q_start && b->n_tokens != b->n_seq)
        return fail(PROX_E_INVALID, "without q_start there is one token per sequence: n_tokens must equal n_seq");
    return PROX_OK;
}

// One of the bf16 activations [n_tokens][heads][head_dim].
prox_status check_rows(const char* name, const void* p, int64_t stride, int64_t width) {
    if (!p) return fail(PROX_E_INVALID, "null %s", name);
    if (!aligned(p, 16)) return fail(PROX_E_INVALID, "%s must be 16-byte aligned", name);
    if (stride < width || stride % 8)
        return fail(PROX_E_INVALID, "%s: the row stride must be a multiple of 8 and at least heads * head_dim", name);
    if (stride > (1ll << 32)) return fail(PROX_E_UNSUPPORTED, "%s: row stride above 2^32", name);
    return PROX_OK;
}

prox_status check_heads(const prox_kv_cache* c, int32_t n_heads) {
    if (n_heads < 1 || n_heads % c->n_kv) return fail(PROX_E_INVALID, "n_heads must be a positive multiple of n_kv");
    if (n_heads > PROX_KV_MAX_HEADS) return fail(PROX_E_UNSUPPORTED, "n_heads above PROX_KV_MAX_HEADS");
    return PROX_OK;
}

prox_status launched(hipError_t e, const char* what) {
    if (e == hipErrorInvalidConfiguration) return fail(PROX_E_UNSUPPORTED, "%s: the batch's bounds are too large for one call", what);
    return e == hipSuccess ? PROX_OK : hip_fail(e, what);
}

}  // namespace

#define PROX_CHECK(x)                           \
    do {                                        \
        const prox_status st_ = (x);            \
        if (st_ != PROX_OK) return st_;         \
    } while (0)

extern "C" int32_t prox_kv_head_pad(int32_t head_dim) {
    if (head_dim < 8 || head_dim % 8 || head_dim > PROX_KV_MAX_HEAD_DIM) return 0;
    return (head_dim + 63) / 64 * 64;
}

extern "C" prox_status prox_kv_append(const prox_kv_cache* c, const prox_kv_batch* b, const void* k, int64_t k_stride,
                                      const void* v, int64_t v_stride, const prox_kv_rotation* r, int32_t n_heads,
                                      const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                                      void* stream) {
    clear_error();
    PROX_CHECK(check_cache(c));
    PROX_CHECK(check_batch(b));
    if (!r) return fail(PROX_E_INVALID, "null rotation");
    if ((!q) != (!q_out)) return fail(PROX_E_INVALID, "q and q_out must both be given or both be null");
    if (q) PROX_CHECK(check_heads(c, n_heads));
    if (r->rot) {
        if (!aligned(r->rot, 8)) return fail(PROX_E_INVALID, "rot must be 8-byte aligned");
        if (r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > c->head_dim)
            return fail(PROX_E_INVALID, "rot_dim must be even, >= 2 and at most head_dim");
        if (r->pairing != PROX_ROPE_INTERLEAVED && r->pairing != PROX_ROPE_HALVES)
            return fail(PROX_E_INVALID, "unknown pairing");
        if (r->pairing == PROX_ROPE_HALVES && r->rot_dim % 16)
            return fail(PROX_E_UNSUPPORTED, "pairs of halves need rot_dim %% 16 == 0");
        if (r->rot_rows < b->max_pages * PROX_KV_PAGE)
            return fail(PROX_E_INVALID, "the rotation table needs a row for each of the 64 * max_pages positions");
    }
    if (!aligned(r->g_q, 4) || !aligned(r->g_k, 4)) return fail(PROX_E_INVALID, "misaligned gain");
    if ((r->g_q || r->g_k) && !(r->eps >= 0.f && r->eps < 3.0e38f)) return fail(PROX_E_INVALID, "eps must be finite and >= 0");
    if (b->n_tokens == 0 || b->max_q == 0) return PROX_OK;
    const int64_t hd = c->head_dim;
    PROX_CHECK(check_rows("k", k, k_stride, c->n_kv * hd));
    PROX_CHECK(check_rows("v", v, v_stride, c->n_kv * hd));
    if (q) {
        PROX_CHECK(check_rows("q", q, q_stride, n_heads * hd));
        PROX_CHECK(check_rows("q_out", q_out, q_out_stride, n_heads * hd));
        if (q == q_out && q_stride != q_out_stride)
            return fail(PROX_E_INVALID, "a call in place needs q_out_stride equal to q_stride");
    }
    return launched(launch_kv_append(*c, *b, static_cast<const uint16_t*>(k), k_stride,
                                     static_cast<const uint16_t*>(v), v_stride, *r, n_heads,
                                     static_cast<const uint16_t*>(q), q_stride, static_cast<uint16_t*>(q_out),
                                     q_out_stride, (hipStream_t)stream),
                    "cache append");
}

extern "C" size_t prox_kv_workspace_bytes(const prox_kv_cache* c, const prox_kv_batch* b, int32_t n_heads) {
    clear_error();
    if (check_cache(c) != PROX_OK || check_batch(b) != PROX_OK || check_heads(c, n_heads) != PROX_OK) return 0;
    return kv_attention_workspace(*c, *b, n_heads);
}

extern "C" prox_status prox_kv_attention(const prox_kv_cache* c, const prox_kv_batch* b, const void* q,
                                         int64_t q_stride, int32_t n_heads, float scale, int32_t window, void* out,
                                         int64_t out_stride, void* workspace, size_t ws_bytes, void* stream) {
    clear_error();
    PROX_CHECK(check_cache(c));
    PROX_CHECK(check_batch(b));
    PROX_CHECK(check_heads(c, n_heads));
    if (!(scale > -3.0e38f && scale < 3.0e38f)) return fail(PROX_E_INVALID, "scale must be finite");
    if (window < 0) return fail(PROX_E_INVALID, "window must be >= 0");
    if (b->n_tokens == 0 || b->max_q == 0) return PROX_OK;
    const int64_t width = (int64_t)n_heads * c->head_dim;
    PROX_CHECK(check_rows("q", q, q_stride, width));
    PROX_CHECK(check_rows("out", out, out_stride, width));
    if (q == out) return fail(PROX_E_INVALID, "out must not be q");
    if (!workspace) return fail(PROX_E_INVALID, "null workspace");
    if (!aligned(workspace, 256)) return fail(PROX_E_INVALID, "workspace must be 256-byte aligned");
    const size_t need = kv_attention_workspace(*c, *b, n_heads);
    if (need == 0) return launched(hipErrorInvalidConfiguration, "cache attention");
    if (ws_bytes < need) return fail(PROX_E_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    return launched(launch_kv_attention(*c, *b, static_cast<const uint16_t*>(q), q_stride, n_heads, scale, window,
                                        static_cast<uint16_t*>(out), out_stride, workspace, (hipStream_t)stream),
                    "cache attention");
}

extern "C" prox_status prox_kv_read(const prox_kv_cache* c, const prox_kv_batch* b, void* k_out, void* v_out,
                                    int32_t out_fp32, void* stream) {
    clear_error();
    PROX_CHECK(check_cache(c));
    PROX_CHECK(check_batch(b));
    if (b->n_tokens == 0 || b->max_q == 0) return PROX_OK;
    if (!k_out || !v_out) return fail(PROX_E_INVALID, "null k_out or v_out");
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return fail(PROX_E_INVALID, "outputs must be 16-byte aligned");
    return launched(launch_kv_read(*c, *b, k_out, v_out, out_fp32 != 0, (hipStream_t)stream), "cache read");
}

static prox_status check_pool(const prox_kv_pool* p) {
    if (!p) return fail(PROX_E_INVALID, "null pool");
    if (p->n_pages < 1 || p->n_seq < 1 || p->max_pages < 1)
        return fail(PROX_E_INVALID, "n_pages, n_seq and max_pages must be >= 1");
    if (p->n_pages > PROX_KV_MAX_POOL || p->n_seq > PROX_KV_MAX_POOL)
        return fail(PROX_E_UNSUPPORTED, "more than PROX_KV_MAX_POOL pages or sequences");
    if (p->max_pages > 0x7fffffff / PROX_KV_PAGE) return fail(PROX_E_UNSUPPORTED, "64 * max_pages above 2^31 - 1");
    if (!p->refs || !p->ctx_len || !p->block_table) return fail(PROX_E_INVALID, "null pool array");
    if (!aligned(p->refs, 4) || !aligned(p->ctx_len, 4) || !aligned(p->block_table, 4))
        return fail(PROX_E_INVALID, "misaligned pool array");
    return PROX_OK;
}

extern "C" size_t prox_kv_pages_workspace_bytes(const prox_kv_pool* p) {
    clear_error();
    return check_pool(p) == PROX_OK ? kv_pages_workspace(*p) : 0;
}

extern "C" prox_status prox_kv_pages(const prox_kv_pool* p, const int32_t* want, const int32_t* parent,
                                     const int32_t* shared, int32_t* q_start, int32_t n_rows, int32_t* slots,
                                     int32_t* status, void* workspace, size_t ws_bytes, void* stream) {
    clear_error();
    PROX_CHECK(check_pool(p));
    if (!want || !q_start || !status) return fail(PROX_E_INVALID, "null want, q_start or status");
    if ((!parent) != (!shared)) return fail(PROX_E_INVALID, "parent and shared must both be given or both be null");
    if (n_rows < 0) return fail(PROX_E_INVALID, "n_rows must be >= 0");
    if (n_rows > 0 && !slots) return fail(PROX_E_INVALID, "null slots");
    if (!aligned(want, 4) || !aligned(parent, 4) || !aligned(shared, 4) || !aligned(q_start, 4) || !aligned(slots, 4) ||
        !aligned(status, 4))
        return fail(PROX_E_INVALID, "misaligned array");
    if (!workspace) return fail(PROX_E_INVALID, "null workspace");
    if (!aligned(workspace, 8)) return fail(PROX_E_INVALID, "workspace must be 8-byte aligned");
    const size_t need = kv_pages_workspace(*p);
    if (ws_bytes < need) return fail(PROX_E_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    return launched(launch_kv_pages(*p, want, parent, shared, q_start, n_rows, slots, status, workspace, (hipStream_t)stream),
                    "page tables");
}

static prox_status check_keep(int32_t n_keep) {
    if (n_keep < 1) return fail(PROX_E_INVALID, "n_keep must be >= 1");
    if (n_keep > 1 << 20) return fail(PROX_E_UNSUPPORTED, "n_keep above 2^20");
    return PROX_OK;
}

extern "C" prox_status prox_kv_page_bounds(const prox_kv_cache* c, const prox_kv_batch* b, void* bounds, void* stream) {
    clear_error();
    PROX_CHECK(check_cache(c));
    PROX_CHECK(check_batch(b));
    if (b->n_tokens == 0 || b->max_q == 0) return PROX_OK;
    if (!bounds) return fail(PROX_E_INVALID, "null bounds");
    if (!aligned(bounds, 16)) return fail(PROX_E_INVALID, "bounds must be 16-byte aligned");
    return launched(launch_kv_bounds(*c, *b, static_cast<int8_t*>(bounds), (hipStream_t)stream), "page bounds");
}

extern "C" size_t prox_kv_select_workspace_bytes(const prox_kv_cache* c, const prox_kv_batch* b, int32_t n_heads) {
    clear_error();
    if (check_cache(c) != PROX_OK || check_batch(b) != PROX_OK || check_heads(c, n_heads) != PROX_OK) return 0;
    if (b->max_pages > PROX_KV_MAX_SELECT_PAGES) return 0;
    return kv_select_workspace(*c, *b, n_heads);
}

extern "C" prox_status prox_kv_select(const prox_kv_cache* c, const prox_kv_batch* b, const void* q, int64_t q_stride,
                                      int32_t n_heads, const void* bounds, int32_t n_keep, int32_t first, int32_t last,
                                      int32_t* pages, void* workspace, size_t ws_bytes, void* stream) {
    clear_error();
    PROX_CHECK(check_cache(c));
    PROX_CHECK(check_batch(b));
    PROX_CHECK(check_heads(c, n_heads));
    PROX_CHECK(check_keep(n_keep));
    if (first < 0 || last < 1 || first > n_keep || last > n_keep - first)
        return fail(PROX_E_INVALID, "first >= 0, last >= 1 and first + last <= n_keep are needed");
    if (b->max_pages > PROX_KV_MAX_SELECT_PAGES) return fail(PROX_E_UNSUPPORTED, "max_pages above PROX_KV_MAX_SELECT_PAGES");
    if (b->n_tokens == 0 || b->max_q == 0) return PROX_OK;
    if (!bounds || !pages) return fail(PROX_E_INVALID, "null bounds or pages");
    if (!aligned(bounds, 16) || !aligned(pages, 4)) return fail(PROX_E_INVALID, "misaligned bounds or pages");
    PROX_CHECK(check_rows("q", q, q_stride, (int64_t)n_heads * c->head_dim));
    if (!workspace) return fail(PROX_E_INVALID, "null workspace");
    if (!aligned(workspace, 256)) return fail(PROX_E_INVALID, "workspace must be 256-byte aligned");
    const size_t need = kv_select_workspace(*c, *b, n_heads);
    if (need == 0) return launched(hipErrorInvalidConfiguration, "page selection");
    if (ws_bytes < need) return fail(PROX_E_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    return launched(launch_kv_select(*c, *b, static_cast<const uint16_t*>(q), q_stride, n_heads,
                                     static_cast<const int8_t*>(bounds), n_keep, first, last, pages, workspace, (hipStream_t)stream),
                    "page selection");
}

extern "C" size_t prox_kv_selected_workspace_bytes(const prox_kv_cache* c, const prox_kv_batch* b, int32_t n_heads,
                                                   int32_t n_keep) {
    clear_error();
    if (check_cache(c) != PROX_OK || check_batch(b) != PROX_OK || check_heads(c, n_heads) != PROX_OK ||
        check_keep(n_keep) != PROX_OK)
        return 0;
    return kv_selected_workspace(*c, *b, n_heads, n_keep);
}

extern "C" prox_status prox_kv_attention_selected(const prox_kv_cache* c, const prox_kv_batch* b, const void* q,
                                                  int64_t q_stride, int32_t n_heads, const int32_t* pages, int32_t n_keep,
                                                  float scale, void* out, int64_t out_stride, void* workspace,
                                                  size_t ws_bytes, void* stream) {
    clear_error();
    PROX_CHECK(check_cache(c));
    PROX_CHECK(check_batch(b));
    PROX_CHECK(check_heads(c, n_heads));
    PROX_CHECK(check_keep(n_keep));
    if (!(scale > -3.0e38f && scale < 3.0e38f)) return fail(PROX_E_INVALID, "scale must be finite");
    if (b->n_tokens == 0 || b->max_q == 0) return PROX_OK;
    const int64_t width = (int64_t)n_heads * c->head_dim;
    PROX_CHECK(check_rows("q", q, q_stride, width));
    PROX_CHECK(check_rows("out", out, out_stride, width));
    if (q == out) return fail(PROX_E_INVALID, "out must not be q");
    if (!pages) return fail(PROX_E_INVALID, "null pages");
    if (!aligned(pages, 4)) return fail(PROX_E_INVALID, "misaligned pages");
    if (!workspace) return fail(PROX_E_INVALID, "null workspace");
    if (!aligned(workspace, 256)) return fail(PROX_E_INVALID, "workspace must be 256-byte aligned");
    const size_t need = kv_selected_workspace(*c, *b, n_heads, n_keep);
    if (need == 0) return launched(hipErrorInvalidConfiguration, "attention over selected pages");
    if (ws_bytes < need) return fail(PROX_E_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    return launched(launch_kv_selected(*c, *b, static_cast<const uint16_t*>(q), q_stride, n_heads, pages, n_keep, scale,
                                       static_cast<uint16_t*>(out), out_stride, workspace, (hipStream_t)stream),
                    "attention over selected pages");
}

static prox_status check_groups(const prox_kv_batch* b, int32_t n_groups) {
    if (n_groups < 1 || n_groups > b->n_seq) return fail(PROX_E_INVALID, "n_groups must be 1 .. n_seq");
    return PROX_OK;
}

extern "C" size_t prox_kv_shared_workspace_bytes(const prox_kv_cache* c, const prox_kv_batch* b, int32_t n_heads,
                                                 int32_t n_groups) {
    clear_error();
    if (check_cache(c) != PROX_OK || check_batch(b) != PROX_OK || check_heads(c, n_heads) != PROX_OK ||
        check_groups(b, n_groups) != PROX_OK)
        return 0;
    return kv_shared_workspace(*c, *b, n_heads, n_groups);
}

extern "C" prox_status prox_kv_attention_shared(const prox_kv_cache* c, const prox_kv_batch* b, const int32_t* group_start,
                                                int32_t n_groups, const int32_t* shared, const void* q, int64_t q_stride,
                                                int32_t n_heads, float scale, void* out, int64_t out_stride,
                                                void* workspace, size_t ws_bytes, void* stream) {
    clear_error();
    PROX_CHECK(check_cache(c));
    PROX_CHECK(check_batch(b));
    PROX_CHECK(check_heads(c, n_heads));
    PROX_CHECK(check_groups(b, n_groups));
    if (!group_start && n_groups != 1) return fail(PROX_E_INVALID, "without group_start there is one group");
    if (!shared) return fail(PROX_E_INVALID, "null shared");
    if (!aligned(group_start, 4) || !aligned(shared, 4)) return fail(PROX_E_INVALID, "misaligned group_start or shared");
    if (!(scale > -3.0e38f && scale < 3.0e38f)) return fail(PROX_E_INVALID, "scale must be finite");
    if (b->n_tokens == 0 || b->max_q == 0) return PROX_OK;
    const int64_t width = (int64_t)n_heads * c->head_dim;
    PROX_CHECK(check_rows("q", q, q_stride, width));
    PROX_CHECK(check_rows("out", out, out_stride, width));
    if (q == out) return fail(PROX_E_INVALID, "out must not be q");
    if (!workspace) return fail(PROX_E_INVALID, "null workspace");
    if (!aligned(workspace, 256)) return fail(PROX_E_INVALID, "workspace must be 256-byte aligned");
    const size_t need = kv_shared_workspace(*c, *b, n_heads, n_groups);
    if (need == 0) return launched(hipErrorInvalidConfiguration, "attention with a shared prefix");
    if (ws_bytes < need) return fail(PROX_E_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    return launched(launch_kv_shared(*c, *b, group_start, n_groups, shared, static_cast<const uint16_t*>(q), q_stride,
                                     n_heads, scale, static_cast<uint16_t*>(out), out_stride, workspace,
                                     (hipStream_t)stream),
                    "attention with a shared prefix");
}
