// Attention over the paged 8-bit key/value cache: the launches of a call.
#include "prox_kv_attn.hpp"

namespace prox {

size_t kv_attention_workspace(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads) {
    if (b.max_q <= 0) return 256;
    const Launches L(c, bounded(b), n_heads);
    return L.fit() ? workspace_of(c, b, n_heads, L) : 0;
}

hipError_t launch_kv_attention(const prox_kv_cache& c, const prox_kv_batch& batch, const uint16_t* q, int64_t q_stride,
                               int n_heads, float scale, int window, uint16_t* out, int64_t out_stride,
                               void* workspace, hipStream_t s) {
    const prox_kv_batch b = bounded(batch);
    // one launch behind the other: they share the workspace
    const Launches L(c, b, n_heads);
    if (!L.fit()) return hipErrorInvalidConfiguration;
    Attend A{};
    set_call(A, c, b, q, q_stride, n_heads, scale, window, out, out_stride);
    A.arrived = static_cast<unsigned long long*>(workspace);
    for (int k = L.few > 0 ? 0 : 1; k < 2; ++k) {
        const Split& p = L.split[k];
        A.rows_lo = k == 0 ? 1 : L.few + 1;
        A.rows_hi = k == 0 ? L.few : b.max_q;
        A.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.part_at);
        set_split(A, p);
        const hipError_t e = c.kind == PROX_KV_INT8 ? attend_kind<PROX_KV_INT8>(A, p, s) : attend_kind<PROX_KV_FP8>(A, p, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace prox
