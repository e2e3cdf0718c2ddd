// Attention over the paged key/value cache for sequences that share a prefix.
//
// A softmax over two sets of positions is put together from the two sets' own
// maxima, sums and results.  So a call is two launches of the attention's kernel
// and one between them:
//   1  the rows of all sequences of a group, as those of one sequence, over the
//      group's shared pages, without a mask; what comes out is each row's
//      maximum, sum, unit and unnormalised result, in fp32, in the workspace;
//   2  a group has few tiles of rows, each cut among many blocks: the parts of a
//      row are joined, all rows at once (by the block that arrives last, as the
//      attention over all pages does it, 64 tokens over 512 shared pages took
//      148 us instead of 60 + 9: 4 MB of parts for one block);
//   3  the rows of each sequence over its other pages, causal; a row's part of 1
//      joins before it is normalised and rounded.
// A page of a prefix is read once for a tile of rows instead of once for each
// sequence: 256 (32 of each of 8 waves) where the groups have more than 128 rows of
// a key head in the mean, 128 up to there and for heads wider than 128, 16 where
// they have no more than 16.  Unlike groups lose by the mean: 63 sequences of 32 / 32
// heads x 128 over 512 shared pages take 111 us in a call of their own, 7 groups of
// one such sequence 342, the eight groups in one call 483.
// A sequence whose first row lies inside the prefix takes no part in it: launch 3
// goes over all of its pages.
#include "prox_kv_attn.hpp"

namespace prox {

namespace {

struct GroupArgs {
    const int32_t *group_start, *shared;
    int n_groups, n_seq;
    int n_heads;
    int blocks;                // of launch 1
    float* row_part;           // [n_tokens][n_heads][head_pad + 4]
    int32_t* skip;             // [n_seq]: pages of a sequence that are taken from its group
    int32_t* joins;            // [n_tokens]: whether the row takes its part of the prefix
    int4* parts;               // [n_tokens][VH of launch 1]: first block, blocks (0: none to join), row of the tile
};

__device__ __forceinline__ int group_at(const GroupArgs& G, int g) {
    return G.group_start ? min(max(G.group_start[g], 0), G.n_seq) : (g == 0 ? 0 : G.n_seq);
}
__device__ __forceinline__ int shared_pages(const GroupArgs& G, const prox_kv_batch& b, int g) {
    return min(max(G.shared[g], 0), b.max_pages);
}
__device__ __forceinline__ size_t row_part_at(const Attend& A, const GroupArgs& G, int row, int head) {
    return ((size_t)row * G.n_heads + head) * (size_t)(A.c.head_pad + 4);
}

// Row of the batch and query head of row r of a segment; row -1 for one that the segment does not have.
struct RowHead {
    int row, head;
};
__device__ __forceinline__ RowHead row_head(const Attend& A, const Seg& S, int r) {
    const int groups = A.VH / A.c.n_kv, head = S.vh / groups, grp = S.vh - head * groups;
    const int i = token_of(A, r), hq = grp * A.HG + r - i * A.HG;
    return RowHead{i >= S.n || hq >= A.rep ? -1 : S.row0 + i, head * A.rep + hq};
}

// ---- launch 1: "sequence" s is group s, A.b.n_seq their number; a group's Row has
// the number of its shared pages as `first`.
struct PrefixOut {
    float* to = nullptr;
    int4* parts = nullptr;
    __device__ __forceinline__ explicit operator bool() const { return to != nullptr; }
};
struct AttendPrefix : Attend {
    typedef PrefixOut Out;
    static constexpr bool kJoinLater = true;
    GroupArgs G;
};

// Which sequences and rows take part, for the other launches.
__device__ __forceinline__ void prologue(const AttendPrefix& A, int wv, int l) {
    const GroupArgs& G = A.G;
    for (int s = blockIdx.x * (int)(blockDim.x >> 6) + wv; s < G.n_seq; s += gridDim.x * (int)(blockDim.x >> 6)) {
        int g = 0;
        if (G.group_start) {
            int upto = 0;                                        // groups that begin at s or before
            for (int base = 0; base < G.n_groups; base += 64)
                upto += __popcll(__ballot(base + l < G.n_groups && G.group_start[min(base + l, G.n_groups - 1)] <= s));
            g = max(upto - 1, 0);
        }
        const KvRows R = kv_rows(A.b, s);
        int pages = s >= group_at(G, g) && s < group_at(G, g + 1) ? shared_pages(G, A.b, g) : 0;
        if (R.first < pages * kKvPage) pages = 0;
        if (l == 0) G.skip[s] = pages;
        const int cap = A.b.max_pages * kKvPage;
        for (int i = l; i < R.n; i += 64) G.joins[R.q0 + i] = pages > 0 && R.first + i < cap;
    }
    // rows before the first and behind the last sequence
    if (!A.b.q_start) return;
    const int lo = min(max(A.b.q_start[0], 0), A.b.n_tokens), hi = min(max(A.b.q_start[G.n_seq], lo), A.b.n_tokens);
    const int t = blockIdx.x * (int)blockDim.x + (int)threadIdx.x, all = gridDim.x * (int)blockDim.x;
    for (int i = t; i < lo; i += all) G.joins[i] = 0;
    for (int i = hi + t; i < A.b.n_tokens; i += all) G.joins[i] = 0;
}
__device__ __forceinline__ KvRows rows_of(const AttendPrefix& A, int g) {
    const int s0 = group_at(A.G, g), s1 = max(group_at(A.G, g + 1), s0);
    KvRows R;
    R.q0 = A.b.q_start ? min(max(A.b.q_start[s0], 0), A.b.n_tokens) : s0;
    R.n = (A.b.q_start ? min(max(A.b.q_start[s1], R.q0), A.b.n_tokens) : s1) - R.q0;
    R.first = shared_pages(A.G, A.b, g);
    R.rows = R.first > 0 ? R.n : 0;
    return R;
}
__device__ __forceinline__ Tile tile_of(const AttendPrefix& A, const KvRows& R, int t) {
    Tile x;
    x.R = R;
    x.i0 = t * A.TQ;
    x.n = min(R.rows - x.i0, A.TQ);
    x.pg0 = 0;
    x.pages = x.n > 0 ? R.first : 0;
    return x;
}
__device__ __forceinline__ const int32_t* table_of(const AttendPrefix& A, int g) {
    return A.b.block_table + (size_t)min(group_at(A.G, g), A.G.n_seq - 1) * A.b.max_pages;
}
// all slots hold tokens: rows of a sequence that has not filled these pages are worked on here, but never joined
__device__ __forceinline__ int ctx_of(const AttendPrefix&, const Tile&) { return 0x7fffffff; }
__device__ __forceinline__ constexpr bool masked(const AttendPrefix&) { return false; }
__device__ __forceinline__ PrefixOut out_row(const AttendPrefix& A, const Seg& S, int r) {
    const RowHead h = row_head(A, S, r);
    PrefixOut x;
    if (h.row < 0) return x;
    x.to = A.G.row_part + row_part_at(A, A.G, h.row, h.head);
    x.parts = A.G.parts + (size_t)h.row * A.VH + S.vh;
    return x;
}
__device__ __forceinline__ void put(const AttendPrefix& A, const PrefixOut& x, int c4, f32x4_t o, const Part& a, float) {
    *reinterpret_cast<f32x4_t*>(x.to + c4) = o;
    if (c4 == 0) {
        *reinterpret_cast<float4*>(x.to + A.c.head_pad) = packed(a);
        *x.parts = make_int4(0, 0, 0, 0);
    }
}
__device__ __forceinline__ void later(const AttendPrefix& A, const Seg& S, int i, int block, int blocks) {
    A.G.parts[(size_t)(S.row0 + i) * A.VH + S.vh] = make_int4(block, blocks, i * A.HG, 0);
}

// ---- launch 2: a thread for each row, query head and four channels.  64 tokens of 32 heads and 32 parts each: 8.7 us
// (35 MB, 4 TB/s); with the parts of a row split among four threads 9.0.
constexpr int kJoinThreads = 256;
int64_t join_blocks(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads) {
    return ((int64_t)b.n_tokens * n_heads * (c.head_pad / 4) + kJoinThreads - 1) / kJoinThreads;
}
template <int NP>
__global__ void __launch_bounds__(kJoinThreads) k_kv_join(AttendPrefix A, int64_t pairs) {
    constexpr int RW = 64 * NP + 4, LPR = 16 * NP;
    const int64_t t = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x, pair = t / LPR;
    const int c4 = 4 * (int)(t % LPR);
    if (pair >= pairs) return;
    const int row = (int)(pair / A.G.n_heads), hq = (int)(pair % A.G.n_heads);
    if (!A.G.joins[row]) return;
    const int groups = A.VH / A.c.n_kv, head = hq / A.rep, in = hq - head * A.rep, grp = in / A.HG;
    const int4 p = A.G.parts[(size_t)row * A.VH + head * groups + grp];
    // (a q_start that does not rise leaves rows that nobody wrote this for: their loop ends too)
    const int parts = min(p.y, A.G.blocks);
    if (parts <= 0) return;
    const __amdgpu_buffer_rsrc_t rp = make_rsrc(A.part, A.part_bytes);
    const uint32_t r = (uint32_t)(p.z + in - grp * A.HG);
    Part a = no_part();
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    for (int p0 = 0; p0 < parts; p0 += 8) {
        u32x4_t v[8], ms[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int k = min(p0 + u, parts - 1);
            const uint32_t at = ((2u * ((uint32_t)p.x + (uint32_t)k) + (k == 0 ? 1u : 0u)) * (uint32_t)A.slot_rows + r) * (uint32_t)(RW * 4);
            v[u] = __builtin_amdgcn_raw_buffer_load_b128(rp, (int)(at + 4 * c4), 0, 0);
            ms[u] = __builtin_amdgcn_raw_buffer_load_b128(rp, (int)(at + 256 * NP), 0, 0);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (p0 + u < parts) join(a, o, unpacked(__builtin_bit_cast(float4, ms[u])), __builtin_bit_cast(f32x4_t, v[u]));
    }
    float* to = A.G.row_part + row_part_at(A, A.G, row, hq);
    *reinterpret_cast<f32x4_t*>(to + c4) = o;
    if (c4 == 0) *reinterpret_cast<float4*>(to + A.c.head_pad) = packed(a);
}

// ---- launch 3
struct RestRows : KvRows {
    int skip;
};
struct RestOut {
    uint16_t* to = nullptr;
    const float* part = nullptr;
    __device__ __forceinline__ explicit operator bool() const { return to != nullptr; }
};
struct AttendRest : Attend {
    typedef RestRows Row;
    typedef RestOut Out;
    GroupArgs G;
};
__device__ __forceinline__ RestRows no_rows(const AttendRest&) { return RestRows{{0, 0, 0, 0}, 0}; }
__device__ __forceinline__ RestRows shuffled(const RestRows& R, int i) {
    return RestRows{shuffled(static_cast<const KvRows&>(R), i), __shfl(R.skip, i)};
}
__device__ __forceinline__ RestRows of_lane(const RestRows& R, int on) {
    return RestRows{of_lane(static_cast<const KvRows&>(R), on), __builtin_amdgcn_readlane(R.skip, on)};
}
__device__ __forceinline__ RestRows rows_of(const AttendRest& A, int s) {
    return RestRows{rows_of(static_cast<const Attend&>(A), s), A.G.skip[s]};
}
__device__ __forceinline__ TileOf<RestRows> tile_of(const AttendRest& A, const RestRows& R, int t) {
    TileOf<RestRows> x;
    x.R = R;
    x.i0 = t * A.TQ;
    x.n = min(R.rows - x.i0, A.TQ);
    const int cap = A.b.max_pages * kKvPage;
    const int p1 = R.first + x.i0 + x.n, hi = min(p1, cap), lo = R.skip * kKvPage;   // positions lo .. hi - 1
    const bool some = hi > 0 && lo < hi;
    x.pg0 = some ? R.skip : 0;
    x.pages = x.n <= 0 ? 0 : some ? (hi - 1) / kKvPage + 1 - x.pg0 : 1;
    return x;
}
__device__ __forceinline__ int ctx_of(const AttendRest&, const TileOf<RestRows>& T) { return T.R.first + T.R.n; }
__device__ __forceinline__ RestOut out_row(const AttendRest& A, const Seg& S, int r) {
    const RowHead h = row_head(A, S, r);
    RestOut x;
    if (h.row < 0) return x;
    x.to = A.out + (int64_t)h.row * A.os + (int64_t)h.head * A.c.head_dim;
    if (A.G.joins[h.row]) x.part = A.G.row_part + row_part_at(A, A.G, h.row, h.head);
    return x;
}
__device__ __forceinline__ void put(const AttendRest& A, const RestOut& x, int c4, f32x4_t o, const Part& a, float) {
    if (c4 >= A.c.head_dim) return;
    Part all = a;
    if (x.part)
        join(all, o, unpacked(*reinterpret_cast<const float4*>(x.part + A.c.head_pad)), *reinterpret_cast<const f32x4_t*>(x.part + c4));
    *reinterpret_cast<uint2*>(x.to + c4) = bf16x4(result(o, inverse(all.sum), all.e));
}

// Splits of the launches, and the workspace (host).
struct SharedPlan {
    prox_kv_batch groups;      // the batch that launch 1 sees
    Split prefix;
    Launches rest;
    bool fits;
    size_t row_part, skip, joins, parts, bytes;
    SharedPlan(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads, int n_groups)
        : groups(b), prefix(), rest(c, b, n_heads) {
        groups.n_seq = n_groups;
        groups.max_q = b.n_tokens;
        // tiles as for groups of the mean size: six groups of 21 tokens in the mean and 7 query heads a key head 37 us,
        // in tiles of twice as many rows 42
        const int64_t usual = (int64_t)((b.n_tokens + n_groups - 1) / n_groups) * (n_heads / c.n_kv);
        prefix = split_of(c, groups, n_heads, b.n_tokens, b.n_tokens, usual);
        fits = prefix.fits && rest.fit() && one_launch(join_blocks(c, b, n_heads), kJoinThreads);
        row_part = align_up(std::max(prefix.bytes, std::max(rest.split[0].bytes, rest.split[1].bytes)), 256);
        skip = row_part + align_up((size_t)b.n_tokens * n_heads * (c.head_pad + 4) * sizeof(float), 256);
        joins = skip + align_up((size_t)b.n_seq * sizeof(int32_t), 256);
        parts = joins + align_up((size_t)b.n_tokens * sizeof(int32_t), 256);
        bytes = parts + align_up((size_t)b.n_tokens * prefix.VH * sizeof(int4), 256);
    }
};

template <typename AT>
hipError_t launch(AT& A, const Split& p, void* workspace, hipStream_t s) {
    A.arrived = static_cast<unsigned long long*>(workspace);
    A.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.part_at);
    set_split(A, p);
    return A.c.kind == PROX_KV_INT8 ? attend_kind<PROX_KV_INT8>(A, p, s) : attend_kind<PROX_KV_FP8>(A, p, s);
}

}  // namespace

size_t kv_shared_workspace(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads, int n_groups) {
    if (b.n_tokens <= 0 || b.max_q <= 0) return 256;
    const SharedPlan P(c, bounded(b), n_heads, n_groups);
    return P.fits ? P.bytes : 0;
}

hipError_t launch_kv_shared(const prox_kv_cache& c, const prox_kv_batch& batch, const int32_t* group_start, int n_groups,
                            const int32_t* shared, const uint16_t* q, int64_t q_stride, int n_heads, float scale,
                            uint16_t* out, int64_t out_stride, void* workspace, hipStream_t s) {
    const prox_kv_batch b = bounded(batch);
    const SharedPlan P(c, b, n_heads, n_groups);
    if (!P.fits) return hipErrorInvalidConfiguration;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const GroupArgs G{group_start, shared, n_groups, b.n_seq, n_heads, P.prefix.blocks, reinterpret_cast<float*>(ws + P.row_part),
                      reinterpret_cast<int32_t*>(ws + P.skip), reinterpret_cast<int32_t*>(ws + P.joins),
                      reinterpret_cast<int4*>(ws + P.parts)};
    AttendPrefix A{};
    set_call(A, c, P.groups, q, q_stride, n_heads, scale, 0, out, out_stride);
    A.G = G;
    hipError_t e = launch(A, P.prefix, workspace, s);
    if (e != hipSuccess) return e;
    const int64_t pairs = (int64_t)b.n_tokens * n_heads;
    const dim3 grid((uint32_t)join_blocks(c, b, n_heads)), threads(kJoinThreads);
    switch (c.head_pad / 64) {
        case 1: hipLaunchKernelGGL((k_kv_join<1>), grid, threads, 0, s, A, pairs); break;
        case 2: hipLaunchKernelGGL((k_kv_join<2>), grid, threads, 0, s, A, pairs); break;
        case 3: hipLaunchKernelGGL((k_kv_join<3>), grid, threads, 0, s, A, pairs); break;
        default: hipLaunchKernelGGL((k_kv_join<4>), grid, threads, 0, s, A, pairs); break;
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    AttendRest B{};
    set_call(B, c, b, q, q_stride, n_heads, scale, 0, out, out_stride);
    B.G = G;
    for (int k = P.rest.few > 0 ? 0 : 1; k < 2; ++k) {
        B.rows_lo = k == 0 ? 1 : P.rest.few + 1;
        B.rows_hi = k == 0 ? P.rest.few : b.max_q;
        e = launch(B, P.rest.split[k], workspace, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace prox
