// Attention over selected pages of the paged key/value cache: for the row at
// position p and a key head
//   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale (q . k_j)
// over the positions j <= p of the pages that a list names, page by page with a
// running maximum (the arithmetic is that of the attention over all pages).
//
// A row, key head and group of up to 16 of its query heads is a unit; its list
// is cut into equal runs of entries, one for each wave of each of its `parts`
// blocks.  The waves of a block meet in LDS; parts of several blocks meet in the
// workspace, where the block that arrives last joins them in order, so results
// do not depend on timing.
//
// What bounds it (kernel times): one token, 64 / 8 heads x 128, 64 pages 11.2 us
// (8.4 MB: latency); 64 ragged sequences, 32 / 8 heads x 128, e4m3, 32 pages 25.5 us
// (105 MB; lists of 12.4 pages in the mean and one block each: those of a page or two
// end after 5.7 us, full ones after 16.7, the last after 24.4, so most CUs are idle in
// the last third); 1000 rows, 28 / 4 heads x 64, 48 pages 133 us: some
// 300 vector instructions for each page and wave, codes to fp16 and weights, of
// whose 16 columns 7 are in use.
#include "prox_kv_attn.hpp"

namespace prox {

namespace {

struct Selected {
    Attend A;
    const int32_t* pages;      // [n_tokens][n_kv][keep]
    int keep, parts;
    int groups;                // head groups of a key head (A.HG heads each)
};

// Entries from .. up - 1 of one row's list, pages of its table all of them, for one
// wave; as Pages, lane i keeps what the table and the scales say of entry base + i.
template <int NP>
struct Listed {
    static constexpr int kBytes = kKvPage * 64 * NP;
    const Attend& A;
    const int32_t *list, *table;
    int first;                     // entry `lane` of the list
    int head, upto, base, at_page, id, ve;
    float ks, vl;
    __device__ __forceinline__ Listed(const Attend& a, const int32_t* lst, int first64, const int32_t* tab, int hd, int from, int up, int l)
        : A(a), list(lst), table(tab), first(first64), head(hd), upto(up) {
        look(from, l);
    }
    __device__ __forceinline__ void look(int e, int l) {
        base = e;
        const int i = min(e + l, upto - 1);
        at_page = upto <= 64 ? __shfl(first, i) : list[i];
        id = table[at_page];
        id = e + l < upto && id >= 0 && id < A.c.n_pages ? id : -1;
        const float k0 = A.c.k_scale[where(id)], v0 = A.c.v_scale[where(id)];
        ks = id >= 0 ? k0 : 0.f;
        const bool some = id >= 0 && v0 > 0.f;
        ve = some ? __builtin_amdgcn_frexp_expf(v0) : kNoUnit;
        vl = kTop + __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(some ? v0 : 1.f));
    }
    __device__ __forceinline__ void follow(int p, int l) {
        if (p + 2 >= base + 64) look(p, l);
    }
    __device__ __forceinline__ int at(int p) const { return __builtin_amdgcn_readlane(id, p - base); }
    __device__ __forceinline__ int base_key(int p) const { return __builtin_amdgcn_readlane(at_page, p - base) * kKvPage; }
    __device__ __forceinline__ float of_page(float x, int p) const {
        return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), p - base));
    }
    __device__ __forceinline__ float k_scale(int p) const { return of_page(ks, p); }
    __device__ __forceinline__ int v_exp(int p) const { return __builtin_amdgcn_readlane(ve, p - base); }
    __device__ __forceinline__ float v_log(int p) const { return of_page(vl, p); }
    __device__ __forceinline__ size_t where(int page) const { return (size_t)max(page, 0) * A.c.n_kv + head; }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t keys(int p) const { return codes(A.c.k, at(p), at(p) >= 0); }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t values(int p) const { return codes(A.c.v, at(p), v_exp(p) != kNoUnit); }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t codes(const void* from, int page, bool there) const {
        return make_rsrc(static_cast<const uint8_t*>(from) + where(page) * kBytes, there ? kBytes : 0);
    }
};

// LDS: [waves][HG][64 NP + 4] floats, the waves' parts.
template <int KIND, int NP, int kWaves>
__global__ void __launch_bounds__(64 * kWaves, NP <= 2 ? 2 : 1) k_kv_selected(Selected S) {
    extern __shared__ __align__(16) float lds[];
    __shared__ int some_s[kWaves];
    __shared__ int last_s;
    constexpr int RW = 64 * NP + 4, LPR = 16 * NP;
    const Attend& A = S.A;
    const int l = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), n = l & 15, g = l >> 4;
    const int unit = (int)(blockIdx.x / (uint32_t)S.parts), part = (int)(blockIdx.x % (uint32_t)S.parts);
    const int row = unit / A.VH, vh = unit - row * A.VH, head = vh / S.groups, h0 = (vh - head * S.groups) * A.HG;
    // the list is on its way while the row's sequence is found
    const int32_t* list = S.pages + ((size_t)row * A.c.n_kv + head) * (size_t)S.keep;
    const int first = list[min(l, S.keep - 1)];
    const int s = kv_seq_find(A.b, row, l), hd = A.c.head_dim;
    const KvRows R = kv_rows(A.b, s);
    if (row < R.q0 || row >= R.q0 + R.rows) return;
    const int pos = R.first + row - R.q0;
    const bool sees = pos >= 0 && pos < A.b.max_pages * kKvPage;
    // entries that count: up to the first that is not above the one before it, or behind the row's own page
    const int own = pos >> 6;
    int count = 0;
    for (int e = 0; sees && count == e && e < S.keep; e += 64) {
        const int i = min(e + l, S.keep - 1), page = e == 0 ? first : list[i];
        const int left = __shfl_up(page, 1), before = l > 0 ? left : e > 0 ? list[e - 1] : -1;
        const uint64_t m = ~__ballot(e + l < S.keep && page > before && page <= own);
        count = e + (m ? __builtin_ctzll(m) : 64);
    }
    const int64_t all = (int64_t)S.parts * kWaves, k = (int64_t)part * kWaves + wv;
    const int from = (int)(count * k / all), upto = (int)(count * (k + 1) / all);
    const bool mine = from < upto;
    if (l == 0) some_s[wv] = mine;
    if (mine) {
        Listed<NP> pages(A, list, first, A.b.block_table + (size_t)s * A.b.max_pages, head, from, upto, l);
        Rows<KIND, NP, 1> w;
        w.live[0] = n < A.HG && h0 + n < A.rep;
        w.key_lo[0] = 0;
        w.key_hi[0] = w.live[0] ? pos + 1 : 0x7fffffff;
        const uint16_t* src = A.q + (int64_t)row * A.qs + (int64_t)(head * A.rep + (w.live[0] ? h0 + n : 0)) * hd;
#pragma unroll
        for (int a = 0; a < NP; ++a)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int ch = 64 * a + 16 * g + 8 * e;
                w.q[0][a][e] = w.live[0] && ch < hd ? *reinterpret_cast<const uint4*>(src + ch) : make_uint4(0, 0, 0, 0);
            }
        walk_pages<KIND, NP, 1>(w, pages, A, R.first + R.n, from, upto, l);
        if (n < A.HG) {
            float* to = lds + (wv * A.HG + n) * RW;
#pragma unroll
            for (int d = 0; d < 4 * NP; ++d) *reinterpret_cast<f32x4_t*>(to + 16 * d + 4 * g) = w.o[0][d];
            if (g == 0) *reinterpret_cast<float4*>(to + 64 * NP) = packed(w.part(0));
        }
    }
    __syncthreads();
    const int lanes = A.HG * LPR;                                   // (head, four channels)
    const __amdgpu_buffer_rsrc_t rp = make_rsrc(A.part, A.part_bytes);
    auto part_at = [&](int p, int r) {
        return ((uint32_t)(unit * S.parts + p) * (uint32_t)A.HG + (uint32_t)r) * (uint32_t)(RW * 4);
    };
    auto store = [&](int e, f32x4_t o, const Part& a) {
        const int r = e / LPR, c4 = 4 * (e % LPR);
        if (h0 + r < A.rep && c4 < hd)
            *reinterpret_cast<uint2*>(A.out + (int64_t)row * A.os + (int64_t)(head * A.rep + h0 + r) * hd + c4) =
                bf16x4(result(o, inverse(a.sum), a.e));
    };
    for (int e = threadIdx.x; e < lanes; e += blockDim.x) {
        const int r = e / LPR, c4 = 4 * (e % LPR);
        Part a = no_part();
        f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const float* at = lds + (i * A.HG + r) * RW;
            if (some_s[i]) join(a, o, unpacked(*reinterpret_cast<const float4*>(at + 64 * NP)), *reinterpret_cast<const f32x4_t*>(at + c4));
        }
        if (S.parts == 1) {
            store(e, o, a);
        } else {
            const uint32_t at = part_at(part, r);
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, o), rp, (int)(at + 4 * c4), 0, kCoherent);
            if (c4 == 0)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, packed(a)), rp, (int)(at + 256 * NP), 0, kCoherent);
        }
    }
    if (S.parts == 1) return;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");               // this wave's stores have completed
    __syncthreads();
    if (wv == 0) {
        const bool last = kv_arrive(A.arrived + (size_t)unit * S.parts, A.tag, part, S.parts, l);
        if (l == 0) last_s = last;
    }
    __syncthreads();
    if (!last_s) return;
    for (int e = threadIdx.x; e < lanes; e += blockDim.x) {
        Part a = no_part();
        f32x4_t o = {0.f, 0.f, 0.f, 0.f};
        for (int p0 = 0; p0 < S.parts; p0 += 8) {
            u32x4_t v[8], ms[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint32_t at = part_at(min(p0 + u, S.parts - 1), e / LPR);
                v[u] = __builtin_amdgcn_raw_buffer_load_b128(rp, (int)(at + 16 * (e % LPR)), 0, kCoherent);
                ms[u] = __builtin_amdgcn_raw_buffer_load_b128(rp, (int)(at + 256 * NP), 0, kCoherent);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (p0 + u < S.parts) join(a, o, unpacked(__builtin_bit_cast(float4, ms[u])), __builtin_bit_cast(f32x4_t, v[u]));
        }
        store(e, o, a);
    }
}

// Waves of a block where there are blocks for every CU twice: shorter prologues and joins among more pages, and
// three blocks a CU (64 channels; 1000 rows of 28 / 4 heads and 48 pages 139 us, with 8 waves 185, with 2 140).
constexpr int kFewWaves = 4;

// How a call is split (host).
struct SelectedSplit {
    int groups, HG, VH, parts, waves;
    int64_t units;
    bool fits;
    size_t part_at, part_bytes, lds, bytes;
};

SelectedSplit selected_split(const prox_kv_cache& c, int n_tokens, int n_heads, int keep) {
    SelectedSplit p;
    const int rep = n_heads / c.n_kv, NP = c.head_pad / 64;
    p.groups = (rep + 15) / 16;
    p.HG = (rep + p.groups - 1) / p.groups;
    p.VH = c.n_kv * p.groups;
    p.units = (int64_t)n_tokens * p.VH;
    p.waves = p.units >= 2 * device_cus() ? kFewWaves : few_waves(NP);
    // enough blocks for the chip, as long as each wave has an entry
    const int64_t want = (device_cus() + p.units - 1) / p.units, most = (keep + p.waves - 1) / p.waves;
    p.parts = (int)std::min(want, most);
    const size_t row = (size_t)(c.head_pad + 4) * sizeof(float);
    p.lds = (size_t)p.waves * p.HG * row;
    p.part_at = align_up((size_t)p.units * p.parts * sizeof(unsigned long long), 256);
    p.part_bytes = p.parts > 1 ? (size_t)p.units * p.parts * p.HG * row : 0;
    p.fits = one_launch(p.units * p.parts, 64 * p.waves);
    p.bytes = align_up(p.parts > 1 ? p.part_at + p.part_bytes : 0, 256) + 256;
    return p;
}

template <int KIND, int NP, int kWaves>
hipError_t selected_launch(const Selected& S, const SelectedSplit& p, hipStream_t s) {
    if (p.lds > 48 * 1024) {
        const hipError_t e = hipFuncSetAttribute((const void*)k_kv_selected<KIND, NP, kWaves>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)p.lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((k_kv_selected<KIND, NP, kWaves>), dim3((uint32_t)(p.units * p.parts)), dim3(64 * kWaves), p.lds, s, S);
    return hipGetLastError();
}

template <int KIND, int NP>
hipError_t selected_np(const Selected& S, const SelectedSplit& p, hipStream_t s) {
    if (p.waves == kFewWaves) return selected_launch<KIND, NP, kFewWaves>(S, p, s);
    return selected_launch<KIND, NP, few_waves(NP)>(S, p, s);
}

template <int KIND>
hipError_t selected_kind(const Selected& S, const SelectedSplit& p, hipStream_t s) {
    switch (S.A.c.head_pad / 64) {
        case 1: return selected_np<KIND, 1>(S, p, s);
        case 2: return selected_np<KIND, 2>(S, p, s);
        case 3: return selected_np<KIND, 3>(S, p, s);
        default: return selected_np<KIND, 4>(S, p, s);
    }
}

}  // namespace

size_t kv_selected_workspace(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads, int keep) {
    if (b.n_tokens <= 0 || b.max_q <= 0) return 256;
    const SelectedSplit p = selected_split(c, b.n_tokens, n_heads, keep);
    return p.fits ? p.bytes : 0;
}

hipError_t launch_kv_selected(const prox_kv_cache& c, const prox_kv_batch& b, const uint16_t* q, int64_t q_stride, int n_heads,
                              const int32_t* pages, int keep, float scale, uint16_t* out, int64_t out_stride,
                              void* workspace, hipStream_t s) {
    const SelectedSplit p = selected_split(c, b.n_tokens, n_heads, keep);
    if (!p.fits) return hipErrorInvalidConfiguration;
    Selected S{};
    Attend& A = S.A;
    set_call(A, c, b, q, q_stride, n_heads, scale, 0, out, out_stride);
    A.arrived = static_cast<unsigned long long*>(workspace);
    A.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.part_at);
    A.part_bytes = (uint32_t)p.part_bytes;
    A.tag = next_call_tag();
    A.HG = p.HG;
    A.VH = p.VH;
    S.pages = pages;
    S.keep = keep;
    S.parts = p.parts;
    S.groups = p.groups;
    return c.kind == PROX_KV_INT8 ? selected_kind<PROX_KV_INT8>(S, p, s) : selected_kind<PROX_KV_FP8>(S, p, s);
}

}  // namespace prox
