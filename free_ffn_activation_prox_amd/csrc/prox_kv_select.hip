// Selection of cache pages by bounds of their keys.
//
// Bounds.  For each page, key head and channel the least and the largest code of
// the page's tokens, int8: lo, hi [2][head_pad].  int8 codes as they are; e4m3
// values v as floor(127 v / 448) and ceil(127 v / 448), so that they still bound
// the channel.  NaN codes count as 0.
//
// Score.  A page's keys k satisfy q . k <= sum_d max(q_d lo_d, q_d hi_d) =
// sum_d (q_d^- lo_d + q_d^+ hi_d): one product over 2 head_pad numbers.  q is
// taken as int8 (unit max|q| / 127, half-even), so the products are whole
// numbers below 2^22 and v_mfma_i32_16x16x64_i8 sums them exactly: which pages
// are kept does not depend on how a kernel orders its sums.  The key of a page
// for the query heads h of a key head is
//   fl32(max_h fl32(dot_h unit_h) page_scale).
#include "prox_kv.hpp"

namespace prox {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}
__device__ __forceinline__ uint32_t pk_min(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}

// Two codes in the low bytes of 16-bit halves -> numbers in the codes' order, 128 for a code of 0.
template <int KIND>
__device__ __forceinline__ uint32_t ordered2(uint32_t w) {
    if constexpr (KIND == PROX_KV_INT8) {
        return w ^ 0x00800080u;
    } else {
        const u16x2_t x = __builtin_bit_cast(u16x2_t, w);
        const u16x2_t size = x & (unsigned short)0x7f, neg = (unsigned short)0 - (x >> (unsigned short)7);   // 0 or 0xffff
        const u16x2_t nan = __builtin_elementwise_max(size, u16x2_t{126, 126}) - (unsigned short)126;       // 1 for a NaN
        const u16x2_t m = size & (nan - (unsigned short)1);
        return __builtin_bit_cast(uint32_t, (u16x2_t)(((m ^ neg) - neg) + (unsigned short)128));
    }
}

// An ordered code as a bound.
template <int KIND>
__device__ __forceinline__ int bound_of(int u, bool upper) {
    if constexpr (KIND == PROX_KV_INT8) {
        return u - 128;
    } else {
        const int m = u < 128 ? 128 - u : u - 128;
        const float v = __builtin_amdgcn_cvt_f32_fp8(u < 128 ? m | 128 : m, 0) * 127.f;   // exact: 11 bits
        // a quotient by 448 = 7 * 64 is a whole number only for 0 and +-448, and else further from one than it is rounded
        const float r = v / 448.f;
        return (int)(upper ? ceilf(r) : floorf(r));
    }
}

struct BoundsArgs {
    prox_kv_cache c;
    prox_kv_batch b;
    int8_t* bounds;
    int pp;               // see page_pairs
};

// One wave for each page that the batch's tokens touch, and key head.  Lane
// (c = l / 16, d = l % 16) reads channels 64 a + 16 c .. + 15 of tokens 16 b + d.
template <int KIND>
__global__ void __launch_bounds__(256) k_kv_bounds(BoundsArgs A, int64_t units) {
    const int l = lane_id(), d = l & 15, hp = A.c.head_pad;
    const int64_t unit = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    if (unit >= units) return;
    const int head = (int)(unit % A.c.n_kv);
    int s, j;
    if (!pair_of(A.b, A.pp, (int)(unit / A.c.n_kv), l, s, j)) return;
    const KvRows R = kv_rows(A.b, s);
    if (R.rows <= 0) return;
    const int cap = A.b.max_pages * kKvPage;
    const int lo = max(R.first, 0), hi = (int)min((int64_t)R.first + R.rows, (int64_t)cap);
    const int pg = lo / kKvPage + j;
    if (hi <= lo || pg * kKvPage >= hi) return;
    const int page = A.b.block_table[(size_t)s * A.b.max_pages + pg];
    if (page < 0 || page >= A.c.n_pages) return;
    const int held = min(hi - pg * kKvPage, kKvPage);            // slots that hold tokens
    const size_t at = (size_t)page * A.c.n_kv + head;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(A.c.k) + at * (size_t)(kKvPage * hp)) + l;
    int8_t* out = A.bounds + at * (size_t)(2 * hp);
    for (int a = 0; a < hp / 64; ++a) {
        uint4 x[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) x[b] = src[(a * 4 + b) * 64];
        uint32_t least[8], most[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            least[i] = 0x00ff00ffu;
            most[i] = 0;
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const bool in = 16 * b + d < held;
            const uint32_t w[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u = ordered2<KIND>((i & 1 ? w[i >> 1] >> 8 : w[i >> 1]) & 0x00ff00ffu);
                least[i] = pk_min(least[i], in ? u : 0x00ff00ffu);
                most[i] = pk_max(most[i], in ? u : 0u);
            }
        }
        // over the 16 lanes of the same channels
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            least[i] = pk_min(least[i], (uint32_t)dpp_ror<8>((int)least[i]));
            least[i] = pk_min(least[i], (uint32_t)dpp_ror<4>((int)least[i]));
            least[i] = pk_min(least[i], (uint32_t)dpp_ror<2>((int)least[i]));
            least[i] = pk_min(least[i], (uint32_t)dpp_ror<1>((int)least[i]));
            most[i] = pk_max(most[i], (uint32_t)dpp_ror<8>((int)most[i]));
            most[i] = pk_max(most[i], (uint32_t)dpp_ror<4>((int)most[i]));
            most[i] = pk_max(most[i], (uint32_t)dpp_ror<2>((int)most[i]));
            most[i] = pk_max(most[i], (uint32_t)dpp_ror<1>((int)most[i]));
        }
        // lane d keeps channel d of the 16: byte d % 4 of dword d / 4
        uint32_t bl = 0, bm = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool mine = (d >> 2) == (i >> 1) && (d & 1) == (i & 1);
            bl = mine ? least[i] : bl;
            bm = mine ? most[i] : bm;
        }
        const int shift = d & 2 ? 16 : 0;
        out[a * 64 + l] = (int8_t)bound_of<KIND>((int)((bl >> shift) & 0xff), false);
        out[hp + a * 64 + l] = (int8_t)bound_of<KIND>((int)((bm >> shift) & 0xff), true);
    }
}

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / kWave;
constexpr int kBins = 256;

struct SelectArgs {
    prox_kv_cache c;
    prox_kv_batch b;
    const uint16_t* q;
    int64_t qs;
    const int8_t* bounds;
    int32_t* pages;
    int keep, first, last;
    int rep;               // query heads of a key head
    int RP;                // columns of a token: rep rounded up to a power of two, 16 at most
    int TQ;                // tokens of a block
    int row_pages;         // keys of a token in LDS (a multiple of 16)
};

// The tile-th group of TQ rows of the batch's sequences: sequence and first row
// in it, found by a whole wave at once; false behind the last one.
__device__ __forceinline__ bool tile_at(const prox_kv_batch& b, int TQ, int tile, int lane, int& s, int& i0) {
    if (!b.q_start) {
        s = tile;
        i0 = 0;
        return tile < b.n_seq;
    }
    for (int base = 0; base < b.n_seq; base += 64) {
        int upto = base + lane < b.n_seq ? (max(kv_rows(b, base + lane).rows, 0) + TQ - 1) / TQ : 0;
        const int n = upto;
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
            const int u = __shfl_up(upto, m);
            if (lane >= m) upto += u;
        }
        const uint64_t m = __ballot(upto > tile);
        if (m) {
            const int on = __builtin_ctzll(m);
            s = base + on;
            i0 = (tile - (__builtin_amdgcn_readlane(upto, on) - __builtin_amdgcn_readlane(n, on))) * TQ;
            return true;
        }
        tile -= __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

constexpr uint32_t kNotThere = 0u, kForced = 0xffffffffu;
// A key as a number that grows with it; NaN below all others.
__device__ __forceinline__ uint32_t ordered_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);                 // -0 as 0
    return x != x ? 1u : (u & 0x80000000u ? ~u : u | 0x80000000u);
}

// The largest of v over groups of RP lanes.
__device__ __forceinline__ float over_columns_max(float v, int RP) {
    if (RP > 1) v = fmaxf(v, __shfl_xor(v, 1));
    if (RP > 2) v = fmaxf(v, __shfl_xor(v, 2));
    if (RP > 4) v = fmaxf(v, __shfl_xor(v, 4));
    if (RP > 8) v = fmaxf(v, __shfl_xor(v, 8));
    return v;
}

// A block: up to TQ rows of one sequence, one key head.
// LDS: keys [TQ][row_pages] (fp32 maxima over heads, then ordered keys), q's
// codes as operands [2 hp / 16][16 columns][16], bins [TQ][256].
// Columns: token i, query head h of a group of up to RP at i RP + h; columns
// beyond the last head hold the group's first one again.
__global__ void __launch_bounds__(kSelThreads) k_kv_select(SelectArgs A) {
    extern __shared__ __align__(16) uint32_t lds[];
    __shared__ float unit_s[16];
    __shared__ int count_s[kSelWaves][2];
    __shared__ int bin_s[16][2];
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave), n16 = l & 15, g = l >> 4;
    const int hp = A.c.head_pad, hd = A.c.head_dim, TQ = A.TQ, RP = A.RP;
    const int tile = blockIdx.x / A.c.n_kv, head = blockIdx.x % A.c.n_kv;
    int s, i0;
    if (!tile_at(A.b, TQ, tile, l, s, i0)) return;
    const KvRows R = kv_rows(A.b, s);
    const int rows = min(R.rows - i0, TQ);
    if (rows <= 0) return;
    uint32_t* const keys = lds;
    uint32_t* const q8 = lds + TQ * A.row_pages;
    uint32_t* const bins = q8 + 2 * hp * 4;
    const int32_t* table = A.b.block_table + (size_t)s * A.b.max_pages;
    // pages that row i sees: 0 for a position that does not exist
    auto sees = [&](int i) {
        const int pos = R.first + i0 + i;
        return i < rows && pos >= 0 && pos < A.b.max_pages * kKvPage ? pos / kKvPage + 1 : 0;
    };
    int most = 0;
    for (int i = 0; i < rows; ++i) most = max(most, sees(i));
    const bool all = most <= A.keep;                              // every page is kept: no scores

    for (int h0 = 0; !all && h0 < A.rep; h0 += 16) {
        // column w: q's codes
        __syncthreads();
        {
            const int i = min(w / RP, rows - 1), h = w % RP + h0 < A.rep ? w % RP + h0 : h0;
            const uint16_t* src = A.q + (int64_t)(R.q0 + i0 + i) * A.qs + (int64_t)(head * A.rep + h) * hd;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (4 * l < hd) {
                const uint2 u = *reinterpret_cast<const uint2*>(src + 4 * l);
                x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
            }
            int big = 0;                                          // bits of the largest finite size
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int b = (int)(__float_as_uint(x[e]) & 0x7fffffffu);
                big = max(big, b < 0x7f800000 ? b : 0);
            }
            const float unit = __int_as_float(wave_max(big)) / 127.f, by = unit > 0.f ? unit : 1.f;
            uint32_t up = 0, down = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float r = x[e] / by;
                const int c = x[e] == x[e] ? (int)rintf(fminf(fmaxf(r, -127.f), 127.f)) : 0;
                up |= (uint32_t)max(c, 0) << (8 * e);
                down |= ((uint32_t)min(c, 0) & 0xffu) << (8 * e);
            }
            if (4 * l < hp) {
                q8[(l / 4 * 16 + w) * 4 + l % 4] = down;
                q8[((hp + 4 * l) / 16 * 16 + w) * 4 + l % 4] = up;
            }
            if (l == 0) unit_s[w] = unit;
        }
        __syncthreads();
        const float unit = unit_s[n16];
        for (int p0 = 16 * w; p0 < most; p0 += 16 * kSelWaves) {
            const int p = p0 + n16, id = p < most ? table[p] : -1;
            const bool there = id >= 0 && id < A.c.n_pages;
            const int8_t* src = A.bounds + ((size_t)(there ? id : 0) * A.c.n_kv + head) * (size_t)(2 * hp) + 16 * g;
            i32x4_t dot = {0, 0, 0, 0};
            for (int k = 0; k < 2 * hp / 64; ++k) {
                const i32x4_t a = *reinterpret_cast<const i32x4_t*>(src + 64 * k);
                const i32x4_t b = *reinterpret_cast<const i32x4_t*>(q8 + ((4 * k + g) * 16 + n16) * 4);
                dot = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, dot, 0, 0, 0);
            }
            float4 v;
            v.x = over_columns_max((float)dot[0] * unit, RP);
            v.y = over_columns_max((float)dot[1] * unit, RP);
            v.z = over_columns_max((float)dot[2] * unit, RP);
            v.w = over_columns_max((float)dot[3] * unit, RP);
            if (n16 % RP == 0 && n16 / RP < rows) {
                float4* to = reinterpret_cast<float4*>(keys + n16 / RP * A.row_pages + p0 + 4 * g);
                if (h0 > 0) {
                    const float4 o = *to;
                    v = make_float4(fmaxf(o.x, v.x), fmaxf(o.y, v.y), fmaxf(o.z, v.z), fmaxf(o.w, v.w));
                }
                *to = v;
            }
        }
    }
    __syncthreads();

    // Teams of waves, one for each row: what follows goes on in all of them at once.
    const int TW = kSelWaves / TQ, team = w / TW, tw = w % TW, t = tw * kWave + l, NT = TW * kWave;
    const int n = sees(team);
    uint32_t* const key = keys + team * A.row_pages;
    uint32_t* const bin = bins + team * kBins;
    // ordered keys
    for (int p = t; p < n; p += NT) {
        const int id = table[p];
        const bool there = id >= 0 && id < A.c.n_pages;
        uint32_t u = kForced;
        if (!(p < A.first || p >= n - A.last) && n > A.keep)
            u = ordered_key(__uint_as_float(key[p]) * A.c.k_scale[(size_t)(there ? id : 0) * A.c.n_kv + head]);
        key[p] = there ? u : kNotThere;
    }
    // The keep-th largest key, eight bits at a time: `prefix` its bits so far,
    // `need` how many keys that share them are kept.
    uint32_t prefix = 0;
    int need = A.keep;
    if (!all) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = t; i < kBins; i += NT) bin[i] = 0;
            __syncthreads();
            if (n > A.keep)
                for (int p = t; p < n; p += NT)
                    if (shift == 24 || key[p] >> (shift + 8) == prefix) atomicAdd(bin + (key[p] >> shift & 255), 1u);
            __syncthreads();
            if (tw == 0) {
                // lane l: bins 255 - 4 l .. 252 - 4 l, from the top
                const uint4 c = *reinterpret_cast<const uint4*>(bin + 252 - 4 * l);
                const int mine = (int)(c.x + c.y + c.z + c.w), upto = (int)wave_incl_scan((uint32_t)mine), above = upto - mine;
                if (above < need && need <= upto) {
                    int at = 255 - 4 * l, over = above;
                    const int each[4] = {(int)c.w, (int)c.z, (int)c.y, (int)c.x};
                    bool on = true;
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        on = on && need > over + each[i];
                        if (on) {
                            over += each[i];
                            --at;
                        }
                    }
                    bin_s[team][0] = at;
                    bin_s[team][1] = over;
                }
            }
            __syncthreads();
            if (n > A.keep) {
                prefix = prefix << 8 | (uint32_t)bin_s[team][0];
                need -= bin_s[team][1];
            }
        }
    } else {
        __syncthreads();
    }
    // Kept: keys above it, and the first `need` of those equal to it.  A wave
    // counts those of its part of the pages, then writes them in order.
    const bool some = n > A.keep;
    const int part = (n + TW * kWave - 1) / (TW * kWave) * kWave, lo = min(tw * part, n), hi = min(lo + part, n);
    int above = 0, equal = 0;
    for (int p = lo; p < hi; p += kWave) {
        const uint32_t u = p + l < hi ? key[p + l] : kNotThere;
        above += __popcll(__ballot(u != kNotThere && (!some || u > prefix)));
        equal += __popcll(__ballot(some && u != kNotThere && u == prefix));
    }
    if (l == 0) {
        count_s[w][0] = above;
        count_s[w][1] = equal;
    }
    __syncthreads();
    if (team >= rows) return;
    int at = 0, eq = 0, total = 0, all_eq = 0;
    for (int i = 0; i < TW; ++i) {
        const int a = count_s[team * TW + i][0], e = count_s[team * TW + i][1];
        if (i < tw) {
            at += a + min(e, max(need - all_eq, 0));
            eq += e;
        }
        total += a + min(e, max(need - all_eq, 0));
        all_eq += e;
    }
    int32_t* out = A.pages + ((size_t)(R.q0 + i0 + team) * A.c.n_kv + head) * (size_t)A.keep;
    for (int p = lo; p < hi; p += kWave) {
        const uint32_t u = p + l < hi ? key[p + l] : kNotThere;
        const uint64_t same = __ballot(some && u != kNotThere && u == prefix);
        const bool kept = u != kNotThere && (!some || u > prefix || (u == prefix && eq + lanes_below(same) < need));
        const uint64_t m = __ballot(kept);
        if (kept) out[at + lanes_below(m)] = p + l;
        at += __popcll(m);
        eq += __popcll(same);
    }
    for (int i = total + t; i < A.keep; i += NT) out[i] = -1;
}

int pow2_up(int v) {
    int p = 1;
    while (p < v) p *= 2;
    return p;
}

}  // namespace

hipError_t launch_kv_bounds(const prox_kv_cache& c, const prox_kv_batch& b, int8_t* bounds, hipStream_t s) {
    BoundsArgs A{c, b, bounds, 0};
    const int64_t units = page_pairs(b, A.pp) * c.n_kv, blocks = (units + 3) / 4;
    if (blocks > 0x7fffffffll || units / c.n_kv > 0x7fffffffll) return hipErrorInvalidConfiguration;
    if (c.kind == PROX_KV_INT8) hipLaunchKernelGGL((k_kv_bounds<PROX_KV_INT8>), dim3((uint32_t)blocks), dim3(256), 0, s, A, units);
    else hipLaunchKernelGGL((k_kv_bounds<PROX_KV_FP8>), dim3((uint32_t)blocks), dim3(256), 0, s, A, units);
    return hipGetLastError();
}

hipError_t launch_kv_select(const prox_kv_cache& c, const prox_kv_batch& b, const uint16_t* q, int64_t q_stride, int n_heads,
                            const int8_t* bounds, int keep, int first, int last, int32_t* pages, hipStream_t s) {
    SelectArgs A{c, b, q, q_stride, bounds, pages, keep, first, last, n_heads / c.n_kv, 0, 0, 0};
    A.RP = std::min(pow2_up(A.rep), 16);
    A.row_pages = (b.max_pages + 15) / 16 * 16;
    // several rows of a sequence share the pages' bounds, as far as their keys fit in LDS
    const int max_q = std::max(std::min(b.q_start ? b.max_q : 1, b.n_tokens), 1);
    A.TQ = std::min(16 / A.RP, pow2_up(max_q));
    auto lds = [&] { return ((size_t)A.TQ * (A.row_pages + kBins) + 2 * (size_t)c.head_pad * 4) * sizeof(uint32_t); };
    while (A.TQ > 1 && lds() > 72 * 1024) A.TQ /= 2;
    const int64_t tiles = b.q_start ? std::min((int64_t)b.n_seq * ((max_q - 1) / A.TQ + 1), (int64_t)b.n_tokens / A.TQ + b.n_seq)
                                    : b.n_seq;
    const int64_t blocks = tiles * c.n_kv;
    if (blocks > 0x7fffffffll) return hipErrorInvalidConfiguration;
    if (lds() > 48 * 1024) {
        const hipError_t e = hipFuncSetAttribute((const void*)k_kv_select, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds());
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k_kv_select, dim3((uint32_t)blocks), dim3(kSelThreads), lds(), s, A);
    return hipGetLastError();
}

}  // namespace prox
