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
//
// What bounds it (kernel times): bounds of 32768 tokens and 8 heads of 128 channels
// 9.0 us (34.6 MB, 3.8 TB/s: a wave's loads of 4 KB wait for the reduction of the 4 KB
// before them).  Selection is a chain of loads (row, table, bounds) and of steps of
// one wave.  32 of up to 512 pages for 64 ragged sequences 14.5 us (7.3 MB): those of
// the longest rows, which have one block each (stamps: rows and table 0.6, keys of 33
// to 128 pages 4.1, of 129 to 320 7.6, of more 10.2, none where all pages are kept,
// selection 1.2 to 1.8).  48 of 250 pages for 1000 rows of 28 / 4 heads 24.0 us, two
// rounds of blocks of 10.7 (rows 1.7, keys 7.9, selection 1.6).  For one token 64 of
// 2048 pages 7.9 + 9.3 us (4.3 MB; in one launch of 8 blocks 31, of which a CU's
// 30 GB/s take 15).
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

constexpr int kSelThreads = 256;
constexpr int kLeastRun = 128;      // least pages of a block, where a tile has several
// Blocks for each CU that a launch is cut into where it can be, by a second launch that selects: one row of 8 heads
// and 2048 pages 15.3 us, in 8 blocks that select by themselves 31; 512 rows and heads of up to 512 pages 18.8 us in
// four times as many, 14.9 in blocks that select by themselves.
constexpr int kBlocksPerCu = 1;
constexpr int kSelBins = 2048;      // of the block's selection (LDS words, with some to spare for its counts)
constexpr int kSelScratch = 64;

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
    int row_pages;         // keys of a token in LDS (a multiple of 64)
    int parts;             // blocks of a tile of tokens and key head; with several their keys go to
    uint32_t* keys;        // [tiles][n_kv][TQ][row_pages] in the workspace
};

// The tile-th group of TQ rows of the batch's sequences: sequence and first row
// in it, found by a whole wave at once; false behind the last one.
__device__ __forceinline__ bool tile_at(const prox_kv_batch& b, int TQ, int tile, int lane, int& s, int& i0) {
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

// fp32 numbers (no NaN) as whole numbers in the same order, and back.
__device__ __forceinline__ int in_order(float x) {
    const int b = __float_as_int(x);
    return b ^ (int)((uint32_t)(b >> 31) >> 1);
}
__device__ __forceinline__ float from_order(int o) { return __int_as_float(o ^ (int)((uint32_t)(o >> 31) >> 1)); }

// The largest of v over groups of RP lanes: pairs, quads, halves of a row of 16, the row.
template <int CTRL>
__device__ __forceinline__ int dpp_max(int v) {
    return max(v, __builtin_amdgcn_update_dpp(v, v, CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ int over_columns_max(int v, int RP) {
    if (RP > 1) v = dpp_max<0xb1>(v);
    if (RP > 2) v = dpp_max<0x4e>(v);
    if (RP > 4) v = dpp_max<0x141>(v);
    if (RP > 8) v = dpp_max<0x140>(v);
    return v;
}

// Ordered keys of the pages from .. most - 1 (from: a multiple of 64) of up to TQ rows, into LDS.
// Columns of the product: token i, query head h of a group of up to RP at
// i RP + h; columns beyond the last head hold the group's first one again.
// LDS: q's codes as operands [2 hp / 16][16 columns][16], the columns' units.
template <int NP, int NT>
__device__ __forceinline__ void page_keys(const SelectArgs& A, uint32_t* keys, uint32_t* q8, float* unit_s, const KvRows& R,
                                          int head, int i0, int rows, const int32_t* table, int from, int most) {
    constexpr int kWaves = NT / kWave, HP = 64 * NP, K = 2 * NP;     // K: products of 64 for a page
    constexpr int U = 2;                               // groups of 16 pages whose bounds are on their way together
    constexpr int kColumns = (16 + kWaves - 1) / kWaves;             // columns whose q a wave turns to codes
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave), n16 = l & 15, g = l >> 4;
    const int hd = A.c.head_dim, RP = A.RP;
    const int mine = min(n16 / RP, rows - 1);                        // this column's token
    float* const scale_s = reinterpret_cast<float*>(q8 + 8 * HP) + w * 16 * U;   // scales of the wave's pages; NaN of kGone: no page
    constexpr uint32_t kGone = 0xffffffffu;
    i32x4_t a[U][K];
    float scale[U];
    auto load = [&](int p0) {
        int id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = table[min(p0 + 16 * u + n16, most - 1)];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool there = p0 + 16 * u + n16 < most && id[u] >= 0 && id[u] < A.c.n_pages;
            const size_t at = (size_t)(there ? id[u] : 0) * A.c.n_kv + head;
            const int8_t* src = A.bounds + at * (size_t)(2 * HP) + 16 * g;
#pragma unroll
            for (int k = 0; k < K; ++k) a[u][k] = *reinterpret_cast<const i32x4_t*>(src + 64 * k);
            const float sc = A.c.k_scale[at];
            scale[u] = there ? (sc == sc ? sc : __builtin_nanf("")) : __uint_as_float(kGone);
        }
    };
    const int p_first = from + 16 * U * w;
    for (int h0 = 0; h0 < A.rep; h0 += 16) {
        uint2 x2[kColumns];
#pragma unroll
        for (int k = 0; k < kColumns; ++k) {
            const int c = w + k * kWaves, h = c % RP + h0 < A.rep ? c % RP + h0 : h0;
            const uint16_t* src = A.q + (int64_t)(R.q0 + i0 + min(c / RP, rows - 1)) * A.qs + (int64_t)(head * A.rep + h) * hd;
            x2[k] = 4 * l < hd ? *reinterpret_cast<const uint2*>(src + 4 * l) : make_uint2(0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);                           // q first: it is turned to codes while the bounds come
        if (p_first < most) load(p_first);
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kColumns; ++k) {
            const int c = w + k * kWaves;
            const float x[4] = {bf16_lo(x2[k].x), bf16_hi(x2[k].x), bf16_lo(x2[k].y), bf16_hi(x2[k].y)};
            int big = 0, sizes = 0;                                  // bits of the largest finite size, and of any
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int b = (int)(__float_as_uint(x[e]) & 0x7fffffffu);
                big = max(big, b < 0x7f800000 ? b : 0);
                sizes = max(sizes, b);
            }
            const float unit = __int_as_float(wave_max(big)) / 127.f;
            const Quotient<PROX_KV_INT8> by(unit, sizes < 0x7f800000);
            uint32_t codes;
            if (by.tame) {
                codes = by.tame4(x);
            } else {
                float r[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) r[e] = x[e] / by.unit;
                codes = kv_codes4<PROX_KV_INT8>(r);
            }
            const uint32_t neg = (codes >> 7 & 0x01010101u) * 0xffu, up = codes & ~neg, down = codes & neg;
            if (4 * l < HP) {
                q8[(l / 4 * 16 + c) * 4 + l % 4] = down;
                q8[((HP + 4 * l) / 16 * 16 + c) * 4 + l % 4] = up;
            }
            if (l == 0) unit_s[c] = unit;
        }
        __syncthreads();
        const float unit = unit_s[n16];
        const bool final = h0 + 16 >= A.rep;
        for (int p0 = p_first; p0 < most; p0 += 16 * U * kWaves) {
            i32x4_t dot[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                dot[u] = i32x4_t{0, 0, 0, 0};
                if (g == 0) scale_s[16 * u + n16] = scale[u];
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const i32x4_t b = *reinterpret_cast<const i32x4_t*>(q8 + ((4 * k + g) * 16 + n16) * 4);
#pragma unroll
                for (int u = 0; u < U; ++u) dot[u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][k], b, dot[u], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (p0 + 16 * U * kWaves < most) load(p0 + 16 * U * kWaves);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                int t[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) t[r] = over_columns_max(in_order((float)dot[u][r] * unit), RP);
                if (n16 % RP == 0 && n16 / RP < rows) {              // pages p0 + 16 u + 4 g .. + 3 of this column's token
                    uint4* to = reinterpret_cast<uint4*>(keys + mine * A.row_pages + p0 + 16 * u + 4 * g);
                    if (h0 > 0) {
                        const uint4 o = *to;
                        t[0] = max(t[0], (int)o.x); t[1] = max(t[1], (int)o.y); t[2] = max(t[2], (int)o.z); t[3] = max(t[3], (int)o.w);
                    }
                    *to = make_uint4((uint32_t)t[0], (uint32_t)t[1], (uint32_t)t[2], (uint32_t)t[3]);
                }
            }
            if (!final) continue;
            // the maxima to keys, a page a lane (a short loop: code that is not there yet takes longer than it runs)
            const int p = p0 + l % (16 * U);
            const float sc = scale_s[l % (16 * U)];
#pragma nounroll
            for (int i = 0; i < rows; ++i) {
                const int pos = R.first + i0 + i, n = pos >= 0 && pos < A.b.max_pages * kKvPage ? pos / kKvPage + 1 : 0;
                uint32_t* to = keys + i * A.row_pages + p;
                const bool forced = n <= A.keep || p < A.first || p >= n - A.last;
                const uint32_t v = ordered_key(from_order((int)*to) * sc);
                if (l < 16 * U) *to = __float_as_uint(sc) == kGone || p >= n ? kNotThere : forced ? kForced : v;
            }
        }
    }
}

// Over the wave; 0x80000000 turns the order of unsigned numbers into that of signed ones.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) { return (uint32_t)wave_max((int)(v ^ 0x80000000u)) ^ 0x80000000u; }
__device__ __forceinline__ uint32_t wave_min_u32(uint32_t v) { return ~wave_max_u32(~v); }

// The pages of keys above T, and the first `equal` of those equal to it.
struct Kept {
    uint32_t T;
    int equal;
};

// What this wave wrote to LDS is there for all of its lanes.
__device__ __forceinline__ void wave_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// One wave's own row: up to 64 R keys, key R lane + r in register r (kNotThere
// behind the last).  The keys between the least and the largest one are counted in
// 64 R equal ranges, and again those of the range that holds the keep-th largest,
// until a range's border divides them.  bins: 64 R words of the wave's own.
template <int R>
__device__ __forceinline__ void select_wave(const uint32_t (&k)[R], int keep, int32_t* out, uint32_t* bins, int l) {
    constexpr int kBits = R == 4 ? 8 : R == 8 ? 9 : 11;
    static_assert(64 * R == 1 << kBits, "as many ranges as keys");
    uint32_t lo = ~0u, hi = 0;
    int there = 0, forced = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = k[r] != kNotThere && k[r] != kForced;
        there += k[r] != kNotThere ? 1 : 0;
        forced += k[r] == kForced ? 1 : 0;
        lo = min(lo, in ? k[r] : ~0u);
        hi = max(hi, in ? k[r] : 0u);
    }
    // counts up to 2^11 each
    const uint32_t both = (uint32_t)__builtin_amdgcn_readlane((int)wave_incl_scan((uint32_t)there | (uint32_t)forced << 16), 63);
    Kept kept{kNotThere, 0};                                         // every page that is there
    if ((int)(both & 0xffffu) > keep) {
        lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)wave_min_u32(lo));
        hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)wave_max_u32(hi));
        int need = keep - (int)(both >> 16);
        kept.T = kForced - 1u;
        while (need > 0) {
            const int bits = hi > lo ? 32 - __builtin_clz(hi - lo) : 0, shift = max(bits - kBits, 0);
#pragma unroll
            for (int i = 0; i < R / 4; ++i) reinterpret_cast<uint4*>(bins)[64 * i + l] = make_uint4(0, 0, 0, 0);
            wave_lds();
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (k[r] >= lo && k[r] <= hi) atomicAdd(bins + ((k[r] - lo) >> shift), 1u);
            wave_lds();
            // lane l: the R ranges from 64 R - 1 - l R downwards
            uint32_t c[R];
#pragma unroll
            for (int i = 0; i < R / 4; ++i) {
                const uint4 b = *reinterpret_cast<const uint4*>(bins + (63 - l) * R + 4 * i);
                c[4 * i] = b.x; c[4 * i + 1] = b.y; c[4 * i + 2] = b.z; c[4 * i + 3] = b.w;
            }
            int sum = 0;
#pragma unroll
            for (int i = 0; i < R; ++i) sum += (int)c[i];
            const int upto = (int)wave_incl_scan((uint32_t)sum);
            const uint64_t reach = __ballot(upto >= need);
            const int on = __builtin_ctzll(reach);                   // (need keys are there: some lane reaches it)
            int above = upto - sum, digit = 0, in = 0;               // of the lane's ranges from the top
            bool found = false;
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                const bool here = !found && above + (int)c[i] >= need;
                digit = here ? i : digit;
                in = here ? (int)c[i] : in;
                found = found || here;
                above += found ? 0 : (int)c[i];
            }
            digit = __builtin_amdgcn_readlane(digit, on) + (63 - on) * R;
            need -= __builtin_amdgcn_readlane(above, on);
            in = __builtin_amdgcn_readlane(in, on);
            lo += (uint32_t)digit << shift;
            hi = lo + min(hi - lo, (1u << shift) - 1u);
            kept.T = lo - 1u;                                        // (keys that are there are 1 at least)
            if (in == need) break;
            if (shift == 0) {
                kept.T = lo;
                kept.equal = need;
                break;
            }
        }
    }
    // places in the list: those of the lanes before, then of this lane's keys
    int above = 0, same = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        above += k[r] > kept.T ? 1 : 0;
        same += k[r] == kept.T ? 1 : 0;
    }
    int before = (int)wave_incl_scan((uint32_t)above | (uint32_t)same << 16);
    const int all = __builtin_amdgcn_readlane(before, 63);
    int eq = (before >> 16 & 0xffff) - same;                         // keys equal to T before
    int at = (before & 0xffff) - above + min(eq, kept.equal);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = k[r] > kept.T || (k[r] == kept.T && eq < kept.equal);
        eq += k[r] == kept.T ? 1 : 0;
        if (in) out[at] = R * l + r;
        at += in ? 1 : 0;
    }
    const int total = (all & 0xffff) + min(all >> 16 & 0xffff, kept.equal);
    for (int i = total + l; i < keep; i += kWave) out[i] = -1;
}

// One row by the whole block, keys in LDS: the keys between the least and the
// largest one are counted in 2048 equal ranges, and again those of the range that
// holds the keep-th largest, until a range's border divides them.
template <int NT>
__device__ __forceinline__ void select_block(const uint32_t* key, int n, int keep, int32_t* out, uint32_t* bins, int* sc) {
    constexpr int kWaves = NT / kWave;
    const int l = lane_id(), w = threadIdx.x / kWave;
    uint32_t lo = ~0u, hi = 0;
    int forced = 0, there = 0;
    for (int p0 = 0; p0 < n; p0 += NT) {
        const int p = p0 + (int)threadIdx.x;
        const uint32_t u = p < n ? key[p] : kNotThere;
        forced += __popcll(__ballot(u == kForced));
        there += __popcll(__ballot(u != kNotThere));
        if (u != kNotThere && u != kForced) {
            lo = min(lo, u);
            hi = max(hi, u);
        }
    }
    lo = wave_min_u32(lo);
    hi = wave_max_u32(hi);
    __syncthreads();
    if (l == 0) {
        bins[4 * w] = lo;
        bins[4 * w + 1] = hi;
        bins[4 * w + 2] = (uint32_t)forced;
        bins[4 * w + 3] = (uint32_t)there;
    }
    __syncthreads();
    forced = there = 0;
    for (int i = 0; i < kWaves; ++i) {
        lo = min(lo, bins[4 * i]);
        hi = max(hi, bins[4 * i + 1]);
        forced += (int)bins[4 * i + 2];
        there += (int)bins[4 * i + 3];
    }
    Kept kept{kNotThere, 0};
    if (there > keep) {
        int need = keep - forced;
        kept.T = kForced - 1;
        while (need > 0) {
            const int bits = hi > lo ? 32 - __builtin_clz(hi - lo) : 0, shift = max(bits - 11, 0);
            __syncthreads();
            for (int i = threadIdx.x; i < kSelBins; i += NT) bins[i] = 0;
            __syncthreads();
            for (int p = threadIdx.x; p < n; p += NT) {
                const uint32_t u = key[p];
                if (u >= lo && u <= hi) atomicAdd(bins + ((u - lo) >> shift), 1u);
            }
            __syncthreads();
            uint32_t digit;
            int above;
            find_bin<NT>(bins, kSelBins, need, sc, digit, above);
            const int in = (int)bins[digit];
            need -= above;
            lo += digit << shift;
            hi = lo + min(hi - lo, (1u << shift) - 1u);
            kept.T = lo - 1;                                         // (keys that are there are 1 at least)
            if (in == need) break;
            if (shift == 0) {
                kept.T = lo;
                kept.equal = need;
                break;
            }
        }
    }
    // a wave counts those of its part of the pages, then writes them in order
    const int part = (n + NT - 1) / NT * kWave, from = min(w * part, n), upto = min(from + part, n);
    int above = 0, equal = 0;
    for (int p = from; p < upto; p += kWave) {
        const uint32_t u = p + l < upto ? key[p + l] : kNotThere;
        above += __popcll(__ballot(u > kept.T));
        equal += __popcll(__ballot(u == kept.T && u != kNotThere));
    }
    __syncthreads();
    if (l == 0) {
        bins[2 * w] = (uint32_t)above;
        bins[2 * w + 1] = (uint32_t)equal;
    }
    __syncthreads();
    int at = 0, eq = 0, total = 0, all_eq = 0;
    for (int i = 0; i < kWaves; ++i) {
        const int a = (int)bins[2 * i], e = (int)bins[2 * i + 1], kept_here = a + min(e, max(kept.equal - all_eq, 0));
        if (i < w) {
            at += kept_here;
            eq += e;
        }
        total += kept_here;
        all_eq += e;
    }
    for (int p = from; p < upto; p += kWave) {
        const uint32_t u = p + l < upto ? key[p + l] : kNotThere;
        const uint64_t same = __ballot(u == kept.T && u != kNotThere);
        const bool in = u > kept.T || (((same >> l) & 1) && eq + lanes_below(same) < kept.equal);
        const uint64_t m = __ballot(in);
        if (in) out[at + lanes_below(m)] = p + l;
        at += __popcll(m);
        eq += __popcll(same);
    }
    for (int i = total + (int)threadIdx.x; i < keep; i += NT) out[i] = -1;
}

// A tile of up to TQ rows of one sequence, and a key head: what a block knows of it.
struct SelectTile {
    KvRows R;
    int head, i0, rows;
    int most;                  // pages that its last row sees
    const int32_t* table;
    __device__ __forceinline__ SelectTile(const SelectArgs& A, int unit, int l) : head(unit % A.c.n_kv), i0(0), rows(0), most(0), table(nullptr) {
        int s;
        const int tile = unit / A.c.n_kv;
        if (A.TQ == 1) {                                             // tiles are rows
            s = kv_seq_find(A.b, tile, l);
            R = kv_rows(A.b, s);
            i0 = tile - R.q0;
            rows = i0 >= 0 && i0 < R.rows ? 1 : 0;
        } else {
            if (!tile_at(A.b, A.TQ, tile, l, s, i0)) return;
            R = kv_rows(A.b, s);
            rows = min(R.rows - i0, A.TQ);
        }
        table = A.b.block_table + (size_t)s * A.b.max_pages;
        for (int i = 0; i < rows; ++i) most = max(most, sees(A, i));
    }
    // pages that row i sees: 0 for a position that does not exist
    __device__ __forceinline__ int sees(const SelectArgs& A, int i) const {
        const int pos = R.first + i0 + i;
        return pos >= 0 && pos < A.b.max_pages * kKvPage ? pos / kKvPage + 1 : 0;
    }
    __device__ __forceinline__ int32_t* out(const SelectArgs& A, int i) const {
        return A.pages + ((size_t)(R.q0 + i0 + i) * A.c.n_kv + head) * (size_t)A.keep;
    }
};

// Selects for the rows of a tile, keys(row, page) giving the keys of four pages,
// any where it is not below row_pages; each wave of
// the block, or for rows of more than 2048 pages (R 0) the block together.
// LDS: R > 0: [waves][64 R], else keys [row_pages], then bins and scratch.
template <int R, typename F>
__device__ __forceinline__ void select_rows(const SelectArgs& A, const SelectTile& t, uint32_t* lds, int w, int waves, int l, F keys) {
    if constexpr (R > 0) {
        for (int i = w; i < t.rows; i += waves) {
            const int n = t.sees(A, i);
            uint32_t k[R];
#pragma unroll
            for (int r = 0; r < R; r += 4) {
                const uint4 u = keys(i, R * l + r);
                k[r] = u.x; k[r + 1] = u.y; k[r + 2] = u.z; k[r + 3] = u.w;
            }
#pragma unroll
            for (int r = 0; r < R; ++r) k[r] = R * l + r < n ? k[r] : kNotThere;
            select_wave<R>(k, A.keep, t.out(A, i), lds + w * 64 * R, l);
        }
    } else {
        const int n = t.sees(A, 0);
        for (int p = 4 * (int)threadIdx.x; p < n; p += 4 * kSelThreads) *reinterpret_cast<uint4*>(lds + p) = keys(0, p);
        __syncthreads();
        uint32_t* const bins = lds + A.row_pages;
        select_block<kSelThreads>(lds, n, A.keep, t.out(A, 0), bins, reinterpret_cast<int*>(bins + kSelBins));
    }
}

// Every page that is there is kept: no scores.
__device__ __forceinline__ uint4 keys_of_all(const SelectArgs& A, const SelectTile& t, int p) {
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int id = t.table[min(p + e, A.b.max_pages - 1)];
        v[e] = id >= 0 && id < A.c.n_pages ? kForced : kNotThere;
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}
// Four keys of a row of the tile's, in LDS or in the workspace.
__device__ __forceinline__ uint4 keys_of(const SelectArgs& A, const uint32_t* keys, int i, int p) {
    return *reinterpret_cast<const uint4*>(keys + i * A.row_pages + min(p, A.row_pages - 4));
}

// A block for each tile, or with several `parts` for a run of its pages, whose
// keys it leaves in the workspace for k_kv_pick.
// LDS: keys [TQ][row_pages], q's codes [8 hp], scales [waves][64], in words; of a
// block that selects, what select_rows needs.
template <int NP, int R>
__global__ void __launch_bounds__(kSelThreads) k_kv_select(SelectArgs A) {
    extern __shared__ __align__(16) uint32_t lds[];
    __shared__ float unit_s[16];
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int unit = blockIdx.x / A.parts, part = blockIdx.x % A.parts;
    const SelectTile t(A, unit, l);
    if (t.rows <= 0) return;
    uint32_t* const keys = lds;
    uint32_t* const rest = lds + A.TQ * A.row_pages;
    const bool all = t.most <= A.keep;
    if (A.parts > 1) {
        const int run = max((t.most + A.parts * 64 - 1) / (A.parts * 64), kLeastRun / 64) * 64, from = run * part;
        if (all || from >= t.most) return;
        const int upto = min(from + run, t.most);
        page_keys<NP, kSelThreads>(A, keys, rest, unit_s, t.R, t.head, t.i0, t.rows, t.table, from, upto);
        __syncthreads();
        uint32_t* to = A.keys + (size_t)unit * A.TQ * A.row_pages;
        for (int i = 0; i < t.rows; ++i)
            for (int p = from + 4 * (int)threadIdx.x; p < upto; p += 4 * kSelThreads)
                *reinterpret_cast<uint4*>(to + i * A.row_pages + p) = *reinterpret_cast<const uint4*>(keys + i * A.row_pages + p);
        return;
    }
    if (!all) page_keys<NP, kSelThreads>(A, keys, rest, unit_s, t.R, t.head, t.i0, t.rows, t.table, 0, t.most);
    __syncthreads();
    if (all) select_rows<R>(A, t, R > 0 ? rest : lds, w, kSelThreads / kWave, l, [&](int, int p) { return keys_of_all(A, t, p); });
    else select_rows<R>(A, t, R > 0 ? rest : lds, w, kSelThreads / kWave, l, [&](int i, int p) { return keys_of(A, keys, i, p); });
}

// The selection from keys in the workspace, a block for each tile.
template <int R>
__global__ void __launch_bounds__(kSelThreads) k_kv_pick(SelectArgs A) {
    extern __shared__ __align__(16) uint32_t lds[];
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const SelectTile t(A, blockIdx.x, l);
    if (t.rows <= 0) return;
    const uint32_t* keys = A.keys + (size_t)blockIdx.x * A.TQ * A.row_pages;
    if (t.most <= A.keep) select_rows<R>(A, t, lds, w, (int)blockDim.x / kWave, l, [&](int, int p) { return keys_of_all(A, t, p); });
    else select_rows<R>(A, t, lds, w, (int)blockDim.x / kWave, l, [&](int i, int p) { return keys_of(A, keys, i, p); });
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
    if (!one_launch(blocks, 256) || units / c.n_kv > 0x7fffffffll) return hipErrorInvalidConfiguration;
    if (c.kind == PROX_KV_INT8) hipLaunchKernelGGL((k_kv_bounds<PROX_KV_INT8>), dim3((uint32_t)blocks), dim3(256), 0, s, A, units);
    else hipLaunchKernelGGL((k_kv_bounds<PROX_KV_FP8>), dim3((uint32_t)blocks), dim3(256), 0, s, A, units);
    return hipGetLastError();
}

namespace {

template <int R>
constexpr size_t select_words(int row_pages, int waves) { return R > 0 ? (size_t)waves * 64 * R : (size_t)row_pages + kSelBins + kSelScratch; }

hipError_t allow_lds(const void* kernel, size_t lds) {
    return lds <= 48 * 1024 ? hipSuccess : hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
}

template <int NP, int R>
hipError_t select_launch(const SelectArgs& A, int64_t units, hipStream_t s) {
    const size_t score = 8 * (size_t)A.c.head_pad + kSelThreads, keys = (size_t)A.TQ * A.row_pages;
    const size_t select = A.parts > 1 ? 0 : select_words<R>(A.row_pages, kSelThreads / kWave);
    // a block of rows of more than 2048 pages selects where its keys are
    const size_t lds = 4 * (R > 0 ? keys + std::max(score, select) : std::max(keys + score, select));
    hipError_t e = allow_lds((const void*)k_kv_select<NP, R>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_kv_select<NP, R>), dim3((uint32_t)(units * A.parts)), dim3(kSelThreads), lds, s, A);
    e = hipGetLastError();
    if (e != hipSuccess || A.parts == 1) return e;
    const int waves = R > 0 ? std::min(A.TQ, kSelThreads / kWave) : kSelThreads / kWave;
    const size_t pick = 4 * select_words<R>(A.row_pages, waves);
    e = allow_lds((const void*)k_kv_pick<R>, pick);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_kv_pick<R>), dim3((uint32_t)units), dim3((uint32_t)(64 * waves)), pick, s, A);
    return hipGetLastError();
}

template <int NP>
hipError_t select_np(const SelectArgs& A, int64_t units, hipStream_t s) {
    // by the table's width: what the rows' lengths are, the host does not see.  A wave's selection of 2048 keys
    // takes 9.3 us, a block's 10.4
    if (A.row_pages > 2048) return select_launch<NP, 0>(A, units, s);
    if (A.row_pages > 512) return select_launch<NP, 32>(A, units, s);
    return A.row_pages > 256 ? select_launch<NP, 8>(A, units, s) : select_launch<NP, 4>(A, units, s);
}

// How a call is split (host).
struct SelectSplit {
    int RP, TQ, row_pages, parts;
    int64_t units;             // tiles of tokens and key heads
    bool fits;
    size_t bytes;              // workspace
    SelectSplit(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads) {
        RP = std::min(pow2_up(n_heads / c.n_kv), 16);
        row_pages = (b.max_pages + 63) / 64 * 64;
        // several rows of a sequence share the pages' bounds; a row of more than 2048 pages has a block of its own
        const int max_q = std::max(std::min(b.q_start ? b.max_q : 1, b.n_tokens), 1);
        TQ = row_pages > 2048 ? 1 : std::min(16 / RP, pow2_up(max_q));
        while (TQ > 1 && TQ * row_pages > 8192) TQ /= 2;             // 32 KB of keys: four blocks a CU have room
        const int64_t tiles = TQ == 1 ? b.n_tokens : std::min((int64_t)b.n_seq * ((max_q - 1) / TQ + 1), (int64_t)b.n_tokens / TQ + b.n_seq);
        units = tiles * c.n_kv;
        const int64_t want = kBlocksPerCu * device_cus() / units, most = (row_pages + kLeastRun - 1) / kLeastRun;
        parts = (int)std::max<int64_t>(std::min(want, most), 1);
        fits = one_launch(units * parts, kSelThreads);               // (k_kv_pick has no more)
        bytes = parts > 1 ? align_up((size_t)units * TQ * row_pages * sizeof(uint32_t), 256) : 256;
    }
};

}  // namespace

size_t kv_select_workspace(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads) {
    if (b.n_tokens <= 0 || b.max_q <= 0) return 256;
    const SelectSplit p(c, b, n_heads);
    return p.fits ? p.bytes : 0;
}

hipError_t launch_kv_select(const prox_kv_cache& c, const prox_kv_batch& b, const uint16_t* q, int64_t q_stride, int n_heads,
                            const int8_t* bounds, int keep, int first, int last, int32_t* pages, void* workspace,
                            hipStream_t s) {
    const SelectSplit p(c, b, n_heads);
    if (!p.fits) return hipErrorInvalidConfiguration;
    const SelectArgs A{c, b, q, q_stride, bounds, pages, keep, first, last, n_heads / c.n_kv, p.RP, p.TQ, p.row_pages, p.parts,
                       static_cast<uint32_t*>(workspace)};
    switch (c.head_pad / 64) {
        case 1: return select_np<1>(A, p.units, s);
        case 2: return select_np<2>(A, p.units, s);
        case 3: return select_np<3>(A, p.units, s);
        default: return select_np<4>(A, p.units, s);
    }
}

}  // namespace prox
