// Kernels of the attention over the paged 8-bit key/value cache, and how a call is
// split among them.
//
// For one row (a token's query head) with the stored codes kc, vc and the
// scales sk, sv of each page:
//   s_j = scale sk (q . kc_j),  o = sum_j exp(s_j - m) sv vc_j / sum_j exp(s_j - m)
// in one pass over the pages with a running maximum m (base 2: log2(e) is
// folded into the scale).
//
// Arithmetic.  Both products run on v_mfma_f32_16x16x32_f16 with fp32 sums.
//   codes  are exact in fp16.  An int8 code c is taken as 1024 + (c + 128): the
//          byte put under the exponent bits 0x64, half an instruction a code
//          where a conversion takes one and a half.  For keys the 1152 too many
//          are subtracted as a start value of the sum, -1152 sum(q), so a
//          score's fp32 sum runs over values up to 1279 / 127 times larger than
//          the codes' own.  For values they are subtracted from each pair of
//          codes (exact in fp16, one instruction): left in sums that run over
//          many pages they cost five bits and more, 1.6e-3 of a mean of 256
//          pages and 1.4e-2 of one of 2048.
//   q      (bf16, 8 bits) is scaled by a power of two to a largest value in
//          [1, 2): exact in fp16 down to 2^-17 of the row's largest, and off
//          by at most 2^-25 of that below.
//   p      the softmax weights are rounded to fp16 (half a step: 2^-11) and
//          held up to 2^15.9, so that fp16's normal numbers reach down to 2^-22
//          of a row's largest (2^-24 but for sv, see there).  The sum that the result is divided by is that
//          of the rounded weights (a product with a row of constants), which
//          keeps the result a weighted mean of the stored values.
//   sv     goes into the weights: p sv / 2^e with 2^e the unit of a row's sums,
//          one more term of the exponent, so the values' sums stay in the matrix
//          unit's accumulators from page to page; the sum of the weights takes
//          it out again.  e moves up where p sv / 2^e leaves the weights' range,
//          so a page that has no weight in a row moves nothing there, and down
//          where sv / 2^e falls below a quarter (smaller ones would cost the
//          small weights, and the sum with them, their bits), as far as the
//          row's sums allow: they stay below 2^100.  A page for which they do
//          not allow it counts as a quarter of the unit, less than 2^-50 of the
//          row's largest sum.
//          m and e are whole numbers: moving them rounds nothing, and value
//          scales of any fp32 size give the same result in their unit.
// m and e move only when a score exceeds m by more than 2^5.9 or an sv leaves its
// range, so most pages rescale nothing.
//
// A wave takes tiles of 16 rows that share a key head and walks their pages.
// With K as the A operand and q as B, lane (g = l / 16, n = l % 16) gets the
// scores of row n and tokens 16 t + 4 g + r of the page, t, r < 4; the V layout
// of the cache puts the same tokens into lane group g, so the weights go
// straight into the second product, whose result has row n in the same lanes:
// nothing but the row's maximum crosses lanes.
//
// How the work is split.  A segment is one tile of rows (TQ tokens x HG query
// heads of one key head) with the pages that some row of it sees.  All segments
// form one line, a unit for each page and a few for what a segment costs by
// itself, cut into pieces of equal length, one for each block, whatever the
// lengths of the sequences.  A block finds its piece from the lengths on the
// device (the host knows bounds only, and a captured call follows the lengths).
// A cut moves to a segment's border where the segment is short or the border
// near.  A segment that a cut divides leaves (maximum, sum, unit,
// unnormalised result) of each part in the workspace, at most two parts for
// each block, and the block that arrives last combines them in order of
// position, so results do not depend on timing.  (A launch of its own for that
// took 5 us of one token's call and up to 100 us of a prompt's.)
//
// What bounds it (medians of kernel time under a profiler and, in brackets, of calls
// back to back; query / key heads x channels; a copy of 2 GiB runs at 4.9 TB/s
// here, a 16384^3 product in bf16 at 1380 TFLOP/s):
//   one token, 32 / 32 x 128, 513 positions    12.5 us  latency; its parts are not measured (4.2 MB)
//   one token, 64 / 8 x 128, 131072 positions  65.4 us  268 MB at 4.1 TB/s: memory, read once (counters: 271 MB)
//   64 ragged sequences, 32 / 8 x 128          52.6 us  224 MB at 4.3 TB/s: memory
//   16 sequences of 1 to 6 tokens, 28 / 4 x 128, window 4096   27.3 us  5 to 7 of a block's 8 waves have no rows (39 MB)
//   4096-token prompt, 32 / 8 x 128           242 (204) us  137 GFLOP at 674 TFLOP/s, see walk_together
//   16384-token prompt                       2530 (2460) us  2199 GFLOP at 890 TFLOP/s: begins and joins weigh less
//   ragged chunks, 40 / 8 x 64                270 (226) us  127 GFLOP at 565 TFLOP/s: twice the exponentials a product
#pragma once

#include <algorithm>

#include "prox_kv.hpp"

namespace prox {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    f16x2_t r;
    r[0] = (_Float16)lo;
    r[1] = (_Float16)hi;
    return __builtin_bit_cast(uint32_t, r);
}

// Eight codes -> eight fp16: e4m3 as they are, int8 plus 1152.
template <int KIND>
__device__ __forceinline__ uint4 codes_f16(uint32_t lo, uint32_t hi) {
    if constexpr (KIND == PROX_KV_INT8) {
        const uint32_t a = lo ^ 0x80808080u, b = hi ^ 0x80808080u;
        return make_uint4(__builtin_amdgcn_perm(0x64646464u, a, 0x04010400u), __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u),
                          __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u), __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u));
    } else {
        return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.f, false)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.f, true)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.f, false)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.f, true)));
    }
}

// The same for values: int8 without the 1152.
template <int KIND>
__device__ __forceinline__ uint4 values_f16(uint32_t lo, uint32_t hi) {
    uint4 x = codes_f16<KIND>(lo, hi);
    if constexpr (KIND == PROX_KV_INT8) {
        auto less = [](uint32_t w) {
            return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, w) - f16x2_t{(_Float16)1152.f, (_Float16)1152.f});
        };
        x = make_uint4(less(x.x), less(x.y), less(x.z), less(x.w));
    }
    return x;
}

// Operands whose product with another one gives that one's sum, or -1152 times it.
__device__ __forceinline__ uint4 ones() { return make_uint4(0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u); }
__device__ __forceinline__ uint4 minus_1152() { return make_uint4(0xe480e480u, 0xe480e480u, 0xe480e480u, 0xe480e480u); }

// e4m3 codes with NaN taken as 0: slots that no token was written to may hold
// any byte, and 0 x NaN would reach the sum.
__device__ __forceinline__ uint32_t no_nan_fp8(uint32_t w) {
    const uint32_t n = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
    return w & ~(n * 0xffu);
}

__device__ __forceinline__ float over_groups_max(float v) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_int(v), __float_as_int(v), false, false);
    v = fmaxf(__int_as_float(a[0]), __int_as_float(a[1]));
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_int(v), __float_as_int(v), false, false);
    return fmaxf(__int_as_float(b[0]), __int_as_float(b[1]));
}

struct Attend {
    typedef KvRows Row;
    typedef uint16_t* Out;
    static constexpr bool kJoinLater = false;   // parts of cut segments are joined by another launch
    prox_kv_cache c;
    prox_kv_batch b;
    const uint16_t* q;
    uint16_t* out;
    int64_t qs, os;
    unsigned long long* arrived;   // [blocks]: arrivals of the cut segment that begins in a block's piece
    float* part;                   // [blocks][2][slot_rows][head_pad + 4]: result, then maximum, sum and unit
    uint32_t part_bytes, tag;
    int rep, window;
    uint32_t HG_inv;       // 2^17 / HG, rounded up
    int HG, VH;            // query heads of a segment; segments of one tile of tokens (key heads x head groups)
    int TQ, tiles;         // tokens of a tile; most tiles of a sequence
    int all_tiles;         // and of the batch: a q_start that does not rise could name more, which are left out
    int rows_lo, rows_hi;  // least and most rows of the sequences that the launch takes
    int slot_rows;
    int seg_cost;          // units of a segment besides its pages
    int no_cut, min_part;  // pages of a segment up to which it is not cut, and least pages of a part
    int min_piece;         // least length of a piece
    float scale2;          // |scale| * log2(e)
    float sign;            // that of scale
};

// What follows up to `Place` is that of a call over the sequences' own pages.  A
// call of another kind has a type of its own derived from Attend, with its own
// Row and Out, and overloads of what its needs differ in: these and out_row(), put().
//
// The rows of sequence s, none if the launch does not take it.
__device__ __forceinline__ KvRows rows_of(const Attend& A, int s) {
    KvRows R = kv_rows(A.b, s);
    if (R.rows < A.rows_lo || R.rows > A.rows_hi) R.rows = 0;
    return R;
}

// Work that a launch does besides, before the attention.
__device__ __forceinline__ void prologue(const Attend&, int, int) {}

__device__ __forceinline__ KvRows no_rows(const Attend&) { return KvRows{0, 0, 0, 0}; }
// A lane's rows from lane i; those of lane `on`, the same for the whole wave.
__device__ __forceinline__ KvRows shuffled(const KvRows& R, int i) {
    return KvRows{__shfl(R.q0, i), __shfl(R.n, i), __shfl(R.rows, i), __shfl(R.first, i)};
}
__device__ __forceinline__ KvRows of_lane(const KvRows& R, int on) {
    return KvRows{__builtin_amdgcn_readlane(R.q0, on), __builtin_amdgcn_readlane(R.n, on),
                  __builtin_amdgcn_readlane(R.rows, on), __builtin_amdgcn_readlane(R.first, on)};
}

// One tile of tokens of one sequence.
template <typename Row>
struct TileOf {
    Row R;
    int i0, n;             // tokens i0 .. i0 + n - 1 of the sequence's rows
    int pg0, pages;        // pages that some row sees: pg0 .. pg0 + pages - 1; at least one (0: no such tile)
};

typedef TileOf<KvRows> Tile;

__device__ __forceinline__ Tile tile_of(const Attend& A, const KvRows& R, int t) {
    Tile x;
    x.R = R;
    x.i0 = t * A.TQ;
    x.n = min(x.R.rows - x.i0, A.TQ);
    const int cap = A.b.max_pages * kKvPage;
    const int p0 = x.R.first + x.i0, p1 = p0 + x.n;                  // positions p0 .. p1 - 1
    const int hi = min(p1, cap), lo = A.window > 0 ? max(max(p0, 0) - A.window + 1, 0) : 0;
    const bool some = hi > 0 && lo < hi;
    x.pg0 = some ? lo / kKvPage : 0;
    x.pages = x.n <= 0 ? 0 : some ? (hi - 1) / kKvPage + 1 - x.pg0 : 1;
    return x;
}

// The table's row of (the launch's) sequence s; the slots of positions from
// ctx_of() on hold no token; whether rows see only what their position allows.
__device__ __forceinline__ const int32_t* table_of(const Attend& A, int s) { return A.b.block_table + (size_t)s * A.b.max_pages; }
__device__ __forceinline__ int ctx_of(const Attend&, const Tile& T) { return T.R.first + T.R.n; }
__device__ __forceinline__ constexpr bool masked(const Attend&) { return true; }

// A segment: key head and head group vh of tile t of sequence s, and the unit
// of the line that it begins at.
struct Place {
    int s, t, vh, begin, pages;
};

// Where a cut at unit x falls that lies in a segment of `pages` pages beginning
// at `begin`: there, or at the segment's nearer border.
__device__ __forceinline__ int cut_in(const Attend& A, int x, int begin, int pages) {
    const int d = x - begin, len = pages + A.seg_cost;
    if (pages <= A.no_cut) return 2 * d < len ? begin : begin + len;
    return d < A.seg_cost + A.min_part ? begin : d > len - A.min_part ? begin + len : x;
}
// The blocks w0 .. w1 that work on such a segment.
__device__ __forceinline__ void blocks_of(const Attend& A, int piece, int begin, int pages, int& w0, int& w1) {
    const int lo = begin + A.seg_cost + A.min_part, hi = begin + A.seg_cost + pages - A.min_part;   // cuts fall in lo .. hi
    w0 = (lo + piece - 1) / piece - 1;
    w1 = hi / piece;
}

// The line of all segments (below 2^31: the host checks all_tiles), seen by one wave.
// It looks at 64 tiles at a time, those that there are of 64 sequences: with
// one prompt among 255 single tokens these are 5 looks, where max_q alone would
// allow 64 tiles for each sequence (256 looks).
template <typename AT>
struct Line {
    typedef typename AT::Row Row;
    typedef TileOf<Row> Tile;
    const AT& A;
    int l, total, looks;   // lane; units; looks that the line takes
    struct Look {
        int s0, j0, base;  // first sequence; first of its chunk's tiles; units before it
        int before;        // tiles before the chunk
    };
    Look from;             // at() begins here
    Row Q;                 // lane: sequence s0 + lane,
    int last, tiles;       // the chunk's tiles up to its end, and all of them
    Row R;                 // lane: a tile's sequence,
    int s, t, pages, upto; // its number, the tile, its pages, and the units up to its end

    static __device__ __forceinline__ int sum_up(int v, int l) {
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
            const int u = __shfl_up(v, m);
            if (l >= m) v += u;
        }
        return v;
    }
    __device__ __forceinline__ void chunk(int s0, int before) {
        Q = s0 + l < A.b.n_seq ? rows_of(A, s0 + l) : no_rows(A);
        if (A.tiles > 1) {
            last = sum_up((int)((uint32_t)(Q.rows + A.TQ - 1) / (uint32_t)A.TQ), l);
            tiles = min(__builtin_amdgcn_readlane(last, 63), A.all_tiles - before);
        } else {
            tiles = 64;        // a lane's sequence is its tile
        }
    }
    __device__ __forceinline__ void look(const Look& k) {
        int i = l;
        R = Q;
        t = 0;
        if (A.tiles > 1) {
            // sequence i, the number of those that end before tile j0 + lane
            const int j = k.j0 + l;
            i = 0;
#pragma unroll
            for (int m = 32; m > 0; m /= 2)
                if (__shfl(last, i + m - 1) <= j) i += m;
            const int before = __shfl(last, i > 0 ? i - 1 : 0);
            t = j - (i > 0 ? before : 0);
            R = shuffled(Q, i);
            if (j >= tiles) R.rows = 0;
        }
        s = k.s0 + i;
        pages = R.rows > 0 ? tile_of(A, R, t).pages : 0;
        upto = k.base + sum_up(pages > 0 ? (pages + A.seg_cost) * A.VH : 0, l);
    }
    // The looks from k on, until one reaches beyond unit x.
    __device__ __forceinline__ Look scan(Look k, int x) {
        chunk(k.s0, k.before);
        for (;;) {
            while (k.j0 >= tiles) {
                k = Look{k.s0 + 64, 0, k.base, k.before + (A.tiles > 1 ? tiles : 0)};
                if (k.s0 >= A.b.n_seq) return k;
                chunk(k.s0, k.before);
            }
            look(k);
            ++looks;
            const int end = __builtin_amdgcn_readlane(upto, 63);
            if (end > x) return k;
            k.j0 += 64;
            k.base = end;
        }
    }
    __device__ __forceinline__ Line(const AT& a, int lane) : A(a), l(lane), looks(0), from{0, 0, 0, 0} {
        total = scan(from, 0x7fffffff).base;
    }
    // x < total; keep: no later call asks for a unit of an earlier look
    __device__ __forceinline__ Place at(int x, Tile& T, bool keep) {
        if (looks > 1) {
            const Look k = scan(from, x);
            if (keep) from = k;
        }
        const int on = __builtin_ctzll(__ballot(upto > x) | (1ull << 63));
        Place p;
        p.s = __builtin_amdgcn_readlane(s, on);
        p.t = __builtin_amdgcn_readlane(t, on);
        p.pages = __builtin_amdgcn_readlane(pages, on);
        const int len = p.pages + A.seg_cost, first = __builtin_amdgcn_readlane(upto, on) - len * A.VH;
        p.vh = (int)((uint32_t)(x - first) / (uint32_t)len);
        p.begin = first + p.vh * len;
        T = tile_of(A, of_lane(R, on), p.t);
        return p;
    }
};

// The segment after p, where there is one.
template <typename AT, typename Tile>
__device__ __forceinline__ void next_segment(const AT& A, Place& p, Tile& T) {
    p.begin += p.pages + A.seg_cost;
    if (++p.vh < A.VH) return;
    p.vh = 0;
    auto R = T.R;
    if (++p.t * A.TQ >= R.rows) {
        p.t = 0;
        do R = rows_of(A, ++p.s);
        while (R.rows <= 0);
    }
    T = tile_of(A, R, p.t);
    p.pages = T.pages;
}

__device__ __forceinline__ uint2 bf16x4(f32x4_t v) {
    typedef __bf16 b4 __attribute__((ext_vector_type(4)));
    b4 x;
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = (__bf16)v[r];
    return __builtin_bit_cast(uint2, x);
}

// 1 / the softmax sum: 0 for a row that has seen nothing; a NaN sum stays.
__device__ __forceinline__ float inverse(float sum) { return sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum); }

// Weights hold up to 2^(kTop + kSlack), 61000 of fp16's 65504: see "Arithmetic" above.  A slack of 5 moves m
// more often: a 4096-token prompt takes 203 us, with 5.9 198.
constexpr float kTop = 10.f, kSlack = 5.9f;
constexpr int kLeast = -2;             // exponent of the least sv / 2^e that goes into the weights
constexpr int kRoom = 100;             // exponent that a row's sums stay below when e moves down
constexpr int kNoUnit = -1000;         // e of a row that has seen no value but zeros
constexpr int kNoPage = -1001;         // unit before the first page with others
constexpr float kNothing = -0x1p126f;  // m of a row that has seen nothing; scores are above
constexpr float kLarge = 0x1p20f;      // maxima from here on: see limits()

// A result in its own units.
__device__ __forceinline__ f32x4_t result(f32x4_t o, float inv, float e) {
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = ldexpf(o[r] * inv, (int)e);
    return o;
}

// What a row's part is besides its results: its maximum, sum and unit.
struct Part {
    float m, sum, e;
};
__device__ __forceinline__ Part no_part() { return Part{kNothing, 0.f, (float)kNoUnit}; }
__device__ __forceinline__ float4 packed(const Part& p) { return make_float4(p.m, p.sum, p.e, 0.f); }
__device__ __forceinline__ Part unpacked(float4 f) { return Part{f.x, f.y, f.z}; }

// Part (p, v) joins (a, o), in the larger of their units 2^(m + e).  m + e is
// never formed: m may be so large that it would swallow e.
__device__ __forceinline__ void join(Part& a, f32x4_t& o, const Part& p, f32x4_t v) {
    const float mn = fmaxf(a.m, p.m), t = (p.m - a.m) + (p.e - a.e);
    const float f = t > 0.f ? __builtin_amdgcn_exp2f(-t) : 1.f, g = t > 0.f ? 1.f : __builtin_amdgcn_exp2f(t);
    a.e = t > 0.f ? p.e + (p.m - mn) : a.e + (a.m - mn);
    a.sum = a.sum * __builtin_amdgcn_exp2f(a.m - mn) + p.sum * __builtin_amdgcn_exp2f(p.m - mn);
    a.m = mn;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = o[r] * f + v[r] * g;
}

// What the rows of a segment need to be put together later.
struct Seg {
    int begin, pages;      // units of the line
    int vh, row0, n;       // key head and head group; rows of the batch row0 .. row0 + n - 1
};
template <typename Tile>
__device__ __forceinline__ Seg seg_of(const Place& P, const Tile& T) {
    return Seg{P.begin, P.pages, P.vh, T.R.q0 + T.i0, T.n};
}

// Where the parts of token i of a segment are, for the launch that joins them.
__device__ __forceinline__ void later(const Attend&, const Seg&, int, int, int) {}

// r / A.HG for r < 256, HG <= 256: r times the rounding of 2^17 / HG stays below 2^17 / HG
__device__ __forceinline__ int token_of(const Attend& A, int r) { return (int)((uint32_t)r * A.HG_inv >> 17); }

// Where row r of a segment goes, or null for a row that the segment does not have.
__device__ __forceinline__ uint16_t* out_row(const Attend& A, const Seg& S, int r) {
    const int groups = A.VH / A.c.n_kv, head = S.vh / groups, grp = S.vh - head * groups;
    const int i = token_of(A, r), hq = grp * A.HG + r - i * A.HG;
    if (i >= S.n || hq >= A.rep) return nullptr;
    return A.out + (int64_t)(S.row0 + i) * A.os + (int64_t)(head * A.rep + hq) * A.c.head_dim;
}

// Four channels of a row's result go there, from c4 on: o unnormalised, a what goes with it, inv the inverse of its sum.
__device__ __forceinline__ void put(const Attend& A, uint16_t* to, int c4, f32x4_t o, const Part& a, float inv) {
    if (c4 < A.c.head_dim) *reinterpret_cast<uint2*>(to + c4) = bf16x4(result(o, inv, a.e));
}

// The rows r0 .. r0 + 16 NT - 1 of a segment's tile in one wave: what they see,
// q, and the running maxima, sums, units and results.
template <int KIND, int NP, int NT>
struct Rows {
    f32x4_t o[NT][4 * NP];      // lane (g, n): channels 16 d + 4 g + r of row 16 u + n, in units of 2^e
    float m[NT], sum[NT];
    int e[NT];
    int unit;                   // e of every row; kNoUnit where they differ or an m is kLarge
    bool live[NT];
    int key_lo[NT], key_hi[NT]; // positions that the row sees: key_lo .. key_hi - 1
    uint4 q[NT][NP][2];
    float row_scale[NT], bias[NT];

    // Where the rows are, and their q on its way.
    template <typename AT>
    __device__ __forceinline__ void load(const AT& A, const Seg& S, int pos0, int r0, int l) {
        const int n = l & 15, g = l >> 4, hd = A.c.head_dim, cap = A.b.max_pages * kKvPage;
        const int groups = A.VH / A.c.n_kv, head = S.vh / groups, grp = S.vh - head * groups;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const int r = r0 + 16 * u + n, i = token_of(A, r), hq = grp * A.HG + r - i * A.HG;
            live[u] = i < S.n && hq < A.rep;
            const int pos = pos0 + i;
            const bool sees = live[u] && pos >= 0 && pos < cap;
            key_lo[u] = sees && A.window > 0 ? pos - A.window + 1 : 0;
            key_hi[u] = !masked(A) ? 0x7fffffff : sees ? pos + 1 : (live[u] ? 0 : 0x7fffffff);    // a row that is not there is not masked
            const uint16_t* src = A.q + (int64_t)(S.row0 + (live[u] ? i : 0)) * A.qs +
                                  (int64_t)(head * A.rep + (live[u] ? hq : 0)) * hd;
#pragma unroll
            for (int a = 0; a < NP; ++a)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int ch = 64 * a + 16 * g + 8 * e;
                    q[u][a][e] = live[u] && ch < hd ? *reinterpret_cast<const uint4*>(src + ch) : make_uint4(0, 0, 0, 0);
                }
        }
    }

    // q scaled to fp16; nothing seen yet.
    __device__ __forceinline__ void begin(const Attend& A) {
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            uint32_t big = 0;
#pragma unroll
            for (int a = 0; a < NP; ++a)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint4 x = q[u][a][e];
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int f = 0; f < 4; ++f) big = max(big, max(w[f] & 0x7fff0000u, (w[f] << 16) & 0x7fff0000u));
                }
            big = __float_as_uint(over_groups_max(__uint_as_float(big > 0x7f800000u ? 0x7f800000u : big)));
            // 2^-E and 2^E with E the exponent of the row's largest value; 1 for a row of zeros or with an infinity or NaN
            const uint32_t ex = big >> 23;
            const bool one = ex == 0 || ex == 255;
            const int E = one ? 0 : (int)ex - 127;
            const float down = ldexpf(A.sign, -E);
            row_scale[u] = ldexpf(A.scale2, E);
            f32x4_t b4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int a = 0; a < NP; ++a)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint4 x = q[u][a][e];
                    q[u][a][e] = make_uint4(pack_f16(bf16_lo(x.x) * down, bf16_hi(x.x) * down),
                                            pack_f16(bf16_lo(x.y) * down, bf16_hi(x.y) * down),
                                            pack_f16(bf16_lo(x.z) * down, bf16_hi(x.z) * down),
                                            pack_f16(bf16_lo(x.w) * down, bf16_hi(x.w) * down));
                    if constexpr (KIND == PROX_KV_INT8) b4 = mfma16(minus_1152(), q[u][a][e], b4);
                }
            bias[u] = b4[0];
            m[u] = kNothing;
            sum[u] = 0.f;
            e[u] = kNoUnit;
#pragma unroll
            for (int d = 0; d < 4 * NP; ++d) o[u][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        unit = kNoPage;
    }

    // The scores of one page, in units of fac: keys(a, t, x, y) gives the two
    // operands of channels 64 a and tokens 16 t.
    template <typename K>
    __device__ __forceinline__ void scores(f32x4_t (&w)[NT][4], K keys) const {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int u = 0; u < NT; ++u) w[u][t] = f32x4_t{bias[u], bias[u], bias[u], bias[u]};
#pragma unroll
            for (int a = 0; a < NP; ++a) {
                uint4 k0, k1;
                keys(a, t, k0, k1);
#pragma unroll
                for (int u = 0; u < NT; ++u) w[u][t] = mfma16(k0, q[u][a][0], w[u][t]);
#pragma unroll
                for (int u = 0; u < NT; ++u) w[u][t] = mfma16(k1, q[u][a][1], w[u][t]);
            }
        }
    }

    // Masks the scores of positions base_key .. + 63 (none is seen if `gone`),
    // moves m and e where this page, of value scale 2^(ve + vl - kTop), needs it,
    // and says what the weights are: 2^(w fac - base), and `back` to their sum.
    __device__ __forceinline__ void limits(f32x4_t (&w)[NT][4], float (&fac)[NT], float (&base)[NT], float (&back)[NT],
                                           int base_key, bool gone, float ks, int ve, float vl, int l) {
#pragma clang fp contract(off)
        const int g = l >> 4;
        // keys that a row does not see; most pages are seen whole by every row
        bool open = !gone;
#pragma unroll
        for (int u = 0; u < NT; ++u) open = open && key_lo[u] <= base_key && key_hi[u] >= base_key + kKvPage;
        if (__ballot(open) != ~0ull) {
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const int s_lo = key_lo[u] - base_key, s_hi = gone ? 0 : key_hi[u] - base_key;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int slot = 16 * t + 4 * g + r;
                        w[u][t][r] = slot >= s_lo && slot < s_hi ? w[u][t][r] : -INFINITY;
                    }
            }
        }
        const bool some = ve != kNoUnit;                // the page has values other than zeros
        if (some && unit == kNoPage) {
            unit = ve;
#pragma unroll
            for (int u = 0; u < NT; ++u) e[u] = ve;
        }
        // a page without counts as one of the unit's scale: its values are read as zeros
        const int under = some ? unit - ve : 0;
        const bool fits = unit != kNoUnit && (uint32_t)under < (uint32_t)-kLeast;
        float top[NT];
        bool large = false;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            // not 0 (a page of zeros): 0 x -inf would be NaN; the scores of such a page vanish all the same.
            // Not above 2^106: the largest w is below 2^19, so scores stay finite
            fac[u] = __builtin_amdgcn_fmed3f(ks * row_scale[u], 1e-37f, 0x1p106f);
            float most = w[u][0][0];
#pragma unroll
            for (int i = 1; i < 16; ++i) most = fmaxf(most, w[u][i >> 2][i & 3]);
            top[u] = over_groups_max(most) * fac[u];
            large = large || (fabsf(top[u]) >= kLarge && top[u] != -INFINITY);
        }
        const float ratio = vl - (float)under, same = __builtin_amdgcn_exp2f(-ratio);
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            base[u] = m[u] - ratio;
            back[u] = same;
        }
        float f[NT];                                    // what o is multiplied by: in one place only
#pragma unroll
        for (int u = 0; u < NT; ++u) f[u] = 1.f;
        if (__builtin_expect(!fits || __ballot(large) != 0, 0)) move(w, top, fac, base, back, f, some, ve, vl);
        // most moves are of m alone, and there is none left behind move()
        bool grow = false;
#pragma unroll
        for (int u = 0; u < NT; ++u) grow = grow || f[u] != 1.f || top[u] - m[u] > kSlack;
        if (__ballot(grow)) {
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const float mn = fmaxf(m[u], floorf(top[u])), keep = __builtin_amdgcn_exp2f(m[u] - mn);
                base[u] = mn > m[u] ? mn - ratio : base[u];
                m[u] = mn;
                sum[u] *= keep;
                f[u] *= keep;
#pragma unroll
                for (int d = 0; d < 4 * NP; ++d) o[u][d] *= f[u];
            }
        }
    }

    // limits() where some row's m or e moves, or the rows differ in e.
    __device__ __forceinline__ void move(f32x4_t (&w)[NT][4], const float (&top)[NT], float (&fac)[NT], float (&base)[NT],
                                         float (&back)[NT], float (&f)[NT], bool some, int ve, float vl) {
#pragma clang fp contract(off)
        uint64_t large = 0;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const float mn = fmaxf(m[u], floorf(top[u])), keep = m[u] - mn;
            int en = e[u];
            bool down = false;
            if (some && mn > kNothing) {
                if (en == kNoUnit) en = unit != kNoUnit && ve <= unit && ve > unit + kLeast ? unit : ve;
                // a page of no weight in this row does not move it far
                else if (ve > en) en = ve - en <= 40 || (top[u] - mn) + (vl + (float)(ve - en)) > kTop + kSlack ? ve : en;
                else down = ve <= en + kLeast;
            }
            if (__ballot(down)) {
                float big = 0.f;
#pragma unroll
                for (int i = 0; i < 16 * NP; ++i) big = fmaxf(big, fabsf(o[u][i >> 2][i & 3]));
                big = over_groups_max(big);
                const int room = kRoom - __builtin_amdgcn_frexp_expf(big) - (int)fmaxf(keep, -500.f);
                if (down) en = big > 0.f ? max(ve, en - min(max(room, 0), 126)) : ve;
            }
            f[u] = __builtin_amdgcn_exp2f(fminf(keep + (float)(e[u] - en), 126.f));
            sum[u] *= __builtin_amdgcn_exp2f(keep);
            m[u] = mn;
            e[u] = en;
            const float ratio = some ? fmaxf(vl + (float)(ve - en), kTop + (float)kLeast) : vl;
            base[u] = mn - ratio;
            back[u] = __builtin_amdgcn_exp2f(-ratio);
            // Scores of 2^20 and more are compared and subtracted as rounded products: the unrounded product
            // would be off the maximum by more than a weight can take
            const bool rounded = mn > kNothing && fabsf(mn) >= kLarge;
            large |= __ballot(rounded);
            if (rounded) {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[u][i >> 2][i & 3] = w[u][i >> 2][i & 3] * fac[u] - mn;
                fac[u] = 1.f;
                base[u] = -ratio;
            }
        }
        // every wave has a row that is there
        int one = kNoUnit;
#pragma unroll
        for (int u = 0; u < NT; ++u) one = m[u] > kNothing ? e[u] : one;
        const uint64_t seen = __ballot(one != kNoUnit);
        one = __builtin_amdgcn_readlane(one, seen ? __builtin_ctzll(seen) : 0);
        bool differ = false;
#pragma unroll
        for (int u = 0; u < NT; ++u) differ = differ || (m[u] > kNothing && e[u] != one);
        unit = kNoUnit;
        if (__ballot(differ) == 0 && large == 0) {
            unit = one;
#pragma unroll
            for (int u = 0; u < NT; ++u) e[u] = one;            // o of a row that has seen nothing is 0
        }
    }

    // The weights of a page as operands.
    __device__ __forceinline__ void weights(const f32x4_t (&w)[NT][4], const float (&fac)[NT], const float (&base)[NT],
                                            uint4 (&pw)[NT][2]) const {
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            uint32_t x[4][2];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    x[t][r] = pack_f16(__builtin_amdgcn_exp2f(fmaf(w[u][t][2 * r], fac[u], -base[u])),
                                       __builtin_amdgcn_exp2f(fmaf(w[u][t][2 * r + 1], fac[u], -base[u])));
            pw[u][0] = make_uint4(x[0][0], x[0][1], x[1][0], x[1][1]);
            pw[u][1] = make_uint4(x[2][0], x[2][1], x[3][0], x[3][1]);
        }
    }

    // The values of a page: vals(d, x, y) gives the two operands of channels
    // 16 d.
    template <typename V>
    __device__ __forceinline__ void values(const uint4 (&pw)[NT][2], const float (&back)[NT], V vals) {
        weigh(pw, back);
#pragma unroll
        for (int d = 0; d < 4 * NP; ++d) {
            uint4 v0, v1;
            vals(d, v0, v1);
#pragma unroll
            for (int u = 0; u < NT; ++u) o[u][d] = mfma16(v0, pw[u][0], o[u][d]);
#pragma unroll
            for (int u = 0; u < NT; ++u) o[u][d] = mfma16(v1, pw[u][1], o[u][d]);
        }
    }
    // scores() and values() from operands in LDS (k, v: this lane's of operand
    // 0, 64 apart): the next few are read before the products of the last few,
    // since a read takes as long as eight products.
    static constexpr int kFew = 2 * NP;
    static __device__ __forceinline__ void fetch(uint4 (&f)[kFew], const uint4* at) {
#pragma unroll
        for (int i = 0; i < kFew; ++i) f[i] = at[i * 64];
    }
    __device__ __forceinline__ void scores_lds(f32x4_t (&w)[NT][4], const uint4* k) const {
        uint4 f[2][kFew];
        // operand 2 (a 4 + t) + e of the keys: those of one t, for all a
        auto read = [&](int t) {
#pragma unroll
            for (int a = 0; a < NP; ++a)
#pragma unroll
                for (int e = 0; e < 2; ++e) f[t & 1][2 * a + e] = k[(2 * (a * 4 + t) + e) * 64];
        };
        read(0);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t < 3) read(t + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < NT; ++u) w[u][t] = f32x4_t{bias[u], bias[u], bias[u], bias[u]};
#pragma unroll
            for (int i = 0; i < kFew; ++i)
#pragma unroll
                for (int u = 0; u < NT; ++u) w[u][t] = mfma16(f[t & 1][i], q[u][i >> 1][i & 1], w[u][t]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // first: the first kFew operands, read before
    __device__ __forceinline__ void values_lds(const uint4 (&pw)[NT][2], const float (&back)[NT], const uint4* v,
                                               const uint4 (&first)[kFew]) {
        uint4 f[2][kFew];
#pragma unroll
        for (int i = 0; i < kFew; ++i) f[0][i] = first[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {                   // channels 16 NP j ..
            if (j < 3) fetch(f[(j + 1) & 1], v + (j + 1) * kFew * 64);
            __builtin_amdgcn_sched_barrier(0);
            if (j == 0) weigh(pw, back);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int u = 0; u < NT; ++u)
                        o[u][j * NP + i] = mfma16(f[j & 1][2 * i + e], pw[u][e], o[u][j * NP + i]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // The weights' own sums.
    __device__ __forceinline__ void weigh(const uint4 (&pw)[NT][2], const float (&back)[NT]) {
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            f32x4_t c = {0.f, 0.f, 0.f, 0.f};
            c = mfma16(ones(), pw[u][0], c);
            c = mfma16(ones(), pw[u][1], c);
            sum[u] = fmaf(c[0], back[u], sum[u]);
        }
    }
    // Behind the last page: o as weights of 1 make it.  (As a step of its own: without one the
    // compiler copies o in every turn of the loop, 12 % of a prompt's time.)
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int d = 0; d < 4 * NP; ++d) o[u][d] *= __builtin_amdgcn_exp2f(-kTop);
    }
    __device__ __forceinline__ Part part(int u) const { return Part{m[u], sum[u], (float)e[u]}; }
};

// Pages of one segment for one wave.  A page that is not there (the table
// names none, or the segment has none) is a buffer of no bytes: its loads
// return zeros and touch no memory, and the number of loads in flight is the
// same in every turn of a loop.  So are the values of a page whose scale is 0.  Lane i keeps what the table and the scales
// say of page base + i: a turn of a loop reads a lane and waits for no memory
// (scalar loads would hold up every wait for LDS, which counts them too).
template <int NP, typename AT>
struct Pages {
    static constexpr int kBytes = kKvPage * 64 * NP;
    const AT& A;
    const int32_t* table;
    int head, upto, pg0, base, id, ve;
    float ks, vl;          // K's scale; V's scale 2^(ve + vl - kTop), -1 <= vl - kTop < 0 (0: ve kNoUnit)
    template <typename Tile>
    __device__ __forceinline__ Pages(const AT& a, const Place& P, const Tile& T, int from, int up, int l)
        : A(a), table(table_of(a, P.s) + T.pg0), head(P.vh / (a.VH / a.c.n_kv)), upto(up),
          pg0(T.pg0) {
        look(from, l);
    }
    __device__ __forceinline__ int base_key(int p) const { return (pg0 + p) * kKvPage; }
    __device__ __forceinline__ void look(int p, int l) {
        base = p;
        id = table[min(p + l, upto - 1)];
        id = p + l < upto && id >= 0 && id < A.c.n_pages ? id : -1;
        // a page that is not there has scales of 0, whatever those at where(-1), another page's, hold
        const float k0 = A.c.k_scale[where(id)], v0 = A.c.v_scale[where(id)];
        ks = id >= 0 ? k0 : 0.f;
        const bool some = id >= 0 && v0 > 0.f;
        ve = some ? __builtin_amdgcn_frexp_expf(v0) : kNoUnit;
        vl = kTop + __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(some ? v0 : 1.f));
    }
    // pages p .. p + 2 are looked at next
    __device__ __forceinline__ void follow(int p, int l) {
        if (p + 2 >= base + 64) look(p, l);
    }
    __device__ __forceinline__ int at(int p) const { return __builtin_amdgcn_readlane(id, p - base); }
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

// One wave walks pages from .. upto - 1 by itself: the next page's keys are
// loaded while this one is weighed, its values while its keys are multiplied.
// 8 such waves keep up to 128 KB of loads in flight in a CU; bare loads of the
// same order read 6.2 TB/s, this loop 4.2.  w's rows are on their way; slots of
// positions from ctx on hold no token.
template <int KIND, int NP, int NT, typename P>
__device__ __forceinline__ void walk_pages(Rows<KIND, NP, NT>& w, P& pages, const Attend& A, int ctx, int from, int upto, int l) {
    uint4 kf[4 * NP], vf[4 * NP];
    auto load = [&](uint4 (&f)[4 * NP], __amdgpu_buffer_rsrc_t r) {
#pragma unroll
        for (int d = 0; d < 4 * NP; ++d) f[d] = buf_load16(r, l * 16, d * 1024);
    };
    load(kf, pages.keys(from));
    __builtin_amdgcn_sched_barrier(0);                              // q and the first keys are on their way
    w.begin(A);
    for (int p = from; p < upto; ++p) {
        pages.follow(p, l);
        const int page = pages.at(p);
        load(vf, pages.values(p));
        __builtin_amdgcn_sched_barrier(0);                          // before the first product
        const int base_key = pages.base_key(p);
        const bool clean = KIND == PROX_KV_FP8 && base_key + kKvPage > ctx;
        f32x4_t sc[NT][4];
        float fac[NT], less[NT], back[NT];
        w.scores(sc, [&](int a, int t, uint4& x, uint4& y) {
            const uint4 c = kf[a * 4 + t];
            x = codes_f16<KIND>(c.x, c.y);
            y = codes_f16<KIND>(c.z, c.w);
        });
        load(kf, pages.keys(p + 1));
        __builtin_amdgcn_sched_barrier(0);
        w.limits(sc, fac, less, back, base_key, page < 0, pages.k_scale(p), pages.v_exp(p), pages.v_log(p), l);
        uint4 pw[NT][2];
        w.weights(sc, fac, less, pw);
        w.values(pw, back, [&](int d, uint4& x, uint4& y) {
            uint4 c = vf[d];
            if (clean) c = make_uint4(no_nan_fp8(c.x), no_nan_fp8(c.y), no_nan_fp8(c.z), no_nan_fp8(c.w));
            x = values_f16<KIND>(c.x, c.y);
            y = values_f16<KIND>(c.z, c.w);
        });
    }
    w.finish();
}

template <int KIND, int NP, int NT, typename AT, typename Tile>
__device__ __forceinline__ void walk_alone(Rows<KIND, NP, NT>& w, const AT& A, const Place& P, const Tile& T, int from,
                                           int upto, int r0, int l) {
    Pages<NP, AT> pages(A, P, T, from, upto, l);
    w.load(A, seg_of(P, T), T.R.first + T.i0, r0, l);
    walk_pages<KIND, NP, NT>(w, pages, A, ctx_of(A, T), from, upto, l);
}

// The waves of a block walk the same pages, each for its own rows.  A page is
// loaded once for the block, each wave turning its share of the codes to fp16
// operands in LDS (two pages' worth: one is filled while the other is used),
// so a page costs the block one barrier.
// Two waves share a SIMD (248 registers).  Measured on a form of this loop that
// took 212 us for a 4096-token prompt (one unit of the sums for a whole wave;
// units of the rows' own cost some 5 %): 297 where each wave loads and converts
// its own operands; the matrix unit is busy 36 % of the time and no single unit
// is the bound: with the LDS reads, exponentials, weights or fills left out in
// turn the time fell by 0 to 20 of 224 us, with the products left out by 24.
// Not kept: the next page's keys multiplied beside the exponentials (322 us,
// spills), two groups of waves half a page apart (220), four waves in each of
// two blocks (244), one tile of 16 rows a wave: 8 waves 299, 12 waves 233, 16
// waves 271.
// LDS: keys [2][4 NP x 2 operands][64] uint4, values the same.
template <int KIND, int NP, int NT, int kWaves, typename AT, typename Tile>
__device__ __forceinline__ void walk_together(Rows<KIND, NP, NT>& w, uint4* lds, const AT& A, const Place& P,
                                              const Tile& T, int from, int upto, int wv, int l) {
    constexpr int kChunks = 4 * NP;                                 // kilobytes of codes of K, and of V
    constexpr int kOwn = (kChunks + kWaves - 1) / kWaves;           // a wave's: chunks wv, wv + kWaves, ...
    constexpr int kSize = kChunks * 128;                            // uint4 of a page's operands
    Pages<NP, AT> pages(A, P, T, from, upto, l);
    const int ctx = ctx_of(A, T);
    const int r0 = 16 * NT * wv;
    const bool busy = r0 < T.n * A.HG;                              // a wave without rows only fills
    w.load(A, seg_of(P, T), T.R.first + T.i0, r0, l);
    uint4* const kl = lds + l;
    uint4* const vl = lds + 2 * kSize + l;
    uint4 kc[kOwn], vc[kOwn];
    auto load = [&](uint4 (&c)[kOwn], __amdgpu_buffer_rsrc_t r) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int ch = wv + j * kWaves;                         // past the last chunk: past the buffer, zeros
            c[j] = buf_load16(r, l * 16 + ch * 1024, 0);
        }
    };
    auto fill_keys = [&](uint4* to) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int ch = wv + j * kWaves;
            if (kChunks % kWaves && ch >= kChunks) continue;
            to[(2 * ch) * 64] = codes_f16<KIND>(kc[j].x, kc[j].y);
            to[(2 * ch + 1) * 64] = codes_f16<KIND>(kc[j].z, kc[j].w);
        }
    };
    auto fill_values = [&](uint4* to, bool clean) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int ch = wv + j * kWaves;
            if (kChunks % kWaves && ch >= kChunks) continue;
            uint4 x = vc[j];
            if (clean) x = make_uint4(no_nan_fp8(x.x), no_nan_fp8(x.y), no_nan_fp8(x.z), no_nan_fp8(x.w));
            to[(2 * ch) * 64] = values_f16<KIND>(x.x, x.y);
            to[(2 * ch + 1) * 64] = values_f16<KIND>(x.z, x.w);
        }
    };
    auto unclean = [&](int p) { return KIND == PROX_KV_FP8 && (T.pg0 + p + 1) * kKvPage > ctx; };
    load(kc, pages.keys(from));
    load(vc, pages.values(from));
    w.begin(A);
    lds_barrier();                                                  // the last segment's pages are done with
    fill_keys(kl);
    load(kc, pages.keys(from + 1));
    fill_values(vl, unclean(from));
    load(vc, pages.values(from + 1));
    lds_barrier();
    for (int p = from; p < upto; ++p) {
        const int buf = (p - from) & 1;
        pages.follow(p, l);
        if (busy) {
            f32x4_t sc[NT][4];
            float fac[NT], less[NT], back[NT];
            w.scores_lds(sc, kl + buf * kSize);
            uint4 first[Rows<KIND, NP, NT>::kFew];
            w.fetch(first, vl + buf * kSize);
            w.limits(sc, fac, less, back, (T.pg0 + p) * kKvPage, pages.at(p) < 0, pages.k_scale(p), pages.v_exp(p),
                     pages.v_log(p), l);
            uint4 pw[NT][2];
            w.weights(sc, fac, less, pw);
            w.values_lds(pw, back, vl + buf * kSize, first);
        }
        // the other half was used a turn ago
        fill_values(vl + (buf ^ 1) * kSize, unclean(p + 1));
        load(vc, pages.values(p + 2));
        fill_keys(kl + (buf ^ 1) * kSize);
        load(kc, pages.keys(p + 2));
        lds_barrier();
    }
    w.finish();
}

// Blocks of up to kWaves waves.
//   ROWS false (a tile of 16 rows at most): the waves cut the block's piece
//     among themselves once more and meet at its end, where segments that
//     several waves worked on are put together in LDS.
//     LDS: [waves][2][slot_rows][64 NP + 4] floats
//   ROWS true: a tile of 16 NT rows for each wave; the waves walk the same pages.
// Rows of cut segments go to the workspace.
template <int KIND, int NP, int NT, bool ROWS, int kWaves, typename AT>
__global__ void __launch_bounds__(64 * kWaves, NP <= 2 ? 2 : 1) k_kv_attend(AT A) {
    extern __shared__ __align__(16) float lds[];
    __shared__ Seg seg_s[16];                     // segment of each wave's two slots, begin -1: none
    __shared__ Seg cut_s[2];                      // the segments that reach over the piece's begin and over its end
    __shared__ int done_s[2];
    constexpr int RW = 64 * NP + 4;               // floats of a row in a slot: result, maximum, sum, unit
    constexpr int LPR = 16 * NP;                  // lanes of a row, four channels each
    const int l = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), n = l & 15, g = l >> 4;
    const int WV = blockDim.x >> 6;
    prologue(A, wv, l);
    Line<AT> line(A, l);
    const int piece = (int)max((uint32_t)line.total / gridDim.x + 1, (uint32_t)A.min_piece);
    if ((int64_t)blockIdx.x * piece >= line.total) return;
    // where the piece begins and ends, and the place of this wave's first unit:
    // one turn each of a loop that stays a loop (code that runs once is fetched once)
    int b0 = 0, b1 = 0, x = 0, end = 0;
    Place P;
    TileOf<typename AT::Row> T;
#pragma nounroll
    for (int k = 0; k < 3; ++k) {
        int64_t at = k < 2 ? ((int64_t)blockIdx.x + k) * piece : x;
        if (at < line.total) {
            P = line.at((int)at, T, k == 0);
            if (k < 2) at = cut_in(A, (int)at, P.begin, P.pages);
        } else {
            at = line.total;
        }
        if (k == 0) b0 = (int)at;
        if (k == 1) {
            b1 = (int)at;
            if (b0 >= b1) return;
            x = ROWS ? b0 : b0 + (int)((int64_t)(b1 - b0) * wv / WV);
            end = ROWS ? b1 : b0 + (int)((int64_t)(b1 - b0) * (wv + 1) / WV);
        }
    }
    const __amdgpu_buffer_rsrc_t rp = make_rsrc(A.part, A.part_bytes);
    bool sent = false;
    // a row of a part in the workspace: bytes
    auto part_at = [&](int block, bool begins, int r) {
        return ((2u * (uint32_t)block + (begins ? 1u : 0u)) * (uint32_t)A.slot_rows + (uint32_t)r) * (uint32_t)(RW * 4);
    };

    if (!ROWS && l < 2) seg_s[2 * wv + l].begin = -1;
    if (threadIdx.x < 2) cut_s[threadIdx.x].begin = -1;
    if (x < end) {
        for (;;) {
            const int first = P.begin + A.seg_cost;                 // the unit of page 0
            const int from = max(x - first, 0), upto = min(P.pages, end - first);
            if (ROWS || from < upto) {
            const int r0 = ROWS ? 16 * NT * wv : 0;
            Rows<KIND, NP, NT> w;
            if constexpr (ROWS) walk_together<KIND, NP, NT, kWaves>(w, reinterpret_cast<uint4*>(lds), A, P, T, from, upto, wv, l);
            else walk_alone<KIND, NP, NT>(w, A, P, T, from, upto, 0, l);
            if (!ROWS || r0 < T.n * A.HG) {
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                    const int r = r0 + 16 * u + n;
                    if (from == 0 && upto == P.pages) {
                        const typename AT::Out to = w.live[u] ? out_row(A, seg_of(P, T), r) : typename AT::Out();
                        const float inv = inverse(w.sum[u]);
                        if (to)
#pragma unroll
                            for (int d = 0; d < 4 * NP; ++d) put(A, to, 16 * d + 4 * g, w.o[u][d], w.part(u), inv);
                    } else if (!ROWS) {
                        const int slot = 2 * wv + (from == 0 ? 1 : 0);
                        if (l == 0) seg_s[slot] = seg_of(P, T);
                        if (n < A.slot_rows) {
                            float* to = lds + (slot * A.slot_rows + n) * RW;
#pragma unroll
                            for (int d = 0; d < 4 * NP; ++d) *reinterpret_cast<f32x4_t*>(to + 16 * d + 4 * g) = w.o[u][d];
                            if (g == 0) *reinterpret_cast<float4*>(to + 64 * NP) = packed(w.part(u));
                        }
                    } else if (w.live[u]) {
                        const uint32_t at = part_at(blockIdx.x, from == 0, r);
                        constexpr int kAux = AT::kJoinLater ? 0 : kCoherent;
#pragma unroll
                        for (int d = 0; d < 4 * NP; ++d)
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, w.o[u][d]), rp,
                                                                   (int)(at + 4 * (16 * d + 4 * g)), 0, kAux);
                        if (g == 0)
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, packed(w.part(u))), rp,
                                                                   (int)(at + 256 * NP), 0, kAux);
                    }
                }
            }
            if (ROWS && (from != 0 || upto != P.pages)) {
                sent = true;
                if (threadIdx.x == 0) cut_s[from != 0 ? 0 : 1] = seg_of(P, T);
            }
            }
            x = first + P.pages;
            if (x >= end) break;
            next_segment(A, P, T);
        }
    }

    if (!ROWS) {
        // The slots in order of position; neighbours of one segment are put
        // together by all threads: thread = (row, four channels) of one of them.
        __syncthreads();
        const int begin = l < 2 * WV ? seg_s[l].begin : -1;
        for (uint64_t left = __ballot(begin >= 0); left;) {
            const int i = __builtin_ctzll(left);
            const uint64_t same = __ballot(begin == __builtin_amdgcn_readlane(begin, i));
            left &= ~same;
            const int j = 64 - __builtin_clzll(same);               // slots i .. j - 1, empty ones between them
            const Seg S = seg_s[i];
            const bool whole = S.begin >= b0 && S.begin + S.pages + A.seg_cost <= b1;
            for (int e = threadIdx.x; e < A.slot_rows * LPR; e += blockDim.x) {
                const int r = e / LPR, c4 = 4 * (e % LPR);
                Part a = no_part();
                f32x4_t o = {0.f, 0.f, 0.f, 0.f};
                for (int k0 = i; k0 < j; k0 += 4) {
                    float4 ms[4];
                    f32x4_t v[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int k = (same >> (k0 + u)) & 1 ? k0 + u : i;
                        const float* from = lds + (k * A.slot_rows + r) * RW;
                        ms[u] = *reinterpret_cast<const float4*>(from + 64 * NP);
                        v[u] = *reinterpret_cast<const f32x4_t*>(from + c4);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if ((same >> (k0 + u)) & 1) join(a, o, unpacked(ms[u]), v[u]);
                }
                if (whole) {
                    const typename AT::Out to = out_row(A, S, r);
                    if (to) put(A, to, c4, o, a, inverse(a.sum));
                } else {
                    const uint32_t at = part_at(blockIdx.x, S.begin >= b0, r);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, o), rp, (int)(at + 4 * c4), 0, kCoherent);
                    if (c4 == 0)
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, packed(a)), rp,
                                                               (int)(at + 256 * NP), 0, kCoherent);
                }
            }
            if (!whole) {
                sent = true;
                if (threadIdx.x == 0) cut_s[S.begin < b0 ? 0 : 1] = S;
            }
        }
    }
    if (!sent) return;                            // uniform over the block
    if constexpr (AT::kJoinLater) {
        __syncthreads();
        const Seg S = cut_s[1];                   // the segment that begins here and goes on behind the piece
        if (S.begin < 0) return;
        int w0, w1;
        blocks_of(A, piece, S.begin, S.pages, w0, w1);
        for (int i = threadIdx.x; i < S.n; i += blockDim.x) later(A, S, i, w0, w1 - w0 + 1);
        return;
    }

    // Arrivals: of the segment that continues into this piece, and of the one
    // that goes on behind it (the same one if it spans the piece).
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's stores have completed
    __syncthreads();
    if (threadIdx.x < 2) {
        const Seg S = cut_s[threadIdx.x];
        int done = 0;
        if (S.begin >= 0) {
            int w0, w1;
            blocks_of(A, piece, S.begin, S.pages, w0, w1);
            done = tile_arrive(A.arrived + w0, A.tag, w1 - w0 + 1);
        }
        done_s[threadIdx.x] = done;
    }
    __syncthreads();
#pragma nounroll
    for (int k = 0; k < 2; ++k) {
        if (!done_s[k]) continue;
        const Seg S = cut_s[k];
        int w0, w1;
        blocks_of(A, piece, S.begin, S.pages, w0, w1);
        const int parts = w1 - w0 + 1;
        const int lanes = A.slot_rows * LPR, bd = blockDim.x;           // (row, four channels)
        auto load = [&](int p, int e, u32x4_t& v, u32x4_t& ms) {
            const uint32_t at = part_at(w0 + p, p == 0, e / LPR);
            v = __builtin_amdgcn_raw_buffer_load_b128(rp, (int)(at + 16 * (e % LPR)), 0, kCoherent);
            ms = __builtin_amdgcn_raw_buffer_load_b128(rp, (int)(at + 256 * NP), 0, kCoherent);
        };
        auto joined = [&](Part& a, f32x4_t& o, u32x4_t ms, u32x4_t v) {
            join(a, o, unpacked(__builtin_bit_cast(float4, ms)), __builtin_bit_cast(f32x4_t, v));
        };
        auto store = [&](int e, f32x4_t o, const Part& a) {
            const typename AT::Out to = out_row(A, S, e / LPR);
            if (to) put(A, to, 4 * (e % LPR), o, a, inverse(a.sum));
        };
        if (2 * lanes > bd) {
            // many rows and few parts: a thread joins four (row, four channels) at once
            for (int e0 = threadIdx.x; e0 < lanes; e0 += 4 * bd) {
                Part a[4];
                f32x4_t o[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    a[u] = no_part();
                    o[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                }
                for (int p0 = 0; p0 < parts; p0 += 2) {
                    u32x4_t v[2][4], ms[2][4];
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int u = 0; u < 4; ++u) load(min(p0 + q, parts - 1), min(e0 + u * bd, lanes - 1), v[q][u], ms[q][u]);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (p0 + q < parts)
#pragma unroll
                            for (int u = 0; u < 4; ++u) joined(a[u], o[u], ms[q][u], v[q][u]);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (e0 + u * bd < lanes) store(e0 + u * bd, o[u], a[u]);
            }
            continue;
        }
        // few rows and many parts: groups of threads take parts in order, eight at once, then the groups are joined
        const int PG = bd / lanes, pg = (int)threadIdx.x / lanes, e = (int)threadIdx.x % lanes;
        Part a = no_part();
        f32x4_t o = {0.f, 0.f, 0.f, 0.f};
        if (pg < PG) {
            const int pe = (pg + 1) * parts / PG;
            for (int p0 = pg * parts / PG; p0 < pe; p0 += 8) {
                u32x4_t v[8], ms[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) load(min(p0 + u, pe - 1), e, v[u], ms[u]);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (p0 + u < pe) joined(a, o, ms[u], v[u]);
            }
        }
        __syncthreads();                                                // LDS is free
        if (pg < PG) {
            *reinterpret_cast<f32x4_t*>(lds + threadIdx.x * 8) = o;
            *reinterpret_cast<float4*>(lds + threadIdx.x * 8 + 4) = packed(a);
        }
        __syncthreads();
        if (pg == 0) {
            for (int u = 1; u < PG; ++u) {
                const float* from = lds + (u * lanes + e) * 8;
                join(a, o, unpacked(*reinterpret_cast<const float4*>(from + 4)), *reinterpret_cast<const f32x4_t*>(from));
            }
            store(e, o, a);
        }
    }
}

// How a call is split (host): a function of the bounds that the batch gives.
struct Split {
    bool rows;                   // a tile of rows for each wave
    int NT, HG, VH, TQ, tiles, slot_rows, waves, blocks, seg_cost, no_cut, min_part, min_piece;
    int64_t all_tiles, units;    // bounds of the batch's tiles and of the line's length
    bool fits;                   // the line can be walked
    size_t part_at, part_bytes, lds, bytes;
};

// Most waves of a block where the waves share a tile: with heads wider than 128
// a wave takes 300 to 371 registers, which 8 waves of a CU do not have.
constexpr int few_waves(int NP) { return NP <= 2 ? 8 : 4; }
// Waves of a block where each has rows of its own: see walk_together.
constexpr int kRowWaves = 8;

// a * b, or anything above 2^62, of numbers up to 2^62
int64_t times(int64_t a, int64_t b) { return a > 0 && b > (1ll << 62) / a ? (1ll << 62) + 1 : a * b; }

// For n_tokens rows in sequences of up to max_q tokens; usual: rows that a sequence has in the mean, where max_q is
// but a bound (0: max_q decides).
[[maybe_unused]] Split split_of(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads, int64_t n_tokens, int max_q,
                                int64_t usual = 0) {
    Split p;
    const int rep = n_heads / c.n_kv, NP = c.head_pad / 64;
    const int64_t most_rows = usual > 0 ? usual : (int64_t)max_q * rep;
    // More than 16 rows get tiles with rows for each wave: sequences of up to 6 tokens and 7 query heads a
    // key head take 27 us so, and 41 in tiles of 16 rows, each of which reads the pages again.  (Up to 128 rows
    // leave most of the 8 waves without any: 64 single tokens with 32 query heads on one key head take 47 us.)
    p.rows = most_rows > 16;
    p.waves = p.rows ? kRowWaves : few_waves(NP);
    // 32 rows a wave use each operand from LDS twice: a prompt 209 us, with 16 rows a wave 299.  Up to 16
    // rows for each of the 8 waves there is nothing to use twice; heads wider than 128 would not fit.
    p.NT = p.rows && most_rows > 16 * kRowWaves && NP <= 2 ? 2 : 1;
    const int RT = p.rows ? 16 * p.NT * kRowWaves : 16;
    const int groups = (rep + RT - 1) / RT;
    p.HG = (rep + groups - 1) / groups;
    p.VH = c.n_kv * groups;
    p.TQ = RT / p.HG;
    p.tiles = (max_q - 1) / p.TQ + 1;
    p.slot_rows = (p.TQ < max_q ? p.TQ : max_q) * p.HG;
    // In pages' time.  Kernel times in us of: one token at 513 positions, at 131072, 64 ragged sequences |
    // sequences of 1 to 6 tokens, a prompt, ragged chunks (those of the head of this file, on the form that
    // walk_together names).
    //   as it is               11.6  63.8  51.6 | 26.8  213  240
    //   seg_cost 0 | 1         11.2  63.3  65.2 | 31.1  303  244
    //   seg_cost 2 | 6         10.9  63.7  51.7 | 27.8  211  241
    //   no_cut 16 | 24         11.6  63.8  51.9 | 27.9  212  246
    //   no_cut 64              11.6  63.5  54.5 |
    //   min_piece 4            11.5  63.7  52.0 | 26.7  217  243
    //   min_piece 16           14.0  64.1  51.2 | 34.8  216  244
    p.seg_cost = p.rows ? 3 : 1;
    p.no_cut = p.rows ? 12 : 32;
    p.min_part = p.rows ? 4 : 8;
    p.min_piece = 8;
    const size_t row = (size_t)(c.head_pad + 4) * sizeof(float);
    p.lds = 32 * 1024 * (size_t)NP;                     // two pages of fp16 operands
    if (!p.rows) {
        while (p.waves * 2 * p.slot_rows * row > 150 * 1024) p.waves /= 2;
        p.lds = p.waves * 2 * p.slot_rows * row;
    }
    if (p.lds < (size_t)p.waves * 64 * 32) p.lds = (size_t)p.waves * 64 * 32;     // the join of parts: 8 floats a thread
    // A sequence of n rows has at most (n - 1) / TQ + 1 tiles: where q_start rises, no more in all than
    // n_tokens / TQ + n_seq, however long max_q lets one sequence be.
    p.all_tiles = std::min((int64_t)b.n_seq * p.tiles, n_tokens / p.TQ + b.n_seq);
    p.units = times(times(p.all_tiles, p.VH), b.max_pages + p.seg_cost);
    const int64_t most = p.units / p.min_piece + 1, cap = device_cus();
    p.blocks = (int)(most < cap ? most : cap);
    // The device counts in 32 bits: units and a piece beyond them (blocks_of()), 64 sequences' tiles.
    p.fits = p.units + p.units / p.blocks + 64 <= 0x7fffffffll && p.tiles < 1 << 24;
    p.part_at = align_up((size_t)p.blocks * sizeof(unsigned long long), 256);
    p.part_bytes = (size_t)p.blocks * 2 * p.slot_rows * row;
    p.bytes = p.part_at + p.part_bytes;
    return p;
}

// Tokens up to which a sequence goes into a launch of its own kind (tiles of 16
// rows, waves that split the pages) before that of the longer ones, 0 where all
// go into one.  In a tile for 8 waves a single token keeps one wave busy, and a
// line of many such segments leaves the long ones too few blocks:
//   a 4096-token prompt and 255 tokens at 1000 positions: one launch 532 us, two 318
//   a 512-token prompt and 31 such tokens:                           66        56
//   2 chunks of 512 and 30 tokens at 20000 positions:               654       280
//   40 chunks of 9 to 243 tokens, none short:                       159.1     159.7
// One launch where the host sees that all sequences are alike, where the longest
// fits one tile, or where there cannot be a short segment for each block: a
// prompt and 15 tokens take 209 us so.  That last rule counts segments, not their
// pages: 2 chunks and 29 tokens at 20000 positions, one segment too few for each
// block, still take 655 us in one launch; with 4 key heads, 2 chunks and 30
// tokens 346 where 62 tokens in two launches take 283.
int short_tokens(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads) {
    const int rep = n_heads / c.n_kv, few = 16 / rep;
    const bool mixed = (int64_t)b.max_q * rep > 256 && b.n_tokens < (int64_t)b.n_seq * b.max_q;
    return mixed && (int64_t)b.n_seq * c.n_kv >= device_cus() ? few : 0;
}

template <int KIND, int NP, int NT, bool ROWS, int kWaves, typename AT>
hipError_t attend_launch(const AT& A, const Split& p, hipStream_t s) {
    if (p.lds > 48 * 1024) {
        const hipError_t e = hipFuncSetAttribute((const void*)k_kv_attend<KIND, NP, NT, ROWS, kWaves, AT>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)p.lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((k_kv_attend<KIND, NP, NT, ROWS, kWaves, AT>), dim3((uint32_t)p.blocks), dim3(64 * p.waves), p.lds, s, A);
    return hipGetLastError();
}

template <int KIND, int NP, typename AT>
hipError_t attend_np(const AT& A, const Split& p, hipStream_t s) {
    if (!p.rows) return attend_launch<KIND, NP, 1, false, few_waves(NP)>(A, p, s);
    if constexpr (NP <= 2)
        if (p.NT == 2) return attend_launch<KIND, NP, 2, true, kRowWaves>(A, p, s);
    return attend_launch<KIND, NP, 1, true, kRowWaves>(A, p, s);
}

template <int KIND, typename AT>
hipError_t attend_kind(const AT& A, const Split& p, hipStream_t s) {
    switch (A.c.head_pad / 64) {
        case 1: return attend_np<KIND, 1>(A, p, s);
        case 2: return attend_np<KIND, 2>(A, p, s);
        case 3: return attend_np<KIND, 3>(A, p, s);
        default: return attend_np<KIND, 4>(A, p, s);
    }
}

// Launches of a call: that of short sequences, if there is one, and that of the others (or all).
struct Launches {
    int few;
    Split split[2];
    Launches(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads) {
        few = short_tokens(c, b, n_heads);
        split[1] = split_of(c, b, n_heads, b.n_tokens, b.max_q);
        split[0] = few > 0 ? split_of(c, b, n_heads, b.n_tokens, few) : split[1];
    }
    bool fit() const { return split[0].fits && split[1].fits; }
};

// The sizes of n_seq, max_q (up to 2^28, as many tokens as a call may have) and max_pages decide, not those of
// n_tokens: a workspace made for a batch serves others of its shape.
size_t workspace_of(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads, const Launches& L) {
    const int max_q = std::min(b.max_q, 1 << 28);
    const size_t all = split_of(c, b, n_heads, times(b.n_seq, max_q), max_q).bytes;
    return align_up(std::max(all, std::max(L.split[0].bytes, L.split[1].bytes)), 256);
}

// No sequence has more rows than the batch.
prox_kv_batch bounded(const prox_kv_batch& b) {
    prox_kv_batch r = b;
    r.max_q = std::max(std::min(b.max_q, b.n_tokens), 1);
    return r;
}

// What a call and what its split give the kernel.
void set_call(Attend& A, const prox_kv_cache& c, const prox_kv_batch& b, const uint16_t* q, int64_t q_stride, int n_heads,
              float scale, int window, uint16_t* out, int64_t out_stride) {
    A.c = c;
    A.b = b;
    A.q = q;
    A.out = out;
    A.qs = q_stride;
    A.os = out_stride;
    A.rep = n_heads / c.n_kv;
    A.window = window;
    A.scale2 = fabsf(scale) * 1.4426950408889634f;
    A.sign = scale < 0.f ? -1.f : 1.f;
}
void set_split(Attend& A, const Split& p) {
    A.part_bytes = (uint32_t)p.part_bytes;
    A.tag = next_call_tag();
    A.HG = p.HG;
    A.HG_inv = (131072u + (uint32_t)p.HG - 1) / (uint32_t)p.HG;
    A.VH = p.VH;
    A.TQ = p.TQ;
    A.tiles = p.tiles;
    A.all_tiles = (int)p.all_tiles;
    A.slot_rows = p.slot_rows;
    A.seg_cost = p.seg_cost;
    A.no_cut = p.no_cut;
    A.min_part = p.min_part;
    A.min_piece = p.min_piece;
}

}  // namespace

}  // namespace prox
