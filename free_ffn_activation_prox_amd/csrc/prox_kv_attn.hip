// Attention over the paged 8-bit key/value cache.
//
// For one row (a token's query head) with the stored codes kc, vc and the
// scales sk, sv of each page:
//   s_j = scale sk (q . kc_j),  o = sum_j exp(s_j - m) sv vc_j / sum_j exp(s_j - m)
// in one pass over the pages with a running maximum m (base 2: log2(e) is
// folded into the scale).  Codes are exact in bf16, so q . kc runs on the bf16
// matrix cores without rounding an operand.  A softmax weight is rounded to
// bf16 (half a step: 2^-9) for the product with the values; dividing by the sum
// of the rounded weights keeps the result a weighted mean, and a row that
// attends to one token alone exact.
//
// A wave takes tiles of 16 rows that share a key head and walks their pages.
// With K as the A operand and q as B, lane (g = l / 16, n = l % 16) gets the scores of row n and tokens
// 16 t + 4 g + r of the page, t, r < 4; the V layout of the cache puts the
// same tokens into lane group g, so the weights go straight into the second
// product, whose result has row n in the same lanes: the running maximum, the
// sums and the rescaling need no exchange but the maximum over the four g.
//
// How the work is split.  A segment is one tile of rows (TQ tokens x HG query
// heads of one key head) with the pages that some row of it sees; all segments'
// pages form one line, cut into equal pieces, one for each wave of the grid,
// whatever the lengths of the sequences.  A wave finds its piece from the
// lengths on the device (the host knows bounds only, and a captured call
// follows the lengths).  A segment inside one piece is finished by its wave;
// one that a cut divides leaves (maximum, sum, unnormalised result) of each
// part in the workspace, at most two parts for each wave, and k_kv_join
// combines them in order of position, so results do not depend on timing.
#include "prox_kv.hpp"

namespace prox {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Eight codes -> eight bf16 (exact).
template <int KIND>
__device__ __forceinline__ uint4 codes_bf16(uint32_t lo, uint32_t hi) {
    if constexpr (KIND == PROX_KV_INT8) {
        uint32_t o[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[4];
            kv_values4<KIND>(h ? hi : lo, v);
#pragma unroll
            for (int e = 0; e < 2; ++e)       // whole numbers below 2^8: the upper halves hold them
                o[2 * h + e] = __builtin_amdgcn_perm(__float_as_uint(v[2 * e + 1]), __float_as_uint(v[2 * e]), 0x07060302u);
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
    } else {
        return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.f, false)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.f, true)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.f, false)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.f, true)));
    }
}

// e4m3 codes with NaN taken as 0: slots that no token was written to may hold
// any byte, and 0 x NaN would reach the sum.
__device__ __forceinline__ uint32_t no_nan_fp8(uint32_t w) {
    const uint32_t n = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
    return w & ~(n * 0xffu);
}

__device__ __forceinline__ float over_groups_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float over_groups_sum(float v) { return xor32_add(xor16_add(v)); }

struct Attend {
    prox_kv_cache c;
    prox_kv_batch b;
    const uint16_t* q;
    uint16_t* out;
    int64_t qs, os;
    float* part_o;         // [workers][2][slot_rows][head_pad]
    float2* part_ml;       // [workers][2][slot_rows]: maximum, sum
    int rep, window;
    int HG, VH;            // query heads of a segment; segments of one tile of tokens (key heads x head groups)
    int TQ, tiles;         // tokens of a tile; most tiles of a sequence
    int slot_rows, workers;
    float scale2;          // scale * log2(e)
};

// One tile of tokens of one sequence.
struct Tile {
    KvRows R;
    int i0, n;             // tokens i0 .. i0 + n - 1 of the sequence's rows
    int pg0, pages;        // pages that some row sees: pg0 .. pg0 + pages - 1; at least one (0: no such tile)
};

__device__ __forceinline__ Tile tile_of(const Attend& A, int s, int t) {
    Tile x;
    x.R = kv_rows(A.b, s);
    x.i0 = t * A.TQ;
    x.n = min(x.R.rows - x.i0, A.TQ);
    const int cap = A.b.max_pages * kKvPage;
    const int p0 = x.R.first + x.i0, p1 = p0 + x.n;                  // positions p0 .. p1 - 1
    const int hi = min(p1, cap), lo = A.window > 0 ? max(p0 - A.window + 1, 0) : 0;
    const bool some = hi > 0 && lo < hi;
    x.pg0 = some ? lo / kKvPage : 0;
    x.pages = x.n <= 0 ? 0 : some ? (hi - 1) / kKvPage + 1 - x.pg0 : 1;
    return x;
}

__device__ __forceinline__ int64_t scan64(int64_t v, int l) {        // inclusive prefix sum over the wave
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        const int64_t u = __shfl_up(v, m);
        if (l >= m) v += u;
    }
    return v;
}

// Pages (over all heads) of the tiles 0 .. count - 1 of the batch, tile =
// sequence * A.tiles + tile of the sequence.
__device__ __forceinline__ int64_t units_before(const Attend& A, int64_t count, int l) {
    int64_t sum = 0;
    for (int64_t j = l; j < count; j += 64) sum += tile_of(A, (int)(j / A.tiles), (int)(j % A.tiles)).pages;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m);
    return sum * A.VH;
}

// The tile that holds unit x of the line, and the unit it begins at.
__device__ __forceinline__ int64_t tile_at(const Attend& A, int64_t x, int l, int64_t* begin) {
    const int64_t all = (int64_t)A.b.n_seq * A.tiles;
    int64_t base = 0;
    for (int64_t j0 = 0; j0 < all; j0 += 64) {
        const int64_t j = j0 + l;
        const int64_t own = j < all ? (int64_t)tile_of(A, (int)(j / A.tiles), (int)(j % A.tiles)).pages * A.VH : 0;
        const int64_t upto = scan64(own, l);
        const uint64_t past = __ballot(base + upto > x);
        if (past) {
            const int at = __builtin_ctzll(past);
            *begin = base + __shfl(upto - own, at);
            return j0 + at;
        }
        base += __shfl(upto, 63);
    }
    *begin = base;
    return all;
}

__device__ __forceinline__ int64_t piece_begin(int64_t w, int64_t total, int workers) { return w * total / workers; }
// The piece that holds unit x: the last w with piece_begin(w) <= x.
__device__ __forceinline__ int64_t piece_of(int64_t x, int64_t total, int workers) {
    return ((x + 1) * workers - 1) / total;
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

// grid: A.workers waves, 64 threads each.  NT tiles of 16 rows a segment.
template <int KIND, int NP, int NT>
__global__ void __launch_bounds__(64) k_kv_attend(Attend A) {
    const int l = threadIdx.x, n = l & 15, g = l >> 4;
    const int hd = A.c.head_dim, cap = A.b.max_pages * kKvPage;
    constexpr int kPageBytes = kKvPage * 64 * NP;
    const int64_t total = units_before(A, (int64_t)A.b.n_seq * A.tiles, l);
    const int64_t end = piece_begin(blockIdx.x + 1, total, A.workers);
    int64_t x = piece_begin(blockIdx.x, total, A.workers);
    if (x >= end) return;
    int64_t begin;
    int64_t tile = tile_at(A, x, l, &begin);
    int s = __builtin_amdgcn_readfirstlane((int)(tile / A.tiles)), t = __builtin_amdgcn_readfirstlane((int)(tile % A.tiles));
    Tile T = tile_of(A, s, t);
    int vh = __builtin_amdgcn_readfirstlane((int)((x - begin) / T.pages));
    int from = __builtin_amdgcn_readfirstlane((int)((x - begin) % T.pages));

    while (x < end) {
        const int upto = (int)min((int64_t)T.pages, from + (end - x));
        const int groups = A.VH / A.c.n_kv, head = vh / groups, grp = vh % groups;
        const int nh = min(A.HG, A.rep - grp * A.HG);                  // heads of this segment
        uint4 q[NT][NP][2];
        int key_lo[NT], key_hi[NT];
        int64_t row_at[NT];                                            // row of the batch and its head, as one
        bool live[NT];
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const int r = 16 * u + n, i = T.i0 + r / A.HG, hq = r % A.HG;
            live[u] = r / A.HG < T.n && hq < nh;
            const int pos = T.R.first + i;
            const bool sees = live[u] && pos >= 0 && pos < cap;
            key_lo[u] = sees && A.window > 0 ? max(pos - A.window + 1, 0) : 0;
            key_hi[u] = sees ? pos + 1 : 0;
            row_at[u] = live[u] ? (int64_t)(T.R.q0 + i) : 0;
            const int h = head * A.rep + grp * A.HG + hq;
            const uint16_t* src = A.q + row_at[u] * A.qs + (int64_t)h * hd;
#pragma unroll
            for (int a = 0; a < NP; ++a)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int ch = 64 * a + 16 * g + 8 * e;
                    q[u][a][e] = live[u] && ch < hd ? *reinterpret_cast<const uint4*>(src + ch) : make_uint4(0, 0, 0, 0);
                }
        }
        const int ctx = T.R.first + T.R.n;                             // slots from here on hold no token
        f32x4_t o[NT][4 * NP];
        float m[NT], sum[NT];
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            m[u] = -INFINITY;
            sum[u] = 0.f;
#pragma unroll
            for (int d = 0; d < 4 * NP; ++d) o[u][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }

        for (int pg = T.pg0 + from; pg < T.pg0 + upto; ++pg) {
            const int page = A.b.block_table[(size_t)s * A.b.max_pages + pg];
            if (page < 0 || page >= A.c.n_pages) continue;
            const size_t where = (size_t)page * A.c.n_kv + head;
            const uint4* kc = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(A.c.k) + where * kPageBytes) + l;
            const uint4* vc = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(A.c.v) + where * kPageBytes) + l;
            const float ks = A.c.k_scale[where] * A.scale2, vs = A.c.v_scale[where];
            float w[NT][4][4];
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                f32x4_t acc[NT];
#pragma unroll
                for (int u = 0; u < NT; ++u) acc[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int a = 0; a < NP; ++a) {
                    const uint4 c = kc[(a * 4 + tt) * 64];
                    const uint4 k0 = codes_bf16<KIND>(c.x, c.y), k1 = codes_bf16<KIND>(c.z, c.w);
#pragma unroll
                    for (int u = 0; u < NT; ++u) acc[u] = mfma16(k0, q[u][a][0], acc[u]);
#pragma unroll
                    for (int u = 0; u < NT; ++u) acc[u] = mfma16(k1, q[u][a][1], acc[u]);
                }
#pragma unroll
                for (int u = 0; u < NT; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int key = pg * kKvPage + 16 * tt + 4 * g + r;
                        w[u][tt][r] = key >= key_lo[u] && key < key_hi[u] ? acc[u][r] * ks : -INFINITY;
                    }
            }
            uint32_t p[NT][4][2];
            float keep[NT];
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                float most = w[u][0][0];
#pragma unroll
                for (int e = 1; e < 16; ++e) most = fmaxf(most, w[u][e >> 2][e & 3]);
                const float m_new = fmaxf(m[u], over_groups_max(most));
                const float base = m_new > -INFINITY ? m_new : 0.f;    // a row that has seen nothing yet
                keep[u] = __builtin_amdgcn_exp2f(m[u] - base);
                m[u] = m_new;
                sum[u] *= keep[u];
#pragma unroll
                for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
                        b2 e;
                        e[0] = (__bf16)__builtin_amdgcn_exp2f(w[u][tt][2 * r] - base);
                        e[1] = (__bf16)__builtin_amdgcn_exp2f(w[u][tt][2 * r + 1] - base);
                        p[u][tt][r] = __builtin_bit_cast(uint32_t, e);
                        sum[u] += bf16_lo(p[u][tt][r]) + bf16_hi(p[u][tt][r]);
                    }
            }
            const bool tail = KIND == PROX_KV_FP8 && (pg + 1) * kKvPage > ctx;
#pragma unroll
            for (int d = 0; d < 4 * NP; ++d) {
                uint4 c = vc[d * 64];
                if (tail) c = make_uint4(no_nan_fp8(c.x), no_nan_fp8(c.y), no_nan_fp8(c.z), no_nan_fp8(c.w));
                const uint4 v0 = codes_bf16<KIND>(c.x, c.y), v1 = codes_bf16<KIND>(c.z, c.w);
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
                    acc = mfma16(v0, make_uint4(p[u][0][0], p[u][0][1], p[u][1][0], p[u][1][1]), acc);
                    acc = mfma16(v1, make_uint4(p[u][2][0], p[u][2][1], p[u][3][0], p[u][3][1]), acc);
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[u][d][r] = fmaf(acc[r], vs, o[u][d][r] * keep[u]);
                }
            }
        }

        const bool done = from == 0 && upto == T.pages;
        const size_t slot = (size_t)blockIdx.x * 2 + (from == 0 ? 1 : 0);
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const float total_sum = over_groups_sum(sum[u]);
            if (!live[u]) continue;
            const int r = 16 * u + n;
            if (done) {
                const float inv = inverse(total_sum);
                uint16_t* to = A.out + row_at[u] * A.os + (int64_t)(head * A.rep + grp * A.HG + r % A.HG) * hd;
#pragma unroll
                for (int d = 0; d < 4 * NP; ++d)
                    if (16 * d + 4 * g < hd) *reinterpret_cast<uint2*>(to + 16 * d + 4 * g) = bf16x4(o[u][d] * inv);
            } else {
                const size_t pr = slot * A.slot_rows + r;
                if (g == 0) A.part_ml[pr] = make_float2(m[u], total_sum);
#pragma unroll
                for (int d = 0; d < 4 * NP; ++d)
                    *reinterpret_cast<f32x4_t*>(A.part_o + pr * (64 * NP) + 16 * d + 4 * g) = o[u][d];
            }
        }

        x += upto - from;
        from = 0;
        if (x < end && ++vh == A.VH) {
            vh = 0;
            do {
                if (++t == A.tiles) {
                    t = 0;
                    ++s;
                }
                T = tile_of(A, s, t);                                   // x < end <= total: a tile follows
            } while (T.pages == 0);
        }
    }
}

// Joins the parts of the segments that more than one wave worked on.  Block:
// one segment and RB of its rows, 256 threads as 64 NP / 4 lanes for each row
// and part; the parts of a row are summed in order of position within a lane
// group and the groups in order, always the same way.
template <int NP, int RB>
__global__ void __launch_bounds__(256) k_kv_join(Attend A, int row_blocks) {
    constexpr int LPR = 16 * NP;                 // lanes of one row, four channels each
    constexpr int GR = 256 / LPR;                // lane groups
    __shared__ float4 acc_s[GR][LPR];
    __shared__ float2 ml_s[GR];
    const int l = threadIdx.x & 63;
    const int64_t seg = blockIdx.x / row_blocks;
    const int rb = blockIdx.x % row_blocks, vh = (int)(seg % A.VH);
    const int64_t tile = seg / A.VH;
    const int s = (int)(tile / A.tiles);
    const Tile T = tile_of(A, s, (int)(tile % A.tiles));
    if (T.pages == 0) return;
    const int64_t all = (int64_t)A.b.n_seq * A.tiles;
    const int64_t before = units_before(A, tile, l);
    int64_t total = before;
    for (int64_t j = tile + l; j - l < all; j += 64) {
        int64_t v = j < all ? (int64_t)tile_of(A, (int)(j / A.tiles), (int)(j % A.tiles)).pages * A.VH : 0;
#pragma unroll
        for (int m = 1; m < 64; m *= 2) v += __shfl_xor(v, m);
        total += v;
    }
    const int64_t a = before + (int64_t)vh * T.pages;
    const int w0 = (int)piece_of(a, total, A.workers), w1 = (int)piece_of(a + T.pages - 1, total, A.workers);
    if (w0 == w1) return;
    const int groups = A.VH / A.c.n_kv, head = vh / groups, grp = vh % groups;
    const int nh = min(A.HG, A.rep - grp * A.HG);
    const int lane = threadIdx.x % LPR, gr = threadIdx.x / LPR;
    const bool in = gr < GR;                     // NP = 3: 16 threads are over
    const int parts = w1 - w0 + 1;
    for (int r = rb * RB; r < min((rb + 1) * RB, A.TQ * A.HG); ++r) {
        const int i = T.i0 + r / A.HG, hq = r % A.HG;
        if (r / A.HG >= T.n || hq >= nh) continue;                      // uniform
        float m = -INFINITY, sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const int pb = gr * parts / GR, pe = in ? (gr + 1) * parts / GR : 0;
        for (int p = pb; p < pe; ++p) {
            // a wave whose piece is empty (more waves than pages) has no part
            if (piece_begin(w0 + p, total, A.workers) == piece_begin(w0 + p + 1, total, A.workers)) continue;
            const size_t pr = ((size_t)(w0 + p) * 2 + (p == 0 ? 1 : 0)) * A.slot_rows + r;
            const float2 ml = A.part_ml[pr];
            const float4 v = reinterpret_cast<const float4*>(A.part_o + pr * (64 * NP))[lane];
            const float mn = fmaxf(m, ml.x), base = mn > -INFINITY ? mn : 0.f;
            const float f = __builtin_amdgcn_exp2f(m - base), e = __builtin_amdgcn_exp2f(ml.x - base);
            m = mn;
            sum = sum * f + ml.y * e;
            o = make_float4(o.x * f + v.x * e, o.y * f + v.y * e, o.z * f + v.z * e, o.w * f + v.w * e);
        }
        __syncthreads();
        if (in) {
            acc_s[gr][lane] = o;
            if (lane == 0) ml_s[gr] = make_float2(m, sum);
        }
        __syncthreads();
        if (gr == 0) {
            for (int p = 1; p < GR; ++p) {
                const float2 ml = ml_s[p];
                const float4 v = acc_s[p][lane];
                const float mn = fmaxf(m, ml.x), base = mn > -INFINITY ? mn : 0.f;
                const float f = __builtin_amdgcn_exp2f(m - base), e = __builtin_amdgcn_exp2f(ml.x - base);
                m = mn;
                sum = sum * f + ml.y * e;
                o = make_float4(o.x * f + v.x * e, o.y * f + v.y * e, o.z * f + v.z * e, o.w * f + v.w * e);
            }
            const float inv = inverse(sum);
            if (4 * lane < A.c.head_dim)
                *reinterpret_cast<uint2*>(A.out + (int64_t)(T.R.q0 + i) * A.os +
                                          (int64_t)(head * A.rep + grp * A.HG + hq) * A.c.head_dim + 4 * lane) =
                    bf16x4(f32x4_t{o.x * inv, o.y * inv, o.z * inv, o.w * inv});
        }
    }
}

// How a call is split (host): a function of the bounds that the batch gives.
struct Split {
    int NT, HG, VH, TQ, tiles, slot_rows, workers;
    size_t part_o, bytes;      // workspace: offset of the results behind the maxima and sums; size
};

Split split_of(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads) {
    Split p;
    const int rep = n_heads / c.n_kv;
    p.NT = (int64_t)b.max_q * rep <= 16 || c.head_pad > 128 ? 1 : 2;
    const int RT = 16 * p.NT;
    const int groups = (rep + RT - 1) / RT;
    p.HG = (rep + groups - 1) / groups;
    p.VH = c.n_kv * groups;
    p.TQ = RT / p.HG;
    p.tiles = (b.max_q + p.TQ - 1) / p.TQ;
    p.slot_rows = (p.TQ < b.max_q ? p.TQ : b.max_q) * p.HG;
    const int64_t most = (int64_t)b.n_seq * p.VH * p.tiles * b.max_pages;
    const int64_t cap = (int64_t)device_cus() * 8;
    p.workers = (int)(most < cap ? most : cap);
    const size_t rows = (size_t)p.workers * 2 * p.slot_rows;
    p.part_o = align_up(rows * sizeof(float2), 256);
    p.bytes = p.part_o + rows * c.head_pad * sizeof(float);
    return p;
}

template <int KIND, int NP>
hipError_t attend_np(const Attend& A, const Split& p, hipStream_t s) {
    const int64_t segs = (int64_t)A.b.n_seq * A.tiles * A.VH;
    const int rb = p.NT == 1 ? p.slot_rows : 1;
    if (segs * rb > 0x7fffffffll) return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)p.workers), join((uint32_t)(segs * rb));
    if (p.NT == 1) {
        hipLaunchKernelGGL((k_kv_attend<KIND, NP, 1>), grid, dim3(64), 0, s, A);
        hipLaunchKernelGGL((k_kv_join<NP, 1>), join, dim3(256), 0, s, A, rb);
    } else if constexpr (NP <= 2) {
        hipLaunchKernelGGL((k_kv_attend<KIND, NP, 2>), grid, dim3(64), 0, s, A);
        hipLaunchKernelGGL((k_kv_join<NP, 32>), join, dim3(256), 0, s, A, rb);
    }
    return hipGetLastError();
}

template <int KIND>
hipError_t attend_kind(const Attend& A, const Split& p, hipStream_t s) {
    switch (A.c.head_pad / 64) {
        case 1: return attend_np<KIND, 1>(A, p, s);
        case 2: return attend_np<KIND, 2>(A, p, s);
        case 3: return attend_np<KIND, 3>(A, p, s);
        default: return attend_np<KIND, 4>(A, p, s);
    }
}

}  // namespace

size_t kv_attention_workspace(const prox_kv_cache& c, const prox_kv_batch& b, int n_heads) {
    return align_up(split_of(c, b, n_heads).bytes + 1, 256);
}

hipError_t launch_kv_attention(const prox_kv_cache& c, const prox_kv_batch& b, const uint16_t* q, int64_t q_stride,
                               int n_heads, float scale, int window, uint16_t* out, int64_t out_stride,
                               void* workspace, hipStream_t s) {
    const Split p = split_of(c, b, n_heads);
    Attend A{};
    A.c = c;
    A.b = b;
    A.q = q;
    A.out = out;
    A.qs = q_stride;
    A.os = out_stride;
    A.part_ml = static_cast<float2*>(workspace);
    A.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.part_o);
    A.rep = n_heads / c.n_kv;
    A.window = window;
    A.HG = p.HG;
    A.VH = p.VH;
    A.TQ = p.TQ;
    A.tiles = p.tiles;
    A.slot_rows = p.slot_rows;
    A.workers = p.workers;
    A.scale2 = scale * 1.4426950408889634f;
    return c.kind == PROX_KV_INT8 ? attend_kind<PROX_KV_INT8>(A, p, s) : attend_kind<PROX_KV_FP8>(A, p, s);
}

}  // namespace prox
