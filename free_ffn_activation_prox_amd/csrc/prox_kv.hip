// Paged 8-bit key/value cache: appending tokens and reading them back.
//
// Append, for a token at position p and a head x of k (q the same, to bf16):
//   y = x / sqrt(mean(x^2) + eps) * g         (optional)
//   (a, b) -> (a cos_p - b sin_p, a sin_p + b cos_p) for the pairs of channels
//   r = fp32(y),  scale = max(old scale, fp32(max|r| / qmax)),  code = r / scale
// The norm and the rotation run in fp64 (bf16 x fp32 products are exact there),
// rounded once, so that a code does not depend on how a kernel orders its sums:
// one code of an 8-bit cache is up to 2^-4 of a value, far more than the
// rounding that would flip it.  The work is a few operations a byte moved; what
// bounds the call is reading q, k, v once and, for one token, the latency of
// the launch.  Kernel times, with 32 query and 8 key heads of 128 channels:
//   one token 4.0 us (latency); 64 sequences of one 7.3 us (10 MB: latency, each
//   page's scale and codes read before they are written); 4096 tokens 23.6 us
//   (117 MB, 5.0 TB/s); read-back of 32768 tokens 50 us (201 MB, 4.0 TB/s), as
//   fp32 105 us (336 MB, 3.2 TB/s).
#include <algorithm>

#include "prox_kv.hpp"

namespace prox {

namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;

struct RotArgs {
    const float2* rot;
    int half;            // rot_dim / 2 (0: no rotation)
    int halves;          // pairing
    int wide;            // table rows are 16-byte aligned
    double eps, inv_hd;  // inv_hd: 1 / head_dim
};

// Channels c .. c + 7 of one head, held by TPT neighbouring lanes (lanes with
// c >= hd take part with zeros): the place of a lane in a head, and the cos and
// sin of its pairs at one position.
template <int TPT>
struct Head8 {
    const RotArgs& a;
    int c, pc, hd;       // channels; halves: those they are paired with
    bool in, turn, lower;
    float2 cs[8];        // halves: of the eight channels; interleaved: of the four pairs

    __device__ __forceinline__ Head8(const RotArgs& r, int ch, int n) : a(r), c(ch), hd(n) {
        in = c < hd;
        turn = in && c < 2 * a.half;
        lower = c < a.half;
        pc = lower ? c + a.half : c - a.half;
    }
    // the table's row of position pos (a loaded pair takes 8 bytes: 16-byte loads where rows are aligned)
    __device__ __forceinline__ void at(int pos) {
        if (!turn) return;
        const float2* src = a.rot + (int64_t)pos * a.half + (a.halves ? (lower ? c : pc) : c / 2);
        if (a.wide && a.halves) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) two(src, e);
        } else if (a.wide && c + 8 <= 2 * a.half) {
#pragma unroll
            for (int e = 0; e < 4; e += 2) two(src, e);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (a.halves || (e < 4 && c + 2 * e < 2 * a.half)) cs[e] = src[e];
        }
    }
    __device__ __forceinline__ void two(const float2* src, int e) {
        const float4 f = *reinterpret_cast<const float4*>(src + e);
        cs[e] = make_float2(f.x, f.y);
        cs[e + 1] = make_float2(f.z, f.w);
    }
    __device__ __forceinline__ void load(const uint16_t* x, uint4& own, uint4& other) const {
        own = other = make_uint4(0, 0, 0, 0);
        if (in) own = *reinterpret_cast<const uint4*>(x + c);
        if (a.halves && turn) other = *reinterpret_cast<const uint4*>(x + pc);
    }
    // normed by `gain` (nullable) and rotated, rounded once
    __device__ __forceinline__ void finish(const uint4& own, const uint4& other, const float* __restrict__ gain, float out[8]) const {
        double v[8], w[8];
        auto wide_of = [](const uint4& u, double o[8]) {
            const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[2 * e] = (double)bf16_lo(d[e]);
                o[2 * e + 1] = (double)bf16_hi(d[e]);
            }
        };
        wide_of(own, v);
        wide_of(other, w);
        if (gain) {
            double ss = 0.0;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fma(v[e], v[e], ss);
#pragma unroll
            for (int m = 1; m < TPT; m *= 2) ss += __shfl_xor(ss, m);
            // 1 / sqrt from the hardware's estimate and two Newton steps: the
            // library's square root and division took most of a chunk's time
            const double x = fma(ss, a.inv_hd, a.eps);
            double inv = __builtin_amdgcn_rsq(x);
#pragma unroll
            for (int e = 0; e < 2; ++e) inv = fma(0.5 * inv, fma(-x * inv, inv, 1.0), inv);
            if (in) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = v[e] * inv * (double)gain[c + e];
            }
            if (a.halves && turn) {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = w[e] * inv * (double)gain[pc + e];
            }
        }
        if (!turn) {
#pragma unroll
            for (int e = 0; e < 8; ++e) out[e] = (float)v[e];
        } else if (a.halves) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double s = lower ? -(double)cs[e].y : (double)cs[e].y;
                out[e] = (float)fma(w[e], s, v[e] * (double)cs[e].x);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const double p = v[2 * e], q = v[2 * e + 1];
                if (c + 2 * e < 2 * a.half) {
                    out[2 * e] = (float)fma(-q, (double)cs[e].y, p * (double)cs[e].x);
                    out[2 * e + 1] = (float)fma(p, (double)cs[e].y, q * (double)cs[e].x);
                } else {
                    out[2 * e] = (float)p;
                    out[2 * e + 1] = (float)q;
                }
            }
        }
    }
};

// Sequence s and page j of it for pair i of the grid (see page_pairs).
__device__ __forceinline__ bool pair_of(const prox_kv_batch& b, int pp, int i, int lane, int& s, int& j) {
    if (pp == 0) return kv_pair_of(b, i, lane, s, j);
    s = i / pp;
    j = i % pp;
    return true;
}

struct Append {
    prox_kv_cache c;
    prox_kv_batch b;
    const uint16_t *k, *v, *q;
    uint16_t* q_out;
    int64_t ks, vs, qs, qos;
    const float *g_q, *g_k;
    RotArgs rot;
    int H, pp;            // query heads; blocks of a sequence, head and side, or 0 (see page_pairs)
    int kv_blocks;
    int head_blocks, per_lane;   // of q: blocks of one row; heads of one lane, at most kHeads
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    b2 r;
    r[0] = (__bf16)lo;
    r[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, r);
}

// Eight codes of each of four tokens (w) -> a dword of four tokens for each of
// the eight channels.
__device__ __forceinline__ void dwords_of_tokens(const uint2 w[4], uint32_t d[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t a = h ? w[0].y : w[0].x, b = h ? w[1].y : w[1].x, c = h ? w[2].y : w[2].x, e = h ? w[3].y : w[3].x;
        const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400u), ab1 = __builtin_amdgcn_perm(b, a, 0x07030602u);
        const uint32_t ce0 = __builtin_amdgcn_perm(e, c, 0x05010400u), ce1 = __builtin_amdgcn_perm(e, c, 0x07030602u);
        d[4 * h] = __builtin_amdgcn_perm(ce0, ab0, 0x05040100u);
        d[4 * h + 1] = __builtin_amdgcn_perm(ce0, ab0, 0x07060302u);
        d[4 * h + 2] = __builtin_amdgcn_perm(ce1, ab1, 0x05040100u);
        d[4 * h + 3] = __builtin_amdgcn_perm(ce1, ab1, 0x07060302u);
    }
}

// A page in LDS: 16 bytes between its kilobytes, so that the same place of
// several kilobytes lies in different banks.
__device__ __forceinline__ int in_image(int at) { return at + (at >> 10) * 16; }

// Codes of x / unit, correctly rounded.  With the rounded reciprocal i of unit,
// y = x i and its exact remainder x - y unit, y + i (x - y unit) is the rounded
// quotient (Markstein) unless the mantissa of unit is all ones or a number
// leaves the normal range; a page with such a scale, or with an infinity or
// NaN, is not `tame` and takes the division and clamp.  The division alone
// takes ten instructions a value, all of the rest six.
template <int KIND>
struct Quotient {
    float unit, inv;
    bool tame, zero;
    __device__ __forceinline__ Quotient(float scale, bool finite) {
        zero = !(scale > 0.f);
        unit = zero ? 1.f : scale;
        tame = finite && scale > 0x1p-90f && scale < 0x1p90f && (__float_as_uint(unit) & 0x7fffffu) != 0x7fffffu;
        inv = 1.f / unit;
    }
    __device__ __forceinline__ uint32_t tame4(const float* x) const {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float q = x[e] * inv;
            y[e] = fmaf(fmaf(-q, unit, x[e]), inv, q);
        }
        return kv_codes4_tame<KIND>(y);
    }
    __device__ __forceinline__ uint32_t codes4(const float* x) const {
        if (tame) return tame4(x);
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = zero ? 0.f : x[e] / unit;
        return kv_codes4<KIND>(y);
    }
};

// Eight channels of one row of K (normed and rotated for position pos) or V;
// a lane that holds none (`off`) takes part with zeros.
template <int TPT, bool VAL>
__device__ __forceinline__ void row8(const Append& A, int row, int head, int c, int pos, bool off, float r[8]) {
    const int hd = A.c.head_dim;
    if constexpr (VAL) {
        const uint16_t* x = A.v + (int64_t)row * A.vs + (int64_t)head * hd;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (!off && c < hd) u = *reinterpret_cast<const uint4*>(x + c);
        const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[2 * e] = bf16_lo(d[e]);
            r[2 * e + 1] = bf16_hi(d[e]);
        }
    } else {
        Head8<TPT> head8(A.rot, c, hd);
        uint4 own, other;
        head8.load(A.k + (int64_t)row * A.ks + (int64_t)head * hd, own, other);
        head8.at(pos);
        head8.finish(own, other, A.g_k, r);
    }
}

// One token into a page that it begins or that keeps its scale (nearly every
// single token): every wave finds out alike, without LDS, and the first lanes
// store.  Returns whether that was the case.
template <int KIND, int TPT, bool VAL>
__device__ __forceinline__ bool append_one(const Append& A, int page, int head, int slot, int row, int pos) {
    const int t = threadIdx.x, c = (t % TPT) * 8, hp = A.c.head_pad;
    const size_t at = (size_t)page * A.c.n_kv + head;
    float* scale = (VAL ? A.c.v_scale : A.c.k_scale) + at;
    const bool fresh = slot == 0;
    const float old = fresh ? 0.f : *scale;
    float r[8];
    row8<TPT, VAL>(A, row, head, c, pos, false, r);
    uint32_t bits = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) bits = max(bits, __float_as_uint(r[e]) << 1);
#pragma unroll
    for (int m = 1; m < TPT; m *= 2) bits = max(bits, (uint32_t)__shfl_xor((int)bits, m));
    const float need = __uint_as_float(bits >> 1) / kv_qmax<KIND>();
    const Quotient<KIND> u(fresh ? need : old, bits < 0xff000000u);
    if (!u.tame || (!fresh && need > old)) return false;
    uint8_t* codes = static_cast<uint8_t*>(VAL ? A.c.v : A.c.k) + at * (size_t)(kKvPage * hp);
    if (fresh) {
        if (t == 0) *scale = need;
        // the other slots' bytes; those of slot 0 lie in 16 bytes of their own (K), or first of 16 (V)
        for (int i = t; i < kKvPage * hp / 16; i += kThreads)
            if (VAL ? (i & 0x30) != 0 : (i & 0xcf) != 0) reinterpret_cast<uint4*>(codes)[i] = make_uint4(0, 0, 0, 0);
    }
    if (t >= TPT || c >= hp) return true;                    // padding channels: zeros
    const uint32_t w[2] = {u.tame4(r), u.tame4(r + 4)};
    if constexpr (VAL) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint8_t* to = codes + kv_v_index(slot, c + e);
            const uint32_t b = (w[e >> 2] >> (8 * (e & 3))) & 0xffu;
            if (fresh) *reinterpret_cast<uint4*>(to) = make_uint4(b, 0, 0, 0);
            else *to = (uint8_t)b;
        }
    } else {
        *reinterpret_cast<uint2*>(codes + kv_k_index(slot, c)) = make_uint2(w[0], w[1]);
    }
    return true;
}

// One side (K or V) of one page and head: slots s0 .. s1 - 1 come from rows
// row0 + (slot - s0).  Block of 256 threads; every thread passes the barriers.
// A thread holds eight channels of four slots: of K, slots 256 / TPT apart, of
// V, neighbours, whose codes make up dwords of the page.
//   few new slots, scale kept: the new codes are stored where they belong;
//   else the page is put together in LDS -- what it held (requantised where the
//   scale grew), cleared where it begins anew -- and stored whole.
template <int KIND, int TPT, bool VAL>
__device__ void append_side(const Append& A, uint8_t* image, uint32_t* red, int page, int head, int s0, int s1,
                            int row0, int pos0) {
    constexpr int RPP = kThreads / TPT;          // slots of one pass over the threads
    constexpr int NP = VAL ? (TPT > 16 ? TPT / 4 : 4) : kKvPage / RPP;
    constexpr int kDirect = 8;                   // at most so many slots are stored on their own
    const int t = threadIdx.x, c = (t % TPT) * 8, hd = A.c.head_dim, hp = A.c.head_pad;
    const size_t at = (size_t)page * A.c.n_kv + head;
    uint8_t* codes = static_cast<uint8_t*>(VAL ? A.c.v : A.c.k) + at * (size_t)(kKvPage * hp);
    float* scale = (VAL ? A.c.v_scale : A.c.k_scale) + at;
    const bool fresh = s0 == 0;
    const float old = fresh ? 0.f : *scale;
    // the slot of this thread's p-th values, and whether pass p has any slot of the call
    auto slot_of = [&](int p) { return VAL ? (p >> 2) * 4 * RPP + (t / TPT) * 4 + (p & 3) : p * RPP + t / TPT; };
    auto idle = [&](int p) { return VAL ? (p >> 2) * 4 * RPP >= s1 || ((p >> 2) + 1) * 4 * RPP <= s0 : p * RPP >= s1 || (p + 1) * RPP <= s0; };

    float r[NP][8];
    uint32_t bits = 0;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        if (idle(p)) continue;                                        // uniform
        const int slot = slot_of(p);
        const bool live = slot >= s0 && slot < s1;
        const int row = row0 + (live ? slot - s0 : 0);
        row8<TPT, VAL>(A, row, head, c, pos0 + (live ? slot - s0 : 0), !live, r[p]);
        if (live) {
#pragma unroll
            for (int e = 0; e < 8; ++e) bits = max(bits, __float_as_uint(r[p][e]) << 1);    // by magnitude, NaN on top
        }
    }
    // the largest magnitude of the block; an infinity or NaN among them (rare)
    // is left out in a second round
    auto over_block = [&](uint32_t v) {
#pragma unroll
        for (int m = 1; m < 64; m *= 2) v = max(v, (uint32_t)__shfl_xor((int)v, m));
        if ((t & 63) == 0) red[t >> 6] = v;
        __syncthreads();
        v = max(max(red[0], red[1]), max(red[2], red[3]));
        __syncthreads();
        return v;
    };
    bits = over_block(bits);
    const bool finite = bits < 0xff000000u;
    if (!finite) {
        bits = 0;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            if (idle(p)) continue;
            const int slot = slot_of(p);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t b = __float_as_uint(r[p][e]) << 1;
                if (slot >= s0 && slot < s1 && b < 0xff000000u) bits = max(bits, b);
            }
        }
        bits = over_block(bits);
    }
    const float most = __uint_as_float(bits >> 1);
    const float sc = fmaxf(old, most / kv_qmax<KIND>());
    const bool grown = sc > old && old > 0.f;
    const bool whole = fresh || grown || s1 - s0 > kDirect;
    if (t == 0 && sc != old) *scale = sc;
    if (t == 0 && fresh) *scale = sc;
    const Quotient<KIND> u(sc, finite);

    if (whole) {
        for (int i = t; i < kKvPage * hp / 16; i += kThreads) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (!fresh) v = reinterpret_cast<const uint4*>(codes)[i];
            if (grown) {
                uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x[4];
                    kv_values4<KIND>(d[e], x);
#pragma unroll
                    for (int f = 0; f < 4; ++f) x[f] = x[f] * old / u.unit;
                    d[e] = kv_codes4<KIND>(x);
                }
                v = make_uint4(d[0], d[1], d[2], d[3]);
            }
            *reinterpret_cast<uint4*>(image + in_image(16 * i)) = v;
        }
        __syncthreads();
    }
    if constexpr (VAL) {
#pragma unroll
        for (int p = 0; p < NP; p += 4) {
            const int slot = slot_of(p);
            if (slot >= s1 || slot + 4 <= s0 || c >= hd) continue;
            uint2 w[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) w[f] = make_uint2(u.codes4(r[p + f]), u.codes4(r[p + f] + 4));
            uint32_t d[8];
            dwords_of_tokens(w, d);
            const bool all = slot >= s0 && slot + 4 <= s1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = kv_v_index(slot, c + e);
                uint8_t* to = whole ? image + in_image(i) : codes + i;
                if (all) {
                    *reinterpret_cast<uint32_t*>(to) = d[e];
                } else {
#pragma unroll
                    for (int f = 0; f < 4; ++f)
                        if (slot + f >= s0 && slot + f < s1) to[f] = (uint8_t)(d[e] >> (8 * f));
                }
            }
        }
    } else {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            if (idle(p)) continue;
            const int slot = slot_of(p);
            if (slot < s0 || slot >= s1 || c >= hd) continue;
            const int i = kv_k_index(slot, c);
            *reinterpret_cast<uint2*>(whole ? image + in_image(i) : codes + i) = make_uint2(u.codes4(r[p]), u.codes4(r[p] + 4));
        }
    }
    if (whole) {
        __syncthreads();
        for (int i = t; i < kKvPage * hp / 16; i += kThreads)
            reinterpret_cast<uint4*>(codes)[i] = *reinterpret_cast<const uint4*>(image + in_image(16 * i));
    }
}

// grid: first one block per (sequence, page that its tokens can touch, head, K
// or V), then blocks of one row and 256 / TPT heads for each of A.per_lane turns,
// which share the row of the table.  K and V of a page
// in one block, one after the other, took 20 us for 4096 tokens of 8 heads
// (each block one long chain of loads, a maximum and stores); as blocks of
// their own they run side by side.
template <int KIND, int TPT>
__global__ void __launch_bounds__(kThreads) k_kv_append(Append A) {
    __shared__ __align__(16) uint8_t image[(kKvPage + 1) * 8 * TPT];    // 16 bytes more for each kilobyte
    __shared__ uint32_t red[4];
    const int t = threadIdx.x;
    if ((int)blockIdx.x < A.kv_blocks) {
        const bool val = blockIdx.x & 1;
        const int head = (blockIdx.x >> 1) % A.c.n_kv;
        const int rest = (blockIdx.x >> 1) / A.c.n_kv;
        int s, j;
        if (!pair_of(A.b, A.pp, rest, t & 63, s, j)) return;
        const KvRows R = kv_rows(A.b, s);
        if (R.rows <= 0 || R.first + R.rows <= 0) return;
        const int lo = max(R.first, 0);
        const int hi = min((int64_t)R.first + R.rows, (int64_t)A.b.max_pages * kKvPage);   // positions lo .. hi - 1
        const int pg = lo / kKvPage + j;
        const int a = max(lo, pg * kKvPage), b = min(hi, (pg + 1) * kKvPage);
        if (a >= b) return;
        const int page = A.b.block_table[(size_t)s * A.b.max_pages + pg];
        if (page < 0 || page >= A.c.n_pages) return;
        const int s0 = a - pg * kKvPage, s1 = b - pg * kKvPage, row0 = R.q0 + (a - R.first);
        if (s1 - s0 == 1) {
            if (val ? append_one<KIND, TPT, true>(A, page, head, s0, row0, a)
                    : append_one<KIND, TPT, false>(A, page, head, s0, row0, a)) return;
        }
        if (val) append_side<KIND, TPT, true>(A, image, red, page, head, s0, s1, row0, a);
        else append_side<KIND, TPT, false>(A, image, red, page, head, s0, s1, row0, a);
        return;
    }
    constexpr int RPP = kThreads / TPT;
    const int bq = (int)blockIdx.x - A.kv_blocks, row = bq / A.head_blocks, c = (t % TPT) * 8, hd = A.c.head_dim;
    const int h0 = (bq - row * A.head_blocks) * RPP * A.per_lane + t / TPT;
    const int s = kv_seq_of(A.b, row, t & 63);
    const KvRows R = kv_rows(A.b, s);
    const int i = row - R.q0;
    if (i < 0 || i >= R.rows) return;
    const int pos = R.first + i;
    const bool seen = pos >= 0 && pos < A.b.max_pages * kKvPage;
    Head8<TPT> head8(A.rot, c, hd);
    uint4 own[kHeads], other[kHeads];
    const uint16_t* x = A.q + (int64_t)row * A.qs;
#pragma unroll
    for (int k = 0; k < kHeads; ++k)
        if (k < A.per_lane) head8.load(x + (int64_t)min(h0 + k * RPP, A.H - 1) * hd, own[k], other[k]);
    head8.at(seen ? pos : 0);
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
        if (k >= A.per_lane) continue;
        float o[8];
        head8.finish(own[k], other[k], A.g_q, o);
        if (c >= hd || h0 + k * RPP >= A.H) continue;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (seen) u = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
        *reinterpret_cast<uint4*>(A.q_out + (int64_t)row * A.qos + (int64_t)(h0 + k * RPP) * hd + c) = u;
    }
}

struct Read {
    prox_kv_cache c;
    prox_kv_batch b;
    void *k, *v;
    int pp;               // blocks of a sequence and head, or 0 (see page_pairs)
};

// Four codes of each of eight channels (a dword a channel, a byte a token) ->
// the eight codes of token e.
__device__ __forceinline__ uint2 token_of_dwords(const uint32_t d[8], int e) {
    const uint32_t one = (uint32_t)e | ((uint32_t)(e + 4) << 8);            // byte e of both operands
    auto pair = [&](uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, one); };
    const uint32_t p0 = pair(d[0], d[1]), p1 = pair(d[2], d[3]), p2 = pair(d[4], d[5]), p3 = pair(d[6], d[7]);
    return make_uint2(__builtin_amdgcn_perm(p1, p0, 0x05040100u), __builtin_amdgcn_perm(p3, p2, 0x05040100u));
}

// grid: one block per (sequence, page that its tokens can touch, head).  A
// thread turns 16 channels of a token (K, as they are stored) or eight channels
// of four tokens (V, bytes exchanged in registers) at a time; eight or sixteen
// neighbouring lanes write one token's channels.  Bound by the output, two or
// four bytes for each byte read.
template <int KIND, bool FP32>
__global__ void __launch_bounds__(kThreads) k_kv_read(Read A) {
    const int hd = A.c.head_dim, hp = A.c.head_pad, t = threadIdx.x;
    const int head = blockIdx.x % A.c.n_kv, rest = blockIdx.x / A.c.n_kv;
    int s, j;
    if (!pair_of(A.b, A.pp, rest, t & 63, s, j)) return;
    const KvRows R = kv_rows(A.b, s);
    if (R.rows <= 0) return;
    auto store = [&](void* out, int row, int c, const float* x) {
        const int64_t o = ((int64_t)row * A.c.n_kv + head) * hd + c;
        if constexpr (FP32) {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + o);
            p[0] = make_float4(x[0], x[1], x[2], x[3]);
            p[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o) =
                make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
        }
    };
    const float zero[8] = {};
    const int cap = A.b.max_pages * kKvPage;
    const int lo = max(R.first, 0), hi = (int)min((int64_t)R.first + R.rows, (int64_t)cap);   // positions that exist
    if (j == 0) {
        // rows whose position does not exist: those before `lo`, those from `hi` on
        const int n8 = hd / 8, before = min(R.rows, max(lo - R.first, 0)), from = min(R.rows, max(max(hi, lo) - R.first, 0));
        const int64_t n = (int64_t)(before + R.rows - from) * n8;
        for (int64_t e = t; e < n; e += kThreads) {
            const int i = (int)(e / n8), row = R.q0 + (i < before ? i : from + i - before), c = (int)(e % n8) * 8;
            store(A.k, row, c, zero);
            store(A.v, row, c, zero);
        }
    }
    const int pg = lo / kKvPage + j;
    const int a = max(lo, pg * kKvPage), b = min(hi, (pg + 1) * kKvPage);
    if (a >= b) return;
    const int page = A.b.block_table[(size_t)s * A.b.max_pages + pg];
    const bool there = page >= 0 && page < A.c.n_pages;
    const int s0 = a - pg * kKvPage, s1 = b - pg * kKvPage, row0 = R.q0 + (a - R.first) - s0;   // slot x: row row0 + x
    const size_t at = (size_t)(there ? page : 0) * A.c.n_kv + head;
    const uint8_t* kc = static_cast<const uint8_t*>(A.c.k) + at * (size_t)(kKvPage * hp);
    const uint8_t* vc = static_cast<const uint8_t*>(A.c.v) + at * (size_t)(kKvPage * hp);
    const float ks = A.c.k_scale[at], vs = A.c.v_scale[at];
    auto put = [&](void* out, int slot, int c, uint2 w, float scale) {
        float x[8];
        kv_values4<KIND>(w.x, x);
        kv_values4<KIND>(w.y, x + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = there ? x[e] * scale : 0.f;
        store(out, row0 + slot, c, x);
    };
    const int n16 = hp / 16, first = s0 / 4 * 4;
    for (int e = t; e < (s1 - first) * n16; e += kThreads) {
        const int slot = first + e / n16, c = e % n16 * 16;
        if (slot < s0 || c >= hd) continue;
        const uint4 u = *reinterpret_cast<const uint4*>(kc + kv_k_index(slot, c));
        put(A.k, slot, c, make_uint2(u.x, u.y), ks);
        if (c + 8 < hd) put(A.k, slot, c + 8, make_uint2(u.z, u.w), ks);
    }
    const int n8 = hp / 8;
    for (int e = t; e < (s1 - first + 3) / 4 * n8; e += kThreads) {
        const int slot = first + e / n8 * 4, c = e % n8 * 8;
        if (c >= hd) continue;
        uint32_t d[8];
#pragma unroll
        for (int f = 0; f < 8; ++f) d[f] = *reinterpret_cast<const uint32_t*>(vc + kv_v_index(slot, c + f));
#pragma unroll
        for (int f = 0; f < 4; ++f)
            if (slot + f >= s0 && slot + f < s1) put(A.v, slot + f, c, token_of_dwords(d, f), vs);
    }
}

template <int KIND>
hipError_t append_kind(const Append& A, int64_t blocks, hipStream_t s) {
    const dim3 g((uint32_t)blocks), t(kThreads);
    if (A.c.head_pad <= 64) hipLaunchKernelGGL((k_kv_append<KIND, 8>), g, t, 0, s, A);
    else if (A.c.head_pad <= 128) hipLaunchKernelGGL((k_kv_append<KIND, 16>), g, t, 0, s, A);
    else hipLaunchKernelGGL((k_kv_append<KIND, 32>), g, t, 0, s, A);
    return hipGetLastError();
}

int lanes_per_head(int hp) { return hp <= 64 ? 8 : hp <= 128 ? 16 : 32; }

}  // namespace

// Blocks for the pages that a batch's tokens can touch.  Each sequence gets as
// many as max_q neighbouring positions can touch (pp, the first of them anywhere
// in a page), or, where that would leave half of the blocks without work, pp is
// 0 and the blocks find their pairs of sequence and page in the lengths: there
// are (n + 126) / 64 at most for n tokens, so (n_tokens + 126 n_seq) / 64 in all.
// A 4096-token prompt beside 255 single tokens of 8 key heads: append 216 us
// with pp blocks a sequence, 55 us so; read 82 and 16 us.  Where few blocks would
// be idle, to find the pairs costs more than it saves: one token 4.0 -> 4.7 us,
// 64 tokens of as many sequences 7.3 -> 9.2, read of 32768 tokens 49 -> 51.
static int64_t page_pairs(const prox_kv_batch& b, int& pp) {
    const int64_t n = ((int64_t)std::min(b.max_q, b.n_tokens) + 2 * kKvPage - 2) / kKvPage;
    pp = (int)(n < b.max_pages ? n : b.max_pages);
    const int64_t each = (int64_t)b.n_seq * pp, found = (b.n_tokens + (2 * kKvPage - 2) * (int64_t)b.n_seq) / kKvPage;
    if (2 * found > each) return each;
    pp = 0;
    return found;
}

hipError_t launch_kv_append(const prox_kv_cache& c, const prox_kv_batch& b, const uint16_t* k, int64_t k_stride,
                            const uint16_t* v, int64_t v_stride, const prox_kv_rotation& r, int n_heads,
                            const uint16_t* q, int64_t q_stride, uint16_t* q_out, int64_t q_out_stride,
                            hipStream_t s) {
    Append A{};
    A.c = c;
    A.b = b;
    A.k = k;
    A.v = v;
    A.q = q;
    A.q_out = q_out;
    A.ks = k_stride;
    A.vs = v_stride;
    A.qs = q_stride;
    A.qos = q_out_stride;
    A.g_q = r.g_q;
    A.g_k = r.g_k;
    A.rot.rot = reinterpret_cast<const float2*>(r.rot);
    A.rot.half = r.rot ? r.rot_dim / 2 : 0;
    A.rot.halves = r.pairing == PROX_ROPE_HALVES;
    A.rot.wide = (uintptr_t)r.rot % 16 == 0 && A.rot.half % 2 == 0;
    A.rot.eps = (double)r.eps;
    A.rot.inv_hd = 1.0 / c.head_dim;
    A.H = q ? n_heads : 1;
    const int64_t kvb = page_pairs(b, A.pp) * c.n_kv * 2;
    const int rpp = kThreads / lanes_per_head(c.head_pad);
    // Several heads a lane share the row of the table (a 4096-token prompt 22.7 us, with one head a lane
    // 27.4); few rows make more blocks of one head a lane (64 tokens 7.3 us, with several 8.0).
    A.per_lane = (int64_t)b.n_tokens * n_heads <= 4 * rpp * device_cus() ? 1 : std::min(kHeads, (n_heads + rpp - 1) / rpp);
    A.head_blocks = (n_heads + rpp * A.per_lane - 1) / (rpp * A.per_lane);
    const int64_t qb = q ? (int64_t)b.n_tokens * A.head_blocks : 0;
    if (kvb + qb > 0x7fffffffll) return hipErrorInvalidConfiguration;
    A.kv_blocks = (int)kvb;
    return c.kind == PROX_KV_INT8 ? append_kind<PROX_KV_INT8>(A, kvb + qb, s)
                                  : append_kind<PROX_KV_FP8>(A, kvb + qb, s);
}

hipError_t launch_kv_read(const prox_kv_cache& c, const prox_kv_batch& b, void* k_out, void* v_out, bool fp32,
                          hipStream_t s) {
    Read A{c, b, k_out, v_out, 0};
    const int64_t blocks = page_pairs(b, A.pp) * c.n_kv;
    if (blocks > 0x7fffffffll) return hipErrorInvalidConfiguration;
    const dim3 g((uint32_t)blocks), t(kThreads);
    if (c.kind == PROX_KV_INT8) {
        if (fp32) hipLaunchKernelGGL((k_kv_read<PROX_KV_INT8, true>), g, t, 0, s, A);
        else hipLaunchKernelGGL((k_kv_read<PROX_KV_INT8, false>), g, t, 0, s, A);
    } else {
        if (fp32) hipLaunchKernelGGL((k_kv_read<PROX_KV_FP8, true>), g, t, 0, s, A);
        else hipLaunchKernelGGL((k_kv_read<PROX_KV_FP8, false>), g, t, 0, s, A);
    }
    return hipGetLastError();
}

}  // namespace prox
