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
// the launch.
#include "prox_kv.hpp"

namespace prox {

namespace {

constexpr int kThreads = 256;

struct RotArgs {
    const float2* rot;
    int half;            // rot_dim / 2 (0: no rotation)
    int halves;          // pairing
    double eps;
};

// Channels c .. c + 7 of one head (TPT neighbouring lanes hold the head; lanes
// with c >= hd take part with zeros), normed by `gain` (nullable) and rotated
// with the table row `rot`.
template <int TPT>
__device__ __forceinline__ void head8(const uint16_t* __restrict__ x, int c, int hd, const float* __restrict__ gain,
                                      const float2* __restrict__ rot, const RotArgs& a, float out[8]) {
    const bool in = c < hd;
    const bool turn = in && c < 2 * a.half;
    double v[8], w[8];
    auto load = [&](int ch, double o[8]) {
        const uint4 u = *reinterpret_cast<const uint4*>(x + ch);
        const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            o[2 * e] = (double)bf16_lo(d[e]);
            o[2 * e + 1] = (double)bf16_hi(d[e]);
        }
    };
    const bool lower = c < a.half;
    const int pc = lower ? c + a.half : c - a.half;      // the other channel of each pair (halves)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = w[e] = 0.0;
    if (in) load(c, v);
    if (a.halves && turn) load(pc, w);
    if (gain) {
        double ss = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fma(v[e], v[e], ss);
#pragma unroll
        for (int m = 1; m < TPT; m *= 2) ss += __shfl_xor(ss, m);
        const double inv = 1.0 / sqrt(ss / (double)hd + a.eps);
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
        const float2* cs = rot + (lower ? c : pc);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 t = cs[e];
            out[e] = (float)(lower ? fma(-w[e], (double)t.y, v[e] * (double)t.x)
                                   : fma(w[e], (double)t.y, v[e] * (double)t.x));
        }
    } else {
        const float2* cs = rot + c / 2;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const double p = v[2 * e], q = v[2 * e + 1];
            if (c + 2 * e < 2 * a.half) {
                const float2 t = cs[e];
                out[2 * e] = (float)fma(-q, (double)t.y, p * (double)t.x);
                out[2 * e + 1] = (float)fma(p, (double)t.y, q * (double)t.x);
            } else {
                out[2 * e] = (float)p;
                out[2 * e + 1] = (float)q;
            }
        }
    }
}

struct Append {
    prox_kv_cache c;
    prox_kv_batch b;
    const uint16_t *k, *v, *q;
    uint16_t* q_out;
    int64_t ks, vs, qs, qos;
    const float *g_q, *g_k;
    RotArgs rot;
    int H, pp;            // query heads; pages that one sequence's tokens can touch
    int kv_blocks;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    b2 r;
    r[0] = (__bf16)lo;
    r[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, r);
}

// One side (K or V) of one page and head: slots s0 .. s1 - 1 come from rows
// row0 + (slot - s0).  Block of 256 threads; every thread passes the barriers.
//   few new slots, scale kept: the new codes are stored where they belong;
//   else the page is put together in LDS -- what it held (requantised where the
//   scale grew), cleared where it begins anew -- and stored whole.
template <int KIND, int TPT, bool VAL>
__device__ void append_side(const Append& A, uint8_t* image, uint32_t* red, int page, int head, int s0, int s1,
                            int row0, int pos0) {
    constexpr int RPP = kThreads / TPT;          // slots of one pass over the threads
    constexpr int NP = kKvPage / RPP;
    constexpr int kDirect = 8;                   // at most so many slots are stored on their own
    const int t = threadIdx.x, c = (t % TPT) * 8, hd = A.c.head_dim, hp = A.c.head_pad;
    const size_t at = (size_t)page * A.c.n_kv + head;
    uint8_t* codes = static_cast<uint8_t*>(VAL ? A.c.v : A.c.k) + at * (size_t)(kKvPage * hp);
    float* scale = (VAL ? A.c.v_scale : A.c.k_scale) + at;
    const bool fresh = s0 == 0;
    const float old = fresh ? 0.f : *scale;

    float r[NP][8];
    uint32_t bits = 0;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        if ((p + 1) * RPP <= s0 || p * RPP >= s1) continue;           // uniform
        const int slot = p * RPP + t / TPT;
        const bool live = slot >= s0 && slot < s1;
        const int row = row0 + (live ? slot - s0 : 0);
        if constexpr (VAL) {
            const uint16_t* x = A.v + (int64_t)row * A.vs + (int64_t)head * hd;
            uint4 u = make_uint4(0, 0, 0, 0);
            if (c < hd) u = *reinterpret_cast<const uint4*>(x + c);
            const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                r[p][2 * e] = bf16_lo(d[e]);
                r[p][2 * e + 1] = bf16_hi(d[e]);
            }
        } else {
            const uint16_t* x = A.k + (int64_t)row * A.ks + (int64_t)head * hd;
            const int pos = pos0 + (live ? slot - s0 : 0);
            head8<TPT>(x, c, hd, A.g_k, A.rot.rot + (int64_t)pos * A.rot.half, A.rot, r[p]);
        }
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
            if ((p + 1) * RPP <= s0 || p * RPP >= s1) continue;
            const int slot = p * RPP + t / TPT;
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
    const float unit = sc > 0.f ? sc : 1.f;
    // x / unit, correctly rounded: with the rounded reciprocal i of unit, y = x i
    // and its exact remainder x - y unit, y + i (x - y unit) is the rounded
    // quotient (Markstein) unless the mantissa of unit is all ones or a number
    // leaves the normal range; those pages, and those with an infinity or NaN,
    // take the division and clamp.  The division alone takes ten instructions
    // a value, all of the rest six.
    const uint32_t ub = __float_as_uint(unit);
    const bool tame = finite && sc > 0x1p-90f && sc < 0x1p90f && (ub & 0x7fffffu) != 0x7fffffu;
    const float inv = 1.f / unit;
    auto codes4 = [&](const float* x) {
        float y[4];
        if (tame) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float q = x[e] * inv;
                y[e] = fmaf(fmaf(-q, unit, x[e]), inv, q);
            }
            return kv_codes4_tame<KIND>(y);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = sc > 0.f ? x[e] / unit : 0.f;
        return kv_codes4<KIND>(y);
    };

    if (whole) {
        for (int i = t; i < kKvPage * hp / 16; i += kThreads) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (!fresh) u = reinterpret_cast<const uint4*>(codes)[i];
            if (grown) {
                uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x[4];
                    kv_values4<KIND>(d[e], x);
#pragma unroll
                    for (int f = 0; f < 4; ++f) x[f] = x[f] * old / unit;
                    d[e] = kv_codes4<KIND>(x);
                }
                u = make_uint4(d[0], d[1], d[2], d[3]);
            }
            reinterpret_cast<uint4*>(image)[i] = u;
        }
        __syncthreads();
    }
    uint8_t* to = whole ? image : codes;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        if ((p + 1) * RPP <= s0 || p * RPP >= s1) continue;
        const int slot = p * RPP + t / TPT;
        if (slot < s0 || slot >= s1 || c >= hd) continue;
        const uint32_t w[2] = {codes4(r[p]), codes4(r[p] + 4)};
        if constexpr (VAL) {
#pragma unroll
            for (int e = 0; e < 8; ++e) to[kv_v_index(slot, c + e)] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
        } else {
            *reinterpret_cast<uint2*>(to + kv_k_index(slot, c)) = make_uint2(w[0], w[1]);
        }
    }
    if (whole) {
        __syncthreads();
        for (int i = t; i < kKvPage * hp / 16; i += kThreads)
            reinterpret_cast<uint4*>(codes)[i] = reinterpret_cast<const uint4*>(image)[i];
    }
}

// grid: first one block per (sequence, page that its tokens can touch, head, K
// or V), then blocks of 256 / TPT (row, query head) pairs.  K and V of a page
// in one block, one after the other, took 20 us for 4096 tokens of 8 heads
// (each block one long chain of loads, a maximum and stores); as blocks of
// their own they run side by side.
template <int KIND, int TPT>
__global__ void __launch_bounds__(kThreads) k_kv_append(Append A) {
    __shared__ __align__(16) uint8_t image[kKvPage * 8 * TPT];
    __shared__ uint32_t red[4];
    const int t = threadIdx.x;
    if ((int)blockIdx.x < A.kv_blocks) {
        const bool val = blockIdx.x & 1;
        const int head = (blockIdx.x >> 1) % A.c.n_kv;
        const int rest = (blockIdx.x >> 1) / A.c.n_kv;
        const int s = rest / A.pp, j = rest % A.pp;
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
        if (val) append_side<KIND, TPT, true>(A, image, red, page, head, s0, s1, row0, a);
        else append_side<KIND, TPT, false>(A, image, red, page, head, s0, s1, row0, a);
        return;
    }
    constexpr int RPP = kThreads / TPT;
    const int64_t id0 = (int64_t)((int)blockIdx.x - A.kv_blocks) * RPP, id = id0 + t / TPT;
    int s = kv_seq_of(A.b, (int)(id0 / A.H), t & 63);
    const int64_t row64 = id / A.H;
    if (row64 >= A.b.n_tokens) return;                       // a head's lanes leave together
    const int row = (int)row64, h = (int)(id - row64 * A.H), c = (t % TPT) * 8, hd = A.c.head_dim;
    s = kv_seq_on(A.b, s, row);
    const KvRows R = kv_rows(A.b, s);
    const int i = row - R.q0;
    if (i < 0 || i >= R.rows) return;
    const int pos = R.first + i;
    const bool seen = pos >= 0 && pos < A.b.max_pages * kKvPage;
    float o[8];
    head8<TPT>(A.q + (int64_t)row * A.qs + (int64_t)h * hd, c, hd, A.g_q,
               A.rot.rot + (int64_t)(seen ? pos : 0) * A.rot.half, A.rot, o);
    if (c >= hd) return;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (seen) u = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
    *reinterpret_cast<uint4*>(A.q_out + (int64_t)row * A.qos + (int64_t)h * hd + c) = u;
}

struct Read {
    prox_kv_cache c;
    prox_kv_batch b;
    void *k, *v;
    int pp;               // pages that one sequence's tokens can touch
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
    const int s = rest / A.pp, j = rest % A.pp;
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

// Pages that the tokens of one sequence can touch: max_q neighbouring
// positions, the first anywhere in a page.
static int pages_touched(const prox_kv_batch& b) {
    const int64_t n = ((int64_t)b.max_q + 2 * kKvPage - 2) / kKvPage;
    return (int)(n < b.max_pages ? n : b.max_pages);
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
    A.rot.eps = (double)r.eps;
    A.H = q ? n_heads : 1;
    A.pp = pages_touched(b);
    const int64_t kvb = (int64_t)b.n_seq * A.pp * c.n_kv * 2;
    const int rpp = kThreads / lanes_per_head(c.head_pad);
    const int64_t qb = q ? ((int64_t)b.n_tokens * n_heads + rpp - 1) / rpp : 0;
    if (kvb + qb > 0x7fffffffll) return hipErrorInvalidConfiguration;
    A.kv_blocks = (int)kvb;
    return c.kind == PROX_KV_INT8 ? append_kind<PROX_KV_INT8>(A, kvb + qb, s)
                                  : append_kind<PROX_KV_FP8>(A, kvb + qb, s);
}

hipError_t launch_kv_read(const prox_kv_cache& c, const prox_kv_batch& b, void* k_out, void* v_out, bool fp32,
                          hipStream_t s) {
    const Read A{c, b, k_out, v_out, pages_touched(b)};
    const int64_t blocks = (int64_t)b.n_seq * A.pp * c.n_kv;
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
