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
// A wave takes 16 rows that share a key head (rows = tokens x query heads of
// the group, token-major) and walks their pages.  With K as the A operand and q
// as B, lane (g = l / 16, n = l % 16) gets the scores of row n and tokens
// 16 t + 4 g + r of the page, t, r < 4; the V layout of the cache puts the
// same tokens into lane group g, so the weights go straight into the second
// product, whose result has row n in the same lanes: the running maximum, the
// sums and the rescaling need no exchange but the maximum over the four g.
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
    int H, rep, tiles, window;
    float scale2;          // scale * log2(e)
};

// grid (row tiles of 16 x key heads x sequences), one wave each.
template <int KIND, int NP>
__global__ void __launch_bounds__(64) k_kv_attend(Attend A) {
    const int tile = blockIdx.x % A.tiles, rest = blockIdx.x / A.tiles;
    const int head = rest % A.c.n_kv, s = rest / A.c.n_kv;
    const int l = threadIdx.x, n = l & 15, g = l >> 4;
    const int hd = A.c.head_dim;
    const KvRows R = kv_rows(A.b, s);
    const int64_t rows = (int64_t)R.rows * A.rep;
    if ((int64_t)tile * 16 >= rows) return;
    const int cap = A.b.max_pages * kKvPage;
    const int64_t row = (int64_t)tile * 16 + n;
    const bool live = row < rows;
    const int i = live ? (int)(row / A.rep) : 0, hq = live ? (int)(row % A.rep) : 0;
    const int pos = R.first + i;
    const bool sees = live && pos >= 0 && pos < cap;
    const int key_lo = sees && A.window > 0 ? max(pos - A.window + 1, 0) : 0, key_hi = sees ? pos + 1 : 0;
    const int64_t at = (int64_t)(R.q0 + i) * A.qs + (int64_t)(head * A.rep + hq) * hd;

    uint4 q[NP][2];
#pragma unroll
    for (int a = 0; a < NP; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int ch = 64 * a + 16 * g + 8 * h;
            q[a][h] = live && ch < hd ? *reinterpret_cast<const uint4*>(A.q + at + ch) : make_uint4(0, 0, 0, 0);
        }

    int lo = sees ? key_lo : 0x7fffffff, hi = key_hi;
#pragma unroll
    for (int m = 1; m < 16; m *= 2) {
        lo = min(lo, __shfl_xor(lo, m));
        hi = max(hi, __shfl_xor(hi, m));
    }
    const int ctx = R.first + R.n;              // slots from here on hold no token
    f32x4_t o[4 * NP];
#pragma unroll
    for (int d = 0; d < 4 * NP; ++d) o[d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, sum = 0.f;
    const int page_bytes = kKvPage * 64 * NP;

    for (int pg = lo / kKvPage; pg * kKvPage < hi; ++pg) {
        const int page = A.b.block_table[(size_t)s * A.b.max_pages + pg];
        if (page < 0 || page >= A.c.n_pages) continue;
        const size_t where = (size_t)page * A.c.n_kv + head;
        const uint4* kc = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(A.c.k) + where * page_bytes) + l;
        const uint4* vc = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(A.c.v) + where * page_bytes) + l;
        const float ks = A.c.k_scale[where] * A.scale2, vs = A.c.v_scale[where];
        float w[4][4];
        float most = -INFINITY;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int a = 0; a < NP; ++a) {
                const uint4 u = kc[(a * 4 + t) * 64];
                acc = mfma16(codes_bf16<KIND>(u.x, u.y), q[a][0], acc);
                acc = mfma16(codes_bf16<KIND>(u.z, u.w), q[a][1], acc);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int key = pg * kKvPage + 16 * t + 4 * g + r;
                w[t][r] = key >= key_lo && key < key_hi ? acc[r] * ks : -INFINITY;
                most = fmaxf(most, w[t][r]);
            }
        }
        const float m_new = fmaxf(m, over_groups_max(most));
        const float base = m_new > -INFINITY ? m_new : 0.f;       // a row that has seen nothing yet
        const float keep = __builtin_amdgcn_exp2f(m - base);
        m = m_new;
        sum *= keep;
        uint32_t p[4][2];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                typedef __bf16 b2 __attribute__((ext_vector_type(2)));
                b2 x;
                x[0] = (__bf16)__builtin_amdgcn_exp2f(w[t][2 * r] - base);
                x[1] = (__bf16)__builtin_amdgcn_exp2f(w[t][2 * r + 1] - base);
                p[t][r] = __builtin_bit_cast(uint32_t, x);
                sum += bf16_lo(p[t][r]) + bf16_hi(p[t][r]);
            }
        const bool tail = KIND == PROX_KV_FP8 && (pg + 1) * kKvPage > ctx;
#pragma unroll
        for (int d = 0; d < 4 * NP; ++d) {
            uint4 u = vc[d * 64];
            if (tail) u = make_uint4(no_nan_fp8(u.x), no_nan_fp8(u.y), no_nan_fp8(u.z), no_nan_fp8(u.w));
            f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
            acc = mfma16(codes_bf16<KIND>(u.x, u.y), make_uint4(p[0][0], p[0][1], p[1][0], p[1][1]), acc);
            acc = mfma16(codes_bf16<KIND>(u.z, u.w), make_uint4(p[2][0], p[2][1], p[3][0], p[3][1]), acc);
#pragma unroll
            for (int r = 0; r < 4; ++r) o[d][r] = fmaf(acc[r], vs, o[d][r] * keep);
        }
    }
    sum = over_groups_sum(sum);
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);   // NaN stays
    if (!live) return;
    uint16_t* to = A.out + (int64_t)(R.q0 + i) * A.os + (int64_t)(head * A.rep + hq) * hd;
#pragma unroll
    for (int d = 0; d < 4 * NP; ++d) {
        const int ch = 16 * d + 4 * g;
        if (ch >= hd) continue;
        typedef __bf16 b4 __attribute__((ext_vector_type(4)));
        b4 x;
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = (__bf16)(o[d][r] * inv);
        *reinterpret_cast<uint2*>(to + ch) = __builtin_bit_cast(uint2, x);
    }
}

template <int KIND>
hipError_t attend_kind(const Attend& A, uint32_t blocks, hipStream_t s) {
    switch (A.c.head_pad / 64) {
        case 1: hipLaunchKernelGGL((k_kv_attend<KIND, 1>), dim3(blocks), dim3(64), 0, s, A); break;
        case 2: hipLaunchKernelGGL((k_kv_attend<KIND, 2>), dim3(blocks), dim3(64), 0, s, A); break;
        case 3: hipLaunchKernelGGL((k_kv_attend<KIND, 3>), dim3(blocks), dim3(64), 0, s, A); break;
        default: hipLaunchKernelGGL((k_kv_attend<KIND, 4>), dim3(blocks), dim3(64), 0, s, A); break;
    }
    return hipGetLastError();
}

}  // namespace

size_t kv_attention_workspace(const prox_kv_cache&, const prox_kv_batch&, int) { return 256; }

hipError_t launch_kv_attention(const prox_kv_cache& c, const prox_kv_batch& b, const uint16_t* q, int64_t q_stride,
                               int n_heads, float scale, int window, uint16_t* out, int64_t out_stride,
                               void* workspace, hipStream_t s) {
    (void)workspace;
    Attend A{};
    A.c = c;
    A.b = b;
    A.q = q;
    A.out = out;
    A.qs = q_stride;
    A.os = out_stride;
    A.H = n_heads;
    A.rep = n_heads / c.n_kv;
    A.window = window;
    A.scale2 = scale * 1.4426950408889634f;
    const int64_t tiles = ((int64_t)b.max_q * A.rep + 15) / 16;
    const int64_t blocks = tiles * c.n_kv * b.n_seq;
    if (blocks > 0x7fffffffll) return hipErrorInvalidConfiguration;
    A.tiles = (int)tiles;
    return c.kind == PROX_KV_INT8 ? attend_kind<PROX_KV_INT8>(A, (uint32_t)blocks, s)
                                  : attend_kind<PROX_KV_FP8>(A, (uint32_t)blocks, s);
}

}  // namespace prox
