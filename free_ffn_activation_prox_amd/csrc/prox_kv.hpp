// Device helpers of the paged 8-bit key/value cache: where a value lies in a
// page, what a code stands for, and which tokens a batch names.
//
// Page layout.  The products of attention run on v_mfma_f32_16x16x32_f16 (codes
// widened to fp16) with the cache as the A operand (lane l: row l % 16, eight
// values of the reduced dimension at 8 (l / 16)).  Scores reduce over channels,
// K rows are tokens; outputs reduce over tokens, V rows are channels.  A page
// stores each kilobyte that one wave loads (16 bytes a lane, two operands)
// contiguously:
//   K block (64 channels a, 16 tokens b): lane (c = l / 16, d = l % 16) holds
//     channels 64 a + 16 c .. + 15 of token 16 b + d
//   V block (16 channels a): lane (b, c) holds tokens 16 d + 4 b + e, d, e < 4,
//     of channel 16 a + c -- the tokens whose scores the same lane group holds
//     after the first product, so the softmax weights need no exchange of lanes
// The order of the reduced dimension is free as long as both operands share it.
#pragma once

#include "prox.h"
#include "prox_device.hpp"
#include "prox_internal.hpp"

namespace prox {

constexpr int kKvPage = PROX_KV_PAGE;

__host__ __device__ __forceinline__ int kv_k_index(int slot, int ch) {
    return ((((ch >> 6) * 4 + (slot >> 4)) * 4 + ((ch >> 4) & 3)) * 16 + (slot & 15)) * 16 + (ch & 15);
}
__host__ __device__ __forceinline__ int kv_v_index(int slot, int ch) {
    return (((ch >> 4) * 4 + ((slot >> 2) & 3)) * 16 + (ch & 15)) * 16 + (slot >> 4) * 4 + (slot & 3);
}

template <int KIND>
__device__ __forceinline__ float kv_qmax() { return KIND == PROX_KV_INT8 ? 127.f : 448.f; }

// Values of the four codes of a dword (exact).
template <int KIND>
__device__ __forceinline__ void kv_values4(uint32_t w, float v[4]) {
    if constexpr (KIND == PROX_KV_INT8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)(int8_t)(w >> (8 * e));
    } else {
        v[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
        v[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
        v[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
        v[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
    }
}

// Four values in units of the scale -> a dword of codes: clamped, half-even;
// NaN becomes 0.
template <int KIND>
__device__ __forceinline__ uint32_t kv_codes4(const float x[4]) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float m = kv_qmax<KIND>();
        const float c = x[e] > m ? m : (x[e] < -m ? -m : x[e]);
        y[e] = x[e] == x[e] ? c : 0.f;
    }
    if constexpr (KIND == PROX_KV_INT8) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) w |= ((uint32_t)(int)rintf(y[e]) & 0xffu) << (8 * e);
        return w;
    } else {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
    }
}

// The same codes for values that are finite and at most qmax (1 + 2^-23) large:
// nothing to clamp.  int8: adding 1.5 2^23 rounds half-even to a whole number
// and leaves it in the low byte.
template <int KIND>
__device__ __forceinline__ uint32_t kv_codes4_tame(const float x[4]) {
    if constexpr (KIND == PROX_KV_INT8) {
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = __float_as_uint(x[e] + 12582912.f);
        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u),
                                     __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
    } else {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
    }
}

// The rows of sequence s: rows q0 .. q0 + n - 1 (clamped to the batch), of
// which the first `rows` are worked on; row i has position first + i.
struct KvRows {
    int q0, n, rows, first;
};
__device__ __forceinline__ KvRows kv_rows(const prox_kv_batch& b, int s) {
    KvRows r;
    if (b.q_start) {
        r.q0 = min(max(b.q_start[s], 0), b.n_tokens);
        r.n = min(max(b.q_start[s + 1], r.q0), b.n_tokens) - r.q0;
    } else {
        r.q0 = s;
        r.n = 1;
    }
    r.rows = min(r.n, b.max_q);
    r.first = max(b.ctx_len[s], -(1 << 29)) - r.n;   // n_tokens <= 2^28: no overflow
    return r;
}

// The sequence that a row belongs to, the last s with q_start[s] <= row (the
// first one if there is none), found by a whole wave at once: row is the same
// for its lanes.
__device__ __forceinline__ int kv_seq_of(const prox_kv_batch& b, int row, int lane) {
    if (!b.q_start) return row;
    int s = 0;
    for (int base = 1; base < b.n_seq; base += 64) {
        const int j = base + lane;
        const uint64_t m = __ballot(j < b.n_seq && b.q_start[min(j, b.n_seq - 1)] <= row);
        s += __builtin_popcountll(m);
        if (m != ~0ull) break;
    }
    return s;
}

// Sequence and page (counted from the first that the sequence's tokens touch)
// of the i-th such pair of the batch, found by a whole wave at once; false
// behind the last pair.  A sequence with rows has one pair at least.
__device__ __forceinline__ bool kv_pair_of(const prox_kv_batch& b, int i, int lane, int& s, int& j) {
    for (int base = 0; base < b.n_seq; base += 64) {
        int n = 0;
        if (base + lane < b.n_seq) {
            const KvRows R = kv_rows(b, base + lane);
            const int64_t cap = (int64_t)b.max_pages * kKvPage, end = (int64_t)R.first + R.rows;
            const int lo = max(R.first, 0), hi = (int)(end < cap ? end : cap);
            if (R.rows > 0) n = hi > lo ? (hi - 1) / kKvPage - lo / kKvPage + 1 : 1;
        }
        int upto = n;
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
            const int u = __shfl_up(upto, m);
            if (lane >= m) upto += u;
        }
        const uint64_t m = __ballot(upto > i);
        if (m) {
            const int on = __builtin_ctzll(m);
            s = base + on;
            j = i - (__builtin_amdgcn_readlane(upto, on) - __builtin_amdgcn_readlane(n, on));
            return true;
        }
        i -= __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}
}  // namespace prox
