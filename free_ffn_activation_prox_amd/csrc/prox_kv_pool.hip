// Page tables of the paged key/value cache, kept on the GPU: sequences grow, are
// cut back, end, or begin with the first pages of another one.
//
// With start_s the tokens that sequence s begins the call with (its own, or 64
// per page taken over from its parent), the call
//   1  takes over pages (each one's count up by one) and gives back those from
//      ceil(want / 64) on (count down),
//   2  numbers the pages without a count, and gives sequence s the
//      ceil(want / 64) - ceil(start / 64) next ones, lowest first, in order of
//      the sequences, as long as they last,
//   3  writes the tables, the new pages' counts and the slots of the new rows.
// Which page goes where depends on the state alone, never on timing: the counts
// are whole numbers, and places come from prefix sums.  A page is free where its
// count is 0, so there is no list to keep in order.
#include "prox_kv.hpp"

namespace prox {

namespace {

constexpr int kPoolThreads = 1024;
constexpr int kPoolWaves = kPoolThreads / kWave;

struct PoolArgs {
    prox_kv_pool p;
    const int32_t *want, *parent, *shared;
    int32_t *q_start, *slots, *status;
    int n_rows;
    int32_t *start, *from, *list;   // workspace: a sequence's start and the first of its new pages in `list`
};

__device__ __forceinline__ int pages_of(int tokens) { return (tokens >> 6) + ((tokens & 63) != 0); }
__device__ __forceinline__ int tokens_of(const PoolArgs& A, int s) {
    return min(max(A.p.ctx_len[s], 0), A.p.max_pages * kKvPage);
}
__device__ __forceinline__ int32_t* row_of(const PoolArgs& A, int s) { return A.p.block_table + (size_t)s * A.p.max_pages; }
__device__ __forceinline__ bool is_page(const PoolArgs& A, int page) { return page >= 0 && page < A.p.n_pages; }

// 1: one wave for each sequence.  Nobody reads a row that this phase writes: a
// sequence that takes pages over had none, so it has none to give.
template <int SCOPE>
__device__ __forceinline__ void take_and_give_back(const PoolArgs& A, int s, int l) {
    const int had = tokens_of(A, s), needs = pages_of(max(A.want[s], 0));
    int start = had;
    if (A.parent && had == 0) {
        const int p = A.parent[s];
        const int first = p >= 0 && p < A.p.n_seq ? max(min(A.shared[s], tokens_of(A, p) / kKvPage), 0) : 0;
        const int32_t* src = row_of(A, first > 0 ? p : s);
        for (int j = l; j < min(first, needs); j += kWave) {
            const int page = src[j];
            row_of(A, s)[j] = page;
            if (is_page(A, page)) __hip_atomic_fetch_add(A.p.refs + page, 1, __ATOMIC_RELAXED, SCOPE);
        }
        start = first * kKvPage;
    }
    for (int j = needs + l; j < pages_of(had); j += kWave) {
        const int page = row_of(A, s)[j];
        if (is_page(A, page)) __hip_atomic_fetch_add(A.p.refs + page, -1, __ATOMIC_RELAXED, SCOPE);
    }
    if (l == 0) A.start[s] = start;
}

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int m) {
    const uint32_t lo = (uint32_t)__shfl_up((int)(uint32_t)v, m), hi = (uint32_t)__shfl_up((int)(uint32_t)(v >> 32), m);
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Sums of v up to and with each thread's, in thread order, and of all of them.
__device__ __forceinline__ int64_t block_sums(int64_t v, int64_t* lds, int64_t& total) {
    const int l = lane_id(), w = threadIdx.x / kWave;
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) {
        const int64_t u = shfl_up64(v, m);
        if (l >= m) v += u;
    }
    if (l == kWave - 1) lds[w] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int i = 0; i < kPoolWaves; ++i) {
        const int64_t c = lds[i];
        total += c;
        if (i < w) v += c;
    }
    __syncthreads();
    return v;
}

// 2: one block.
__device__ __forceinline__ void number_pages(const PoolArgs& A) {
    __shared__ int64_t sums[kPoolWaves];
    __shared__ int free_s[kPoolWaves];
    const int l = lane_id(), w = threadIdx.x / kWave;
    // free pages: a wave counts those of its part of the pool
    const int part = (A.p.n_pages + kPoolWaves - 1) / kPoolWaves;
    const int lo = min(w * part, A.p.n_pages), hi = min(lo + part, A.p.n_pages);
    int n = 0;
    for (int i = lo; i < hi; i += kWave) n += __popcll(__ballot(i + l < hi && A.p.refs[min(i + l, hi - 1)] <= 0));
    if (l == 0) free_s[w] = n;
    __syncthreads();
    int all = 0, before = 0;
#pragma unroll
    for (int i = 0; i < kPoolWaves; ++i) {
        before += i < w ? free_s[i] : 0;
        all += free_s[i];
    }
    // what the sequences get
    int64_t given = 0, rows = 0;       // pages asked for and rows of the sequences so far
    int taken = 0;                     // pages given
    int refused = 0;
    for (int s0 = 0; s0 < A.p.n_seq; s0 += kPoolThreads) {
        const int s = s0 + threadIdx.x;
        const bool there = s < A.p.n_seq;
        int start = 0, want = 0, more = 0;
        bool no = false;
        if (there) {
            start = A.start[s];
            want = max(A.want[s], 0);
            const int has = pages_of(start), needs = pages_of(want);
            no = needs > A.p.max_pages;
            if (want > start && (start & 63) != 0) {           // goes on in a page: it must be its own
                const int page = row_of(A, s)[start >> 6];
                no = no || (is_page(A, page) && A.p.refs[page] > 1);
            }
            more = no ? 0 : max(needs - has, 0);
        }
        int64_t all_more, all_rows;
        const int64_t upto = given + block_sums(more, sums, all_more);
        no = no || (more > 0 && upto > all);
        const int length = no ? start : want;
        const int64_t behind = rows + block_sums(max(length - start, 0), sums, all_rows);
        if (there) {
            A.from[s] = (int)min(upto - more, (int64_t)all);
            A.p.ctx_len[s] = length;
            A.q_start[s + 1] = (int)behind;
            if (!no && more > 0) taken = max(taken, (int)upto);
            refused += no ? 1 : 0;
        }
        given += all_more;
        rows += all_rows;
    }
    int64_t none;
    taken = wave_max(taken);
    if (l == 0) free_s[w] = taken;
    block_sums(refused, sums, none);
#pragma unroll
    for (int i = 0; i < kPoolWaves; ++i) taken = max(taken, free_s[i]);
    if (threadIdx.x == 0) {
        A.q_start[0] = 0;
        A.status[0] = (int)none;
        A.status[1] = all - taken;
    }
    // the lowest free pages, as many as are given
    for (int i = lo; i < hi && before < taken; i += kWave) {
        const bool is = i + l < hi && A.p.refs[min(i + l, hi - 1)] <= 0;
        const uint64_t m = __ballot(is);
        const int at = before + lanes_below(m);
        if (is && at < taken) A.list[at] = i + l;
        before += __popcll(m);
    }
}

// 3: one wave for each sequence.
__device__ __forceinline__ void fill(const PoolArgs& A, int s, int l) {
    const int start = A.start[s], length = A.p.ctx_len[s], from = A.from[s];
    const int has = pages_of(start), needs = pages_of(length);
    int32_t* row = row_of(A, s);
    const int row0 = A.q_start[s];
    for (int i = l; i < length - start && row0 + i < A.n_rows; i += kWave) {
        const int pos = start + i, j = pos >> 6, page = j < has ? row[j] : A.list[from + j - has];
        A.slots[row0 + i] = is_page(A, page) ? page * kKvPage + (pos & 63) : -1;
    }
    for (int j = has + l; j < needs; j += kWave) {
        const int page = A.list[from + j - has];
        row[j] = page;
        A.p.refs[page] = 1;
    }
    for (int j = needs + l; j < has; j += kWave) row[j] = -1;
}

// Rows behind the last sequence's; i: this thread of n.
__device__ __forceinline__ void clear_rows(const PoolArgs& A, int i, int n) {
    for (int r = A.q_start[A.p.n_seq] + i; r < A.n_rows; r += n) A.slots[r] = -1;
}

// What the block's waves stored and counted is there for all of them.
__device__ __forceinline__ void all_done() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// The whole call in one block.  Counts move by atomics of the block's own scope, in the L2 cache that its
// loads read, and are loaded only after the last of them.
__global__ void __launch_bounds__(kPoolThreads) k_kv_pages(PoolArgs A) {
    const int l = lane_id(), w = threadIdx.x / kWave;
    for (int s = w; s < A.p.n_seq; s += kPoolWaves) take_and_give_back<__HIP_MEMORY_SCOPE_WORKGROUP>(A, s, l);
    all_done();
    number_pages(A);
    all_done();
    for (int s = w; s < A.p.n_seq; s += kPoolWaves) fill(A, s, l);
    clear_rows(A, threadIdx.x, kPoolThreads);
}

}  // namespace

size_t kv_pages_workspace(const prox_kv_pool& p) {
    return align_up(((size_t)p.n_seq * 2 + (size_t)p.n_pages) * sizeof(int32_t), 256);
}

hipError_t launch_kv_pages(const prox_kv_pool& p, const int32_t* want, const int32_t* parent, const int32_t* shared,
                           int32_t* q_start, int n_rows, int32_t* slots, int32_t* status, void* workspace, hipStream_t s) {
    PoolArgs A{p, want, parent, shared, q_start, slots, status, n_rows, nullptr, nullptr, nullptr};
    A.start = static_cast<int32_t*>(workspace);
    A.from = A.start + p.n_seq;
    A.list = A.from + p.n_seq;
    hipLaunchKernelGGL(k_kv_pages, dim3(1), dim3(kPoolThreads), 0, s, A);
    return hipGetLastError();
}

}  // namespace prox
