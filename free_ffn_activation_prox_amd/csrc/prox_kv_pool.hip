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
//
// What bounds it: latency.  A step of 64 sequences 6.9 us in one block (8.7 with a
// wave for each sequence).  256 sequences of 290 pages in a pool of 131072, half of
// them ending and half beginning with 256 shared pages, in two launches: 30.6 + 4.9
// (the last block's numbering about half of it; a form that did it all in one block
// took 237).
#include "prox_kv.hpp"

namespace prox {

namespace {

constexpr int kPoolThreads = 1024;
constexpr int kPoolWaves = kPoolThreads / kWave;
constexpr int kChunk4 = 4 * kWave;      // table entries that a wave takes at once
constexpr int kFillBlocks = 1 << 20;    // of k_kv_pages_fill in x: 2^24 sequences of 256 threads would be more than a launch has

struct PoolArgs {
    prox_kv_pool p;
    const int32_t *want, *parent, *shared;
    int32_t *q_start, *slots, *status;
    int n_rows;
    int chunks;                     // of kChunk4 entries in a table row
    uint32_t tag;
    // workspace: arrivals of blocks; what a sequence begins the call with and the first of its new pages in `list`;
    // a bit for each page, set where it is free; the pages given, in order
    unsigned long long* arrived;
    int32_t *start, *from;
    uint32_t* free;
    int32_t* list;
};

__device__ __forceinline__ int pages_of(int tokens) { return (tokens >> 6) + ((tokens & 63) != 0); }
__device__ __forceinline__ int tokens_of(const PoolArgs& A, int s) {
    return min(max(A.p.ctx_len[s], 0), A.p.max_pages * kKvPage);
}
__device__ __forceinline__ int32_t* row_of(const PoolArgs& A, int s) { return A.p.block_table + (size_t)s * A.p.max_pages; }
__device__ __forceinline__ bool is_page(const PoolArgs& A, int page) { return page >= 0 && page < A.p.n_pages; }

// What a sequence takes over and gives back.
struct Move {
    int parent, first;              // its first pages (of `parent`)
    int start;                      // tokens that it begins with
    int lo, hi;                     // table entries given back
};
__device__ __forceinline__ Move move_of(const PoolArgs& A, int s) {
    Move m;
    const int had = tokens_of(A, s), needs = pages_of(max(A.want[s], 0));
    m.parent = -1;
    m.first = 0;
    m.start = had;
    m.lo = needs;
    m.hi = pages_of(had);
    if (A.parent && had == 0) {
        m.parent = A.parent[s];
        const bool is = m.parent >= 0 && m.parent < A.p.n_seq;
        const int first = is ? max(min(A.shared[s], tokens_of(A, m.parent) / kKvPage), 0) : 0;
        m.start = first * kKvPage;
        m.first = min(first, needs);
    }
    return m;
}

// Entries j0 .. j0 + 255 of a sequence's row, one wave each.  Nobody reads a row
// that is written here: a sequence that takes pages over had none.
__device__ __forceinline__ void take_over(const PoolArgs& A, int s, const Move& m, int j0, int l) {
    if (m.first <= j0) return;
    const int32_t* src = row_of(A, m.parent);
    int page[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) page[i] = src[min(j0 + 64 * i + l, m.first - 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + 64 * i + l;
        if (j >= m.first) continue;
        row_of(A, s)[j] = page[i];
        if (is_page(A, page[i])) __hip_atomic_fetch_add(A.p.refs + page[i], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}
template <int SCOPE>
__device__ __forceinline__ void give_back(const PoolArgs& A, int s, int lo, int hi, int j0, int l) {
    if (hi <= j0 || lo >= j0 + kChunk4) return;
    int page[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) page[i] = row_of(A, s)[min(j0 + 64 * i + l, hi - 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + 64 * i + l;
        if (j >= lo && j < hi && is_page(A, page[i])) __hip_atomic_fetch_add(A.p.refs + page[i], -1, __ATOMIC_RELAXED, SCOPE);
    }
}

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int m) {
    const uint32_t lo = (uint32_t)__shfl_up((int)(uint32_t)v, m), hi = (uint32_t)__shfl_up((int)(uint32_t)(v >> 32), m);
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Sums of a and of b up to and with each thread's, in thread order, and of all of them.
__device__ __forceinline__ void block_sums(int64_t& a, int64_t& b, int64_t (*lds)[2], int64_t& all_a, int64_t& all_b) {
    const int l = lane_id(), w = threadIdx.x / kWave;
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) {
        const int64_t u = shfl_up64(a, m), v = shfl_up64(b, m);
        if (l >= m) {
            a += u;
            b += v;
        }
    }
    __syncthreads();
    if (l == kWave - 1) {
        lds[w][0] = a;
        lds[w][1] = b;
    }
    __syncthreads();
    all_a = all_b = 0;
#pragma unroll
    for (int i = 0; i < kPoolWaves; ++i) {
        const int64_t u = lds[i][0], v = lds[i][1];
        all_a += u;
        all_b += v;
        if (i < w) {
            a += u;
            b += v;
        }
    }
}

// Numbers the free pages and gives them out; one block.  FAR: what the launch's
// other blocks counted and stored is read past this one's caches.
template <bool FAR>
__device__ __forceinline__ void number_pages(const PoolArgs& A) {
    __shared__ int64_t sums[kPoolWaves][2];
    __shared__ int free_s[kPoolWaves], taken_s[kPoolWaves], refused_s[kPoolWaves];
    constexpr int kAux = FAR ? kCoherent : 0;
    const int l = lane_id(), w = threadIdx.x / kWave;
    // Free pages: a wave makes the bits of its part of the pool, eight pages a lane and turn, and counts them.
    const __amdgpu_buffer_rsrc_t refs = make_rsrc(A.p.refs, (uint32_t)A.p.n_pages * 4u);
    const int part = (A.p.n_pages + kPoolWaves * 2048 - 1) / (kPoolWaves * 2048) * 2048;
    const int lo = min(w * part, A.p.n_pages), hi = min(lo + part, A.p.n_pages);
    uint8_t* const bytes = reinterpret_cast<uint8_t*>(A.free);
    int n = 0;
    for (int i0 = lo; i0 < hi; i0 += 2048) {
        uint32_t r[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + 512 * k + 8 * l;
            if (i + 8 <= A.p.n_pages) {
                const u32x4_t u = __builtin_amdgcn_raw_buffer_load_b128(refs, 4 * i, 0, kAux);
                const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(refs, 4 * i + 16, 0, kAux);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    r[k][e] = u[e];
                    r[k][4 + e] = v[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)   // loads past the pool give 0: masked below
                    r[k][e] = __builtin_amdgcn_raw_buffer_load_b32(refs, 4 * (i + e), 0, kAux);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t b = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) b |= (i0 + 512 * k + 8 * l + e < hi && (int)r[k][e] <= 0) ? 1u << e : 0u;
            n += __popc(b);
            if (i0 + 512 * k + 8 * l < hi) bytes[(i0 + 512 * k) / 8 + l] = (uint8_t)b;
        }
    }
    n = (int)wave_incl_scan((uint32_t)n);
    if (l == kWave - 1) free_s[w] = n;
    __syncthreads();
    int all = 0, before = 0;
#pragma unroll
    for (int i = 0; i < kPoolWaves; ++i) {
        before += i < w ? free_s[i] : 0;
        all += free_s[i];
    }
    // What the sequences get.  Rows are summed as if none was refused for want of pages, which only the
    // last turns of the loop have to take back.
    int64_t given = 0, rows = 0;       // pages asked for, and rows, of the sequences so far
    int taken = 0, refused = 0;
    for (int s0 = 0; s0 < A.p.n_seq; s0 += kPoolThreads) {
        const int s = s0 + threadIdx.x;
        const bool there = s < A.p.n_seq;
        int start = 0, want = 0, more = 0;
        bool no = false;
        if (there) {
            start = FAR ? __hip_atomic_load(A.start + s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : A.start[s];
            want = max(A.want[s], 0);
            const int has = pages_of(start), needs = pages_of(want);
            no = needs > A.p.max_pages;
            if (want > start && (start & 63) != 0) {           // goes on in a page: it must be its own
                const int page = row_of(A, s)[start >> 6];
                no = no || (is_page(A, page) && (int)__builtin_amdgcn_raw_buffer_load_b32(refs, 4 * page, 0, kAux) > 1);
            }
            more = no ? 0 : max(needs - has, 0);
        }
        int64_t upto = more, behind = no ? 0 : max(want - start, 0), all_more, all_rows;
        block_sums(upto, behind, sums, all_more, all_rows);
        upto += given;
        const bool none_left = more > 0 && upto > all;
        int length = no ? start : want;
        if (given + all_more > all) {                          // some sequence of this turn, or a later one, goes without
            no = no || none_left;
            length = no ? start : want;
            int64_t zero = 0, none;
            behind = max(length - start, 0);
            block_sums(behind, zero, sums, all_rows, none);
        }
        if (there) {
            A.from[s] = (int)min(upto - more, (int64_t)all);
            A.p.ctx_len[s] = length;
            A.q_start[s + 1] = (int)(rows + behind);
            if (!no && more > 0) taken = max(taken, (int)upto);
        }
        refused += __popcll(__ballot(no));
        given += all_more;
        rows += all_rows;
    }
    taken = wave_max(taken);
    if (l == 0) {
        taken_s[w] = taken;
        refused_s[w] = refused;
    }
    __syncthreads();
    refused = 0;
#pragma unroll
    for (int i = 0; i < kPoolWaves; ++i) {
        taken = max(taken, taken_s[i]);
        refused += refused_s[i];
    }
    if (threadIdx.x == 0) {
        A.q_start[0] = 0;
        A.status[0] = refused;
        A.status[1] = all - taken;
    }
    // The lowest free pages, as many as are given: 32 pages a lane and turn.
    for (int i = lo; i < hi && before < taken; i += 2048) {
        const int here = hi - (i + 32 * l);                        // pages of this lane's word
        uint32_t b = here > 0 ? A.free[i / 32 + l] : 0u;
        if (here < 32) b &= here > 0 ? (1u << here) - 1u : 0u;
        const int c = __popc(b), upto = (int)wave_incl_scan((uint32_t)c);
        for (int at = before + upto - c; b && at < taken; ++at, b &= b - 1) A.list[at] = i + 32 * l + __builtin_ctz(b);
        before += __builtin_amdgcn_readlane(upto, 63);
    }
}

// One sequence's new and given-back entries and its rows' slots.
struct Fill {
    int start, length, from, row0;
};
__device__ __forceinline__ Fill fill_of(const PoolArgs& A, int s) {
    return Fill{A.start[s], A.p.ctx_len[s], A.from[s], A.q_start[s]};
}
__device__ __forceinline__ void fill_row(const PoolArgs& A, int s, const Fill& f, int i) {
    const int pos = f.start + i, j = pos >> 6, has = pages_of(f.start);
    const int page = j < has ? row_of(A, s)[j] : A.list[f.from + j - has];
    A.slots[f.row0 + i] = is_page(A, page) ? page * kKvPage + (pos & 63) : -1;
}
__device__ __forceinline__ void fill_entry(const PoolArgs& A, int s, const Fill& f, int j) {
    const int has = pages_of(f.start), needs = pages_of(f.length);
    if (j >= has && j < needs) {
        const int page = A.list[f.from + j - has];
        row_of(A, s)[j] = page;
        A.p.refs[page] = 1;
    } else if (j >= needs && j < has) {
        row_of(A, s)[j] = -1;
    }
}

// Rows behind the last sequence's; i: this thread of n.
__device__ __forceinline__ void clear_rows(const PoolArgs& A, int64_t i, int64_t n) {
    for (int64_t r = A.q_start[A.p.n_seq] + i; r < A.n_rows; r += n) A.slots[r] = -1;
}

// What the block's waves stored and counted is there for all of them.
__device__ __forceinline__ void all_done() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// A call without parents in one block: a lane for each sequence, a wave for those
// with more to do.  Counts move by atomics of the block's own scope, in the L2 cache
// that its loads read, and are loaded only after the last of them.
__global__ void __launch_bounds__(kPoolThreads) k_kv_pages_one(PoolArgs A) {
    constexpr int kFew = 2;                                        // entries and rows that a lane takes by itself
    const int l = lane_id(), w = threadIdx.x / kWave;
    for (int s0 = w * kWave; s0 < A.p.n_seq; s0 += kPoolThreads) {
        int lo = 0, hi = 0;
        if (s0 + l < A.p.n_seq) {
            const int had = tokens_of(A, s0 + l);
            A.start[s0 + l] = had;
            lo = pages_of(max(A.want[s0 + l], 0));
            hi = pages_of(had);
        }
        for (uint64_t some = __ballot(hi > lo); some; some &= some - 1) {
            const int i = __builtin_ctzll(some), from = __builtin_amdgcn_readlane(lo, i), upto = __builtin_amdgcn_readlane(hi, i);
            for (int j = from / kChunk4 * kChunk4; j < upto; j += kChunk4)
                give_back<__HIP_MEMORY_SCOPE_WORKGROUP>(A, s0 + i, from, upto, j, l);
        }
    }
    all_done();
    number_pages<false>(A);
    all_done();
    for (int s0 = w * kWave; s0 < A.p.n_seq; s0 += kPoolThreads) {
        Fill f{0, 0, 0, 0};
        if (s0 + l < A.p.n_seq) f = fill_of(A, s0 + l);
        const int has = pages_of(f.start), needs = pages_of(f.length), rows = max(f.length - f.start, 0);
        const int lo = min(has, needs), hi = max(has, needs);
        const bool few = rows <= kFew && hi - lo <= kFew;
        if (few) {
            for (int i = 0; i < rows && f.row0 + i < A.n_rows; ++i) fill_row(A, s0 + l, f, i);
            for (int j = lo; j < hi; ++j) fill_entry(A, s0 + l, f, j);
        }
        for (uint64_t many = __ballot(!few); many; many &= many - 1) {
            const int i = __builtin_ctzll(many);
            const Fill x{__builtin_amdgcn_readlane(f.start, i), __builtin_amdgcn_readlane(f.length, i),
                         __builtin_amdgcn_readlane(f.from, i), __builtin_amdgcn_readlane(f.row0, i)};
            for (int k = l; k < x.length - x.start && x.row0 + k < A.n_rows; k += kWave) fill_row(A, s0 + i, x, k);
            const int end = __builtin_amdgcn_readlane(hi, i);
            for (int j = __builtin_amdgcn_readlane(lo, i) + l; j < end; j += kWave) fill_entry(A, s0 + i, x, j);
        }
    }
    clear_rows(A, threadIdx.x, kPoolThreads);
}

// A wave for each sequence and kChunk4 entries; the block that arrives last gives the pages out.
__global__ void __launch_bounds__(kPoolThreads) k_kv_pages_move(PoolArgs A) {
    __shared__ int last_s;
    const int l = lane_id(), w = threadIdx.x / kWave;
    const int64_t units = (int64_t)A.p.n_seq * A.chunks;
    for (int64_t u = (int64_t)blockIdx.x * kPoolWaves + w; u < units; u += (int64_t)gridDim.x * kPoolWaves) {
        const int s = (int)(u / A.chunks), c = (int)(u % A.chunks);
        const Move m = move_of(A, s);
        if (c == 0 && l == 0) __hip_atomic_store(A.start + s, m.start, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        take_over(A, s, m, c * kChunk4, l);
        give_back<__HIP_MEMORY_SCOPE_AGENT>(A, s, m.lo, m.hi, c * kChunk4, l);
    }
    all_done();
    if (w == 0) {
        const bool last = kv_arrive(A.arrived, A.tag, blockIdx.x, gridDim.x, l);
        if (l == 0) last_s = last;
    }
    __syncthreads();
    if (last_s) number_pages<true>(A);
}

// blockIdx.x: a sequence (and those kFillBlocks behind it); blockIdx.y: its runs of 256 rows or entries.
__global__ void __launch_bounds__(256) k_kv_pages_fill(PoolArgs A) {
    const int step = gridDim.y * 256, t = blockIdx.y * 256 + threadIdx.x;
    for (int s = blockIdx.x; s < A.p.n_seq; s += gridDim.x) {
        const Fill f = fill_of(A, s);
        const int rows = max(f.length - f.start, 0), entries = max(pages_of(f.start), pages_of(f.length));
        for (int i = t; i < rows && f.row0 + i < A.n_rows; i += step) fill_row(A, s, f, i);
        for (int j = min(pages_of(f.start), pages_of(f.length)) + t; j < entries; j += step) fill_entry(A, s, f, j);
    }
    clear_rows(A, ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x, (int64_t)gridDim.x * gridDim.y * 256);
}

// Most blocks of k_kv_pages_move.
int pool_blocks(const prox_kv_pool& p) {
    const int64_t units = (int64_t)p.n_seq * ((p.max_pages + kChunk4 - 1) / kChunk4);
    return (int)std::min((units + kPoolWaves - 1) / kPoolWaves, (int64_t)2 * device_cus());
}

// Parts of the workspace, in 32-bit words.
struct PoolSpace {
    size_t start, from, free, list, words;
    explicit PoolSpace(const prox_kv_pool& p) {
        start = 2 * (size_t)pool_blocks(p);
        from = start + (size_t)p.n_seq;
        free = from + (size_t)p.n_seq;
        list = free + ((size_t)p.n_pages + 31) / 32;
        words = list + (size_t)p.n_pages;
    }
};

}  // namespace

size_t kv_pages_workspace(const prox_kv_pool& p) { return align_up(PoolSpace(p).words * sizeof(int32_t), 256); }

hipError_t launch_kv_pages(const prox_kv_pool& p, const int32_t* want, const int32_t* parent, const int32_t* shared,
                           int32_t* q_start, int n_rows, int32_t* slots, int32_t* status, void* workspace, hipStream_t s) {
    PoolArgs A{};
    A.p = p;
    A.want = want;
    A.parent = parent;
    A.shared = shared;
    A.q_start = q_start;
    A.slots = slots;
    A.status = status;
    A.n_rows = n_rows;
    A.chunks = (p.max_pages + kChunk4 - 1) / kChunk4;
    A.tag = next_call_tag();
    int32_t* ws = static_cast<int32_t*>(workspace);
    const PoolSpace w(p);
    A.arrived = reinterpret_cast<unsigned long long*>(ws);
    A.start = ws + w.start;
    A.from = ws + w.from;
    A.free = reinterpret_cast<uint32_t*>(ws + w.free);
    A.list = ws + w.list;
    // One block for a step of a token or two each, where the sequences' lanes do it all (calls back to back): 64
    // sequences 9.5 us, in two launches 13.3; 256 sequences and 65000 pages 10.2 and 14.5; 1024 sequences 11.6 and
    // 15.5.  Two launches where sequences begin or take pages over, which are a wave's work each: 16 sequences that
    // end or begin with 200 to 500 tokens 13.3 us, in one block 22.4; 64 with 16 shared pages 15.6 and 72.6.  The
    // rule sees neither what is given back nor how long the tables are: 256 sequences of 290 pages that end in a
    // call of no rows take 179 us in one block, where two launches would take 17.
    if (!parent && n_rows <= 2 * (int64_t)p.n_seq && p.n_seq <= 4096) {
        hipLaunchKernelGGL(k_kv_pages_one, dim3(1), dim3(kPoolThreads), 0, s, A);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(k_kv_pages_move, dim3((uint32_t)pool_blocks(p)), dim3(kPoolThreads), 0, s, A);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // rows of one sequence go to several blocks where there are few sequences
    const int runs = (int)std::min<int64_t>(std::max<int64_t>(device_cus() * 4 / p.n_seq, 1), ((int64_t)n_rows + 255) / 256 + 1);
    hipLaunchKernelGGL(k_kv_pages_fill, dim3((uint32_t)std::min(p.n_seq, kFillBlocks), (uint32_t)runs), dim3(256), 0, s, A);
    return hipGetLastError();
}

}  // namespace prox
