// Managing the pages of a paged KV cache (decode_attn_paged.h): the pages that no sequence uses,
// rows that continue other rows, and the pages in use moved to the front of the cache.
//
// All of it follows from the block table and the lengths, so nothing is kept between calls and
// nothing can fall out of step with them. A bitmap with one bit per page says what is in use;
// the number of used pages before a page (a population count of the words before it) gives its
// place in every list, so the lists come out in ascending order whatever the timing:
//
//     free page f:      free_pages[f - used_before(f)] = f
//     n pages in use:   hole i < n, not used,  holes[i - used_before(i)] = i
//                       mover i >= n, used,    movers[used_before(i) - used_before(n)] = i
//     (as many holes as movers), and the k-th mover goes to the k-th hole.
//
// What bounds them: the copies the bytes (512 beams with half a page of 512 KB each 35.8 us, 6.3 TB/s read and written;
// 1.5 thousand pages of 128 KB moved 70 us, of which 60 the copy, 6.5 TB/s), the lists latency: three launches that wait for one
// another, each with one or two loads that do (357000 pages, 257000 entries 12.9 us; a small pool by one block 4.8 us).

#include "paged_common.cuh"

namespace da_impl {

constexpr int kPageThreads = 256;
constexpr int kCopyUnits = 4;                                  // 16-byte units per thread and chunk
constexpr int kCopyChunk = kPageThreads * kCopyUnits;          // units per chunk
constexpr int kOneThreads = 1024;                              // of the block that plans alone
constexpr int kOneWords = 7168;                                // words of its bitmap
constexpr int kOneRows = 1024;                                 // rows that it takes
constexpr int kRowEntries = 128;                               // block-table entries that a warp takes at a time

struct RowsParams {
    const int32_t* lens;
    const int32_t* table;
    uint32_t* err;
    int B, max_pages, table_stride, P, num_pages;

    // The length of row b as it counts, and its pages.
    __device__ __forceinline__ int length(int b) const {
        const int len = ld_cg_s32(lens + b);
        if (len >= 0 && len <= static_cast<int64_t>(max_pages) * P) return len;
        flag_error(err, DA_DEVERR_SEQLENS);
        return 0;
    }
    __device__ __forceinline__ int pages(int b) const { return pages_of(length(b), P); }
};

// The workspace of a plan: bitmap, count of movers, lists.
struct PlanSpace {
    uint32_t* bits;      // [words]
    int32_t* count;      // {movers, pages in use}
    int32_t* holes;      // [num_pages]
    int32_t* movers;     // [num_pages]
    int32_t* rank;       // [num_pages]: of a mover among the movers
};

// Marks the pages that the rows use: a warp per run of entries, or (below) one block.
template <int THREADS>
__device__ __forceinline__ void mark_pages(const RowsParams& p, uint32_t* bits) {
    const int lane = threadIdx.x & 31;
    const int64_t pieces = (p.max_pages + kRowEntries - 1) / kRowEntries, items = p.B * pieces;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (THREADS / 32);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5); i < items; i += warps) {
        const int b = static_cast<int>(i / pieces), from = static_cast<int>(i - b * pieces) * kRowEntries;
        const int to = min(p.pages(b), from + kRowEntries);
        const int32_t* row = p.table + static_cast<int64_t>(b) * p.table_stride;
#pragma unroll 4
        for (int e = from + lane; e < to; e += 32) {
            const int page = ld_cg_s32(row + e);
            if (page >= 0 && page < p.num_pages) atomicOr(bits + (page >> 5), 1u << (page & 31));
            else flag_error(p.err, DA_DEVERR_PAGE);
        }
    }
}

// One block: the rows' pages first, then all entries alike, so that no load waits for another row's length.
__device__ __forceinline__ void mark_pages_one(const RowsParams& p, int* pages, uint32_t* marked) {
    for (int b = threadIdx.x; b < p.B; b += kOneThreads) pages[b] = p.pages(b);
    __syncthreads();
    const int all = p.B * p.max_pages;
    constexpr int kAhead = 8;
    for (int i0 = threadIdx.x; i0 < all; i0 += kAhead * kOneThreads) {
        int page[kAhead];
        bool live[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * kOneThreads, b = i / p.max_pages, e = i - b * p.max_pages;
            live[j] = i < all && e < pages[b];
            page[j] = live[j] ? ld_cg_s32(p.table + static_cast<int64_t>(b) * p.table_stride + e) : 0;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (!live[j]) continue;
            if (page[j] >= 0 && page[j] < p.num_pages) atomicOr(marked + (page[j] >> 5), 1u << (page[j] & 31));
            else flag_error(p.err, DA_DEVERR_PAGE);
        }
    }
}

// (A kernel of its own, not a memset: each of the kernels here is launched before the one in front of it has ended.)
__global__ void __launch_bounds__(kPageThreads) page_clear_kernel(uint32_t* bits, int words) {
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_dependents_launch();
    for (int w = blockIdx.x * kPageThreads + threadIdx.x; w < words; w += gridDim.x * kPageThreads) bits[w] = 0;
}

__global__ void __launch_bounds__(kPageThreads) page_mark_kernel(const RowsParams p, uint32_t* bits) {
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_dependents_launch();
    mark_pages<kPageThreads>(p, bits);
}

// Sum over the block of one int per thread.
template <int THREADS>
__device__ __forceinline__ int block_sum(int x, int* scratch) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    int sum = 0;
    for (int w = 0; w < THREADS / 32; ++w) sum += scratch[w];
    __syncthreads();
    return sum;
}

// The lists, a run of words per block (each counts what lies before its own). With ONE a single block marks the
// pages too, in shared memory.
template <bool COMPACT, bool ONE>
__global__ void __launch_bounds__(ONE ? kOneThreads : kPageThreads)
page_plan_kernel(const RowsParams p, const PlanSpace s, int32_t* free_pages, int32_t* count) {
    constexpr int kT = ONE ? kOneThreads : kPageThreads;
    __shared__ int scratch[kT / 32];
    __shared__ uint32_t marked[ONE ? kOneWords : 1];
    __shared__ int row_pages[ONE ? kOneRows : 1];
    __shared__ uint32_t run_word[kT];
    __shared__ int run_used[kT];
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_dependents_launch();
    const int num_pages = p.num_pages, words = (num_pages + 31) / 32;
    if (ONE) {
        for (int w = threadIdx.x; w < words; w += kT) marked[w] = 0;
        __syncthreads();
        mark_pages_one(p, row_pages, marked);
        __syncthreads();
    }
    auto word_at = [&](int w) { return ONE ? marked[w] : __ldcg(s.bits + w); };
    // used pages among the first `pages`
    auto used_before = [&](int pages) {
        int n = 0;
        const int whole = pages >> 5;
#pragma unroll 8
        for (int w = threadIdx.x; w < whole; w += kT) n += __popc(word_at(w));
        if (threadIdx.x == 0 && (pages & 31)) n += __popc(word_at(whole) & ((1u << (pages & 31)) - 1));
        return block_sum<kT>(n, scratch);
    };
    const int per = (words + gridDim.x - 1) / gridDim.x;
    const int w0 = min(words, static_cast<int>(blockIdx.x) * per), w1 = min(words, w0 + per);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int before = ONE ? 0 : used_before(static_cast<int>(min(static_cast<int64_t>(num_pages), static_cast<int64_t>(w0) * 32)));
    int n = 0, before_n = 0;
    if (COMPACT) {
        n = used_before(num_pages);
        before_n = used_before(n);
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            *count = n;
            s.count[0] = n - before_n;
            s.count[1] = n;
        }
    }
    for (int base = w0; base < w1; base += kT) {
        const int w = base + static_cast<int>(threadIdx.x);
        const uint32_t mine = w < w1 ? word_at(w) : 0u;
        const int own = __popc(mine);
        int run = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, run, off);
            if (lane >= off) run += y;
        }
        if (lane == 31) scratch[warp] = run;
        __syncthreads();
        int at = before + run - own;
        for (int i = 0; i < kT / 32; ++i) {
            if (i < warp) at += scratch[i];
            before += scratch[i];
        }
        run_word[threadIdx.x] = mine;
        run_used[threadIdx.x] = at;
        __syncthreads();
        for (int i = warp; i < min(kT, w1 - base); i += kT / 32) {   // a warp per word, a lane per page
            const uint32_t word = run_word[i];
            const int used0 = run_used[i];
            const int64_t page = static_cast<int64_t>(base + i) * 32 + lane;
            if (page >= num_pages) continue;
            const bool used = (word >> lane) & 1;
            const int k = used0 + __popc(word & ((1u << lane) - 1));
            if (!COMPACT) {
                if (!used) free_pages[page - k] = static_cast<int>(page);
            } else if (page < n) {
                if (!used) s.holes[page - k] = static_cast<int>(page);
            } else if (used) {
                s.movers[k - before_n] = static_cast<int>(page);
                s.rank[page] = k - before_n;
            }
        }
        __syncthreads();
    }
    if (!COMPACT && blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) *count = num_pages - before;
}

struct MoveParams {
    RowsParams rows;
    PlanSpace s;
    uint4 *k, *v;
    float *ks, *vs;
    int Hkv;
    int64_t page_units;      // 16-byte units of a page's keys (or values)
    int32_t* table_out;
    int table_out_stride;
};

// Moves the pages, and writes the table with their new numbers.
__global__ void __launch_bounds__(kPageThreads) page_move_kernel(const MoveParams p) {
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_dependents_launch();
    const int moves = __ldcg(p.s.count), in_use = __ldcg(p.s.count + 1);
    const int64_t chunks = (p.page_units + kCopyChunk - 1) / kCopyChunk;
    const int64_t items = 2 * chunks * moves;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int64_t pair = i / chunks, c = i - pair * chunks;
        const int m = static_cast<int>(pair >> 1);
        const int64_t src = __ldcg(p.s.movers + m), dst = __ldcg(p.s.holes + m);
        uint4* base = (pair & 1) ? p.v : p.k;
        const uint4* from = base + src * p.page_units;
        uint4* to = base + dst * p.page_units;
        const int64_t u0 = c * kCopyChunk + threadIdx.x;
        uint4 x[kCopyUnits];
#pragma unroll
        for (int j = 0; j < kCopyUnits; ++j)
            if (u0 + j * kPageThreads < p.page_units) x[j] = __ldcs(from + u0 + j * kPageThreads);
#pragma unroll
        for (int j = 0; j < kCopyUnits; ++j)
            if (u0 + j * kPageThreads < p.page_units) __stcs(to + u0 + j * kPageThreads, x[j]);
        if (p.ks != nullptr && c == 0) {
            float* scale = (pair & 1) ? p.vs : p.ks;
            for (int h = threadIdx.x; h < p.Hkv; h += kPageThreads) scale[dst * p.Hkv + h] = scale[src * p.Hkv + h];
        }
    }
    const RowsParams& r = p.rows;
    const int lane = threadIdx.x & 31;
    const int64_t pieces = (r.max_pages + kRowEntries - 1) / kRowEntries, all = r.B * pieces;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kPageThreads / 32);
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kPageThreads + threadIdx.x) >> 5; i < all; i += warps) {
        const int b = static_cast<int>(i / pieces), begin = static_cast<int>(i - b * pieces) * kRowEntries;
        const int end = min(r.pages(b), begin + kRowEntries);
        const int32_t* row = r.table + static_cast<int64_t>(b) * r.table_stride;
        int32_t* out = p.table_out + static_cast<int64_t>(b) * p.table_out_stride;
        for (int e = begin + lane; e < end; e += 32) {
            int page = ld_cg_s32(row + e);
            if (page >= in_use && page < r.num_pages) page = __ldcg(p.s.holes + __ldcg(p.s.rank + page));
            out[e] = page;
        }
    }
}

struct ForkParams {
    RowsParams rows;
    const int32_t* parents;
    const int32_t* new_pages;
    int32_t* lens_out;
    int32_t* table_out;
    int table_out_stride, n_out;
    uint4 *k, *v;
    float *ks, *vs;
    int Hkv, layout;
    int row_units;           // 16-byte units of one token and head
    int64_t page_units;
};

// A block per (child, share of its work): what it has to know of the child is four loads that wait for one another, so it
// then copies all its chunks, `split` of them apart.
__global__ void __launch_bounds__(kPageThreads, 6) page_fork_kernel(const ForkParams p, int split) {
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_dependents_launch();
    const RowsParams& r = p.rows;
    const int64_t items = static_cast<int64_t>(p.n_out) * split;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int child = static_cast<int>(i / split), share = static_cast<int>(i - static_cast<int64_t>(child) * split);
        const int parent = ld_cg_s32(p.parents + child), fresh = ld_cg_s32(p.new_pages + child);
        int len = 0;
        if (parent >= 0 && parent < r.B) len = r.length(parent);
        else if (share == 0 && threadIdx.x == 0) flag_error(r.err, DA_DEVERR_SEQLENS);
        const int pages = pages_of(len, r.P), used = len - (pages - 1) * r.P;   // tokens of the last page
        const bool own = fresh >= 0 && len > 0 && used < r.P, writable = own && fresh < r.num_pages;
        const int32_t* row = r.table + static_cast<int64_t>(parent) * r.table_stride;
        const int64_t old = writable ? ld_cg_s32(row + pages - 1) : -1;
        // the row
        if (share == 0 && threadIdx.x == 0) {
            p.lens_out[child] = len;
            if (own && !writable) flag_error(r.err, DA_DEVERR_PAGE);
        }
        int32_t* out = p.table_out + static_cast<int64_t>(child) * p.table_out_stride;
        for (int e = share * kPageThreads + static_cast<int>(threadIdx.x); e < pages; e += split * kPageThreads) {
            const int page = ld_cg_s32(row + e);
            const bool there = page >= 0 && page < r.num_pages;
            if (!there) flag_error(r.err, DA_DEVERR_PAGE);
            out[e] = own && there && e == pages - 1 ? fresh : page;
        }
        if (old < 0 || old >= r.num_pages) continue;
        // the used tokens of its last page: one run, or one per head (a page has at most kMostUnits units)
        const bool thd = p.layout == DA_LAYOUT_VARLEN;
        const uint32_t run = static_cast<uint32_t>(used) * p.row_units * (thd ? p.Hkv : 1), units = thd ? run : run * p.Hkv;
        const uint32_t stride = static_cast<uint32_t>(r.P) * p.row_units;   // of heads, where they lie outside the tokens
        const uint32_t chunks = (units + kCopyChunk - 1) / kCopyChunk;
        for (uint32_t c = share; c < 2 * chunks; c += split) {
            const bool values = c >= chunks;
            const uint32_t u0 = (values ? c - chunks : c) * kCopyChunk + threadIdx.x;
            const uint4* from = (values ? p.v : p.k) + old * p.page_units;
            uint4* to = (values ? p.v : p.k) + fresh * p.page_units;
            uint4 x[kCopyUnits];
            uint32_t at[kCopyUnits];
#pragma unroll
            for (int j = 0; j < kCopyUnits; ++j) {
                const uint32_t u = u0 + j * kPageThreads;
                at[j] = thd ? u : u / run * stride + u % run;
                if (u < units) x[j] = __ldcs(from + at[j]);
            }
#pragma unroll
            for (int j = 0; j < kCopyUnits; ++j)
                if (u0 + j * kPageThreads < units) __stcs(to + at[j], x[j]);
        }
        if (p.ks != nullptr && share == 0) {
            for (int h = threadIdx.x; h < 2 * p.Hkv; h += kPageThreads) {
                float* scale = h < p.Hkv ? p.ks : p.vs;
                const int hh = h < p.Hkv ? h : h - p.Hkv;
                scale[static_cast<int64_t>(fresh) * p.Hkv + hh] = scale[old * p.Hkv + hh];
            }
        }
    }
}

// ------------------------------------------------------------ host side
constexpr int kPageBlocks = 152 * 8;                       // blocks of a kernel that loops over its work
constexpr int64_t kMostUnits = 0x7fffffff;                 // of a page's keys in a fork, which counts them in 32 bits: 32 GB
constexpr int kPlanWords = 64;                             // words of the bitmap that a block plans, at least
constexpr int64_t kOneEntries = 4096;                      // table entries up to which one block plans alone: one launch, not three
                                                           // (1024 entries 4.9 us against 4.4 in a graph, but 5.8 against 9.7
                                                           // of host time; 6300: 5.5 against 5.2; 20000: 10.7 against 8.0)

inline size_t pages_space(int num_pages, PlanSpace* s, uint8_t* ws) {
    const size_t words = (static_cast<size_t>(num_pages) + 31) / 32 * 4, list = static_cast<size_t>(num_pages) * 4;
    size_t at = kPagedHeadBytes;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    const size_t bits = take(words), count = take(8), holes = take(list), movers = take(list), rank = take(list);
    if (s) {
        s->bits = reinterpret_cast<uint32_t*>(ws + bits);
        s->count = reinterpret_cast<int32_t*>(ws + count);
        s->holes = reinterpret_cast<int32_t*>(ws + holes);
        s->movers = reinterpret_cast<int32_t*>(ws + movers);
        s->rank = reinterpret_cast<int32_t*>(ws + rank);
    }
    return at;
}

inline bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + static_cast<uintptr_t>(b_bytes) && y < x + static_cast<uintptr_t>(a_bytes);
}

inline int64_t table_bytes(int rows, int stride, int max_pages) {
    return 4 * (static_cast<int64_t>(rows - 1) * stride + max_pages);
}

inline da_status check_rows(const da_paged_rows* r) {
    if (!r || r->max_pages < 1 || r->table_stride < r->max_pages || r->B < 1) return DA_ERR_INVALID_ARG;
    if (r->page_size < 16 || r->page_size > DA_MAX_PAGE_SIZE || r->page_size % 16 || r->num_pages < 1) return DA_ERR_INVALID_ARG;
    if (r->B > DA_MAX_PAGED_ROWS) return DA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(r->num_pages) * r->page_size > 0x7fffff00ll ||
        static_cast<int64_t>(r->max_pages) * r->page_size > 0x7fffff00ll ||
        static_cast<int64_t>(r->B) * r->max_pages > 0x7fffffffll)
        return DA_ERR_INVALID_ARG;
    if (!r->kv_lens || !r->block_table || !r->workspace) return DA_ERR_INVALID_ARG;
    if (!aligned(r->kv_lens, 4) || !aligned(r->block_table, 4) || !aligned(r->workspace, 256)) return DA_ERR_ALIGNMENT;
    if (r->workspace_bytes < decode_attn_paged_pages_workspace_size(r->num_pages)) return DA_ERR_WORKSPACE_TOO_SMALL;
    return DA_OK;
}

// Checks of the cache beside the rows, and of the table that a call writes.
inline da_status check_moves(const da_paged_rows& r, const da_paged_cache* c, const int32_t* out, int out_stride, int n_out) {
    if (!c) return DA_ERR_INVALID_ARG;
    const da_status st = check_cache(c, c->kv_dtype == DA_BF16 ? DA_BF16 : DA_F16, r.kv_lens, r.block_table, r.max_pages,
                                     r.table_stride, 1, c->Hkv);
    if (st != DA_OK) return st;
    if (c->page_size != r.page_size || c->num_pages != r.num_pages) return DA_ERR_INVALID_ARG;
    if (!out || out_stride < r.max_pages) return DA_ERR_INVALID_ARG;
    if (!aligned(out, 4)) return DA_ERR_ALIGNMENT;
    if (overlap(out, table_bytes(n_out, out_stride, r.max_pages), r.block_table, table_bytes(r.B, r.table_stride, r.max_pages)) ||
        overlap(out, table_bytes(n_out, out_stride, r.max_pages), r.kv_lens, 4 * static_cast<int64_t>(r.B)))
        return DA_ERR_INVALID_ARG;
    return DA_OK;
}

inline RowsParams rows_params(const da_paged_rows& r) {
    RowsParams p;
    p.lens = r.kv_lens;
    p.table = r.block_table;
    p.err = static_cast<uint32_t*>(r.workspace);
    p.B = r.B;
    p.max_pages = r.max_pages;
    p.table_stride = r.table_stride;
    p.P = r.page_size;
    p.num_pages = r.num_pages;
    return p;
}

template <class... Formal, class... Args>
inline bool launch_after(void (*kern)(Formal...), int grid, int threads, cudaStream_t stream, Args... args) {
    cudaLaunchAttribute attrs[1] = {pdl_attr()};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

template <bool COMPACT>
da_status launch_plan(const RowsParams& p, const PlanSpace& s, int32_t* free_pages, int32_t* count, cudaStream_t stream) {
    const int words = (p.num_pages + 31) / 32;
    const int64_t entries = static_cast<int64_t>(p.B) * p.max_pages;
    if (words <= kOneWords && p.B <= kOneRows && entries <= kOneEntries)
        return launch_after(page_plan_kernel<COMPACT, true>, 1, kOneThreads, stream, p, s, free_pages, count) ? DA_OK : DA_ERR_CUDA;
    if (!launch_after(page_clear_kernel, std::max(1, std::min(152, words / kPageThreads)), kPageThreads, stream, s.bits, words))
        return DA_ERR_CUDA;
    const int64_t items = p.B * ((p.max_pages + kRowEntries - 1ll) / kRowEntries), per = kPageThreads / 32;
    if (!launch_after(page_mark_kernel, static_cast<int>(std::min<int64_t>(kPageBlocks, (items + per - 1) / per)), kPageThreads, stream,
                      p, s.bits))
        return DA_ERR_CUDA;
    const int blocks = std::max(1, std::min(152, words / kPlanWords));
    return launch_after(page_plan_kernel<COMPACT, false>, blocks, kPageThreads, stream, p, s, free_pages, count) ? DA_OK : DA_ERR_CUDA;
}

}  // namespace da_impl

using namespace da_impl;

extern "C" {

size_t decode_attn_paged_pages_workspace_size(int num_pages) {
    if (num_pages < 1 || static_cast<int64_t>(num_pages) * 16 > 0x7fffff00ll) return 0;
    return pages_space(num_pages, nullptr, nullptr);
}

da_status decode_attn_paged_free_pages(const da_paged_rows* rows, int32_t* free_pages, int32_t* num_free, void* stream) {
    const da_status st = check_rows(rows);
    if (st != DA_OK) return st;
    if (!free_pages || !num_free) return DA_ERR_INVALID_ARG;
    if (!aligned(free_pages, 4) || !aligned(num_free, 4)) return DA_ERR_ALIGNMENT;
    const int64_t list = 4 * static_cast<int64_t>(rows->num_pages), table = table_bytes(rows->B, rows->table_stride, rows->max_pages);
    for (const void* out : {static_cast<const void*>(free_pages), static_cast<const void*>(num_free)}) {
        const int64_t bytes = out == free_pages ? list : 4;
        if (overlap(out, bytes, rows->block_table, table) || overlap(out, bytes, rows->kv_lens, 4 * static_cast<int64_t>(rows->B)))
            return DA_ERR_INVALID_ARG;
    }
    if (overlap(free_pages, list, num_free, 4)) return DA_ERR_INVALID_ARG;
    PlanSpace s;
    pages_space(rows->num_pages, &s, static_cast<uint8_t*>(rows->workspace));
    return launch_plan<false>(rows_params(*rows), s, free_pages, num_free, static_cast<cudaStream_t>(stream));
}

da_status decode_attn_paged_fork(const da_paged_rows* rows, const da_paged_cache* cache, const int32_t* parents,
                                 const int32_t* new_pages, int n_out, int32_t* kv_lens_out, int32_t* block_table_out,
                                 int table_out_stride, void* stream) {
    da_status st = check_rows(rows);
    if (st != DA_OK) return st;
    if (n_out < 1) return DA_ERR_INVALID_ARG;
    if (n_out > DA_MAX_PAGED_ROWS) return DA_ERR_UNSUPPORTED;
    const da_paged_rows& r = *rows;
    st = check_moves(r, cache, block_table_out, table_out_stride, n_out);
    if (st != DA_OK) return st;
    if (!parents || !new_pages || !kv_lens_out) return DA_ERR_INVALID_ARG;
    if (!aligned(parents, 4) || !aligned(new_pages, 4) || !aligned(kv_lens_out, 4)) return DA_ERR_ALIGNMENT;
    const int64_t list = 4 * static_cast<int64_t>(n_out), table = table_bytes(n_out, table_out_stride, r.max_pages);
    if (overlap(kv_lens_out, list, r.kv_lens, 4 * static_cast<int64_t>(r.B)) ||
        overlap(kv_lens_out, list, r.block_table, table_bytes(r.B, r.table_stride, r.max_pages)) ||
        overlap(kv_lens_out, list, parents, list) || overlap(kv_lens_out, list, new_pages, list) ||
        overlap(block_table_out, table, parents, list) || overlap(block_table_out, table, new_pages, list) ||
        overlap(block_table_out, table, kv_lens_out, list))
        return DA_ERR_INVALID_ARG;
    const da_paged_cache& c = *cache;
    ForkParams p;
    p.rows = rows_params(r);
    p.parents = parents;
    p.new_pages = new_pages;
    p.lens_out = kv_lens_out;
    p.table_out = block_table_out;
    p.table_out_stride = table_out_stride;
    p.n_out = n_out;
    p.k = static_cast<uint4*>(c.k);
    p.v = static_cast<uint4*>(c.v);
    p.ks = c.kv_dtype == DA_E4M3 ? c.k_scale : nullptr;
    p.vs = c.kv_dtype == DA_E4M3 ? c.v_scale : nullptr;
    p.Hkv = c.Hkv;
    p.layout = c.layout;
    p.row_units = c.D * (c.kv_dtype == DA_E4M3 ? 1 : 2) / 16;
    p.page_units = static_cast<int64_t>(c.page_size) * c.Hkv * p.row_units;
    if (p.page_units > kMostUnits) return DA_ERR_UNSUPPORTED;
    // as many blocks for a child as there is work for, and as fill the device
    const int64_t work = std::max<int64_t>(2 * ((p.page_units + kCopyChunk - 1) / kCopyChunk), (r.max_pages + kPageThreads - 1) / kPageThreads);
    const int split = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(work, kPageBlocks / n_out)));
    const int grid = static_cast<int>(std::min<int64_t>(kPageBlocks, static_cast<int64_t>(split) * n_out));
    return launch_after(page_fork_kernel, grid, kPageThreads, static_cast<cudaStream_t>(stream), p, split) ? DA_OK : DA_ERR_CUDA;
}

da_status decode_attn_paged_compact(const da_paged_rows* rows, const da_paged_cache* cache, int32_t* block_table_out,
                                    int table_out_stride, int32_t* num_used, void* stream) {
    da_status st = check_rows(rows);
    if (st != DA_OK) return st;
    const da_paged_rows& r = *rows;
    st = check_moves(r, cache, block_table_out, table_out_stride, r.B);
    if (st != DA_OK) return st;
    if (!num_used) return DA_ERR_INVALID_ARG;
    if (!aligned(num_used, 4)) return DA_ERR_ALIGNMENT;
    if (overlap(num_used, 4, r.kv_lens, 4 * static_cast<int64_t>(r.B)) ||
        overlap(num_used, 4, r.block_table, table_bytes(r.B, r.table_stride, r.max_pages)) ||
        overlap(num_used, 4, block_table_out, table_bytes(r.B, table_out_stride, r.max_pages)))
        return DA_ERR_INVALID_ARG;
    const da_paged_cache& c = *cache;
    MoveParams p;
    p.rows = rows_params(r);
    pages_space(r.num_pages, &p.s, static_cast<uint8_t*>(r.workspace));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = launch_plan<true>(p.rows, p.s, nullptr, num_used, s);
    if (st != DA_OK) return st;
    p.k = static_cast<uint4*>(c.k);
    p.v = static_cast<uint4*>(c.v);
    p.ks = c.kv_dtype == DA_E4M3 ? c.k_scale : nullptr;
    p.vs = c.kv_dtype == DA_E4M3 ? c.v_scale : nullptr;
    p.Hkv = c.Hkv;
    p.page_units = static_cast<int64_t>(c.page_size) * c.Hkv * (c.D * (c.kv_dtype == DA_E4M3 ? 1 : 2) / 16);
    p.table_out = block_table_out;
    p.table_out_stride = table_out_stride;
    // as many moves as half the pages at most
    const int64_t chunks = (p.page_units + kCopyChunk - 1) / kCopyChunk;
    const int64_t items = std::max<int64_t>(r.num_pages / 2 * 2 * chunks, (r.B + 7) / 8);
    const int grid = static_cast<int>(std::min<int64_t>(kPageBlocks, std::max<int64_t>(1, items)));
    return launch_after(page_move_kernel, grid, kPageThreads, s, p) ? DA_OK : DA_ERR_CUDA;
}

}  // extern "C"
