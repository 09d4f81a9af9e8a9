// Attention of a chunk of new tokens of each sequence over the paged KV cache
// (decode_attn_paged.h) on the Blackwell tensor cores, for GB300 / sm_103a.
//
// An item is 256 rows of one sequence and KV head, a row one (token, query head of the group)
// pair, in two tiles of 128 rows that take turns on the tensor cores. Over the 128-key tiles that
// some row sees, in one pass with a running maximum m per row,
//
//     S = Q K^T,   P = 2^(S scale log2e - m),   O += P V,   l += sum P;   out = O / l.
//
// S, P and O live in tensor memory (S and P in the same columns), Q, K and V in shared memory.
// One thread per row holds the row's scores in registers. One warp copies K and V by TMA, a box
// per page, or per 16 to 128 keys of it; one warp issues the products:
//
//     ... P0(j) V(j), Q0 K(j+1), P1(j) V(j), Q1 K(j+1), P0(j+1) V(j+1) ...
//
// so that the softmax of one row tile runs beside the products of the other. (At head size 64 tensor memory
// has room for P beside S, and the next scores are computed while the softmax of these runs.)
//
// The work of the whole call, in units of a key tile of an item, is cut into as many equal ranges
// as there are CTAs, one per SM, whatever the lengths, the causal triangle and the window leave of it. An item that lies in
// one range is written by it; otherwise each of its ranges leaves a partial result (two per range at
// most), and a second kernel joins them, in the order of the ranges: the results do not depend on timing.
//
// A tile is special if some row does not see some of its keys. There the scores of the others are taken
// out, values that no row sees are zeroed, and so are elements that are not finite (0 times NaN is no
// zero), which the end of the piece then adds to the rows that see them.
//
// e4m3 pages: four warps convert each tile to fp16, exactly. Queries enter as fp16, bf16 ones scaled by a
// power of two per row into the top of its range; ks multiplies the scores and vs the weights, page by page,
// relative to a reference per row (`dv`, the distance of the weights' maximum from the scores' m) that keeps the
// fp16 weights in range however unequal the scales are.
//
// Sums, maxima, accumulators and partial results are float32. Rounded to fewer bits are the outputs, once, and the
// weights, once, to the 16-bit type of their product: the tensor cores have no wider one at this rate, and a second
// term (as in the decode kernel, which waits for bytes) would add half of all products. The outputs' error is 1.3 (fp16)
// to 1.4 times (bf16) that of float32 weights (16-bit pages; over e4m3 pages 1.0, where fp16 weights meet a bf16 output).
//
// What bounds it (times in a graph of 20 calls, and of calls in a row, where the power limit lowers the clock). Head size 128:
// the tensor cores, 75 % of the time active (2048 of 8192 tokens, 32 / 8 heads, bf16: 145 and 157 us, 1.66 and 1.53 PFLOP/s, 86 %
// of cuBLAS's burst and 90 % of its sustained rate; 4096 of 32768: 1.18 to 1.32 and 1.34 ms, 1.54 PFLOP/s in a row). A pair of row
// tiles takes 2048 cycles of products and 2900 in all; their operands and the copies keep shared memory busy for the 2048, too, and
// a shorter softmax (1280 cycles from scores to weights) changes nothing. e4m3 pages: shared memory, which a pair of tiles keeps busy
// for 2560 cycles (the products' operands 1536, the raw tile in and out 512, the converted one in 512): 206 us for the first call
// above, 1.46 and 1.48 ms for the second. Head size 64: the rows' threads: an exponent takes 4 cycles of a scheduler's unit, two
// warps 1024 cycles per pair of tiles that the products need 1024 for; 2000 in all (16 / 2 heads, 8192 of 16384 tokens: 371 us,
// 1.11 PFLOP/s; over e4m3 pages 528 us with fp16 queries, 543 with bf16 ones). Short calls: latency, 2 us to the plan, 2 to the first
// scores, 1.4 per key tile, 2.5 for a piece's end and 3 for the join (107 of 1131 tokens 17.5 us). Row tiles without a row are
// computed like the others: 64 sequences with one token each over 8192 keys take 326 us in 16-bit pages, bound by the bytes, and
// 404 in e4m3 ones, whose bytes would take 158.

#include "paged_common.cuh"
#include "tcgen05.cuh"

namespace da_impl {

constexpr int kTileRows = 128;
constexpr int kItemRows = 2 * kTileRows;
constexpr int kTileKeys = 128;
constexpr int kMaxRanges = 160;       // CTAs at most (GB300 has 152 SMs)
// An item's begin and end, in key tiles: what its pipeline's filling and draining cost. (4 prompts of 4096 tokens 411 us with 2,
// 375 with 3, 370 with 4, 376 with 5; the ragged batch of 24 667, 600, 611 and 625.)
constexpr int kItemCost = 4;
// Of a range: a short call takes more CTAs, and joins more parts (107 of 1131 tokens 23.7 us with 7, 21.5 with 5, 19.0 with 3; 64 of
// 8192 29.3, 28.4 and 30.7).
constexpr int kLeastCost = 4;
constexpr int kLeastPart = 1;         // key tiles of a partial result at least (with 4 the ragged batch takes 677 us, with 2 611, with 1 579)
constexpr int kScaleRing = 4;         // tiles whose scales are in shared memory
constexpr int kPieceRing = 4;         // pieces whose description is
constexpr int kJoinSlices = 8;        // blocks that join one split item, 32 rows each

struct ChunkCut {            // a place in the order of the work: before key tile `tile` of an item
    int b, kvh, rt, tile;
};

struct ChunkJoin {           // a split item, at the range that holds its first part
    int parts;               // 0: none
    int n, r0, kvh, rt, pad[3];
};

struct ChunkParams {
    const uint16_t* q;
    const uint8_t* v;
    const float *ks, *vs;
    const int32_t *cu, *lens, *table;
    uint16_t* out;
    float* lse;              // or nullptr
    uint32_t* err;
    ChunkJoin* join;         // [ranges]
    float2* part_sum;        // [2 * range][row] {m, l}
    float4* part;            // [2 * range][D / 4][row], sums of weighted values relative to m
    int64_t q_stride, out_stride;
    int B, T, Hq, Hkv, G, P, max_pages, table_stride, num_pages, layout, window, sinks;
    int box_keys;            // keys of a TMA box: gcd(page size, 128)
    uint32_t group_mul;      // f / G by multiplication (token())
    int group_shift;
    int q_zero;              // the scale is 0: so are the queries (0 times what is not finite is NaN), and the factor is 1
    uint32_t q_xor;          // the scale's sign, on two query elements
    float scale_log2;        // |scale| log2e (1 if it is 0)
    int out_wide;            // every row of out begins on a 32-byte border
    unsigned long long wait_limit_ns;

    // Token of row f of a sequence (f < 2^31).
    __device__ __forceinline__ int token(int f) const {
        return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(f)) * group_mul) >> group_shift);
    }
};

struct ChunkSeq {
    int n, L, r0;            // rows (0: none, or none that can be), keys, first row
};

__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams& p, int b, bool flag) {
    ChunkSeq s;
    s.r0 = ld_cg_s32(p.cu + b);
    const int r1 = ld_cg_s32(p.cu + b + 1);
    s.L = ld_cg_s32(p.lens + b);
    s.n = r1 - s.r0;
    if (s.r0 < 0 || r1 < s.r0 || r1 > p.T) {
        if (flag) flag_error(p.err, DA_DEVERR_SEQLENS);
        s.n = 0;
    }
    if (s.L < 0 || s.L > static_cast<int64_t>(p.max_pages) * p.P) {
        if (flag) flag_error(p.err, DA_DEVERR_SEQLENS);
        s.L = 0;
    }
    return s;
}

// The key tiles of an item: 0 .. ns - 1 (first tokens), then lo on, nt in all (one, all of it hidden, if no row sees a key).
struct ChunkTiles {
    ChunkTiles() = default;
    int first, last;         // positions of its first and last token (may be < 0)
    int low;                 // the first key that the first token sees through the window
    int ns, lo, nt;
    int sure, from, to;      // every row sees every key of the tiles 0 .. sure - 1 and from .. to - 1

    __device__ __forceinline__ ChunkTiles(const ChunkParams& p, const ChunkSeq& s, int rt) {
        const int f = rt * kItemRows;
        first = s.L - s.n + p.token(f);
        last = s.L - s.n + min(s.n - 1, p.token(f + kItemRows - 1));
        low = p.window ? max(0, max(first, 0) - p.window + 1) : 0;
        ns = (min(p.sinks, low) + kTileKeys - 1) / kTileKeys;
        lo = max(ns, low / kTileKeys);
        nt = ns + max(last, 0) / kTileKeys - lo + 1;
        // tiles of first tokens before the first token's window, and tiles from lo on that end at or before the first token and
        // begin in the last token's window
        sure = min(p.sinks, low) / kTileKeys;
        to = ns + max((first + 1) / kTileKeys - lo, 0);
        from = ns;
        if (p.window) from += max((max(0, max(last, 0) - p.window + 1) + kTileKeys - 1) / kTileKeys - lo, 0);
    }
    __device__ __forceinline__ int key(int tile) const { return (tile < ns ? tile : lo + tile - ns) * kTileKeys; }
    __device__ __forceinline__ bool plain(int tile) const { return tile < sure || (tile >= from && tile < to); }
    // whether some row sees a key in [k, k + keys), or the key k
    __device__ __forceinline__ bool wanted(const ChunkParams& p, int k, int keys) const {
        return k <= last && (k + keys > low || k < p.sinks);
    }
};

__device__ __forceinline__ int chunk_items(const ChunkParams& p, int n) { return (n * p.G + kItemRows - 1) / kItemRows; }

// Where a cut at distance x into an item falls: the item's begin, a key tile of it, or (nt) its end.
__device__ __forceinline__ int cut_tile(int x, int nt) {
    const int tile = x - kItemCost;
    return tile < kLeastPart ? 0 : nt - tile < kLeastPart ? nt : tile;
}

// A piece: key tiles t0 .. t1 - 1 of an item. The warp that copies tiles walks through the range and leaves the pieces'
// descriptions in shared memory, where the others read them when they need them: their registers are the rows'.
struct ChunkPiece {
    int valid, b, kvh, rt, t0, t1;
    ChunkSeq s;
    ChunkTiles tiles;
    int dirty;               // special tiles had values that are not finite
};

// A CTA's range: its cuts, and the split item that begins in it.
struct ChunkPlan {
    ChunkCut cuts[2];
    ChunkSeq seqs[2];        // of the sequences that they lie in
    ChunkJoin join;
};

struct ChunkWalk {
    ChunkCut at, end;
    ChunkSeq s;
    __device__ __forceinline__ explicit ChunkWalk(const ChunkPlan& plan) : at(plan.cuts[0]), end(plan.cuts[1]), s(plan.seqs[0]) {}
    __device__ __forceinline__ bool next(const ChunkParams& p, ChunkPiece& x) {
        if (at.b >= p.B || (at.b == end.b && at.kvh == end.kvh && at.rt == end.rt && at.tile >= end.tile)) return false;
        x.tiles = ChunkTiles(p, s, at.rt);
        x.s = s;
        x.b = at.b;
        x.kvh = at.kvh;
        x.rt = at.rt;
        x.t0 = at.tile;
        x.t1 = x.tiles.nt;
        x.valid = 1;
        x.dirty = 0;
        if (at.b == end.b && at.kvh == end.kvh && at.rt == end.rt) {
            x.t1 = end.tile;
            at.tile = end.tile;
        } else {
            at.tile = 0;
            if (++at.rt == chunk_items(p, s.n)) {
                at.rt = 0;
                if (++at.kvh == p.Hkv) {
                    at.kvh = 0;
                    do {
                        if (++at.b >= p.B) break;
                        s = chunk_seq(p, at.b, false);
                    } while (s.n == 0);
                }
            }
        }
        return true;
    }
};

// ------------------------------------------------------------ the plan
template <int D, bool KV8>
struct ChunkShape {
    // warps: 0 - 7 rows, 8 copies, 9 products, 10 and 11 queries, 12 - 15 conversion. The rows' threads take most of the launch's registers.
    static constexpr int kRowWarps = 8, kThreads = KV8 ? 512 : 384;
    static constexpr int kRowRegs = KV8 ? 192 : 208, kOtherRegs = KV8 ? 64 : 88;
    static_assert(256 * kRowRegs + (kThreads - 256) * kOtherRegs <= kThreads * (65536 / kThreads / 8 * 8), "registers of the launch");
    static constexpr int kSlices = D / 64;                     // 128-byte columns of a tile in 16 bits
    static constexpr int kSliceBytes = 128 * 128;
    static constexpr int kTileBytes = kSlices * kSliceBytes;
    static constexpr int kRing = D == 64 ? 8 : KV8 ? 4 : 5;    // K and V tiles in 16 bits
    static constexpr int kRawBytes = KV8 ? kTileKeys * D : 0;  // and as they come, in 8
    static constexpr int kRaw = KV8 ? (D == 128 ? 2 : 8) : 0;
    static constexpr int kRawRow = D;
    static constexpr int kQOff = 0;
    static constexpr int kRingOff = 2 * kTileBytes;
    static constexpr int kRawOff = kRingOff + kRing * kTileBytes;
    static constexpr int kScaleOff = kRawOff + kRaw * kRawBytes;          // [tile][16-key box] {ks, log2 vs}
    static constexpr int kFactorOff = kScaleOff + (KV8 ? kScaleRing * 8 * 8 : 0);   // [row] factor of a row's scores
    static constexpr int kPieceOff = kFactorOff + (KV8 ? kItemRows * 4 : 0);
    static constexpr int kPlanOff = kPieceOff + (kPieceRing * static_cast<int>(sizeof(ChunkPiece)) + 7) / 8 * 8;
    static constexpr int kBarOff = kPlanOff + (static_cast<int>(sizeof(ChunkPlan)) + 7) / 8 * 8;
    static constexpr int kNumBars = 2 * kRing + 2 * kRaw + 2 * kScaleRing + 2 * kPieceRing + 15;
    static constexpr int kPieceReaders = kRowWarps + 3 + (KV8 ? 4 : 0);               // warps
    static constexpr int kTmemOff = kBarOff + kNumBars * 8;               // where the tensor memory begins
    static constexpr int kSmemBytes = kTmemOff + 8;
    static constexpr int kPlanBytes = (DA_MAX_PAGED_BATCH + 1) * 8 + DA_MAX_PAGED_BATCH * 12;
    static_assert(kPlanBytes <= kRing * kTileBytes, "the plan is made where the ring is later");
    // tensor memory
    // S0, S1, O0, O1 and, where there is room (head size 64), P0 and P1: the next scores then need not wait for the
    // products of these weights. Otherwise P lies where S was.
    static constexpr int kCols = 512, kO = 2 * kTileKeys;
    static constexpr bool kApart = D == 64;
    static constexpr int kP = kApart ? kO + 2 * D : 0, kPStep = kApart ? kTileKeys / 2 : kTileKeys;
    static_assert(!kApart || kP + 2 * kPStep <= kCols, "tensor memory");
};

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Cost of an item per tile and once, summed over a sequence's items of one KV head (by a warp).
__device__ __forceinline__ int64_t chunk_cost(const ChunkParams& p, const ChunkSeq& s) {
    int64_t cost = 0;
    for (int rt = threadIdx.x & 31; rt < chunk_items(p, s.n); rt += 32) cost += ChunkTiles(p, s, rt).nt + kItemCost;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) cost += __shfl_xor_sync(0xffffffffu, cost, off);
    return cost;
}
__device__ __forceinline__ int64_t scan_add(int64_t x) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
        if ((threadIdx.x & 31) >= off) x += y;
    }
    return x;
}

// Cut number r (by a warp, in all lanes alike), the sequence it lies in, and for a cut within an item what is known of
// the cuts after it. pre(b): cost of the sequences before b; seq(b): the sequence.
template <class Pre, class Seq>
__device__ __forceinline__ void chunk_cut(const ChunkParams& p, int r, Pre pre, Seq seq, ChunkCut& cut, ChunkSeq& s, ChunkJoin* join) {
    const int lane = threadIdx.x & 31;
    const int64_t all = pre(p.B);
    const int ranges = static_cast<int>(max(int64_t(1), min(static_cast<int64_t>(gridDim.x), all / kLeastCost)));
    const int64_t q = all / ranges;
    const int rem = static_cast<int>(all - q * ranges);
    auto raw = [&](int i) { return i * q + min(i, rem); };
    cut = {p.B, 0, 0, 0};
    s = {0, 0, 0};
    if (r >= ranges || all == 0) return;     // (no rows at all: no work, and nothing to divide by)
    const int64_t at = raw(r);
    int lo = 0, hi = p.B - 1;       // last b with pre(b) <= at
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre(mid) <= at) lo = mid;
        else hi = mid - 1;
    }
    s = seq(lo);
    int64_t begin = pre(lo);
    const int64_t head = (pre(lo + 1) - begin) / p.Hkv;
    const int items = chunk_items(p, s.n);
    cut.b = lo;
    cut.kvh = static_cast<int>((at - begin) / head);
    begin += cut.kvh * head;
    int nt = 0;
    for (int rt0 = 0; rt0 < items; rt0 += 32) {
        const int mine = rt0 + lane < items ? ChunkTiles(p, s, rt0 + lane).nt : 0;
        const int64_t run = scan_add(rt0 + lane < items ? mine + kItemCost : 0);
        const uint32_t past = __ballot_sync(0xffffffffu, begin + run > at);
        if (past != 0) {
            const int i = __ffs(past) - 1;
            cut.rt = rt0 + i;
            nt = __shfl_sync(0xffffffffu, mine, i);
            begin += __shfl_sync(0xffffffffu, run, i) - nt - kItemCost;
            break;
        }
        begin += __shfl_sync(0xffffffffu, run, 31);
    }
    cut.tile = cut_tile(static_cast<int>(at - begin), nt);
    if (join && cut.tile > 0 && cut.tile < nt) {
        // the cuts of other ranges in the same item
        int inside = 0;
        bool more = true;
        for (int r0 = r + 1; more; r0 += 32) {
            const int64_t x = r0 + lane < ranges ? raw(r0 + lane) - begin : int64_t(1) << 40;
            int tile = nt;
            if (x < nt + kItemCost) tile = cut_tile(static_cast<int>(x), nt);
            const uint32_t in = __ballot_sync(0xffffffffu, tile < nt);
            inside += __popc(in);
            more = in == 0xffffffffu;
        }
        join->parts = 2 + inside;
        join->n = s.n;
        join->r0 = s.r0;
        join->kvh = cut.kvh;
        join->rt = cut.rt;
    }
    if (cut.tile == nt) {            // the next item's begin
        cut.tile = 0;
        if (++cut.rt == items) {
            cut.rt = 0;
            if (++cut.kvh == p.Hkv) {
                cut.kvh = 0;
                do ++cut.b;
                while (cut.b < p.B && pre(cut.b + 1) == pre(cut.b));
                if (cut.b < p.B) s = seq(cut.b);
            }
        }
    }
}

// This CTA's range, by all threads; `space` is shared memory that the pipeline uses later.
template <int THREADS>
__device__ void chunk_plan(const ChunkParams& p, uint8_t* space, ChunkPlan& plan) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = static_cast<int>(blockIdx.x) + warp;       // warp 0: the range's begin, warp 1: its end
    ChunkCut cut;
    ChunkSeq s;
    ChunkJoin join = {};
    if (p.B <= 32) {
        // a lane per sequence, in either of the two warps: nothing to wait for
        if (warp < 2) {
            ChunkSeq mine = {0, 0, 0};
            if (lane < p.B) mine = chunk_seq(p, lane, blockIdx.x == 0 && warp == 0);
            const int items = chunk_items(p, mine.n);
            int64_t cost = 0;
            if (items == 1) cost = ChunkTiles(p, mine, 0).nt + kItemCost;
            uint32_t many = __ballot_sync(0xffffffffu, items > 1);
            while (many != 0) {
                const int b = __ffs(many) - 1;
                many &= many - 1;
                const ChunkSeq x = {__shfl_sync(0xffffffffu, mine.n, b), __shfl_sync(0xffffffffu, mine.L, b), 0};
                const int64_t sum = chunk_cost(p, x);
                if (lane == b) cost = sum;
            }
            const int64_t run = scan_add(cost * p.Hkv);      // (0 beyond the last sequence)
            auto pre = [&](int b) {
                const int64_t x = __shfl_sync(0xffffffffu, run, max(b - 1, 0));
                return b == 0 ? int64_t(0) : x;
            };
            auto seq = [&](int b) {
                return ChunkSeq{__shfl_sync(0xffffffffu, mine.n, b), __shfl_sync(0xffffffffu, mine.L, b),
                                __shfl_sync(0xffffffffu, mine.r0, b)};
            };
            chunk_cut(p, r, pre, seq, cut, s, warp == 1 ? &join : nullptr);
        }
    } else {
        int64_t* before = reinterpret_cast<int64_t*>(space);                   // [B + 1] cost before a sequence
        ChunkSeq* seqs = reinterpret_cast<ChunkSeq*>(before + p.B + 1);        // [B]
        constexpr int kFew = 4;                                                // items that a thread counts by itself
        for (int b = threadIdx.x; b < p.B; b += THREADS) {
            const ChunkSeq x = chunk_seq(p, b, blockIdx.x == 0);
            seqs[b] = x;
            const int items = chunk_items(p, x.n);
            int64_t cost = 0;
            for (int rt = 0; rt < min(items, kFew); ++rt) cost += ChunkTiles(p, x, rt).nt + kItemCost;
            before[b + 1] = items > kFew ? -1 : cost * p.Hkv;
        }
        __syncthreads();
        for (int b = warp; b < p.B; b += THREADS / 32) {
            if (before[b + 1] >= 0) continue;
            const int64_t cost = chunk_cost(p, seqs[b]);
            __syncwarp();
            if (lane == 0) before[b + 1] = cost * p.Hkv;
        }
        __syncthreads();
        if (warp == 0) {
            int64_t sum = 0;
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const int64_t run = scan_add(b0 + lane < p.B ? before[b0 + lane + 1] : 0);
                if (b0 + lane < p.B) before[b0 + lane + 1] = sum + run;
                sum += __shfl_sync(0xffffffffu, run, 31);
            }
            if (lane == 0) before[0] = 0;
        }
        __syncthreads();
        if (warp < 2)
            chunk_cut(p, r, [&](int b) { return before[b]; }, [&](int b) { return seqs[b]; }, cut, s, warp == 1 ? &join : nullptr);
        proxy_fence();                 // this memory is the ring from here on
    }
    if (warp < 2 && lane == 0) {
        plan.cuts[warp] = cut;
        plan.seqs[warp] = s;
        if (warp == 1) plan.join = join;
    }
}

// The split item that begins in this range, for the kernel that joins its parts (none if it began in an earlier one).
__device__ __forceinline__ void leave_join(const ChunkParams& p, const ChunkPlan& plan) {
    const ChunkCut &a = plan.cuts[0], &e = plan.cuts[1];
    ChunkJoin join = plan.join;
    if (a.b == e.b && a.kvh == e.kvh && a.rt == e.rt && a.tile > 0) join.parts = 0;
    p.join[blockIdx.x] = join;
}

// ------------------------------------------------------------ arithmetic on pairs
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// tmem_ld32 and tmem_st16 without the wait.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, float* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
                 : "r"(taddr));
}
// Nothing that reads the values moves before this.
__device__ __forceinline__ void hold32(float* r) {
    asm volatile("" : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]), "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31]));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16_start(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a));
    return x;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 x) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}

// Bits 0 .. n - 1 (any n).
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 0 times two 16-bit elements, added to y.
template <int DT>
__device__ __forceinline__ uint32_t zero_times(uint32_t x, uint32_t y) {
    uint32_t r;
    if constexpr (DT == DA_F16) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(y));
    else asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(y));
    return r;
}

template <int D, int DT, bool KV8>
struct ChunkKernel {
    using Sh = ChunkShape<D, KV8>;
    static constexpr int MT = KV8 ? DA_F16 : DT;                 // type of the products
    static constexpr bool kRowFactors = KV8 && DT == DA_BF16;    // queries scaled to fp16, row by row
    // A weight enters its product as 2^kLift times itself and is at most 2^kHeadroom times the largest one at the
    // time that its row's reference was set; fp16 then holds all bits of a weight down to 2^-25 of the largest (bf16 any).
    static constexpr float kHeadroom = MT == DA_F16 ? 4.f : 8.f;
    static constexpr float kLift = MT == DA_F16 ? 15.f - kHeadroom : 0.f;
    static constexpr uint32_t kIdS = umma_idesc<MT>(kTileRows, kTileKeys, false);
    static constexpr uint32_t kIdPV = umma_idesc<MT>(kTileRows, D, true);

    struct Ctx {
        uint8_t* smem;
        uint32_t base, tmem;
        uint32_t kv_full, kv_empty, raw_full, raw_empty, sc_full, sc_empty, x_full, x_empty, q_full, q_empty, s_full, s_free, p_half, p_full, pv_done, fin;
        const ChunkPlan* plan;
        ChunkPiece* pieces;
    };

    static __device__ __forceinline__ uint32_t ring(const Ctx& c, int i) { return c.base + Sh::kRingOff + i * Sh::kTileBytes; }
    // 16-byte chunk `chunk` of row `row` of a 16-bit tile
    static __device__ __forceinline__ uint32_t tile_addr(uint32_t tile, int row, int chunk) {
        return tile + (chunk >> 3) * Sh::kSliceBytes + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
    }
    static __device__ __forceinline__ bool wait(const ChunkParams& p, uint32_t bar, uint32_t parity) {
        const bool ok = wait_warp(bar, parity, p.wait_limit_ns);
        if (!ok && (threadIdx.x & 31) == 0) flag_error(p.err, DA_DEVERR_TIMEOUT);
        return ok;
    }

    // A wait for the end of a piece, which may be long: 20 us for each of its key tiles more than other waits.
    static __device__ __forceinline__ unsigned long long piece_limit(const ChunkParams& p, int tiles) {
        return p.wait_limit_ns + static_cast<unsigned long long>(tiles) * 20000ull;
    }

    // wait, for warps that are not in a hurry: each question reads shared memory, of which the 8-bit kernel has no time to
    // spare (4096 of 32768 tokens 1992 us with the queries' warps asking all the time, 1827 so).
    template <int NS>
    static __device__ __forceinline__ bool wait_calmly(const ChunkParams& p, uint32_t bar, uint32_t parity, int tiles = 0) {
        const unsigned long long limit = piece_limit(p, tiles), start = global_ns();
        while (!mbar_try_wait(bar, parity) && global_ns() - start <= limit) __nanosleep(NS);
        return wait(p, bar, parity);
    }

    // Piece number i, or nullptr after the last one (or a wait that timed out), by a whole warp and with one answer for all of
    // its lanes: a time-out that only some of them saw must not split them. It is given back with drop_piece.
    static __device__ __forceinline__ ChunkPiece* take_piece(const Ctx& c, const ChunkParams& p, uint32_t i, int tiles = 0) {
        const bool ok = wait_lane(c.x_full + 8 * (i % kPieceRing), (i / kPieceRing) & 1, piece_limit(p, tiles));
        if (!ok) flag_error(p.err, DA_DEVERR_TIMEOUT);
        ChunkPiece* x = c.pieces + i % kPieceRing;
        return __any_sync(0xffffffffu, !ok || !x->valid) ? nullptr : x;
    }
    static __device__ __forceinline__ void drop_piece(const Ctx& c, uint32_t i) {   // (one lane of a warp)
        mbar_arrive(c.x_empty + 8 * (i % kPieceRing));
    }

    // ------------------------------------------------------------ copies
    static __device__ void producer(const Ctx& c, const ChunkParams& p, const CUtensorMap* tmK, const CUtensorMap* tmV) {
        constexpr uint32_t kSlots = KV8 ? Sh::kRaw : Sh::kRing;
        uint32_t slot = 0;             // K and V tiles so far
        if (copy_tiles(c, p, tmK, tmV, slot)) return;
        // after a wait that timed out, copies still in flight into this CTA's shared memory get another bounded one each
        for (uint32_t i = slot < kSlots ? 0 : slot - kSlots; i < slot; ++i)
            wait_lane((KV8 ? c.raw_full : c.kv_full) + 8 * (i % kSlots), (i / kSlots) & 1, p.wait_limit_ns);
    }

    static __device__ __forceinline__ bool copy_tiles(const Ctx& c, const ChunkParams& p, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                                      uint32_t& slot) {
        constexpr int kSlots = KV8 ? Sh::kRaw : Sh::kRing;
        constexpr int kBytes = KV8 ? Sh::kRawBytes : Sh::kTileBytes;
        constexpr int kRow = KV8 ? Sh::kRawRow : 128;                       // bytes of a row of a box
        const uint32_t space = c.base + (KV8 ? Sh::kRawOff : Sh::kRingOff);
        const uint32_t full = KV8 ? c.raw_full : c.kv_full, empty = KV8 ? c.raw_empty : c.kv_empty;
        const int lane = threadIdx.x & 31;
        const int boxes = kTileKeys / p.box_keys, batch = 32 / boxes;       // tiles whose boxes the lanes look up at once
        const int my_tile = lane / boxes, my_box = lane - my_tile * boxes;
        ChunkWalk walk(*c.plan);
        uint32_t count = 0;                // key tiles so far
        for (uint32_t piece = 0;; ++piece) {
            ChunkPiece x;
            x.valid = 0;
            walk.next(p, x);
            const int place = piece % kPieceRing;
            if (!wait_calmly<500>(p, c.x_empty + 8 * place, ((piece / kPieceRing) & 1) ^ 1)) return false;
            if (lane == 0) {
                c.pieces[place] = x;
                mbar_arrive(c.x_full + 8 * place);
            }
            __syncwarp();
            if (!x.valid) break;
            const ChunkTiles& tiles = x.tiles;
            const int32_t* row = p.table + static_cast<int64_t>(x.b) * p.table_stride;
            auto entry = [&](int t) {      // block-table entry of this lane's box of tile t + my_tile, or -1
                t += my_tile;
                if (t >= x.t1) return -1;
                const int k = tiles.key(t) + my_box * p.box_keys;
                return tiles.wanted(p, k, p.box_keys) ? ld_cg_s32(row + k / p.P) : -1;
            };
            int ahead = entry(x.t0);
            for (int t0 = x.t0; t0 < x.t1; t0 += batch) {
                int page = ahead;
                const int mine = t0 + my_tile;
                const bool want = mine < x.t1 && tiles.wanted(p, tiles.key(mine) + my_box * p.box_keys, p.box_keys);
                const bool good = page >= 0 && page < p.num_pages;
                if (want && !good) flag_error(p.err, DA_DEVERR_PAGE);
                if (!good) page = p.num_pages;     // past the cache, which the copy fills with zeros
                ahead = entry(t0 + batch);
                float ks = 0.f, lv = 0.f;
                if constexpr (KV8) {
                    float vs = 0.f;
                    if (good) {
                        const int64_t at = static_cast<int64_t>(page) * p.Hkv + x.kvh;
                        ks = __ldcg(p.ks + at);
                        vs = __ldcg(p.vs + at);
                    }
                    lv = log2_of_scale(vs);
                }
                for (int t = t0; t < min(t0 + batch, x.t1); ++t) {
                    const int k0 = tiles.key(t);
                    const int from = (t - t0) * boxes;      // this tile's lanes
                    if constexpr (KV8) {
                        const int at = count % kScaleRing;
                        if (!wait_calmly<100>(p, c.sc_empty + 8 * at, ((count / kScaleRing) & 1) ^ 1)) return false;
                        const int owner = (from + (lane * 16) / p.box_keys) & 31;
                        const float a = __shfl_sync(0xffffffffu, ks, owner), b = __shfl_sync(0xffffffffu, lv, owner);
                        if (lane < 8) reinterpret_cast<float2*>(c.smem + Sh::kScaleOff)[at * 8 + lane] = make_float2(a, b);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(c.sc_full + 8 * at);
                        ++count;
                    }
                    const int my_page = __shfl_sync(0xffffffffu, page, (from + lane) & 31);
                    const int pos = k0 + lane * p.box_keys, in_page = pos % p.P;
                    const bool thd = p.layout == DA_LAYOUT_VARLEN;
                    // (a box of a page that is none starts past the last page)
                    const bool none = my_page == p.num_pages;
                    const int c1 = thd ? x.kvh : in_page;
                    const int c2 = thd ? my_page * p.P + (none ? 0 : in_page) : my_page * p.Hkv + (none ? 0 : x.kvh);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++slot) {
                        const int at = slot % kSlots;
                        if (!wait(p, empty + 8 * at, ((slot / kSlots) & 1) ^ 1)) return false;
                        const uint32_t bar = full + 8 * at;
                        if (lane == 0) mbar_arrive_expect_tx(bar, kBytes);
                        __syncwarp();
                        if (lane < boxes) {
                            const uint32_t dst = space + at * kBytes + lane * p.box_keys * kRow;
                            const CUtensorMap* map = kv ? tmV : tmK;
                            if constexpr (KV8) {
                                tma_load_3d(dst, map, 0, c1, c2, bar);
                            } else {
#pragma unroll
                                for (int sl = 0; sl < Sh::kSlices; ++sl) tma_load_3d(dst + sl * Sh::kSliceBytes, map, sl * 64, c1, c2, bar);
                            }
                        }
                    }
                }
            }
        }
        return true;
    }

    // ------------------------------------------------------------ e4m3 to fp16
    static __device__ void converter(const Ctx& c, const ChunkParams& p) {
        constexpr int kChunks = D / 16;                        // 16-byte chunks of a raw row
        constexpr int kStep = 128 / kChunks, kPer = kTileKeys / kStep;    // rows that the threads take at a time; times
        const int tid = threadIdx.x & 127, lane = threadIdx.x & 31;
        // A thread's chunk of its rows row0, row0 + kStep ... Eight lanes at a time read 8 x 16 bytes of raw rows and write as much of
        // 16-bit rows, both swizzled: rows r and r ^ 5, four neighbouring chunks each, meet in no bank either way (head size
        // 64: two neighbouring rows of four chunks).
        const int four = tid & 3, other = (tid >> 2) & 1, pr = (tid >> 3) & 3;
        const int row0 = kChunks == 8 ? ((tid >> 5) & 1) * 8 + (other ? pr ^ 5 : pr) : tid / 4;
        const int ch = kChunks == 8 ? (tid >> 6) * 4 + four : four;
        const int sw = kChunks == 8 ? row0 & 7 : (row0 >> 1) & 3;         // the copy's swizzle
        const uint32_t from0 = row0 * Sh::kRawRow + ((ch ^ sw) << 4);
        const uint32_t to0 = tile_addr(0, row0, 2 * ch), to1 = tile_addr(0, row0, 2 * ch + 1);
        static_assert(kStep % 8 == 0, "a thread's rows have one swizzle");
        uint32_t slot = 0;
        for (uint32_t piece = 0;; ++piece) {
            ChunkPiece* x = take_piece(c, p, piece);
            if (!x) break;
            for (int t = x->t0, t1 = x->t1; t < t1; ++t) {
                const bool plain = x->tiles.plain(t);
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++slot) {
                    const uint32_t from = slot % Sh::kRaw, to = slot % Sh::kRing;
                    const uint32_t landed = c.raw_full + 8 * from, free = c.kv_empty + 8 * to;
                    const uint32_t landed_phase = (slot / Sh::kRaw) & 1, free_phase = ((slot / Sh::kRing) & 1) ^ 1;
                    // (both asked at once)
                    const bool a = mbar_try_wait(landed, landed_phase), b = mbar_try_wait(free, free_phase);
                    if (!__all_sync(0xffffffffu, a && b) && (!wait(p, landed, landed_phase) || !wait(p, free, free_phase))) return;
                    const uint32_t src = c.base + Sh::kRawOff + from * Sh::kRawBytes + from0;
                    const uint32_t dst = c.base + Sh::kRingOff + to * Sh::kTileBytes;
                    uint4 in[kPer];
#pragma unroll
                    for (int i = 0; i < kPer; ++i) in[i] = lds128(src + i * kStep * Sh::kRawRow);
                    uint32_t found = 0;
                    if (kv == 1 && !plain) {
                        const int k0 = x->tiles.key(t) + row0;
#pragma unroll
                        for (int i = 0; i < kPer; ++i) {
                            const bool seen = x->tiles.wanted(p, k0 + i * kStep, 1);
                            uint32_t* e = &in[i].x;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t bad = __vcmpeq4(e[j] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                if (seen) found |= bad;
                                e[j] = seen ? e[j] & ~bad : 0u;
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        uint4 lo, hi;
                        e4m3x4_to_f16(in[i].x, lo.x, lo.y);
                        e4m3x4_to_f16(in[i].y, lo.z, lo.w);
                        e4m3x4_to_f16(in[i].z, hi.x, hi.y);
                        e4m3x4_to_f16(in[i].w, hi.z, hi.w);
                        sts128(dst + to0 + i * kStep * 128, lo);
                        sts128(dst + to1 + i * kStep * 128, hi);
                    }
                    if (found) x->dirty = 1;
                    proxy_fence();
                    __syncwarp();
                    // (the raw tile is given back here, where what was read of it has been used: an arrival overtakes reads in flight)
                    if (lane == 0) {
                        mbar_arrive(c.raw_empty + 8 * from);
                        mbar_arrive(c.kv_full + 8 * to);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) drop_piece(c, piece);
        }
    }

    // ------------------------------------------------------------ products (one warp, all lanes alike)
    static __device__ void multiplier(const Ctx& c, const ChunkParams& p) {
        multiply(c, p);
        // nothing is in flight when the tensor memory is freed, after a wait that timed out neither
        umma_commit_elect(c.fin);
        wait_warp(c.fin, 0, p.wait_limit_ns);
    }

    static __device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

    static __device__ __forceinline__ void multiply(const Ctx& c, const ChunkParams& p) {
        const uint32_t tmem = uniform(c.tmem), base = uniform(c.base);
        const uint64_t q0 = umma_desc_sw128(base + Sh::kQOff, 16, 1024);
        const uint64_t k0 = umma_desc_sw128(base + Sh::kRingOff, 16, 1024), v0 = umma_desc_sw128(base + Sh::kRingOff, Sh::kSliceBytes, 1024);
        uint32_t at = 0, phase = 0;            // the next tile's place in the ring, and its parity
        uint32_t tiles = 0;
        auto ready = [&](uint32_t bar, uint32_t parity) {
            const bool ok = wait(p, bar, parity);
            tmem_fence_after_sync();
            return ok;
        };
        auto advance = [&]() {
            if (++at == Sh::kRing) {
                at = 0;
                phase ^= 1;
            }
        };
        auto scores = [&](int w, uint32_t place) {
            const uint64_t kd = k0 + ((place * Sh::kTileBytes) >> 4), qd = q0 + ((w * Sh::kTileBytes) >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((k >> 2) * Sh::kSliceBytes + (k & 3) * 32) >> 4;
                umma_ss_elect(tmem + w * kTileKeys, qd + off, kd + off, kIdS, k > 0);
            }
            umma_commit_elect(c.s_full + 8 * w);
        };
        // (a half of the tile's keys at a time: the second half's weights are computed beside the first product)
        auto weigh = [&](int w, uint32_t place, int half, bool first) {
            const uint64_t vd = v0 + ((place * Sh::kTileBytes) >> 4);
#pragma unroll
            for (int j = 0; j < kTileKeys / 32; ++j) {
                const int k = half * (kTileKeys / 32) + j;
                umma_ts_elect(tmem + Sh::kO + w * D, tmem + Sh::kP + w * Sh::kPStep + k * 8, vd + ((k * 16 * 128) >> 4), kIdPV, !(first && k == 0));
            }
            if (half == 1) umma_commit_elect(c.pv_done + 8 * w);
        };
        for (uint32_t piece = 0;; ++piece) {
            const ChunkPiece* x = take_piece(c, p, piece);
            if (!x) return;
            const int nt = uniform(x->t1 - x->t0);
            __syncwarp();
            if ((threadIdx.x & 31) == 0) drop_piece(c, piece);
            // the ring: K, V, K, V ...
            if (!ready(c.kv_full + 8 * at, phase)) return;
            const uint32_t begin = at;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                // (Where the next scores do not wait for products, the second row tile begins half a softmax after the first
                // and stays behind it: both at once would take turns at the same units, exponents here, maxima there.)
                if (Sh::kApart && w == 1 && !ready(c.p_half, tiles & 1)) return;
                if (!ready(c.q_full + 8 * w, piece & 1)) return;
                scores(w, begin);
                if (nt == 1) umma_commit_elect(c.q_empty + 8 * w);
            }
            umma_commit_elect(c.kv_empty + 8 * begin);
            advance();
            for (int t = 0; t < nt; ++t, ++tiles) {
                const uint32_t v = at, v_phase = phase;
                const bool more = t + 1 < nt;
                advance();
                const uint32_t k = at;
                if (Sh::kApart && more) {
                    // the next scores as soon as these are read
                    if (!ready(c.kv_full + 8 * k, phase)) return;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        if (!ready(c.s_free + 8 * w, tiles & 1)) return;
                        scores(w, k);
                        if (t + 2 == nt) umma_commit_elect(c.q_empty + 8 * w);
                    }
                    umma_commit_elect(c.kv_empty + 8 * k);
                }
                if (!ready(c.kv_full + 8 * v, v_phase)) return;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (!ready(c.p_half + 8 * w, tiles & 1)) return;
                    weigh(w, v, 0, t == 0);
                    if (!ready(c.p_full + 8 * w, tiles & 1)) return;
                    weigh(w, v, 1, false);
                    if (w == 1) umma_commit_elect(c.kv_empty + 8 * v);
                    if (!Sh::kApart && more) {
                        if (w == 0 && !ready(c.kv_full + 8 * k, phase)) return;
                        scores(w, k);
                        if (t + 2 == nt) umma_commit_elect(c.q_empty + 8 * w);
                        if (w == 1) umma_commit_elect(c.kv_empty + 8 * k);
                    }
                }
                if (more) advance();
            }
        }
    }

    // ------------------------------------------------------------ rows
    // Queries of rows first .. first + ROWS - 1 of tile w into shared memory, by a warp.
    template <int ROWS>
    static __device__ __forceinline__ void fetch_queries(const Ctx& c, const ChunkParams& p, const ChunkPiece& x, int w, int first) {
        constexpr int kChunks = D / 8, kPerPass = 32 / kChunks, kPasses = ROWS / kPerPass, kBatch = 8;
        const int lane = threadIdx.x & 31, ch = lane % kChunks, sub = lane / kChunks;
        const uint32_t tile = c.base + Sh::kQOff + w * Sh::kTileBytes;
        const bool asis = !kRowFactors && !p.q_zero && p.q_xor == 0;
        const int rows = x.s.n * p.G;
        int f = x.rt * kItemRows + w * kTileRows + first + sub, t = p.token(f), g = f - t * p.G;
        const uint16_t* q = p.q + (x.s.r0 + t) * p.q_stride + static_cast<int64_t>(x.kvh) * p.G * D + ch * 8;   // of token t
        auto next = [&]() {            // kPerPass rows on
            f += kPerPass;
            g += kPerPass;
            while (g >= p.G) {
                g -= p.G;
                q += p.q_stride;
            }
        };
        if (asis) {
#pragma unroll 4
            for (int i = 0; i < kPasses; ++i, next()) {
                const bool live = f < rows;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tile_addr(tile, first + i * kPerPass + sub, ch)),
                             "l"(live ? q + g * D : p.q), "r"(live ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        } else {
#pragma unroll 1
            for (int i0 = 0; i0 < kPasses; i0 += kBatch) {
                uint4 v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i, next())   // (from the L2: the kernel before, which this one overlaps, may have written q)
                    v[i] = f < rows ? __ldcg(reinterpret_cast<const uint4*>(q + g * D)) : make_uint4(0, 0, 0, 0);
                // the largest exponent field of each row, all rows of the batch a step at a time
                uint32_t top[kBatch];
                if constexpr (kRowFactors) {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const uint32_t e[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                        top[i] = 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j) top[i] = max(top[i], max(e[j] & 0x7f80u, (e[j] >> 16) & 0x7f80u));
                    }
#pragma unroll
                    for (int off = 1; off < kChunks; off <<= 1)
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], off));
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) put_query(c, p, v[i], kRowFactors ? top[i] >> 7 : 0u, w, first + (i0 + i) * kPerPass + sub, ch);
            }
        }
        proxy_fence();
        __syncwarp();
    }

    // The queries of every piece but the first (which the rows' warps fetch, four of them a tile), a warp per row tile, as
    // soon as the piece before is done with its own. Queries that have to be scaled to fp16 are too much work for one warp (9 us a
    // tile): the rows' warps fetch those of every piece, and these only pull them into the L2.
    static __device__ void queries(const Ctx& c, const ChunkParams& p, int w) {
        const int lane = threadIdx.x & 31;
        int before = 0, tiles = 0;         // key tiles of the piece before, and of this one
        for (uint32_t piece = 0;; ++piece) {
            const ChunkPiece* x = take_piece(c, p, piece, tiles);
            if (!x) return;
            before = tiles;
            tiles = x->t1 - x->t0;
            if (piece > 0) {
                // (into the L2 while the tensor cores still read the tile)
                for (int r = lane; r < kTileRows; r += 32) {
                    const int f = x->rt * kItemRows + w * kTileRows + r;
                    if (f >= x->s.n * p.G) break;
                    const int t = p.token(f);
                    const uint16_t* line = p.q + (x->s.r0 + t) * p.q_stride + (static_cast<int64_t>(x->kvh) * p.G + f - t * p.G) * D;
                    for (int d = 0; d < D; d += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(line + d));
                }
                if constexpr (!kRowFactors) {
                    if (!wait_calmly<500>(p, c.q_empty + 8 * w, (piece & 1) ^ 1, before)) return;
                    fetch_queries<kTileRows>(c, p, *x, w, 0);
                    if (lane < 4) mbar_arrive(c.q_full + 8 * w);
                }
            }
            __syncwarp();
            if (lane == 0) drop_piece(c, piece);
        }
    }

    // 16 bytes of a query: the sign of the scale, and for bf16 over 8-bit pages fp16, with a factor per row (`top`: the largest
    // exponent field of the row).
    static __device__ __forceinline__ void put_query(const Ctx& c, const ChunkParams& p, const uint4& v, uint32_t top, int w, int r, int ch) {
        uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = p.q_zero ? zero_times<DT>(e[j], 0u) : e[j] ^ p.q_xor;
        if constexpr (kRowFactors) {
            // 2^e takes the largest element to [2^14, 2^15); an infinity or a NaN stays one
            const int field = top == 255 ? 127 : min(max(268 - static_cast<int>(top), 14), 240);
            const float up = __uint_as_float(static_cast<uint32_t>(field) << 23);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                e[j] = pack2<DA_F16>(__uint_as_float(e[j] << 16) * up, __uint_as_float(e[j] & 0xffff0000u) * up);
            if (ch == 0)
                reinterpret_cast<float*>(c.smem + Sh::kFactorOff)[w * kTileRows + r] =
                    __uint_as_float(static_cast<uint32_t>(254 - field) << 23) * p.scale_log2;
        }
        sts128(tile_addr(c.base + Sh::kQOff + w * Sh::kTileBytes, r, ch), make_uint4(e[0], e[1], e[2], e[3]));
    }

    // A special tile's values, 16-bit pages (by the 128 threads of row tile 0): zeros for what no row sees and for what
    // is not finite.
    static __device__ __forceinline__ bool clean_values(const ChunkParams& p, const ChunkTiles& tiles, int k0, uint32_t tile) {
        constexpr int kChunks = D / 8, kStep = 128 / kChunks, kTimes = kTileKeys / kStep;
        const int tid = threadIdx.x & 127, ch = tid % kChunks, r0 = tid / kChunks;
        uint32_t probe = 0;      // a sum of zero times the elements that some row sees: 0, or NaN
#pragma unroll 4
        for (int i = 0; i < kTimes; ++i) {
            const int r = r0 + i * kStep;
            const uint32_t at = tile_addr(tile, r, ch);
            if (tiles.wanted(p, k0 + r, 1)) {
                const uint4 v = lds128(at);
                probe = zero_times<MT>(v.x, zero_times<MT>(v.y, zero_times<MT>(v.z, zero_times<MT>(v.w, probe))));
            } else {
                sts128(at, make_uint4(0, 0, 0, 0));
            }
        }
        const bool found = (probe & 0x7fff7fffu) != 0;
        if (found) {
            constexpr uint32_t kExp = MT == DA_BF16 ? 0x7f807f80u : 0x7c007c00u;
#pragma unroll 1
            for (int i = 0; i < kTimes; ++i) {
                const int r = r0 + i * kStep;
                const uint32_t at = tile_addr(tile, r, ch);
                if (!tiles.wanted(p, k0 + r, 1)) continue;
                const uint4 v = lds128(at);
                sts128(at, make_uint4(v.x & ~__vcmpeq2(v.x & kExp, kExp), v.y & ~__vcmpeq2(v.y & kExp, kExp),
                                      v.z & ~__vcmpeq2(v.z & kExp, kExp), v.w & ~__vcmpeq2(v.w & kExp, kExp)));
            }
        }
        proxy_fence();
        return found;
    }

    // Adds to the accumulator `to` of this warp's rows what was taken out of the special tiles' values that a row sees.
    static __device__ __noinline__ void add_non_finite(const ChunkParams& p, const ChunkPiece& x, int pos, uint32_t to) {
        const ChunkTiles& tiles = x.tiles;
        for (int d0 = 0; d0 < D; d0 += 16) {
            uint32_t o[16];
            tmem_ld16(to + d0, o);
            float add[16];
#pragma unroll
            for (int d = 0; d < 16; ++d) add[d] = 0.f;
            for (int t = x.t0; t < x.t1; ++t) {
                const int k0 = tiles.key(t);
                if (tiles.plain(t)) continue;
                for (int k = k0; k <= min(k0 + kTileKeys - 1, pos); ++k) {
                    if (p.window && k <= pos - p.window && k >= p.sinks) continue;
                    const int page = ld_cg_s32(p.table + static_cast<int64_t>(x.b) * p.table_stride + k / p.P);
                    if (page < 0 || page >= p.num_pages) continue;
                    const int64_t at = page_row(p.layout, page, k % p.P, x.kvh, p.P, p.Hkv) * D + d0;
#pragma unroll
                    for (int d = 0; d < 16; ++d) {
                        float v;
                        if constexpr (KV8) v = (p.v[at + d] & 0x7f) == 0x7f ? NAN : 0.f;
                        else v = bits_to_f32<DT>(reinterpret_cast<const uint16_t*>(p.v)[at + d]);
                        if (!isfinite(v)) add[d] += v;
                    }
                }
            }
            __syncwarp();
#pragma unroll
            for (int d = 0; d < 16; ++d) o[d] = __float_as_uint(__uint_as_float(o[d]) + add[d]);
            tmem_st16_start(to + d0, o);
            tmem_st_wait();
        }
    }

    // Multiplies the accumulator of this warp's rows, at `to`, by `by`: its last product is done then, the next one waits
    // for this tile's weights.
    static __device__ __forceinline__ bool rescale(const Ctx& c, const ChunkParams& p, uint32_t to, uint32_t done, uint32_t count, float by) {
        if (!wait(p, done, (count - 1) & 1)) return false;
        tmem_fence_after_sync();
#pragma unroll 1
        for (int d = 0; d < D; d += 16) {
            uint32_t u[16];
            tmem_ld16(to + d, u);
#pragma unroll
            for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(u[j]));
#pragma unroll
            for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * by);
            tmem_st16_start(to + d, u);
        }
        tmem_st_wait();
        return true;
    }

    static __device__ __forceinline__ float max16(const float* s) {
        float a = s[0], b = s[1];
#pragma unroll
        for (int j = 2; j < 14; j += 4) {
            a = max3(a, s[j], s[j + 1]);
            b = max3(b, s[j + 2], s[j + 3]);
        }
        return fmaxf(max3(a, s[14], s[15]), b);
    }

    static __device__ void rows(const Ctx& c, const ChunkParams& p) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t ts = c.tmem + lanes + w * kTileKeys, tp = c.tmem + lanes + Sh::kP + w * Sh::kPStep, to = c.tmem + lanes + Sh::kO + w * D;
        uint32_t count = 0;            // key tiles so far
        for (uint32_t piece = 0;; ++piece) {
            ChunkPiece* const taken = take_piece(c, p, piece);
            if (!taken) return;
            ChunkPiece& x = *taken;
            // (the scores of the piece before are complete: the queries are no longer read)
            if (kRowFactors || piece == 0) {
                fetch_queries<32>(c, p, x, w, quarter * 32);
                if (lane == 0) mbar_arrive(c.q_full + 8 * w);
            }
            float factor = p.scale_log2;
            if constexpr (kRowFactors) factor = reinterpret_cast<const float*>(c.smem + Sh::kFactorOff)[w * kTileRows + r];
            const int f = x.rt * kItemRows + w * kTileRows + r, token = p.token(f);
            const bool live = f < x.s.n * p.G;
            const int pos = live ? x.s.L - x.s.n + token : -1;
            // references: scores' maximum m (16-bit pages: less kLift), and (8-bit pages) dv, how far the weights' is above it
            float m = kNoKey, dv = 0.f, l = 0.f;
            bool asked = false;            // the scores of the coming tile are known to be there
            const int t0 = x.t0, t1 = x.t1, sure = x.tiles.sure, plain0 = x.tiles.from, plain1 = x.tiles.to;
            for (int t = t0; t < t1; ++t, ++count) {
                const bool plain = t < sure || (t >= plain0 && t < plain1), first = t == t0;
                if (!(Sh::kApart && asked) && !wait(p, c.s_full + 8 * w, count & 1)) return;
                tmem_fence_after_sync();
                float s[kTileKeys];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld32_start(ts + 32 * i, s + 32 * i);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i) hold32(s + 32 * i);
                bool done = first;       // the weights before are no longer read (asked here, needed after the maxima)
                if constexpr (Sh::kApart) {
                    if (!first) done = mbar_try_wait(c.pv_done + 8 * w, (count - 1) & 1);
                    tmem_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(c.s_free + 8 * w);
                }
                float lv[8];             // 8-bit pages: log2 of the value scale, of 16 keys each
                if constexpr (KV8) {
                    if (!wait(p, c.sc_full + 8 * (count % kScaleRing), (count / kScaleRing) & 1)) return;
                    const float4* sc = reinterpret_cast<const float4*>(c.smem + Sh::kScaleOff) + (count % kScaleRing) * 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 f = sc[i];
                        lv[2 * i] = f.y;
                        lv[2 * i + 1] = f.w;
#pragma unroll
                        for (int g = 2 * i; g < 2 * i + 2; ++g) {
                            const float by = factor * (g & 1 ? f.z : f.x);
                            const uint64_t by2 = pair(by, by);
#pragma unroll
                            for (int j = 16 * g; j < 16 * g + 16; j += 2) unpair(mul2(pair(s[j], s[j + 1]), by2), s[j], s[j + 1]);
                        }
                    }
                }
                if (!plain) {
                    const int k0 = x.tiles.key(t), hi = pos - k0;
                    if (p.window == 0) {
#pragma unroll
                        for (int i = 0; i < kTileKeys; ++i) s[i] = i <= hi ? s[i] : -INFINITY;
                    } else {
                        const int low = max(pos, 0) - p.window + 1 - k0, sink = p.sinks - k0;
#pragma unroll
                        for (int i = 0; i < kTileKeys; i += 32) {      // a bit per key: two instructions for each, not four
                            const uint32_t seen = bits_below(hi + 1 - i) & (~bits_below(low - i) | bits_below(sink - i));
#pragma unroll
                            for (int j = 0; j < 32; ++j) s[i + j] = seen & (1u << j) ? s[i + j] : -INFINITY;
                        }
                    }
                }
                uint64_t sum0 = 0, sum1 = 0;
                // weights of keys 32 i on, relative to m
                const auto weights = [&](int i, uint32_t (&o)[16]) {
                    const uint64_t by2 = pair(factor, factor), m2 = pair(-m, -m);
                    float lift = 1.f;
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const int k = 32 * i + j;
                        float a, b;
                        unpair(KV8 ? add2(pair(s[k], s[k + 1]), m2) : fma2(pair(s[k], s[k + 1]), by2, m2), a, b);
                        a = fast_exp2(a);
                        b = fast_exp2(b);
                        uint64_t e = pair(a, b);
                        if (j & 2) sum1 = add2(sum1, e);
                        else sum0 = add2(sum0, e);
                        if constexpr (KV8) {
                            if (j % 16 == 0) lift = fast_exp2(fminf(lv[k / 16] - dv, 127.f));
                            e = mul2(e, pair(lift, lift));
                            unpair(e, a, b);
                        }
                        o[j / 2] = pack2<MT>(a, b);
                    }
                };
                uint32_t o0[16], o1[16];
                // 16-bit pages: the first half's weights by the reference as it is, beside the maxima, which seldom move it: the exponents'
                // unit and the maxima's need not wait for each other (16 heads of size 64, 16384 tokens 383 -> 370 us)
                if constexpr (!KV8) {
                    weights(0, o0);
                    weights(1, o1);
                }
                // maxima of 16 keys, the size of the smallest page
                float top[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) top[i] = max16(s + 16 * i);
                float best = max3(max3(top[0], top[1], top[2]), max3(top[3], top[4], top[5]), fmaxf(top[6], top[7]));
                if constexpr (KV8) {
                    // a weight that is too large moves the references as a score does
                    bool move = best - m > kHeadroom;
#pragma unroll
                    for (int i = 0; i < 8; ++i) move = move || (top[i] - m) + (lv[i] - dv) > kHeadroom + kLift;
                    if (first || __any_sync(0xffffffffu, move)) {
                        const float mn = fmaxf(m, best);
                        // (not below kNoKey: with no value that counts so far, as behind a first tile that the row does not see, the
                        // sum is -inf, and a tile whose value scales are all 0 would leave lv - dv without a value)
                        float dn = first ? kNoKey : fmaxf(kNoKey, (m - mn) + dv);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dn = fmaxf(dn, (top[i] - mn) + (lv[i] - kLift));
                        if (!first) {
                            l *= fast_exp2(m - mn);
                            if (!rescale(c, p, to, c.pv_done + 8 * w, count, fast_exp2((m - mn) + (dv - dn)))) return;
                        }
                        m = mn;
                        dv = dn;
                    }
                } else {
                    best *= factor;
                    const bool move = first || best - m > kHeadroom + kLift;
                    if (__any_sync(0xffffffffu, move)) {
                        const float mn = move ? fmaxf(m, best - kLift) : m, by = fast_exp2(m - mn);
                        l *= by;
                        m = mn;
                        if (!first && !rescale(c, p, to, c.pv_done + 8 * w, count, by)) return;
                        sum0 = sum1 = 0;
                        weights(0, o0);
                        weights(1, o1);
                    }
                    if (w == 0 && !plain) {
                        const uint32_t v = 2 * count + 1;
                        if (!wait(p, c.kv_full + 8 * (v % Sh::kRing), (v / Sh::kRing) & 1)) return;
                        if (clean_values(p, x.tiles, x.tiles.key(t), ring(c, v % Sh::kRing))) x.dirty = 1;
                    }
                }
                if constexpr (Sh::kApart) {
                    if (!__all_sync(0xffffffffu, done) && !wait(p, c.pv_done + 8 * w, (count - 1) & 1)) return;
                    tmem_fence_after_sync();
                }
                if constexpr (KV8) weights(0, o0);
                tmem_st16_start(tp, o0);
                if constexpr (KV8) weights(1, o1);
                tmem_st16_start(tp + 16, o1);
                tmem_st_wait();
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(c.p_half + 8 * w);
                weights(2, o0);
                tmem_st16_start(tp + 32, o0);
                weights(3, o1);
                tmem_st16_start(tp + 48, o1);
                if constexpr (Sh::kApart) asked = mbar_try_wait(c.s_full + 8 * w, (count + 1) & 1) && t + 1 < t1;   // the next scores
                tmem_st_wait();
                tmem_fence_before_sync();
                __syncwarp();
                if constexpr (Sh::kApart) asked = __all_sync(0xffffffffu, asked);
                if (lane == 0) {
                    mbar_arrive(c.p_full + 8 * w);
                    if constexpr (KV8) mbar_arrive(c.sc_empty + 8 * (count % kScaleRing));
                }
                float a, b;
                unpair(add2(sum0, sum1), a, b);
                l += a + b;
            }
            // ---- the piece's end
            if (!wait(p, c.pv_done + 8 * w, (count - 1) & 1)) return;
            tmem_fence_after_sync();
            const bool whole = t0 == 0 && t1 == x.tiles.nt;
            if (*static_cast<volatile int*>(&x.dirty) != 0) add_non_finite(p, x, pos, to);
            const bool none = m == kNoKey && l == 0.f;
            const float by = none ? 0.f : 1.f / l;
            const int64_t row = x.s.r0 + token, head = static_cast<int64_t>(x.kvh) * p.G + (f - token * p.G);
            const int slot = 2 * static_cast<int>(blockIdx.x) + (t0 == 0 ? 1 : 0);
            const float root = KV8 ? fast_exp2(0.5f * dv) : 1.f;   // 2^dv in two steps, which stay normal floats for every scale
#pragma unroll
            for (int d0 = 0; d0 < D; d0 += 64) {
                float o[64];
                tmem_ld32_start(to + d0, o);
                tmem_ld32_start(to + d0 + 32, o + 32);
                tmem_ld_wait();
                hold32(o);
                hold32(o + 32);
                if constexpr (KV8) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) o[j] = o[j] * root * root;
                }
                if (whole) {
                    if (live) {
                        uint16_t* out = p.out + row * p.out_stride + head * D + d0;
#pragma unroll
                        for (int j = 0; j < 64; j += 16) {
                            uint32_t y[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) y[i] = pack2<DT>(o[j + 2 * i] * by, o[j + 2 * i + 1] * by);
                            if (p.out_wide) {      // a sector each
                                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + j), "r"(y[0]), "r"(y[1]),
                                             "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                                             : "memory");
                            } else {
                                *reinterpret_cast<uint4*>(out + j) = make_uint4(y[0], y[1], y[2], y[3]);
                                *reinterpret_cast<uint4*>(out + j + 8) = make_uint4(y[4], y[5], y[6], y[7]);
                            }
                        }
                    }
                } else if (live) {
                    float4* out = p.part + (static_cast<int64_t>(slot) * (D / 4) + d0 / 4) * kItemRows + w * kTileRows + r;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        out[j * kItemRows] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                }
            }
            if (!whole && live) p.part_sum[static_cast<int64_t>(slot) * kItemRows + w * kTileRows + r] = make_float2(m, l);
            if (whole && p.lse != nullptr && live) p.lse[row * p.Hq + head] = none ? -INFINITY : (m + fast_log2(l)) * kLn2;
            tmem_fence_before_sync();
            __syncwarp();
            if (lane == 0) drop_piece(c, piece);
        }
    }
};

template <int D, int DT, bool KV8>
__global__ void __launch_bounds__(ChunkShape<D, KV8>::kThreads, 1)
chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const ChunkParams p) {
    using K = ChunkKernel<D, DT, KV8>;
    using Sh = typename K::Sh;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    typename K::Ctx c;
    c.smem = smem_raw;
    c.base = smem_addr(c.smem);
    if (c.base & 1023) {   // (it begins the block's shared memory, there is no room to move it)
        grid_dependency_wait();
        if (threadIdx.x == 0) {
            p.join[blockIdx.x] = {};   // no parts that the second kernel could join
            flag_error(p.err, DA_DEVERR_TIMEOUT);
        }
        return;
    }
    ChunkPlan& plan = *reinterpret_cast<ChunkPlan*>(c.smem + Sh::kPlanOff);
    uint32_t bar = c.base + Sh::kBarOff;
    auto bars = [&](int n) {
        const uint32_t at = bar;
        bar += 8 * n;
        return at;
    };
    c.kv_full = bars(Sh::kRing);
    c.kv_empty = bars(Sh::kRing);
    c.raw_full = bars(Sh::kRaw);
    c.raw_empty = bars(Sh::kRaw);
    c.sc_full = bars(kScaleRing);
    c.sc_empty = bars(kScaleRing);
    c.x_full = bars(kPieceRing);
    c.x_empty = bars(kPieceRing);
    c.q_full = bars(2);
    c.q_empty = bars(2);
    c.s_full = bars(2);
    c.s_free = bars(2);
    c.p_half = bars(2);
    c.p_full = bars(2);
    c.pv_done = bars(2);
    c.fin = bars(1);
    c.plan = &plan;
    c.pieces = reinterpret_cast<ChunkPiece*>(c.smem + Sh::kPieceOff);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kRing; ++i) {
            mbar_init(c.kv_full + 8 * i, KV8 ? 4 : 1);
            mbar_init(c.kv_empty + 8 * i, 1);
        }
        for (int i = 0; i < Sh::kRaw; ++i) {
            mbar_init(c.raw_full + 8 * i, 1);
            mbar_init(c.raw_empty + 8 * i, 4);
        }
        for (int i = 0; i < kScaleRing; ++i) {
            mbar_init(c.sc_full + 8 * i, 1);
            mbar_init(c.sc_empty + 8 * i, Sh::kRowWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(c.q_full + 8 * i, 4);
            mbar_init(c.q_empty + 8 * i, 1);
            mbar_init(c.s_full + 8 * i, 1);
            mbar_init(c.s_free + 8 * i, 4);
            mbar_init(c.p_half + 8 * i, 4);
            mbar_init(c.p_full + 8 * i, 4);
            mbar_init(c.pv_done + 8 * i, 1);
        }
        mbar_init(c.fin, 1);
        for (int i = 0; i < kPieceRing; ++i) {
            mbar_init(c.x_full + 8 * i, 1);
            mbar_init(c.x_empty + 8 * i, Sh::kPieceReaders);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == Sh::kRowWarps + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(c.base + Sh::kTmemOff), "r"(Sh::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // From here on this grid touches global memory: wait for the previous kernel.
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_dependents_launch();
    chunk_plan<Sh::kThreads>(p, c.smem + Sh::kRingOff, plan);
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    if (threadIdx.x == 0) leave_join(p, plan);
    c.tmem = *reinterpret_cast<const volatile uint32_t*>(c.smem + Sh::kTmemOff);
    if (warp < Sh::kRowWarps) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Sh::kRowRegs));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Sh::kOtherRegs));
    if (warp < Sh::kRowWarps) K::rows(c, p);
    else if (warp == Sh::kRowWarps) K::producer(c, p, &tmK, &tmV);
    else if (warp == Sh::kRowWarps + 1) {
        K::multiplier(c, p);
    } else if (warp < Sh::kRowWarps + 4) {
        K::queries(c, p, warp - Sh::kRowWarps - 2);
    }
    if constexpr (KV8) {
        if (warp >= Sh::kRowWarps + 4) K::converter(c, p);
    }
    tmem_fence_before_sync();
    __syncthreads();
    if (warp == Sh::kRowWarps + 1) {
        tmem_fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(c.tmem), "r"(Sh::kCols));
    }
}

// Joins the parts of the split items: block (range, slice) 32 rows of the item whose first part that range holds, a
// thread 16 dims of a row.
template <int D, int DT>
__global__ void __launch_bounds__(32 * D / 16) chunk_join_kernel(const ChunkParams p) {
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_dependents_launch();
    const int range = blockIdx.x / kJoinSlices, slice = blockIdx.x % kJoinSlices;
    const ChunkJoin join = p.join[range];
    const int r = slice * 32 + (threadIdx.x & 31), f = join.rt * kItemRows + r, d = threadIdx.x / 32 * 16;
    if (join.parts == 0 || f >= join.n * p.G) return;
    auto slot = [&](int j) { return static_cast<int64_t>(j == 0 ? 2 * range + 1 : 2 * (range + j)); };
    // a few parts at a time, all of their loads before any is needed
    constexpr int kAhead = 4;
    float m = kNoKey, l = 0.f, o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.f;
    for (int j0 = 0; j0 < join.parts; j0 += kAhead) {
        float2 sum[kAhead];
        float4 x[kAhead][4];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const bool some = j0 + j < join.parts;
            const float4* part = p.part + (slot(some ? j0 + j : 0) * (D / 4) + d / 4) * kItemRows + r;
            sum[j] = some ? __ldcg(p.part_sum + slot(j0 + j) * kItemRows + r) : make_float2(kNoKey, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[j][i] = some ? __ldcg(part + i * kItemRows) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float top = m;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) top = fmaxf(top, sum[j].x);
        const float old = fast_exp2(m - top);
        m = top;
        l *= old;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] *= old;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (j0 + j >= join.parts) break;
            const float w = fast_exp2(sum[j].x - m);
            l = fmaf(w, sum[j].y, l);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[4 * i] = fmaf(w, x[j][i].x, o[4 * i]);
                o[4 * i + 1] = fmaf(w, x[j][i].y, o[4 * i + 1]);
                o[4 * i + 2] = fmaf(w, x[j][i].z, o[4 * i + 2]);
                o[4 * i + 3] = fmaf(w, x[j][i].w, o[4 * i + 3]);
            }
        }
    }
    const bool none = m == kNoKey && l == 0.f;
    const float by = none ? 0.f : 1.f / l;
    const int token = p.token(f);
    const int64_t row = join.r0 + token, head = static_cast<int64_t>(join.kvh) * p.G + (f - token * p.G);
    uint4* out = reinterpret_cast<uint4*>(p.out + row * p.out_stride + head * D + d);
#pragma unroll
    for (int j = 0; j < 2; ++j)
        out[j] = make_uint4(pack2<DT>(o[8 * j] * by, o[8 * j + 1] * by), pack2<DT>(o[8 * j + 2] * by, o[8 * j + 3] * by),
                            pack2<DT>(o[8 * j + 4] * by, o[8 * j + 5] * by), pack2<DT>(o[8 * j + 6] * by, o[8 * j + 7] * by));
    if (p.lse != nullptr && d == 0) p.lse[row * p.Hq + head] = none ? -INFINITY : (m + fast_log2(l)) * kLn2;
}

template <int D, int DT, bool KV8>
da_status launch_chunk(const da_paged_cache& c, ChunkParams& p, cudaStream_t stream) {
    using Sh = ChunkShape<D, KV8>;
    constexpr int kInner = KV8 ? D : 64;
    p.box_keys = gcd_of(c.page_size, kTileKeys);
    CUtensorMap mk, mv;
    if (!make_page_map(&mk, c.k, c, kInner, p.box_keys) || !make_page_map(&mv, c.v, c, kInner, p.box_keys)) return DA_ERR_CUDA;
    auto kern = chunk_kernel<D, DT, KV8>;
    static DeviceCache cache;
    int resident = 0;
    if (persistent_grid(kern, Sh::kThreads, Sh::kSmemBytes, cache, &resident) != cudaSuccess) return DA_ERR_CUDA;
    const int grid = std::min(std::min(resident, device_sms()), kMaxRanges);
    cudaLaunchAttribute attrs[1] = {pdl_attr()};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(Sh::kThreads);
    cfg.dynamicSmemBytes = Sh::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, mk, mv, p) != cudaSuccess) return DA_ERR_CUDA;
    cfg.gridDim = dim3(grid * kJoinSlices);
    cfg.blockDim = dim3(32 * D / 16);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, chunk_join_kernel<D, DT>, p) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

template <int D, int DT>
da_status launch_chunk_any(const da_paged_cache& c, ChunkParams& p, cudaStream_t s) {
    return c.kv_dtype == DA_E4M3 ? launch_chunk<D, DT, true>(c, p, s) : launch_chunk<D, DT, false>(c, p, s);
}

}  // namespace da_impl

using namespace da_impl;

extern "C" {

size_t decode_attn_paged_chunk_workspace_size(int Hq, int Hkv, int D) {
    if (Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
    return kPagedHeadBytes + round_up(kMaxRanges * sizeof(ChunkJoin), 256) +
           static_cast<size_t>(2 * kMaxRanges) * kItemRows * (sizeof(float2) + D * sizeof(float));
}

da_status decode_attn_paged_chunk(const da_paged_chunk* args, void* stream) {
    if (!args) return DA_ERR_INVALID_ARG;
    const da_paged_chunk& a = *args;
    const da_status st = check_cache(a.cache, a.dtype, a.kv_lens, a.block_table, a.max_pages, a.table_stride, a.B, a.Hq);
    if (st != DA_OK) return st;
    const da_paged_cache& c = *a.cache;
    if (a.Hq < 1 || a.T_new < 0 || !std::isfinite(a.scale) || a.window < 0 || a.sinks < 0) return DA_ERR_INVALID_ARG;
    if (!a.cu_new || !a.workspace) return DA_ERR_INVALID_ARG;
    if (!aligned(a.cu_new, 4) || !aligned(a.workspace, 256)) return DA_ERR_ALIGNMENT;
    const int64_t row = static_cast<int64_t>(a.Hq) * c.D;
    if (a.q_stride < row || a.out_stride < row) return DA_ERR_INVALID_ARG;
    if (a.q_stride % 8 || a.out_stride % 8) return DA_ERR_ALIGNMENT;
    // rows of the items are numbered in 32 bits
    if (static_cast<int64_t>(a.T_new) * (a.Hq / c.Hkv) > 0x3fffffffll) return DA_ERR_INVALID_ARG;
    if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.lse, 4)) return DA_ERR_ALIGNMENT;
    if (a.workspace_bytes < decode_attn_paged_chunk_workspace_size(a.Hq, c.Hkv, c.D)) return DA_ERR_WORKSPACE_TOO_SMALL;
    if (a.T_new == 0) return DA_OK;
    if (!a.q || !a.out) return DA_ERR_INVALID_ARG;
    ChunkParams p;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    p.q = static_cast<const uint16_t*>(a.q);
    p.v = static_cast<const uint8_t*>(c.v);
    p.ks = c.k_scale;
    p.vs = c.v_scale;
    p.cu = a.cu_new;
    p.lens = a.kv_lens;
    p.table = a.block_table;
    p.out = static_cast<uint16_t*>(a.out);
    p.lse = a.lse;
    p.err = reinterpret_cast<uint32_t*>(ws);
    p.join = reinterpret_cast<ChunkJoin*>(ws + kPagedHeadBytes);
    p.part = reinterpret_cast<float4*>(ws + kPagedHeadBytes + round_up(kMaxRanges * sizeof(ChunkJoin), 256));
    p.part_sum = reinterpret_cast<float2*>(p.part + static_cast<size_t>(2 * kMaxRanges) * kItemRows * (c.D / 4));
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.out_wide = aligned(a.out, 32) && a.out_stride % 16 == 0;
    p.B = a.B;
    p.T = a.T_new;
    p.Hq = a.Hq;
    p.Hkv = c.Hkv;
    p.G = a.Hq / c.Hkv;
    // floor(f / G) = f * ceil(2^(31 + l) / G) >> (31 + l) for every f < 2^31, with 2^l >= G > 2^(l - 1)
    int l = 0;
    while ((1ll << l) < p.G) ++l;
    p.group_shift = 31 + l;
    p.group_mul = static_cast<uint32_t>(((1ull << p.group_shift) + p.G - 1) / p.G);
    p.P = c.page_size;
    p.max_pages = a.max_pages;
    p.table_stride = a.table_stride;
    p.num_pages = c.num_pages;
    p.layout = c.layout;
    p.window = std::min(a.window, 0x7fffff00);   // (no sequence is longer; the kernel subtracts it)
    p.sinks = a.sinks;
    p.scale_log2 = std::fabs(a.scale) * kLog2e;
    const bool zero = p.scale_log2 == 0.f;       // (a factor of 0 would make NaN of the scores taken out)
    if (zero) p.scale_log2 = 1.f;
    p.q_zero = zero;
    p.q_xor = !zero && a.scale < 0.f ? 0x80008000u : 0u;
    p.wait_limit_ns = kWaitLimitNs;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (c.D == 128) return a.dtype == DA_F16 ? launch_chunk_any<128, DA_F16>(c, p, s) : launch_chunk_any<128, DA_BF16>(c, p, s);
    return a.dtype == DA_F16 ? launch_chunk_any<64, DA_F16>(c, p, s) : launch_chunk_any<64, DA_BF16>(c, p, s);
}

}  // extern "C"
