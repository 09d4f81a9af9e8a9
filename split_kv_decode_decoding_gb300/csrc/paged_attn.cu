// Decode attention over a paged KV cache (decode_attn_paged.h) for GB300 / sm_103a, with
// pages of 16-bit or of e4m3 elements.
//
// Per (sequence b, KV head, chunk of up to 8 or 16 packed (token, head) columns):
//     x_j = scale * ks * (q . k_j),   out = sum_j 2^(x_j log2e - m) vs v_j / sum_j 2^(x_j log2e - m)
// in one pass over the keys with a running maximum m (ks, vs: the scales of key j's page and
// head, 1 in 16-bit pages).
//
// What bounds it: the K/V bytes. A key costs 4 D (16-bit) or 2 D (e4m3) bytes for 4 D
// operations per column, far below what the tensor cores deliver, so everything here serves
// the stream. Short calls are bound by latency: a chain of kv_lens, block table, first copy,
// a few stages, the merge of the warps, a partial result's way through the L2. 16-column
// e4m3 calls by the consumer warps' instructions (40 % of the issue slots at 2.4 warps
// per scheduler, each waiting for its own results).
//
// How the work is cut. The unit is a stage of 64 or 128 keys of a sequence. The units of
// the batch, in order, are cut into about as many equal ranges as there are persistent CTAs
// per KV head and chunk, whatever the lengths are: the host knows none of them, and no split
// count has to be chosen. A range may hold the end of one sequence, several whole ones and the
// beginning of another; a sequence that lies in one range is written by it directly, otherwise
// each of its ranges leaves a partial result (at most two per range, so the workspace does not
// grow with the batch) and the warp that finishes a column last merges that column's partials,
// in range order whoever it is: the result does not depend on timing. Every KV head is cut
// alike and the heads of a range run at the same time, so that the interleaved rows of a page
// are read together (16 sequences of 8192 keys, e4m3, tokens outside heads: 68.0 us with one
// cut through all heads, 51.3 us so).
//
// A CTA is one producer warp and four or eight consumer warps around a ring of stages, as in the
// split kernel for contiguous caches. With four, two CTAs share an SM (three at head size 64).
// 16-bit pages of head size 128 have one CTA of eight per SM: as many warps on half as many ranges, so
// half the partial results, and a short range streams twice as fast (16 x 131072 keys 1189 -> 1153 us,
// the ragged batch 89 -> 85 us, one sequence of 32768 keys 31.0 -> 28.5 us), unless the table's rows hold
// few keys (256 sequences of 256: 18.6 us against 16.3, 64 of 512: 25.8 against 25.4, of 960: 45.3 against
// 42.8, where two CTAs cover each other's ends; of 1024: 46.0 against 44.6, but 16 of 1024 15.3 against 16.4
// and 16 of 2048 24.5 against 27.4). e4m3 pages, whose consumers work harder, lose by it (four tokens
// 191 us against 169), as does head size 64. The producer's lanes read the block table (and the
// scales) of the next 32 boxes at once, one batch ahead of the copies, and each lane issues its own
// box: TMA boxes of gcd(page size, stage) keys, 16-key boxes at a sequence's ragged end, so that a
// box never crosses a page.
//
// e4m3 pages. The products run as fp16 tensor-core products: every e4m3 value is an fp16
// value, and one conversion takes two elements, 0.5 cycles per SM (measured), 2 of the 11
// cycles that a key of 2 x 128 bytes takes to stream. Queries in bf16 are scaled by a power of
// two per column into the top of the fp16 range (an element below 2^-28 of its column's largest
// loses bits, by at most 2^-39 of that largest). The order of the dims inside a 16-dim step is
// free, so one ldmatrix of 16-bit pairs feeds two steps. The scales never touch the elements: ks
// multiplies the score, and vs goes into the exponent of the weight, 2^((x - m) + (log2 vs - dv)),
// with m + dv a running maximum of its own, so that the fp16 weights keep their precision however
// unequal the pages' scales are. It is held as its distance dv from m: beside a large score log2 vs
// would lose its last bits.
//
// Sums, maxima, accumulators and partial results are float32. A partial result keeps its maximum and its
// sum apart, so that scores of any size are joined with no more loss than they were computed with. Rounded to fewer bits are the
// weights, in 16-bit pages to two terms of their type and in 8-bit pages to one of fp16 (weights16), and the outputs, once.
//
// Measured (one GB300, mean of a graph of calls): 16 sequences of 131072 keys, 32 / 8 heads, bf16
// 1156 us, 7.4 TB/s; 64 sequences of 512 to 8192 keys, 28 / 4 heads 86.2 us, 6.4 TB/s, over e4m3
// pages 51.3 us, 5.4 TB/s; one sequence of 1024 keys 9.0 us, of 8192 keys over e4m3 pages 11.1 us.

#include "paged_common.cuh"

namespace da_impl {

constexpr int kPagedShares = 2048;   // bound of shares (range, KV head, chunk), each with two partial results
constexpr int kWriters = 4;          // consumer warps that write a piece's columns, two of every eight each
constexpr size_t kPagedCounterBytes = static_cast<size_t>(kPagedShares) * kWriters * 4;
constexpr int kAlignRange = 16;      // ranges of an even batch up to so long follow its sequences in any case
constexpr int kMaxSlack = 4;         // units that a cut may move to avoid a partial result
constexpr int kFewUnits = 8;         // units per SM of a full table up to which CTAs have an SM each
constexpr int kShortCapacity = 1023; // keys of the block table's rows up to which CTAs of four consumer warps do better
constexpr float kNoKey = -3.402823466e38f;   // running maximum of a column that has seen no key: the least finite
                                             // value, so that every finite score is above it and no NaN arises

template <int D, bool KV8, int NT, int NW>
struct PagedShape {
    static constexpr int kWarps = NW;                               // consumer warps
    static constexpr int kThreads = (kWarps + 1) * 32;
    static constexpr int kKeys = kWarps == 8 || KV8 ? 128 : 64;     // keys per stage
    static constexpr int kBoxes = kKeys / kWarps / 16;              // 16-key boxes per consumer warp
    static constexpr int kRowBytes = KV8 ? D : 2 * D;
    static constexpr int kSliceRow = kRowBytes < 128 ? kRowBytes : 128;   // bytes per row of a TMA box
    static constexpr int kSlices = kRowBytes / kSliceRow;
    static constexpr int kSliceBytes = kKeys * kSliceRow;
    static constexpr int kTileBytes = kSlices * kSliceBytes;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kRing = kWarps == 8 ? (196608 / kStageBytes < 8 ? 196608 / kStageBytes : 8) : 3;
    static constexpr int kRingBytes = kRing * kStageBytes;
    static constexpr int kCols = 8 * NT;
    static constexpr int kLeast = kKeys == 64 || KV8 ? 2 : 1;       // units of a range at least (see Ranges)
    // the merge of the warps, in a ring stage: [warp][8] rows of accumulators, free of bank conflicts both ways by
    // four floats of padding, or where the stage has no room for it, by dim d of column c at d ^ 4 (c % 8); and
    // beside the ring [warp][8] maxima, the weights' distance from them, sums
    static constexpr int kMergeRow = kWarps == 8 ? D : D + 4;
    static __device__ __forceinline__ int merge_dim(int d, int col) { return kWarps == 8 ? d ^ (4 * (col & 7)) : d; }
    static_assert(kWarps * 8 * kMergeRow * 4 <= kStageBytes, "item merge must fit in one ring stage");
    static constexpr int kQBytes = kCols * D * 2;
    static constexpr int kQOff = kRingBytes;
    static constexpr int kSlotOff = kQOff + kItemSlots * kQBytes;
    static constexpr int kSlotBytes = 64;
    static constexpr int kScaleOff = kSlotOff + kItemSlots * kSlotBytes;   // [stage][box] {ks, log2 vs}
    static constexpr int kScaleBytes = KV8 ? kRing * (kKeys / 16) * 8 : 0;
    static constexpr int kRedOff = kScaleOff + kScaleBytes;
    static constexpr int kRedFloats = 3 * kWarps * 8;                      // twice, used in turn
    static constexpr int kLastOff = kRedOff + 2 * kRedFloats * 4;          // [writer][2] merges to do
    static constexpr int kBarOff = kLastOff + kWriters * 2 * kSlotBytes;
    static constexpr int kNumBars = 2 * kRing + 2 * kItemSlots + 2;
    static constexpr int kSeqOff = kBarOff + kNumBars * 8;                 // prefix[B + 1], even, then pad[B]
    static constexpr int smem_bytes(int B) { return 1024 + kSeqOff + (4 * (B + 2) + B + 15) / 16 * 16; }
};

struct PagedParams {
    const uint16_t* q;
    const float* ks;
    const float* vs;
    const int32_t* lens;
    const int32_t* table;
    uint16_t* out;
    float* lse;              // or nullptr
    uint32_t* err;
    uint32_t* arrived;       // [share][consumer warp] partials written, at the share that begins a (sequence, head)
    float2* part_sum;        // [2 * share][columns] {maximum m, sum of 2^(x - m)}: a logarithm of the sum would lose
                             // its last bits beside a large m
    float* part;             // [2 * share][columns][D], sums of weighted values relative to the same m
    int B, tq, Hq, Hkv, G, P, max_pages, table_stride, num_pages, layout, chunks;
    int lanes;               // CTAs per range: Hkv * chunks
    int slots, one;          // ranges that run at once, and ranges that have an SM to themselves
    int box_keys;            // keys of a full TMA box: gcd(page size, stage keys)
    uint32_t page_mul;       // position / P by multiplication (page())
    int page_shift;
    float scale_log2;
    unsigned long long wait_limit_ns;

    __device__ __forceinline__ int page(int pos) const {
        return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(pos)) * page_mul) >> page_shift);
    }
};

struct PagedItem {           // one piece of a (sequence, KV head): what a range holds of it
    int32_t valid, b, kvh, c0, nh;
    int32_t key0, nkeys, ntiles;
    int32_t vis0;            // keys of the piece that query token 0 may see (may be <= 0)
    int32_t part;            // partial result to write, or -1: the piece is the whole
    int32_t first_share;     // share that holds the (sequence, head)'s first key
    int32_t nparts;
};
static_assert(sizeof(PagedItem) <= 64, "PagedItem fits its slot");

// The cut of the batch's `units` into n ranges, for every KV head and chunk alike: k raw cuts at equal
// distances (q or q + 1 units) in every w units.
//
// Few units go to one range per SM, more to all the CTAs that run at once. A batch of unequal lengths is
// one period of w = units. Where every sequence has the same t units and ranges are short, a period
// is one of them (cut into k parts) or several whole ones (k = 1), so that no range holds the end of one
// and the beginning of the next: that costs a second merge of the warps and a partial result, 2 to 3 us
// against the 1 to 1.5 us that a unit takes to stream with every SM busy (256 sequences of 256 keys, 2 KV
// heads: 24.0 us with plain equal cuts, 16.6 us with whole sequences).
// Otherwise a raw cut within `slack` units of a border moves there (4 slack <= q keeps the ranges in order).
//
// A division by a number that is not known at compile time takes some 70 ns and nothing streams before
// these are done, so independent ones stand together, where they overlap.
struct Ranges {
    int units, n, w, k, q, rem, split, slack;
    // t: units of every sequence, or 0. slots: ranges that run at once; `one` of them take an SM each. least:
    // units of a range at least where every sequence has eight or more of them (two where it has sixteen, twice
    // as many in a batch of unequal lengths, and sequences shorter than that stay whole). streams: the bytes bound
    // the kernel (not the 16-column products of e4m3 pages).
    __device__ __forceinline__ Ranges(int u, int t, int slots, int one, int short_range, int least,
                                      bool streams)
        : units(u) {
        const int share1 = (u + one - 1) / one, share = (u + slots - 1) / slots;
        // one range per SM while it is short, then all slots
        int size = max(t >= 16 ? 2 : t >= 8 ? least : 2 * least, share1);
        if (size > (t >= size ? kAlignRange : short_range)) size = max(short_range, share);
        const int cuts = (u + size - 1) / size, parts = t / size, whole = (size + t - 1) / max(t, 1), seqs = u / max(t, 1);
        // long ranges too, where four fifths of the slots are enough because the stream bounds them
        const bool follow = t > 0 && (size <= kAlignRange || (streams && size < t && 5 * parts * seqs >= 4 * slots));
        w = !follow ? units : size < t ? t : whole * t;
        k = !follow ? min(cuts, slots) : size < t ? parts : 1;
        const int periods = (units + w - 1) / w;
        q = w / k;
        n = periods * k;
        rem = w - q * k;
        split = rem * (q + 1);
        slack = min(q / 4, kMaxSlack);
    }
    // cut r, and the first r with raw(r) >= x
    __device__ __forceinline__ int raw(int r) const {
        const int p = r / k, j = r - p * k;
        return p * w + j * q + min(j, rem);
    }
    __device__ __forceinline__ int first_from(int x) const {
        const int p = x / w, y = x - p * w;
        const bool low = y <= split;
        const int j = (low ? y + q : y - split + q - 1) / (low ? q + 1 : q);
        return p * k + (low ? j : rem + j);
    }
    // Ranges that hold parts of the sequence of units [a, b): the first, and their number.
    __device__ __forceinline__ void parts(int a, int b, int& first, int& count) const {
        const int lo = first_from(a + slack + 1), end = first_from(b - slack);
        first = lo - 1;                // cuts lo .. end - 1 lie inside
        count = max(end - lo, 0) + 1;
    }
};

// mbar_wait and mbar_wait_warp with their loop kept a loop: unrolled at some twenty places it makes up a
// third of the kernel's code, and a call on a short sequence spends a microsecond fetching code.
__device__ __forceinline__ bool wait_lane(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
#pragma unroll 1
    do {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
    } while (global_ns() - t0 <= limit_ns);
    return false;
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
    const bool ok = wait_lane(bar, parity, limit_ns);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void fence_acq_rel() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// yes ? a : b, kept a selection: of several from one array the compiler makes an index, and the array goes to local memory.
__device__ __forceinline__ float select(bool yes, float a, float b) {
    float r;
    asm("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %3, 0;\n\tselp.f32 %0, %1, %2, p;\n\t}"
        : "=f"(r)
        : "f"(a), "f"(b), "r"(static_cast<int>(yes)));
    return r;
}

// log2 of a scale, a subnormal one too (-inf of 0).
__device__ __forceinline__ float log2_of_scale(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// pack2, rounded towards zero.
template <int DT>
__device__ __forceinline__ uint32_t pack2_down(float a, float b) {
    uint32_t r;
    if constexpr (DT == DA_F16) asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Two e4m3 values to two fp16 values (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}

template <int D, int DT, bool KV8, int NT, int NW>
struct PagedKernel {
    using Sh = PagedShape<D, KV8, NT, NW>;

    // A weight enters its product as 2^kLift times itself, and is at most 2^kHeadroom times the largest one at the time
    // that its column's reference was set (a larger one moves the reference). bf16 holds any of them. fp16 ends at 2^-24,
    // and at 2^16: lifted by 11 to the top of it, weights keep all their bits down to 2^-25 of the largest, and count down
    // to 2^-36. (Unlifted, down to 2^-14 and 2^-25: 10^5 keys of 2^-26 beside one are 2^-9 of the sum, and went missing.)
    // Less headroom means more moves, which the 16-column kernel of 8-bit pages feels: four tokens 172.4 us with 8 and
    // 7, 176.3 with 4 and 11, 171.7 unlifted; it is given the first, 2^-21 and 2^-32. One token: 50.7, 50.9 and 50.6.
    static constexpr bool kFp16Weights = KV8 || DT == DA_F16;
    static constexpr bool kFewMoves = KV8 && NT == 2;
    static constexpr float kHeadroom = kFp16Weights && !kFewMoves ? 4.f : kLazyRescale;
    static constexpr float kLift = kFp16Weights ? 15.f - kHeadroom : 0.f;
    // In 16-bit pages a factor of the weights (2^kLift), beside the sum that keeps them as they are (fp16, four tokens 116.3 ->
    // 118.2 us, one token 86.5 both); in 8-bit pages, whose weights have a reference of their own, part of that one (dv).
    static constexpr float kLiftBy = !KV8 && kFp16Weights ? 2048.f : 1.f;
    static_assert(kLiftBy == 1.f || kLift == 11.f, "kLiftBy is 2^kLift");

    struct Layout {
        uint8_t* smem;
        PagedItem* slots;
        float2* scales;
        int32_t* prefix;
        uint8_t* pad;
        uint32_t ring, qbuf, full0, empty0, ifull0, iempty0, mfull, mdone;
    };

    static __device__ __forceinline__ Layout layout(uint8_t* raw, const PagedParams& p) {
        Layout s;
        s.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
        s.slots = reinterpret_cast<PagedItem*>(s.smem + Sh::kSlotOff);
        s.scales = reinterpret_cast<float2*>(s.smem + Sh::kScaleOff);
        s.prefix = reinterpret_cast<int32_t*>(s.smem + Sh::kSeqOff);
        s.pad = reinterpret_cast<uint8_t*>(s.prefix + p.B + 2);
        s.ring = smem_addr(s.smem);
        s.qbuf = s.ring + Sh::kQOff;
        s.full0 = s.ring + Sh::kBarOff;
        s.empty0 = s.full0 + 8 * Sh::kRing;
        s.ifull0 = s.empty0 + 8 * Sh::kRing;
        s.iempty0 = s.ifull0 + 8 * kItemSlots;
        s.mfull = s.iempty0 + 8 * kItemSlots;
        s.mdone = s.mfull + 8;
        return s;
    }

    static __device__ __forceinline__ PagedItem* slot_of(const Layout& s, int i) {
        return reinterpret_cast<PagedItem*>(reinterpret_cast<uint8_t*>(s.slots) + i * Sh::kSlotBytes);
    }

    static __device__ __forceinline__ PagedItem* last_of(const Layout& s, int warp, int i) {
        return reinterpret_cast<PagedItem*>(s.smem + Sh::kLastOff + (2 * warp + i) * Sh::kSlotBytes);
    }

    // A length as it counts, and the stages of sequence b (keeping how many keys its last one lacks).
    static __device__ __forceinline__ int checked_length(const PagedParams& p, int L) {
        if (L < 0 || L > static_cast<int64_t>(p.max_pages) * p.P) {
            if (blockIdx.x == 0) flag_error(p.err, DA_DEVERR_SEQLENS);
            L = 0;
        }
        return L;
    }
    static __device__ __forceinline__ int count_stages(const Layout& s, const PagedParams& p, int b, int L) {
        L = checked_length(p, L);
        const int n = L == 0 ? 1 : (L + Sh::kKeys - 1) / Sh::kKeys;   // an empty sequence: one empty stage
        s.pad[b] = static_cast<uint8_t>(n * Sh::kKeys - L);
        return n;
    }

    // prefix[b]: stages before sequence b; prefix[B + 1]: the stages that every sequence has, or 0 where they
    // differ. Up to 32 sequences by the producer warp, which alone needs them, ...
    static __device__ __forceinline__ void count_units_warp(const Layout& s, const PagedParams& p) {
        const int lane = threadIdx.x & 31;
        const int n = lane < p.B ? count_stages(s, p, lane, ld_cg_s32(p.lens + lane)) : 0;
        int run = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, run, off);
            if (lane >= off) run += y;
        }
        const int first = __shfl_sync(0xffffffffu, n, 0);
        const bool same = __all_sync(0xffffffffu, lane >= p.B || n == first);
        if (lane < p.B) s.prefix[lane + 1] = run;
        if (lane == 0) {
            s.prefix[0] = 0;
            s.prefix[p.B + 1] = same ? first : 0;
        }
        __syncwarp();
    }
    // ... more by the whole CTA.
    static __device__ __forceinline__ void count_units(const Layout& s, const PagedParams& p) {
        constexpr int kThreads = Sh::kThreads;
        __shared__ int32_t warp_sum[kThreads / 32];
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        constexpr int kMost = (DA_MAX_PAGED_BATCH + kThreads - 1) / kThreads;
        const int per = (p.B + kThreads - 1) / kThreads, b0 = tid * per;
        int len[kMost], mine = 0;
        bool same = true;
        int first = ld_cg_s32(p.lens);
        if (per == 1) {
            if (tid < p.B) mine = len[0] = count_stages(s, p, tid, ld_cg_s32(p.lens + tid));
        } else {
#pragma unroll
            for (int i = 0; i < kMost; ++i) len[i] = i < per && b0 + i < p.B ? ld_cg_s32(p.lens + b0 + i) : 0;
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                if (i >= per || b0 + i >= p.B) break;
                len[i] = count_stages(s, p, b0 + i, len[i]);
                mine += len[i];
            }
        }
        first = checked_length(p, first);
        first = first == 0 ? 1 : (first + Sh::kKeys - 1) / Sh::kKeys;
        int run = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, run, off);
            if (lane >= off) run += y;
        }
        if (lane == 31) warp_sum[warp] = run;
        if (per == 1) {
            same = tid >= p.B || len[0] == first;
        } else {
#pragma unroll
            for (int i = 0; i < kMost; ++i) same = same && (i >= per || b0 + i >= p.B || len[i] == first);
        }
        same = __syncthreads_and(same);
        int sum = run - mine;
        for (int w = 0; w < warp; ++w) sum += warp_sum[w];
        if (per == 1) {
            if (tid < p.B) s.prefix[tid + 1] = sum + len[0];
        } else {
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                if (i >= per || b0 + i >= p.B) break;
                sum += len[i];
                s.prefix[b0 + i + 1] = sum;
            }
        }
        if (tid == 0) {
            s.prefix[0] = 0;
            s.prefix[p.B + 1] = same ? first : 0;
        }
        __syncthreads();
    }

    // Up to this many units a range has an SM to itself in a batch of unequal lengths, from there on as many run as
    // fit (200 sequences of 25 to 400 keys: 18.5 us with 8, 16.8 with 4).
    static constexpr int kShortRange = D == 128 ? 4 : 3;

    static __device__ __forceinline__ Ranges cut(const Layout& s, const PagedParams& p) {
        return Ranges(s.prefix[p.B], s.prefix[p.B + 1], p.slots, p.one, kShortRange, Sh::kLeast, !KV8 || NT == 1);
    }

    // ------------------------------------------------------------ producer
    struct Box {        // what a lane knows of its box: one page and head
        int page;
        float ks, vs;
    };

    // The block-table entry of this lane's box, and what follows from it: the entry's read is on its way while
    // other work is done.
    static __device__ __forceinline__ int box_entry(const PagedParams& p, const PagedItem& it, int box) {
        const int key = box * p.box_keys;
        if (static_cast<uint32_t>(key) >= static_cast<uint32_t>(it.nkeys)) return -1;   // (a product past 2^31 is none)
        return ld_cg_s32(p.table + static_cast<int64_t>(it.b) * p.table_stride + p.page(it.key0 + key));
    }
    static __device__ __forceinline__ Box box_of(const PagedParams& p, const PagedItem& it, int box, int entry) {
        Box x;
        x.page = p.num_pages;   // a bad page: a coordinate past the cache, which the copy fills with zeros
        x.ks = 0.f;
        x.vs = 0.f;
        if (static_cast<uint32_t>(box * p.box_keys) < static_cast<uint32_t>(it.nkeys)) {
            const bool good = entry >= 0 && entry < p.num_pages;
            if (good) x.page = entry;
            else flag_error(p.err, DA_DEVERR_PAGE);
            if constexpr (KV8) {
                if (good) {
                    const int64_t at = static_cast<int64_t>(entry) * p.Hkv + it.kvh;
                    x.ks = __ldcg(p.ks + at);
                    x.vs = __ldcg(p.vs + at);   // its logarithm waits until the copies are on their way
                }
            }
        }
        return x;
    }
    static __device__ __forceinline__ Box load_box(const PagedParams& p, const PagedItem& it, int box) {
        return box_of(p, it, box, box_entry(p, it, box));
    }

    // Copy one box of keys or values to `dst`.
    static __device__ __forceinline__ void copy_box(const PagedParams& p, uint32_t dst, const CUtensorMap* map, int c1, int c2,
                                                    uint32_t bar) {
        constexpr int kInner = Sh::kSliceRow / (KV8 ? 1 : 2);
#pragma unroll
        for (int hf = 0; hf < Sh::kSlices; ++hf) tma_load_3d(dst + hf * Sh::kSliceBytes, map, hf * kInner, c1, c2, bar);
    }

    static __device__ void producer(const Layout& s, const PagedParams& p, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                    const CUtensorMap* tmK16, const CUtensorMap* tmV16) {
        const int lane = threadIdx.x & 31;
        if (p.B <= 32) count_units_warp(s, p);
        const Ranges ranges = cut(s, p);
        const int shares = ranges.n * p.lanes;

        // cursor: where this CTA's next unit lies, and the units left of its share. Lane 0 looks up the share's
        // begin, lane 1 its end.
        const int share = static_cast<int>(blockIdx.x);
        const int range = share / p.lanes, sub = share - range * p.lanes;
        const int kvh = p.chunks == 1 ? sub : sub / p.chunks, chunk = sub - kvh * p.chunks;
        int b = 0, stage = 0, left = 0;
        if (share < shares) {
            const int r = range + (lane == 1 ? 1 : 0);
            const int u = min(ranges.raw(r), ranges.units - 1);
            int lo = 0, hi = p.B - 1;   // last b with prefix[b] <= u
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s.prefix[mid] <= u) lo = mid;
                else hi = mid - 1;
            }
            int at = u, st = u - s.prefix[lo];
            const int rest = s.prefix[lo + 1] - u;
            if (st <= ranges.slack) {          // a cut near a border moves there
                at -= st;
                st = 0;
            } else if (rest <= ranges.slack) {
                at += rest;
                st = 0;
                ++lo;
            }
            if (r >= ranges.n) at = ranges.units;
            b = __shfl_sync(0xffffffffu, lo, 0);
            stage = __shfl_sync(0xffffffffu, st, 0);
            left = __shfl_sync(0xffffffffu, at, 1) - __shfl_sync(0xffffffffu, at, 0);
        }
        // the next piece: valid 0 when this CTA has none left
        auto next_piece = [&](PagedItem& it) {
            it.valid = 0;
            if (left == 0) return;
            const int n = s.prefix[b + 1] - s.prefix[b];
            const int L = n * Sh::kKeys - s.pad[b];
            const int count = min(n - stage, left), last = stage + count;
            it.valid = 1;
            it.b = b;
            it.kvh = kvh;
            it.c0 = chunk * Sh::kCols;
            it.nh = min(Sh::kCols, p.G * p.tq - it.c0);
            it.key0 = stage * Sh::kKeys;
            it.nkeys = min(L, last * Sh::kKeys) - it.key0;
            it.ntiles = (it.nkeys + Sh::kKeys - 1) / Sh::kKeys;
            it.vis0 = L - p.tq + 1 - it.key0;
            it.part = -1;
            if (count < n) it.part = 2 * share + (stage == 0 ? 1 : 0);
            left -= count;
            stage = last;
            if (stage == n) {
                stage = 0;
                ++b;
            }
        };
        auto publish = [&](uint32_t i, const PagedItem& it) -> bool {
            const int slot = i % kItemSlots;
            if (!wait_warp(s.iempty0 + 8 * slot, ((i / kItemSlots) & 1) ^ 1, p.wait_limit_ns)) {
                if (lane == 0) flag_error(p.err, DA_DEVERR_TIMEOUT);
                return false;
            }
            const uint32_t bar = s.ifull0 + 8 * slot;
            if (lane == 0) {
                *slot_of(s, slot) = it;
                if (it.valid) mbar_arrive_expect_tx(bar, it.nh * D * 2);
                else mbar_arrive(bar);
            }
            __syncwarp();
            if (it.valid) {
                const uint32_t dst = s.qbuf + slot * Sh::kQBytes;
                const int64_t row = static_cast<int64_t>(it.b) * p.tq * p.Hq + it.kvh * p.G;
                if (p.tq == 1) {
                    if (lane == 0) bulk_load(dst, p.q + (row + it.c0) * D, it.nh * D * 2, bar);
                } else if (lane < it.nh) {
                    const int c = it.c0 + lane;
                    bulk_load(dst + lane * D * 2, p.q + (row + static_cast<int64_t>(c / p.G) * p.Hq + c % p.G) * D, D * 2, bar);
                }
            }
            return true;
        };

        PagedItem item;
        item.valid = 0;
        int st = 0;
        uint32_t ph = 0;
        const int per_stage = Sh::kKeys / p.box_keys;
        for (uint32_t i = 0;; ++i) {
            // the next piece's descriptor, queries and table entries go out before the last one's merge
            PagedItem next;
            next_piece(next);
            int entry = -1;
            if (next.valid) entry = box_entry(p, next, lane);
            if (!publish(i, next)) return;
            Box cur = {};
            if (next.valid) cur = box_of(p, next, lane, entry);
            if (item.valid) {
                // hand the consumers the next stage, empty, for that merge
                if (!wait_warp(s.empty0 + 8 * st, ph ^ 1, p.wait_limit_ns)) {
                    if (lane == 0) flag_error(p.err, DA_DEVERR_TIMEOUT);
                    return;
                }
                if (lane == 0) mbar_arrive(s.full0 + 8 * st);
                if (++st == Sh::kRing) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (!next.valid) return;
            item = next;
            Box ahead = load_box(p, item, 32 + lane);   // the next batch of boxes
            for (int t = 0; t < item.ntiles; ++t) {
                const int box0 = t * per_stage, in32 = box0 % 32;
                if (t > 0 && in32 == 0) {
                    cur = ahead;
                    ahead = load_box(p, item, box0 + 32 + lane);
                }
                if (!wait_warp(s.empty0 + 8 * st, ph ^ 1, p.wait_limit_ns)) {
                    if (lane == 0) flag_error(p.err, DA_DEVERR_TIMEOUT);
                    return;
                }
                // A full stage in boxes of box_keys keys, the ragged end of a sequence in 16-key boxes up to it:
                // lane l copies box l.
                const int keys = min(Sh::kKeys, item.nkeys - t * Sh::kKeys);
                const bool full = keys == Sh::kKeys;
                const int box = full ? p.box_keys : 16, boxes = full ? per_stage : (keys + 15) / 16;
                const uint32_t fb = s.full0 + 8 * st;
                if (lane == 0) mbar_expect_tx(fb, 2 * boxes * box * Sh::kRowBytes);
                __syncwarp();
                const int off = lane * box;
                const int page = __shfl_sync(0xffffffffu, cur.page, (in32 + off / p.box_keys) & 31);
                if (lane < boxes) {
                    const int pos = item.key0 + t * Sh::kKeys + off;
                    const int slot = pos - p.page(pos) * p.P;
                    const bool thd = p.layout == DA_LAYOUT_VARLEN;
                    const int c1 = thd ? item.kvh : slot, c2 = thd ? page * p.P + slot : page * p.Hkv + item.kvh;
                    const uint32_t dst = s.ring + st * Sh::kStageBytes + off * Sh::kSliceRow;
                    copy_box(p, dst, full ? tmK : tmK16, c1, c2, fb);
                    copy_box(p, dst + Sh::kTileBytes, full ? tmV : tmV16, c1, c2, fb);
                }
                if constexpr (KV8) {
                    // the scales of the stage's 16-key boxes
                    const int from = (in32 + lane * 16 / p.box_keys) & 31;
                    const float ks = __shfl_sync(0xffffffffu, cur.ks, from);
                    const float vs = __shfl_sync(0xffffffffu, cur.vs, from);
                    if (lane < Sh::kKeys / 16) s.scales[st * (Sh::kKeys / 16) + lane] = make_float2(ks, log2_of_scale(vs));
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(fb);
                if (++st == Sh::kRing) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (item.part >= 0) {
                // which ranges hold the other parts, for the consumers' end of the piece (they read it after the
                // hand-over above)
                int first, count;
                ranges.parts(s.prefix[item.b], s.prefix[item.b + 1], first, count);
                if (lane == 0) {
                    PagedItem* at = slot_of(s, i % kItemSlots);
                    at->first_share = first * p.lanes + sub;
                    at->nparts = count;
                }
            }
        }
    }

    // ------------------------------------------------------------ consumers
    static __device__ __forceinline__ uint32_t chunk_addr(uint32_t tile, int row, int chunk) {
        constexpr int kChunks = Sh::kSliceRow / 16;
        const int x = kChunks == 8 ? row & 7 : (row >> 1) & 3;   // the copy's 128- or 64-byte swizzle
        return tile + (chunk / kChunks) * Sh::kSliceBytes + row * Sh::kSliceRow + (((chunk % kChunks) ^ x) << 4);
    }

    // Query fragments (B operand, k16 x n8) of n-tile n, and the factor that takes a product to
    // the exp2 domain for this thread's two columns.
    static __device__ __forceinline__ void load_queries(const PagedParams& p, uint32_t qrows, int nh,
                                                        uint32_t (&qf)[D / 16][NT][2], float (&qs)[NT][2]) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool live = 8 * n + g < nh;
            const uint32_t row = qrows + (live ? 8 * n + g : 0) * D * 2;
            qs[n][0] = qs[n][1] = p.scale_log2;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t a0, a1;
                if constexpr (KV8) {
                    // dims 16 ks + 4 t4 .. + 3: where an e4m3 row's ldmatrix puts a lane's four bytes
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a0), "=r"(a1) : "r"(row + (ks * 16 + 4 * t4) * 2));
                } else {
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a0) : "r"(row + (ks * 16 + 2 * t4) * 2));
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a1) : "r"(row + (ks * 16 + 8 + 2 * t4) * 2));
                }
                qf[ks][n][0] = live ? a0 : 0u;
                qf[ks][n][1] = live ? a1 : 0u;
            }
            if constexpr (KV8 && DT == DA_BF16) {
                uint32_t top = 0;   // largest exponent field of the column
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        top = max(top, max((qf[ks][n][j] >> 7) & 0xffu, (qf[ks][n][j] >> 23) & 0xffu));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^e takes the largest element to [2^14, 2^15); an infinity or a NaN stays one
                const int field = top == 255 ? 127 : min(max(268 - static_cast<int>(top), 14), 240);
                const float up = __uint_as_float(static_cast<uint32_t>(field) << 23);
                const float down = __uint_as_float(static_cast<uint32_t>(254 - field) << 23);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        qf[ks][n][j] = pack2<DA_F16>(__uint_as_float(qf[ks][n][j] << 16) * up,
                                                     __uint_as_float(qf[ks][n][j] & 0xffff0000u) * up);
                qs[n][0] *= __shfl_sync(0xffffffffu, down, 8 * t4);       // column 2 t4 is row g = 2 t4 of the operand
                qs[n][1] *= __shfl_sync(0xffffffffu, down, 8 * t4 + 4);
            }
        }
    }

    // S^T[16 keys, 8 columns per n-tile] of box `row0`.
    static __device__ __forceinline__ void scores(uint32_t tile, int row0, const uint32_t (&qf)[D / 16][NT][2],
                                                  float (&x)[NT][4]) {
        const int lane = threadIdx.x & 31, mi = lane >> 3, r8 = lane & 7;
        const int row = row0 + (mi & 1) * 8 + r8;
        if constexpr (KV8) {
            // two chains where there is one n-tile (more give each box as many anyway)
            constexpr int kChains = NT == 1 ? 2 : 1;
            float y[NT][kChains][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < kChains; ++c) y[n][c][0] = y[n][c][1] = y[n][c][2] = y[n][c][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
                uint32_t w[4];   // rows lo / hi of 16 dims, then of the next 16
                ldsm_x4(chunk_addr(tile, row, 2 * kk + (mi >> 1)), w);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a[4];
                    e4m3x4_to_f16(w[2 * h], a[0], a[2]);
                    e4m3x4_to_f16(w[2 * h + 1], a[1], a[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_16816<DA_F16>(y[n][h % kChains], a, qf[2 * kk + h][n][0], qf[2 * kk + h][n][1]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[n][j] = kChains == 2 ? y[n][0][j] + y[n][kChains - 1][j] : y[n][0][j];
        } else {
            float y[NT][4];   // two independent chains
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[n][j] = y[n][j] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t a[4];
                ldsm_x4(chunk_addr(tile, row, 2 * ks + (mi >> 1)), a);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (ks & 1) mma_16816<DT>(y[n], a, qf[ks][n][0], qf[ks][n][1]);
                    else mma_16816<DT>(x[n], a, qf[ks][n][0], qf[ks][n][1]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[n][j] += y[n][j];
        }
    }

    // Weights to the type of their product. In 16-bit pages a weight enters as two terms, a 16-bit value and what it
    // leaves: off by 2^-15 of itself in bf16, in fp16 by 2^-21, or 2^-36 of the largest. One term, off by 2^-8 and 2^-11,
    // made the outputs' error 1.2 to 1.4 times that of float32 weights. The first is rounded down (in fp16 from 2^-20 of
    // the weight and the least fp16 below it) and the second (in bf16 of 2^-20 of the weight more) is above 0: an infinite
    // value stays one, as it meets no 0 and no other sign. The second products cost one token next to nothing
    // (16 x 131072 keys 1154 -> 1156 us, the ragged batch 86.7 both), 16 columns 1 to 7 % (16 x 8192 keys, four tokens, bf16
    // 81.9 -> 82.7 us; 64 ragged sequences, fp16 117.9 -> 125.6). 8-bit pages, bound by instructions, have one (fp16)
    // term: a second takes four tokens from 172.6 to 201.2 us and 16 x 32768 keys of head size 64 from 94.1 to 97.4.
    static constexpr int kTerms = KV8 ? 1 : 2;
    static __device__ __forceinline__ void weights16(float a, float b, uint32_t (&term)[kTerms]) {
        if constexpr (KV8) {
            term[0] = pack2<DA_F16>(a, b);
        } else if constexpr (DT == DA_F16) {
            constexpr float kLess = 1.f - 0x1p-20f, kLeast = 0x1p-24f;
            term[0] = pack2_down<DT>(fmaxf(fmaf(a, kLess, -kLeast), 0.f), fmaxf(fmaf(b, kLess, -kLeast), 0.f));
            term[1] = pack2<DT>(a - bits_to_f32<DT>(term[0] & 0xffffu), b - bits_to_f32<DT>(term[0] >> 16));
        } else {
            constexpr float kMore = 1.f + 0x1p-20f;
            term[0] = pack2_down<DT>(a, b);
            term[1] = pack2<DT>(fmaf(a, kMore, -bits_to_f32<DT>(term[0] & 0xffffu)), fmaf(b, kMore, -bits_to_f32<DT>(term[0] >> 16)));
        }
    }

    // O^T[D, 8 columns per n-tile] += V^T P^T of box `row0`; in 8-bit tiles rows g and g + 8 of
    // step i are dims 16 i + 2 g and 16 i + 2 g + 1, in 16-bit tiles 16 i + g and 16 i + g + 8.
    static __device__ __forceinline__ void weigh(uint32_t tile, int row0, const uint32_t (&pb)[kTerms][NT][2],
                                                 float (&acc)[D / 16][NT][4]) {
        const int lane = threadIdx.x & 31, mi = lane >> 3, r8 = lane & 7;
        if constexpr (KV8) {
            const int row = row0 + (mi & 1) * 8 + r8;
#pragma unroll
            for (int ii = 0; ii < D / 32; ++ii) {
                uint32_t w[4];   // keys lo / hi of 16 dims, then of the next 16: two keys x two dims each
                ldsm_x4_trans(chunk_addr(tile, row, 2 * ii + (mi >> 1)), w);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a[4];
                    e4m3x4_to_f16(__byte_perm(w[2 * h], 0, 0x3120), a[0], a[1]);
                    e4m3x4_to_f16(__byte_perm(w[2 * h + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_16816<DA_F16>(acc[2 * ii + h][n], a, pb[0][n][0], pb[0][n][1]);
                }
            }
        } else {
            const int row = row0 + (mi >> 1) * 8 + r8;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t a[4];
                ldsm_x4_trans(chunk_addr(tile, row, 2 * i + (mi & 1)), a);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < kTerms; ++k) mma_16816<DT>(acc[i][n], a, pb[k][n][0], pb[k][n][1]);
            }
        }
    }

    // A token does not see the keys of the tokens after it, and its weights for them are 0; but 0 * NaN and 0 * Inf
    // are not, so a value row of theirs that holds either must not enter the product. Such rows are rare: they are
    // looked for where a stage has keys that some column does not see (at most T_q - 1, at a sequence's end), taken
    // into the columns that see them one by one, and zeroed before the product. Rows are rows of the tile. (The search and
    // the registers of the rare case cost four tokens over e4m3 pages 1.5 %: 169.4 -> 171.9 us; one token nothing.)
    static __device__ __forceinline__ bool any_non_finite(uint32_t vtile, int from, int to) {
        constexpr int kPerRow = Sh::kRowBytes / 16;
        constexpr uint32_t kOnes = KV8 ? 0x7f7f7f7fu : DT == DA_BF16 ? 0x7f807f80u : 0x7c007c00u;
        uint32_t found = 0;
        for (int c = threadIdx.x & 31; c < (to - from) * kPerRow; c += 32) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(chunk_addr(vtile, from + c / kPerRow, c % kPerRow)));
#pragma unroll
            for (int i = 0; i < 4; ++i) found |= KV8 ? __vcmpeq4(w[i] & kOnes, kOnes) : __vcmpeq2(w[i] & kOnes, kOnes);
        }
        return __any_sync(0xffffffffu, found != 0);
    }
    static __device__ __forceinline__ void zero_rows(uint32_t vtile, int from, int to) {
        constexpr int kPerRow = Sh::kRowBytes / 16;
        for (int c = threadIdx.x & 31; c < (to - from) * kPerRow; c += 32)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                             chunk_addr(vtile, from + c / kPerRow, c % kPerRow)),
                         "r"(0u)
                         : "memory");
        __syncwarp();
    }
    // acc += w[n][c] v over the columns with sees[n][c], v the value row `row`.
    static __device__ __forceinline__ void weigh_row(uint32_t vtile, int row, const float (&w)[NT][2], const bool (&sees)[NT][2],
                                                     float (&acc)[D / 16][NT][4]) {
        const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            float v[2];   // of the dims that acc[i][n][0 .. 1] and acc[i][n][2 .. 3] hold
            uint16_t x, y;
            if constexpr (KV8) {
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(chunk_addr(vtile, row, i) + 2 * g));
                uint32_t h2;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(x));
                v[0] = bits_to_f32<DA_F16>(h2 & 0xffffu);
                v[1] = bits_to_f32<DA_F16>(h2 >> 16);
            } else {
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(chunk_addr(vtile, row, 2 * i) + 2 * g));
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(y) : "r"(chunk_addr(vtile, row, 2 * i + 1) + 2 * g));
                v[0] = bits_to_f32<DT>(x);
                v[1] = bits_to_f32<DT>(y);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (sees[n][c]) {
                        acc[i][n][c] = fmaf(w[n][c], v[0], acc[i][n][c]);
                        acc[i][n][c + 2] = fmaf(w[n][c], v[1], acc[i][n][c + 2]);
                    }
        }
    }

    static __device__ __forceinline__ int64_t output_row(const PagedParams& p, const PagedItem& it, int col) {
        const int c = it.c0 + col;
        return (static_cast<int64_t>(it.b) * p.tq + c / p.G) * p.Hq + it.kvh * p.G + c % p.G;
    }

    // Outputs are written by half a warp per column: the halves of warp w have columns w and w + 4 of an
    // n-tile. A lane has kVec times four dims, 64 v + 4 (lane % 16) on.
    static constexpr int kVec = D / 64;

    static __device__ __forceinline__ void scale4(float4& a, float by) {
        a.x *= by;
        a.y *= by;
        a.z *= by;
        a.w *= by;
    }
    static __device__ __forceinline__ void fma4(float4& a, float w, const float4& b) {
        a.x = fmaf(w, b.x, a.x);
        a.y = fmaf(w, b.y, a.y);
        a.z = fmaf(w, b.z, a.z);
        a.w = fmaf(w, b.w, a.w);
    }

    // One column whose sums o and l, relative to m, are complete: its output and its lse. One that saw no key has
    // output 0 and lse -inf. (NaN scores leave m alone and make l NaN.) l >= 1 otherwise (the key that set m weighs 1).
    static __device__ __forceinline__ void finish_column(const PagedParams& p, int64_t row, float4 (&o)[kVec], float m, float l) {
        const int l16 = threadIdx.x & 15;
        const bool none = m == kNoKey && l == 0.f;
        const float by = none ? 0.f : 1.f / l, lse2 = none ? -INFINITY : m + fast_log2(l);
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            scale4(o[v], by);
            *reinterpret_cast<uint2*>(p.out + row * D + 64 * v + 4 * l16) =
                make_uint2(pack2<DT>(o[v].x, o[v].y), pack2<DT>(o[v].z, o[v].w));
        }
        if (p.lse != nullptr && l16 == 0) p.lse[row] = lse2 * kLn2;
    }

    // Where part j of a (sequence, head)'s column lies, in units of columns: j = 0 is the part with the first
    // key, which its range left in its second place (a range's first place is for the end of a sequence).
    static __device__ __forceinline__ int64_t part_row(const PagedParams& p, int first_share, int j, int col) {
        return static_cast<int64_t>(j == 0 ? 2 * first_share + 1 : 2 * (first_share + j * p.lanes)) * Sh::kCols + col;
    }

    // Columns 8n .. 8n + 7 of a piece from the consumer warps' states. With `direct` the piece is the first of two
    // parts and the second one is written: they are merged here, in the order and with the roundings of merge_parts.
    static __device__ __forceinline__ void write_piece(const PagedParams& p, const PagedItem& it, const float* red_acc,
                                                       const float* red_m, int n, bool direct) {
        const float* red_dv = red_m + Sh::kWarps * 8;
        const float* red_l = red_dv + Sh::kWarps * 8;
        const int l16 = threadIdx.x & 15;
        const int hh = (threadIdx.x >> 5) + kWriters * ((threadIdx.x >> 4) & 1), col = 8 * n + hh;
        const bool live = col < it.nh;
        float2 sum1 = make_float2(kNoKey, 0.f);
        float4 o1[kVec];
        if (direct && live) {
            const int64_t at = part_row(p, it.first_share, 1, col);
            sum1 = __ldcg(p.part_sum + at);
#pragma unroll
            for (int v = 0; v < kVec; ++v)
                o1[v] = __ldcg(reinterpret_cast<const float4*>(p.part + at * D + 64 * v + 4 * l16));
        }
        float M = kNoKey, dV = kNoKey;
#pragma unroll
        for (int w = 0; w < Sh::kWarps; ++w) M = fmaxf(M, red_m[w * 8 + hh]);
        if constexpr (KV8) {
#pragma unroll
            for (int w = 0; w < Sh::kWarps; ++w) dV = fmaxf(dV, (red_m[w * 8 + hh] - M) + red_dv[w * 8 + hh]);
        }
        float4 o[kVec];
#pragma unroll
        for (int v = 0; v < kVec; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < Sh::kWarps; ++w) {
            const float wl = fast_exp2(red_m[w * 8 + hh] - M);
            const float wt = KV8 ? fast_exp2((red_m[w * 8 + hh] - M) + (red_dv[w * 8 + hh] - dV)) : wl * (1.f / kLiftBy);
            l = fmaf(wl, red_l[w * 8 + hh], l);
            const float* row = red_acc + (w * 8 + hh) * Sh::kMergeRow + Sh::merge_dim(4 * l16, hh);
#pragma unroll
            for (int v = 0; v < kVec; ++v) fma4(o[v], wt, *reinterpret_cast<const float4*>(row + 64 * v));
        }
        if (!live) return;
        if constexpr (KV8) {   // o is relative to M + dV, l to M: in two steps, which stay normal floats for every scale
            const float by = fast_exp2(0.5f * dV);
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                scale4(o[v], by);
                scale4(o[v], by);
            }
        }
        if (direct) {
            const float m = fmaxf(M, sum1.x), w0 = fast_exp2(M - m), w1 = fast_exp2(sum1.x - m);
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);   // (merge_parts' first term: a product of -0 becomes +0)
                fma4(sum, w0, o[v]);
                fma4(sum, w1, o1[v]);
                o[v] = sum;
            }
            l = __fadd_rn(__fmul_rn(w0, l), __fmul_rn(w1, sum1.y));
            M = m;
        }
        if (it.part < 0 || direct) {
            finish_column(p, output_row(p, it, col), o, M, l);
        } else {
            const int64_t at = static_cast<int64_t>(it.part) * Sh::kCols + col;
#pragma unroll
            for (int v = 0; v < kVec; ++v) *reinterpret_cast<float4*>(p.part + at * D + 64 * v + 4 * l16) = o[v];
            if (l16 == 0) p.part_sum[at] = make_float2(M, l);
        }
    }

    // Merge this warp's columns of a (sequence, head) whose partials are all written. Lane j of a half warp
    // takes part j's maximum, sum and weight, so that every load is issued before any of them is needed; the order
    // of the sums is that of the parts.
    static __device__ __forceinline__ void merge_parts(const PagedParams& p, const PagedItem& it) {
        constexpr int kAhead = NT == 1 ? 16 / kVec : 4 / kVec;   // parts in flight
        const int l16 = threadIdx.x & 15, nparts = it.nparts, nh = it.nh, first_share = it.first_share;
#pragma unroll 1
        for (int c0 = threadIdx.x >> 5; c0 < nh; c0 += 2 * kWriters) {
            const int c = c0 + kWriters * ((threadIdx.x >> 4) & 1);
            const bool live = c < nh;
            float m = kNoKey, z = 0.f;
            float4 acc[kVec];
#pragma unroll
            for (int v = 0; v < kVec; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int j0 = 0; j0 < nparts; j0 += 16) {
                const int count = live ? min(16, nparts - j0) : 0;
                const float2 part = l16 < count ? __ldcg(p.part_sum + part_row(p, first_share, j0 + l16, c))
                                                : make_float2(kNoKey, 0.f);
                float w = 0.f;
#pragma unroll 1
                for (int j = 0; j < min(16, nparts - j0); j += kAhead) {
                    float4 o[kAhead][kVec];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        const float* at = p.part + part_row(p, first_share, j0 + j + i, c) * D + 4 * l16;
#pragma unroll
                        for (int v = 0; v < kVec; ++v)
                            o[i][v] = j + i < count ? __ldcg(reinterpret_cast<const float4*>(at + 64 * v))
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                    if (j == 0) {
                        float top = part.x;
#pragma unroll
                        for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                        const float mn = fmaxf(m, top);       // stays kNoKey while no part has seen a key
                        w = fast_exp2(part.x - mn);
                        float sum = __fmul_rn(w, part.y);
#pragma unroll
                        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                        const float al = fast_exp2(m - mn);
                        m = mn;
                        z = fmaf(z, al, sum);
#pragma unroll
                        for (int v = 0; v < kVec; ++v) scale4(acc[v], al);
                    }
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        const float wi = __shfl_sync(0xffffffffu, w, (j + i) & 15, 16);
#pragma unroll
                        for (int v = 0; v < kVec; ++v) fma4(acc[v], wi, o[i][v]);
                    }
                }
            }
            if (live) finish_column(p, output_row(p, it, c), acc, m, z);
        }
    }

    static __device__ void consumer(const Layout& s, const PagedParams& p) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
        constexpr int kRows = 16 * Sh::kBoxes;   // keys of a stage that are this warp's
        bool ok = true;
        uint32_t bad_bar = 0, bad_ph = 0;
        int st = 0;
        uint32_t ph = 0, mz = 0, md = 0;
        int merges = 0;
        for (uint32_t i = 0;; ++i) {
            const int slot = i % kItemSlots;
            if (!wait_warp(s.ifull0 + 8 * slot, (i / kItemSlots) & 1, p.wait_limit_ns)) {
                if (lane == 0) flag_error(p.err, DA_DEVERR_TIMEOUT);
                ok = false;
                break;
            }
            // stays in shared memory (the slot is handed back at the piece's end): the loop below needs
            // every register
            const PagedItem& item = *slot_of(s, slot);
            if (!item.valid) break;
            uint32_t qf[D / 16][NT][2];
            float qs[NT][2];
            load_queries(p, s.qbuf + slot * Sh::kQBytes, item.nh, qf, qs);
            const int nkeys = item.nkeys, ntiles = item.ntiles;
            const int hide = item.vis0 - warp * kRows;   // this warp's first row that token 0 does not see, from the first
                                                         // stage on (with one token: past the last)

            int vis[NT][2];   // keys of the piece that this thread's columns may see
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    vis[n][c] = nkeys;
                    if (p.tq > 1) vis[n][c] = min(nkeys, item.vis0 + (item.c0 + 8 * n + 2 * t4 + c) / p.G);
                }
            float acc[D / 16][NT][4];
#pragma unroll
            for (int a = 0; a < D / 16; ++a)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[a][n][0] = acc[a][n][1] = acc[a][n][2] = acc[a][n][3] = 0.f;
            // running maximum of the scores, (8-bit) how far that of the weights is above it, less kLift, this thread's
            // share of the sum
            float m[NT][2], dv[NT][2], l[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    m[n][c] = kNoKey;
                    dv[n][c] = KV8 ? -kLift : 0.f;
                    l[n][c] = 0.f;
                }

            for (int t = 0; t < ntiles; ++t) {
                const uint32_t fb = s.full0 + 8 * st;
                if (ok && !wait_warp(fb, ph, p.wait_limit_ns)) {
                    ok = false;
                    bad_bar = fb;
                    bad_ph = ph;
                    if (lane == 0) flag_error(p.err, DA_DEVERR_TIMEOUT);
                }
                const int keys = min(Sh::kKeys, nkeys - t * Sh::kKeys);
                const int valid = keys - warp * kRows;
                bool zeroed = false;
                if (ok && valid > 0) {
                    const uint32_t ktile = s.ring + st * Sh::kStageBytes;
                    const uint32_t vtile = ktile + Sh::kTileBytes;
                    if (valid < kRows) {
                        // rows past the end hold anything: their weight is 0, but 0 * NaN is not
                        zero_rows(vtile, warp * kRows + valid, (warp + 1) * kRows);
                        zeroed = true;
                    }
                    float x[Sh::kBoxes][NT][4], lv[Sh::kBoxes];
                    bool move = false;
#pragma unroll
                    for (int bx = 0; bx < Sh::kBoxes; ++bx) {
                        scores(ktile, warp * kRows + bx * 16, qf, x[bx]);
                        float ks = 1.f;
                        lv[bx] = 0.f;
                        if constexpr (KV8) {
                            const float2 f = s.scales[st * (Sh::kKeys / 16) + warp * Sh::kBoxes + bx];
                            ks = f.x;
                            lv[bx] = f.y;
                        }
                        const int key = t * Sh::kKeys + warp * kRows + bx * 16 + g;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float f = KV8 ? qs[n][j & 1] * ks : qs[n][j & 1];
                                const bool seen = key + 8 * (j >> 1) < vis[n][j & 1];
                                x[bx][n][j] = seen ? x[bx][n][j] * f : -INFINITY;
                                const float above = KV8 ? fmaxf(lv[bx] - dv[n][j & 1], kLift) : kLift;
                                move = move || x[bx][n][j] - m[n][j & 1] > kHeadroom + kLift - above;
                            }
                    }
                    // The reference of a column moves only when a score passes it by more than
                    // kHeadroom, so the shuffles and the rescale run on a few stages per piece.
                    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                float top = m[n][c];
#pragma unroll
                                for (int bx = 0; bx < Sh::kBoxes; ++bx)
                                    top = fmaxf(top, fmaxf(x[bx][n][c], x[bx][n][c + 2]));
#pragma unroll
                                for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                                const float al = fast_exp2(m[n][c] - top);
                                float av = al;
                                if constexpr (KV8) {
                                    float dnew = fmaxf(kNoKey, (m[n][c] - top) + dv[n][c]);
#pragma unroll
                                    for (int bx = 0; bx < Sh::kBoxes; ++bx)
                                        dnew = fmaxf(dnew, (fmaxf(x[bx][n][c], x[bx][n][c + 2]) - top) + (lv[bx] - kLift));
#pragma unroll
                                    for (int off = 4; off < 32; off <<= 1)
                                        dnew = fmaxf(dnew, __shfl_xor_sync(0xffffffffu, dnew, off));
                                    av = fast_exp2((m[n][c] - top) + (dv[n][c] - dnew));
                                    dv[n][c] = dnew;
                                }
                                m[n][c] = top;
                                l[n][c] *= al;
#pragma unroll
                                for (int a = 0; a < D / 16; ++a) {
                                    acc[a][n][c] *= av;
                                    acc[a][n][c + 2] *= av;
                                }
                            }
                    }
                    const int hidden = max(hide - t * Sh::kKeys, 0), rows = min(valid, kRows);
                    if (hidden < rows && any_non_finite(vtile, warp * kRows + hidden, warp * kRows + rows)) {
#pragma unroll 1
                        for (int r = hidden; r < rows; ++r) {
                            float w[NT][2], lr = lv[0];
                            bool sees[NT][2];
                            if constexpr (Sh::kBoxes == 2) lr = r < 16 ? lv[0] : lv[Sh::kBoxes - 1];
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    float score = x[0][n][c];
#pragma unroll
                                    for (int k = 1; k < 2 * Sh::kBoxes; ++k)
                                        score = select(r >> 3 == k, x[k >> 1][n][2 * (k & 1) + c], score);
                                    const float d = __shfl_sync(0xffffffffu, score, 4 * (r & 7) + t4) - m[n][c];
                                    w[n][c] = fast_exp2(KV8 ? d + (lr - dv[n][c]) : d) * kLiftBy;
                                    sees[n][c] = t * Sh::kKeys + warp * kRows + r < vis[n][c];
                                }
                            weigh_row(vtile, warp * kRows + r, w, sees, acc);
                        }
                        __syncwarp();
                        zero_rows(vtile, warp * kRows + hidden, warp * kRows + rows);
                        zeroed = true;
                    }
#pragma unroll
                    for (int bx = 0; bx < Sh::kBoxes; ++bx) {
                        uint32_t pb[kTerms][NT][2];
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float d = x[bx][n][j] - m[n][j & 1];
                                w[j] = fast_exp2(d);
                                l[n][j & 1] += w[j];
                                if constexpr (KV8) w[j] = fast_exp2(d + (lv[bx] - dv[n][j & 1]));
                                else w[j] *= kLiftBy;
                            }
                            uint32_t lo[kTerms], hi[kTerms];
                            weights16(w[0], w[1], lo);
                            weights16(w[2], w[3], hi);
#pragma unroll
                            for (int k = 0; k < kTerms; ++k) {
                                pb[k][n][0] = movmatrix_trans(lo[k]);
                                pb[k][n][1] = movmatrix_trans(hi[k]);
                            }
                        }
                        weigh(vtile, warp * kRows + bx * 16, pb, acc);
                    }
                }
                // order the generic-proxy stores above before the copy that refills the stage
                if (zeroed) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(s.empty0 + 8 * st);
                if (++st == Sh::kRing) {
                    st = 0;
                    ph ^= 1;
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], off);

            // ---- merge the consumer warps in the stage that the producer handed over, 8 columns a round
            if (ok && !wait_warp(s.full0 + 8 * st, ph, p.wait_limit_ns)) {
                ok = false;
                if (lane == 0) flag_error(p.err, DA_DEVERR_TIMEOUT);
            }
            // A range ends with the beginning of a sequence, whose end the next range began with: where that is
            // all of it, it is written by now, and this piece needs no partial result of its own (8-column
            // kernels: the others have no registers for it).
            uint32_t* count = p.arrived + item.first_share * kWriters + warp;   // (a writer's)
            const bool writer = Sh::kWarps == kWriters || warp < kWriters;
            const bool two = NT == 1 && writer && item.part >= 0 && (item.part & 1) != 0 && item.nparts == 2;
            uint32_t arrived = 0;
            if (two && lane == 0) arrived = ld_acquire(count);
            float* red = reinterpret_cast<float*>(s.smem + st * Sh::kStageBytes);
            bool direct = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n > 0) {
                    // every warp has read the previous round's rows
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s.mdone);
                    if (ok && !wait_warp(s.mdone, md & 1, p.wait_limit_ns)) {
                        ok = false;
                        if (lane == 0) flag_error(p.err, DA_DEVERR_TIMEOUT);
                    }
                    ++md;
                }
                // in turn: a warp may be a round ahead of one that still reads the last
                float* red_m = reinterpret_cast<float*>(s.smem + Sh::kRedOff) + (mz & 1) * Sh::kRedFloats;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = warp * 8 + 2 * t4 + c;
                    if (g == 0) {
                        red_m[col] = m[n][c];
                        red_m[Sh::kWarps * 8 + col] = dv[n][c];
                        red_m[2 * Sh::kWarps * 8 + col] = l[n][c];
                    }
                    float* row = red + col * Sh::kMergeRow;
#pragma unroll
                    for (int a = 0; a < D / 16; ++a) {
                        if constexpr (KV8) {
                            *reinterpret_cast<float2*>(row + Sh::merge_dim(a * 16 + 2 * g, col)) = make_float2(acc[a][n][c], acc[a][n][c + 2]);
                        } else {
                            row[Sh::merge_dim(a * 16 + g, col)] = acc[a][n][c];
                            row[Sh::merge_dim(a * 16 + g + 8, col)] = acc[a][n][c + 2];
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(s.mfull);
                if (ok && !wait_warp(s.mfull, mz & 1, p.wait_limit_ns)) {
                    ok = false;
                    if (lane == 0) flag_error(p.err, DA_DEVERR_TIMEOUT);
                }
                ++mz;
                if (NT == 1) {
                    direct = __shfl_sync(0xffffffffu, arrived, 0) == 1;
                    __syncwarp();
                }
                if (ok && writer) write_piece(p, item, red, red_m, n, direct);
            }
            // release the stage: order these generic-proxy stores before the copy that refills it
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(s.empty0 + 8 * st);
            if (++st == Sh::kRing) {
                st = 0;
                ph ^= 1;
            }
            if (!ok) break;
            if (direct) {
                if (lane == 0) *count = 0;
            } else if (writer && item.part >= 0) {
                // Warp w wrote the same columns of every partial, so the writers count apart: the
                // one whose arrival completes the count merges its columns, and sets the count back.
                uint32_t n = 0;
                __syncwarp();
                if (lane == 0) {
                    fence_acq_rel();
                    n = atomicAdd(count, 1u) + 1;
                    if (n == static_cast<uint32_t>(item.nparts)) {
                        atomicExch(count, 0u);
                        fence_acq_rel();
                    }
                }
                n = __shfl_sync(0xffffffffu, n, 0);
                // The merge waits for the end of the range (at most its first and last piece need one): it
                // then has the registers of the loop above to itself.
                if (n == static_cast<uint32_t>(item.nparts)) {
                    if (lane == 0) *last_of(s, warp, merges) = item;
                    ++merges;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(s.iempty0 + 8 * slot);
        }
        __syncwarp();
        for (int i = 0; i < merges; ++i) merge_parts(p, *last_of(s, warp, i));
        // after a timed-out wait, a copy still in flight into this CTA's shared memory gets one more
        // bounded wait before the CTA exits
        if (!ok && bad_bar != 0) wait_lane(bad_bar, bad_ph, p.wait_limit_ns);
    }
};

template <int D, int DT, bool KV8, int NT, int NW>
__global__ void __launch_bounds__(PagedShape<D, KV8, NT, NW>::kThreads, NW == 8 ? 1 : 2)
paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
             const __grid_constant__ CUtensorMap tmK16, const __grid_constant__ CUtensorMap tmV16, const PagedParams p) {
    using K = PagedKernel<D, DT, KV8, NT, NW>;
    using Sh = typename K::Sh;
    extern __shared__ uint8_t smem_raw[];
    const auto s = K::layout(smem_raw, p);
    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kRing; ++i) {
            mbar_init(s.full0 + 8 * i, 1);
            mbar_init(s.empty0 + 8 * i, Sh::kWarps);
        }
        for (int i = 0; i < kItemSlots; ++i) {
            mbar_init(s.ifull0 + 8 * i, 1);
            mbar_init(s.iempty0 + 8 * i, Sh::kWarps);
        }
        mbar_init(s.mfull, Sh::kWarps);
        mbar_init(s.mdone, Sh::kWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
        prefetch_tensormap(&tmK16);
        prefetch_tensormap(&tmV16);
    }
    __syncthreads();
    // From here on this grid touches global memory: wait for the previous kernel.
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_dependents_launch();
    if (p.B > 32) K::count_units(s, p);
    if ((threadIdx.x >> 5) == Sh::kWarps) K::producer(s, p, &tmK, &tmV, &tmK16, &tmV16);
    else K::consumer(s, p);
}

// ------------------------------------------------------------ host side
inline int gcd_of(int a, int b) {
    while (b) {
        const int r = a % b;
        a = b;
        b = r;
    }
    return a;
}

// Tensor map of a cache's keys or values: boxes of `rows` tokens of one head, slices of `inner` elements.
inline bool make_page_map(CUtensorMap* map, const void* base, const da_paged_cache& c, int inner, int rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t size = c.kv_dtype == DA_E4M3 ? 1 : 2;
    cuuint64_t dims[3], strides[2];
    cuuint32_t box[3], step[3] = {1, 1, 1};
    dims[0] = c.D;
    strides[0] = c.D * size;
    box[0] = inner;
    if (c.layout == DA_LAYOUT_VARLEN) {
        dims[1] = c.Hkv;
        dims[2] = static_cast<cuuint64_t>(c.num_pages) * c.page_size;
        strides[1] = static_cast<cuuint64_t>(c.Hkv) * c.D * size;
        box[1] = 1;
        box[2] = rows;
    } else {
        dims[1] = c.page_size;
        dims[2] = static_cast<cuuint64_t>(c.num_pages) * c.Hkv;
        strides[1] = static_cast<cuuint64_t>(c.page_size) * c.D * size;
        box[1] = rows;
        box[2] = 1;
    }
    const CUtensorMapDataType type = c.kv_dtype == DA_E4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : c.kv_dtype == DA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return fn(map, type, 3, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              inner * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device (152 if it cannot be queried).
inline int device_sms() {
    static std::atomic<int> known[64] = {};
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    sms = known[dev].load(std::memory_order_relaxed);
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 152;
        known[dev].store(sms, std::memory_order_relaxed);
    }
    return sms;
}

template <int D, int DT, bool KV8, int NT, int NW>
da_status launch_paged(const da_paged_cache& c, PagedParams& p, cudaStream_t stream) {
    using Sh = PagedShape<D, KV8, NT, NW>;
    constexpr int kInner = Sh::kSliceRow / (KV8 ? 1 : 2);
    p.chunks = (p.G * p.tq + Sh::kCols - 1) / Sh::kCols;
    p.box_keys = gcd_of(c.page_size, Sh::kKeys);
    CUtensorMap mk, mv, mk16, mv16;
    if (!make_page_map(&mk, c.k, c, kInner, p.box_keys) || !make_page_map(&mv, c.v, c, kInner, p.box_keys) ||
        !make_page_map(&mk16, c.k, c, kInner, 16) || !make_page_map(&mv16, c.v, c, kInner, 16))
        return DA_ERR_CUDA;
    // units of the largest batch that the table can describe
    const int64_t stages = (static_cast<int64_t>(p.max_pages) * p.P + Sh::kKeys - 1) / Sh::kKeys;
    const int64_t units = static_cast<int64_t>(p.B) * stages, lanes = static_cast<int64_t>(p.Hkv) * p.chunks;
    if (units > 0x3fff0000ll || lanes > 0x1000000ll) return DA_ERR_INVALID_ARG;
    auto kern = paged_kernel<D, DT, KV8, NT, NW>;
    static DeviceCache cache;
    int resident = 0;
    if (persistent_grid(kern, Sh::kThreads, Sh::smem_bytes(DA_MAX_PAGED_BATCH), cache, &resident) != cudaSuccess)
        return DA_ERR_CUDA;
    p.lanes = static_cast<int>(lanes);
    p.slots = std::max(1, std::min(resident, kPagedShares) / p.lanes);
    p.one = std::max(1, device_sms() / p.lanes);
    // A table whose rows hold few keys gets one CTA per SM (idle ones beside it cost a short call 1.7 us of 12).
    if (units <= static_cast<int64_t>(p.one) * kFewUnits) p.slots = p.one;
    // CTAs for the most ranges that the kernel can make of these units (see Ranges)
    const int64_t most = std::min<int64_t>(p.slots, (units + Sh::kLeast - 1) / Sh::kLeast);
    const int grid = static_cast<int>(most) * p.lanes;
    cudaLaunchAttribute attrs[1] = {pdl_attr()};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(Sh::kThreads);
    cfg.dynamicSmemBytes = Sh::smem_bytes(p.B);
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, mk, mv, mk16, mv16, p) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

template <int D, int DT, bool KV8, int NT>
da_status launch_paged_warps(const da_paged_cache& c, PagedParams& p, cudaStream_t s) {
    if constexpr (D == 128 && !KV8) {
        if (static_cast<int64_t>(p.max_pages) * p.P > kShortCapacity) return launch_paged<D, DT, KV8, NT, 8>(c, p, s);
    }
    return launch_paged<D, DT, KV8, NT, 4>(c, p, s);
}

template <int D, int DT>
da_status launch_paged_any(const da_paged_cache& c, PagedParams& p, cudaStream_t s) {
    const bool wide = item_cols(static_cast<int64_t>(p.G) * p.tq) > kHeadsPerCta;
    if (c.kv_dtype == DA_E4M3)
        return wide ? launch_paged_warps<D, DT, true, 2>(c, p, s) : launch_paged_warps<D, DT, true, 1>(c, p, s);
    return wide ? launch_paged_warps<D, DT, false, 2>(c, p, s) : launch_paged_warps<D, DT, false, 1>(c, p, s);
}

}  // namespace da_impl

using namespace da_impl;

extern "C" {

size_t decode_attn_paged_workspace_size(int T_q, int Hq, int Hkv, int D) {
    if (T_q < 1 || T_q > DA_MAX_QUERY_TOKENS || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
    const int cols = item_cols(static_cast<int64_t>(Hq / Hkv) * T_q);
    return kPagedHeaderBytes + kPagedCounterBytes + static_cast<size_t>(2 * kPagedShares) * cols * (D + 2) * 4;
}

da_status decode_attn_paged_workspace_init(void* workspace, size_t workspace_bytes, void* stream) {
    const size_t head = kPagedHeaderBytes + kPagedCounterBytes;
    if (!workspace || workspace_bytes < head) return DA_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return DA_ERR_ALIGNMENT;
    return cudaMemsetAsync(workspace, 0, head, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

da_status decode_attn_paged(const da_paged_attn* args, void* stream) {
    if (!args) return DA_ERR_INVALID_ARG;
    const da_paged_attn& a = *args;
    da_status st = check_cache(a.cache, a.dtype, a.kv_lens, a.block_table, a.max_pages, a.table_stride, a.B, a.Hq);
    if (st != DA_OK) return st;
    const da_paged_cache& c = *a.cache;
    if (a.Hq < 1 || a.T_q < 1 || a.T_q > DA_MAX_QUERY_TOKENS || !std::isfinite(a.scale)) return DA_ERR_INVALID_ARG;
    if (!a.q || !a.out || !a.workspace) return DA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(a.B) * a.T_q * a.Hq * c.D > 0x7fffffffll) return DA_ERR_INVALID_ARG;
    if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.lse, 4) || !aligned(a.workspace, 256)) return DA_ERR_ALIGNMENT;
    if (a.workspace_bytes < decode_attn_paged_workspace_size(a.T_q, a.Hq, c.Hkv, c.D)) return DA_ERR_WORKSPACE_TOO_SMALL;
    PagedParams p;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    p.q = static_cast<const uint16_t*>(a.q);
    p.ks = c.k_scale;
    p.vs = c.v_scale;
    p.lens = a.kv_lens;
    p.table = a.block_table;
    p.out = static_cast<uint16_t*>(a.out);
    p.lse = a.lse;
    p.err = reinterpret_cast<uint32_t*>(ws);
    p.arrived = reinterpret_cast<uint32_t*>(ws + kPagedHeaderBytes);
    p.G = a.Hq / c.Hkv;
    const int cols = item_cols(static_cast<int64_t>(p.G) * a.T_q);
    p.part = reinterpret_cast<float*>(ws + kPagedHeaderBytes + kPagedCounterBytes);
    p.part_sum = reinterpret_cast<float2*>(p.part + static_cast<size_t>(2 * kPagedShares) * cols * c.D);
    p.B = a.B;
    p.tq = a.T_q;
    p.Hq = a.Hq;
    p.Hkv = c.Hkv;
    p.P = c.page_size;
    // floor(pos / P) = pos * ceil(2^(31 + l) / P) >> (31 + l) for every pos < 2^31, with 2^l >= P > 2^(l - 1)
    int l = 0;
    while ((1 << l) < p.P) ++l;
    p.page_shift = 31 + l;
    p.page_mul = static_cast<uint32_t>(((1ull << p.page_shift) + p.P - 1) / p.P);
    p.max_pages = a.max_pages;
    p.table_stride = a.table_stride;
    p.num_pages = c.num_pages;
    p.layout = c.layout;
    p.scale_log2 = a.scale * kLog2e;
    p.wait_limit_ns = kWaitLimitNs;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (c.D == 128) return a.dtype == DA_F16 ? launch_paged_any<128, DA_F16>(c, p, s) : launch_paged_any<128, DA_BF16>(c, p, s);
    return a.dtype == DA_F16 ? launch_paged_any<64, DA_F16>(c, p, s) : launch_paged_any<64, DA_BF16>(c, p, s);
}

}  // extern "C"
