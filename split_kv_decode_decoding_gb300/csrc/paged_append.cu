// Append to a paged KV cache (decode_attn_paged.h): rotate new queries and keys by their
// positions, write keys and values into their pages, in 16 bits or as e4m3 with one scale
// per page and KV head.
//
// The mathematics. A pair (x, y) of a query or key at position p turns into
// (x c - y s, y c + x s); products and sum are each rounded to float32 (no fused
// multiply-add), so the result is the one that a step-by-step float32 evaluation gives, bit
// for bit, and an 8-bit code never depends on how the compiler contracted the expression.
// 8-bit pages: s = 2^e with the least e for which amax <= 448 * 2^e, over the new tokens of
// the page and head. With amax = m * 2^x, 1 <= m < 2, and 448 = 1.75 * 2^8, that is
// e = x - 8 for m <= 1.75, else x - 7: read off the bits of amax, no logarithm.
//
// What bounds it: bytes for prompts (each element read and written once), latency for a
// decode step (a chain of dependent reads: cu_new and kv_lens, block table, scale, then the
// stores).
//
// Threads: one thread owns 16 elements of one head's row, the two 16-byte chunks whose
// elements pair up (dims [8u, 8u + 8) and [rot/2 + 8u, ...) for the half rotation, 16
// consecutive dims for the interleaved one), so a rotation needs no exchange, loads and
// stores are 16 bytes wide, and a row may be rotated in place. The rotation runs on pairs of
// float32, two at a time. Instructions count here: with the rotation style as a run-time
// choice inside the loops, or a division's slow path beside every product, the same kernels
// took 20 to 60 % longer.
//
// Measured (one GB300): 16-bit pages, 9887 tokens of 32 + 2 x 8 heads in 5 prompts 39.3 us,
// 6.3 TB/s; 64 tokens, one per sequence, 28 + 2 x 4 heads 2.8 us. e4m3 pages: the same prompts 40.8 us,
// 5.5 TB/s (bound by the latency of a page's two passes and by instructions, not by its bytes); 256 tokens,
// one per sequence, 16 + 2 x 2 heads 4.1 us.

#include "paged_common.cuh"

namespace da_impl {

constexpr int kAppendThreads = 256;

struct AppendParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    uint64_t minus_zero;     // two float32 -0 (see mul2)
    const float* cos_sin;
    const int32_t* cu;       // [B + 1]
    const int32_t* lens;     // [B]
    const int32_t* table;    // [B][table_stride]
    uint16_t* q_out;
    uint8_t* kc;
    uint8_t* vc;
    float* ks;
    float* vs;
    uint32_t* err;
    int B, T, Hq, Hkv, P, max_pages, table_stride, num_pages, layout;
    int max_pos, rot, rope;
    int head_lanes;          // rows: threads that share a token's heads (per unit)
    int page_blocks;         // 8-bit pages: blocks for pages, before the ones for rows
};

// New tokens of sequence b: rows first .. first + n - 1 at positions start ...; n = 0 for a
// sequence that cannot be appended to.
struct NewTokens {
    int first, n, start;
    bool bad;
};

__device__ __forceinline__ NewTokens new_tokens(const AppendParams& p, int c0, int c1, int len) {
    NewTokens t;
    const int64_t n = static_cast<int64_t>(c1) - c0;
    t.bad = c0 < 0 || n < 0 || c1 > p.T || len < n || len > static_cast<int64_t>(p.max_pages) * p.P;
    t.first = c0;
    t.n = t.bad ? 0 : static_cast<int>(n);
    t.start = t.bad ? 0 : len - static_cast<int>(n);
    return t;
}

// Two float32 at once: products and sums are rounded one by one, as the scalar instructions do.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    return static_cast<uint64_t>(__float_as_uint(x)) | (static_cast<uint64_t>(__float_as_uint(y)) << 32);
}
// (The product as a fused multiply-add of -0, which rounds the same. The compiler turns a paired product
// and a paired sum into one rounding, and sees through a -0 that it knows, so this one comes with the
// call's parameters. Seen in 16 of 1.5 million bf16 results.)
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b, uint64_t minus_zero) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(minus_zero));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float lo2(uint64_t a) { return __uint_as_float(static_cast<uint32_t>(a)); }
__device__ __forceinline__ float hi2(uint64_t a) { return __uint_as_float(static_cast<uint32_t>(a >> 32)); }

// The 16 elements of one thread in float32, as eight rotation pairs (x, y): two pairs per step.
struct Chunk16 {
    uint64_t x[4], y[4];
};

// Elements of the two 16-byte chunks: with the half rotation x are a's and y are b's, with the
// interleaved one x are the even and y the odd elements of a, then of b.
template <int DT, bool HALF>
__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, Chunk16& e) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = bits_to_f32<DT>(w[i] & 0xffffu);
        hi[i] = bits_to_f32<DT>(w[i] >> 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        e.x[i] = HALF ? pair(lo[i], hi[i]) : pair(lo[2 * i], lo[2 * i + 1]);
        e.y[i] = HALF ? pair(lo[4 + i], hi[4 + i]) : pair(hi[2 * i], hi[2 * i + 1]);
    }
}

// Element j (0 .. 7) of chunk a (or b) of e.
template <bool HALF>
__device__ __forceinline__ float element(const Chunk16& e, bool of_b, int j) {
    if constexpr (HALF) {
        const uint64_t v = of_b ? e.y[j >> 1] : e.x[j >> 1];
        return (j & 1) ? hi2(v) : lo2(v);
    } else {
        const int k = (of_b ? 4 : 0) + (j >> 1);   // the pair
        const uint64_t v = (j & 1) ? e.y[k >> 1] : e.x[k >> 1];
        return (k & 1) ? hi2(v) : lo2(v);
    }
}

template <int DT, bool HALF>
__device__ __forceinline__ uint4 pack_chunk(const Chunk16& e, bool of_b) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<DT>(element<HALF>(e, of_b, 2 * i), element<HALF>(e, of_b, 2 * i + 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Cosines and sines of the eight pairs of unit u at one position.
struct Turn {
    uint64_t c[4], s[4];
};

// (Plain loads: the table may come from the kernel before, whose end this kernel awaits while it runs.)
__device__ __forceinline__ void load_turn(Turn& t, const float* cos_sin, int rot, int pos, int u) {
    const float* at = cos_sin + static_cast<int64_t>(pos) * rot + 8 * u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const ulonglong2 c = reinterpret_cast<const ulonglong2*>(at)[i];
        const ulonglong2 s = reinterpret_cast<const ulonglong2*>(at + rot / 2)[i];
        t.c[2 * i] = c.x;
        t.c[2 * i + 1] = c.y;
        t.s[2 * i] = s.x;
        t.s[2 * i + 1] = s.y;
    }
}

__device__ __forceinline__ void rotate(Chunk16& e, const Turn& t, uint64_t minus_zero) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t x = sub2(mul2(e.x[i], t.c[i], minus_zero), mul2(e.y[i], t.s[i], minus_zero));
        e.y[i] = add2(mul2(e.y[i], t.c[i], minus_zero), mul2(e.x[i], t.s[i], minus_zero));
        e.x[i] = x;
    }
}

// First dims of unit u's two chunks. (HALF: the half rotation. Units past rot_dim pass as they are, and
// so do all without a rotation, rot = 0.)
template <bool HALF>
__device__ __forceinline__ void unit_dims(const AppendParams& p, int u, int& da, int& db) {
    const bool paired = HALF && 16 * u < p.rot;
    da = paired ? 8 * u : 16 * u;
    db = paired ? p.rot / 2 + 8 * u : 16 * u + 8;
}

// Stage cu_new and kv_lens in shared memory; AT_ONCE: every read on its way before the first is waited for
// (256 tokens, one per sequence, into e4m3 pages 4.2 -> 4.1 us; 9887 tokens 43.6 -> 42.2). Where the threads hold rows
// meanwhile and few registers are left (16-bit pages, the rows of a decode step) it costs more than it gives:
// 9887 tokens into 16-bit pages 39.5 -> 41.3 us.
template <bool AT_ONCE>
__device__ __forceinline__ void stage_sequences(const AppendParams& p, int32_t* cu, int32_t* lens) {
    if constexpr (AT_ONCE) {
        constexpr int kMost = (DA_MAX_PAGED_BATCH + kAppendThreads - 1) / kAppendThreads;
        const int tid = threadIdx.x;
        int32_t c[kMost], l[kMost], c0 = 0;
        if (tid == 0) c0 = ld_cg_s32(p.cu);
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
            const int i = tid + k * kAppendThreads;
            if (i < p.B) {
                c[k] = ld_cg_s32(p.cu + i + 1);
                l[k] = ld_cg_s32(p.lens + i);
            }
        }
        if (tid == 0) cu[0] = c0;
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
            const int i = tid + k * kAppendThreads;
            if (i < p.B) {
                cu[i + 1] = c[k];
                lens[i] = l[k];
            }
        }
    } else {
        for (int i = threadIdx.x; i <= p.B; i += kAppendThreads) {
            cu[i] = ld_cg_s32(p.cu + i);
            if (i < p.B) lens[i] = ld_cg_s32(p.lens + i);
        }
    }
    __syncthreads();
}

// The sequence whose rows hold `row`, or -1: the last b with cu[b] <= row, checked.
__device__ __forceinline__ int sequence_of(const AppendParams& p, const int32_t* cu, int row) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= row) lo = mid;
        else hi = mid - 1;
    }
    return cu[lo] <= row && row < cu[lo + 1] ? lo : -1;
}

// A sequence's page that holds position pos, or -1 (flagged) for a bad table entry.
__device__ __forceinline__ int page_of(const AppendParams& p, int b, int pos) {
    const int page = ld_cg_s32(p.table + static_cast<int64_t>(b) * p.table_stride + pos / p.P);
    if (page >= 0 && page < p.num_pages) return page;
    flag_error(p.err, DA_DEVERR_PAGE);
    return -1;
}

// Rows of tokens x heads: the queries and, with KV16, the keys and values of a 16-bit cache. A block
// takes as many tokens as its threads hold; a thread goes through its heads of one token, the loads of
// the first ones issued before anything is known of the token's sequence (they depend on the row
// alone), and keeps its pairs' cosines and sines for all of them.
template <int D, int DT, bool HALF, bool KV16>
struct AppendRows {
    static constexpr int kUnits = D / 16;
    // query heads in flight: as many as the registers hold (e4m3 pages, 9887 tokens: 42.2 us with two, 41.5 with four)
    static constexpr int kAhead = KV16 ? 2 : 4;
    struct Chunk {
        uint4 a, b;
    };
    const AppendParams& p;
    const int u, lane;
    const int64_t row;
    int da, db;
    Chunk wq[kAhead], wk, wv;

    static __device__ __forceinline__ Chunk get(const uint16_t* at, int da, int db) {
        Chunk w;
        w.a = *reinterpret_cast<const uint4*>(at + da);
        w.b = *reinterpret_cast<const uint4*>(at + db);
        return w;
    }
    static __device__ __forceinline__ void put(uint16_t* at, int da, int db, const Chunk& w) {
        *reinterpret_cast<uint4*>(at + da) = w.a;
        *reinterpret_cast<uint4*>(at + db) = w.b;
    }
    __device__ __forceinline__ void turn_chunk(Chunk& w, const Turn& turn) const {
        Chunk16 e;
        unpack16<DT, HALF>(w.a, w.b, e);
        rotate(e, turn, p.minus_zero);
        w.a = pack_chunk<DT, HALF>(e, false);
        w.b = pack_chunk<DT, HALF>(e, true);
    }
    __device__ __forceinline__ void load_q(int h0) {
        const uint16_t* at = p.q + row * p.q_stride + h0 * D;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (h0 + k * p.head_lanes < p.Hq) wq[k] = get(at + k * p.head_lanes * D, da, db);
    }
    __device__ __forceinline__ void load_kv(int h) {
        if (h >= p.Hkv) return;
        wk = get(p.k + row * p.k_stride + h * D, da, db);
        wv = get(p.v + row * p.v_stride + h * D, da, db);
    }
    __device__ __forceinline__ AppendRows(const AppendParams& params, int64_t group)
        : p(params),
          u(threadIdx.x % kUnits),
          lane((threadIdx.x / kUnits) % params.head_lanes),
          row(group * (kAppendThreads / (kUnits * params.head_lanes)) + threadIdx.x / (kUnits * params.head_lanes)) {
        unit_dims<HALF>(p, u, da, db);
        if (row >= p.T) return;
        if constexpr (KV16) load_kv(lane);
        load_q(lane);
    }
    __device__ __forceinline__ void finish(const int32_t* cu, const int32_t* lens) {
        if (row >= p.T) return;
        const int b = sequence_of(p, cu, static_cast<int>(row));
        if (b < 0) return;
        const NewTokens t = new_tokens(p, cu[b], cu[b + 1], lens[b]);
        if (t.n == 0) return;
        const int pos = t.start + static_cast<int>(row) - t.first;
        if (p.rope != DA_ROPE_NONE && pos >= p.max_pos) {
            if (u == 0 && lane == 0) flag_error(p.err, DA_DEVERR_POSITION);
            return;
        }
        const bool turns = 16 * u < p.rot;
        Turn turn;
        if (turns) load_turn(turn, p.cos_sin, p.rot, pos, u);
        if constexpr (KV16) {
            const int page = page_of(p, b, pos);
            if (page >= 0) {
                const int64_t at = page_row(p.layout, page, pos % p.P, 0, p.P, p.Hkv) * D;
                const int64_t step = (p.layout == DA_LAYOUT_VARLEN ? 1 : p.P) * D;
                for (int h = lane; h < p.Hkv; h += p.head_lanes) {
                    if (h != lane) load_kv(h);
                    if (turns) turn_chunk(wk, turn);
                    put(reinterpret_cast<uint16_t*>(p.kc) + at + h * step, da, db, wk);
                    put(reinterpret_cast<uint16_t*>(p.vc) + at + h * step, da, db, wv);
                }
            }
        }
        uint16_t* out = p.q_out + row * p.q_out_stride;
        for (int h0 = lane; h0 < p.Hq; h0 += kAhead * p.head_lanes) {
            if (h0 != lane) load_q(h0);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int h = h0 + k * p.head_lanes;
                if (h < p.Hq) {
                    if (turns) turn_chunk(wq[k], turn);
                    put(out + h * D, da, db, wq[k]);
                }
            }
        }
    }
};

__device__ __forceinline__ void flag_bad_sequences(const AppendParams& p, const int32_t* cu, const int32_t* lens) {
    for (int b = threadIdx.x; b < p.B; b += kAppendThreads)
        if (new_tokens(p, cu[b], cu[b + 1], lens[b]).bad) flag_error(p.err, DA_DEVERR_SEQLENS);
}

template <int D, int DT, bool HALF>
__global__ void __launch_bounds__(kAppendThreads, 4) append16_kernel(const AppendParams p) {
    extern __shared__ int32_t append_smem[];
    int32_t* cu = append_smem;
    int32_t* lens = append_smem + p.B + 1;
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_dependents_launch();
    AppendRows<D, DT, HALF, true> rows(p, blockIdx.x);
    stage_sequences<false>(p, cu, lens);
    if (blockIdx.x == 0) flag_bad_sequences(p, cu, lens);
    rows.finish(cu, lens);
}

// ------------------------------------------------------------ 8-bit pages
// Least power of two s with amax <= 448 s (at least 2^-126).
__device__ __forceinline__ float needed_scale(float amax) {
    const uint32_t w = __float_as_uint(amax);
    const int x = static_cast<int>(w >> 23);                   // biased exponent (amax >= 0)
    const int e = x - 8 + ((w & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
}

// Four float32 to four e4m3 codes, to nearest even, saturating.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Four e4m3 codes times `by`, rounded to e4m3 again.
__device__ __forceinline__ uint32_t scale_e4m3x4(uint32_t w, float by) {
    float f[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(w >> (16 * i))));
        f[2 * i] = bits_to_f32<DA_F16>(h2 & 0xffffu) * by;
        f[2 * i + 1] = bits_to_f32<DA_F16>(h2 >> 16) * by;
    }
    return to_e4m3x4(f[0], f[1], f[2], f[3]);
}

// The new tokens of one page, as a unit's threads need them.
struct PagePart {
    int row0, n, slot0, pos0, page;   // first row, tokens, first slot and its position, the page

    __device__ __forceinline__ void locate(const AppendParams& p, const NewTokens& t, int b, int nth_page) {
        const int first_page = t.start / p.P;
        const int page_pos = (first_page + nth_page) * p.P;   // position of the page's first slot
        slot0 = nth_page == 0 ? t.start - page_pos : 0;
        pos0 = page_pos + slot0;
        row0 = t.first + (pos0 - t.start);
        n = min(p.P - slot0, t.start + t.n - pos0);
        page = ld_cg_s32(p.table + static_cast<int64_t>(b) * p.table_stride + first_page + nth_page);
    }
    // Whether anything is to be written (flags what is not).
    __device__ __forceinline__ bool check(const AppendParams& p, bool first_thread) {
        if (p.rope != DA_ROPE_NONE && pos0 + n > p.max_pos) {
            if (first_thread) flag_error(p.err, DA_DEVERR_POSITION);
            n = p.max_pos - pos0;
        }
        const bool good = page >= 0 && page < p.num_pages;
        if (!good && first_thread) flag_error(p.err, DA_DEVERR_PAGE);
        return good && n > 0;
    }
};

// The new scale of a page and head: `before` is the old one (0 for a page that begins here). Where it
// grew, kLanes threads round the page's earlier elements again.
template <int D, int kLanes>
__device__ __forceinline__ float grow_scale(const AppendParams& p, const PagePart& x, int head, bool is_v, float before,
                                            float amax, int lane) {
    const float scale = fmaxf(before, needed_scale(amax));
    if (lane == 0 && scale != before) (is_v ? p.vs : p.ks)[static_cast<int64_t>(x.page) * p.Hkv + head] = scale;
    if (scale > before && x.slot0 > 0) {
        const float by = before / scale;
        const int chunks = x.slot0 * (D / 16);
        for (int i = lane; i < chunks; i += kLanes) {
            uint4* at = reinterpret_cast<uint4*>((is_v ? p.vc : p.kc) +
                                                 page_row(p.layout, x.page, i / (D / 16), head, p.P, p.Hkv) * D + (i % (D / 16)) * 16);
            uint4 c = *at;
            c.x = scale_e4m3x4(c.x, by);
            c.y = scale_e4m3x4(c.y, by);
            c.z = scale_e4m3x4(c.z, by);
            c.w = scale_e4m3x4(c.w, by);
            *at = c;
        }
    }
    return scale;
}

// Barrier of a unit's threads.
template <int kLanes>
__device__ __forceinline__ void unit_sync() {
    if constexpr (kLanes == kAppendThreads) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x) / kLanes), "n"(kLanes) : "memory");
}

// A unit is the new tokens of one page and KV head, keys or values, by kLanes threads: a warp for the few
// tokens of a decode step, up to the block for prompts (run_append). A thread holds kKeep rows in registers between the
// pass that finds the largest element and the one that rounds (further rows are read twice): rotated, in
// float32, where it is one row (256 tokens, one per sequence: 4.2 us against 4.3), as they were read where
// twice as many such registers would cost a third of the blocks (9887 tokens: 43.3 us against 49).
template <int D, int DT, bool HALF, int kLanes>
struct AppendPage {
    static constexpr int kUnits = D / 16;
    static constexpr int kRows = kLanes / kUnits;   // rows at once
    static constexpr int kKeep = kLanes == 32 ? 1 : 2;
    static constexpr bool kKeepTurned = kKeep == 1;
    struct Chunk {
        uint4 a, b;
    };
    const AppendParams& p;
    const int lane, u, r0;
    PagePart x;
    int hv;                // head, keys (even) or values
    int da, db;
    bool turns;
    const uint16_t* src;   // the first new row
    int64_t stride;
    Chunk kept[kKeep];
    Chunk16 kept_turned[kKeepTurned ? kKeep : 1];

    __device__ __forceinline__ AppendPage(const AppendParams& params, int l) : p(params), lane(l), u(l % kUnits), r0(l / kUnits) {
        unit_dims<HALF>(p, u, da, db);
    }
    __device__ __forceinline__ void load(const NewTokens& t, int b, int nth_page, int unit_hv) {
        hv = unit_hv;
        const bool is_v = (hv & 1) != 0;
        x.locate(p, t, b, nth_page);
        turns = !is_v && 16 * u < p.rot;
        stride = is_v ? p.v_stride : p.k_stride;
        src = (is_v ? p.v : p.k) + x.row0 * stride + static_cast<int64_t>(hv >> 1) * D;
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (r0 + i * kRows < x.n) kept[i] = read(r0 + i * kRows);
    }
    __device__ __forceinline__ Chunk read(int r) const {
        Chunk w;
        const uint16_t* at = src + r * stride;
        w.a = *reinterpret_cast<const uint4*>(at + da);
        w.b = *reinterpret_cast<const uint4*>(at + db);
        return w;
    }
    __device__ __forceinline__ void turned(const Chunk& w, int r, Chunk16& e) const {
        unpack16<DT, HALF>(w.a, w.b, e);
        if (turns) {
            Turn turn;
            load_turn(turn, p.cos_sin, p.rot, x.pos0 + r, u);
            rotate(e, turn, p.minus_zero);
        }
    }
    template <class F>
    __device__ __forceinline__ void rows(F&& f) const {
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (r0 + i * kRows < x.n) {
                Chunk16 e;
                if constexpr (kKeepTurned) e = kept_turned[i];
                else turned(kept[i], r0 + i * kRows, e);
                f(r0 + i * kRows, e);
            }
        for (int r = r0 + kKeep * kRows; r < x.n; r += kRows) {
            Chunk16 e;
            turned(read(r), r, e);
            f(r, e);
        }
    }
    // The largest magnitude of the unit, NaN ignored, and infinities too with FINITE.
    template <bool FINITE>
    __device__ __forceinline__ float largest(float* red) const {
        float amax = 0.f;
        rows([&](int, const Chunk16& e) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float f[4] = {fabsf(lo2(e.x[j])), fabsf(hi2(e.x[j])), fabsf(lo2(e.y[j])), fabsf(hi2(e.y[j]))};
#pragma unroll
                for (int k = 0; k < 4; ++k) amax = fmaxf(amax, FINITE && f[k] == INFINITY ? 0.f : f[k]);
            }
        });
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        if constexpr (kLanes > 32) {
            if ((threadIdx.x & 31) == 0) red[lane >> 5] = amax;
            unit_sync<kLanes>();
#pragma unroll
            for (int w = 0; w < kLanes / 32; ++w) amax = fmaxf(amax, red[w]);
        } else {
            __syncwarp();
        }
        return amax;
    }
    // Round the rows to e4m3 at the scale; EXACT: a power of two, whose reciprocal is exact.
    template <bool EXACT>
    __device__ __forceinline__ void write(uint8_t* to, int64_t row_step, float scale) const {
        const float inv = 1.f / scale;
        rows([&](int r, const Chunk16& e) {
            uint8_t* at = to + r * row_step;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float y = element<HALF>(e, c == 1, j);
                    f[j] = EXACT ? y * inv : y / scale;
                }
                *reinterpret_cast<uint2*>(at + (c == 0 ? da : db)) =
                    make_uint2(to_e4m3x4(f[0], f[1], f[2], f[3]), to_e4m3x4(f[4], f[5], f[6], f[7]));
            }
        });
    }

    // red: shared, a float per warp of the unit, not the one that the last call used. Whether this one used it: a unit
    // that is left out returns before its barrier, with the last call's maxima perhaps still being read.
    __device__ __forceinline__ bool finish(float* red) {
        if (!x.check(p, lane == 0)) return false;   // for the whole unit
        const int head = hv >> 1;
        const bool is_v = (hv & 1) != 0;
        const float* scale_at = (is_v ? p.vs : p.ks) + static_cast<int64_t>(x.page) * p.Hkv + head;
        const float before = x.slot0 > 0 ? *reinterpret_cast<const volatile float*>(scale_at) : 0.f;
        if constexpr (kKeepTurned) {
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (r0 + i * kRows < x.n) turned(kept[i], r0 + i * kRows, kept_turned[i]);
        }
        float amax = largest<false>(red);
        if (amax == INFINITY) {   // the same for every thread
            if constexpr (kLanes > 32) unit_sync<kLanes>();   // `red` has been read
            amax = largest<true>(red);
        }
        // every thread has read `before` by now
        const float scale = grow_scale<D, kLanes>(p, x, head, is_v, before, amax, lane);
        uint8_t* to = (is_v ? p.vc : p.kc) + page_row(p.layout, x.page, x.slot0, head, p.P, p.Hkv) * D;
        const int64_t row_step = static_cast<int64_t>(p.layout == DA_LAYOUT_VARLEN ? p.Hkv : 1) * D;
        if ((__float_as_uint(scale) & 0x7fffffu) == 0) write<true>(to, row_step, scale);
        else write<false>(to, row_step, scale);
        return true;
    }
};

// 8-bit pages, and the queries' rows. Page units are (touched page, KV head, keys or values) of all
// sequences, head fastest.
template <int D, int DT, bool HALF, int kLanes>
__global__ void __launch_bounds__(kAppendThreads, kLanes == 32 ? 2 : 3) append8_kernel(const AppendParams p) {
    extern __shared__ int32_t append_smem[];
    __shared__ int32_t warp_sum[kAppendThreads / 32];
    __shared__ float red[2][kAppendThreads / 32];   // used in turn
    int32_t* cu = append_smem;
    int32_t* lens = cu + p.B + 1;
    int32_t* prefix = lens + p.B;      // touched pages before sequence b, [B + 1]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    if (tid == 0) grid_dependents_launch();
    if (static_cast<int>(blockIdx.x) >= p.page_blocks) {
        AppendRows<D, DT, HALF, false> rows(p, blockIdx.x - p.page_blocks);
        stage_sequences<(kLanes > 32)>(p, cu, lens);
        rows.finish(cu, lens);
        return;
    }
    stage_sequences<true>(p, cu, lens);
    if (blockIdx.x == 0) flag_bad_sequences(p, cu, lens);
    // running count of touched pages: each thread sums its run of sequences, then one scan
    const int per = (p.B + kAppendThreads - 1) / kAppendThreads;
    int mine = 0;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= p.B) break;
        const NewTokens t = new_tokens(p, cu[b], cu[b + 1], lens[b]);
        if (t.n > 0) mine += (t.start + t.n - 1) / p.P - t.start / p.P + 1;
    }
    int run = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, run, off);
        if (lane >= off) run += y;
    }
    if (lane == 31) warp_sum[warp] = run;
    __syncthreads();
    int before = run - mine;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= p.B) break;
        prefix[b] = before;
        const NewTokens t = new_tokens(p, cu[b], cu[b + 1], lens[b]);
        if (t.n > 0) before += (t.start + t.n - 1) / p.P - t.start / p.P + 1;
        if (b == p.B - 1) prefix[p.B] = before;
    }
    __syncthreads();
    const uint32_t groups = 2u * p.Hkv, units = prefix[p.B] * groups;   // below 2^31: checked by the host
    constexpr int kPerBlock = kAppendThreads / kLanes;
    const uint32_t step = static_cast<uint32_t>(p.page_blocks) * kPerBlock;
    AppendPage<D, DT, HALF, kLanes> page(p, tid % kLanes);
    const int sub = tid / kLanes;
    int turn = 0;
    // the bound is uniform over a unit's threads
    for (uint32_t unit = blockIdx.x * kPerBlock + sub; unit < units; unit += step) {
        const int nth = static_cast<int>(unit / groups), hv = static_cast<int>(unit - nth * groups);
        int lo = 0, hi = p.B - 1;   // last b with prefix[b] <= nth
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= nth) lo = mid;
            else hi = mid - 1;
        }
        page.load(new_tokens(p, cu[lo], cu[lo + 1], lens[lo]), lo, nth - prefix[lo], hv);
        if (page.finish(&red[turn][sub * (kLanes / 32)])) turn ^= 1;
    }
}

// ------------------------------------------------------------ host side
template <class K>
da_status launch_append(K kern, int grid, size_t smem, const AppendParams& p, cudaStream_t stream) {
    cudaLaunchAttribute attrs[1] = {pdl_attr()};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kAppendThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

// Blocks for pages: what fits the GPU at once, times the pages' share of the work, an element of theirs taken for
// kPageWeight of a query's. Each takes several units, so that rows, which are bound by bytes, run beside pages,
// which are bound by latency and instructions, from the first to the last (7200 tokens of 3 x 32 128-dim heads:
// 66.2 us, with two thirds for pages 92.5, with all 68.4; 9887 tokens of 32 + 2 x 8 heads 41.2, all 43.0, a block
// for each unit 49.8). Rows take over what pages leave, not the other way round, hence the large weight (8; 3 or 4:
// 5.8 us where 8 has 4.3, 200 tokens of 28 + 2 x 4 heads).
constexpr int kPageWeight = 8;
constexpr int kManyHeads = 8;                // heads per thread where there are many tokens
constexpr int64_t kManyThreads = 152 * 512;  // threads that keep the GPU busy

template <int D, int DT, bool HALF>
da_status run_append(AppendParams& p, bool e4m3, cudaStream_t stream) {
    constexpr int kUnits = D / 16;
    // Threads per token and unit: one for each head while the tokens leave the GPU's threads idle; with many
    // tokens each takes up to kManyHeads of them, and finds its token's sequence, cosines and page once for
    // all (9887 tokens, 48 heads: 39.3 us, 42.6 with half as many, 41.7 with twice as many).
    const int heads = p.Hq + (e4m3 ? 0 : 2 * p.Hkv);
    while (p.head_lanes < kAppendThreads / kUnits && p.head_lanes < std::max(p.Hq, e4m3 ? 0 : p.Hkv) &&
           (p.head_lanes * kManyHeads < heads || static_cast<int64_t>(p.T) * kUnits * p.head_lanes < kManyThreads))
        p.head_lanes *= 2;
    const int tokens = kAppendThreads / kUnits / p.head_lanes;
    const int row_blocks = e4m3 && p.Hq == 0 ? 0 : 1 + (p.T - 1) / tokens;   // (T >= 1, up to 2^31 - 1)
    const size_t smem = (3 * p.B + 2) * sizeof(int32_t);
    if (!e4m3) return launch_append(append16_kernel<D, DT, HALF>, row_blocks, smem, p, stream);
    // a sequence's n new tokens touch at most min(n, n / P + 2) pages
    const int64_t touched = std::min<int64_t>(p.T, p.T / p.P + 2ll * p.B);
    // Threads per page and head: a warp while pages get few tokens each, else as many as hold a page of 32 or of
    // 64 tokens in registers: fewer read rows twice (pages of 64 tokens, half the threads: 18.7 us against 17.8, and
    // 15.3 against 9.3), more idle and have fewer bytes in flight (pages of 32 tokens, twice the threads: 16.6 us
    // against 14.2; 64-dim heads, pages of 64, the whole block: 51.9 against 37.6).
    // (A warp for up to three tokens per sequence: 64 sequences of 3 tokens, 32 + 2 x 8 heads, 4.2 us against 8.7. It is
    // ahead further than that: of 4 tokens 5.1 against 8.7, of 16 8.2 against 11.6; of 32 17.5 against 16.7.)
    const bool few = p.T < 4 * static_cast<int64_t>(p.B);
    const int lanes = few ? 32 : p.P <= 32 ? D : 2 * D;
    const int64_t units = touched * p.Hkv * 2;
    if (units > 0x3fffffffll) return DA_ERR_INVALID_ARG;
    const int64_t page_work = 2ll * kPageWeight * p.Hkv, resident = 152 * (few ? 2 : 3);
    const int64_t most = std::max<int64_t>(1, resident * page_work / (page_work + p.Hq));
    const int per_block = kAppendThreads / lanes;
    p.page_blocks = static_cast<int>(std::min<int64_t>((units + per_block - 1) / per_block, most));
    const int grid = p.page_blocks + row_blocks;
    if (lanes == 32) return launch_append(append8_kernel<D, DT, HALF, 32>, grid, smem, p, stream);
    if (lanes == D) return launch_append(append8_kernel<D, DT, HALF, D>, grid, smem, p, stream);
    return launch_append(append8_kernel<D, DT, HALF, 2 * D>, grid, smem, p, stream);
}

template <int D, int DT>
da_status run_append_any(AppendParams& p, bool half, bool e4m3, cudaStream_t s) {
    return half ? run_append<D, DT, true>(p, e4m3, s) : run_append<D, DT, false>(p, e4m3, s);
}

}  // namespace da_impl

using namespace da_impl;

extern "C" da_status decode_attn_paged_append(const da_paged_append* args, void* stream) {
    if (!args) return DA_ERR_INVALID_ARG;
    const da_paged_append& a = *args;
    da_status st = check_cache(a.cache, a.dtype, a.kv_lens, a.block_table, a.max_pages, a.table_stride, a.B, a.Hq);
    if (st != DA_OK) return st;
    const da_paged_cache& c = *a.cache;
    if (a.T_new < 0 || !a.cu_new || !a.workspace) return DA_ERR_INVALID_ARG;
    if (a.rope != DA_ROPE_NONE && a.rope != DA_ROPE_HALF && a.rope != DA_ROPE_INTERLEAVED) return DA_ERR_INVALID_ARG;
    const bool turns = a.rope != DA_ROPE_NONE;
    if (turns && (!a.cos_sin || a.max_pos < 1 || a.rot_dim < 16 || a.rot_dim > c.D || a.rot_dim % 16)) return DA_ERR_INVALID_ARG;
    const int Hq = a.q ? a.Hq : 0;
    if (Hq > 0 && !a.q_out) return DA_ERR_INVALID_ARG;
    if (a.T_new > 0 && (!a.k || !a.v)) return DA_ERR_INVALID_ARG;
    const int64_t kv_row = static_cast<int64_t>(c.Hkv) * c.D, q_row = static_cast<int64_t>(Hq) * c.D;
    if (a.k_stride < kv_row || a.v_stride < kv_row || (Hq > 0 && (a.q_stride < q_row || a.q_out_stride < q_row)))
        return DA_ERR_INVALID_ARG;
    if (!aligned(a.workspace, 256) || !aligned(a.cu_new, 4) || !aligned(a.k, 16) || !aligned(a.v, 16) || a.k_stride % 8 ||
        a.v_stride % 8)
        return DA_ERR_ALIGNMENT;
    if (Hq > 0 && (!aligned(a.q, 16) || !aligned(a.q_out, 16) || a.q_stride % 8 || a.q_out_stride % 8)) return DA_ERR_ALIGNMENT;
    if (turns && !aligned(a.cos_sin, 16)) return DA_ERR_ALIGNMENT;
    if (a.T_new == 0) return DA_OK;
    AppendParams p;
    p.q = static_cast<const uint16_t*>(a.q);
    p.k = static_cast<const uint16_t*>(a.k);
    p.v = static_cast<const uint16_t*>(a.v);
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.q_out_stride = a.q_out_stride;
    p.minus_zero = 0x8000000080000000ull;
    p.cos_sin = a.cos_sin;
    p.cu = a.cu_new;
    p.lens = a.kv_lens;
    p.table = a.block_table;
    p.q_out = static_cast<uint16_t*>(a.q_out);
    p.kc = static_cast<uint8_t*>(c.k);
    p.vc = static_cast<uint8_t*>(c.v);
    p.ks = c.k_scale;
    p.vs = c.v_scale;
    p.err = static_cast<uint32_t*>(a.workspace);
    p.B = a.B;
    p.T = a.T_new;
    p.Hq = Hq;
    p.Hkv = c.Hkv;
    p.P = c.page_size;
    p.max_pages = a.max_pages;
    p.table_stride = a.table_stride;
    p.num_pages = c.num_pages;
    p.layout = c.layout;
    p.max_pos = turns ? a.max_pos : 0x7fffffff;
    p.rot = turns ? a.rot_dim : 0;
    p.rope = a.rope;
    p.head_lanes = 1;
    p.page_blocks = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool e4m3 = c.kv_dtype == DA_E4M3;
    const bool half = a.rope == DA_ROPE_HALF;
    if (c.D == 128)
        return a.dtype == DA_F16 ? run_append_any<128, DA_F16>(p, half, e4m3, s) : run_append_any<128, DA_BF16>(p, half, e4m3, s);
    return a.dtype == DA_F16 ? run_append_any<64, DA_F16>(p, half, e4m3, s) : run_append_any<64, DA_BF16>(p, half, e4m3, s);
}
