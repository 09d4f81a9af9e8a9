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
// decode step (a chain of four dependent reads: cu_new and kv_lens, block table, scale and
// rows, then the stores).
//
// Threads: one thread owns 16 elements of one head's row, the two 16-byte chunks whose
// elements pair up (dims [8u, 8u + 8) and [rot/2 + 8u, ...) for the half rotation, 16
// consecutive dims for the interleaved one), so a rotation needs no exchange, loads and
// stores are 16 bytes wide, and a row may be rotated in place.

#include "paged_common.cuh"

namespace da_impl {

constexpr int kAppendThreads = 256;

struct AppendParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
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
    int tokens_per_block;    // row kernel: tokens a block handles at once
    int row_blocks;          // 8-bit call: blocks that rotate queries, after the page blocks
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

struct Chunk16 {     // the 16 elements of one thread, in float32
    float a[8], b[8];
};

template <int DT>
__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bits_to_f32<DT>(x[i] & 0xffffu);
        f[2 * i + 1] = bits_to_f32<DT>(x[i] >> 16);
    }
}

template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7]));
}

// Eight cosines and sines of one position: the pairs of unit u.
struct Turn {
    float c[8], s[8];
};

__device__ __forceinline__ void load_turn(Turn& t, const float* cos_sin, int rot, int pos, int u) {
    const float4* c = reinterpret_cast<const float4*>(cos_sin + static_cast<int64_t>(pos) * rot + 8 * u);
    const float4* s = reinterpret_cast<const float4*>(cos_sin + static_cast<int64_t>(pos) * rot + rot / 2 + 8 * u);
    const float4 c0 = __ldg(c), c1 = __ldg(c + 1), s0 = __ldg(s), s1 = __ldg(s + 1);
    t.c[0] = c0.x; t.c[1] = c0.y; t.c[2] = c0.z; t.c[3] = c0.w;
    t.c[4] = c1.x; t.c[5] = c1.y; t.c[6] = c1.z; t.c[7] = c1.w;
    t.s[0] = s0.x; t.s[1] = s0.y; t.s[2] = s0.z; t.s[3] = s0.w;
    t.s[4] = s1.x; t.s[5] = s1.y; t.s[6] = s1.z; t.s[7] = s1.w;
}

__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
    const float p = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    const float r = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = p;
    y = r;
}

__device__ __forceinline__ void rotate(Chunk16& e, const Turn& t, bool half) {
    if (half) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(e.a[i], e.b[i], t.c[i], t.s[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            turn_pair(e.a[2 * i], e.a[2 * i + 1], t.c[i], t.s[i]);
            turn_pair(e.b[2 * i], e.b[2 * i + 1], t.c[4 + i], t.s[4 + i]);
        }
    }
}

// First dims of unit u's two chunks.
__device__ __forceinline__ void unit_dims(const AppendParams& p, int u, int& da, int& db) {
    const bool paired = p.rope == DA_ROPE_HALF && 16 * u < p.rot;
    da = paired ? 8 * u : 16 * u;
    db = paired ? p.rot / 2 + 8 * u : 16 * u + 8;
}

// Stage cu_new and kv_lens in shared memory.
__device__ __forceinline__ void stage_sequences(const AppendParams& p, int32_t* cu, int32_t* lens) {
    for (int i = threadIdx.x; i <= p.B; i += kAppendThreads) {
        cu[i] = ld_cg_s32(p.cu + i);
        if (i < p.B) lens[i] = ld_cg_s32(p.lens + i);
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

// Rows [block's tokens] x heads: the queries and, with KV16, the keys and values of a
// 16-bit cache. `block` of `blocks` blocks; every thread keeps its pairs' cosines and sines
// for all the heads of a token.
template <int D, int DT, bool KV16>
__device__ __forceinline__ void append_rows(const AppendParams& p, const int32_t* cu, const int32_t* lens, int block,
                                            int blocks) {
    constexpr int kUnits = D / 16;
    const int head_lanes = kAppendThreads / (kUnits * p.tokens_per_block);
    const int u = threadIdx.x % kUnits;
    const int hl = (threadIdx.x / kUnits) % head_lanes;
    const int tk = threadIdx.x / (kUnits * head_lanes);
    const int heads = KV16 ? p.Hq + 2 * p.Hkv : p.Hq;
    const bool half = p.rope == DA_ROPE_HALF;
    const bool turns = p.rope != DA_ROPE_NONE && 16 * u < p.rot;
    int da, db;
    unit_dims(p, u, da, db);
    for (int64_t row0 = static_cast<int64_t>(block) * p.tokens_per_block; row0 < p.T;
         row0 += static_cast<int64_t>(blocks) * p.tokens_per_block) {
        const int64_t row = row0 + tk;
        if (row >= p.T) continue;
        const int b = sequence_of(p, cu, static_cast<int>(row));
        if (b < 0) continue;
        const NewTokens t = new_tokens(p, cu[b], cu[b + 1], lens[b]);
        if (t.n == 0) continue;
        const int pos = t.start + static_cast<int>(row) - t.first;
        if (p.rope != DA_ROPE_NONE && pos >= p.max_pos) {
            if (u == 0 && hl == 0) flag_error(p.err, DA_DEVERR_POSITION);
            continue;
        }
        int page = 0;
        if constexpr (KV16) page = page_of(p, b, pos);
        Turn turn;
        if (turns) load_turn(turn, p.cos_sin, p.rot, pos, u);
        constexpr int kAhead = 3;   // head rows in flight per thread
        for (int h0 = hl; h0 < heads; h0 += kAhead * head_lanes) {
            uint4 wa[kAhead], wb[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int h = h0 + i * head_lanes;
                if (h >= heads) continue;
                const uint16_t* src = h < p.Hq ? p.q + row * p.q_stride + static_cast<int64_t>(h) * D
                                     : h < p.Hq + p.Hkv ? p.k + row * p.k_stride + static_cast<int64_t>(h - p.Hq) * D
                                                        : p.v + row * p.v_stride + static_cast<int64_t>(h - p.Hq - p.Hkv) * D;
                wa[i] = *reinterpret_cast<const uint4*>(src + da);
                wb[i] = *reinterpret_cast<const uint4*>(src + db);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int h = h0 + i * head_lanes;
                if (h >= heads) continue;
                const bool is_v = h >= p.Hq + p.Hkv;
                if (turns && !is_v) {
                    Chunk16 e;
                    unpack8<DT>(wa[i], e.a);
                    unpack8<DT>(wb[i], e.b);
                    rotate(e, turn, half);
                    wa[i] = pack8<DT>(e.a);
                    wb[i] = pack8<DT>(e.b);
                }
                uint16_t* dst;
                if (h < p.Hq) {
                    dst = p.q_out + row * p.q_out_stride + static_cast<int64_t>(h) * D;
                } else {
                    if (page < 0) continue;
                    const int kvh = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
                    dst = reinterpret_cast<uint16_t*>(is_v ? p.vc : p.kc) +
                          page_row(p.layout, page, pos % p.P, kvh, p.P, p.Hkv) * D;
                }
                *reinterpret_cast<uint4*>(dst + da) = wa[i];
                *reinterpret_cast<uint4*>(dst + db) = wb[i];
            }
        }
    }
}

__device__ __forceinline__ void flag_bad_sequences(const AppendParams& p, const int32_t* cu, const int32_t* lens) {
    for (int b = threadIdx.x; b < p.B; b += kAppendThreads)
        if (new_tokens(p, cu[b], cu[b + 1], lens[b]).bad) flag_error(p.err, DA_DEVERR_SEQLENS);
}

template <int D, int DT>
__global__ void __launch_bounds__(kAppendThreads) append16_kernel(const AppendParams p) {
    extern __shared__ int32_t append_smem[];
    int32_t* cu = append_smem;
    int32_t* lens = append_smem + p.B + 1;
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_dependents_launch();
    stage_sequences(p, cu, lens);
    if (blockIdx.x == 0) flag_bad_sequences(p, cu, lens);
    append_rows<D, DT, true>(p, cu, lens, blockIdx.x, gridDim.x);
}

// ------------------------------------------------------------ 8-bit pages
// Least power of two s with amax <= 448 s (at least 2^-126).
__device__ __forceinline__ float needed_scale(float amax) {
    const uint32_t w = __float_as_uint(amax);
    const int x = static_cast<int>(w >> 23);                   // biased exponent (amax >= 0)
    const int e = x - 8 + ((w & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
}

// x / s for a fixed s: a multiplication where 1 / s is exact.
struct Divide {
    float s, inv;
    bool exact;
    __device__ __forceinline__ explicit Divide(float scale) : s(scale) {
        inv = 1.f / scale;
        exact = (__float_as_uint(scale) & 0x7fffffu) == 0;
    }
    __device__ __forceinline__ float operator()(float x) const { return exact ? x * inv : x / s; }
};

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

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.f;   // Inf and NaN do not move a scale
}

// One unit: the new tokens of one page, one KV head, keys or values, by kLanes threads (a
// warp, or the block) of which `lane` is this one.
template <int D, int DT, int kLanes>
__device__ __forceinline__ void append_page(const AppendParams& p, const NewTokens& t, int b, int nth_page, int head,
                                            bool is_v, int lane, float* red) {
    constexpr int kUnits = D / 16;
    constexpr int kRows = kLanes / kUnits;
    const int first_page = t.start / p.P;
    const int page_pos = (first_page + nth_page) * p.P;                  // position of the page's first slot
    const int slot0 = nth_page == 0 ? t.start - page_pos : 0;
    const int pos0 = page_pos + slot0;
    const int row0 = t.first + (pos0 - t.start);
    int n = min(p.P - slot0, t.start + t.n - pos0);
    if (p.rope != DA_ROPE_NONE && pos0 + n > p.max_pos) {
        if (lane == 0) flag_error(p.err, DA_DEVERR_POSITION);
        n = p.max_pos - pos0;
        if (n <= 0) return;
    }
    const int page = ld_cg_s32(p.table + static_cast<int64_t>(b) * p.table_stride + first_page + nth_page);
    if (page < 0 || page >= p.num_pages) {
        if (lane == 0) flag_error(p.err, DA_DEVERR_PAGE);
        return;
    }
    const int u = lane % kUnits, r0 = lane / kUnits;
    int da, db;
    unit_dims(p, u, da, db);
    const bool turns = !is_v && p.rope != DA_ROPE_NONE && 16 * u < p.rot;
    const uint16_t* src = (is_v ? p.v : p.k) + static_cast<int64_t>(head) * D;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    float* scale_at = (is_v ? p.vs : p.ks) + static_cast<int64_t>(page) * p.Hkv + head;
    uint8_t* cache = is_v ? p.vc : p.kc;
    const float before = slot0 == 0 ? 0.f : *reinterpret_cast<volatile float*>(scale_at);

    auto load_row = [&](int r, Chunk16& e) {
        const uint16_t* at = src + static_cast<int64_t>(row0 + r) * stride;
        unpack8<DT>(*reinterpret_cast<const uint4*>(at + da), e.a);
        unpack8<DT>(*reinterpret_cast<const uint4*>(at + db), e.b);
        if (turns) {
            Turn turn;
            load_turn(turn, p.cos_sin, p.rot, pos0 + r, u);
            rotate(e, turn, p.rope == DA_ROPE_HALF);
        }
    };
    float amax = 0.f;
    for (int r = r0; r < n; r += kRows) {
        Chunk16 e;
        load_row(r, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(finite_abs(e.a[i]), finite_abs(e.b[i])));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if constexpr (kLanes > 32) {
        if ((lane & 31) == 0) red[lane >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kLanes / 32; ++w) amax = fmaxf(amax, red[w]);
        __syncthreads();   // `red` is free for the next unit
    } else {
        __syncwarp();
    }
    // every thread has read `before` by now
    const float scale = fmaxf(before, needed_scale(amax));
    if (lane == 0 && scale != before) *scale_at = scale;
    const Divide over(scale);
    if (scale > before && slot0 > 0) {
        const float by = before / scale;
        const int chunks = slot0 * (D / 16);
        for (int i = lane; i < chunks; i += kLanes) {
            uint4* at = reinterpret_cast<uint4*>(
                cache + page_row(p.layout, page, i / (D / 16), head, p.P, p.Hkv) * D + (i % (D / 16)) * 16);
            uint4 w = *at;
            w.x = scale_e4m3x4(w.x, by);
            w.y = scale_e4m3x4(w.y, by);
            w.z = scale_e4m3x4(w.z, by);
            w.w = scale_e4m3x4(w.w, by);
            *at = w;
        }
    }
    for (int r = r0; r < n; r += kRows) {
        Chunk16 e;
        load_row(r, e);
        uint8_t* at = cache + page_row(p.layout, page, slot0 + r, head, p.P, p.Hkv) * D;
        *reinterpret_cast<uint2*>(at + da) =
            make_uint2(to_e4m3x4(over(e.a[0]), over(e.a[1]), over(e.a[2]), over(e.a[3])),
                       to_e4m3x4(over(e.a[4]), over(e.a[5]), over(e.a[6]), over(e.a[7])));
        *reinterpret_cast<uint2*>(at + db) =
            make_uint2(to_e4m3x4(over(e.b[0]), over(e.b[1]), over(e.b[2]), over(e.b[3])),
                       to_e4m3x4(over(e.b[4]), over(e.b[5]), over(e.b[6]), over(e.b[7])));
    }
}

// The page blocks come first (gridDim.x - row_blocks of them): units (touched page, KV head,
// keys or values) of all sequences, head fastest. kLanes = 32: a warp per unit.
template <int D, int DT, int kLanes>
__global__ void __launch_bounds__(kAppendThreads) append8_kernel(const AppendParams p) {
    extern __shared__ int32_t append_smem[];
    __shared__ int32_t warp_sum[kAppendThreads / 32];
    __shared__ float red[kAppendThreads / 32];
    int32_t* cu = append_smem;
    int32_t* lens = cu + p.B + 1;
    int32_t* prefix = lens + p.B;      // touched pages before sequence b, [B + 1]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    if (tid == 0) grid_dependents_launch();
    stage_sequences(p, cu, lens);
    const int page_blocks = static_cast<int>(gridDim.x) - p.row_blocks;
    if (static_cast<int>(blockIdx.x) >= page_blocks) {
        append_rows<D, DT, false>(p, cu, lens, blockIdx.x - page_blocks, p.row_blocks);
        return;
    }
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
    const int64_t units = static_cast<int64_t>(prefix[p.B]) * p.Hkv * 2;
    constexpr int kPerBlock = kAppendThreads / kLanes;
    const int64_t step = static_cast<int64_t>(page_blocks) * kPerBlock;
    // with kLanes = 32 the bound is uniform over a warp, with a block per unit over the block
    for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kPerBlock + (kLanes == 32 ? warp : 0); unit < units;
         unit += step) {
        const int hv = static_cast<int>(unit % (2 * p.Hkv));
        const int nth = static_cast<int>(unit / (2 * p.Hkv));
        int lo = 0, hi = p.B - 1;   // last b with prefix[b] <= nth
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= nth) lo = mid;
            else hi = mid - 1;
        }
        append_page<D, DT, kLanes>(p, new_tokens(p, cu[lo], cu[lo + 1], lens[lo]), lo, nth - prefix[lo], hv >> 1,
                                   (hv & 1) != 0, kLanes == 32 ? lane : tid, red);
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

constexpr int kAppendGrid = 152 * 8;   // one wave of 256-thread blocks

template <int D, int DT>
da_status run_append(AppendParams& p, bool e4m3, cudaStream_t stream) {
    constexpr int kUnits = D / 16;
    // One token per block while that still fills the GPU's blocks; more of them share one
    // as the batch grows, so that a thread reuses its cosines over more heads.
    p.tokens_per_block = 1;
    while (p.tokens_per_block < kAppendThreads / kUnits / 4 && p.T / (2 * p.tokens_per_block) >= kAppendGrid)
        p.tokens_per_block *= 2;
    const int rows = std::min((p.T + p.tokens_per_block - 1) / p.tokens_per_block, kAppendGrid);
    if (!e4m3) {
        p.row_blocks = rows;
        return launch_append(append16_kernel<D, DT>, rows, (2 * p.B + 1) * sizeof(int32_t), p, stream);
    }
    p.row_blocks = p.Hq > 0 ? rows : 0;
    // A warp per (page, head) while pages get few tokens each, the block where they get many.
    const bool few = p.T < 4 * static_cast<int64_t>(p.B) || p.P <= 16;
    const int64_t touched = std::min<int64_t>(p.T, p.T / p.P + 2ll * p.B);
    const int64_t units = touched * p.Hkv * 2;
    const int blocks = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>(few ? (units + kAppendThreads / 32 - 1) / (kAppendThreads / 32) : units, kAppendGrid)));
    const size_t smem = (3 * p.B + 2) * sizeof(int32_t);
    return few ? launch_append(append8_kernel<D, DT, 32>, blocks + p.row_blocks, smem, p, stream)
               : launch_append(append8_kernel<D, DT, kAppendThreads>, blocks + p.row_blocks, smem, p, stream);
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
    p.tokens_per_block = 1;
    p.row_blocks = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool e4m3 = c.kv_dtype == DA_E4M3;
    if (c.D == 128)
        return a.dtype == DA_F16 ? run_append<128, DA_F16>(p, e4m3, s) : run_append<128, DA_BF16>(p, e4m3, s);
    return a.dtype == DA_F16 ? run_append<64, DA_F16>(p, e4m3, s) : run_append<64, DA_BF16>(p, e4m3, s);
}
