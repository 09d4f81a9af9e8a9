// Attention of a chunk of new tokens of each sequence over the paged KV cache
// (decode_attn_paged.h): a warp per (token, query head), in one pass over the keys that the
// token sees with a running maximum m,
//
//     x_j = scale * ks * (q . k_j),   out = sum_j e^(x_j - m) vs v_j / sum_j e^(x_j - m).
//
// A lane holds D / 32 dims of the query and of the accumulator. All of it is float32.

#include "paged_common.cuh"

namespace da_impl {

constexpr int kRowWarps = 8;

struct ChunkParams {
    const uint16_t* q;
    const uint8_t *k, *v;
    const float *ks, *vs;
    const int32_t *cu, *lens, *table;
    uint16_t* out;
    float* lse;              // or nullptr
    uint32_t* err;
    int64_t q_stride, out_stride;
    int B, T, Hq, Hkv, G, P, max_pages, table_stride, num_pages, layout, window, sinks;
    float scale;
};

template <int D, int DT, bool KV8>
__global__ void __launch_bounds__(kRowWarps * 32) chunk_row_kernel(const ChunkParams p) {
    constexpr int kDims = D / 32;
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_dependents_launch();
    const int lane = threadIdx.x & 31;
    const int64_t warp = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kRowWarps;
    auto element = [&](const uint8_t* base, int64_t at) {
        if constexpr (KV8) {
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(base[at])));
            return bits_to_f32<DA_F16>(h2 & 0xffffu);
        } else {
            return bits_to_f32<DT>(reinterpret_cast<const uint16_t*>(base)[at]);
        }
    };
    for (int b = 0; b < p.B; ++b) {
        const int r0 = ld_cg_s32(p.cu + b), r1 = ld_cg_s32(p.cu + b + 1);
        if (r0 < 0 || r1 < r0 || r1 > p.T) {
            if (lane == 0) flag_error(p.err, DA_DEVERR_SEQLENS);
            continue;
        }
        int L = ld_cg_s32(p.lens + b);
        if (L < 0 || L > static_cast<int64_t>(p.max_pages) * p.P) {
            if (lane == 0) flag_error(p.err, DA_DEVERR_SEQLENS);
            L = 0;
        }
        for (int64_t i = warp; i < static_cast<int64_t>(r1 - r0) * p.Hq; i += warps) {
            const int t = static_cast<int>(i / p.Hq), h = static_cast<int>(i - static_cast<int64_t>(t) * p.Hq), kvh = h / p.G;
            const int pos = L - (r1 - r0) + t;
            const int low = p.window ? max(0, pos - p.window + 1) : 0, sinks = min(p.sinks, low);
            float q[kDims], acc[kDims], m = -INFINITY, l = 0.f;
#pragma unroll
            for (int d = 0; d < kDims; ++d) {
                q[d] = bits_to_f32<DT>(p.q[(r0 + t) * p.q_stride + static_cast<int64_t>(h) * D + 32 * d + lane]);
                acc[d] = 0.f;
            }
            for (int j = 0; j <= pos; ++j) {
                if (j == sinks) j = low;
                const int page = ld_cg_s32(p.table + static_cast<int64_t>(b) * p.table_stride + j / p.P);
                const bool good = page >= 0 && page < p.num_pages;
                if (!good && lane == 0) flag_error(p.err, DA_DEVERR_PAGE);
                const int64_t at = page_row(p.layout, good ? page : 0, j % p.P, kvh, p.P, p.Hkv) * D + lane;
                float x = 0.f, ks = 1.f, vs = 1.f;
                if constexpr (KV8) {
                    ks = good ? p.ks[static_cast<int64_t>(page) * p.Hkv + kvh] : 0.f;
                    vs = good ? p.vs[static_cast<int64_t>(page) * p.Hkv + kvh] : 0.f;
                }
#pragma unroll
                for (int d = 0; d < kDims; ++d) x = fmaf(q[d], good ? element(p.k, at + 32 * d) : 0.f, x);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
                x *= p.scale * ks;
                const float top = fmaxf(m, x), none = top == -INFINITY ? 0.f : top;
                const float old = expf(m - none), w = expf(x - none);
                m = top;
                l = fmaf(l, old, w);
#pragma unroll
                for (int d = 0; d < kDims; ++d)
                    acc[d] = fmaf(acc[d], old, good ? w * (vs * element(p.v, at + 32 * d)) : 0.f);
            }
            const bool none = m == -INFINITY && l == 0.f;
            const int64_t row = (r0 + t) * p.out_stride + static_cast<int64_t>(h) * D;
#pragma unroll
            for (int d = 0; d < kDims; ++d) p.out[row + 32 * d + lane] = to_bits<DT>(none ? 0.f : acc[d] / l);
            if (p.lse != nullptr && lane == 0)
                p.lse[static_cast<int64_t>(r0 + t) * p.Hq + h] = none ? -INFINITY : m + logf(l);
        }
    }
}

template <int D, int DT, bool KV8>
da_status launch_chunk(const ChunkParams& p, cudaStream_t stream) {
    cudaLaunchAttribute attrs[1] = {pdl_attr()};
    cudaLaunchConfig_t cfg = {};
    const int64_t rows = static_cast<int64_t>(p.T) * p.Hq;
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(152 * 8, (rows + kRowWarps - 1) / kRowWarps)));
    cfg.blockDim = dim3(kRowWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, chunk_row_kernel<D, DT, KV8>, p) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

template <int D, int DT>
da_status launch_chunk_any(const ChunkParams& p, bool kv8, cudaStream_t s) {
    return kv8 ? launch_chunk<D, DT, true>(p, s) : launch_chunk<D, DT, false>(p, s);
}

}  // namespace da_impl

using namespace da_impl;

extern "C" {

size_t decode_attn_paged_chunk_workspace_size(int Hq, int Hkv, int D) {
    if (Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
    return kPagedHeadBytes;
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
    // rows of the accumulators' tiles, one per (token, head of a group)
    if (static_cast<int64_t>(a.T_new) * (a.Hq / c.Hkv) > 0x3fffffffll) return DA_ERR_INVALID_ARG;
    if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.lse, 4)) return DA_ERR_ALIGNMENT;
    if (a.workspace_bytes < decode_attn_paged_chunk_workspace_size(a.Hq, c.Hkv, c.D)) return DA_ERR_WORKSPACE_TOO_SMALL;
    if (a.T_new == 0) return DA_OK;
    if (!a.q || !a.out) return DA_ERR_INVALID_ARG;
    ChunkParams p;
    p.q = static_cast<const uint16_t*>(a.q);
    p.k = static_cast<const uint8_t*>(c.k);
    p.v = static_cast<const uint8_t*>(c.v);
    p.ks = c.k_scale;
    p.vs = c.v_scale;
    p.cu = a.cu_new;
    p.lens = a.kv_lens;
    p.table = a.block_table;
    p.out = static_cast<uint16_t*>(a.out);
    p.lse = a.lse;
    p.err = static_cast<uint32_t*>(a.workspace);
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.B = a.B;
    p.T = a.T_new;
    p.Hq = a.Hq;
    p.Hkv = c.Hkv;
    p.G = a.Hq / c.Hkv;
    p.P = c.page_size;
    p.max_pages = a.max_pages;
    p.table_stride = a.table_stride;
    p.num_pages = c.num_pages;
    p.layout = c.layout;
    p.window = a.window;
    p.sinks = a.sinks;
    p.scale = a.scale;
    const bool kv8 = c.kv_dtype == DA_E4M3;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (c.D == 128) return a.dtype == DA_F16 ? launch_chunk_any<128, DA_F16>(p, kv8, s) : launch_chunk_any<128, DA_BF16>(p, kv8, s);
    return a.dtype == DA_F16 ? launch_chunk_any<64, DA_F16>(p, kv8, s) : launch_chunk_any<64, DA_BF16>(p, kv8, s);
}

}  // extern "C"
