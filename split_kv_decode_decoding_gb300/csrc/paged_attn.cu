// Decode attention over a paged KV cache (decode_attn_paged.h): a warp per query row.
//
// Each lane owns D / 32 dims of the row; per key one dot product by shuffles and one step of
// the online softmax in the exp2 domain, float32 throughout.

#include "paged_common.cuh"

namespace da_impl {

constexpr int kPagedShares = 2048;   // bound of the workspace's partial results

struct PagedParams {
    const uint16_t* q;
    const uint8_t* k;
    const uint8_t* v;
    const float* ks;
    const float* vs;
    const int32_t* lens;
    const int32_t* table;
    uint16_t* out;
    float* lse;
    uint32_t* err;
    int B, tq, Hq, Hkv, P, max_pages, table_stride, num_pages, layout;
    float scale_log2;
};

template <int DT, bool KV8>
__device__ __forceinline__ float element(const uint8_t* base, int64_t i) {
    if constexpr (KV8) {
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(base[i])));
        return bits_to_f32<DA_F16>(h2 & 0xffffu);
    } else {
        return bits_to_f32<DT>(reinterpret_cast<const uint16_t*>(base)[i]);
    }
}

template <int D, int DT, bool KV8>
__global__ void __launch_bounds__(128) paged_kernel(const PagedParams p) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= static_cast<int64_t>(p.B) * p.tq * p.Hq) return;
    const int h = static_cast<int>(row % p.Hq), t = static_cast<int>(row / p.Hq % p.tq);
    const int b = static_cast<int>(row / p.Hq / p.tq), kvh = h / (p.Hq / p.Hkv);
    int L = p.lens[b];
    if (L < 0 || L > static_cast<int64_t>(p.max_pages) * p.P) {
        if (lane == 0) flag_error(p.err, DA_DEVERR_SEQLENS);
        L = 0;
    }
    const int seen = min(L, L - p.tq + t + 1);
    constexpr int kDims = D / 32;
    float q[kDims], acc[kDims], m = -INFINITY, l = 0.f;
    for (int i = 0; i < kDims; ++i) {
        q[i] = bits_to_f32<DT>(p.q[row * D + i * 32 + lane]);
        acc[i] = 0.f;
    }
    for (int j = 0; j < seen; ++j) {
        const int page = p.table[static_cast<int64_t>(b) * p.table_stride + j / p.P];
        const bool good = page >= 0 && page < p.num_pages;
        if (!good && lane == 0) flag_error(p.err, DA_DEVERR_PAGE);
        const int64_t at = page_row(p.layout, good ? page : 0, j % p.P, kvh, p.P, p.Hkv) * D;
        const int64_t sc = static_cast<int64_t>(good ? page : 0) * p.Hkv + kvh;
        float dot = 0.f;
        for (int i = 0; i < kDims; ++i) dot += good ? q[i] * element<DT, KV8>(p.k, at + i * 32 + lane) : 0.f;
        for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        const float x = dot * p.scale_log2 * (KV8 ? p.ks[sc] : 1.f);
        const float mn = fmaxf(m, x);
        const float w = fast_exp2(x - mn), al = fast_exp2(m - mn);
        m = mn;
        l = l * al + w;
        for (int i = 0; i < kDims; ++i)
            acc[i] = acc[i] * al + (good ? w * element<DT, KV8>(p.v, at + i * 32 + lane) * (KV8 ? p.vs[sc] : 1.f) : 0.f);
    }
    for (int i = 0; i < kDims; ++i) p.out[row * D + i * 32 + lane] = to_bits<DT>(seen > 0 ? acc[i] / l : 0.f);
    if (p.lse && lane == 0) p.lse[row] = seen > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <int D, int DT, bool KV8>
da_status launch_paged(const PagedParams& p, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.tq * p.Hq;
    paged_kernel<D, DT, KV8><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

template <int D, int DT>
da_status launch_paged_kv(const PagedParams& p, bool e4m3, cudaStream_t s) {
    return e4m3 ? launch_paged<D, DT, true>(p, s) : launch_paged<D, DT, false>(p, s);
}

}  // namespace da_impl

using namespace da_impl;

extern "C" {

size_t decode_attn_paged_workspace_size(int T_q, int Hq, int Hkv, int D) {
    if (T_q < 1 || T_q > DA_MAX_QUERY_TOKENS || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
    const int cols = item_cols(static_cast<int64_t>(Hq / Hkv) * T_q);
    return kPagedHeaderBytes + kPagedShares * 16 + static_cast<size_t>(2 * kPagedShares) * cols * (D + 1) * 4;
}

da_status decode_attn_paged_workspace_init(void* workspace, size_t workspace_bytes, void* stream) {
    const size_t head = kPagedHeaderBytes + kPagedShares * 16;
    if (!workspace || workspace_bytes < head) return DA_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return DA_ERR_ALIGNMENT;
    return cudaMemsetAsync(workspace, 0, head, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

da_status decode_attn_paged(const void* q, const da_paged_cache* cache, const int32_t* kv_lens,
                            const int32_t* block_table, int max_pages, int table_stride, int B, int T_q, int Hq,
                            da_dtype dtype, float scale, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream) {
    da_status st = check_cache(cache, dtype, kv_lens, block_table, max_pages, table_stride, B, Hq);
    if (st != DA_OK) return st;
    const da_paged_cache& c = *cache;
    if (Hq < 1 || T_q < 1 || T_q > DA_MAX_QUERY_TOKENS || !std::isfinite(scale)) return DA_ERR_INVALID_ARG;
    if (!q || !out || !workspace) return DA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(B) * T_q * Hq * c.D > 0x7fffffffll) return DA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 256)) return DA_ERR_ALIGNMENT;
    if (workspace_bytes < decode_attn_paged_workspace_size(T_q, Hq, c.Hkv, c.D)) return DA_ERR_WORKSPACE_TOO_SMALL;
    PagedParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint8_t*>(c.k);
    p.v = static_cast<const uint8_t*>(c.v);
    p.ks = c.k_scale;
    p.vs = c.v_scale;
    p.lens = kv_lens;
    p.table = block_table;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.err = static_cast<uint32_t*>(workspace);
    p.B = B;
    p.tq = T_q;
    p.Hq = Hq;
    p.Hkv = c.Hkv;
    p.P = c.page_size;
    p.max_pages = max_pages;
    p.table_stride = table_stride;
    p.num_pages = c.num_pages;
    p.layout = c.layout;
    p.scale_log2 = scale * kLog2e;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool e4m3 = c.kv_dtype == DA_E4M3;
    if (c.D == 128)
        return dtype == DA_F16 ? launch_paged_kv<128, DA_F16>(p, e4m3, s) : launch_paged_kv<128, DA_BF16>(p, e4m3, s);
    return dtype == DA_F16 ? launch_paged_kv<64, DA_F16>(p, e4m3, s) : launch_paged_kv<64, DA_BF16>(p, e4m3, s);
}

}  // extern "C"
