// Pieces shared by the paged-cache translation units (paged_*.cu): what a workspace begins with, the checks of a
// cache description, where a page's rows lie, waits and conversions of the kernels, the tensor maps of the pages.
#ifndef DECODE_ATTN_PAGED_COMMON_CUH
#define DECODE_ATTN_PAGED_COMMON_CUH

#include "decode_attn_paged.h"
#include "split_common.cuh"

namespace da_impl {

constexpr size_t kPagedHeaderBytes = kHeaderBytes;
constexpr int kPagedShares = 2048;   // decode attention: bound of shares (range, KV head, chunk), each with two partial results
constexpr int kWriters = 4;          // consumer warps that write a piece's columns, two of every eight each
constexpr size_t kPagedCounterBytes = static_cast<size_t>(kPagedShares) * kWriters * 4;
// what workspace_init clears: every workspace begins so, whichever call it is for, so that one can serve them all
constexpr size_t kPagedHeadBytes = kPagedHeaderBytes + kPagedCounterBytes;

constexpr float kNoKey = -3.402823466e38f;   // running maximum of a row that has seen no key: the least finite value,
                                             // so that every finite score is above it and no NaN arises

// Host checks of a cache description and of the block table's geometry, for calls
// whose queries and new tokens are `dt`.
inline da_status check_cache(const da_paged_cache* c, int dt, const int32_t* kv_lens, const int32_t* table,
                             int max_pages, int table_stride, int B, int Hq) {
    if (!c) return DA_ERR_INVALID_ARG;
    if (dt != DA_F16 && dt != DA_BF16) return DA_ERR_INVALID_ARG;
    if (c->kv_dtype != DA_E4M3 && c->kv_dtype != dt) return DA_ERR_INVALID_ARG;
    if (c->layout != DA_LAYOUT_VARLEN && c->layout != DA_LAYOUT_BHSD) return DA_ERR_INVALID_ARG;
    if (c->D != 64 && c->D != 128) return DA_ERR_UNSUPPORTED;
    if (c->num_pages < 1 || c->Hkv < 1 || c->page_size < 16 || c->page_size > DA_MAX_PAGE_SIZE || c->page_size % 16)
        return DA_ERR_INVALID_ARG;
    // rows and (page, head) slabs are int32 coordinates of the tensor maps, with room for a
    // coordinate past the end
    if (static_cast<int64_t>(c->num_pages) * c->page_size > 0x7fffff00ll ||
        static_cast<int64_t>(c->num_pages) * c->Hkv > 0x7fffff00ll)
        return DA_ERR_INVALID_ARG;
    if (B < 1 || Hq < 0 || Hq % c->Hkv != 0 || max_pages < 1 || table_stride < max_pages) return DA_ERR_INVALID_ARG;
    if (B > DA_MAX_PAGED_BATCH) return DA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_pages) * c->page_size > 0x7fffff00ll) return DA_ERR_INVALID_ARG;
    if (!c->k || !c->v || !kv_lens || !table) return DA_ERR_INVALID_ARG;
    if (c->kv_dtype == DA_E4M3 && (!c->k_scale || !c->v_scale)) return DA_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(kv_lens, 4) || !aligned(table, 4)) return DA_ERR_ALIGNMENT;
    if (c->kv_dtype == DA_E4M3 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))) return DA_ERR_ALIGNMENT;
    return DA_OK;
}

// Row (of D elements) of a page's slot and head in k or v.
__device__ __forceinline__ int64_t page_row(int layout, int page, int slot, int head, int page_size, int Hkv) {
    return layout == DA_LAYOUT_VARLEN ? (static_cast<int64_t>(page) * page_size + slot) * Hkv + head
                                      : (static_cast<int64_t>(page) * Hkv + head) * page_size + slot;
}

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

// log2 of a scale, a subnormal one too (-inf of 0).
__device__ __forceinline__ float log2_of_scale(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two e4m3 values to two fp16 values (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
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

}  // namespace da_impl

#endif
