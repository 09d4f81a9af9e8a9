// Pieces shared by the paged-cache translation units (paged_attn.cu,
// paged_append.cu): the checks of a cache description, and where a page's rows lie.
#ifndef DECODE_ATTN_PAGED_COMMON_CUH
#define DECODE_ATTN_PAGED_COMMON_CUH

#include "decode_attn_paged.h"
#include "split_common.cuh"

namespace da_impl {

constexpr size_t kPagedHeaderBytes = kHeaderBytes;

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

}  // namespace da_impl

#endif
