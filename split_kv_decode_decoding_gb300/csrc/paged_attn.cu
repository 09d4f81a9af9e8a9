// Decode attention over all keys of a paged KV cache (the kernel: paged_attn.cuh), and its workspace.

#include "paged_attn.cuh"

using namespace da_impl;

extern "C" {

size_t decode_attn_paged_workspace_size(int T_q, int Hq, int Hkv, int D) {
    if (T_q < 1 || T_q > DA_MAX_QUERY_TOKENS || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
    const int cols = item_cols(static_cast<int64_t>(Hq / Hkv) * T_q);
    return kPagedHeadBytes + static_cast<size_t>(2 * kPagedShares) * cols * (D + 2) * 4;
}

da_status decode_attn_paged_workspace_init(void* workspace, size_t workspace_bytes, void* stream) {
    const size_t head = kPagedHeadBytes;
    if (!workspace || workspace_bytes < head) return DA_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return DA_ERR_ALIGNMENT;
    return cudaMemsetAsync(workspace, 0, head, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

da_status decode_attn_paged(const da_paged_attn* args, void* stream) { return attend<false>(args, 0, 0, stream); }

}  // extern "C"
