// Decode attention over a paged KV cache with a sliding window and first tokens that stay
// visible (the kernel: paged_attn.cuh).

#include "paged_attn.cuh"

using namespace da_impl;

extern "C" da_status decode_attn_paged_window(const da_paged_attn* args, int window, int sinks, void* stream) {
    if (window < 1 || sinks < 0) return DA_ERR_INVALID_ARG;
    return attend<true>(args, window, sinks, stream);
}
