// twell_kv.cuh -- the device view of a paged key-value cache (twell_kv_cache in twell.h).
#pragma once

#include "twell_common.cuh"

namespace twell {

struct KvView {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int64_t page_stride, head_stride, token_stride;  // elements
    int64_t scale_page, scale_head;                  // floats; a page's tokens are adjacent
    int n_pages, page_shift, heads, hd, q8;

    // First element of the row of `slot` (page * page_size + offset) and `head`; 64-bit throughout.
    __device__ __forceinline__ int64_t row(int slot, int head) const
    {
        return (slot >> page_shift) * page_stride + head * head_stride +
               (slot & ((1 << page_shift) - 1)) * token_stride;
    }
    __device__ __forceinline__ int64_t scale_row(int slot, int head) const
    {
        return (slot >> page_shift) * scale_page + head * scale_head + (slot & ((1 << page_shift) - 1));
    }
};

}  // namespace twell

namespace twell_host {
// Validate a cache descriptor (twell_kv.cu) and make its device view.
twell_status check_kv(const twell_kv_cache* c, twell::KvView* out);
}  // namespace twell_host
