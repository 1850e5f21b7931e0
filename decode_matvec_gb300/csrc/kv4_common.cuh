// Shared by the kernels around the 4-bit paged key/value cache (layout: kv4_cache in qmoe.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"

namespace kv4 {

// What the kernels need of a kv4_cache.
struct CacheView {
    unsigned char* pages;
    int n_pages;
    int page_shift;    // log2(page_size)
    int n_kv_heads;
    uint32_t head_bytes;  // one kv head of one page
    uint64_t page_bytes;
};

// Start of kv head h of a page; 64-bit, a cache may pass 2^32 bytes.
__device__ __forceinline__ unsigned char* head_ptr(const CacheView& c, int page, int h) {
    return c.pages + (uint64_t)page * c.page_bytes + (uint64_t)h * c.head_bytes;
}

// An int32, past the first-level cache where a kernel reads it ahead of its depend_wait.
template <bool kAhead>
__device__ __forceinline__ int load_i32(const int32_t* p) {
    return kAhead ? __ldcg(p) : *p;
}

// The request that query token t belongs to (q_start[b] <= t < q_start[b + 1]), or -1; with q_start[b + 1] and kv_len[b].  In a
// decode step it is t itself: that is looked at first, in one go.
template <bool kAhead>
__device__ __forceinline__ int request_of(const int32_t* q_start, const int32_t* kv_len, int B, int t, int* end, int* kv) {
    if (t < B) {
        const int s = load_i32<kAhead>(q_start + t);
        *end = load_i32<kAhead>(q_start + t + 1), *kv = load_i32<kAhead>(kv_len + t);
        if (s == t && *end == t + 1) return t;
    }
    int lo = 0, hi = B;         // the last b with q_start[b] <= t is in [lo - 1, hi - 1]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (load_i32<kAhead>(q_start + mid) <= t) lo = mid + 1;
        else hi = mid;
    }
    *end = load_i32<kAhead>(q_start + lo);
    if (lo == 0 || t >= *end) return -1;
    *kv = load_i32<kAhead>(kv_len + lo - 1);
    return lo - 1;
}

// Checks a descriptor and fills the view; `who` names the call in the message.
inline int view_of(const kv4_cache* c, const char* who, CacheView* v) {
    if (!c || !c->pages) return qmoe::fail(QMOE_EINVAL, std::string(who) + ": NULL cache");
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64)
        return qmoe::fail(QMOE_EINVAL, std::string(who) + ": page_size must be 16, 32 or 64");
    if (c->head_dim != 64 && c->head_dim != 128)
        return qmoe::fail(QMOE_EUNSUPPORTED, std::string(who) + ": head_dim must be 64 or 128");
    if (c->n_kv_heads < 1 || c->n_kv_heads > 1024 || c->n_pages < 1 ||
        (int64_t)c->n_pages * c->page_size > 0x7FFFFFFFLL)
        return qmoe::fail(QMOE_EINVAL, std::string(who) + ": n_kv_heads outside 1 .. 1024, or n_pages * page_size outside int32");
    if ((uintptr_t)c->pages & 15) return qmoe::fail(QMOE_EINVAL, std::string(who) + ": pages not 16-byte aligned");
    v->pages = (unsigned char*)c->pages;
    v->n_pages = c->n_pages;
    v->page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : 6;
    v->n_kv_heads = c->n_kv_heads;
    v->head_bytes = (uint32_t)c->page_size * (uint32_t)(c->head_dim + 8);
    v->page_bytes = (uint64_t)v->head_bytes * c->n_kv_heads;
    return QMOE_OK;
}

using qmoe::depend_launch;
using qmoe::depend_wait;
using qmoe::launch_dependent;

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace kv4
