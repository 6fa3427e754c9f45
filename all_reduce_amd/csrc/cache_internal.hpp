// cache_internal.hpp -- what the entry points of ar_cache.h and their kernel
// files share.
#pragma once

#include "ar_cache.h"
#include "ar_internal.hpp"

namespace ar {

// A cache's layout as the kernels take it: strides in elements.
struct CacheShape {
    uint64_t page_stride, head_stride, token_stride;
    uint32_t pages, page_tokens;
    uint32_t heads;
    uint32_t dim;
    uint32_t page_mul, page_shift;  // see set_division

    // t / page_tokens for t below 2^31 is (t * mul) >> (32 + shift), with mul the
    // quotient 2^(31 + s) / page_tokens rounded up, 2^s the power of two from
    // page_tokens on and shift = s - 1: mul * page_tokens exceeds 2^(31 + s) by at
    // most 2^s, which t below 2^31 does not raise to a whole.
    void set_division()
    {
        uint32_t s = 0;
        while (((uint64_t)1 << s) < page_tokens)
            ++s;
        page_mul = s == 0 ? 0 : (uint32_t)(((uint64_t)1 << (31 + s)) / page_tokens + 1);
        page_shift = s == 0 ? 0 : s - 1;
    }
    __host__ __device__ uint32_t page_of(uint32_t t) const
    {
        return page_mul == 0 ? t : (uint32_t)((uint64_t)t * page_mul >> 32) >> page_shift;
    }
    // Element offset of place `o` of page `p` of a head.
    __host__ __device__ uint64_t at(uint32_t p, uint32_t o, uint32_t head) const
    {
        return p * page_stride + o * token_stride + head * head_stride;
    }
    // The same among the scales.
    __host__ __device__ uint64_t scale_at(uint32_t p, uint32_t o, uint32_t head) const
    {
        return ((uint64_t)p * heads + head) * page_tokens + o;
    }
    // A slot's page and place; false for a number that is none of the cache's.
    __host__ __device__ bool place(int64_t slot, uint32_t *p, uint32_t *o) const
    {
        if (slot < 0 || slot >= (int64_t)pages * page_tokens)
            return false;
        *p = page_of((uint32_t)slot);
        *o = (uint32_t)slot - *p * page_tokens;
        return true;
    }
};

// Rank tables by value in the kernel arguments, as in block_internal.hpp.
// arCacheWrite: from rows into pages; arCacheRead: from pages into rows.
struct CacheCopyArgs {
    char *rows[2][AR_MAX_RANKS];    // keys, values
    char *pages[2][AR_MAX_RANKS];
    float *scales[2][AR_MAX_RANKS]; // unused where the cache has the element type
    const int64_t *slots;
    CacheShape cache;
    uint64_t row_stride;            // elements
    uint32_t tokens;
};

struct CacheAttentionArgs {
    const char *q[AR_MAX_RANKS];
    const char *keys[AR_MAX_RANKS];
    const char *values[AR_MAX_RANKS];
    const float *key_scales[AR_MAX_RANKS];
    const float *value_scales[AR_MAX_RANKS];
    char *out[AR_MAX_RANKS];
    float *out_scales[AR_MAX_RANKS];  // unused without an 8-bit output
    float *lse[AR_MAX_RANKS];         // unused where has_lse is 0
    const int32_t *table;
    const int32_t *lengths;
    CacheShape cache;
    uint64_t q_stride;  // elements
    uint64_t table_pages;
    uint64_t window;    // 0: all
    char *work;         // the workspace's counters
    float *slots;       // its partial sums
    uint32_t seqs;
    uint32_t heads;     // query heads
    uint32_t group;     // of a key-value head
    uint32_t nranks;
    uint32_t has_lse;
    uint32_t passes;    // of a step, as a power of two (the launcher sets it)
    float scale;
};

// Launchers: validate nothing (the entry points did).
hipError_t launch_cache_write(const CacheCopyArgs &args, int dtype, bool eight, int nranks,
                              int cu_count, hipStream_t stream);
hipError_t launch_cache_read(const CacheCopyArgs &args, int dtype, bool eight, int nranks,
                             int cu_count, hipStream_t stream);
hipError_t launch_cache_attention(const CacheAttentionArgs &args, int dtype, bool eight,
                                  bool eight_out, int cu_count, hipStream_t stream);
// Bytes of workspace for heads of `dim`, `group` query heads to a key-value head: counters
// (AR_CACHE_WORKSPACE_ZEROS), then partial sums.
uint64_t cache_attention_workspace(uint32_t dim, uint32_t group, int cu_count);

}  // namespace ar
