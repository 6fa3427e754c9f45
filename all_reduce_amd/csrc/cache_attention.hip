// cache_attention.hip -- the choice among the cached attention's kernel families
// (cache_attention.hpp) and the size of its workspace.
#include "cache_attention.hpp"

namespace ar {

// Counters, in the same place whatever call uses the workspace, then two slots a team.
// (A wave that is a team has at most 32 queries, four together at most 128.  Heads above 128
// have half the workgroups, and a little less than twice as many floats a query.)
uint64_t cache_attention_workspace(uint32_t dim, uint32_t group, int cu_count)
{
    const uint32_t dp = padded_dim(dim), queries = group < 32u ? group : 32u;
    auto floats = [&](int per_cu, uint32_t padded) {
        return (uint64_t)attend_most(per_cu, cu_count) * kAttendWaves * 2u * queries * (padded + 2u);
    };
    uint64_t most = floats(2, dp < 128 ? dp : 128);
    if (dp == 256 && floats(1, dp) > most)
        most = floats(1, dp);
    return AR_CACHE_WORKSPACE_ZEROS + most * sizeof(float);
}

// 16 query heads a wave, or 32 where a key-value head has more: the keys and values in
// registers then serve twice as many (32 windows of 4096 tokens x 4 ranks, 32 query heads
// of 256: 114 us in place of 120; 64 x 8192 tokens x 8 ranks, 32 of 128: 327 in place of
// 416).  Float32 heads of 256 leave no registers for that.
uint32_t attend_queries(uint32_t group, int dtype, uint32_t dim)
{
    return group <= 16u || (dtype == kFp32 && padded_dim(dim) == 256) ? 4u : 5u;
}

hipError_t launch_cache_attention(const CacheAttentionArgs &args, int dtype, bool eight,
                                  bool eight_out, int cu_count, hipStream_t stream)
{
    auto typed = [&](auto type) {
        typedef decltype(type) T;
        if (attend_queries(args.group, dtype, args.cache.dim) == 4u)
            return eight ? launch_attend<T, true, 1>(args, eight_out, cu_count, stream)
                         : launch_attend<T, false, 1>(args, eight_out, cu_count, stream);
        return eight ? launch_attend<T, true, 2>(args, eight_out, cu_count, stream)
                     : launch_attend<T, false, 2>(args, eight_out, cu_count, stream);
    };
    switch (dtype) {
    case kBf16: return typed(Bf16{});
    case kFp16: return typed(Fp16{});
    default: return typed(Fp32{});
    }
}

}  // namespace ar
