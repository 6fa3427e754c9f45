// cache_attention.hip -- the choice among the cached attention's kernel families
// (cache_attention.hpp) and the size of its workspace.
#include "cache_attention.hpp"

namespace ar {

// Counters, in the same place whatever call uses the workspace, then two slots a team.
// (A wave that is a team has at most 16 queries, four together at most 64.)
uint64_t cache_attention_counters(int cu_count)
{
    return (uint64_t)attend_most(2, cu_count) * kAttendWaves * 4u * sizeof(uint32_t);
}

uint64_t cache_attention_workspace(uint32_t dim, uint32_t group, int cu_count)
{
    const uint64_t teams = (uint64_t)attend_most(2, cu_count) * kAttendWaves;
    const uint32_t queries = group < kTileQueries ? group : kTileQueries;
    return cache_attention_counters(cu_count) +
           teams * 2u * queries * (padded_dim(dim) + 2u) * sizeof(float);
}

hipError_t launch_cache_attention(const CacheAttentionArgs &args, int dtype, bool eight,
                                  bool eight_out, int cu_count, hipStream_t stream)
{
    switch (dtype) {
    case kBf16:
        return eight ? launch_attend<Bf16, true>(args, eight_out, cu_count, stream)
                     : launch_attend<Bf16, false>(args, eight_out, cu_count, stream);
    case kFp16:
        return eight ? launch_attend<Fp16, true>(args, eight_out, cu_count, stream)
                     : launch_attend<Fp16, false>(args, eight_out, cu_count, stream);
    default:
        return eight ? launch_attend<Fp32, true>(args, eight_out, cu_count, stream)
                     : launch_attend<Fp32, false>(args, eight_out, cu_count, stream);
    }
}

}  // namespace ar
