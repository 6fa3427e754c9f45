// cache_plan.hpp -- how the workgroups of the cached attention share its work,
// for the kernel and for tests on the host.
//
// The host does not know the lengths (they change between replays of a graph),
// so the grid is fixed and each workgroup finds its own share.  A unit is the
// attention of 16 query heads (or fewer) of one key-value head of one rank over
// one sequence; its work comes in steps of `step` tokens, at least one, so that
// an empty sequence is visited too.  All units' steps stand in one row, unit
// group (rank, key-value head, query tile) after unit group and sequence after
// sequence, and are cut into equal shares of whole steps.  A share's first and
// last piece may be parts of a unit: such a piece's sums wait in the
// workspace, and the last of the unit's workgroups to arrive joins them.
// Shares that are equal whatever the lengths are keep a batch of one long and
// many short sequences as balanced as one of equal ones.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ar {

// a / b; the 32-bit quotient is several times cheaper.
__host__ __device__ inline uint64_t divide(uint64_t a, uint64_t b)
{
    if (((a | b) >> 32) == 0)
        return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// The tokens of a sequence that are attended to: [first, end).  False where the
// length is none.
__host__ __device__ inline bool attended(int32_t length, uint64_t capacity, uint64_t window,
                                         uint32_t *first, uint32_t *end)
{
    *first = *end = 0;
    if (length < 0 || (uint64_t)length > capacity)
        return false;
    *end = (uint32_t)length;
    if (window != 0 && (uint64_t)length > window)
        *first = (uint32_t)(length - (int64_t)window);
    return true;
}

__host__ __device__ inline uint32_t steps_of(uint32_t first, uint32_t end, uint32_t step)
{
    const uint32_t n = end - first;
    return n == 0 ? 1u : (n - 1u) / step + 1u;
}

// `total` steps over `sharers` workgroups, of which the first `extra` take one
// more than `per`.
struct CachePlan {
    uint64_t per;
    uint32_t extra, sharers;
    __host__ __device__ CachePlan(uint64_t total, uint32_t grid, uint32_t least)
    {
        const uint64_t most = divide(total + least - 1u, least);
        sharers = most < grid ? (uint32_t)most : grid;
        per = divide(total, sharers);
        extra = (uint32_t)(total - per * sharers);
    }
    __host__ __device__ uint64_t start(uint32_t w) const
    {
        return w * per + (w < extra ? w : extra);
    }
    // The workgroup whose share holds step i.
    __host__ __device__ uint32_t owner(uint64_t i) const
    {
        const uint64_t cut = (per + 1u) * extra;
        return (uint32_t)(i < cut ? divide(i, per + 1u) : extra + divide(i - cut, per));
    }
    // The share of workgroup `block` of the grid, or ~0: none.  Workgroup b runs on
    // XCD b % 8; shares that follow one another lie on one XCD, and few shares on
    // all of them.
    __host__ __device__ uint32_t share(uint32_t block) const
    {
        const uint32_t each = (sharers + 7u) / 8u, w = block % 8u * each + block / 8u;
        return block / 8u < each && w < sharers ? w : ~0u;
    }
};

// The workspace: counters first, then two slots of partial sums a workgroup, one
// for the unit that its share begins inside, one for the unit that it ends inside.
// Partial sums are joined in two steps, 16 consecutive workgroups first, so that
// one long sequence is not joined by one workgroup alone.
constexpr uint32_t kJoinGroup = 16;
struct CacheJoin {
    uint32_t w0, w1;  // the unit's first and last workgroup
    __host__ __device__ uint32_t slot(uint32_t w) const { return 2u * w + (w == w0 ? 1u : 0u); }
    // The group of w: its first and last member.
    __host__ __device__ uint32_t first(uint32_t w) const
    {
        const uint32_t g = w / kJoinGroup * kJoinGroup;
        return g > w0 ? g : w0;
    }
    __host__ __device__ uint32_t last(uint32_t w) const
    {
        const uint32_t g = w / kJoinGroup * kJoinGroup + kJoinGroup - 1u;
        return g < w1 ? g : w1;
    }
    __host__ __device__ uint32_t groups() const { return w1 / kJoinGroup - w0 / kJoinGroup + 1u; }
    // A workgroup begins at most one group inside its share (its last piece's unit
    // starts there) and one as the first of 16; and at most one unit.
    __host__ __device__ uint32_t group_counter(uint32_t w) const
    {
        const uint32_t f = first(w);
        return 4u * f + (f == w0 ? 0u : 1u);
    }
    __host__ __device__ uint32_t unit_counter() const { return 4u * w0 + 2u; }
};

}  // namespace ar
