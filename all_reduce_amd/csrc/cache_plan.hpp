// cache_plan.hpp -- how the workgroups of the cached attention share its work,
// for the kernel and for tests on the host.
//
// The host does not know the lengths (they change between replays of a graph),
// so the grid is fixed and each team of waves finds its own share.  A unit is the
// attention of up to 16 query heads of one key-value head of one rank over one sequence
// (of up to 128 where there are more: CacheTeams); its work comes in steps of some
// tokens, at least one, so that an empty sequence is visited too.
// All units' steps stand in one row, by rank, then sequence, then key-value head and
// tile of query heads (heads that lie side by side in memory are read side by side),
// and are cut into equal shares of whole steps.  A share's first
// and last piece may be parts of a unit: such a piece's sums wait in the workspace,
// and the last of the unit's teams to arrive joins them.  Shares that are equal
// whatever the lengths are keep a batch of one long and many short sequences as
// balanced as one of equal ones.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ar {

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

// The tokens that no sequence attends to more than (lengths have 31 bits).
inline uint64_t most_attended(uint64_t capacity, uint64_t window)
{
    const uint64_t most = capacity < INT32_MAX ? capacity : INT32_MAX;
    return window != 0 && window < most ? window : most;
}

// Steps of 2^shift tokens.
__host__ __device__ inline uint32_t steps_of(uint32_t first, uint32_t end, uint32_t shift)
{
    const uint32_t n = end - first;
    return n == 0 ? 1u : ((n - 1u) >> shift) + 1u;
}

// `total` steps over `sharers` teams, of which the first `extra` take one more than
// `per`.  There are at most `teams`, a multiple of 8.
struct CachePlan {
    uint32_t per, extra, sharers;
    __host__ __device__ CachePlan(uint32_t total, uint32_t teams)
    {
        // (divisions are long chains: a call of few steps has none)
        sharers = total < teams ? total : teams;
        per = total <= teams ? 1u : total / teams;
        extra = total - per * sharers;
    }
    __host__ __device__ uint32_t start(uint32_t w) const
    {
        return w * per + (w < extra ? w : extra);
    }
    // The team whose share holds step i.
    __host__ __device__ uint32_t owner(uint32_t i) const
    {
        const uint32_t cut = (per + 1u) * extra;
        if (i < cut)
            return i / (per + 1u);
        return extra + (per == 1u ? i - cut : (i - cut) / per);
    }
    // The share of team `team` of workgroup `block`, or ~0: none.  Workgroup b runs on
    // XCD b % 8; shares that follow one another lie on one XCD, and few shares on all
    // of them, and on all their compute units before one has two.
    __host__ __device__ uint32_t share(uint32_t block, uint32_t team, uint32_t grid) const
    {
        const uint32_t each = (sharers + 7u) / 8u, i = block / 8u + team * (grid / 8u);
        const uint32_t w = block % 8u * each + i;
        return i < each && w < sharers ? w : ~0u;
    }
};

// How a launch's waves make teams.  A wave takes 16 query heads of a key-value head, or
// 32 where there are more.  Four waves of a workgroup share a unit's tokens; with more
// than 32 query heads, two or all four of them take the same tokens and 32 heads each.
// Where there are more units than workgroups, and short ones, each wave is a team, with
// longer steps: a team's way into and out of a unit is a chain of loads that four waves
// do not shorten.  On MI355X 2048 units of 33 tokens on the average (lengths from 1 to three
// times as many) take 16 us that way and 26 with four waves, of 133 tokens 36 and 46, of 200
// 51 and 60, of 333 81 and 85, but of 500 176 and 113, where a few waves have the longest
// alone.  (Of equal lengths single waves are 4 to 10 % faster up to 1000 tokens; the rule
// keeps clear of the loss.)
struct CacheTeams {
    uint32_t waves;  // of a team
    uint32_t side;   // waves that take the same tokens
    uint32_t tiles;  // of a team's query heads: units of a sequence and key-value head
    uint32_t pass;   // tokens that the team takes at once
    uint32_t shift;  // 2^shift tokens are a step
    // 2^queries and 2^tokens are a wave's; 2^passes a step's.
    __host__ __device__ CacheTeams(uint32_t group, uint32_t queries, uint32_t tokens, uint32_t passes,
                                   bool alone)
    {
        const uint32_t t = (group + (1u << queries) - 1u) >> queries;
        const uint32_t beside = alone || t == 1u ? 0u : t == 2u ? 1u : 2u, behind = alone ? 0u : 2u - beside;
        waves = alone ? 1u : 4u;
        side = 1u << beside;
        tiles = (t + side - 1u) >> beside;
        pass = 1u << (behind + tokens);
        shift = behind + tokens + passes;
    }
};

// Whether each wave is to be a team, for a batch whose sequences have `tiles` tiles of
// tokens together; and the passes of its step, a power of two that takes most sequences
// whole.
__host__ __device__ inline bool waves_alone(uint32_t tiles, uint32_t seqs)
{
    return tiles <= 8u * seqs;
}

__host__ __device__ inline uint32_t passes_alone(uint32_t tiles, uint32_t seqs)
{
    return tiles <= seqs ? 2u : tiles <= 2u * seqs ? 3u : tiles <= 4u * seqs ? 4u : 5u;
}

// How long a step of teams of four is: one pass where a team's share is many, else 2, 4
// or 8, where that leaves no more steps than teams: splitting a unit costs a joining of
// its parts (4 us on MI355X; a pass takes 1.2).  64 units of 200 tokens take 9.3 us whole
// and 10.3 in two parts, 435 of 333 tokens on the average 17.7 and 22.0.  Few units that
// are longer gain by more teams: 8 of 1000 tokens take 10.7 us in eight parts, 11.2 in four
// and 12.6 in two.
//
// This is the exponent to try for `seqs` sequences of `per` units and `steps` steps of
// one pass each; it is taken if there are no more steps than teams then.
__host__ __device__ inline uint32_t passes_to_try(uint32_t steps, uint32_t seqs, uint32_t per, uint32_t teams)
{
    const uint32_t all = steps * per;
    if (steps == seqs || (all <= teams && steps > 4u * seqs) || all > 8u * teams)
        return 0;
    return all > 4u * teams ? 3u : all > 2u * teams ? 2u : 1u;
}

// What the teams' sharing depends on besides the lengths.
struct CacheCall {
    uint32_t seqs, ranks, heads, group;
    uint32_t queries, tokens;  // 2^queries and 2^tokens are a wave's
    uint32_t passes;           // of a step, at least (passes_of_a_step)
    uint32_t grid;
    uint32_t token_bytes;      // of a key and a value of a head
};

// Whether keys and values of `tokens` tokens of all sequences together are loaded past the
// caches (non-temporal loads): where they are more than half of the last-level cache, which
// would not keep them.  64 x 8192 tokens x 8 ranks, 8 query heads of 128, take 321 in place of
// 355 us, but 256 of 67 tokens (70 MB, which the cache holds) 23.4 in place of 21.3, and 128 of
// 200 (105 MB) 34.3 in place of 29.8.  Not where several waves or units read the same tokens
// for other query heads: 136 in place of 117 us for 32 windows of 4096 tokens x 4 ranks and
// 32 query heads of 256 as two waves, 120.5 in place of 118.2 for 256 of 200 tokens x 8 ranks
// and 64 of 128 as two units.
__host__ __device__ inline bool streamed(const CacheCall &c, const CacheTeams &teams, uint64_t tokens)
{
    return teams.side == 1u && teams.tiles == 1u &&
           tokens * c.ranks * c.heads * c.token_bytes >= (uint64_t)128 << 20;
}

// How a call's waves share its work, from the lengths.  `sum_up(shift, most)` gives the steps of
// 2^shift tokens of all sequences (of one unit each), `most` of a sequence at most, as its
// member `all`, with whatever else it finds; that of the steps chosen is left in `steps`.
struct CacheChoice {
    CacheTeams teams;
    bool alone;   // each wave is a team
    bool stream;
};

template <typename SumUp, typename Steps>
__host__ __device__ inline CacheChoice choose(const CacheCall &c, SumUp sum_up, Steps *steps)
{
    CacheTeams teams(c.group, c.queries, c.tokens, c.passes, false);
    const uint32_t per = c.ranks * c.heads * teams.tiles;  // units of a sequence
    // Whole steps and tiles bound the tokens, which are summed up only where that is not enough.
    // (As many of a sequence as leave the sum 32 bits.)
    auto stream_of = [&](uint64_t bound) {
        uint32_t most = 0x80000000u;
        for (uint32_t n = 1; n < c.seqs; n *= 2u)
            most /= 2u;
        return streamed(c, teams, bound) && streamed(c, teams, sum_up(0u, most).all);
    };
    bool alone = false, stream;
    if (c.seqs * per > c.grid) {
        // (so many tiles of a sequence say enough of how long it is)
        const uint32_t tiles = sum_up(c.tokens, 0xffffu).all;
        alone = waves_alone(tiles, c.seqs);
        if (alone)
            teams = CacheTeams(c.group, c.queries, c.tokens, c.passes + passes_alone(tiles, c.seqs), true);
        stream = stream_of((uint64_t)tiles << c.tokens);
        *steps = sum_up(teams.shift, ~0u);
    } else {
        *steps = sum_up(teams.shift, ~0u);
        stream = stream_of((uint64_t)steps->all << teams.shift);
        const uint32_t more = passes_to_try(steps->all, c.seqs, per, c.grid);
        if (more != 0) {
            const Steps fewer = sum_up(teams.shift + more, ~0u);
            if (fewer.all * per <= c.grid) {
                teams.shift += more;
                *steps = fewer;
            }
        }
    }
    return {teams, alone, stream};
}

// The smallest power of two of passes to a step (as its exponent) with which all steps
// of a call can be counted in 31 bits whatever its lengths are: 0, but for calls of
// extreme sizes.  With at most 2^24 units it is at most 20 for waves of 32 tokens and 21 for
// waves of 16, and no step, at most 2^5 times longer, is more than 2^30 tokens.
inline uint32_t passes_of_a_step(uint64_t seqs, uint64_t ranks, uint64_t heads, uint32_t group,
                                 uint32_t tokens, uint64_t most_tokens)
{
    const uint64_t units = seqs * ranks * heads * ((group + 15u) / 16u);
    uint32_t passes = 0;
    while (units * ((most_tokens >> (tokens + passes)) + 1u) >= (uint64_t)1 << 31)
        ++passes;
    return passes;
}

// The workspace: counters first, then two slots of partial sums a team, one for
// the unit that its share begins inside, one for the unit that it ends inside.
// Partial sums of up to 16 teams are joined by the last of them; those of more in two
// steps, by the last of groups of consecutive teams and then by the last of the groups,
// so that one long sequence is not joined by one team alone.  (On MI355X: 8 units of
// 4000 tokens, 32 teams each, 12.7 us by eights and 15.3 by one team, 8 of 8192 in 8 bits,
// 64 teams each, 16.3 by eights and 17.3 by 16; 128 windows of 4096, 2 or 3 teams each,
// 113.5 in one step, 116.5 where groups began at multiples of 16 and some took two.)
struct CacheJoin {
    uint32_t w0, w1;  // the unit's first and last team
    uint32_t shift;   // groups of 2^shift teams
    __host__ __device__ CacheJoin(uint32_t first, uint32_t last) : w0(first), w1(last)
    {
        const uint32_t apart = last - first;
        shift = apart < 16u ? 4u : apart < 64u ? 3u : apart < 256u ? 4u : 5u;
    }
    __host__ __device__ uint32_t slot(uint32_t w) const { return 2u * w + (w == w0 ? 1u : 0u); }
    // The group of w: its first and last member.
    __host__ __device__ uint32_t first(uint32_t w) const { return w0 + ((w - w0) >> shift << shift); }
    __host__ __device__ uint32_t last(uint32_t w) const
    {
        const uint32_t l = first(w) + (1u << shift) - 1u;
        return l < w1 ? l : w1;
    }
    __host__ __device__ uint32_t groups() const { return ((w1 - w0) >> shift) + 1u; }
    // A team is the first of a group of the unit that its share begins inside, and of
    // the unit that it ends inside, which has its counter there too.
    __host__ __device__ uint32_t group_counter(uint32_t w) const
    {
        const uint32_t f = first(w);
        return 4u * f + (f == w0 ? 0u : 1u);
    }
    __host__ __device__ uint32_t unit_counter() const { return 4u * w0 + 2u; }
    // The slots that w joins in stage 1, its group's teams', or 2, the groups': `first`,
    // then `next`, next + `by` and so on.
    struct Parts {
        uint32_t first, next, by;
    };
    __host__ __device__ Parts parts(uint32_t w, uint32_t stage) const
    {
        const uint32_t f = stage == 1u ? first(w) : w0, by = stage == 1u ? 1u : 1u << shift;
        return {slot(f), 2u * (f + by), 2u * by};
    }
};

}  // namespace ar
