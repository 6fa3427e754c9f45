// cache_api.hip -- the entry points declared in include/ar_cache.h: argument
// checks on the host without touching the device, then one launch on the
// caller's stream.
#include <math.h>

#include "api_checks.hpp"
#include "cache_internal.hpp"
#include "cache_plan.hpp"

using namespace ar;

namespace {

typedef unsigned __int128 u128;

constexpr size_t kMostHeads = 4096, kMostSeqs = 65536;

// A step of a layout: blocks of `inner` elements from their first to their last,
// `stride` apart.
struct Step {
    size_t count, stride, inner;
};

// The layout in the kernels' form, its steps, the innermost first, and the elements
// from a pool's first to its last.  Strides of which there is only one step do not count.
arResult_t check_layout(const arCacheLayout_t *c, size_t page_bytes, CacheShape *shape,
                        Step (&steps)[3], size_t *span)
{
    if (c == nullptr)
        return reject(arInvalidArgument, "NULL cache layout");
    if (c->dim < 16 || c->dim > AR_CACHE_MAX_DIM || c->dim % 16 != 0)
        return reject(arUnsupported, "dim must be a multiple of 16 in 16..256");
    if (c->heads < 1 || c->heads > kMostHeads)
        return reject(arUnsupported, "cache heads must be in 1..4096");
    if (c->pages < 1 || c->pageTokens < 1 || c->pages > INT32_MAX || c->pageTokens > INT32_MAX ||
        c->pages * c->pageTokens > INT32_MAX)
        return reject(arInvalidArgument, "pages * pageTokens must be in 1..2^31 - 1");
    steps[0] = {c->pages, c->pageStride, 0};
    steps[1] = {c->heads, c->headStride, 0};
    steps[2] = {c->pageTokens, c->tokenStride, 0};
    std::sort(steps, steps + 3, [](const Step &a, const Step &b) { return a.stride < b.stride; });
    u128 extent = c->dim;
    for (Step &s : steps) {
        s.inner = (size_t)extent;
        if (s.count == 1)
            continue;
        if (s.stride % (16 / page_bytes) != 0)
            return reject(arInvalidArgument, "cache strides must be multiples of 16 bytes");
        if (s.stride < extent)
            return reject(arInvalidArgument, "rows of the cache overlap");
        extent += (u128)(s.count - 1) * s.stride;
        if (extent > SIZE_MAX >> 4)
            return reject(arInvalidArgument, "cache too large");
    }
    shape->page_stride = c->pages > 1 ? c->pageStride : 0;
    shape->head_stride = c->heads > 1 ? c->headStride : 0;
    shape->token_stride = c->pageTokens > 1 ? c->tokenStride : 0;
    shape->pages = (uint32_t)c->pages;
    shape->page_tokens = (uint32_t)c->pageTokens;
    shape->heads = (uint32_t)c->heads;
    shape->dim = (uint32_t)c->dim;
    shape->set_division();
    *span = (size_t)extent;
    return arSuccess;
}

// Rows of `heads` * dim elements `stride` apart: the elements from the first to
// the last.
arResult_t check_rows(size_t rows, size_t row, size_t stride, int dtype, size_t *span)
{
    if (stride < row || stride % (16 / elem_bytes(dtype)) != 0)
        return reject(arInvalidArgument, "a row stride must hold a row and be a multiple of 16 bytes");
    const u128 most = (u128)(rows - 1) * stride + row;
    if (most > SIZE_MAX >> 4)
        return reject(arInvalidArgument, "too many rows");
    *span = (size_t)most;
    return arSuccess;
}

// The ranges of a rank's keys and values, written both, `bytes` each, which may lie next to
// each other inside the blocks of a step (elements of `es` bytes): the values' parts then lie
// behind the keys' or the other way round, and neither's reach into the next block, here or
// in the steps around it.
template <size_t N>
bool add_pair(Ranges *mem, const void *a, const void *b, size_t bytes, const Step (&steps)[N], size_t es)
{
    const uintptr_t lo = std::min((uintptr_t)a, (uintptr_t)b), hi = std::max((uintptr_t)a, (uintptr_t)b);
    const size_t apart = hi - lo;
    bool beside = false;
    for (const Step &s : steps) {
        if (s.count == 1)
            continue;
        const bool inside = apart < s.stride * es && s.inner * es <= s.stride * es - apart;
        beside = inside && (beside || apart >= s.inner * es);
    }
    if (beside && lo != 0 && (lo & 15u) == 0 && (hi & 15u) == 0)
        return mem->add((const void *)lo, apart + bytes, true);
    return mem->add(a, bytes, true) && mem->add(b, bytes, true);
}

// The steps of 2^shift tokens of sequences whose lengths are known, for `choose`.
struct TotalSteps {
    uint32_t all;
};
TotalSteps total_steps(const int32_t *lengths, size_t seqs, size_t capacity, size_t window, uint32_t shift,
                       uint32_t most)
{
    TotalSteps t = {0};
    for (size_t i = 0; i < seqs; ++i) {
        uint32_t first, end;
        attended(lengths[i], capacity, window, &first, &end);
        t.all += std::min(steps_of(first, end, shift), most);
    }
    return t;
}

struct Copy {
    const void *const *rows[2];
    const void *const *pages[2];
    const float *const *scales[2];
};

// arCacheWrite and arCacheRead: `write` says which side is written.
arResult_t copy(const Copy &c, bool write, size_t row_stride, const int64_t *slots, size_t tokens,
                const arCacheLayout_t *cache, arDataType_t dtype_arg, int nranks, arComm_t comm,
                arStream_t stream)
{
    const int dtype = raw(dtype_arg);
    if (!is_dtype(dtype))
        return reject(arUnsupported, "dtype must be bf16, fp16 or fp32");
    if (nranks < 1 || nranks > AR_MAX_RANKS)
        return reject(arUnsupported, "nranks must be in 1..32");
    const bool eight = c.scales[0] != nullptr;
    if (eight != (c.scales[1] != nullptr))
        return reject(arInvalidArgument, "scales of keys and of values, or of neither");
    const size_t page_bytes = eight ? 1 : elem_bytes(dtype);
    CacheCopyArgs args = {};
    Step steps[3];
    size_t span, row_span;
    arResult_t r = check_layout(cache, page_bytes, &args.cache, steps, &span);
    if (r != arSuccess)
        return r;
    if (tokens == 0)
        return arSuccess;
    if (tokens > INT32_MAX)
        return reject(arInvalidArgument, "tokens must be below 2^31");
    const size_t row = cache->heads * cache->dim, es = elem_bytes(dtype);
    r = check_rows(tokens, row, row_stride, dtype, &row_span);
    if (r != arSuccess)
        return r;
    for (int i = 0; i < 2; ++i)
        if (c.rows[i] == nullptr || c.pages[i] == nullptr)
            return reject(arInvalidArgument, "NULL buffer array");
    Ranges mem;
    const size_t places = cache->pages * cache->pageTokens * cache->heads;
    const Step rows[1] = {{tokens, row_stride, row}};
    bool ok = mem.add(slots, tokens * sizeof(int64_t), false, 8);
    for (int i = 0; i < nranks && ok; ++i) {
        if (write) {
            ok = mem.add(c.rows[0][i], row_span * es, false) &&
                 mem.add(c.rows[1][i], row_span * es, false) &&
                 add_pair(&mem, c.pages[0][i], c.pages[1][i], span * page_bytes, steps, page_bytes);
        } else {
            ok = mem.add(c.pages[0][i], span * page_bytes, false) &&
                 mem.add(c.pages[1][i], span * page_bytes, false) &&
                 add_pair(&mem, c.rows[0][i], c.rows[1][i], row_span * es, rows, es);
        }
        for (int k = 0; k < 2 && eight && ok; ++k)
            ok = mem.add(c.scales[k][i], places * sizeof(float), write);
    }
    if (!ok || !mem.disjoint())
        return reject(arInvalidArgument, mem.why());
    r = check_comm(comm);
    if (r != arSuccess)
        return r;
    for (int i = 0; i < nranks; ++i)
        for (int k = 0; k < 2; ++k) {
            args.rows[k][i] = (char *)c.rows[k][i];
            args.pages[k][i] = (char *)c.pages[k][i];
            args.scales[k][i] = eight ? (float *)c.scales[k][i] : nullptr;
        }
    args.slots = slots;
    args.row_stride = row_stride;
    args.tokens = (uint32_t)tokens;
    auto launch = write ? launch_cache_write : launch_cache_read;
    return launched(launch(args, dtype, eight, nranks, comm->cu_count, (hipStream_t)stream));
}

}  // namespace

extern "C" {

arResult_t arCacheWrite(const void *const *keys, const void *const *values, size_t rowStride,
                        const int64_t *slots, size_t tokens, const arCacheLayout_t *cache,
                        void *const *keyPages, void *const *valuePages, float *const *keyScales,
                        float *const *valueScales, arDataType_t dtype, int nranks, arComm_t comm,
                        arStream_t stream)
{
    return copy({{keys, values}, {keyPages, valuePages}, {keyScales, valueScales}}, true, rowStride,
                slots, tokens, cache, dtype, nranks, comm, stream);
}

arResult_t arCacheRead(const int64_t *slots, size_t tokens, const arCacheLayout_t *cache,
                       const void *const *keyPages, const void *const *valuePages,
                       const float *const *keyScales, const float *const *valueScales,
                       void *const *keys, void *const *values, size_t rowStride,
                       arDataType_t dtype, int nranks, arComm_t comm, arStream_t stream)
{
    return copy({{keys, values}, {keyPages, valuePages}, {keyScales, valueScales}}, false, rowStride,
                slots, tokens, cache, dtype, nranks, comm, stream);
}

arResult_t arCacheAttention(const void *const *queries, size_t queryStride,
                            const arCacheLayout_t *cache, const void *const *keyPages,
                            const void *const *valuePages, const float *const *keyScales,
                            const float *const *valueScales, const int32_t *pageTable,
                            size_t tablePages, const int32_t *lengths, size_t seqs, size_t heads,
                            float scale, size_t window, void *const *outbufs,
                            float *const *outScales, float *const *lse, void *workspace,
                            size_t workspaceBytes, arDataType_t dtype_arg, int nranks,
                            arComm_t comm, arStream_t stream)
{
    const int dtype = raw(dtype_arg);
    if (!is_dtype(dtype))
        return reject(arUnsupported, "dtype must be bf16, fp16 or fp32");
    if (nranks < 1 || nranks > AR_MAX_RANKS)
        return reject(arUnsupported, "nranks must be in 1..32");
    const bool eight = keyScales != nullptr, eight_out = outScales != nullptr;
    if (eight != (valueScales != nullptr))
        return reject(arInvalidArgument, "scales of keys and of values, or of neither");
    const size_t es = elem_bytes(dtype), page_bytes = eight ? 1 : es;
    CacheAttentionArgs args = {};
    Step steps[3];
    size_t span, q_span;
    arResult_t r = check_layout(cache, page_bytes, &args.cache, steps, &span);
    if (r != arSuccess)
        return r;
    if (heads < 1 || heads > kMostHeads || heads % cache->heads != 0)
        return reject(arUnsupported, "heads must be a multiple of the cache's, at most 4096");
    if (eight_out && cache->dim % AR_SCALE_BLOCK != 0)
        return reject(arUnsupported, "8-bit outputs need heads of 128 or 256");
    if (!(fabsf(scale) <= 0x1p126f))  // (the kernel takes it times log2 e)
        return reject(arInvalidArgument, "scale must be at most 2^126 in magnitude");
    if (seqs == 0)
        return arSuccess;
    if (seqs > kMostSeqs)
        return reject(arUnsupported, "seqs must be at most 65536");
    if (seqs * heads * (size_t)nranks > (size_t)1 << 24)
        return reject(arUnsupported, "seqs * heads * nranks must be at most 2^24");
    if (tablePages < 1 || tablePages > INT32_MAX)
        return reject(arInvalidArgument, "tablePages must be in 1..2^31 - 1");
    const size_t row = heads * cache->dim;
    r = check_rows(seqs, row, queryStride, dtype, &q_span);
    if (r != arSuccess)
        return r;
    if (queries == nullptr || keyPages == nullptr || valuePages == nullptr || outbufs == nullptr)
        return reject(arInvalidArgument, "NULL buffer array");
    Ranges mem;
    const size_t places = cache->pages * cache->pageTokens * cache->heads;
    bool ok = mem.add(pageTable, seqs * tablePages * sizeof(int32_t), false, 4) &&
              mem.add(lengths, seqs * sizeof(int32_t), false, 4) &&
              mem.add(workspace, workspaceBytes, true) &&
              mem.add_ranks(queries, nranks, q_span * es, false) &&
              mem.add_ranks(keyPages, nranks, span * page_bytes, false) &&
              mem.add_ranks(valuePages, nranks, span * page_bytes, false) &&
              mem.add_ranks(outbufs, nranks, seqs * row * (eight_out ? 1 : es), true);
    if (eight)
        ok = ok && mem.add_ranks((const void *const *)keyScales, nranks, places * sizeof(float), false) &&
             mem.add_ranks((const void *const *)valueScales, nranks, places * sizeof(float), false);
    if (eight_out)
        ok = ok && mem.add_ranks((const void *const *)outScales, nranks,
                                 scale_blocks(row) * seqs * sizeof(float), true);
    if (lse != nullptr)
        ok = ok && mem.add_ranks((const void *const *)lse, nranks, seqs * heads * sizeof(float), true);
    if (!ok || !mem.disjoint())
        return reject(arInvalidArgument, mem.why());
    r = check_comm(comm);
    if (r != arSuccess)
        return r;
    if (workspaceBytes < cache_attention_workspace(args.cache.dim, (uint32_t)(heads / cache->heads),
                                                   comm->cu_count))
        return reject(arInvalidArgument, "workspace too small");
    for (int i = 0; i < nranks; ++i) {
        args.q[i] = (const char *)queries[i];
        args.keys[i] = (const char *)keyPages[i];
        args.values[i] = (const char *)valuePages[i];
        args.key_scales[i] = eight ? keyScales[i] : nullptr;
        args.value_scales[i] = eight ? valueScales[i] : nullptr;
        args.out[i] = (char *)outbufs[i];
        args.out_scales[i] = eight_out ? outScales[i] : nullptr;
        args.lse[i] = lse != nullptr ? lse[i] : nullptr;
    }
    args.table = pageTable;
    args.lengths = lengths;
    args.q_stride = queryStride;
    args.table_pages = tablePages;
    args.window = window;
    args.work = (char *)workspace;
    args.slots = (float *)((char *)workspace + AR_CACHE_WORKSPACE_ZEROS);
    args.seqs = (uint32_t)seqs;
    args.heads = (uint32_t)heads;
    args.group = (uint32_t)(heads / cache->heads);
    args.nranks = (uint32_t)nranks;
    args.has_lse = lse != nullptr;
    args.scale = scale;
    return launched(launch_cache_attention(args, dtype, eight, eight_out, comm->cu_count,
                                           (hipStream_t)stream));
}

arResult_t arCacheAttentionWorkspace(size_t dim, size_t group, arComm_t comm, size_t *bytes)
{
    if (bytes == nullptr)
        return reject(arInvalidArgument, "NULL result");
    if (dim < 16 || dim > AR_CACHE_MAX_DIM || dim % 16 != 0)
        return reject(arUnsupported, "dim must be a multiple of 16 in 16..256");
    if (group < 1 || group > kMostHeads)
        return reject(arUnsupported, "group must be in 1..4096");
    if (comm == nullptr)
        return reject(arInvalidArgument, "NULL comm");
    *bytes = (size_t)cache_attention_workspace((uint32_t)dim, (uint32_t)group, comm->cu_count);
    return arSuccess;
}

// For tests, on the host: whether a call whose lengths are known loads keys and values past the
// caches.
int ar_cache_attention_streams(const int32_t *lengths, size_t seqs, size_t capacity, size_t window,
                               uint32_t queries, uint32_t tokens, uint32_t ranks, uint32_t heads,
                               uint32_t group, uint32_t grid, uint32_t token_bytes)
{
    const uint32_t passes = passes_of_a_step(seqs, ranks, heads, group, tokens,
                                             most_attended(capacity, window));
    const CacheCall call = {(uint32_t)seqs, ranks, heads, group, queries, tokens, passes, grid, token_bytes};
    TotalSteps steps;
    return choose(call, [&](uint32_t shift, uint32_t most) { return total_steps(lengths, seqs, capacity, window, shift, most); },
                  &steps).stream;
}

// For tests, on the host: the pieces of the share of team `team` of workgroup `block`
// of an attention whose lengths are known, as the kernel walks them (cache_plan.hpp).
// 2^queries and 2^tokens are a wave's.  Thirteen numbers a piece: rank, sequence,
// key-value head and tile of query heads, first step, step after the last, steps of the
// unit, first token, token after the last, slot of partial sums, counter of the group and
// teams in it, counter of the unit and groups in it.  `teams`: waves of a team, waves that take
// the same tokens, tiles of query heads, tokens of a pass and of a step.  Returns the
// number of pieces, of which `most` are written.
size_t ar_cache_attention_share(const int32_t *lengths, size_t seqs, size_t capacity, size_t window,
                                uint32_t queries, uint32_t tokens, uint32_t ranks,
                                uint32_t heads, uint32_t group, uint32_t grid, uint32_t block,
                                uint32_t team, uint32_t teams[5], uint32_t (*pieces)[13], size_t most)
{
    uint32_t first, end;
    const uint32_t passes = passes_of_a_step(seqs, ranks, heads, group, tokens,
                                             most_attended(capacity, window));
    const CacheCall call = {(uint32_t)seqs, ranks, heads, group, queries, tokens, passes, grid, 0};
    TotalSteps steps_of_all;
    const CacheChoice choice =
        choose(call, [&](uint32_t shift, uint32_t most) { return total_steps(lengths, seqs, capacity, window, shift, most); },
               &steps_of_all);
    const CacheTeams &t = choice.teams;
    const bool alone = choice.alone;
    const uint32_t across = heads * t.tiles;
    auto steps_at = [&](size_t i) {
        attended(lengths[i], capacity, window, &first, &end);
        return steps_of(first, end, t.shift);
    };
    uint32_t row = 0;
    for (size_t i = 0; i < seqs; ++i)
        row += steps_at(i) * across;
    const uint32_t told[5] = {t.waves, t.side, t.tiles, t.pass, 1u << t.shift};
    memcpy(teams, told, sizeof told);
    const CachePlan plan(row * ranks, alone ? grid * 4u : grid);
    const uint32_t share = team < 4u / t.waves ? plan.share(block, team, grid) : ~0u;
    if (share == ~0u)
        return 0;
    const uint32_t begin = plan.start(share);
    uint32_t left = plan.start(share + 1u) - begin, rank = begin / row, at = begin % row, seq = 0;
    size_t count = 0;
    for (uint32_t x = steps_at(seq) * across; at >= x; x = steps_at(++seq) * across)
        at -= x;
    uint32_t unit = at / steps_at(seq), step0 = at % steps_at(seq), here = begin - step0;
    for (;;) {
        const uint32_t steps = steps_at(seq);
        const uint32_t step1 = left < steps - step0 ? step0 + left : steps;
        const CacheJoin join(plan.owner(here), plan.owner(here + steps - 1u));
        const uint32_t piece[13] = {
            rank, seq, unit, step0, step1, steps, first + (step0 << t.shift),
            step1 == steps ? end : first + (step1 << t.shift), join.slot(share), join.group_counter(share),
            join.last(share) - join.first(share) + 1u, join.unit_counter(), join.groups()};
        if (count < most)
            memcpy(pieces[count], piece, sizeof piece);
        ++count;
        left -= step1 - step0;
        if (left == 0)
            return count;
        here += steps;
        step0 = 0;
        if (++unit == across) {
            unit = 0;
            if (++seq == seqs) {
                seq = 0;
                ++rank;
            }
        }
    }
}

// For tests, on the host: the slot of part i of what team w joins in `stage` for a unit
// of teams w0 .. w1.
uint32_t ar_cache_attention_part(uint32_t w0, uint32_t w1, uint32_t w, uint32_t stage, uint32_t i)
{
    const CacheJoin::Parts parts = CacheJoin(w0, w1).parts(w, stage);
    return i == 0 ? parts.first : parts.next + (i - 1u) * parts.by;
}

// For tests, on the host: the page and place of a slot; 0 for one of no cache.
int ar_cache_place(size_t pages, size_t page_tokens, int64_t slot, uint32_t at[2])
{
    CacheShape shape = {};
    shape.pages = (uint32_t)pages;
    shape.page_tokens = (uint32_t)page_tokens;
    shape.set_division();
    return shape.place(slot, &at[0], &at[1]);
}

}  // extern "C"
