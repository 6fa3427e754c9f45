// cache_attention.hpp -- attention of one new token a sequence over the paged
// cache: the kernel.
//
//     x_t = scale sum_d q_d k_td;   out = sum_t e^{x_t} v_t / sum_t e^{x_t}
//
// It is bound by reading the cache, once for all query heads of a key-value
// head.  These (16 of them; fewer leave columns unused) are the columns of both
// products, so that scores, softmax statistics and results of a query head stay
// in the same four lanes, and nothing crosses lanes inside the loop:
//
//     S [token][query] = K Q^T     the matrix instruction's rows are 16 tokens;
//                                  lane (g, n), g = lane / 16, n = lane % 16, gets
//                                  the scores of query n and tokens 4 g .. 4 g + 3
//     O^T [dim][query] = V^T P^T   rows are 16 dims, and its sum runs over 32
//                                  tokens, eight a lane: tokens 4 g .. 4 g + 3 of two
//                                  groups of 16, which are the ones whose scores the
//                                  lane holds
//
// A wave takes tiles of 32 tokens, its keys straight from memory into the
// registers of the first operand (lane: token n, 16 bytes of it), its values with
// lane n on 16 bytes of each of the lane's eight tokens: the eight-fold transpose
// that the instruction wants is then inside the lane, one byte permutation for two
// values.  Which dim a row of O^T is follows from that load and is undone when
// results are stored.  While a tile is multiplied the next one's keys and values
// are on the way; waves wait for nothing but their own loads, and meet when a
// piece of a unit (cache_plan.hpp) is done.
//
// The softmax keeps a reference r per query: weights are 2^(x - r) and r moves
// only when a score is more than kRoom above it, which rescales the accumulators.
// That is rare, so the loop has no reductions across lanes.
#pragma once

#include "block_device.hpp"
#include "block_matmul.hpp"
#include "cache_internal.hpp"
#include "cache_plan.hpp"

namespace ar {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr uint32_t kAttendWaves = 4, kAttendThreads = 64 * kAttendWaves;

// Queries a workgroup takes at once.
constexpr uint32_t kTileQueries = 16;

// Floats of a slot of partial sums: [16][DP] sums, 16 pairs of reference and sum of weights.
constexpr uint32_t attend_slot(uint32_t dp) { return kTileQueries * (dp + 2u); }

constexpr uint32_t padded_dim(uint32_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// (by value: a bit cast of a vector's element in place reads its first one)
__device__ inline float as_float(uint32_t x) { return __builtin_bit_cast(float, x); }

// Two floats as one word of the matrix instruction's type, rounded to nearest.
template <typename M>
__device__ inline uint32_t pack2(float a, float b)
{
    const float f[2] = {a, b};
    return M::narrow(f);
}

// The same of eight floats in PARTS words each: part i is the rounding of what
// the parts before it leave.  An infinity or NaN stays in the first.
template <typename M, int PARTS>
__device__ inline void split8(const float (&x)[8], u32x4 (&out)[PARTS])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
        for (int s = 0; s < PARTS; ++s) {
            const uint32_t w = pack2<M>(a, b);
            out[s][i] = w;
            if (s + 1 < PARTS) {
                float f[2];
                M::widen(w, f);
                a = a - f[0];
                b = b - f[1];
            }
        }
    }
}

template <typename M>
__device__ inline f32x4 multiply(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (M::kId == Bf16::kId)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Two e4m3 values (the lower or upper half of a word), exactly.
template <typename M, bool UPPER>
__device__ inline uint32_t widen_pair(uint32_t w)
{
    if constexpr (M::kId == Bf16::kId)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, UPPER));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, UPPER));
}

// What a wave holds of a tile.  T: the queries' and outputs' type; EIGHT: the
// cache is e4m3; DP: dim rounded up to 64, 128 or 256.
//
// 16-bit caches multiply in their own type.  An e4m3 cache is widened (exactly) to
// the queries' 16-bit type for the scores, to bfloat16 for a float32's, which is
// split in three parts of 8 bits, and to bfloat16 for the values, whose scale goes
// into the weight: float16 might not hold the product.  float32 caches use the
// binary32 instruction.
template <typename T, bool EIGHT, int DP>
struct Tile {
    static constexpr bool kWide = !EIGHT && T::kBytes == 4;
    static constexpr int kBytes = EIGHT ? 1 : T::kBytes;      // of a cached value
    // A float32 cache of 256 takes one group of 16 tokens a tile: two would not
    // leave registers.
    static constexpr int kGroups = kWide && DP == 256 ? 1 : 2;
    static constexpr uint32_t kTokens = 16 * kGroups;
    static constexpr int kE = 16 / kBytes;                    // values in 16 bytes
    static constexpr int kKeyLoads = DP / (4 * kE);           // a group of 16 tokens
    static constexpr int kVE = EIGHT ? DP / 16 : (DP / 16 < kE ? DP / 16 : kE);  // values a load
    static constexpr int kVH = DP / (16 * kVE);               // loads a token
    static constexpr int kVW = kVE * kBytes / 4;              // words a load
    using KeyType = std::conditional_t<T::kId == Fp16::kId, Fp16, Bf16>;
    using ValueType = std::conditional_t<!EIGHT && T::kId == Fp16::kId, Fp16, Bf16>;
    static constexpr int kQueryParts = EIGHT && T::kBytes == 4 ? 3 : 1;
    static constexpr int kWeightParts = T::kBytes == 4 ? 3 : 2;
    // Weights are at most 2^kRoom, and the largest of those that set the reference
    // 2^kBias: float16 keeps more of the small ones that way.
    static constexpr float kBias = ValueType::kId == Fp16::kId ? 8.0f : 0.0f;
    static constexpr float kRoom = ValueType::kId == Fp16::kId ? 15.0f : 8.0f;
    // Workgroups of a compute unit: registers of a wave.
    static constexpr int kPerCu = DP == 256 || (kWide && DP == 128) ? 1 : 2;

    // query: dims of the lane's k index, for the wide instruction one a register
    static constexpr int kQueryRegs = kWide ? DP / 16 : DP / 32;
    u32x4 q[kQueryParts][kQueryRegs];
    u32x4 k[kGroups][kKeyLoads];
    uint32_t v[kGroups][4][kVH][kVW];
    f32x4 o[DP / 16];

    // The first dim of the lane's 16 bytes (8-bit: of either half) of load s.
    static __device__ uint32_t key_dim(int s, uint32_t g) { return (s * 4 + g) * kE; }
    static __device__ uint32_t value_dim(int h, uint32_t n) { return h * 16 * kVE + n * kVE; }

    template <bool EXACT>
    __device__ void load_query(const char *row, bool there, uint32_t g, uint32_t dim)
    {
#pragma unroll
        for (int s = 0; s < kQueryRegs; ++s) {
            u32x4 x[2] = {};
            // dims of register s: as the key's load has them
            constexpr int kQE = 16 / T::kBytes;
            uint32_t d;
            if constexpr (kWide)
                d = key_dim(s, g);
            else if constexpr (EIGHT)
                d = key_dim(s / 2, g) + s % 2 * 8;
            else
                d = key_dim(s, g);
            if (there && (EXACT || d < dim)) {
                x[0] = load_piece<false>(row + (uint64_t)d * T::kBytes);
                if constexpr (EIGHT && kQE == 4)
                    x[1] = load_piece<false>(row + (uint64_t)d * T::kBytes + 16);
            }
            if constexpr (kQueryParts == 1) {
                q[0][s] = x[0];
            } else {
                // Cut, not rounded, so that the largest values stay finite: three
                // parts of 8 bits hold all of a float32.
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a = as_float(x[i / 2][i % 2 * 2]), b = as_float(x[i / 2][i % 2 * 2 + 1]);
#pragma unroll
                    for (int t = 0; t < kQueryParts; ++t) {
                        const uint32_t ua = __builtin_bit_cast(uint32_t, a) & 0xffff0000u;
                        const uint32_t ub = __builtin_bit_cast(uint32_t, b) & 0xffff0000u;
                        q[t][s][i] = ua >> 16 | ub;
                        a = __builtin_isfinite(a) ? a - as_float(ua) : 0.0f;
                        b = __builtin_isfinite(b) ? b - as_float(ub) : 0.0f;
                    }
                }
            }
        }
    }

    template <bool EXACT>
    __device__ void load_keys(const char *const (&row)[kGroups], uint32_t g, uint32_t dim)
    {
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
            for (int s = 0; s < kKeyLoads; ++s) {
                if (EXACT || key_dim(s, g) < dim)
                    k[gr][s] = load_piece<false>(row[gr] + s * 64);
                else
                    k[gr][s] = u32x4{0, 0, 0, 0};
            }
    }

    template <bool EXACT>
    __device__ void load_values(const char *const (&row)[kGroups][4], uint32_t n, uint32_t dim)
    {
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < kVH; ++h) {
                    // (columns past dim are stored nowhere)
                    if (EXACT || value_dim(h, n) < dim)
                        __builtin_memcpy(v[gr][i][h], __builtin_assume_aligned(row[gr][i] + h * 16 * kVE * kBytes, kVE * kBytes),
                                         kVE * kBytes);
                }
    }

    __device__ void scores(f32x4 (&s)[kGroups]) const
    {
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr)
            s[gr] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int l = 0; l < kKeyLoads; ++l)
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
                if constexpr (kWide) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[gr] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                            as_float(k[gr][l][e]), as_float(q[0][l][e]), s[gr], 0, 0, 0);
                } else if constexpr (EIGHT) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        u32x4 a;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            a[2 * i] = widen_pair<KeyType, false>(k[gr][l][2 * half + i]);
                            a[2 * i + 1] = widen_pair<KeyType, true>(k[gr][l][2 * half + i]);
                        }
                        // the small parts first
#pragma unroll
                        for (int t = kQueryParts - 1; t >= 0; --t)
                            s[gr] = multiply<KeyType>(a, q[t][2 * l + half], s[gr]);
                    }
                } else {
                    s[gr] = multiply<KeyType>(k[gr][l], q[0][l], s[gr]);
                }
            }
    }

    // Values of tokens that are none: whatever their places hold, they add nothing.
    __device__ void drop_values(int gr, int i)
    {
#pragma unroll
        for (int h = 0; h < kVH; ++h)
#pragma unroll
            for (int w = 0; w < kVW; ++w)
                v[gr][i][h][w] = 0;
    }

    // o += V^T P^T; `p`: weights (8-bit values: times their scales) of the lane's tokens.
    __device__ void accumulate(const float (&p)[kGroups][4])
    {
        if constexpr (kWide) {
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int h = 0; h < kVH; ++h)
#pragma unroll
                        for (int j = 0; j < kVE; ++j)
                            o[h * kVE + j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                as_float(v[gr][i][h][j]), p[gr][i], o[h * kVE + j], 0, 0, 0);
        } else {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = p[e / 4][e % 4];
            u32x4 w[kWeightParts];
            split8<ValueType, kWeightParts>(x, w);
#pragma unroll
            for (int h = 0; h < kVH; ++h)
#pragma unroll
                for (int c = 0; c < kVW; ++c) {
                    if constexpr (EIGHT) {
                        u32x4 a[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {  // tokens 2 r, 2 r + 1 of the eight
                            const uint32_t x0 = v[r / 2][r % 2 * 2][h][c], x1 = v[r / 2][r % 2 * 2 + 1][h][c];
                            const uint32_t lo = __builtin_amdgcn_perm(x1, x0, 0x05010400u);
                            const uint32_t hi = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
                            a[0][r] = widen_pair<ValueType, false>(lo);
                            a[1][r] = widen_pair<ValueType, true>(lo);
                            a[2][r] = widen_pair<ValueType, false>(hi);
                            a[3][r] = widen_pair<ValueType, true>(hi);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            add_parts(o[h * kVE + 4 * c + j], a[j], w);
                    } else {
                        u32x4 a[2];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t x0 = v[r / 2][r % 2 * 2][h][c], x1 = v[r / 2][r % 2 * 2 + 1][h][c];
                            a[0][r] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
                            a[1][r] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            add_parts(o[h * kVE + 2 * c + j], a[j], w);
                    }
                }
        }
    }

    static __device__ void add_parts(f32x4 &c, u32x4 a, const u32x4 (&w)[kWeightParts])
    {
#pragma unroll
        for (int t = kWeightParts - 1; t >= 0; --t)
            c = multiply<ValueType>(a, w[t], c);
    }

    // The dim of value i of accumulator t.
    static __device__ uint32_t result_dim(int t, uint32_t g, int i)
    {
        return t / kVE * 16 * kVE + (4 * g + i) * kVE + t % kVE;
    }
};

// A value that is the same in every lane, in a scalar register.
__device__ inline uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ inline uint64_t uniform(uint64_t x)
{
    return (uint64_t)uniform((uint32_t)(x >> 32)) << 32 | uniform((uint32_t)x);
}

// A sum of the lanes that hold a query, in each of them.
__device__ inline float sum_query(float x)
{
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

__device__ inline float max_query(float x)
{
    float y = __shfl_xor(x, 16);
    x = y > x ? y : x;
    y = __shfl_xor(x, 32);
    return y > x ? y : x;
}

// Partial sums go from one workgroup to another past the caches of their XCDs: a
// store of this scope has reached the memory that all of them see when its wave's
// counter says that it is done, and a load of this scope reads there.  (With
// ordinary accesses between fences, which write back and drop whole caches, one
// sequence of 1000 tokens x 8 ranks took 16.3 us in place of @A, 29 odd ones 142 in
// place of @B.)
__device__ inline void share_pair(float *to, float a, float b)
{
    const f32x2 v = {a, b};
    __hip_atomic_store((uint64_t *)to, __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ inline f32x2 shared_pair(const float *from)
{
    return __builtin_bit_cast(f32x2, __hip_atomic_load((const uint64_t *)from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

__device__ inline void shared_stores_done()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <typename T, bool EIGHT, int DP, bool EXACT, bool EIGHT_OUT>
__global__ __launch_bounds__(kAttendThreads, (Tile<T, EIGHT, DP>::kPerCu)) void cache_attend(CacheAttentionArgs p)
{
    typedef Tile<T, EIGHT, DP> X;
    constexpr uint32_t kStep = X::kTokens * kAttendWaves;
    constexpr uint32_t kRow = DP + 4;  // floats of a query's sums in LDS
    // a tile's rows (byte offsets in a pool) and scales, of the next tile
    __shared__ uint64_t rows_at[kAttendWaves][X::kTokens];
    __shared__ float scales_at[EIGHT ? kAttendWaves : 1][2][X::kTokens];
    __shared__ __align__(16) float sums[kAttendWaves][kTileQueries][kRow];
    __shared__ float refs[kAttendWaves][kTileQueries], weights[kAttendWaves][kTileQueries];
    __shared__ uint32_t flags[kAttendWaves];
    __shared__ uint64_t found[6];

    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = uniform(threadIdx.x >> 6);
    const uint32_t n = lane & 15u, g = lane >> 4;
    const uint32_t dim = EXACT ? (uint32_t)DP : p.cache.dim;
    const uint32_t group = p.heads / p.cache.heads;
    const uint32_t tiles = (group + kTileQueries - 1u) / kTileQueries;
    const uint64_t capacity = p.table_pages * p.cache.page_tokens;

    // ---- this workgroup's share -----------------------------------------------
    auto steps_at = [&](uint32_t seq) {
        uint32_t first, end;
        attended(p.lengths[seq], capacity, p.window, &first, &end);
        return steps_of(first, end, kStep);
    };
    const uint32_t chunk = (p.seqs + kAttendThreads - 1u) / kAttendThreads;
    const uint32_t from = threadIdx.x * chunk, to = from + chunk < p.seqs ? from + chunk : p.seqs;
    uint64_t mine = 0;
    for (uint32_t s = from; s < to; ++s)
        mine += steps_at(s);
    uint64_t before = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint64_t x = (uint64_t)__shfl_up((unsigned long long)before, d);
        before += lane >= (uint32_t)d ? x : 0u;
    }
    if (lane == 63)
        found[wave] = before;
    __syncthreads();
    before -= mine;
    uint64_t each = 0;  // steps of all sequences
#pragma unroll
    for (uint32_t w = 0; w < kAttendWaves; ++w) {
        before += w < wave ? found[w] : 0u;
        each += found[w];
    }
    each = uniform(each);
    const uint32_t units = p.nranks * p.cache.heads * tiles;
    const CachePlan plan(each * units, gridDim.x, 1u);
    const uint32_t share = plan.share(blockIdx.x);
    if (share == ~0u)
        return;
    const uint64_t begin = plan.start(share);
    uint64_t left = plan.start(share + 1u) - begin;
    uint32_t unit = (uint32_t)divide(begin, each);
    const uint64_t at = begin - unit * each;
    if (at >= before && at < before + mine) {
        uint64_t b = before;
        uint32_t s = from;
        for (uint32_t x = steps_at(s); at - b >= x; x = steps_at(s)) {
            b += x;
            ++s;
        }
        found[4] = s;
        found[5] = at - b;
    }
    __syncthreads();
    uint32_t seq = uniform((uint32_t)found[4]);
    uint32_t step0 = uniform((uint32_t)found[5]);
    uint64_t here = begin - step0;  // the unit's first step

    const float factor = p.scale * kLog2e;
    uint32_t *counters = (uint32_t *)p.work;
    float *slots = (float *)(p.work + (uint64_t)gridDim.x * 16u);

    for (;;) {
        // ---- a piece: steps [step0, step1) of a unit --------------------------
        const uint32_t rank = unit / (p.cache.heads * tiles);
        const uint32_t kv = unit / tiles % p.cache.heads, tile = unit % tiles;
        uint32_t first, end;
        const int32_t length = p.lengths[seq];
        const bool fine = attended(length, capacity, p.window, &first, &end);
        const uint32_t steps = steps_of(first, end, kStep);
        const uint32_t step1 = left < steps - step0 ? step0 + (uint32_t)left : steps;
        const uint32_t t1 = step1 == steps ? end : first + step1 * kStep;
        const uint32_t queries = group - tile * kTileQueries < kTileQueries ? group - tile * kTileQueries : kTileQueries;
        const uint32_t head0 = kv * group + tile * kTileQueries;

        X x;
        x.template load_query<EXACT>(p.q[rank] + (seq * p.q_stride + (uint64_t)(head0 + n) * dim) * T::kBytes,
                                     n < queries, g, dim);
#pragma unroll
        for (int t = 0; t < DP / 16; ++t)
            x.o[t] = f32x4{0, 0, 0, 0};
        if constexpr (!EXACT)
#pragma unroll
            for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x.drop_values(gr, i);
        float ref = -__builtin_inff(), sum = 0.0f;
        bool bad = !fine;

        const char *keys = p.keys[rank], *values = p.values[rank];
        const float *scales = EIGHT ? (lane < 32u ? p.key_scales[rank] : p.value_scales[rank]) : nullptr;
        const int32_t *table = p.table + seq * p.table_pages;
        const uint32_t mine_at = lane % X::kTokens;
        const uint32_t kd = X::key_dim(0, g) * X::kBytes, vd = X::value_dim(0, n) * X::kBytes;
        uint32_t t0 = first + step0 * kStep + wave * X::kTokens;

        // page and place of the lane's token of the tile at t (past the end: none)
        auto look = [&](uint32_t t, uint32_t &place) {
            t += mine_at;
            int32_t page = -1;
            place = 0;
            if (t < t1) {
                const uint32_t i = p.cache.page_of(t);
                place = t - i * p.cache.page_tokens;
                page = table[i];
            }
            return page;
        };
        const char *krow[X::kGroups], *vrow[X::kGroups][4];
        float scale_next = 0.0f;
        // A token without a place stands for the cache's first one.
        auto rows = [&](uint32_t t, int32_t page, uint32_t place) {
            if ((uint32_t)page >= p.cache.pages) {
                bad = bad || t + mine_at < t1;
                page = 0;
                place = 0;
            }
            rows_at[wave][mine_at] = p.cache.at((uint32_t)page, place, kv) * X::kBytes;
            if constexpr (EIGHT)
                scale_next = scales[p.cache.scale_at((uint32_t)page, place, kv)];
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int gr = 0; gr < X::kGroups; ++gr) {
                krow[gr] = keys + rows_at[wave][gr * 16 + n] + kd;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    vrow[gr][i] = values + rows_at[wave][gr * 16 + 4 * g + i] + vd;
            }
            __builtin_amdgcn_wave_barrier();
        };
        if (t0 < t1) {
            uint32_t place, place_next;
            int32_t page = look(t0, place), page_next = look(t0 + kStep, place_next);
            rows(t0, page, place);
            x.template load_keys<EXACT>(krow, g, dim);
            x.template load_values<EXACT>(vrow, n, dim);
            for (; t0 < t1; t0 += kStep) {
                float ks[X::kGroups][4], vs[X::kGroups][4];
                if constexpr (EIGHT) {
                    scales_at[wave][lane / 32u][mine_at] = scale_next;
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            ks[gr][i] = scales_at[wave][0][gr * 16 + 4 * g + i];
                            vs[gr][i] = scales_at[wave][1][gr * 16 + 4 * g + i];
                        }
                    __builtin_amdgcn_wave_barrier();
                }
                rows(t0 + kStep, page_next, place_next);
                page_next = look(t0 + 2 * kStep, place_next);
                f32x4 s[X::kGroups];
                x.scores(s);
                x.template load_keys<EXACT>(krow, g, dim);

                const bool whole = t0 + X::kTokens <= t1;
                float w[X::kGroups][4], most = -__builtin_inff();
#pragma unroll
                for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float c = factor;
                        if constexpr (EIGHT)
                            c = c * ks[gr][i];
                        w[gr][i] = s[gr][i] * c;
                    }
                if (!whole) {
#pragma unroll
                    for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (t0 + gr * 16 + 4 * g + i >= t1) {
                                w[gr][i] = -__builtin_inff();
                                if constexpr (EIGHT)
                                    vs[gr][i] = 0.0f;
                                x.drop_values(gr, i);
                            }
                }
#pragma unroll
                for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        most = w[gr][i] > most ? w[gr][i] : most;
                if (__ballot(most > ref + (X::kRoom - X::kBias)) != 0) {
                    // (a NaN raises nothing; it reaches the sums by its own weight)
                    const float next = max_query(most) > ref ? max_query(most) : ref;
                    const float shift = next == -__builtin_inff() ? 0.0f : next;
                    const float keep = __builtin_amdgcn_exp2f(ref - shift);
                    sum = sum * keep;
#pragma unroll
                    for (int t = 0; t < DP / 16; ++t)
                        x.o[t] = x.o[t] * keep;
                    ref = next;
                }
                const float shift = (ref == -__builtin_inff() ? 0.0f : ref) - X::kBias;
#pragma unroll
                for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w[gr][i] = __builtin_amdgcn_exp2f(w[gr][i] - shift);
                        sum += w[gr][i];
                        if constexpr (EIGHT)
                            w[gr][i] = w[gr][i] * vs[gr][i];
                    }
                x.accumulate(w);
                x.template load_values<EXACT>(vrow, n, dim);
            }
        }

        // ---- the waves' sums together -----------------------------------------
        sum = sum_query(sum);
        if (g == 0) {
            refs[wave][n] = ref;
            weights[wave][n] = sum;
        }
        const bool any_bad = __ballot(bad) != 0;
        if (lane == 0)
            flags[wave] = any_bad;
#pragma unroll
        for (int t = 0; t < DP / 16; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sums[wave][n][X::result_dim(t, g, i)] = x.o[t][i];
        __syncthreads();

        // A thread takes eight dims of one query, or of two.
        constexpr uint32_t kPieces = DP / 8, kAtOnce = kAttendThreads / kPieces;
        constexpr uint32_t kTurns = (kTileQueries + kAtOnce - 1) / kAtOnce;
        const uint32_t d0 = threadIdx.x % kPieces * 8u;
        float top[kTurns], total[kTurns], y[kTurns][8];
#pragma unroll
        for (uint32_t u = 0; u < kTurns; ++u) {
            const uint32_t q = (threadIdx.x / kPieces + u * kAtOnce) % kTileQueries;
            top[u] = -__builtin_inff();
            total[u] = 0.0f;
#pragma unroll
            for (uint32_t w = 0; w < kAttendWaves; ++w)
                top[u] = refs[w][q] > top[u] ? refs[w][q] : top[u];
            const float shift = top[u] == -__builtin_inff() ? 0.0f : top[u];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[u][e] = 0.0f;
#pragma unroll
            for (uint32_t w = 0; w < kAttendWaves; ++w) {
                const float keep = __builtin_amdgcn_exp2f(refs[w][q] - shift);
                total[u] += weights[w][q] * keep;
                if (flags[w] != 0)
                    total[u] = __builtin_nanf("");
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[u][e] += sums[w][q][d0 + e] * keep;
            }
        }

        // ---- and the workgroups', where several share the unit ----------------
        bool done = step0 == 0 && step1 == steps;
        if (!done) {
            const CacheJoin join = {plan.owner(here), plan.owner(here + steps - 1u)};
            auto keep_slot = [&](uint32_t slot) {
                float *to = slots + (uint64_t)slot * attend_slot(DP);
#pragma unroll
                for (uint32_t u = 0; u < kTurns; ++u) {
                    const uint32_t q = threadIdx.x / kPieces + u * kAtOnce;
                    if (q >= queries)
                        continue;
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        share_pair(to + q * DP + d0 + e, y[u][e], y[u][e + 1]);
                    if (d0 == 0)
                        share_pair(to + kTileQueries * DP + 2 * q, top[u], total[u]);
                }
            };
            // Whether this workgroup is the last of `count` to come here.
            auto arrive = [&](uint32_t counter, uint32_t count) {
                shared_stores_done();
                __syncthreads();
                if (threadIdx.x == 0) {
                    const uint32_t old = __hip_atomic_fetch_add(counters + counter, 1u, __ATOMIC_RELAXED,
                                                                __HIP_MEMORY_SCOPE_AGENT);
                    flags[0] = old + 1u == count;
                    if (old + 1u == count)
                        __hip_atomic_store(counters + counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                }
                __syncthreads();
                return flags[0] != 0;
            };
            // The slots' sums together, in order, four slots' loads under way at once.
            auto add_slots = [&](auto slot_of, uint32_t count) {
#pragma unroll
                for (uint32_t u = 0; u < kTurns; ++u) {
                    const uint32_t q = (threadIdx.x / kPieces + u * kAtOnce) % kTileQueries;
                    top[u] = -__builtin_inff();
                    total[u] = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[u][e] = 0.0f;
                    if (q >= queries)
                        continue;
                    constexpr uint32_t kBatch = 4;
                    for (uint32_t i = 0; i < count; i += kBatch) {
                        f32x2 f[kBatch][4], s[kBatch];
#pragma unroll
                        for (uint32_t j = 0; j < kBatch; ++j) {
                            // (past the last: the last again, without weight)
                            const float *at = slots + (uint64_t)slot_of(i + j < count ? i + j : count - 1u) * attend_slot(DP);
                            s[j] = shared_pair(at + kTileQueries * DP + 2 * q);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                f[j][e] = shared_pair(at + q * DP + d0 + 2 * e);
                        }
#pragma unroll
                        for (uint32_t j = 0; j < kBatch; ++j) {
                            if (i + j >= count)
                                break;
                            const float next = s[j][0] > top[u] ? s[j][0] : top[u];
                            const float shift = next == -__builtin_inff() ? 0.0f : next;
                            const float a = __builtin_amdgcn_exp2f(top[u] - shift), b = __builtin_amdgcn_exp2f(s[j][0] - shift);
                            top[u] = next;
                            total[u] = total[u] * a + s[j][1] * b;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                y[u][e] = y[u][e] * a + f[j][e / 2][e % 2] * b;
                        }
                    }
                }
            };
            keep_slot(join.slot(share));
            const uint32_t f = join.first(share), l = join.last(share);
            if (arrive(join.group_counter(share), l - f + 1u)) {
                add_slots([&](uint32_t i) { return join.slot(f + i); }, l - f + 1u);
                done = join.groups() == 1u;
                if (!done) {
                    __syncthreads();
                    keep_slot(join.slot(f));
                    if (arrive(join.unit_counter(), join.groups())) {
                        const uint32_t g0 = join.w0 / kJoinGroup;
                        add_slots([&](uint32_t i) { return join.slot(join.first((g0 + i) * kJoinGroup > join.w0 ? (g0 + i) * kJoinGroup : join.w0)); },
                                  join.groups());
                        done = true;
                    }
                }
            }
        }

        // ---- the unit's results ------------------------------------------------
        if (done) {
#pragma unroll
            for (uint32_t u = 0; u < kTurns; ++u) {
                const uint32_t q = threadIdx.x / kPieces + u * kAtOnce;
                const bool there = q < queries && d0 < dim;
                const uint64_t row = (uint64_t)seq * p.heads + head0 + q;
                const bool empty = length == 0;
                float r[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    r[e] = empty ? 0.0f : y[u][e] / total[u];
                if (p.has_lse != 0 && there && d0 == 0)
                    p.lse[rank][row] = empty ? -__builtin_inff()
                                             : ((top[u] == -__builtin_inff() ? 0.0f : top[u]) - X::kBias) * kLn2 +
                                                   __builtin_logf(total[u]);
                if constexpr (EIGHT_OUT) {
                    // 16 neighbouring lanes hold the 128 columns of a scale
                    const float s = scale_of(max16(max_bits(r)));
                    const Eights<8> e = to_eights(r, s);
                    if (there) {
                        store_eights<false>(p.out[rank] + row * dim + d0, e);
                        if (d0 % AR_SCALE_BLOCK == 0)
                            p.out_scales[rank][((uint64_t)(head0 + q) * dim + d0) / AR_SCALE_BLOCK * p.seqs + seq] = s;
                    }
                } else if (there) {
                    char *at_out = p.out[rank] + (row * dim + d0) * T::kBytes;
                    constexpr int E = kPiece<T>;
#pragma unroll
                    for (int i = 0; i < 8 / E; ++i) {
                        float f[E];
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            f[e] = r[i * E + e];
                        store_piece<false>(at_out + i * 16, narrow_piece<T>(f));
                    }
                }
            }
        }

        left -= step1 - step0;
        if (left == 0)
            return;
        here += steps;
        step0 = 0;
        if (++seq == p.seqs) {
            seq = 0;
            ++unit;
        }
        __syncthreads();  // the sums in LDS are read before the next piece's are written
    }
}

// Workgroups of a launch at most: what fits the compute units at once.
inline uint32_t attend_most(int per_cu, int cu_count) { return (uint32_t)(per_cu * cu_count) / 8u * 8u; }

template <typename T, bool EIGHT, int DP, bool EXACT, bool EIGHT_OUT>
hipError_t enqueue_attend(const CacheAttentionArgs &args, int cu_count, hipStream_t stream)
{
    typedef Tile<T, EIGHT, DP> X;
    const uint64_t capacity = args.table_pages * args.cache.page_tokens;
    const uint64_t tokens = args.window != 0 && args.window < capacity ? args.window : capacity;
    const uint64_t steps = (tokens - 1u) / (X::kTokens * kAttendWaves) + 1u;
    const uint32_t group = args.heads / args.cache.heads;
    const uint64_t units = (uint64_t)args.nranks * args.cache.heads * args.seqs *
                           ((group + kTileQueries - 1u) / kTileQueries);
    uint64_t grid = attend_most(X::kPerCu, cu_count);
    if (steps < grid && units * steps < grid)
        grid = (units * steps + 7u) / 8u * 8u;
    hipLaunchKernelGGL((cache_attend<T, EIGHT, DP, EXACT, EIGHT_OUT>), dim3((uint32_t)grid),
                       dim3(kAttendThreads), 0, stream, args);
    return hipGetLastError();
}

template <typename T, bool EIGHT, int DP>
hipError_t pick_attend(const CacheAttentionArgs &args, bool eight_out, int cu_count, hipStream_t stream)
{
    if (args.cache.dim != DP)
        return enqueue_attend<T, EIGHT, DP, false, false>(args, cu_count, stream);
    if constexpr (DP % AR_SCALE_BLOCK == 0)
        if (eight_out)
            return enqueue_attend<T, EIGHT, DP, true, true>(args, cu_count, stream);
    return enqueue_attend<T, EIGHT, DP, true, false>(args, cu_count, stream);
}

// One of the six kernel families, each compiled in a file of its own.
template <typename T, bool EIGHT>
hipError_t launch_attend(const CacheAttentionArgs &args, bool eight_out, int cu_count,
                         hipStream_t stream)
#ifdef AR_ATTEND_FAMILY
{
    switch (padded_dim(args.cache.dim)) {
    case 64: return pick_attend<T, EIGHT, 64>(args, eight_out, cu_count, stream);
    case 128: return pick_attend<T, EIGHT, 128>(args, eight_out, cu_count, stream);
    default: return pick_attend<T, EIGHT, 256>(args, eight_out, cu_count, stream);
    }
}
#else
    ;
#endif

}  // namespace ar
