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
//
// Measured on MI355X, where reading alone reaches 7.1 TB/s: 64 x 8192 tokens x 8 ranks,
// 8 query heads of 128, 318 us (6.75 TB/s of keys and values; 8 bits 174 us, 6.4);
// 4 ranks with heads of 256 315 us (6.8); heads of 64 163 us (6.6).  A call of few tokens
// is one chain of loads (lengths, page, keys, queries), the waves' sums in LDS and, for a
// unit of several teams, one or two joins through memory of 3 to 4 us: one sequence of
// 20 tokens x 8 ranks 7.6 us, of 1000 10.6, of 8192 in 8 bits 16.0.
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

// A slot of partial sums: [queries][DP] sums, then as many pairs of reference and sum
// of weights.  A lane has eight sums of a query; they lie in pairs, the first pairs of
// all lanes, then the second ones and so on, so that each access is of whole lines.

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
// the parts before it leave.
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
// cache is e4m3; DP: dim rounded up to 64, 128 or 256; QT: tiles of 16 queries.
//
// 16-bit caches multiply in their own type.  An e4m3 cache is widened (exactly) to
// the queries' 16-bit type for the scores, to bfloat16 for a float32's, which is
// split in three parts of 8 bits, and to bfloat16 for the values, whose scale goes
// into the weight: float16 might not hold the product.  float32 caches use the
// binary32 instruction.
template <typename T, bool EIGHT, int DP, int QT>
struct Tile {
    static constexpr bool kWide = !EIGHT && T::kBytes == 4;
    static constexpr int kBytes = EIGHT ? 1 : T::kBytes;      // of a cached value
    // A float32 cache of 256 takes one group of 16 tokens a tile: two would not
    // leave registers.
    static constexpr int kGroups = kWide && DP == 256 ? 1 : 2;
    static constexpr uint32_t kTokenShift = kGroups == 1 ? 4 : 5;
    static constexpr uint32_t kTokens = 1u << kTokenShift;
    static constexpr int kE = 16 / kBytes;                    // values in 16 bytes
    static constexpr int kKeyLoads = DP / (4 * kE);           // a group of 16 tokens
    static constexpr int kVE = EIGHT ? DP / 16 : (DP / 16 < kE ? DP / 16 : kE);  // values a load
    static constexpr int kVH = DP / (16 * kVE);               // loads a token
    static constexpr int kVW = kVE * kBytes / 4;              // words a load
    typedef uint32_t Words __attribute__((ext_vector_type(kVW)));
    using KeyType = std::conditional_t<T::kId == Fp16::kId, Fp16, Bf16>;
    using ValueType = std::conditional_t<!EIGHT && T::kId == Fp16::kId, Fp16, Bf16>;
    static constexpr int kQueryParts = EIGHT && T::kBytes == 4 ? 3 : 1;
    // The parts of a weight, each the rounding of what is left, hold a binary32's bits:
    // three of bfloat16 all, two of float16 all but 2^-23 of the weight or 2^-33 of the
    // largest.  (Two of bfloat16, 2^-18 off, took 64 x 8192 tokens x 8 ranks in 318.0 us in
    // place of 318.4, 8-bit heads of 64 in 91 in place of 94.5, one rank's 64 query heads
    // in 72 in place of 75.)
    static constexpr int kWeightParts = ValueType::kId == Fp16::kId ? 2 : 3;
    // Weights are at most 2^kRoom, and the largest of those that set the reference
    // 2^kBias: float16 keeps more of the small ones that way.
    static constexpr float kBias = ValueType::kId == Fp16::kId ? 8.0f : 0.0f;
    static constexpr float kRoom = ValueType::kId == Fp16::kId ? 15.0f : 8.0f;
    // Workgroups of a compute unit: registers of a wave.
    static constexpr int kPerCu = DP == 256 || (DP == 128 && (kWide || QT == 2)) ? 1 : 2;
    static constexpr uint32_t kQueries = 16 * QT, kQueryShift = QT == 1 ? 4 : 5;

    // query: dims of the lane's k index, for the wide instruction one a register
    static constexpr int kQueryRegs = kWide ? DP / 16 : DP / 32;
    u32x4 q[QT][kQueryParts][kQueryRegs];
    u32x4 k[kGroups][kKeyLoads];
    uint32_t v[kGroups][4][kVH][kVW];
    f32x4 o[QT][DP / 16];

    // The first dim of the lane's 16 bytes (8-bit: of either half) of load s.
    static __device__ uint32_t key_dim(int s, uint32_t g) { return (s * 4 + g) * kE; }
    static __device__ uint32_t value_dim(int h, uint32_t n) { return h * 16 * kVE + n * kVE; }

    template <bool EXACT>
    __device__ void load_query(int tile, const char *row, bool there, uint32_t g, uint32_t dim)
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
                q[tile][0][s] = x[0];
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
                        q[tile][t][s][i] = ua >> 16 | ub;
                        a = __builtin_isfinite(a) ? a - as_float(ua) : 0.0f;
                        b = __builtin_isfinite(b) ? b - as_float(ub) : 0.0f;
                    }
                }
            }
        }
    }

    template <bool EXACT, bool NT>
    __device__ void load_keys(const char *const (&row)[kGroups], uint32_t g, uint32_t dim)
    {
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
            for (int s = 0; s < kKeyLoads; ++s) {
                if (EXACT || key_dim(s, g) < dim)
                    k[gr][s] = load_piece<NT>(row[gr] + s * 64);
                else
                    k[gr][s] = u32x4{0, 0, 0, 0};
            }
    }

    template <bool EXACT, bool NT>
    __device__ void load_values(const char *const (&row)[kGroups][4], uint32_t n, uint32_t dim)
    {
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < kVH; ++h) {
                    // (columns past dim are stored nowhere)
                    if (EXACT || value_dim(h, n) < dim) {
                        const Words *from = (const Words *)(row[gr][i] + h * 16 * kVE * kBytes);
                        const Words x = NT ? __builtin_nontemporal_load(from) : *from;
                        __builtin_memcpy(v[gr][i][h], &x, sizeof x);
                    }
                }
    }

    __device__ void scores(f32x4 (&s)[QT][kGroups]) const
    {
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr)
                s[t][gr] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int l = 0; l < kKeyLoads; ++l)
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
                if constexpr (kWide) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int t = 0; t < QT; ++t)
                            s[t][gr] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                as_float(k[gr][l][e]), as_float(q[t][0][l][e]), s[t][gr], 0, 0, 0);
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
                        for (int part = kQueryParts - 1; part >= 0; --part)
#pragma unroll
                            for (int t = 0; t < QT; ++t)
                                s[t][gr] = multiply<KeyType>(a, q[t][part][2 * l + half], s[t][gr]);
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < QT; ++t)
                        s[t][gr] = multiply<KeyType>(k[gr][l], q[t][0][l], s[t][gr]);
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
    __device__ void accumulate(const float (&p)[QT][kGroups][4])
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
#pragma unroll
                            for (int t = 0; t < QT; ++t)
                                o[t][h * kVE + j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                    as_float(v[gr][i][h][j]), p[t][gr][i], o[t][h * kVE + j], 0, 0, 0);
        } else {
            u32x4 w[QT][kWeightParts];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = p[t][e / 4][e % 4];
                split8<ValueType, kWeightParts>(x, w[t]);
            }
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
                            add_parts(h * kVE + 4 * c + j, a[j], w);
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
                            add_parts(h * kVE + 2 * c + j, a[j], w);
                    }
                }
        }
    }

    __device__ void add_parts(int c, u32x4 a, const u32x4 (&w)[QT][kWeightParts])
    {
#pragma unroll
        for (int part = kWeightParts - 1; part >= 0; --part)
#pragma unroll
            for (int t = 0; t < QT; ++t)
                o[t][c] = multiply<ValueType>(a, w[t][part], o[t][c]);
    }

    // The dim of value i of accumulator t.
    static __device__ uint32_t result_dim(int t, uint32_t g, int i)
    {
        return t / kVE * 16 * kVE + (4 * g + i) * kVE + t % kVE;
    }
};

// A matrix instruction's result is ready some issue slots after it, for which the
// compiler fills in waits; of a branch that is taken in between it counts too few
// (binary32 scores read behind one came out with old values in their last register).
// So no branch follows such instructions before these waits.  (A test follows the paths
// through the built code.)
__device__ inline void matrix_done()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7");
    __builtin_amdgcn_sched_barrier(0);
}

template <int QT, int GROUPS>
__device__ inline void matrix_done(f32x4 (&c)[QT][GROUPS])
{
    // (the last of them first; the others are older)
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" : "+v"(c[QT - 1][GROUPS - 1]));
#pragma unroll
    for (int i = 0; i < QT * GROUPS - 1; ++i)
        asm volatile("" : "+v"(c[i / GROUPS][i % GROUPS]));
}

// A value that is the same in every lane, in a scalar register.
__device__ inline uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

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
// sequence of 1000 tokens x 8 ranks took 16.3 us in place of 9.6, 29 odd ones 142 in
// place of 22.)
__device__ inline void share_pair(float *to, float a, float b)
{
    const f32x2 v = {a, b};
    __hip_atomic_store((uint64_t *)to, __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}

__device__ inline f32x2 shared_pair(const float *from)
{
    const uint64_t v = __hip_atomic_load((const uint64_t *)from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return __builtin_bit_cast(f32x2, v);
}

__device__ inline void shared_stores_done()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// The inclusive sum over the lanes up to this one.
__device__ inline uint32_t scan64(uint32_t x)
{
    x += lane_move<0x111>(x);  // within rows of 16: 1, 2, 4 and 8 lanes on
    x += lane_move<0x112>(x);
    x += lane_move<0x114>(x);
    x += lane_move<0x118>(x);
    x += __builtin_amdgcn_update_dpp(0u, x, 0x142, 0xa, 0xf, false);  // the row before's last
    x += __builtin_amdgcn_update_dpp(0u, x, 0x143, 0xc, 0xf, false);  // the half before's
    return x;
}

// Parts of a sum that are loaded at once.  (With eight, one sequence of 1000 tokens x 8
// ranks took 10.4 us in place of 10.7, but 29 odd ones 17.5 in place of 16.9 and 32 windows
// of 4096 x 4 ranks with 32 query heads of 256 108.8 in place of 106.6.)
constexpr uint32_t kJoinLoads = 4;

// Sequences that a wave has in its lanes.
constexpr uint32_t kSmallBatch = 64;

// What a workgroup has in LDS.
template <typename X, int DP>
struct AttendShared {
    uint64_t rows[kAttendWaves][X::kTokens];      // a tile's rows: byte offsets in a pool
    float scales[kAttendWaves][2][X::kTokens];    // a tile's scales, of keys and of values
    float sums[kAttendWaves][X::kQueries][DP + 4];
    float refs[kAttendWaves][X::kQueries], weights[kAttendWaves][X::kQueries];
    uint32_t bad[kAttendWaves], last;
    uint32_t found[kAttendWaves][2];
};

// (The code is kept short, with one copy of everything: a call of few tokens runs
// through it once, from memory.)
template <typename T, bool EIGHT, int DP, int QT, bool EXACT, bool EIGHT_OUT>
__global__ __launch_bounds__(kAttendThreads, (Tile<T, EIGHT, DP, QT>::kPerCu))
void cache_attend(CacheAttentionArgs p)
{
    typedef Tile<T, EIGHT, DP, QT> X;
    __shared__ __align__(16) AttendShared<X, DP> lds;
    const uint32_t lane = threadIdx.x & 63u, wave = uniform(threadIdx.x >> 6);
    const uint32_t n = lane & 15u, g = lane >> 4;
    const uint32_t dim = EXACT ? (uint32_t)DP : p.cache.dim;
    const uint32_t group = p.group;
    const uint64_t capacity = p.table_pages * p.cache.page_tokens;
    const float factor = p.scale * kLog2e;
    uint32_t *counters = (uint32_t *)p.work;

    // ---- this team's share of the row of all steps ---------------------------------
    // A small batch: a lane has a sequence, and every wave all of them.  Else a thread
    // has some, and the workgroup all.
    const bool small = p.seqs <= kSmallBatch;
    const int32_t lane_length = small && lane < p.seqs ? p.lengths[lane] : 0;
    // The pointer tables' first use costs a trip to memory, on the way beside this one.
    touch(p.q);
    touch(p.keys);
    touch(p.values);
    touch(p.out);
    if constexpr (EIGHT) {
        touch(p.key_scales);
        touch(p.value_scales);
    }
    auto length_of = [&](uint32_t seq) {  // (the same in every lane)
        return small ? __builtin_amdgcn_readlane(lane_length, seq) : p.lengths[seq];
    };
    const uint32_t chunk = (p.seqs + kAttendThreads - 1u) / kAttendThreads;
    const uint32_t from = small ? lane : threadIdx.x * chunk;
    const uint32_t to = small ? lane + 1u : from + chunk;
    // Steps of all sequences (of one unit each), of the lane's, and of those before.
    struct Steps {
        uint32_t all, mine, before;
    };
    auto sum_up = [&](uint32_t shift, uint32_t most) {  // of 2^shift tokens, `most` of a sequence at most
        uint32_t mine = 0;
        for (uint32_t s = from; s < to && s < p.seqs; ++s) {
            uint32_t first, end;
            attended(small ? lane_length : p.lengths[s], capacity, p.window, &first, &end);
            const uint32_t steps = steps_of(first, end, shift);
            mine += steps < most ? steps : most;
        }
        uint32_t before = scan64(mine);
        uint32_t all = __builtin_amdgcn_readlane(before, 63);
        before -= mine;
        if (!small) {
            __syncthreads();
            if (lane == 0)
                lds.found[wave][0] = all;
            __syncthreads();
            all = 0;
            for (uint32_t w = 0; w < kAttendWaves; ++w) {
                before += w < wave ? lds.found[w][0] : 0u;
                all += lds.found[w][0];
            }
            all = uniform(all);
        }
        return Steps{all, mine, before};
    };
    const CacheCall call = {p.seqs,          p.nranks,       p.cache.heads, group, X::kQueryShift, X::kTokenShift,
                            p.passes, gridDim.x, dim * 2u * X::kBytes};
    Steps sums;
    const CacheChoice choice = choose(call, sum_up, &sums);
    const CacheTeams &teams = choice.teams;
    const bool alone = choice.alone;
    auto steps_in = [&](uint32_t first, uint32_t end) { return steps_of(first, end, teams.shift); };
    auto steps_at = [&](int32_t length) {
        uint32_t first, end;
        attended(length, capacity, p.window, &first, &end);
        return steps_in(first, end);
    };
    const uint32_t across = p.cache.heads * teams.tiles;  // units of a sequence and rank
    const uint32_t row = sums.all * across;  // steps of a rank
    const uint32_t mine = sums.mine * across, before = sums.before * across;
    const CachePlan plan(row * p.nranks, alone ? gridDim.x * kAttendWaves : gridDim.x);
    const uint32_t team = alone ? wave : 0u;
    const uint32_t share = plan.share(blockIdx.x, team, gridDim.x);
    const uint32_t begin = share == ~0u ? 0u : plan.start(share);
    uint32_t left = share == ~0u ? 0u : plan.start(share + 1u) - begin;
    uint32_t rank = p.nranks == 1u ? 0u : begin / row, seq, unit;
    if (small) {
        const uint32_t at = begin - rank * row;
        seq = (uint32_t)__builtin_ctzll(__ballot(at >= before && at - before < mine));
        unit = at - __builtin_amdgcn_readlane(before, seq);
    } else {
        __syncthreads();
        for (uint32_t i = 0; i < (alone ? kAttendWaves : 1u); ++i) {
            const uint32_t s = plan.share(blockIdx.x, i, gridDim.x);
            const uint32_t at = s == ~0u ? 0u : plan.start(s) % row;
            if (at >= before && at - before < mine) {
                uint32_t b = before, e = from;
                for (uint32_t x; x = steps_at(p.lengths[e]) * across, at - b >= x; ++e)
                    b += x;
                lds.found[i][0] = e;
                lds.found[i][1] = at - b;
            }
        }
        __syncthreads();
        seq = uniform(lds.found[team][0]);
        unit = uniform(lds.found[team][1]);
    }
    if (left == 0)  // (from here on waves that are alone meet no more)
        return;
    int32_t length = length_of(seq);
    uint32_t step0 = unit;  // the sequence's step, until the unit's number is known
    unit = across == 1u ? 0u : step0 / steps_at(length);
    step0 -= unit * steps_at(length);
    uint32_t here = begin - step0;  // the unit's first step in the row

    const uint32_t wave0 = alone ? wave : 0u;                // the team's first
    const uint32_t member = alone ? lane : threadIdx.x;      // lane of the team
    const uint32_t beside = alone ? 0u : wave % teams.side;  // the wave's place among those on its tokens
    const uint32_t behind = alone ? 0u : wave / teams.side;
    const uint32_t most_queries = X::kQueries * teams.side < group ? X::kQueries * teams.side : group;
    const uint32_t waves_deep = teams.waves / teams.side;
    const uint32_t mine0 = beside * X::kQueries;            // the wave's queries among the team's
    auto meet = [&] {
        if (alone)
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        else
            __syncthreads();
    };

    auto pieces = [&](auto nt) {
        constexpr bool NT = decltype(nt)::value;
        for (;;) {
            // ---- a piece: steps [step0, step1) of a unit ----------------------------
            const uint32_t kv = teams.tiles == 1u ? unit : unit / teams.tiles, tile = unit - kv * teams.tiles;
            uint32_t first, end;
            const bool fine = attended(length, capacity, p.window, &first, &end);
            const uint32_t steps = steps_in(first, end);
            const uint32_t step1 = left < steps - step0 ? step0 + left : steps;
            const uint32_t t1 = step1 == steps ? end : first + (step1 << teams.shift);
            const uint32_t query0 = tile * X::kQueries * teams.side;  // of the group
            const uint32_t queries = group - query0 < most_queries ? group - query0 : most_queries;
            const uint32_t head0 = kv * group + query0;

            X x;
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                const uint32_t q = mine0 + 16 * t + n;
                const char *at = p.q[rank] + (seq * p.q_stride + (uint64_t)(head0 + q) * dim) * T::kBytes;
                x.template load_query<EXACT>(t, at, q < queries, g, dim);
            }
            float ref[QT], sum[QT];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                ref[t] = -__builtin_inff();
                sum[t] = 0.0f;
#pragma unroll
                for (int c = 0; c < DP / 16; ++c)
                    x.o[t][c] = f32x4{0, 0, 0, 0};
            }
            // (where dim is not DP some lanes load none)
#pragma unroll
            for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x.drop_values(gr, i);
            bool bad = !fine;

            const char *keys = p.keys[rank], *values = p.values[rank];
            const float *scales = EIGHT ? (lane < 32u ? p.key_scales[rank] : p.value_scales[rank]) : nullptr;
            const int32_t *table = p.table + seq * p.table_pages;
            const uint32_t mine_at = lane % X::kTokens;
            const uint32_t kd = X::key_dim(0, g) * X::kBytes, vd = X::value_dim(0, n) * X::kBytes;
            uint32_t t0 = first + (step0 << teams.shift) + behind * X::kTokens;
            const uint32_t tend = mine0 < queries ? t1 : 0u;  // a wave without queries has no tokens

            // page and place of the lane's token of the tile at t (past the end: of the last one)
            auto look = [&](uint32_t t, uint32_t &place) {
                t += mine_at;
                t = t < t1 ? t : t1 - 1u;
                const uint32_t i = p.cache.page_of(t);
                place = t - i * p.cache.page_tokens;
                return table[i];
            };
            float scale_next = 0.0f;
            // A tile's rows to LDS.  (A page that is none: the cache's first row, and NaN in the end.)
            auto rows = [&](int32_t page, uint32_t place) {
                if ((uint32_t)page >= p.cache.pages) {
                    bad = true;
                    page = 0;
                    place = 0;
                }
                lds.rows[wave][mine_at] = p.cache.at((uint32_t)page, place, kv) * X::kBytes;
                if constexpr (EIGHT)
                    scale_next = scales[p.cache.scale_at((uint32_t)page, place, kv)];
                __builtin_amdgcn_wave_barrier();
            };
            // Where the tile's rows are: read from LDS ahead of its loads where there are
            // registers for that, beside the scores' instructions (QT 1: 64 x 8192 tokens x 8
            // ranks 318 us; before those 324, each at its loads 322 where the rest took 314).
            const char *krow[X::kGroups], *vrow[X::kGroups][4];
            auto find_keys = [&] {
#pragma unroll
                for (int gr = 0; gr < X::kGroups; ++gr)
                    krow[gr] = keys + lds.rows[wave][gr * 16 + n] + kd;
            };
            auto find_values = [&] {
#pragma unroll
                for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        vrow[gr][i] = values + lds.rows[wave][gr * 16 + 4 * g + i] + vd;
            };
            auto load_keys = [&] {
                if constexpr (QT != 1)
                    find_keys();
                x.template load_keys<EXACT, NT>(krow, g, dim);
            };
            auto load_values = [&] {
                if constexpr (QT != 1)
                    find_values();
                x.template load_values<EXACT, NT>(vrow, n, dim);
                __builtin_amdgcn_wave_barrier();
            };
            if (t0 < tend) {
                uint32_t place, place_next;
                int32_t page = look(t0, place), page_next = look(t0 + teams.pass, place_next);
                rows(page, place);
                if constexpr (QT == 1) {
                    find_keys();
                    find_values();
                }
                load_keys();
                load_values();
                for (; t0 < t1; t0 += teams.pass) {
                    float ks[X::kGroups][4], vs[X::kGroups][4];
                    if constexpr (EIGHT) {
                        lds.scales[wave][lane / 32u][mine_at] = scale_next;
                        __builtin_amdgcn_wave_barrier();
#pragma unroll
                        for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                ks[gr][i] = lds.scales[wave][0][gr * 16 + 4 * g + i];
                                vs[gr][i] = lds.scales[wave][1][gr * 16 + 4 * g + i];
                            }
                        __builtin_amdgcn_wave_barrier();
                    }
                    rows(page_next, place_next);
                    page_next = look(t0 + 2 * teams.pass, place_next);
                    f32x4 s[QT][X::kGroups];
                    x.scores(s);
                    if constexpr (QT == 1) {
                        find_keys();
                        find_values();
                    }
                    matrix_done(s);
                    // (also behind the last tile, where there is nothing to load: behind a branch the
                    // compiler would wait for the keys where it needs the values)
                    load_keys();
                    float w[QT][X::kGroups][4];
#pragma unroll
                    for (int t = 0; t < QT; ++t)
#pragma unroll
                        for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float f = factor;
                                if constexpr (EIGHT)
                                    f = f * ks[gr][i];
                                w[t][gr][i] = s[t][gr][i] * f;
                            }
                    if (t0 + X::kTokens > t1) {
#pragma unroll
                        for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (t0 + gr * 16 + 4 * g + i >= t1) {
#pragma unroll
                                    for (int t = 0; t < QT; ++t)
                                        w[t][gr][i] = -__builtin_inff();
                                    if constexpr (EIGHT)
                                        vs[gr][i] = 0.0f;
                                    x.drop_values(gr, i);
                                }
                    }
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                        float most = -__builtin_inff();
#pragma unroll
                        for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                most = w[t][gr][i] > most ? w[t][gr][i] : most;
                        if (__ballot(most > ref[t] + (X::kRoom - X::kBias)) != 0) {
                            // (a NaN raises nothing; it reaches the sums by its own weight)
                            // The reference stays finite: a score of infinity has an infinite weight.
                            most = __builtin_fminf(max_query(most), __FLT_MAX__);
                            const float next = most > ref[t] ? most : ref[t];
                            const float shift = next == -__builtin_inff() ? 0.0f : next;
                            const float keep = __builtin_amdgcn_exp2f(ref[t] - shift);
                            sum[t] = sum[t] * keep;
#pragma unroll
                            for (int c = 0; c < DP / 16; ++c)
                                x.o[t][c] = x.o[t][c] * keep;
                            ref[t] = next;
                        }
                        const float shift = (ref[t] == -__builtin_inff() ? 0.0f : ref[t]) - X::kBias;
#pragma unroll
                        for (int gr = 0; gr < X::kGroups; ++gr)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                w[t][gr][i] = __builtin_amdgcn_exp2f(w[t][gr][i] - shift);
                                sum[t] += w[t][gr][i];
                                if constexpr (EIGHT)
                                    w[t][gr][i] = w[t][gr][i] * vs[gr][i];
                            }
                    }
                    x.accumulate(w);
                    if constexpr (!EXACT)  // (whose loads have branches)
                        matrix_done();
                    load_values();
                    if constexpr (EXACT)
                        matrix_done();
                }
            }

            // ---- the waves' sums to LDS -----------------------------------------------
            const bool any_bad = __ballot(bad) != 0;
            if (lane == 0)
                lds.bad[wave] = any_bad;
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                sum[t] = sum_query(sum[t]);
                if (g == 0) {
                    lds.refs[wave][16 * t + n] = ref[t];
                    lds.weights[wave][16 * t + n] = sum[t];
                }
#pragma unroll
                for (int c = 0; c < DP / 16; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        lds.sums[wave][16 * t + n][X::result_dim(c, g, i)] = x.o[t][c][i];
            }
            meet();

            // ---- and together: the waves', then, where several teams share the unit, those of
            // a group of teams, then those of the groups; by the last team to arrive ---------
            // A lane of the team takes eight dims of a query, then of another.
            constexpr uint32_t kPieces = DP / 8;
            const uint32_t d0 = member % kPieces * 8u;
            const uint32_t slot_floats = most_queries * (DP + 2u);
            const bool whole = step0 == 0 && step1 == steps;
            const CacheJoin join(whole ? share : plan.owner(here),
                                 whole ? share : plan.owner(here + steps - 1u));
            // An infinite value times a later part of its weight, which is zero or negative as
            // often as not, makes NaN of the infinity that it stands for.  A column that is NaN
            // although its weights are finite is the sum of the infinities and NaNs in it.
            // (Looked for here, among the eight sums of a lane, it costs 1 x 1000 tokens 0.2 us of 10.2
            // and windows with 32 heads of 256 1 of 106; among a wave's accumulators 4 of 106.)
            auto infinities = [&](float (&y)[8]) {
                float f[8] = {};
#pragma unroll 1
                for (uint32_t t = first + (step0 << teams.shift); t < t1; ++t) {
                    const uint32_t i = p.cache.page_of(t), place = t - i * p.cache.page_tokens;
                    const uint32_t page = (uint32_t)table[i];
                    if (page >= p.cache.pages)
                        continue;
                    const char *at = values + (p.cache.at(page, place, kv) + d0) * X::kBytes;
                    float v[8];
                    if constexpr (EIGHT) {
                        const float s = p.value_scales[rank][p.cache.scale_at(page, place, kv)];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] = __builtin_amdgcn_cvt_f32_fp8((int)((const uint8_t *)at)[e], 0) * s;
                    } else if constexpr (!X::kWide) {
                        widen_piece<T>(load_piece<false>(at), v);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[e] += __builtin_isfinite(v[e]) ? 0.0f : v[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = __builtin_isnan(y[e]) && !__builtin_isfinite(f[e]) ? f[e] : y[e];
            };
            uint32_t stage = 0, parts = 0;  // slots of a sum
            for (;;) {
                const CacheJoin::Parts from_slots = join.parts(share, stage);
                const bool done = stage == 0 ? whole : stage == 2 || join.groups() == 1u;
                for (uint32_t q = member / kPieces; q < queries; q += 64u * teams.waves / kPieces) {
                    float top = -__builtin_inff(), total = 0.0f, y[8] = {};
                    const uint32_t in_slot = q * DP + d0 / 4u;
                    // `count` parts of references r, sums of weights l and sums f
                    auto add = [&](auto parts_at_once, uint32_t count, const float *r, const float *l,
                                   const float (*f)[8]) {
                        constexpr uint32_t N = decltype(parts_at_once)::value;
                        const float last = top;
#pragma unroll
                        for (uint32_t j = 0; j < N; ++j)
                            top = r[j] > top ? r[j] : top;
                        const float shift = top == -__builtin_inff() ? 0.0f : top;
                        const float a = __builtin_amdgcn_exp2f(last - shift);
                        total = total * a;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            y[e] = y[e] * a;
#pragma unroll
                        for (uint32_t j = 0; j < N; ++j)
                            if (j < count) {
                                const float b = __builtin_amdgcn_exp2f(r[j] - shift);
                                total += l[j] * b;
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    y[e] += f[j][e] * b;
                            }
                    };
                    // All loads are under way at once; past the last part the last again, left out.
                    if (stage == 0) {
                        float r[kAttendWaves], l[kAttendWaves], f[kAttendWaves][8];
#pragma unroll
                        for (uint32_t j = 0; j < kAttendWaves; ++j) {
                            const uint32_t deep = j < waves_deep ? j : waves_deep - 1u;
                            const uint32_t w = wave0 + q / X::kQueries + deep * teams.side;
                            const uint32_t k = q % X::kQueries;
                            r[j] = lds.refs[w][k];
                            l[j] = lds.bad[w] != 0 ? __builtin_nanf("") : lds.weights[w][k];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                f[j][e] = lds.sums[w][k][d0 + e];
                        }
                        add(std::integral_constant<uint32_t, kAttendWaves>{}, waves_deep, r, l, f);
                        if constexpr (!X::kWide) {
                            float zero = 0.0f;  // NaN behind an infinity or NaN
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                zero = __builtin_fmaf(y[e], 0.0f, zero);
                            // (columns past dim are no part of a row)
                            if (__builtin_expect(__builtin_isnan(zero) && __builtin_isfinite(total) &&
                                                     (EXACT || d0 < dim),
                                                 false))
                                infinities(y);
                        }
                    } else {
                        for (uint32_t i = 0; i < parts; i += kJoinLoads) {
                            float r[kJoinLoads], l[kJoinLoads], f[kJoinLoads][8];
#pragma unroll
                            for (uint32_t j = 0; j < kJoinLoads; ++j) {
                                const uint32_t at = i + j < parts ? i + j : parts - 1u;
                                const uint32_t part =
                                    at == 0 ? from_slots.first : from_slots.next + (at - 1u) * from_slots.by;
                                const float *slot = p.slots + (uint64_t)part * slot_floats;
                                const float *pairs = slot + in_slot;
                                const f32x2 s = shared_pair(slot + most_queries * DP + 2 * q);
                                r[j] = s[0];
                                l[j] = s[1];
#pragma unroll
                                for (int e = 0; e < 8; e += 2) {
                                    const f32x2 v = shared_pair(pairs + e * kPieces);
                                    f[j][e] = v[0];
                                    f[j][e + 1] = v[1];
                                }
                            }
                            add(std::integral_constant<uint32_t, kJoinLoads>{}, parts - i, r, l, f);
                        }
                    }
                    if (!done) {
                        // (a group's sums: in the place of its first, which this wave alone has read)
                        const uint32_t to_slot = join.slot(stage == 0 ? share : join.first(share));
                        float *slot = p.slots + (uint64_t)to_slot * slot_floats;
#pragma unroll
                        for (int e = 0; e < 8; e += 2)
                            share_pair(slot + in_slot + e * kPieces, y[e], y[e + 1]);
                        if (d0 == 0)
                            share_pair(slot + most_queries * DP + 2 * q, top, total);
                        continue;
                    }
                    const bool empty = length == 0;
                    const uint64_t out_row = (uint64_t)seq * p.heads + head0 + q;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = empty ? 0.0f : y[e] / total;
                    if (p.has_lse != 0 && d0 == 0) {
                        const float shift = (top == -__builtin_inff() ? 0.0f : top) - X::kBias;
                        p.lse[rank][out_row] = empty ? -__builtin_inff() : shift * kLn2 + __builtin_logf(total);
                    }
                    if constexpr (EIGHT_OUT) {
                        // 16 neighbouring lanes hold the 128 columns of a scale
                        const float s = scale_of(max16(max_bits(y)));
                        store_eights<false>(p.out[rank] + out_row * dim + d0, to_eights(y, s));
                        if (d0 % AR_SCALE_BLOCK == 0) {
                            const uint64_t block = ((uint64_t)(head0 + q) * dim + d0) / AR_SCALE_BLOCK;
                            p.out_scales[rank][block * p.seqs + seq] = s;
                        }
                    } else if (EXACT || d0 < dim) {
                        char *at = p.out[rank] + (out_row * dim + d0) * T::kBytes;
                        constexpr int E = kPiece<T>;
#pragma unroll
                        for (int i = 0; i < 8 / E; ++i) {
                            float f[E];
#pragma unroll
                            for (int e = 0; e < E; ++e)
                                f[e] = y[i * E + e];
                            store_piece<false>(at + i * 16, narrow_piece<T>(f));
                        }
                    }
                }
                if (done)
                    break;
                // Whether this team is the last to come here.
                const uint32_t counter = stage == 0 ? join.group_counter(share) : join.unit_counter();
                const uint32_t count = stage == 0 ? join.last(share) - join.first(share) + 1u : join.groups();
                shared_stores_done();
                meet();
                uint32_t last = 0;
                if (member == 0) {
                    const uint32_t old = __hip_atomic_fetch_add(counters + counter, 1u, __ATOMIC_RELAXED,
                                                                __HIP_MEMORY_SCOPE_AGENT);
                    last = old + 1u == count;
                    if (last != 0)
                        __hip_atomic_store(counters + counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    lds.last = last;
                }
                meet();
                if ((alone ? uniform(last) : uniform(lds.last)) == 0)
                    break;
                ++stage;
                parts = count;
            }

            left -= step1 - step0;
            if (left == 0)
                return;
            here += steps;
            step0 = 0;
            if (++unit == across) {
                unit = 0;
                if (++seq == p.seqs) {
                    seq = 0;
                    ++rank;
                }
                length = length_of(seq);
            }
            meet();  // the sums in LDS are read before the next piece's are written
        }
    };
    if (choice.stream)
        pieces(std::true_type{});
    else
        pieces(std::false_type{});
}

// Workgroups of a launch at most: what fits the compute units at once (of 512 at most: the
// workspace's counters have room for so many).
inline uint32_t attend_most(int per_cu, int cu_count)
{
    static_assert(2 * 512 * kAttendWaves * 4 * sizeof(uint32_t) <= AR_CACHE_WORKSPACE_ZEROS, "four counters a team");
    return (uint32_t)(per_cu * (cu_count < 512 ? cu_count : 512)) / 8u * 8u;
}

template <typename T, bool EIGHT, int DP, int QT, bool EXACT, bool EIGHT_OUT>
hipError_t enqueue_attend(CacheAttentionArgs args, int cu_count, hipStream_t stream)
{
    typedef Tile<T, EIGHT, DP, QT> X;
    const uint64_t tokens = most_attended(args.table_pages * args.cache.page_tokens, args.window);
    args.passes = passes_of_a_step(args.seqs, args.nranks, args.cache.heads, args.group,
                                   X::kTokenShift, tokens);
    // (a call of few steps has fewer workgroups)
    const CacheTeams teams(args.group, X::kQueryShift, X::kTokenShift, args.passes, false);
    const uint64_t units = (uint64_t)args.nranks * args.cache.heads * args.seqs * teams.tiles;
    const uint64_t steps = ((tokens - 1u) >> teams.shift) + 1u;
    uint64_t grid = attend_most(X::kPerCu, cu_count);
    if (steps < grid && units * steps < grid)
        grid = (units * steps + 7u) / 8u * 8u;
    hipLaunchKernelGGL((cache_attend<T, EIGHT, DP, QT, EXACT, EIGHT_OUT>), dim3((uint32_t)grid),
                       dim3(kAttendThreads), 0, stream, args);
    return hipGetLastError();
}

// One of the kernel families, each compiled in a file of its own.
template <typename T, bool EIGHT, int QT>
hipError_t launch_attend(const CacheAttentionArgs &args, bool eight_out, int cu_count,
                         hipStream_t stream)
#ifdef AR_ATTEND_FAMILY
{
    auto pick = [&](auto padded) {
        constexpr int DP = decltype(padded)::value;
        if (args.cache.dim != DP)
            return enqueue_attend<T, EIGHT, DP, QT, false, false>(args, cu_count, stream);
        if constexpr (DP % AR_SCALE_BLOCK == 0)
            if (eight_out)
                return enqueue_attend<T, EIGHT, DP, QT, true, true>(args, cu_count, stream);
        return enqueue_attend<T, EIGHT, DP, QT, true, false>(args, cu_count, stream);
    };
    switch (padded_dim(args.cache.dim)) {
    case 64: return pick(std::integral_constant<int, 64>{});
    case 128: return pick(std::integral_constant<int, 128>{});
    }
    if constexpr (QT == 1 || T::kBytes == 2)
        return pick(std::integral_constant<int, 256>{});
    return hipErrorInvalidValue;
}
#else
    ;
#endif

}  // namespace ar
