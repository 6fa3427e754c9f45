// block_matmul_tile.hip -- the block-scaled 8-bit product for many rows.
//
// A workgroup computes a tile of 256 rows x 256 output columns with eight
// waves, or 128 x 128 with four where there would be too few of the larger
// ones; a step is one block of 128 of k (of all ranks' k, one rank after the
// other, in the form that sums over the ranks).  A step's inputs go from
// global memory straight to LDS (no registers in between), two steps' worth
// in turn, so that one is loaded while the other is multiplied.  A wave
// computes 64 rows x 128 (64) columns in 32x32 tiles: the columns of a wave
// lie in one weight scale block, so a step's scale is one number a lane and
// row tile, applied with a fused multiply-add to the running sums.
//
// LDS rows are the 128 bytes of a step, in eight pieces of 16; piece c of row
// r is kept at place c ^ (r / 2 % 8).  Two rows cover all banks once, so 16
// rows of one piece, read together, lie in 16 different places (with r % 8,
// rows 8 apart met: half of the LDS cycles were conflicts).  A direct load
// writes its lanes' pieces one after the other, so the exchange is made in
// the lanes' global addresses.
#include <type_traits>

#include "block_device.hpp"
#include "block_internal.hpp"
#include "block_matmul.hpp"

namespace ar {

// NT: 32-column tiles of a wave (it has two 32-row ones).  WM, WN: waves along
// rows and columns.
template <int NT, int WM, int WN>
struct TileShape {
    static constexpr uint32_t kRows = WM * 64u, kCols = WN * NT * 32u, kWaves = WM * WN;
    static constexpr uint32_t kRowBytes = kRows * 128u, kColBytes = kCols * 128u;  // of a step
    static constexpr uint32_t kLoadsM = kRows / 8u / kWaves, kLoadsN = kCols / 8u / kWaves;
};

template <typename T, int NT, int WM, int WN, bool REDUCE>
__global__ __launch_bounds__(WM * WN * 64, 2) void matmul_tile(MatmulArgs p)
{
    constexpr bool kExact = T::kBytes == 4;
    typedef TileShape<NT, WM, WN> S;
    // rows of both steps, then columns of both
    __shared__ __align__(128) char lds[2 * (S::kRowBytes + S::kColBytes)];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // Workgroup w runs on XCD w % 8: each XCD takes consecutive tiles, and 32
    // consecutive tiles are 8 x 4, which its second-level cache serves with 12
    // tiles' inputs instead of 64.
    const uint32_t mt = (p.rows + S::kRows - 1) / S::kRows, nt = (p.n + S::kCols - 1) / S::kCols;
    const uint32_t tiles = mt * nt * (REDUCE ? 1u : p.nranks);
    uint32_t t = (blockIdx.x & 7u) * ((tiles + 7u) / 8u) + blockIdx.x / 8u;
    if (blockIdx.x / 8u >= (tiles + 7u) / 8u || t >= tiles)
        return;
    const uint32_t rank0 = REDUCE ? 0u : t / (mt * nt);
    t -= rank0 * mt * nt;
    const uint32_t band = t / (mt * 4u);                      // four columns of tiles
    const uint32_t wide = nt - band * 4u < 4u ? nt - band * 4u : 4u;
    t -= band * mt * 4u;
    const uint32_t m0 = t / wide * S::kRows, n0 = (band * 4u + t % wide) * S::kCols;

    // This wave loads rows and columns eight at a time; rows past the end
    // repeat the last one, and what comes of them is not stored.
    uint32_t offm[S::kLoadsM], offn[S::kLoadsN];
    const uint32_t piece16 = ((lane & 7u) ^ (lane >> 4)) * 16u;  // even groups of eight; odd ^ 64
#pragma unroll
    for (uint32_t i = 0; i < S::kLoadsM; ++i) {
        const uint32_t r = (wave * S::kLoadsM + i) * 8u + (lane >> 3);
        offm[i] = (r < p.rows - m0 ? r : p.rows - m0 - 1u) * p.k + (piece16 ^ (i & 1u) * 64u);
    }
#pragma unroll
    for (uint32_t i = 0; i < S::kLoadsN; ++i) {
        const uint32_t r = (wave * S::kLoadsN + i) * 8u + (lane >> 3);
        offn[i] = (r < p.n - n0 ? r : p.n - n0 - 1u) * p.k + (piece16 ^ (i & 1u) * 64u);
    }
    static_assert(S::kLoadsM % 2 == 0 && S::kLoadsN % 2 == 0, "odd groups start on odd i");
    const uint32_t lds0 =
        __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds);
    const uint32_t tom = lds0 + wave * S::kLoadsM * 1024u;
    const uint32_t ton = lds0 + 2u * S::kRowBytes + wave * S::kLoadsN * 1024u;

    // This wave multiplies rows wm .. wm + 63 and columns wn .. wn + 32 NT - 1.
    const uint32_t wm = wave % WM * 64u, wn = wave / WM * (NT * 32u);
    const uint32_t l32 = lane & 31u, half = lane >> 5;
    const uint32_t place = l32 * 128u + ((half * 2u) ^ (l32 >> 1 & 7u)) * 16u;
    uint32_t m[2];
#pragma unroll
    for (uint32_t j = 0; j < 2; ++j) {
        const uint32_t row = m0 + wm + j * 32u + l32;
        m[j] = row < p.rows ? row : p.rows - 1u;
    }

    // What the next load reads: block kb of rank r, from these on.  The weight
    // scale is loaded like the others, by a vector instruction: a scalar one
    // shares its wait counter with LDS reads, which would then wait for it in
    // every step.
    const uint32_t nranks = REDUCE ? p.nranks : 1u;
    uint32_t r = 0, kb = 0;
    const char *a, *b;
    const float *sa, *sb;
    uint32_t sb_off = n0 + wn < p.n ? (n0 + wn) / 128u * p.kblocks : 0u;
    asm volatile("" : "+v"(sb_off));
    auto at_rank = [&] {
        a = p.a[rank0 + r] + (uint64_t)m0 * p.k;
        b = p.b[rank0 + r] + (uint64_t)n0 * p.k;
        sa = p.sa[rank0 + r];
        sb = p.sb[rank0 + r];
    };
    // Part `i` of its loads into half `stage` of LDS: eight rows and eight
    // columns.  A piece past the end of its row repeats the row's last one.
    auto load = [&](uint32_t stage, uint32_t i) {
        const int32_t over = (int32_t)(piece16 ^ (i & 1u) * 64u) - (int32_t)(p.k - 16u - kb * 128u);
        const uint32_t back = over > 0 ? (uint32_t)over : 0u;
        if (i < S::kLoadsM)
            to_lds(a, offm[i] - back, tom + stage * S::kRowBytes + i * 1024u);
        if (i < S::kLoadsN)
            to_lds(b, offn[i] - back, ton + stage * S::kColBytes + i * 1024u);
    };
    constexpr uint32_t kParts = S::kLoadsM > S::kLoadsN ? S::kLoadsM : S::kLoadsN;
    // Their scales (multiplied later: here that would wait for the loads
    // before), then on to the next block; after the last one the loads repeat.
    auto load_scales = [&](float (&s)[3]) {
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j)
            s[j] = sa[m[j]];
        s[2] = sb[sb_off];
        if (kb + 1u < p.kblocks) {
            ++kb;
            a += 128;
            b += 128;
            sa += p.rows;
            sb += 1;
        } else if (r + 1u < nranks) {
            kb = 0;
            ++r;
            at_rank();
        }
    };

    f32x16 acc[NT][2] = {};
    float s_next[3];
    at_rank();
#pragma unroll
    for (uint32_t i = 0; i < kParts; ++i)
        load(0, i);
    load_scales(s_next);

    // One step: multiplies half `stage`, loads the other one.  `left`: bytes of
    // the block that are in the row; those past it (TAIL) are zero in the
    // weights, and in the activations a repeat of the row's own, so that a NaN
    // there is one that the row has anyway.
    auto step = [&](uint32_t stage, auto tail, uint32_t left) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        // After this every wave's loads of this step are in LDS, and no wave
        // reads the other half any more.
        __syncthreads();
        float s[2] = {s_next[0] * s_next[2], s_next[1] * s_next[2]};
        // (here, where they are at hand: a wait for them further down would
        // also wait for the next step's loads)
        asm volatile("" : "+v"(s[0]), "+v"(s[1]));
        const char *pm = lds + stage * S::kRowBytes + wm * 128u;
        const char *pn = lds + 2u * S::kRowBytes + stage * S::kColBytes + wn * 128u;
        auto weights = [&](uint32_t i, uint32_t h) {
            i32x8 w = pieces(pn + i * 4096u, place ^ (h * 64u));
            if constexpr (decltype(tail)::value) {
#pragma unroll
                for (uint32_t e = 0; e < 8; ++e)
                    w[e] = (h * 4u + half * 2u + e / 4u) * 16u < left ? w[e] : 0;
            }
            return w;
        };
        i32x8 x[2][2], w[2];
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            x[0][h] = pieces(pm, place ^ (h * 64u));
            w[h] = weights(0, h);
        }
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h)
            x[1][h] = pieces(pm + 4096u, place ^ (h * 64u));
        __builtin_amdgcn_sched_barrier(0);
        // A tile's products are under way while the one before it is scaled.
        // The next step's loads go out between the products: all of them at
        // once would hold the first product back.
        f32x16 c[2];
#pragma unroll
        for (uint32_t i = 0; i < NT; ++i) {
            if (i > 0) {
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h)
                    w[h] = weights(i, h);
            }
#pragma unroll
            for (uint32_t j = 0; j < 2; ++j) {
                c[j] = block_sums32<kExact>(w, x[j]);
                __builtin_amdgcn_sched_barrier(0);
                if (i + j > 0) {
                    const uint32_t pi = j == 0 ? i - 1u : i, pj = j ^ 1u;
#pragma unroll
                    for (uint32_t e = 0; e < 16; ++e)
                        acc[pi][pj][e] = __builtin_fmaf(c[pj][e], s[pj], acc[pi][pj][e]);
                    // (done here: put off, it keeps every tile's registers)
                    asm volatile("" : "+v"(acc[pi][pj]));
                }
                if (i * 2u + j < kParts)
                    load(stage ^ 1u, i * 2u + j);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        load_scales(s_next);
#pragma unroll
        for (uint32_t e = 0; e < 16; ++e)
            acc[NT - 1][1][e] = __builtin_fmaf(c[1][e], s[1], acc[NT - 1][1][e]);
        asm volatile("" : "+v"(acc[NT - 1][1]));
    };
    uint32_t stage = 0;
    const uint32_t full = p.k / 128u;
    for (uint32_t q = 0; q < nranks; ++q) {
        for (uint32_t i = 0; i < full; ++i, stage ^= 1u)
            step(stage, std::false_type{}, 128u);
        if (full != p.kblocks) {
            step(stage, std::true_type{}, p.k % 128u);
            stage ^= 1u;
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    // The sums go through LDS, 32 rows x 32 NT columns of a wave at a time, so
    // that a store covers whole lines: 16-byte pieces, piece c of row r at
    // place c ^ (r % 8).
    __syncthreads();
    constexpr uint32_t kRow = NT * 32u * T::kBytes;
    static_assert(S::kWaves * 32u * kRow <= sizeof(lds), "the waves' parts fit");
    char *mine = lds + wave * (32u * kRow);
#pragma unroll
    for (uint32_t j = 0; j < 2; ++j) {
#pragma unroll
        for (uint32_t i = 0; i < NT; ++i) {
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) {
                const uint32_t col = i * 32u + q * 8u + half * 4u;
                float f[4];
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e)
                    f[e] = acc[i][j][q * 4u + e];
                uint32_t v[T::kBytes];
#pragma unroll
                for (uint32_t e = 0; e < 4 / T::kPerWord; ++e)
                    v[e] = T::narrow(f + e * T::kPerWord);
                const uint32_t at = col * T::kBytes;
                char *to = mine + l32 * kRow + (((at >> 4) ^ (l32 & 7u)) << 4) + (at & 15u);
                __builtin_memcpy(__builtin_assume_aligned(to, 4 * T::kBytes), v, 4 * T::kBytes);
            }
        }
        // (a wave's own LDS accesses are in order, and no other wave's are here)
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        constexpr uint32_t kPieces = kRow / 16u, kEach = 16u / T::kBytes;
#pragma unroll
        for (uint32_t u = 0; u < 32u * kPieces / 64u; ++u) {
            const uint32_t row = u * (64u / kPieces) + lane / kPieces;
            const uint32_t c = lane % kPieces;
            const u32x4 v = *(const u32x4 *)(mine + row * kRow + ((c ^ (row & 7u)) << 4));
            const uint32_t gm = m0 + wm + j * 32u + row, gn = n0 + wn + c * kEach;
            if (gm < p.rows && gn < p.n) {
                const uint64_t at = ((uint64_t)gm * p.n + gn) * T::kBytes;
                if constexpr (REDUCE) {
                    for (uint32_t o = 0; o < p.nranks; ++o)
                        store_row_piece<T>(p.out[o] + at, v, p.n - gn);
                } else {
                    store_row_piece<T>(p.out[rank0] + at, v, p.n - gn);
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

namespace {

template <typename T, int NT, int WM, int WN>
hipError_t enqueue_tile(const MatmulArgs &args, bool reduce, hipStream_t stream)
{
    typedef TileShape<NT, WM, WN> S;
    const uint32_t tiles = (args.rows + S::kRows - 1) / S::kRows *
                           ((args.n + S::kCols - 1) / S::kCols) * (reduce ? 1u : args.nranks);
    const dim3 grid((tiles + 7u) / 8u * 8u);
    if (reduce)
        hipLaunchKernelGGL((matmul_tile<T, NT, WM, WN, true>), grid, dim3(S::kWaves * 64), 0, stream,
                           args);
    else
        hipLaunchKernelGGL((matmul_tile<T, NT, WM, WN, false>), grid, dim3(S::kWaves * 64), 0, stream,
                           args);
    return hipGetLastError();
}

template <typename T>
hipError_t pick_tile(const MatmulArgs &args, bool reduce, bool large, hipStream_t stream)
{
    if constexpr (T::kBytes == 2)
        if (large)
            return enqueue_tile<T, 4, 4, 2>(args, reduce, stream);
    return enqueue_tile<T, 2, 2, 2>(args, reduce, stream);
}

}  // namespace

hipError_t launch_matmul_tile(const MatmulArgs &args, int out_dtype, bool reduce, bool large,
                              hipStream_t stream)
{
    switch (out_dtype) {
    case kBf16: return pick_tile<Bf16>(args, reduce, large, stream);
    case kFp16: return pick_tile<Fp16>(args, reduce, large, stream);
    default: return pick_tile<Fp32>(args, reduce, large, stream);
    }
}

}  // namespace ar
