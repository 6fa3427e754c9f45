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
// row tile, applied with a fused multiply-add to the running sums.  (Four
// 16x16x128 instructions in place of two 32x32x64 ones: 2 % slower.)
//
// On MI355X 8 x (4096 x 7168 x 8192) takes 1740 to 1840 us on random values,
// 2.09 to 2.21 PFLOP/s, and 1416 us, 2.72 PFLOP/s, on constant ones: the
// card's power sets the clock (1.5 to 1.8 against 2.3 GHz).  Of copies on
// random values, one without the scaling took 12 % less, one without the LDS
// reads 8 %, one without the loads 12 %.  The instructions alone reach 4.1
// PFLOP/s with the scaling on constant values, 3.25 on random ones.
//
// LDS rows are the 128 bytes of a step, in eight pieces of 16; piece c of row
// r is kept at place c ^ (r / 2 % 8).  Two rows cover all banks once, so 16
// rows of one piece, read together, lie in 16 different places (with r % 8,
// rows 8 apart met: half of the LDS cycles were conflicts).  A direct load
// writes its lanes' pieces one after the other, so the exchange is made in
// the lanes' global addresses.
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
    // LDS: rows of both steps, columns of both, scales of both (a float a row,
    // then 64 times the same for each 128 columns), a place that nothing reads
    static constexpr uint32_t kScaleWaves = kRows / 64u + kCols / 128u;
    static constexpr uint32_t kScaleBytes = kScaleWaves * 256u;
    static constexpr uint32_t kScalesAt = 2u * (kRowBytes + kColBytes);
    static constexpr uint32_t kUnusedAt = kScalesAt + 2u * kScaleBytes;
    static constexpr uint32_t kBytes = kUnusedAt + (kWaves - kScaleWaves) * 256u;
    static_assert(kScaleWaves < kWaves, "a wave is left to bring lines");
};

template <typename T, int NT, int WM, int WN, bool REDUCE>
__global__ __launch_bounds__(WM * WN * 64, 2) void matmul_tile(MatmulArgs p)
{
    constexpr bool kExact = T::kBytes == 4;
    typedef TileShape<NT, WM, WN> S;
    __shared__ __align__(128) char lds[S::kBytes];
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
    // What the next load reads: block kb of rank r, from these on.
    const uint32_t nranks = REDUCE ? p.nranks : 1u;
    uint32_t r = 0, kb = 0;
    const char *a, *b;
    const float *sa, *sb;
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
    // One more load a wave, then on to the next block (after the last one the
    // loads repeat).  The first waves load the scales, 64 rows' or a block of
    // columns' each (nothing in the loop goes through registers that the
    // compiler would wait for).  The other waves bring lines of the block
    // after the next into the second-level cache, so that the direct loads,
    // which are waited for within a step, do not wait for memory: a quarter of
    // the rows' and an eighth of the columns', the rest being the same tiles'
    // to the sides and above, which run at the same time.  (On constant values,
    // where power is no limit, 8 x 4096 x 7168 x 8192 takes 1416 against
    // 1571 us; on random ones the two are within 2 %.)
    const uint32_t helper = wave - S::kScaleWaves;  // (used where wave >= kScaleWaves)
    uint32_t off1;
    if (wave < S::kRows / 64u) {
        const uint32_t row = wave * 64u + lane;
        off1 = (m0 + row < p.rows ? m0 + row : p.rows - 1u) * 4u;
    } else if (wave < S::kScaleWaves) {
        const uint32_t col = n0 + (wave - S::kRows / 64u) * 128u;
        off1 = (col < p.n ? col / 128u : 0u) * p.kblocks * 4u;
    } else {
        const uint32_t i = helper * 64u + lane;
        uint32_t row = t / wide % 8u * (S::kCols / 8u) + (i - S::kRows / 4u) % (S::kCols / 8u), end = p.n - n0;
        if (i < S::kRows / 4u) {
            row = t % wide * (S::kRows / 4u) + i;
            end = p.rows - m0;
        }
        off1 = (row < end ? row : end - 1u) * p.k;
    }
    auto finish = [&](uint32_t stage) {
        const uint32_t to = lds0 + S::kScalesAt + stage * S::kScaleBytes + wave * 256u;
        const uint32_t far = kb + 2u < p.kblocks ? 256u : 0u;
        if (wave < S::kRows / 64u)
            to_lds4((const char *)sa + off1, to);
        else if (wave < S::kScaleWaves)
            to_lds4((const char *)sb + off1, to);
        else
            to_lds4((helper * 64u + lane < S::kRows / 4u ? a : b) + far + off1, lds0 + S::kUnusedAt + helper * 256u);
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

    // The steps run into one another: the wave waits for the others (all have
    // read this step's LDS, all have the next step's loads in it) before its
    // last two tiles, whose operands are in registers, so that their products
    // cover the wait and the next step's first reads.  A tile's products are
    // under way while the one before it is scaled, across steps too.  The
    // loads of the step after next go out between the products of the two
    // tiles before and after a step's end: all at once they would hold the
    // products back.
    f32x16 acc[NT][2] = {};
    f32x16 c[2] = {};
    i32x8 x[2][2], w[2];
    float s[2], s_last = 0.0f;
    auto rows = [&](uint32_t stage, uint32_t j) {
        const char *pm = lds + stage * S::kRowBytes + wm * 128u + j * 4096u;
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h)
            x[j][h] = pieces(pm, place ^ (h * 64u));
    };
    auto columns = [&](uint32_t stage, uint32_t i) {
        const char *pn = lds + 2u * S::kRowBytes + stage * S::kColBytes + wn * 128u + i * 4096u;
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h)
            w[h] = pieces(pn, place ^ (h * 64u));
    };
    auto arrived = [&](uint32_t stage) {
        if (wave < S::kScaleWaves)
            wait_loads<0>();
        else
            wait_loads<1>();
        __syncthreads();
        const float *scales = (const float *)(lds + S::kScalesAt + stage * S::kScaleBytes);
        const float sw = scales[S::kRows + wn / 128u * 64u + lane];
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j)
            s[j] = scales[wm + j * 32u + l32] * sw;
    };

    // One step: half `stage`.  `left`: bytes of the block that are in the row;
    // those past it are zero in the weights, and in the activations a repeat
    // of the row's own, so that a NaN there is one that the row has anyway.
    auto step = [&](uint32_t stage, uint32_t left) {
        float s_this[2] = {s[0], s[1]};
#pragma unroll
        for (uint32_t i = 0; i < NT; ++i) {
            if (left < 128u) {
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h)
#pragma unroll
                    for (uint32_t e = 0; e < 8; ++e)
                        w[h][e] = (h * 4u + half * 2u + e / 4u) * 16u < left ? w[h][e] : 0;
            }
            if (i == NT - 1u) {
                __builtin_amdgcn_sched_barrier(0);
                arrived(stage ^ 1u);
            }
#pragma unroll
            for (uint32_t j = 0; j < 2; ++j) {
                c[j] = block_sums32<kExact>(w, x[j]);
                __builtin_amdgcn_sched_barrier(0);
                if (i == NT - 1u)
                    rows(stage ^ 1u, j);
                if (j == 1)
                    columns(i == NT - 1u ? stage ^ 1u : stage, i == NT - 1u ? 0u : i + 1u);
                __builtin_amdgcn_sched_barrier(0);
                const uint32_t pi = j == 1 ? i : i == 0 ? NT - 1u : i - 1u, pj = j ^ 1u;
                const float ps = i + j == 0 ? s_last : s_this[pj];
#pragma unroll
                for (uint32_t e = 0; e < 16; ++e)
                    acc[pi][pj][e] = __builtin_fmaf(c[pj][e], ps, acc[pi][pj][e]);
                // (done here: put off, it keeps every tile's registers)
                asm volatile("" : "+v"(acc[pi][pj]));
                if (i == 0) {
#pragma unroll
                    for (uint32_t q = kParts / 2u + j * (kParts / 4u);
                         q < kParts / 2u + (j + 1u) * (kParts / 4u); ++q)
                        load(stage ^ 1u, q);
                    if (j == 1)
                        finish(stage ^ 1u);
                }
                if (i == NT - 1u) {
#pragma unroll
                    for (uint32_t q = j * (kParts / 4u); q < (j + 1u) * (kParts / 4u); ++q)
                        load(stage, q);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        s_last = s_this[1];
    };
    static_assert(kParts % 4 == 0, "the loads go out in four parts");

    at_rank();
#pragma unroll
    for (uint32_t q = 0; q < kParts; ++q)
        load(0, q);
    finish(0);
    arrived(0);
    rows(0, 0);
    columns(0, 0);
    rows(0, 1);
#pragma unroll
    for (uint32_t q = 0; q < kParts / 2u; ++q)
        load(1, q);
    uint32_t left = p.k;
    for (uint32_t n = 0; n < p.kblocks * nranks; ++n) {
        step(n & 1u, left);
        left = left > 128u ? left - 128u : p.k;
    }
#pragma unroll
    for (uint32_t e = 0; e < 16; ++e)
        acc[NT - 1][1][e] = __builtin_fmaf(c[1][e], s_last, acc[NT - 1][1][e]);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    // The sums go through LDS, 32 rows x 32 NT columns of a wave at a time, so
    // that a store covers whole lines: 16-byte pieces, piece c of row r at
    // place c ^ (r % 8).
    __syncthreads();
    constexpr uint32_t kRow = NT * 32u * T::kBytes;
    static_assert(S::kWaves * 32u * kRow <= S::kScalesAt, "the waves' parts fit");
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
