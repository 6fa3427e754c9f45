// block_matmul_mid.hip -- the block-scaled 8-bit product for a decode batch
// (three rows to a few hundred; one or two where workgroups share k).
//
// It is bound by reading the weights, so each weight byte goes through a
// compute unit once a tile of rows, and the reads are kept deep: a wave has a
// ring of D places in LDS, each one block of 128 of k of its rows and
// columns, and loads D - 1 blocks ahead straight from memory to LDS (whole
// 128-byte lines, no registers).  The waves of a workgroup share a tile of
// MT * 32 rows x NT * 32 columns and take every waves-th block of k (of all
// ranks' k, one rank after the other, when REDUCE).  They wait for nothing
// but their own loads until their sums are added, in wave order, at the end.
//
// Tiles are 32x32 (see block_matmul_tile.hip for the layout in LDS).
//
// Where a sum over the ranks has few tiles, p.split workgroups share a tile's
// k as well, and a second kernel adds their binary32 sums in order.  These lie
// in the output buffers until then, which are as many as there are ranks:
// workgroup s's sum of an element is where the element goes in buffer s, or
// for 16-bit outputs in two halves in buffers 2 s and 2 s + 1.  A lane of the
// second kernel reads all sums of its elements before it writes any, and no
// other lane touches them.  (8 x (91 x 66 x 6224), float32: 14 us in place of
// 57.)
#include <type_traits>

#include "block_device.hpp"
#include "block_internal.hpp"
#include "block_matmul.hpp"

namespace ar {

template <int MT, int NT>
struct MidPlace {
    static constexpr uint32_t kColumns = MT * 4096u;             // where the weights start
    static constexpr uint32_t kScales = kColumns + NT * 4096u;   // MT * 32 floats, the weights'
    // (a load of scales writes 256 bytes)
    static constexpr uint32_t kBytes = kScales + (MT == 1 ? 256u : MT * 128u + 256u);
    // loads of one place: eight rows or columns each, then the scales
    static constexpr int kLoads = (MT + NT) * 4 + MT / 2 + 1;
};

// Eight consecutive columns of a row, `left` of them to its end.
template <typename T>
__device__ inline void store8(char *to, const float (&c)[8], uint32_t left)
{
    constexpr uint32_t E = kPiece<T>;
#pragma unroll
    for (uint32_t i = 0; i < 8u / E; ++i) {
        float f[E];
#pragma unroll
        for (uint32_t e = 0; e < E; ++e)
            f[e] = c[i * E + e];
        if (left > i * E)
            store_row_piece<T>(to + i * 16u, narrow_piece<T>(f), left - i * E);
    }
}

// Workgroup `part`'s sums of them, to wait in the outputs.
template <typename T>
__device__ inline void store_part(const MatmulArgs &p, uint32_t part, uint64_t at, uint32_t left,
                                  const float (&c)[8])
{
    if constexpr (T::kBytes == 4) {
        store8<T>(p.out[part] + at * 4u, c, left);
    } else {
        u32x4 hi, lo;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            const uint32_t x = __builtin_bit_cast(uint32_t, c[2 * i]);
            const uint32_t y = __builtin_bit_cast(uint32_t, c[2 * i + 1]);
            hi[i] = x >> 16 | (y & 0xffff0000u);
            lo[i] = (x & 0xffffu) | y << 16;
        }
        store_row_piece<T>(p.out[2u * part] + at * 2u, hi, left);
        store_row_piece<T>(p.out[2u * part + 1u] + at * 2u, lo, left);
    }
}

// Adds the workgroups' sums of a piece of the outputs (ONE: of one element),
// in order, and stores the result to all ranks.
template <typename T, bool ONE>
__device__ inline void join(const MatmulArgs &p, uint64_t at)
{
    constexpr uint32_t E = ONE ? 1 : kPiece<T>;
    constexpr uint32_t kParts = T::kBytes == 4 ? 1 : 2;
    auto load = [&](uint32_t o) {
        const char *from = p.out[o] + at * T::kBytes;
        return ONE ? load_some<T>(from, 1) : load_piece<false>(from);
    };
    float sum[kPiece<T>] = {};
    // (splits are powers of two: four at a time, loaded before any is added)
    for (uint32_t s = 0; s < p.split; s += 4u) {
        u32x4 v[4][kParts];
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u)
            if (s + u < p.split)
#pragma unroll
                for (uint32_t h = 0; h < kParts; ++h)
                    v[u][h] = load((s + u) * kParts + h);
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u)
            if (s + u < p.split)
#pragma unroll
                for (uint32_t e = 0; e < E; ++e) {
                    uint32_t b;
                    if constexpr (kParts == 1)
                        b = v[u][0][e];
                    else
                        b = (v[u][0][e / 2u] >> 16u * (e % 2u)) << 16 |
                            (v[u][kParts - 1][e / 2u] >> 16u * (e % 2u) & 0xffffu);
                    sum[e] = sum[e] + __builtin_bit_cast(float, b);
                }
    }
    const u32x4 y = narrow_piece<T>(sum);
    for (uint32_t o = 0; o < p.nranks; ++o) {
        char *to = p.out[o] + at * T::kBytes;
        if constexpr (ONE)
            store_some<T>(to, y, 1);
        else
            store_piece<false>(to, y);
    }
}

// All pieces, and one by one the elements after the last whole one.
template <typename T>
__global__ __launch_bounds__(256) void matmul_join(MatmulArgs p)
{
    constexpr uint32_t E = kPiece<T>;
    const uint64_t count = (uint64_t)p.rows * p.n, pieces = count / E;
    for (uint64_t i = (uint64_t)blockIdx.x * 256u + threadIdx.x; i < pieces;
         i += (uint64_t)gridDim.x * 256u)
        join<T, false>(p, i * E);
    if (blockIdx.x == gridDim.x - 1u && threadIdx.x < count % E)
        join<T, true>(p, pieces * E + threadIdx.x);
}

template <typename T, int MT, int NT, int D, bool REDUCE>
__global__ __launch_bounds__(512) void matmul_mid(MatmulArgs p)
{
    constexpr bool kExact = T::kBytes == 4;
    typedef MidPlace<MT, NT> Place;
    constexpr uint32_t kRows = MT * 32u, kCols = NT * 32u;
    extern __shared__ __align__(128) char lds[];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t waves = blockDim.x >> 6;
    const uint32_t l32 = lane & 31u, half = lane >> 5;

    // Workgroup w runs on XCD w % 8: each XCD takes consecutive tiles, rows
    // first, so that the row tiles of the same weights meet in one cache.
    const uint32_t mtiles = (p.rows + kRows - 1) / kRows, ntiles = (p.n + kCols - 1) / kCols;
    const uint32_t tiles = mtiles * ntiles * (REDUCE ? p.split : p.nranks);
    const uint32_t each = (tiles + 7u) / 8u;
    const uint32_t tile = (blockIdx.x & 7u) * each + blockIdx.x / 8u;
    if (blockIdx.x / 8u >= each || tile >= tiles)
        return;
    const uint32_t m0 = tile % mtiles * kRows, n0 = tile / mtiles % ntiles * kCols;
    const uint32_t rank0 = REDUCE ? 0u : tile / (mtiles * ntiles);
    const uint32_t part = REDUCE ? tile / (mtiles * ntiles) : 0u;
    const uint32_t first = part * waves + wave, stride = REDUCE ? p.split * waves : waves;
    const uint32_t nranks = REDUCE ? p.nranks : 1u;

    // Rows and columns past the end repeat the last one, and what comes of
    // them is not stored.
    uint32_t offm[MT * 4], offn[NT * 4], offs[MT / 2 + 1];
    const uint32_t piece16 = ((lane & 7u) ^ (lane >> 4)) * 16u;  // even groups of eight; odd ^ 64
#pragma unroll
    for (uint32_t i = 0; i < MT * 4; ++i) {
        const uint32_t r = i * 8u + (lane >> 3);
        offm[i] = (r < p.rows - m0 ? r : p.rows - m0 - 1u) * p.k + (piece16 ^ (i & 1u) * 64u);
    }
#pragma unroll
    for (uint32_t i = 0; i < NT * 4; ++i) {
        const uint32_t r = i * 8u + (lane >> 3);
        offn[i] = (r < p.n - n0 ? r : p.n - n0 - 1u) * p.k + (piece16 ^ (i & 1u) * 64u);
    }
    // Scales: the rows' (64 a load), in the last load's upper half the
    // weights' (NT * 32 columns lie in one scale block).
#pragma unroll
    for (uint32_t i = 0; i < MT / 2 + 1; ++i) {
        const uint32_t r = i * 64u + lane;
        offs[i] = (r < p.rows - m0 ? r : p.rows - m0 - 1u) * 4u;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    const uint32_t ring = wave * (D * Place::kBytes);
    const uint32_t to0 = __builtin_amdgcn_readfirstlane(lds0) + ring;

    // What the next load reads: block kb of rank r.
    struct At {
        uint32_t r, kb;
    };
    auto normal = [&](At &at) {
        while (at.kb >= p.kblocks) {
            at.kb -= p.kblocks;
            ++at.r;
        }
    };
    At next = {0, first};
    normal(next);
    uint32_t known = ~0u;  // the rank that these belong to
    const char *a = nullptr, *b = nullptr;
    const float *sa = nullptr, *sb = nullptr;
    auto load = [&](uint32_t slot) {
        if (next.r != known) {
            known = next.r;
            a = p.a[rank0 + known] + (uint64_t)m0 * p.k;
            b = p.b[rank0 + known] + (uint64_t)n0 * p.k;
            sa = p.sa[rank0 + known] + m0;
            sb = p.sb[rank0 + known] + (uint64_t)(n0 / 128u) * p.kblocks;
        }
        const uint32_t to = to0 + slot * Place::kBytes;
        const uint64_t skip = (uint64_t)next.kb * 128u;
        // a piece past the end of its row repeats the row's last one
        const int32_t room = (int32_t)(p.k - 16u - next.kb * 128u);
        const int32_t over0 = (int32_t)piece16 - room, over1 = (int32_t)(piece16 ^ 64u) - room;
        const uint32_t back[2] = {over0 > 0 ? (uint32_t)over0 : 0u, over1 > 0 ? (uint32_t)over1 : 0u};
#pragma unroll
        for (uint32_t i = 0; i < NT * 4; ++i)
            to_lds(b + skip, offn[i] - back[i & 1u], to + Place::kColumns + i * 1024u);
#pragma unroll
        for (uint32_t i = 0; i < MT * 4; ++i)
            to_lds(a + skip, offm[i] - back[i & 1u], to + i * 1024u);
        const char *s = (const char *)(sa + (uint64_t)next.kb * p.rows);
        if constexpr (MT == 1) {
            to_lds4(half == 0 ? s + offs[0] : (const char *)(sb + next.kb), to + Place::kScales);
        } else {
#pragma unroll
            for (uint32_t i = 0; i < MT / 2; ++i)
                to_lds4(s + offs[i], to + Place::kScales + i * 256u);
            to_lds4((const char *)(sb + next.kb), to + Place::kScales + MT * 128u);
        }
        next.kb += stride;
        normal(next);
    };

    const uint32_t place = l32 * 128u + ((half * 2u) ^ (l32 >> 1 & 7u)) * 16u;
    f32x16 acc[NT][MT] = {};
    const uint32_t blocks = p.kblocks * nranks;
    const uint32_t steps = first < blocks ? (blocks - first + stride - 1u) / stride : 0u;
    uint32_t issued = 0, slot_in = 0, slot_out = 0;
    for (; issued < D - 1u && issued < steps; ++issued)
        load(slot_in++);
    At now = {0, first};
    normal(now);
    for (uint32_t step = 0; step < steps; ++step) {
        if (issued < steps) {
            load(slot_in);
            slot_in = slot_in + 1u == D ? 0u : slot_in + 1u;
            ++issued;
            wait_loads<(D - 1) * Place::kLoads>();
        } else {
            wait_loads<0>();
        }
        const char *at = lds + ring + slot_out * Place::kBytes;
        slot_out = slot_out + 1u == D ? 0u : slot_out + 1u;
        const uint32_t left = p.k - now.kb * 128u;
        now.kb += stride;
        normal(now);
        i32x8 x[MT][2];
        float s[MT];
        const float sbk = *(const float *)(at + Place::kScales + MT * 128u);
#pragma unroll
        for (uint32_t j = 0; j < MT; ++j) {
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h)
                x[j][h] = pieces(at + j * 4096u, place ^ (h * 64u));
            s[j] = *(const float *)(at + Place::kScales + (j * 32u + l32) * 4u) * sbk;
        }
#pragma unroll
        for (uint32_t i = 0; i < NT; ++i) {
            i32x8 w[2];
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h)
                w[h] = pieces(at + Place::kColumns + i * 4096u, place ^ (h * 64u));
            // past the row's end the weights are zero, and the activations a
            // repeat of the row's own: a NaN there is one that the row has
            if (left < 128u) {
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h)
#pragma unroll
                    for (uint32_t e = 0; e < 8; ++e)
                        w[h][e] = (h * 4u + half * 2u + e / 4u) * 16u < left ? w[h][e] : 0;
            }
#pragma unroll
            for (uint32_t j = 0; j < MT; ++j) {
                const f32x16 c = block_sums32<kExact>(w, x[j]);
#pragma unroll
                for (uint32_t e = 0; e < 16; ++e)
                    acc[i][j][e] = __builtin_fmaf(c[e], s[j], acc[i][j][e]);
            }
        }
        // every read of this place has returned before the place is loaded again
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }

    // The waves' sums: [wave][tile][16][64] floats in LDS, added in wave order.
    __syncthreads();
    float *sums = (float *)lds;
#pragma unroll
    for (uint32_t i = 0; i < NT; ++i)
#pragma unroll
        for (uint32_t j = 0; j < MT; ++j)
#pragma unroll
            for (uint32_t e = 0; e < 16; ++e)
                sums[(((wave * NT + i) * MT + j) * 16u + e) * 64u + lane] = acc[i][j][e];
    __syncthreads();
    // Eight consecutive columns of a row each: elements 4 q .. 4 q + 3 of a
    // tile, of both halves of the wave.
    for (uint32_t it = threadIdx.x; it < NT * MT * 128u; it += blockDim.x) {
        const uint32_t t = it / 128u, r32 = it / 4u % 32u, q = it & 3u;
        float c[8] = {};
        for (uint32_t w = 0; w < waves; ++w)
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e)
                c[e] += sums[((w * (NT * MT) + t) * 16u + q * 4u + e % 4u) * 64u + e / 4u * 32u + r32];
        const uint32_t row = m0 + t % MT * 32u + r32, col = n0 + t / MT * 32u + q * 8u;
        if (row < p.rows && col < p.n) {
            const uint64_t at = (uint64_t)row * p.n + col;
            if constexpr (REDUCE) {
                if (p.split > 1u)
                    store_part<T>(p, part, at, p.n - col, c);
                else
                    for (uint32_t o = 0; o < p.nranks; ++o)
                        store8<T>(p.out[o] + at * T::kBytes, c, p.n - col);
            } else {
                store8<T>(p.out[rank0] + at * T::kBytes, c, p.n - col);
            }
        }
    }
}

namespace {

template <typename T, int MT, int NT, int D>
hipError_t enqueue_mid(const MatmulArgs &args, uint32_t waves, bool reduce, hipStream_t stream)
{
    const size_t ring = (size_t)waves * D * MidPlace<MT, NT>::kBytes;
    const size_t part = (size_t)waves * NT * MT * 4096u;
    const size_t lds = ring > part ? ring : part;
    const uint32_t tiles = (args.rows + MT * 32u - 1) / (MT * 32u) *
                           ((args.n + NT * 32u - 1) / (NT * 32u)) *
                           (reduce ? args.split : args.nranks);
    const dim3 grid((tiles + 7u) / 8u * 8u);
    if (reduce)
        hipLaunchKernelGGL((matmul_mid<T, MT, NT, D, true>), grid, dim3(waves * 64), lds, stream, args);
    else
        hipLaunchKernelGGL((matmul_mid<T, MT, NT, D, false>), grid, dim3(waves * 64), lds, stream, args);
    return hipGetLastError();
}

template <typename T>
hipError_t pick_mid(const MatmulArgs &args, bool reduce, int mt, int nt, uint32_t waves,
                    hipStream_t stream)
{
    // two places a wave: three or four of them measured no faster
    if (mt == 1)
        return enqueue_mid<T, 1, 1, 2>(args, waves, reduce, stream);
    return nt == 1 ? enqueue_mid<T, 2, 1, 2>(args, waves, reduce, stream)
                   : enqueue_mid<T, 2, 2, 2>(args, waves, reduce, stream);
}

}  // namespace

hipError_t launch_matmul_mid(const MatmulArgs &given, int out_dtype, bool reduce, int mt, int nt,
                             uint32_t waves, uint32_t split, hipStream_t stream)
{
    MatmulArgs args = given;
    args.split = split;
    hipError_t e;
    switch (out_dtype) {
    case kBf16: e = pick_mid<Bf16>(args, reduce, mt, nt, waves, stream); break;
    case kFp16: e = pick_mid<Fp16>(args, reduce, mt, nt, waves, stream); break;
    default: e = pick_mid<Fp32>(args, reduce, mt, nt, waves, stream); break;
    }
    if (e != hipSuccess || split == 1u)
        return e;
    const uint64_t pieces = ((uint64_t)args.rows * args.n * (out_dtype == kFp32 ? 4u : 2u) + 15u) / 16u;
    const dim3 grid((uint32_t)(pieces < ((uint64_t)1 << 28) ? (pieces + 255u) / 256u : 1u << 20));
    switch (out_dtype) {
    case kBf16: hipLaunchKernelGGL((matmul_join<Bf16>), grid, dim3(256), 0, stream, args); break;
    case kFp16: hipLaunchKernelGGL((matmul_join<Fp16>), grid, dim3(256), 0, stream, args); break;
    default: hipLaunchKernelGGL((matmul_join<Fp32>), grid, dim3(256), 0, stream, args); break;
    }
    return hipGetLastError();
}

}  // namespace ar
