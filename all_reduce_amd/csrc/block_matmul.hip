// block_matmul.hip -- the product of 8-bit activations and weights with a
// scale per block of 128, per rank or summed over the ranks: the kernel for
// one or two rows, and the choice among the kernels.
//
//     c[t][j] = sum_b sa[b][t] * sb[j / 128][b] * sum_{i in b} a[t][i] * w[j][i]
//
// The matrix instruction 16x16x128 (f8f6f4) takes one block of 128 in one go.
// The weights are its first operand and the activations its second, so that a
// lane of the result holds four consecutive output columns of ONE activation
// row: its scale is one number a lane, and a block costs one multiplication
// for the scale and four fused multiply-adds for the running sums.
//
// Operand layout: lane l holds row l % 16 and, of each 128, bytes
// [16 g, 16 g + 16) and [64 + 16 g, +16) with g = l / 16.  Both operands are
// loaded alike, so the instruction's own order of k inside the 128 does not
// matter.  Result: lane l holds column (activation row) l % 16 and rows
// (output columns) 4 (l / 16) .. + 3.
#include <math.h>

#include "block_device.hpp"
#include "block_internal.hpp"
#include "block_matmul.hpp"

namespace ar {

constexpr uint32_t kRowsWaves = 8;

// The lane's 32 bytes of one whole block (`at`: the row's start plus the
// lane's 16 g plus 128 a block).
__device__ inline i32x8 load_block(const char *at)
{
    const u32x4 lo = *(const u32x4 *)at, hi = *(const u32x4 *)(at + 64);
    i32x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = (int)lo[i];
        r[4 + i] = (int)hi[i];
    }
    return r;
}

// The same of a row's last block, of which the lane has `left` bytes; rows end
// on a multiple of 16, so a 16-byte piece is inside or outside whole.
__device__ inline i32x8 load_last(const char *at, int32_t left)
{
    const u32x4 zero = {0, 0, 0, 0};
    const u32x4 lo = left > 0 ? *(const u32x4 *)at : zero;
    const u32x4 hi = left > 64 ? *(const u32x4 *)(at + 64) : zero;
    i32x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = (int)lo[i];
        r[4 + i] = (int)hi[i];
    }
    return r;
}

// A workgroup computes 16 output columns of up to 16 rows (it is called for
// two at most: more are faster in the other kernels); its waves take every
// waves-th block of k (of all ranks' k, one rank after the other, when
// REDUCE), kAhead of them at a time, and their sums are added through LDS in
// wave order.  Weights go straight from memory to the registers of the one
// wave that multiplies them, each byte once: it is bound by that.  On MI355X
// 8 x (1 x 7168 x 8192) takes 76 to 80 us, 5.9 to 6.2 TB/s (measured beside 76: two
// blocks at a time 78 us, one 83 us; 32 columns a workgroup 84 us; through
// LDS, as in block_matmul_mid.hip, 87 us).
template <typename T, bool REDUCE>
__global__ __launch_bounds__(kRowsWaves * 64) void matmul_rows(MatmulArgs p)
{
    constexpr bool kExact = T::kBytes == 4;
    constexpr uint32_t kAhead = 4;
    __shared__ float part[kRowsWaves * 4 * 64];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t g = lane >> 4, l16 = lane & 15u;
    const uint32_t nranks = REDUCE ? p.nranks : 1u;
    const uint32_t ntiles = (p.n + 15u) / 16u;
    const uint32_t full = p.k / 128u;
    // rows and columns past the end repeat the last one; what comes of them is
    // not stored
    const uint32_t m = l16 < p.rows ? l16 : p.rows - 1u;
    const uint32_t n0 = blockIdx.x % ntiles * 16u, rank0 = blockIdx.x / ntiles;
    const uint32_t col = n0 + l16 < p.n ? n0 + l16 : p.n - 1u;
    const uint64_t m_at = (uint64_t)m * p.k + 16u * g, n_at = (uint64_t)col * p.k + 16u * g;
    f32x4 acc = {};
    uint32_t turn = wave;  // blocks until this wave's next one
    for (uint32_t r = 0; r < nranks; ++r) {
        const char *a = p.a[rank0 + r], *b = p.b[rank0 + r];
        const float *sa = p.sa[rank0 + r] + m;
        // 16 columns lie in one scale block
        const float *sb = p.sb[rank0 + r] + (uint64_t)(n0 / 128u) * p.kblocks;
        i32x8 w[kAhead], x[kAhead];
        float s[kAhead];
        auto load = [&](uint32_t u, uint32_t kb) {
            w[u] = load_block(b + n_at + (uint64_t)kb * 128u);
            x[u] = load_block(a + m_at + (uint64_t)kb * 128u);
            s[u] = sb[kb] * sa[(uint64_t)kb * p.rows];
        };
        auto multiply = [&](uint32_t u) {
            const f32x4 c = block_sums<kExact>(w[u], x[u]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[e] = __builtin_fmaf(c[e], s[u], acc[e]);
        };
        uint32_t kb = turn;
        for (; kb + (kAhead - 1u) * kRowsWaves < full; kb += kAhead * kRowsWaves) {
#pragma unroll
            for (uint32_t u = 0; u < kAhead; ++u)
                load(u, kb + u * kRowsWaves);
#pragma unroll
            for (uint32_t u = 0; u < kAhead; ++u)
                multiply(u);
        }
        for (; kb < full; kb += kRowsWaves) {
            load(0, kb);
            multiply(0);
        }
        if (kb < p.kblocks) {  // the row's last block, shorter than 128
            const int32_t left = (int32_t)(p.k % 128u) - (int32_t)(16u * g);
            w[0] = load_last(b + n_at + (uint64_t)kb * 128u, left);
            x[0] = load_last(a + m_at + (uint64_t)kb * 128u, left);
            s[0] = sb[kb] * sa[(uint64_t)kb * p.rows];
            multiply(0);
            kb += kRowsWaves;
        }
        turn = kb - p.kblocks;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        part[(wave * 4 + e) * 64 + lane] = acc[e];
    __syncthreads();
    if (wave != 0)
        return;
    f32x4 c = {};
    for (uint32_t w = 0; w < kRowsWaves; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c[e] += part[(w * 4 + e) * 64 + lane];
    const uint32_t col4 = n0 + 4u * g;
    if (l16 < p.rows && col4 < p.n) {
        if constexpr (REDUCE) {
            for (uint32_t r = 0; r < p.nranks; ++r)
                store4<T>(p.out[r], l16, p.n, col4, c);
        } else {
            store4<T>(p.out[rank0], l16, p.n, col4, c);
        }
    }
}

namespace {

template <typename T>
hipError_t enqueue_rows(const MatmulArgs &args, bool reduce, hipStream_t stream)
{
    const dim3 grid((args.n + 15u) / 16u * (reduce ? 1u : args.nranks));
    if (reduce)
        hipLaunchKernelGGL((matmul_rows<T, true>), grid, dim3(kRowsWaves * 64), 0, stream, args);
    else
        hipLaunchKernelGGL((matmul_rows<T, false>), grid, dim3(kRowsWaves * 64), 0, stream, args);
    return hipGetLastError();
}

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

}  // namespace

// The kernels for any number of rows: tiles of rows x columns whose `waves`
// share k, `resident` workgroups to a compute unit, and the time they take (us)
//
//     base + each * Q + MB written / 4
//          + max(alone * ceil(Q / resident) * S, full * W * S, MB read / rate)
//
// for Q = ceil(W) workgroups a compute unit (W of them on average) of S steps
// (blocks of k to a wave): a step takes `alone` where nothing else is on the
// compute unit and `full` a workgroup where it is filled.  Inputs of up to 64
// MB may still be in a cache from the call before; larger ones (the weights of
// a decode step, read once a step) come from memory, where a step's loads take
// longer and what counts is how many are under way: these have numbers of
// their own, a rate of 6.4 MB/us, and less where some compute units have no
// workgroup.  (With the numbers of cached inputs, 8 x 16 x 8192 x 3584 summed
// went to two waves a tile and 58 us in place of four and 41, 8 x 4 x 7168 x
// 8192 to 91 in place of 79.)  In a summed form workgroups may share a tile's k
// too (block_matmul_mid.hip), at the price of a second kernel.
//
// The numbers were fitted on MI355X to 900 shapes measured with the same inputs
// call after call (3 to 8192 rows, 64 to 8192 columns, k 128 to 8192, 1 to 8
// ranks, each rank's product and the sum; 8 to 19 % off in the mean) and, for
// more than 64 MB, to 3700 with 600 MB of inputs in turn (10 % off).  The kernel
// chosen by them takes 1.05 times the fastest one's time in the mean over 300
// other shapes of the first kind, 1.02 times over 1200 of the second up to 400
// rows and 1.003 times above.  What they tell apart, for example (us, bfloat16
// out, the same inputs):
//
//                                    64x32   64x64   128x128  256x256
//     1 rank,    64 x 8192 x 8192     14      17       52       85
//     1 rank,   128 x 8192 x 8192     23      18       53       86
//     1 rank,   512 x 8192 x 8192     77      61       55       87
//     1 rank,  2048 x 8192 x 8192              309     163      111
//     8 ranks,  100 x 8192 x 8192             157      108      125
//     8 ranks,  256 x 8192 x 8192             273      191      155
//     8 ranks, 1024 x 8192 x 8192            1023      632      448
struct Choice {
    uint32_t rows, cols, waves, resident;
    float base, alone, full, each;
};

constexpr int kChoices = 9;
constexpr Choice kChoice16[kChoices] = {
    {32, 32, 8, 1, 2.40f, 0.71f, 1.19f, 1.05f}, {32, 32, 4, 2, 3.15f, 0.43f, 0.54f, 0.27f},
    {32, 32, 2, 4, 3.33f, 0.37f, 0.31f, 0.0f},  {64, 32, 4, 1, 2.53f, 0.60f, 0.98f, 1.33f},
    {64, 32, 2, 3, 3.79f, 0.49f, 0.53f, 0.0f},  {64, 64, 4, 1, 2.95f, 0.84f, 1.30f, 1.83f},
    {64, 64, 2, 2, 4.40f, 0.68f, 0.71f, 0.29f}, {128, 128, 1, 2, 3.92f, 0.81f, 0.70f, 0.0f},
    {256, 256, 1, 1, 4.65f, 1.40f, 1.40f, 0.78f}};
// With exact products; 256 x 256 tiles have no registers left for those.
constexpr Choice kChoice32[kChoices - 1] = {
    {32, 32, 8, 1, 2.45f, 0.85f, 1.24f, 1.10f}, {32, 32, 4, 2, 3.29f, 0.52f, 0.57f, 0.23f},
    {32, 32, 2, 4, 3.39f, 0.49f, 0.33f, 0.0f},  {64, 32, 4, 1, 2.61f, 0.72f, 1.03f, 1.37f},
    {64, 32, 2, 3, 3.71f, 0.66f, 0.58f, 0.0f},  {64, 64, 4, 1, 2.35f, 1.20f, 1.37f, 2.31f},
    {64, 64, 2, 2, 4.07f, 1.06f, 0.81f, 0.48f}, {128, 128, 1, 2, 4.22f, 1.21f, 0.81f, 0.0f}};

// For inputs from memory.
constexpr Choice kMemory16[kChoices] = {
    {32, 32, 8, 1, 5.05f, 0.94f, 1.00f, 2.10f}, {32, 32, 4, 2, 7.18f, 0.48f, 0.51f, 0.16f},
    {32, 32, 2, 4, 7.43f, 0.45f, 0.28f, 0.20f}, {64, 32, 4, 1, 3.15f, 0.68f, 0.74f, 2.35f},
    {64, 32, 2, 3, 6.69f, 0.53f, 0.43f, 0.05f}, {64, 64, 4, 1, 5.14f, 0.93f, 1.01f, 3.89f},
    {64, 64, 2, 2, 10.43f, 0.65f, 0.69f, 0.0f}, {128, 128, 1, 2, 8.23f, 1.11f, 0.78f, 0.88f},
    {256, 256, 1, 1, 3.65f, 1.81f, 1.81f, 5.06f}};
constexpr Choice kMemory32[kChoices - 1] = {
    {32, 32, 8, 1, 5.76f, 0.97f, 1.04f, 2.30f},  {32, 32, 4, 2, 7.58f, 0.59f, 0.52f, 0.39f},
    {32, 32, 2, 4, 10.96f, 0.49f, 0.28f, 0.07f}, {64, 32, 4, 1, 4.10f, 0.72f, 0.77f, 2.75f},
    {64, 32, 2, 3, 10.88f, 0.59f, 0.46f, 0.0f},  {64, 64, 4, 1, 6.36f, 1.09f, 1.19f, 4.86f},
    {64, 64, 2, 2, 12.37f, 0.96f, 0.84f, 0.23f}, {128, 128, 1, 2, 7.18f, 1.53f, 1.05f, 2.16f}};

namespace {

// A launch has fewer than 2^32 threads.
constexpr double kMostThreads = 4.0e9;

double tiles_of(const Choice &c, uint64_t rows, uint64_t n)
{
    return (double)(ceil_div(rows, c.rows) * ceil_div(n, c.cols));
}

bool fits(const Choice &c, double tiles)
{
    return tiles * 64.0 * (c.rows == 256u ? 8.0 : c.rows == 128u ? 4.0 : c.waves) <= kMostThreads;
}

}  // namespace

bool matmul_fits(uint64_t rows, uint64_t n, int out_dtype)
{
    for (int i = 0; i < (out_dtype == kFp32 ? kChoices - 1 : kChoices); ++i)
        if (fits(kChoice16[i], tiles_of(kChoice16[i], rows, n)))
            return true;
    return false;
}

bool choose_matmul(const MatmulArgs &args, int out_dtype, bool reduce, int cu_count,
                   MatmulChoice *choice)
{
    const bool exact = out_dtype == kFp32;
    const Choice *best = nullptr;
    uint32_t best_split = 1;
    double best_us = 0.0;
    const double ranks = args.nranks, steps = (double)args.kblocks * (reduce ? ranks : 1.0);
    const double read = ((double)args.rows + args.n) * args.k * ranks * 1e-6;
    const bool memory = read > 64.0;
    const Choice *choices = memory ? (exact ? kMemory32 : kMemory16) : (exact ? kChoice32 : kChoice16);
    // (what is written is the same for all, but that sums are read again)
    const double join = 3.0 + (double)args.rows * args.n * ranks * (exact ? 4.0 : 2.0) * 0.1e-6;
    const uint32_t splits = reduce ? matmul_most_split(out_dtype, args.nranks) : 1u;
    for (int i = 0; i < (exact ? kChoices - 1 : kChoices); ++i) {
        const Choice &c = choices[i];
        const double tiles = tiles_of(c, args.rows, args.n) * (reduce ? 1.0 : ranks);
        for (uint32_t split = 1; split <= (c.rows < 128u ? splits : 1u); split *= 2u) {
            if (!fits(c, tiles * split))
                continue;
            const double w = tiles * split / cu_count, q = ceil(w);
            const double s = ceil(steps / (c.waves * split));
            const double rate = memory ? 6.4 * fmin(1.0, 2.0 * w)
                                       : 5.0 * fmin(1.0, 0.5 + (double)args.rows / c.rows);
            const double us = c.base + c.each * q + (split > 1u ? join : 0.0) +
                              fmax(fmax(c.alone * ceil(q / c.resident) * s, c.full * w * s), read / rate);
            if (best == nullptr || us < best_us) {
                best = &c;
                best_split = split;
                best_us = us;
            }
        }
    }
    // One or two rows take the kernel made for them, but where the model would
    // have workgroups share k: it has few columns there, and too few workgroups
    // (8 x (1 x 512 x 8192) summed: 14 in place of 41 us).  The model does not
    // know that kernel's own time.
    if (args.rows <= 2 && best_split == 1u && 32.0 * args.n * args.nranks < kMostThreads) {
        *choice = {16u, 16u, kRowsWaves, 1u};
        return true;
    }
    if (best == nullptr)
        return false;
    *choice = {best->rows, best->cols, best->waves, best_split};
    return true;
}

hipError_t launch_matmul(const MatmulArgs &args, int out_dtype, bool reduce, int cu_count,
                         hipStream_t stream)
{
    MatmulChoice c;
    if (!choose_matmul(args, out_dtype, reduce, cu_count, &c)) {
        // Too many tiles for one launch: half of the ranks, and the others.
        // (One rank's fit: the entry point has asked matmul_fits.)
        if (reduce || args.nranks == 1)
            return hipErrorInvalidConfiguration;
        const uint32_t half = args.nranks / 2u;
        MatmulArgs part = args;
        part.nranks = half;
        const hipError_t e = launch_matmul(part, out_dtype, reduce, cu_count, stream);
        if (e != hipSuccess)
            return e;
        part.nranks = args.nranks - half;
        for (uint32_t r = 0; r < part.nranks; ++r) {
            part.a[r] = args.a[half + r];
            part.sa[r] = args.sa[half + r];
            part.b[r] = args.b[half + r];
            part.sb[r] = args.sb[half + r];
            part.out[r] = args.out[half + r];
        }
        return launch_matmul(part, out_dtype, reduce, cu_count, stream);
    }
    if (c.rows == 16u) {
        switch (out_dtype) {
        case kBf16: return enqueue_rows<Bf16>(args, reduce, stream);
        case kFp16: return enqueue_rows<Fp16>(args, reduce, stream);
        default: return enqueue_rows<Fp32>(args, reduce, stream);
        }
    }
    if (c.rows >= 128u)
        return launch_matmul_tile(args, out_dtype, reduce, c.rows == 256u, stream);
    return launch_matmul_mid(args, out_dtype, reduce, (int)c.rows / 32, (int)c.cols / 32, c.waves,
                             c.split, stream);
}

}  // namespace ar
