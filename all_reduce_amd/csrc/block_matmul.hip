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
// 8 x (1 x 7168 x 8192) takes 76 us, 6.2 TB/s (two blocks at a time 78 us,
// one 83 us; 32 columns a workgroup 84 us; through LDS, as in
// block_matmul_mid.hip, 87 us).
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

// The kernel that is expected to be fastest.  Each one's time is rounds of
// workgroups over the chip times blocks of k (a wave's share of them in the
// decode-batch kernel) times what one block takes, and not less than the
// weights take from memory; the constants were measured on MI355X over 1 to
// 2048 rows, 512 to 8192 columns, k 1024 and 8192, 1 and 8 ranks, each rank's
// own product and the sum.  Some of what they tell apart (us, bfloat16 out):
//
//                                    64x32   64x64   128x128  256x256
//     1 rank,    64 x 8192 x 8192     14      17       52       85
//     1 rank,   128 x 8192 x 8192     23      18       53       86
//     1 rank,   512 x 8192 x 8192     77      61       55       87
//     1 rank,  2048 x 8192 x 8192              309     163      111
//     8 ranks,  100 x 8192 x 8192             157      108      125
//     8 ranks,  256 x 8192 x 8192             273      191      155
//     8 ranks, 1024 x 8192 x 8192            1023      632      448
hipError_t launch_matmul(const MatmulArgs &args, int out_dtype, bool reduce, int cu_count,
                         hipStream_t stream)
{
    if (args.rows <= 2) {
        switch (out_dtype) {
        case kBf16: return enqueue_rows<Bf16>(args, reduce, stream);
        case kFp16: return enqueue_rows<Fp16>(args, reduce, stream);
        default: return enqueue_rows<Fp32>(args, reduce, stream);
        }
    }
    const uint64_t cus = (uint64_t)cu_count;
    const uint64_t steps = (uint64_t)args.kblocks * (reduce ? args.nranks : 1u);
    auto tiles = [&](uint32_t m, uint32_t n) {
        return ceil_div(args.rows, m) * ceil_div(args.n, n) * (reduce ? 1u : args.nranks);
    };
    if (args.rows <= 32) {
        // 32 x 32 tiles; eight waves where one workgroup a compute unit is all
        // there is, else more workgroups of fewer waves
        const uint32_t waves = tiles(32, 32) <= cus ? 8 : steps < 32 ? 2 : 4;
        return launch_matmul_mid(args, out_dtype, reduce, 1, 1, waves, stream);
    }
    const double memory = (double)args.n * args.k * args.nranks / 5.2e6;
    auto at_least = [&](double us) { return us > memory ? us : memory; };
    // a binary32 output's products are exact, and take three times as long
    const bool exact = out_dtype == kFp32;
    const uint64_t t21 = tiles(64, 32), t22 = tiles(64, 64), t1 = tiles(128, 128), t2 = tiles(256, 256);
    const double share = (double)ceil_div(steps, 4);
    const double us21 = 2.5 + at_least((double)ceil_div(t21, cus) * share * 0.70);
    const double us22 = 2.5 + at_least((double)ceil_div(t22, cus) * share * 0.95);
    const double us1 = 3.0 + at_least((t1 <= cus ? 0.80 : 1.20 * (double)ceil_div(t1, 2 * cus)) *
                                      (double)steps * (exact ? 1.5 : 1.0));
    // (256 x 256 tiles have no registers left for the exact products)
    const double us2 = exact ? us1 + 1.0
                             : 3.0 + at_least((double)ceil_div(t2, cus) * (double)steps *
                                              (t2 <= cus ? 1.33 : 1.65));
    if (us2 < us1 && us2 < us22 && us2 < us21)
        return launch_matmul_tile(args, out_dtype, reduce, true, stream);
    if (us1 < us22 && us1 < us21)
        return launch_matmul_tile(args, out_dtype, reduce, false, stream);
    if (us21 < us22)
        return launch_matmul_mid(args, out_dtype, reduce, 2, 1, t21 > cus && steps < 32 ? 2 : 4, stream);
    return launch_matmul_mid(args, out_dtype, reduce, 2, 2, t22 > cus && steps < 32 ? 2 : 4, stream);
}

}  // namespace ar
