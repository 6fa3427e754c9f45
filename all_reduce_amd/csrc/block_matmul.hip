// block_matmul.hip -- the product of 8-bit activations and weights with a
// scale per block of 128, per rank or summed over the ranks.
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

// The lane's 32 bytes of one block of one row (`row_at`: the row's start plus
// the lane's 16 g; `left`: bytes of the row from there on; rows end on a
// multiple of 16, so a 16-byte piece is inside or outside whole).
__device__ inline i32x8 load_block(const char *row_at, uint32_t kb, int32_t left)
{
    const int32_t at = (int32_t)(kb * 128u);
    const u32x4 zero = {0, 0, 0, 0};
    const u32x4 lo = at < left ? *(const u32x4 *)(row_at + at) : zero;
    const u32x4 hi = at + 64 < left ? *(const u32x4 *)(row_at + at + 64) : zero;
    i32x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = (int)lo[i];
        r[4 + i] = (int)hi[i];
    }
    return r;
}

// Four consecutive columns of a row, those below `n`.
template <typename T>
__device__ inline void store4(char *out, uint64_t row, uint32_t n, uint32_t col, f32x4 c)
{
    const uint64_t at = row * n + col;
    float f[4] = {c[0], c[1], c[2], c[3]};
    uint32_t w[2 * T::kBytes / 2];
#pragma unroll
    for (int i = 0; i < 4 / T::kPerWord; ++i)
        w[i] = T::narrow(f + i * T::kPerWord);
    if (col + 4u <= n) {
        __builtin_memcpy(out + at * T::kBytes, w, 4 * T::kBytes);
    } else {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            if (col + i < n)
                __builtin_memcpy(out + (at + i) * T::kBytes, (const char *)w + i * T::kBytes, T::kBytes);
    }
}

// A workgroup computes 16 output columns of MT * 16 rows; its waves take
// every waves-th block of k (of all ranks' k when REDUCE) and their sums are
// added through LDS in wave order.
template <typename T, int MT, bool REDUCE>
__global__ __launch_bounds__(1024) void matmul_rows(MatmulArgs p)
{
    extern __shared__ float part[];  // [waves][MT][4][64]
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t waves = blockDim.x >> 6;
    const uint32_t g = lane >> 4, l16 = lane & 15u;
    const uint32_t nranks = REDUCE ? p.nranks : 1u;
    const uint64_t ntiles = (p.n + 15u) / 16u, mtiles = (p.rows + 16u * MT - 1u) / (16u * MT);
    const uint64_t tiles = ntiles * mtiles * (REDUCE ? 1u : p.nranks);
    for (uint64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const uint32_t n0 = (uint32_t)(tile % ntiles) * 16u;
    const uint32_t m0 = (uint32_t)(tile / ntiles % mtiles) * (16u * MT);
    const uint32_t rank0 = (uint32_t)(tile / ntiles / mtiles);
    const uint32_t col = n0 + l16 < p.n ? n0 + l16 : p.n - 1u;
    const int32_t left = (int32_t)(p.k - 16u * g);
    uint32_t m[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const uint32_t x = m0 + t * 16u + l16;
        m[t] = x < p.rows ? x : p.rows - 1u;
    }
    f32x4 acc[MT] = {};
    for (uint32_t r = 0; r < nranks; ++r) {
        const char *b = p.b[rank0 + r] + (uint64_t)col * p.k + 16u * g;
        const char *a = p.a[rank0 + r] + 16u * g;
        const float *sa = p.sa[rank0 + r];
        const float *sb = p.sb[rank0 + r] + (uint64_t)(n0 / 128u) * p.kblocks;
        for (uint32_t kb = wave; kb < p.kblocks; kb += waves) {
            const i32x8 w = load_block(b, kb, left);
            const float s = sb[kb];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const i32x8 x = load_block(a + (uint64_t)m[t] * p.k, kb, left);
                const float st = s * sa[(uint64_t)kb * p.rows + m[t]];
                const f32x4 c = block_sums<T::kBytes == 4>(w, x);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[t][i] = __builtin_fmaf(c[i], st, acc[t][i]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            part[((wave * MT + t) * 4 + i) * 64 + lane] = acc[t][i];
    __syncthreads();
    for (uint32_t t = wave; t < MT; t += waves) {
        f32x4 c = {};
        for (uint32_t w = 0; w < waves; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c[i] += part[((w * MT + t) * 4 + i) * 64 + lane];
        const uint32_t row = m0 + t * 16u + l16, col4 = n0 + 4u * g;
        if (row < p.rows && col4 < p.n) {
            if constexpr (REDUCE) {
                for (uint32_t r = 0; r < p.nranks; ++r)
                    store4<T>(p.out[r], row, p.n, col4, c);
            } else {
                store4<T>(p.out[rank0], row, p.n, col4, c);
            }
        }
    }
    __syncthreads();
    }
}

namespace {

template <typename T, int MT>
hipError_t enqueue(const MatmulArgs &args, bool reduce, hipStream_t stream)
{
    const uint32_t waves = 4;
    const size_t lds = waves * MT * 4 * 64 * sizeof(float);
    uint64_t tiles = ((uint64_t)args.n + 15u) / 16u * ((args.rows + 16u * MT - 1u) / (16u * MT)) *
                     (reduce ? 1u : args.nranks);
    const dim3 grid((uint32_t)(tiles < (1u << 20) ? tiles : (1u << 20)));
    if (reduce)
        hipLaunchKernelGGL((matmul_rows<T, MT, true>), grid, dim3(waves * 64), lds, stream, args);
    else
        hipLaunchKernelGGL((matmul_rows<T, MT, false>), grid, dim3(waves * 64), lds, stream, args);
    return hipGetLastError();
}

template <typename T>
hipError_t pick(const MatmulArgs &args, bool reduce, hipStream_t stream)
{
    if (args.rows > 128 && args.k <= kTileMaxK)
        return launch_matmul_tile(args, T::kId, reduce, stream);
    return args.rows <= 16 ? enqueue<T, 1>(args, reduce, stream)
                           : enqueue<T, 4>(args, reduce, stream);
}

}  // namespace

hipError_t launch_matmul(const MatmulArgs &args, int out_dtype, bool reduce, int cu_count,
                         hipStream_t stream)
{
    (void)cu_count;
    switch (out_dtype) {
    case kBf16: return pick<Bf16>(args, reduce, stream);
    case kFp16: return pick<Fp16>(args, reduce, stream);
    default: return pick<Fp32>(args, reduce, stream);
    }
}

}  // namespace ar
