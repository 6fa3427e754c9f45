// block_gate.hip -- SiLU gate (or nothing) and quantisation to 8 bits with a
// scale per row and 128 columns, for R rank buffers in one launch.
//
// Sixteen (binary32: 32) neighbouring lanes hold the 128 columns of a scale,
// a piece each: the block's largest magnitude is a few lane rotations away,
// and each value is read once and written once.  A workgroup takes 16 rows of
// one block, or of four, so that their scales, next to each other in memory,
// are written together; all loads are issued before the first is used.  Bound
// by memory: 4 bytes read and 1 written a value for 16-bit gated inputs.  On
// MI355X 8 x 8192 x 3584 bfloat16 takes 195 us (6.0 TB/s; block by block along
// a row, one load in flight and an IEEE division a value, it took 251).
#include <type_traits>

#include "block_device.hpp"
#include "block_internal.hpp"

namespace ar {

// g / (1 + exp(-g)), by exp(-|g|): nothing overflows.  For g from kFar on; the
// hardware's exponential has no results below 2^-126.
constexpr float kFar = -80.0f;

__device__ inline float silu(float g)
{
    const float e = __builtin_amdgcn_exp2f(-__builtin_fabsf(g) * 1.44269504088896341f);
    return g * ((g < 0.0f ? e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + e));
}

// g / (1 + exp(-g)) * u for g below kFar, where 1 + exp(g) is 1: g exp(g) u,
// which a large u keeps an ordinary number to g = -200.  With exp(g) = f 2^n the
// powers of two are multiplied in around u, so that nothing leaves the range on
// the way (below -400 the result is 0 for every finite u).
__device__ inline float silu_far(float g, float u)
{
    const float near = g < -400.0f ? -400.0f : g;
    const float x = near * 1.44269504088896341f, n = __builtin_rintf(x);
    const float gf = near * __builtin_amdgcn_exp2f(x - n);
    const float y = __builtin_ldexpf(__builtin_ldexpf(gf, -64) * u, (int)n + 64);
    // an infinite g divides by an infinity
    return g < -__FLT_MAX__ ? __builtin_nanf("") : y;
}

// kTurns: blocks of a group of lanes.  One rank per grid row (blockIdx.y).  A
// workgroup has 256 / kLanes groups of lanes: `tall` consecutive rows of them
// side by side in columns.
template <typename T, bool GATED, bool NT, uint32_t kTurns>
__global__ __launch_bounds__(256) void gate_quant(GateArgs p)
{
    constexpr uint32_t E = kPiece<T>, kLanes = AR_SCALE_BLOCK / E, kGroups = 256 / kLanes;
    const uint32_t rank = blockIdx.y;
    const char *in = p.in[rank];
    char *out = p.out[rank];
    float *scales = p.scales[rank];
    const uint64_t blocks = (p.cols + AR_SCALE_BLOCK - 1) / AR_SCALE_BLOCK;
    const uint64_t wide = GATED ? 2 * p.cols : p.cols;
    const uint32_t side = kGroups / p.tall;             // blocks next to each other
    const uint64_t across = (blocks + side * kTurns - 1) / (side * kTurns);  // workgroups
    const uint32_t group = threadIdx.x / kLanes;
    const uint64_t works = (p.rows + p.tall - 1) / p.tall * across;
    for (uint64_t w = blockIdx.x; w < works; w += gridDim.x) {
        const uint64_t row = w / across * p.tall + group % p.tall;
        const uint64_t block0 = w % across * (side * kTurns) + group / p.tall;
        const uint32_t lane_col = threadIdx.x % kLanes * E;
        auto load = [&](uint32_t t, u32x4 &x, u32x4 &u) {
            const uint64_t col = (block0 + t * side) * AR_SCALE_BLOCK + lane_col;
            x = u = u32x4{0, 0, 0, 0};
            if (row < p.rows && col < p.cols) {
                const char *at = in + (row * wide + col) * T::kBytes;
                if (col + E <= p.cols) {
                    x = load_piece<NT>(at);
                    if constexpr (GATED)
                        u = load_piece<NT>(at + p.cols * T::kBytes);
                } else {
                    const uint32_t n = (uint32_t)(p.cols - col);
                    x = load_some<T>(at, n);
                    if constexpr (GATED)
                        u = load_some<T>(at + p.cols * T::kBytes, n);
                }
            }
        };
        uint32_t most = 0;
        // FAR: with gates below kFar.
        auto finish = [&](auto far, uint32_t t, u32x4 x, u32x4 u) {
            const uint64_t block = block0 + t * side;
            const uint64_t col = block * AR_SCALE_BLOCK + lane_col;
            float y[E];
            widen_piece<T>(x, y);
            if constexpr (GATED) {
                float f[E];
                widen_piece<T>(u, f);
                // (columns past the row are 0 / 2 * 0)
#pragma unroll
                for (uint32_t e = 0; e < E; ++e) {
                    const float g = y[e];
                    y[e] = silu(g) * f[e];
                    if constexpr (decltype(far)::value)
                        y[e] = g < kFar ? silu_far(g, f[e]) : y[e];
                    const uint32_t bits = __builtin_bit_cast(uint32_t, g);
                    most = most > bits ? most : bits;
                }
            }
            const float s = scale_of(max_block<T>(max_bits(y)));
            const Eights<E> q = to_eights(y, s);
            if (row < p.rows && col < p.cols) {
                if (col + E <= p.cols)
                    store_eights<NT>(out + row * p.cols + col, q);
                else
                    store_eights_some(out + row * p.cols + col, q, (uint32_t)(p.cols - col));
                if (threadIdx.x % kLanes == 0)
                    scales[block * p.rows + row] = s;
            }
        };
        u32x4 x[kTurns], u[kTurns];
#pragma unroll
        for (uint32_t t = 0; t < kTurns; ++t)
            load(t, x[t], u[t]);
#pragma unroll
        for (uint32_t t = 0; t < kTurns; ++t)
            finish(std::false_type{}, t, x[t], u[t]);
        // A gate below kFar (its bits are above kFar's, as no positive one's
        // are): the wave takes its blocks again, from memory.  They are rare,
        // and here they cost the others half an instruction a value; chosen in
        // place, value by value, 8 x 8192 x 3584 took 201 in place of 194 us.
        if constexpr (GATED) {
            if (__ballot(most > __builtin_bit_cast(uint32_t, kFar)) != 0) {
#pragma unroll 1
                for (uint32_t t = 0; t < kTurns; ++t) {
                    u32x4 xt, ut;
                    load(t, xt, ut);
                    finish(std::true_type{}, t, xt, ut);
                }
            }
        }
    }
}

namespace {

template <typename T, bool GATED, bool NT, uint32_t TURNS>
hipError_t enqueue(const GateArgs &args, int nranks, int cu_count, hipStream_t stream)
{
    constexpr uint32_t kGroups = 256 / (AR_SCALE_BLOCK / kPiece<T>);
    const uint64_t blocks = (args.cols + AR_SCALE_BLOCK - 1) / AR_SCALE_BLOCK;
    const uint64_t each = kGroups / args.tall * TURNS;
    uint64_t grid = (args.rows + args.tall - 1) / args.tall * ((blocks + each - 1) / each);
    const uint64_t most = (uint64_t)cu_count * 256;
    grid = grid < most ? grid : most;
    hipLaunchKernelGGL((gate_quant<T, GATED, NT, TURNS>), dim3((uint32_t)grid, (uint32_t)nranks),
                       dim3(256), 0, stream, args);
    return hipGetLastError();
}

// Non-temporal accesses from 64 MiB moved, as in block_norm.hip, and four
// blocks a group of lanes from there on; below, one: the shorter chain counts
// (8 x 64 x 3584: 4.0 against 4.4 us).
template <typename T, bool GATED>
hipError_t sized(GateArgs args, int nranks, int cu_count, hipStream_t stream)
{
    constexpr uint32_t kGroups = 256 / (AR_SCALE_BLOCK / kPiece<T>);
    args.tall = args.rows >= kGroups ? kGroups : 1u;
    const uint64_t moved = args.rows * args.cols * nranks * (T::kBytes * (GATED ? 2u : 1u) + 1u);
    return moved >= (uint64_t)64 << 20 ? enqueue<T, GATED, true, 4>(args, nranks, cu_count, stream)
                                       : enqueue<T, GATED, false, 1>(args, nranks, cu_count, stream);
}

template <typename T>
hipError_t pick(const GateArgs &args, bool gated, int nranks, int cu_count, hipStream_t stream)
{
    return gated ? sized<T, true>(args, nranks, cu_count, stream)
                 : sized<T, false>(args, nranks, cu_count, stream);
}

}  // namespace

hipError_t launch_gate(const GateArgs &args, int dtype, int act, int nranks, int cu_count,
                       hipStream_t stream)
{
    const bool gated = act == arActSiLU;
    switch (dtype) {
    case kBf16: return pick<Bf16>(args, gated, nranks, cu_count, stream);
    case kFp16: return pick<Fp16>(args, gated, nranks, cu_count, stream);
    default: return pick<Fp32>(args, gated, nranks, cu_count, stream);
    }
}

}  // namespace ar
