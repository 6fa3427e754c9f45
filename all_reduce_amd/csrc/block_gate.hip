// block_gate.hip -- SiLU gate (or nothing) and quantisation to 8 bits with a
// scale per row and 128 columns, for R rank buffers in one launch.
//
// Sixteen neighbouring lanes hold the 128 columns of a scale, eight each: the
// block's largest magnitude is four lane rotations away, and each value is
// read once and written once.  Bound by memory: 4 bytes read and 1 written a
// value for 16-bit gated inputs.
#include "block_device.hpp"
#include "block_internal.hpp"

namespace ar {

// One rank per grid row (blockIdx.y).
template <typename T, bool GATED>
__global__ __launch_bounds__(256) void gate_quant(GateArgs p)
{
    const uint32_t rank = blockIdx.y;
    const char *in = p.in[rank];
    char *out = p.out[rank];
    float *scales = p.scales[rank];
    const uint64_t blocks = (p.cols + AR_SCALE_BLOCK - 1) / AR_SCALE_BLOCK;
    const uint64_t units = p.rows * blocks;  // one scale each
    const uint64_t wide = GATED ? 2 * p.cols : p.cols;
    for (uint64_t u = (uint64_t)blockIdx.x * 16u + threadIdx.x / 16u; u < units;
         u += (uint64_t)gridDim.x * 16u) {
        const uint64_t row = u / blocks, block = u % blocks;
        const uint64_t col = block * AR_SCALE_BLOCK + (threadIdx.x & 15u) * 8u;
        const uint32_t n = col >= p.cols ? 0u : p.cols - col < 8u ? (uint32_t)(p.cols - col) : 8u;
        float y[8] = {};
        if (n != 0) {
            const char *at = in + (row * wide + col) * T::kBytes;
            widen8<T>(n == 8u ? load8<T, false>(at) : load_some<T>(at, n), y);
            if constexpr (GATED) {
                const char *at2 = at + p.cols * T::kBytes;
                float f[8];
                widen8<T>(n == 8u ? load8<T, false>(at2) : load_some<T>(at2, n), f);
                // (columns past the row are 0 / 2 * 0)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = y[e] / (1.0f + __expf(-y[e])) * f[e];
            }
        }
        const float s = scale_of(max16(max_bits8(y)));
        const u32x2 q = eight_of(y, 1.0f / s);
        if (n == 8u)
            store_eight<false>(out + row * p.cols + col, q);
        else if (n != 0)
            store_eight_some(out + row * p.cols + col, q, n);
        if ((threadIdx.x & 15u) == 0)
            scales[block * p.rows + row] = s;
    }
}

namespace {

template <typename T>
hipError_t pick(const GateArgs &args, bool gated, int nranks, int cu_count, hipStream_t stream)
{
    const uint64_t blocks = (args.cols + AR_SCALE_BLOCK - 1) / AR_SCALE_BLOCK;
    uint64_t grid = (args.rows * blocks + 15) / 16;
    const uint64_t most = (uint64_t)cu_count * 64;
    grid = grid < most ? grid : most;
    const dim3 g((uint32_t)grid, (uint32_t)nranks);
    if (gated)
        hipLaunchKernelGGL((gate_quant<T, true>), g, dim3(256), 0, stream, args);
    else
        hipLaunchKernelGGL((gate_quant<T, false>), g, dim3(256), 0, stream, args);
    return hipGetLastError();
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
