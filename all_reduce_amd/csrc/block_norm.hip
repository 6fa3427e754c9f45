// block_norm.hip -- all-reduce, residual addition and root-mean-square norm of
// R rank buffers in one kernel, with an output in the element type or in 8
// bits with a scale per 128 columns.
//
// A workgroup takes a row: its lanes sum their columns over the ranks (rank
// order, binary32), add the residual and keep h in registers; the sum of
// squares crosses the workgroup through LDS; then every lane scales its own
// columns and stores them to all ranks.  So each input is read once and each
// output written once, and a row's reads are complete before its first write
// (which is what makes the exact in-place forms safe).
//
// It is bound by memory: R + 1 reads and 2 R writes a column at two or three
// operations each.
#include "block_device.hpp"
#include "block_internal.hpp"

namespace ar {

// acc += the values of `COUNT` ranks from rank `r0` on, every load issued
// before the first addition.
template <typename T, int COUNT, bool NT>
__device__ inline void add_ranks(const NormArgs &p, uint32_t r0, uint64_t at, float (&acc)[8])
{
    Raw8<T> x[COUNT];
#pragma unroll
    for (int j = 0; j < COUNT; ++j)
        x[j] = load8<T, NT>(p.send[r0 + j] + at);
#pragma unroll
    for (int j = 0; j < COUNT; ++j) {
        float f[8];
        widen8<T>(x[j], f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            acc[e] = acc[e] + f[e];
    }
}

// V: groups of eight columns a lane holds (lane i holds groups i, i + threads,
// ..).  EIGHT: 8-bit output with scales.  NT: non-temporal accesses.
template <typename T, int V, bool EIGHT, bool NT>
__global__ __launch_bounds__(1024) void norm_rows(NormArgs p)
{
    __shared__ float part[2][16];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t waves = blockDim.x >> 6;
    uint32_t turn = 0;
    for (uint64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1u) {
        const uint64_t row_at = row * p.cols;
        float h[V][8];
        float sq = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t col = (v * blockDim.x + threadIdx.x) * 8u;
            // -0 + x is x for every x: the sum starts from rank 0's value
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[v][e] = -0.0f;
            if (col + 8u <= p.cols) {
                const uint64_t at = (row_at + col) * T::kBytes;
                uint32_t r = 0;
                for (; r + 8u <= p.nranks; r += 8u)
                    add_ranks<T, 8, NT>(p, r, at, h[v]);
                if (p.nranks & 4u) {
                    add_ranks<T, 4, NT>(p, r, at, h[v]);
                    r += 4u;
                }
                if (p.nranks & 2u) {
                    add_ranks<T, 2, NT>(p, r, at, h[v]);
                    r += 2u;
                }
                if (p.nranks & 1u)
                    add_ranks<T, 1, NT>(p, r, at, h[v]);
                if (p.residual != nullptr) {
                    float f[8];
                    widen8<T>(load8<T, NT>(p.residual + at), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        h[v][e] = h[v][e] + f[e];
                }
            } else if (col < p.cols) {
                const uint64_t at = (row_at + col) * T::kBytes;
                const uint32_t n = p.cols - col;
                for (uint32_t r = 0; r <= p.nranks; ++r) {
                    const char *from = r < p.nranks ? p.send[r] : p.residual;
                    if (from == nullptr)
                        break;
                    float f[8];
                    widen8<T>(load_some<T>(from + at, n), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        h[v][e] = h[v][e] + f[e];
                }
            }
            // (columns past the row hold -0 or 0 and add nothing)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sq = __builtin_fmaf(h[v][e], h[v][e], sq);
        }
        sq = sum64(sq);
        if (lane == 0)
            part[turn][wave] = sq;
        // One barrier a row: the next row writes the other half, and the row
        // after that only once every wave has passed the next row's barrier.
        __syncthreads();
        float total = 0.0f;
        for (uint32_t w = 0; w < waves; ++w)
            total += part[turn][w];
        const float inv = 1.0f / __builtin_sqrtf(total / (float)p.cols + p.eps);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t col = (v * blockDim.x + threadIdx.x) * 8u;
            const bool full = col + 8u <= p.cols;
            const uint32_t n = col < p.cols ? p.cols - col : 0u;
            const uint64_t at = row_at + col;
            if (p.has_res_out != 0 && n != 0) {
                const Raw8<T> x = narrow8<T>(h[v]);
                for (uint32_t r = 0; r < p.nranks; ++r) {
                    if (full)
                        store8<T, NT>(p.res_out[r] + at * T::kBytes, x);
                    else
                        store_some<T>(p.res_out[r] + at * T::kBytes, x, n);
                }
            }
            float y[8] = {};
            if (n != 0) {
                const char *w = p.weight + (uint64_t)col * T::kBytes;
                float f[8];
                widen8<T>(full ? load8<T, false>(w) : load_some<T>(w, n), f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = full || (uint32_t)e < n ? h[v][e] * inv * f[e] : 0.0f;
            }
            if constexpr (EIGHT) {
                // all lanes of a scale's 16 take part; those past the row hold 0
                const float s = scale_of(max16(max_bits8(y)));
                const u32x2 q = eight_of(y, 1.0f / s);
                if (n != 0) {
                    const uint64_t sat = (uint64_t)(col / AR_SCALE_BLOCK) * p.rows + row;
                    for (uint32_t r = 0; r < p.nranks; ++r) {
                        if (full)
                            store_eight<NT>(p.out[r] + at, q);
                        else
                            store_eight_some(p.out[r] + at, q, n);
                        if ((lane & 15u) == 0)
                            p.scales[r][sat] = s;
                    }
                }
            } else if (n != 0) {
                const Raw8<T> x = narrow8<T>(y);
                for (uint32_t r = 0; r < p.nranks; ++r) {
                    if (full)
                        store8<T, NT>(p.out[r] + at * T::kBytes, x);
                    else
                        store_some<T>(p.out[r] + at * T::kBytes, x, n);
                }
            }
        }
    }
}

namespace {

template <typename T, int V, bool EIGHT>
hipError_t enqueue(const NormArgs &args, uint32_t threads, bool nt, hipStream_t stream)
{
    const uint32_t grid = args.rows < (1u << 20) ? (uint32_t)args.rows : (1u << 20);
    if (nt)
        hipLaunchKernelGGL((norm_rows<T, V, EIGHT, true>), dim3(grid), dim3(threads), 0, stream, args);
    else
        hipLaunchKernelGGL((norm_rows<T, V, EIGHT, false>), dim3(grid), dim3(threads), 0, stream, args);
    return hipGetLastError();
}

template <typename T, bool EIGHT>
hipError_t pick(const NormArgs &args, hipStream_t stream)
{
    const uint32_t groups = (args.cols + 7u) / 8u;
    uint32_t threads = (groups + 63u) / 64u * 64u;
    if (threads > 1024u)
        threads = 1024u;
    const uint32_t v = (groups + threads - 1u) / threads;
    const bool nt = args.rows * args.cols * T::kBytes * args.nranks > ((uint64_t)128 << 20);
    if (v <= 1)
        return enqueue<T, 1, EIGHT>(args, threads, nt, stream);
    if (v <= 2)
        return enqueue<T, 2, EIGHT>(args, threads, nt, stream);
    return enqueue<T, 4, EIGHT>(args, threads, nt, stream);
}

}  // namespace

hipError_t launch_norm(const NormArgs &args, int dtype, bool eight, int cu_count,
                       hipStream_t stream)
{
    (void)cu_count;
    switch (dtype) {
    case kBf16: return eight ? pick<Bf16, true>(args, stream) : pick<Bf16, false>(args, stream);
    case kFp16: return eight ? pick<Fp16, true>(args, stream) : pick<Fp16, false>(args, stream);
    default: return eight ? pick<Fp32, true>(args, stream) : pick<Fp32, false>(args, stream);
    }
}

}  // namespace ar
