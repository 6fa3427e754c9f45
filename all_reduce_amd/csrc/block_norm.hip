// block_norm.hip -- all-reduce, residual addition and root-mean-square norm of
// R rank buffers in one kernel, with an output in the element type or in 8
// bits with a scale per 128 columns.
//
// A workgroup takes a row: its lanes sum their columns over the ranks (rank
// order, binary32), add the residual and keep h in registers; the sum of
// squares crosses the workgroup through LDS; then every lane scales its own
// columns and stores them to all ranks.  So each input is read once and each
// output written once, and a row's reads are complete before its first write
// (which is what makes the exact in-place forms safe).  Where there are fewer
// rows than compute units, several workgroups take a row, each sums all of it
// and each stores to its share of the ranks: a row's stores are more bytes
// than its reads and take longer than reading it again from the cache.
//
// The sum of squares is binary32 where that holds the mean; rows beyond 1e18
// and, where eps does not cover them, below 1e-12 take it again in binary64,
// which loses no square of a finite h.  (A binary64 sum for every row: 64 rows
// of 8 ranks x 8192 take 7.4 in place of 7.2 us.)
//
// It is bound by memory: R + 1 reads and 2 R writes a column at two or three
// operations each.  On MI355X 8 x 8192 x 8192 bfloat16 with residual takes
// 656 us (5.1 TB/s; a large copy runs at 5.1), 16 x 1024 x 7168 float32 with
// an 8-bit output 210 us (5.2 TB/s).  In a graph one row of 8 x 8192 takes
// 4.4 us (5.5 with one workgroup a row) and 64 rows 6.9, bound by a row's chain
// of loads, sum and stores.
#include <type_traits>

#include "block_device.hpp"
#include "block_internal.hpp"

namespace ar {

// h += the values of `COUNT` ranks from rank `r0` on, in rank order.  Every
// load is issued before the first addition.  `back`: columns that a lane's
// piece starts early, to end with the row; they are dropped again.
template <typename T, int V, int COUNT, bool NT, bool RAGGED>
__device__ inline void add_ranks(const NormArgs &p, uint32_t r0, uint64_t row_at,
                                 const uint32_t (&col)[V], const uint32_t (&back)[V],
                                 float (&h)[V][kPiece<T>])
{
    u32x4 x[V][COUNT];
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (col[v] < p.cols)
#pragma unroll
            for (int j = 0; j < COUNT; ++j)
                x[v][j] = load_piece<NT>(p.send[r0 + j] +
                                         (row_at + col[v] - (RAGGED ? back[v] : 0u)) * T::kBytes);
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (col[v] < p.cols) {
            if (RAGGED && back[v] != 0)
#pragma unroll
                for (int j = 0; j < COUNT; ++j)
                    x[v][j] = drop<T>(x[v][j], back[v]);
#pragma unroll
            for (int j = 0; j < COUNT; ++j) {
                float f[kPiece<T>];
                widen_piece<T>(x[v][j], f);
#pragma unroll
                for (int e = 0; e < kPiece<T>; ++e)
                    h[v][e] = h[v][e] + f[e];
            }
        }
}

// 1 / sqrt(m) for m in 2^-100 .. 2^126, with one rounding but for 2^-45 of it:
// the root's reciprocal, off by e / 2 of itself with e = 1 - m r r.  So h times
// it rounds as often as h divided by a rounded root.
__device__ inline float inverse_root(float m)
{
    const float r = 1.0f / __builtin_sqrtf(m);
    const float mr = m * r, low = __builtin_fmaf(m, r, -mr);
    const float e = __builtin_fmaf(-low, r, __builtin_fmaf(-mr, r, 1.0f));
    return __builtin_fmaf(0.5f * r, e, r);
}

// V: pieces a lane holds (lane i holds pieces i, i + threads, ..).  EIGHT:
// 8-bit output with scales.  NT: non-temporal accesses.  RAGGED: cols is not a
// multiple of a piece's.
template <typename T, int V, bool EIGHT, bool NT, bool RAGGED>
__global__ __launch_bounds__(1024) void norm_rows(NormArgs p)
{
    constexpr uint32_t E = kPiece<T>;
    constexpr uint32_t kBatch = 8 / V;  // ranks whose loads are under way at once: 8 pieces a lane
    __shared__ float part[2][16];
    __shared__ double wide[16];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t waves = blockDim.x >> 6;
    // The tables of where to store are touched here: their first use costs a
    // trip to memory, one after the other where they are used.
    touch(p.res_out);
    touch(p.out);
    touch(p.scales);
    // A row's last columns, fewer than a piece, are read with a piece that
    // starts early (one load like the others'; element by element, rank after
    // rank, 3 x 333 x 5001 took 7.5 us); a row that is shorter than a piece is
    // read by elements.
    const bool tiny = RAGGED && p.cols < E;
    uint32_t col[V], back[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        col[v] = (v * blockDim.x + threadIdx.x) * E;
        back[v] = RAGGED && col[v] < p.cols && col[v] + E > p.cols && !tiny ? col[v] + E - p.cols : 0u;
    }
    auto load_at = [&](auto nt, const char *row, int v) {
        if (tiny)
            return col[v] < p.cols ? load_some<T>(row, p.cols) : u32x4{0, 0, 0, 0};
        if (col[v] >= p.cols)
            return u32x4{0, 0, 0, 0};
        const u32x4 x = load_piece<decltype(nt)::value>(row + (uint64_t)(col[v] - back[v]) * T::kBytes);
        return back[v] != 0 ? drop<T>(x, back[v]) : x;
    };
    auto load_weight = [&](int v) { return load_at(std::false_type{}, p.weight, v); };
    auto load_residual = [&](uint64_t row_at, int v) {
        return load_at(std::integral_constant<bool, NT>{}, p.residual + row_at * T::kBytes, v);
    };
    // The weights are loaded here, and a row's residual before its sum, so that
    // a single row does not wait for them one after the other; a lane with
    // many pieces has no registers for it.
    constexpr bool kEarly = V <= 2;
    u32x4 weight[V];
    if constexpr (kEarly) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            weight[v] = load_weight(v);
    }
    // The p.split workgroups of a row each sum all of it, and each stores to
    // every split-th rank.  Rows go round the eight XCDs (workgroup w runs on
    // XCD w % 8) and a row's workgroups share one, and its cache.
    const uint32_t share = blockIdx.x / 8u % p.split;
    uint32_t turn = 0;
    for (uint64_t row = blockIdx.x / (8u * p.split) * 8u + blockIdx.x % 8u; row < p.rows;
         row += gridDim.x / p.split, turn ^= 1u) {
        const uint64_t row_at = row * p.cols;
        float h[V][E];
        u32x4 res[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            // -0 + x is x for every x: the sum starts from rank 0's value
#pragma unroll
            for (uint32_t e = 0; e < E; ++e)
                h[v][e] = -0.0f;
            if (kEarly && p.residual != nullptr)
                res[v] = load_residual(row_at, v);
        }
        uint32_t r = tiny ? p.nranks : 0u;
        for (; r + kBatch <= p.nranks; r += kBatch)
            add_ranks<T, V, kBatch, NT, RAGGED>(p, r, row_at, col, back, h);
        if constexpr (kBatch > 4) {
            if (p.nranks & 4u && !tiny) {
                add_ranks<T, V, 4, NT, RAGGED>(p, r, row_at, col, back, h);
                r += 4u;
            }
        }
        if constexpr (kBatch > 2) {
            if (p.nranks & 2u && !tiny) {
                add_ranks<T, V, 2, NT, RAGGED>(p, r, row_at, col, back, h);
                r += 2u;
            }
        }
        if constexpr (kBatch > 1) {
            if (p.nranks & 1u && !tiny)
                add_ranks<T, V, 1, NT, RAGGED>(p, r, row_at, col, back, h);
        }
        float sq = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (tiny && col[v] < p.cols) {
                for (uint32_t q = 0; q < p.nranks; ++q) {
                    float f[E];
                    widen_piece<T>(load_some<T>(p.send[q] + row_at * T::kBytes, p.cols), f);
#pragma unroll
                    for (uint32_t e = 0; e < E; ++e)
                        h[v][e] = h[v][e] + f[e];
                }
            }
            if (p.residual != nullptr) {
                float f[E];
                if constexpr (!kEarly)
                    res[v] = load_residual(row_at, v);
                widen_piece<T>(res[v], f);
#pragma unroll
                for (uint32_t e = 0; e < E; ++e)
                    h[v][e] = h[v][e] + f[e];
            }
            // (columns past the row hold -0 or 0 and add nothing)
#pragma unroll
            for (uint32_t e = 0; e < E; ++e)
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
        // (the same in every lane of the workgroup)
        const float mean = __builtin_bit_cast(
            float, __builtin_amdgcn_readfirstlane(
                       __builtin_bit_cast(int, total / (float)p.cols + p.eps)));
        float inv;
        int up = 0;
        if (std::is_same<T, Fp16>::value || (mean >= 0x1p-80f && mean <= 0x1p120f)) {
            // (33 float16 values and their squares stay in range, but for
            // infinities; of a row of zeros without eps NaN is to come)
            inv = mean < __builtin_inff() ? inverse_root(mean) : 1.0f / __builtin_sqrtf(mean);
        } else {
            // h * inv is scaled by 2^-up and 2^up, with which the root lies in
            // [0.7, 1.5).  (`wide` is written again only behind the next row's
            // barrier, which every wave reaches after it has read it here.)
            double square = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (uint32_t e = 0; e < E; ++e)
                    square = __builtin_fma((double)h[v][e], (double)h[v][e], square);
            square = sum64(square);
            if (lane == 0)
                wide[wave] = square;
            __syncthreads();
            double sum = 0.0;
            for (uint32_t w = 0; w < waves; ++w)
                sum += wide[w];
            sum = sum / (double)p.cols + (double)p.eps;
            up = __builtin_amdgcn_frexp_exp(sum) >> 1;  // (0 for 0, infinity and NaN)
            const float m = (float)__builtin_ldexp(sum, -2 * up);
            inv = m > 0.0f && m < __builtin_inff() ? inverse_root(m) : 1.0f / __builtin_sqrtf(m);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool full = !RAGGED || col[v] + E <= p.cols;
            const uint32_t n = col[v] < p.cols ? p.cols - col[v] : 0u;
            const uint64_t at = row_at + col[v];
            if (p.has_res_out != 0 && n != 0) {
                const u32x4 x = narrow_piece<T>(h[v]);
                for (uint32_t r = share; r < p.nranks; r += p.split) {
                    if (full)
                        store_piece<NT>(p.res_out[r] + at * T::kBytes, x);
                    else
                        store_some<T>(p.res_out[r] + at * T::kBytes, x, n);
                }
            }
            float y[E], f[E];
            if constexpr (!kEarly)
                weight[v] = load_weight(v);
            if (up != 0)
#pragma unroll
                for (uint32_t e = 0; e < E; ++e)
                    h[v][e] = __builtin_ldexpf(h[v][e], -up);
            widen_piece<T>(weight[v], f);
#pragma unroll
            for (uint32_t e = 0; e < E; ++e)
                y[e] = (RAGGED ? e < n : n != 0) ? h[v][e] * inv * f[e] : 0.0f;
            if constexpr (EIGHT) {
                // all lanes of a scale take part; those past the row hold 0
                const float s = scale_of(max_block<T>(max_bits(y)));
                const Eights<E> q = to_eights(y, s);
                if (n != 0) {
                    const uint64_t sat = (uint64_t)(col[v] / AR_SCALE_BLOCK) * p.rows + row;
                    for (uint32_t r = share; r < p.nranks; r += p.split) {
                        if (full)
                            store_eights<NT>(p.out[r] + at, q);
                        else
                            store_eights_some(p.out[r] + at, q, n);
                        if (col[v] % AR_SCALE_BLOCK == 0)
                            p.scales[r][sat] = s;
                    }
                }
            } else if (n != 0) {
                const u32x4 x = narrow_piece<T>(y);
                for (uint32_t r = share; r < p.nranks; r += p.split) {
                    if (full)
                        store_piece<NT>(p.out[r] + at * T::kBytes, x);
                    else
                        store_some<T>(p.out[r] + at * T::kBytes, x, n);
                }
            }
        }
    }
}

namespace {

template <typename T, int V, bool EIGHT, bool NT>
hipError_t enqueue(const NormArgs &args, uint32_t threads, hipStream_t stream)
{
    const uint64_t rows = args.rows < (1u << 20) ? args.rows : (1u << 20);
    const uint32_t grid = (uint32_t)((rows + 7u) / 8u * 8u * args.split);
    if (args.cols % kPiece<T> != 0)
        hipLaunchKernelGGL((norm_rows<T, V, EIGHT, NT, true>), dim3(grid), dim3(threads), 0, stream, args);
    else
        hipLaunchKernelGGL((norm_rows<T, V, EIGHT, NT, false>), dim3(grid), dim3(threads), 0, stream, args);
    return hipGetLastError();
}

template <typename T, int V, bool EIGHT>
hipError_t enqueue(const NormArgs &args, uint32_t threads, bool nt, hipStream_t stream)
{
    return nt ? enqueue<T, V, EIGHT, true>(args, threads, stream)
              : enqueue<T, V, EIGHT, false>(args, threads, stream);
}

// As many lanes a row as it has pieces where rows are few (the pieces' loads
// are then all under way at once: one row of 8 ranks x 8192 takes 6.0 us with
// 1024 lanes and 8.0 with 512); two pieces a lane where there are rows for
// every compute unit (the smaller workgroups overlap one row's stores with
// another's loads: 1 x 8192 x 8192 takes 96 against 111 us, 8 x 512 x 8192
// 32.6 against 33.9, 8 x 8192 x 8192 638 against 645).
// Non-temporal accesses from 64 MiB moved (8 x 512 x 8192: 33 against 43 us;
// 8 x 4096 x 512, 88 MB: 19.7 against 19.9; below that the two are equal, and
// what reads the results next finds them in the last-level cache).
template <typename T, bool EIGHT>
hipError_t pick(NormArgs args, int cu_count, hipStream_t stream)
{
    const uint32_t pieces = (args.cols + kPiece<T> - 1u) / kPiece<T>;
    const bool many = args.rows >= 2u * (uint64_t)cu_count;
    uint32_t v = many && pieces >= 128u ? 2u : 1u;
    while (v * 1024u < pieces)
        v *= 2u;
    const uint32_t threads = (pieces + 64u * v - 1u) / (64u * v) * 64u;
    const uint64_t moved = args.rows * args.cols * args.nranks *
                           (T::kBytes * (args.has_res_out != 0 ? 2u : 1u) + (EIGHT ? 1u : T::kBytes));
    const bool nt = moved >= (uint64_t)64 << 20;
    // Fewer rows than compute units: a row's stores are shared out by rank.
    // (In place that would write what another workgroup has yet to read.)
    uint64_t split = args.in_place != 0 ? 1u : (uint64_t)cu_count / args.rows;
    split = split < args.nranks ? split : args.nranks;
    args.split = split < 1u ? 1u : (uint32_t)split;
    switch (v) {
    case 1: return enqueue<T, 1, EIGHT>(args, threads, nt, stream);
    case 2: return enqueue<T, 2, EIGHT>(args, threads, nt, stream);
    case 4: return enqueue<T, 4, EIGHT>(args, threads, nt, stream);
    }
    // (a 16-bit row of 32768 columns has four pieces a lane)
    if constexpr (kPiece<T> == 4)
        return enqueue<T, 8, EIGHT>(args, threads, nt, stream);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_norm(const NormArgs &args, int dtype, bool eight, int cu_count,
                       hipStream_t stream)
{
    switch (dtype) {
    case kBf16: return eight ? pick<Bf16, true>(args, cu_count, stream) : pick<Bf16, false>(args, cu_count, stream);
    case kFp16: return eight ? pick<Fp16, true>(args, cu_count, stream) : pick<Fp16, false>(args, cu_count, stream);
    default: return eight ? pick<Fp32, true>(args, cu_count, stream) : pick<Fp32, false>(args, cu_count, stream);
    }
}

}  // namespace ar
