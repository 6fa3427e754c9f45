// cache_copy.hip -- new keys and values into the pages of the cache, in the
// element type or in 8 bits with a scale per token and head, and back.
//
// LANES neighbouring lanes hold the `dim` values of a token and head, 16 bytes
// of the row each: the largest magnitude is a few lane moves away, each value is
// read once and written once.  A row's slot and its values are loaded at once,
// and the address follows from the slot.  Bound by memory: on MI355X 16384 tokens x 8
// ranks with 2 heads of 128 are written from bfloat16 to 8 bits in 37.6 us and read
// back in 31.4 (185 MB: 4.9 and 5.9 TB/s; a copy reaches 5.1); few tokens take a
// launch, 4.7 us.
#include "block_device.hpp"
#include "cache_internal.hpp"

namespace ar {

// The largest of LANES neighbouring lanes, in each of them.
template <int LANES>
__device__ inline uint32_t max_lanes(uint32_t x)
{
    auto with = [&](uint32_t y) { x = x > y ? x : y; };
    with(lane_move<0xB1>(x));   // the neighbour, the other pair of four,
    with(lane_move<0x4E>(x));
    with(lane_move<0x141>(x));  // the other four of eight
    if constexpr (LANES >= 16)
        with(lane_move<0x140>(x));
    if constexpr (LANES >= 32)
        with((uint32_t)__shfl_xor((int)x, 16));
    if constexpr (LANES >= 64)
        with((uint32_t)__shfl_xor((int)x, 32));
    return x;
}

// The token of row `r` of `count` (in 64 bits a division is several times longer).
__device__ inline uint32_t token_of(uint64_t r, uint64_t count, uint32_t heads)
{
    return heads == 1 ? (uint32_t)r : count >> 32 == 0 ? (uint32_t)r / heads : (uint32_t)(r / heads);
}

// One rank per blockIdx.y, keys or values per blockIdx.z, TURNS rows a group of
// lanes.
template <typename T, bool EIGHT, int LANES, int TURNS, bool NT>
__global__ __launch_bounds__(256) void cache_write(CacheCopyArgs p)
{
    constexpr uint32_t E = kPiece<T>, kGroups = 256 / LANES;
    const char *rows = p.rows[blockIdx.z][blockIdx.y];
    char *pages = p.pages[blockIdx.z][blockIdx.y];
    float *scales = p.scales[blockIdx.z][blockIdx.y];
    const uint32_t d = threadIdx.x % LANES * E;
    const uint64_t count = (uint64_t)p.tokens * p.cache.heads;
    for (uint64_t r0 = (uint64_t)blockIdx.x * kGroups * TURNS + threadIdx.x / LANES; r0 < count;
         r0 += (uint64_t)gridDim.x * kGroups * TURNS) {
        u32x4 x[TURNS];
        int64_t slot[TURNS];
        uint32_t head[TURNS];
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            const uint64_t r = r0 + t * kGroups;
            x[t] = u32x4{0, 0, 0, 0};
            slot[t] = -1;
            head[t] = 0;
            if (r < count) {
                const uint32_t token = token_of(r, count, p.cache.heads);
                head[t] = (uint32_t)(r - (uint64_t)token * p.cache.heads);
                slot[t] = p.slots[token];
                if (d < p.cache.dim)
                    x[t] = load_piece<NT>(
                        rows + (token * p.row_stride + head[t] * p.cache.dim + d) * T::kBytes);
            }
        }
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            uint32_t page = 0, place = 0;
            const bool there = p.cache.place(slot[t], &page, &place);
            const uint64_t at = p.cache.at(page, place, head[t]) + d;
            if constexpr (EIGHT) {
                float y[E];
                widen_piece<T>(x[t], y);
                const float s = scale_of(max_lanes<LANES>(max_bits(y)));
                const Eights<E> q = to_eights(y, s);
                if (there && d < p.cache.dim)
                    store_eights<NT>(pages + at, q);
                if (there && d == 0)
                    scales[p.cache.scale_at(page, place, head[t])] = s;
            } else {
                if (there && d < p.cache.dim)
                    store_piece<NT>(pages + at * T::kBytes, x[t]);
            }
        }
    }
}

// Four or eight e4m3 values times a scale, in binary32 (the product is exact but
// for its one rounding).
template <int N>
__device__ inline void from_eights(const uint32_t (&w)[N / 4], float s, float (&y)[N])
{
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        y[4 * i] = lo[0] * s;
        y[4 * i + 1] = lo[1] * s;
        y[4 * i + 2] = hi[0] * s;
        y[4 * i + 3] = hi[1] * s;
    }
}

template <typename T, bool EIGHT, int LANES, int TURNS, bool NT>
__global__ __launch_bounds__(256) void cache_read(CacheCopyArgs p)
{
    constexpr uint32_t E = kPiece<T>, kGroups = 256 / LANES;
    char *rows = p.rows[blockIdx.z][blockIdx.y];
    const char *pages = p.pages[blockIdx.z][blockIdx.y];
    const float *scales = p.scales[blockIdx.z][blockIdx.y];
    const uint32_t d = threadIdx.x % LANES * E;
    const uint64_t count = (uint64_t)p.tokens * p.cache.heads;
    for (uint64_t r0 = (uint64_t)blockIdx.x * kGroups * TURNS + threadIdx.x / LANES; r0 < count;
         r0 += (uint64_t)gridDim.x * kGroups * TURNS) {
        u32x4 x[TURNS];
        float s[TURNS];
        uint64_t to[TURNS];
        bool there[TURNS];
        int64_t slot[TURNS];
        uint32_t head[TURNS];
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            const uint64_t r = r0 + t * kGroups;
            slot[t] = -1;
            head[t] = 0;
            to[t] = 0;
            if (r < count) {
                const uint32_t token = token_of(r, count, p.cache.heads);
                head[t] = (uint32_t)(r - (uint64_t)token * p.cache.heads);
                slot[t] = p.slots[token];
                to[t] = token * p.row_stride + head[t] * p.cache.dim + d;
            }
        }
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            uint32_t page = 0, place = 0;
            there[t] = p.cache.place(slot[t], &page, &place) && d < p.cache.dim;
            const uint64_t at = p.cache.at(page, place, head[t]) + d;
            if (there[t]) {
                if constexpr (!EIGHT) {
                    x[t] = load_piece<NT>(pages + at * T::kBytes);
                } else {
                    s[t] = scales[p.cache.scale_at(page, place, head[t])];
                    if constexpr (E == 8) {
                        const u32x2_any v = *(const u32x2_any *)(pages + at);
                        x[t][0] = v[0];
                        x[t][1] = v[1];
                    } else {
                        x[t][0] = *(const u32_any *)(pages + at);
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            if (!there[t])
                continue;
            if constexpr (EIGHT) {
                uint32_t w[E / 4];
#pragma unroll
                for (uint32_t i = 0; i < E / 4; ++i)
                    w[i] = x[t][i];
                float y[E];
                from_eights<E>(w, s[t], y);
                x[t] = narrow_piece<T>(y);
            }
            store_piece<NT>(rows + to[t] * T::kBytes, x[t]);
        }
    }
}

namespace {

template <bool WRITE, typename T, bool EIGHT, int LANES, int TURNS, bool NT>
hipError_t enqueue(const CacheCopyArgs &args, int nranks, int cu_count, hipStream_t stream)
{
    const uint64_t each = 256 / LANES * TURNS;
    uint64_t grid = ((uint64_t)args.tokens * args.cache.heads + each - 1) / each;
    const uint64_t most = (uint64_t)cu_count * 256;
    grid = grid < most ? grid : most;
    const dim3 blocks((uint32_t)grid, (uint32_t)nranks, 2);
    if constexpr (WRITE)
        hipLaunchKernelGGL((cache_write<T, EIGHT, LANES, TURNS, NT>), blocks, dim3(256), 0, stream, args);
    else
        hipLaunchKernelGGL((cache_read<T, EIGHT, LANES, TURNS, NT>), blocks, dim3(256), 0, stream, args);
    return hipGetLastError();
}

// By the bytes that a call reads and writes (us on MI355X; 8 ranks, a head of 128):
//   four rows a group of lanes from 64 MiB on, so that more loads are on the way at
//   once: 134 MB of bfloat16 written in 22.6 in place of 24.2, 101 MB from bfloat16 to
//   8 bits in 20.9 in place of 22.4; at 34 MB the same (7.4 and 7.6);
//   non-temporal from 160 MiB on, where the last-level cache would not keep them: 201 MB
//   of bfloat16 and 8 bits written in 38.5 in place of 43.0, read in 31.3 in place of
//   40.0; but 134 MB written in 23.9 in place of 22.8.
template <bool WRITE, typename T, bool EIGHT, int LANES>
hipError_t sized(const CacheCopyArgs &args, int nranks, int cu_count, hipStream_t stream)
{
    const uint64_t moved = (uint64_t)args.tokens * args.cache.heads * args.cache.dim * nranks * 2u *
                           (T::kBytes + (EIGHT ? 1u : T::kBytes));
    if (moved >= (uint64_t)160 << 20)
        return enqueue<WRITE, T, EIGHT, LANES, 4, true>(args, nranks, cu_count, stream);
    if (moved >= (uint64_t)64 << 20)
        return enqueue<WRITE, T, EIGHT, LANES, 4, false>(args, nranks, cu_count, stream);
    return enqueue<WRITE, T, EIGHT, LANES, 1, false>(args, nranks, cu_count, stream);
}

template <bool WRITE, typename T, bool EIGHT>
hipError_t pick(const CacheCopyArgs &args, int nranks, int cu_count, hipStream_t stream)
{
    const uint32_t pieces = args.cache.dim / kPiece<T>;
    if (pieces <= 8)
        return sized<WRITE, T, EIGHT, 8>(args, nranks, cu_count, stream);
    if (pieces <= 16)
        return sized<WRITE, T, EIGHT, 16>(args, nranks, cu_count, stream);
    if (pieces <= 32)
        return sized<WRITE, T, EIGHT, 32>(args, nranks, cu_count, stream);
    if constexpr (kPiece<T> == 4)  // (a 16-bit row of 256 has 32 pieces)
        return sized<WRITE, T, EIGHT, 64>(args, nranks, cu_count, stream);
    return hipErrorInvalidValue;
}

template <bool WRITE>
hipError_t typed(const CacheCopyArgs &args, int dtype, bool eight, int nranks, int cu_count,
                 hipStream_t stream)
{
    switch (dtype) {
    case kBf16:
        return eight ? pick<WRITE, Bf16, true>(args, nranks, cu_count, stream)
                     : pick<WRITE, Bf16, false>(args, nranks, cu_count, stream);
    case kFp16:
        return eight ? pick<WRITE, Fp16, true>(args, nranks, cu_count, stream)
                     : pick<WRITE, Fp16, false>(args, nranks, cu_count, stream);
    default:
        return eight ? pick<WRITE, Fp32, true>(args, nranks, cu_count, stream)
                     : pick<WRITE, Fp32, false>(args, nranks, cu_count, stream);
    }
}

}  // namespace

hipError_t launch_cache_write(const CacheCopyArgs &args, int dtype, bool eight, int nranks,
                              int cu_count, hipStream_t stream)
{
    return typed<true>(args, dtype, eight, nranks, cu_count, stream);
}

hipError_t launch_cache_read(const CacheCopyArgs &args, int dtype, bool eight, int nranks,
                             int cu_count, hipStream_t stream)
{
    return typed<false>(args, dtype, eight, nranks, cu_count, stream);
}

}  // namespace ar
