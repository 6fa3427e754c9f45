// cache_attention.hip -- attention of one new token a sequence over the paged
// cache.  One workgroup a rank, sequence and query head; each wave takes every
// fourth token with its lanes over the head's values, and the waves' sums are
// joined in LDS.
#include "block_device.hpp"
#include "cache_internal.hpp"

namespace ar {

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

template <typename T>
__device__ inline float element(const char *p, uint64_t i)
{
    if constexpr (T::kBytes == 4) {
        return ((const float *)p)[i];
    } else {
        float f[2];
        T::widen(((const uint16_t *)p)[i], f);
        return f[0];
    }
}

template <typename T, bool EIGHT>
__device__ inline float cached(const char *p, uint64_t i, float scale)
{
    if constexpr (EIGHT)
        return __builtin_amdgcn_cvt_pk_f32_fp8((int)((const uint8_t *)p)[i], false)[0] * scale;
    else
        return element<T>(p, i);
}

template <typename T, bool EIGHT, bool EIGHT_OUT>
__global__ __launch_bounds__(256) void cache_attention(CacheAttentionArgs p)
{
    __shared__ float acc[4][AR_CACHE_MAX_DIM];
    __shared__ float most[4], total[4];
    const uint32_t head = blockIdx.x, seq = blockIdx.y, rank = blockIdx.z;
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t dim = p.cache.dim, kv = head / (p.heads / p.cache.heads);
    const int64_t len = p.lengths[seq];
    bool bad = len < 0 || (uint64_t)len > p.table_pages * p.cache.page_tokens;
    const int64_t n = bad ? 0 : len;
    const int64_t first = p.window != 0 && (uint64_t)n > p.window ? n - (int64_t)p.window : 0;
    const uint64_t q_at = seq * p.q_stride + (uint64_t)head * dim;
    float q[4], o[4] = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
        q[i] = lane + 64 * i < dim ? element<T>(p.q[rank], q_at + lane + 64 * i) : 0.0f;
    const float scale = p.scale * kLog2e;
    float m = -__builtin_inff(), sum = 0.0f;
    for (int64_t t = first + wave; t < n; t += 4) {
        const int32_t page = p.table[seq * p.table_pages + (uint64_t)t / p.cache.page_tokens];
        if (page < 0 || (uint32_t)page >= p.cache.pages) {
            bad = true;
            continue;
        }
        const uint32_t place = (uint32_t)((uint64_t)t % p.cache.page_tokens);
        const uint64_t at = p.cache.at((uint32_t)page, place, kv);
        const uint64_t sat = p.cache.scale_at((uint32_t)page, place, kv);
        const float ks = EIGHT ? p.key_scales[rank][sat] : 1.0f;
        const float vs = EIGHT ? p.value_scales[rank][sat] : 1.0f;
        float x = 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            if (lane + 64 * i < dim)
                x += q[i] * cached<T, EIGHT>(p.keys[rank], at + lane + 64 * i, ks);
        x = sum64(x) * scale;
        const float next = x > m ? x : m;
        const float shift = next == -__builtin_inff() ? 0.0f : next;
        const float keep = __builtin_amdgcn_exp2f(m - shift), w = __builtin_amdgcn_exp2f(x - shift);
        m = next;
        sum = sum * keep + w;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            if (lane + 64 * i < dim)
                o[i] = o[i] * keep + w * cached<T, EIGHT>(p.values[rank], at + lane + 64 * i, vs);
    }
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
        acc[wave][lane + 64 * i] = o[i];
    if (lane == 0) {
        most[wave] = m;
        total[wave] = bad ? __builtin_nanf("") : sum;
    }
    __syncthreads();
    float all = most[0];
    for (int w = 1; w < 4; ++w)
        all = most[w] > all ? most[w] : all;
    const float shift = all == -__builtin_inff() ? 0.0f : all;
    float l = 0.0f, y = 0.0f;
    for (int w = 0; w < 4; ++w) {
        const float keep = __builtin_amdgcn_exp2f(most[w] - shift);
        l += total[w] * keep;
        y += acc[w][threadIdx.x] * keep;
    }
    const bool empty = n == 0 && !bad && len == 0;
    y = empty ? 0.0f : y / l;
    const uint64_t row = (uint64_t)seq * p.heads + head;
    if (p.has_lse != 0 && threadIdx.x == 0)
        p.lse[rank][row] = empty ? -__builtin_inff() : shift * kLn2 + __builtin_logf(l);
    const uint32_t d = threadIdx.x;
    if constexpr (EIGHT_OUT) {
        __shared__ uint32_t bits[2];
        if (threadIdx.x < 2)
            bits[threadIdx.x] = 0;
        __syncthreads();
        if (d < dim)
            atomicMax(&bits[d / 128], __builtin_bit_cast(uint32_t, y) & 0x7fffffffu);
        __syncthreads();
        if (d < dim) {
            const float s = scale_of(bits[d / 128]);
            const float v = quotient(y, reciprocal(s));
            p.out[rank][row * dim + d] = (char)__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false);
            if (d % 128 == 0)
                p.out_scales[rank][((uint64_t)head * dim + d) / 128 * p.seqs + seq] = s;
        }
    } else if (d < dim) {
        float f[2] = {y, y};
        const uint32_t w = T::narrow(f);
        if constexpr (T::kBytes == 4)
            ((uint32_t *)p.out[rank])[row * dim + d] = w;
        else
            ((uint16_t *)p.out[rank])[row * dim + d] = (uint16_t)w;
    }
}

namespace {

template <typename T, bool EIGHT>
hipError_t pick(const CacheAttentionArgs &args, bool eight_out, hipStream_t stream)
{
    const dim3 grid(args.heads, args.seqs, args.nranks);
    if (eight_out)
        hipLaunchKernelGGL((cache_attention<T, EIGHT, true>), grid, dim3(256), 0, stream, args);
    else
        hipLaunchKernelGGL((cache_attention<T, EIGHT, false>), grid, dim3(256), 0, stream, args);
    return hipGetLastError();
}

}  // namespace

uint64_t cache_attention_workspace(uint32_t, int) { return 256; }

hipError_t launch_cache_attention(const CacheAttentionArgs &args, int dtype, bool eight,
                                  bool eight_out, int, hipStream_t stream)
{
    switch (dtype) {
    case kBf16:
        return eight ? pick<Bf16, true>(args, eight_out, stream) : pick<Bf16, false>(args, eight_out, stream);
    case kFp16:
        return eight ? pick<Fp16, true>(args, eight_out, stream) : pick<Fp16, false>(args, eight_out, stream);
    default:
        return eight ? pick<Fp32, true>(args, eight_out, stream) : pick<Fp32, false>(args, eight_out, stream);
    }
}

}  // namespace ar
