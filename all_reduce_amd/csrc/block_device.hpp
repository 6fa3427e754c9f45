// block_device.hpp -- device-side building blocks of the operators of
// ar_block.h: 16-byte pieces of a row, sums and maxima across lanes, 8-bit
// values.
//
// A lane works on pieces of 16 bytes: eight consecutive columns of a 16-bit
// type, four of binary32, so that neighbouring lanes always cover whole lines
// (two pieces a lane for binary32 leave gaps: 16 ranks of 1024 x 7168 took
// 311 us that way and take 211 us this way).  The 128 columns that share a
// scale are the pieces of 16 or 32 neighbouring lanes.  A row may start at
// any element, so the vector types carry the element's alignment; gfx950
// serves such accesses with the same instructions as aligned ones.
#pragma once

#include "ar_allreduce.h"
#include "ar_device.hpp"

namespace ar {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));

constexpr float kEightMax = 448.0f;        // largest e4m3 value
constexpr float kScaleMin = 0x1p-126f;     // smallest scale: its reciprocal is finite

// Brings a rank table's first eight entries into the scalar cache.
template <typename P>
__device__ inline void touch(P *const (&table)[AR_MAX_RANKS])
{
    asm volatile("" : : "s"(table[0]));
}

// Elements of a 16-byte piece.
template <typename T>
constexpr int kPiece = 16 / T::kBytes;

template <bool NT>
__device__ inline u32x4 load_piece(const char *p)
{
    if constexpr (NT)
        return __builtin_nontemporal_load((const u32x4_any *)p);
    else
        return *(const u32x4_any *)p;
}

template <bool NT>
__device__ inline void store_piece(char *p, u32x4 v)
{
    if constexpr (NT)
        __builtin_nontemporal_store((u32x4_any)v, (u32x4_any *)p);
    else
        *(u32x4_any *)p = v;
}

// The first `n` (less than a piece's) elements; the others read as zero.
template <typename T>
__device__ inline u32x4 load_some(const char *p, uint32_t n)
{
    u32x4 r = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t i = 0; i < (uint32_t)kPiece<T>; ++i) {
        if (i < n) {
            if constexpr (T::kBytes == 2)
                r[i / 2] |= (uint32_t)((const uint16_t *)p)[i] << (16 * (i % 2));
            else
                r[i] = ((const uint32_t *)p)[i];
        }
    }
    return r;
}

// A piece without its first `n` elements, zeros behind the others.
template <typename T>
__device__ inline u32x4 drop(u32x4 v, uint32_t n)
{
    const uint32_t bits = n * 8u * T::kBytes;  // 16 .. 112
    uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
    if (bits >= 64u) {
        lo = hi >> (bits - 64u);
        hi = 0;
    } else {
        lo = lo >> bits | hi << (64u - bits);
        hi >>= bits;
    }
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

template <typename T>
__device__ inline void store_some(char *p, u32x4 v, uint32_t n)
{
#pragma unroll
    for (uint32_t i = 0; i < (uint32_t)kPiece<T>; ++i) {
        if (i < n) {
            if constexpr (T::kBytes == 2)
                ((uint16_t *)p)[i] = (uint16_t)(v[i / 2] >> (16 * (i % 2)));
            else
                ((uint32_t *)p)[i] = v[i];
        }
    }
}

template <typename T>
__device__ inline void widen_piece(u32x4 v, float (&f)[kPiece<T>])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        T::widen(v[i], f + i * T::kPerWord);
}

template <typename T>
__device__ inline u32x4 narrow_piece(const float (&f)[kPiece<T>])
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = T::narrow(f + i * T::kPerWord);
    return v;
}

template <int CTRL>
__device__ inline uint32_t lane_move(uint32_t x)
{
    return __builtin_amdgcn_update_dpp(0u, x, CTRL, 0xf, 0xf, false);
}

// The largest of 16 neighbouring lanes, in each of them (lane rotations by 8,
// 4, 2 and 1 within the row of 16).
__device__ inline uint32_t max16(uint32_t x)
{
    uint32_t y = lane_move<0x128>(x);
    x = x > y ? x : y;
    y = lane_move<0x124>(x);
    x = x > y ? x : y;
    y = lane_move<0x122>(x);
    x = x > y ? x : y;
    y = lane_move<0x121>(x);
    return x > y ? x : y;
}

// The largest of the lanes that hold the 128 columns of a scale, in each of
// them: 16 lanes, or 32 where a piece has four columns.
template <typename T>
__device__ inline uint32_t max_block(uint32_t x)
{
    x = max16(x);
    if constexpr (kPiece<T> == 4) {
        const uint32_t y = (uint32_t)__shfl_xor((int)x, 16);
        x = x > y ? x : y;
    }
    return x;
}

template <int CTRL>
__device__ inline double lane_move(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)lane_move<CTRL>((uint32_t)(b >> 32)) << 32 |
                                          lane_move<CTRL>((uint32_t)b));
}

template <int CTRL>
__device__ inline float lane_move(float x)
{
    return __builtin_bit_cast(float, lane_move<CTRL>(__builtin_bit_cast(uint32_t, x)));
}

// The sum over a wave, in every lane, in a fixed order.
template <typename F>
__device__ inline F sum64(F x)
{
    x += lane_move<0x128>(x);
    x += lane_move<0x124>(x);
    x += lane_move<0x122>(x);
    x += lane_move<0x121>(x);
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

// Magnitude bits order like the magnitudes, with infinity above every finite
// value and NaN above infinity, so a maximum over them keeps a NaN.
template <int N>
__device__ inline uint32_t max_bits(const float (&y)[N])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t b = __builtin_bit_cast(uint32_t, y[i]) & 0x7fffffffu;
        m = m > b ? m : b;
    }
    return m;
}

// The scale of a block whose largest magnitude has the bits `m`.
__device__ inline float scale_of(uint32_t m)
{
    const float s = __builtin_bit_cast(float, m) / kEightMax;
    return s < kScaleMin ? kScaleMin : s;  // keeps NaN
}

// 1 / s in two parts, so that y / s is a product and a fused multiply-add,
// within 2^-46 before its one rounding (the product with 1 / s alone is up to
// 2^-23 off; above s = 2^100 the low part has fewer bits, down to 2^-30).  An
// infinite s gives 0 for finite values and NaN for infinite ones.
struct Reciprocal {
    float high, low;
};

__device__ inline Reciprocal reciprocal(float s)
{
    const float high = 1.0f / s;
    const float low = high * __builtin_fmaf(-high, s, 1.0f);
    return {high, high == 0.0f ? 0.0f : low};
}

__device__ inline float quotient(float y, Reciprocal r)
{
    return __builtin_fmaf(y, r.high, y * r.low);
}

// The e4m3 values of y / s, rounded to nearest even, four to a word.  |y| / s
// is at most 448 but for a few units in the last place, which round back to
// 448, so the conversion's overflow is never reached.  (Ties between two e4m3
// values are common where y has few bits: y * (1 / s) took one of 2000 normal
// bfloat16 values to the other side.)
template <int N>
struct Eights {
    uint32_t w[N / 4];
};

template <int N>
__device__ inline Eights<N> to_eights(const float (&y)[N], float s)
{
    const Reciprocal r = reciprocal(s);
    Eights<N> q;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        int w = 0;
        w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(y[4 * i], r), quotient(y[4 * i + 1], r), w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(y[4 * i + 2], r), quotient(y[4 * i + 3], r), w, true);
        q.w[i] = (uint32_t)w;
    }
    return q;
}

template <bool NT, int N>
__device__ inline void store_eights(char *p, const Eights<N> &q)
{
    if constexpr (N == 8) {
        const u32x2_any v = {q.w[0], q.w[1]};
        if constexpr (NT)
            __builtin_nontemporal_store(v, (u32x2_any *)p);
        else
            *(u32x2_any *)p = v;
    } else {
        if constexpr (NT)
            __builtin_nontemporal_store(q.w[0], (u32_any *)p);
        else
            *(u32_any *)p = q.w[0];
    }
}

template <int N>
__device__ inline void store_eights_some(char *p, const Eights<N> &q, uint32_t n)
{
#pragma unroll
    for (uint32_t i = 0; i < (uint32_t)N; ++i)
        if (i < n)
            p[i] = (char)(q.w[i / 4] >> (8 * (i % 4)));
}

}  // namespace ar
