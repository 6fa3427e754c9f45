// block_device.hpp -- device-side building blocks of the operators of
// ar_block.h: groups of eight elements, sums and maxima across lanes, 8-bit
// values.
//
// A lane works on groups of eight consecutive columns: one 16-byte access for
// the 16-bit types, two for binary32, 8 bytes of 8-bit values; the 128
// columns that share a scale are the groups of 16 neighbouring lanes (one row
// of the lane network).  A row may start at any element, so the vector types
// carry the element's alignment; gfx950 serves such accesses with the same
// instructions as aligned ones.
#pragma once

#include "ar_device.hpp"

namespace ar {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

constexpr float kEightMax = 448.0f;        // largest e4m3 value
constexpr float kScaleMin = 0x1p-126f;     // smallest scale: its reciprocal is finite

// Eight elements as they lie in memory.
template <typename T>
struct Raw8 {
    static constexpr int kVecs = T::kBytes / 2;  // 16-byte vectors
    u32x4 v[kVecs];
};

template <typename T, bool NT>
__device__ inline Raw8<T> load8(const char *p)
{
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < Raw8<T>::kVecs; ++i) {
        const u32x4_any *q = (const u32x4_any *)p + i;
        if constexpr (NT)
            r.v[i] = __builtin_nontemporal_load(q);
        else
            r.v[i] = *q;
    }
    return r;
}

template <typename T, bool NT>
__device__ inline void store8(char *p, const Raw8<T> &r)
{
#pragma unroll
    for (int i = 0; i < Raw8<T>::kVecs; ++i) {
        u32x4_any *q = (u32x4_any *)p + i;
        if constexpr (NT)
            __builtin_nontemporal_store((u32x4_any)r.v[i], q);
        else
            *q = r.v[i];
    }
}

// The first `n` (1..7) of eight elements; the others read as zero.
template <typename T>
__device__ inline Raw8<T> load_some(const char *p, uint32_t n)
{
    uint32_t w[T::kBytes * 2] = {};
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
        if (i < n) {
            if constexpr (T::kBytes == 2)
                w[i / 2] |= (uint32_t)((const uint16_t *)p)[i] << (16 * (i % 2));
            else
                w[i] = ((const uint32_t *)p)[i];
        }
    }
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < Raw8<T>::kVecs; ++i)
        r.v[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    return r;
}

template <typename T>
__device__ inline void store_some(char *p, const Raw8<T> &r, uint32_t n)
{
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
        if (i < n) {
            if constexpr (T::kBytes == 2)
                ((uint16_t *)p)[i] = (uint16_t)(r.v[0][i / 2] >> (16 * (i % 2)));
            else
                ((uint32_t *)p)[i] = r.v[i / 4][i % 4];
        }
    }
}

template <typename T>
__device__ inline void widen8(const Raw8<T> &r, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 8 / T::kPerWord; ++i)
        T::widen(r.v[i / 4][i % 4], f + i * T::kPerWord);
}

template <typename T>
__device__ inline Raw8<T> narrow8(const float (&f)[8])
{
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < 8 / T::kPerWord; ++i)
        r.v[i / 4][i % 4] = T::narrow(f + i * T::kPerWord);
    return r;
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

// The sum over a wave, in every lane, in a fixed order.
__device__ inline float sum64(float x)
{
    x += __builtin_bit_cast(float, lane_move<0x128>(__builtin_bit_cast(uint32_t, x)));
    x += __builtin_bit_cast(float, lane_move<0x124>(__builtin_bit_cast(uint32_t, x)));
    x += __builtin_bit_cast(float, lane_move<0x122>(__builtin_bit_cast(uint32_t, x)));
    x += __builtin_bit_cast(float, lane_move<0x121>(__builtin_bit_cast(uint32_t, x)));
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

// Magnitude bits order like the magnitudes, with infinity above every finite
// value and NaN above infinity, so a maximum over them keeps a NaN.
__device__ inline uint32_t max_bits8(const float (&y)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
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

// Eight e4m3 values of y * inv, rounded to nearest even.  |y| * inv is at most
// 448 but for a few units in the last place, which round back to 448, so the
// conversion's overflow is never reached.  The reciprocal in place of a
// division moves a value by 2^-23 of itself before a rounding of 2^-4.
__device__ inline u32x2 eight_of(const float (&y)[8], float inv)
{
    u32x2 q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = 0;
        w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i] * inv, y[4 * i + 1] * inv, w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2] * inv, y[4 * i + 3] * inv, w, true);
        q[i] = (uint32_t)w;
    }
    return q;
}

template <bool NT>
__device__ inline void store_eight(char *p, u32x2 q)
{
    if constexpr (NT)
        __builtin_nontemporal_store((u32x2_any)q, (u32x2_any *)p);
    else
        *(u32x2_any *)p = q;
}

__device__ inline void store_eight_some(char *p, u32x2 q, uint32_t n)
{
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i)
        if (i < n)
            p[i] = (char)(q[i / 4] >> (8 * (i % 4)));
}

}  // namespace ar
