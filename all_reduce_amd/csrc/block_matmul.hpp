// block_matmul.hpp -- device code that the kernels of the block-scaled 8-bit
// product share: one block's sums, in either matrix instruction's shape.
#pragma once

#include "block_device.hpp"
#include "block_internal.hpp"

namespace ar {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Bytes 8 s .. 8 s + 7 of a lane's block as bfloat16, exactly.
__device__ inline bf16x8 widen_eight(i32x8 x, int s)
{
    bf16x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2 v = i % 2 == 0
                             ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * s + i / 2], 1.0f, false)
                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * s + i / 2], 1.0f, true);
        r[2 * i] = v[0];
        r[2 * i + 1] = v[1];
    }
    return r;
}

// The sums of one block of 128 products, 16 x 16 of them.
//
// The 8-bit instruction adds products in groups of eight (8 consecutive k);
// inside a group each product is cut, toward zero, at 2^-13 of the largest
// one's leading bit, and the groups' sums are added in binary32.  Measured on
// MI355X: normal inputs come out 1.4e-5 off in the 2-norm (a binary32 sum is
// 1e-7 off).  That is far below an output's rounding to 16 bits (up to 2^-8 and
// 2^-11 of a value), so 16-bit outputs take it; a binary32 output (EXACT) would
// show it, so there the values are widened to bfloat16, which holds them exactly, and
// multiplied at that type's rate, a third of the 8-bit one (1320 against 4460
// TFLOP/s of instructions alone), to binary32 sums 1e-8 off.
template <bool EXACT>
__device__ inline f32x4 block_sums(i32x8 a, i32x8 b)
{
    f32x4 c = {0, 0, 0, 0};
    if constexpr (EXACT) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_eight(a, s), widen_eight(b, s), c, 0, 0,
                                                        0);
        return c;
    } else {
        // formats 0 and 0: e4m3 for both operands; no hardware scales
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
    }
}

// The same for 32 x 32 of them: operands of 64 of k each, two to a block.
template <bool EXACT>
__device__ inline f32x16 block_sums32(const i32x8 (&a)[2], const i32x8 (&b)[2])
{
    f32x16 c = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (EXACT) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
                c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_eight(a[h], s),
                                                            widen_eight(b[h], s), c, 0, 0, 0);
        } else {
            c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[h], b[h], c, 0, 0, 0, 0, 0, 0);
        }
    }
    return c;
}

// A lane's 32 bytes of an operand kept in LDS in pieces of 16: the piece at
// `at` and the next one, which is the neighbour by the lowest bit of its place.
__device__ inline i32x8 pieces(const char *base, uint32_t at)
{
    const u32x4 lo = *(const u32x4 *)(base + at), hi = *(const u32x4 *)(base + (at ^ 16u));
    i32x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = (int)lo[i];
        r[4 + i] = (int)hi[i];
    }
    return r;
}

// 16 bytes a lane from base + off to LDS at `to` + 16 * lane (`base` and `to`
// are the same in every lane).  The compiler does not see the load: whoever
// reads the bytes waits for vmcnt first.
__device__ inline void to_lds(const char *base, uint32_t off, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(to), "v"(off), "s"(base)
                 : "memory", "m0");
}

// Four bytes a lane from an address of its own to LDS at `to` + 4 * lane.
__device__ inline void to_lds4(const char *at, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
                 :
                 : "s"(to), "v"(at)
                 : "memory", "m0");
}

// Waits until at most N of the wave's loads are under way.
template <int N>
__device__ inline void wait_loads()
{
    static_assert(N < 64, "the counter has six bits");
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
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

// 16 bytes of an output row with `left` elements to its end.
template <typename T>
__device__ inline void store_row_piece(char *p, u32x4 v, uint32_t left)
{
    if (left >= (uint32_t)kPiece<T>)
        store_piece<false>(p, v);
    else
        store_some<T>(p, v, left);
}

}  // namespace ar
