// fp8_mma.h -- matrix instructions over e4m3 codes (gfx950).  Internal;
// included by the product kernels of the 8-bit floating-point route.
//
// Both operands of v_mfma_f32_16x16x128_f8f6f4 take a lane's row (lane % 16)
// and 32 codes of it; which k the 4 x 32 codes of the lanes of a row are does
// not matter as long as both operands agree.  Here lane group g = lane / 16
// holds bytes 16g..16g+15 and 64+16g..64+16g+15 of a block of 128: two 16-byte
// reads from LDS, whose quarter waves meet different banks (fp8_lds.h).  Result
// register i of a lane is row 4g + i of the first operand, row lane % 16 of the
// second.
//
// The instruction does not add its products in fp32: of eight that it takes
// together (eight consecutive codes of a lane) it drops what is below about
// 2^-13 of the largest (measured: 2^16 + 7.03 gives 2^16, 2^16 + 14.06 does
// not; sums of different eights are fp32).  On normal values that is 1.6e-5 of
// the result's norm, 9e-5 where a block holds an outlier of 30 times the rest:
// 1/100 to 1/20 of what rounding the result to bf16 costs (1.7e-3), and less
// against e4m3's.  An fp32 result would lose eight bits, so there the codes are
// widened to bf16, which is exact, and multiplied by the bf16 instruction at
// half the rate (1e-8 of the norm): EXACT below.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bpg {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

template <bool EXACT> struct Operand;

template <> struct Operand<false> {
    v8i c;
    __device__ __forceinline__ Operand() {}
    __device__ __forceinline__ Operand(v4i lo, v4i hi)
    {
        c = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
};

// eight codes (two registers) as bf16
__device__ __forceinline__ v8b widen(int lo, int hi)
{
    const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const v2b c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const v2b d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return v8b{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <> struct Operand<true> {
    v8b q[4];
    __device__ __forceinline__ Operand() {}
    __device__ __forceinline__ Operand(v4i lo, v4i hi)
    {
        q[0] = widen(lo[0], lo[1]);
        q[1] = widen(lo[2], lo[3]);
        q[2] = widen(hi[0], hi[1]);
        q[3] = widen(hi[2], hi[3]);
    }
};

// the 16 x 16 dot products over one block
__device__ __forceinline__ v4f dot(const Operand<false> &a, const Operand<false> &b)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.c, b.c, v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0,
                                                            0);
}

__device__ __forceinline__ v4f dot(const Operand<true> &a, const Operand<true> &b)
{
    v4f c{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; i++)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.q[i], b.q[i], c, 0, 0, 0);
    return c;
}

// acc += s d: the block's dot products under both scales, the one rounding in
// fp32 that a block costs
__device__ __forceinline__ void add_scaled(v4f &acc, v4f d, float s)
{
#pragma unroll
    for (int i = 0; i < 4; i++)
        acc[i] = __builtin_fmaf(d[i], s, acc[i]);
}

__device__ __forceinline__ uint32_t bf16_bits(float v)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}

// Values of columns n..n+3 of a row whose first is at index i; `vec`: rows of
// y begin at a multiple of four values and y is aligned to four.
__device__ __forceinline__ void store4(void *y, bool bf16, bool vec, int64_t i, int left, v4f v)
{
    if (bf16) {
        uint16_t *p = static_cast<uint16_t *>(y) + i;
        if (vec && left >= 4) {
            const uint32_t lo = bf16_bits(v[0]) | bf16_bits(v[1]) << 16;
            const uint32_t hi = bf16_bits(v[2]) | bf16_bits(v[3]) << 16;
            *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (j < left)
                p[j] = (uint16_t)bf16_bits(v[j]);
        return;
    }
    float *p = static_cast<float *>(y) + i;
    if (vec && left >= 4) {
        *reinterpret_cast<v4f *>(p) = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (j < left)
            p[j] = v[j];
}

inline bool vector_rows(const void *y, int64_t ldy, bool bf16)
{
    return ldy % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & (bf16 ? 7u : 15u)) == 0;
}

} // namespace
} // namespace bpg
