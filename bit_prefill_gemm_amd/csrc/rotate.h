// rotate.h -- the 32-value blocks of activations in registers (gfx950).
// Internal; included by the kernel sources only, which must be compiled with
// -ffp-contract=off.
//
// A quad of lanes owns a block.  The exchanges across lanes (quad_swap,
// cross_stage, cross_quad_stage) are shared by the quantizers (quantize.hip)
// and the norm and the decoding (norm.hip).  load8, rotate_p and quantize_block
// are the quantizers' alone: there lane t holds elements {4t..4t+3} and
// {16+4t..16+4t+3}, while norm.hip's lanes hold 8t..8t+7.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bpg {
namespace {

constexpr int kQuadXor1 = 0xB1;         // DPP quad_perm [1,0,3,2]
constexpr int kQuadXor2 = 0x4E;         // DPP quad_perm [2,3,0,1]

template <int CTRL>
__device__ __forceinline__ float quad_swap(float v)
{
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}

// One butterfly stage across lanes: the lane whose `upper` flag is set holds
// the upper element b and gets partner - own = a - b; the lower lane gets
// own + partner = a + b.  Negation by flipping the sign bit is exact, so
// partner + (-own) is the IEEE a - b.
template <int CTRL>
__device__ __forceinline__ void cross_stage(float (&v)[8], bool upper)
{
    const uint32_t flip = upper ? 0x80000000u : 0u;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        float p = quad_swap<CTRL>(v[i]);
        v[i] = p + __uint_as_float(__float_as_uint(v[i]) ^ flip);
    }
}

// The same across the quads of a span: lane l pairs with l ^ (PATTERN's XOR
// mask); ds_swizzle bit mode, and mask 0x1F, XOR mask in bits 14:10.
template <int PATTERN>
__device__ __forceinline__ void cross_quad_stage(float (&v)[8], bool upper)
{
    const uint32_t flip = upper ? 0x80000000u : 0u;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float p = __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v[i]), PATTERN));
        v[i] = p + __uint_as_float(__float_as_uint(v[i]) ^ flip);
    }
}
constexpr int kSwzXor4 = (4 << 10) | 0x1F;
constexpr int kSwzXor8 = (8 << 10) | 0x1F;

__device__ __forceinline__ void load8(const float *src, int t, float (&v)[8])
{
    float4 lo = *reinterpret_cast<const float4 *>(src + 4 * t);
    float4 hi = *reinterpret_cast<const float4 *>(src + 16 + 4 * t);
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
}

__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }

__device__ __forceinline__ void load8(const uint16_t *src, int t, float (&v)[8])
{
    uint2 lo = *reinterpret_cast<const uint2 *>(src + 4 * t);
    uint2 hi = *reinterpret_cast<const uint2 *>(src + 16 + 4 * t);
    v[0] = bf16_to_f32(lo.x & 0xFFFFu); v[1] = bf16_to_f32(lo.x >> 16);
    v[2] = bf16_to_f32(lo.y & 0xFFFFu); v[3] = bf16_to_f32(lo.y >> 16);
    v[4] = bf16_to_f32(hi.x & 0xFFFFu); v[5] = bf16_to_f32(hi.x >> 16);
    v[6] = bf16_to_f32(hi.y & 0xFFFFu); v[7] = bf16_to_f32(hi.y >> 16);
}

// The rotation of one block (span ROT = 0: none, 32, 64, 128): lane t holds
// elements {4t..4t+3} and {16+4t..16+4t+3} (v[0..3], v[4..7]); h = 1, 2
// inside the lane, h = 4 with lane t^1, h = 8 with t^2 (the lane with the
// bit clear is lower), h = 16 inside the lane (v[i] with v[i+4]), h = 32, 64
// with the adjacent quads of a longer span; then times fp32(1/sqrt(ROT)).
template <int ROT>
__device__ __forceinline__ void rotate_p(float (&v)[8], int t, int lane)
{
    if constexpr (ROT != 0) {
#pragma unroll
        for (int base = 0; base < 8; base += 4) {
            const float a0 = v[base], a1 = v[base + 1], a2 = v[base + 2], a3 = v[base + 3];
            v[base] = a0 + a1;
            v[base + 1] = a0 - a1;
            v[base + 2] = a2 + a3;
            v[base + 3] = a2 - a3;
        }
#pragma unroll
        for (int base = 0; base < 8; base += 4) {
            const float a0 = v[base], a1 = v[base + 1], a2 = v[base + 2], a3 = v[base + 3];
            v[base] = a0 + a2;
            v[base + 2] = a0 - a2;
            v[base + 1] = a1 + a3;
            v[base + 3] = a1 - a3;
        }
        cross_stage<kQuadXor1>(v, (t & 1) != 0);
        cross_stage<kQuadXor2>(v, (t & 2) != 0);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float a = v[i], c = v[i + 4];
            v[i] = a + c;
            v[i + 4] = a - c;
        }
        if constexpr (ROT >= 64)
            cross_quad_stage<kSwzXor4>(v, (lane & 4) != 0);
        if constexpr (ROT >= 128)
            cross_quad_stage<kSwzXor8>(v, (lane & 8) != 0);
        const float c = ROT == 64 ? 0.125f
                                  : __uint_as_float(ROT == 128 ? 0x3DB504F3u : 0x3E3504F3u);
#pragma unroll
        for (int i = 0; i < 8; i++)
            v[i] = v[i] * c;
    }
}

// Rotate and quantize one block whose 8 values (this lane's share) are in v.
// rot: 0 (no rotation), 32, 64 or 128 (span of the rotation).
template <int BITS>
__device__ __forceinline__ void quantize_block(float (&v)[8], int t, int rot, int64_t row,
                                               int64_t b, int64_t k, int64_t nb,
                                               uint8_t *__restrict__ codes,
                                               float *__restrict__ scales)
{
    if (rot) {
        // h = 1: pairs (4t, 4t+1), (4t+2, 4t+3) and the same in the upper half
#pragma unroll
        for (int base = 0; base < 8; base += 4) {
            float a0 = v[base], a1 = v[base + 1], a2 = v[base + 2], a3 = v[base + 3];
            v[base] = a0 + a1; v[base + 1] = a0 - a1;
            v[base + 2] = a2 + a3; v[base + 3] = a2 - a3;
        }
        // h = 2: pairs (4t, 4t+2), (4t+1, 4t+3)
#pragma unroll
        for (int base = 0; base < 8; base += 4) {
            float a0 = v[base], a1 = v[base + 1], a2 = v[base + 2], a3 = v[base + 3];
            v[base] = a0 + a2; v[base + 2] = a0 - a2;
            v[base + 1] = a1 + a3; v[base + 3] = a1 - a3;
        }
        // h = 4: element 4t+i pairs with 4(t^1)+i; the even lane is lower
        cross_stage<kQuadXor1>(v, (t & 1) != 0);
        // h = 8: lane t pairs with t^2; lanes 0,1 are lower
        cross_stage<kQuadXor2>(v, (t & 2) != 0);
        // h = 16: element j (v[i]) pairs with j+16 (v[i+4]) in the same lane
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float a = v[i], c = v[i + 4];
            v[i] = a + c;
            v[i + 4] = a - c;
        }
        // h = 32, 64: the blocks of a longer span, in adjacent quads
        const int lane = threadIdx.x & 63;
        if (rot >= 64)
            cross_quad_stage<kSwzXor4>(v, (lane & 4) != 0);
        if (rot >= 128)
            cross_quad_stage<kSwzXor8>(v, (lane & 8) != 0);
        // fp32 nearest to 1/sqrt(rot): 1/sqrt(32), 1/8 and half of 1/sqrt(32)
        const float c = rot == 64 ? 0.125f
                                  : __uint_as_float(rot == 128 ? 0x3DB504F3u : 0x3E3504F3u);
#pragma unroll
        for (int i = 0; i < 8; i++)
            v[i] = v[i] * c;
    }

    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++)
        amax = fmaxf(amax, fabsf(v[i]));
    amax = fmaxf(amax, quad_swap<kQuadXor1>(amax));
    amax = fmaxf(amax, quad_swap<kQuadXor2>(amax));

    constexpr float kQmax = BITS == 4 ? 7.0f : 127.0f;
    constexpr float kQmin = BITS == 4 ? -8.0f : -127.0f;
    // a scale of 0 (an all-zero block, or amax / kQmax underflowing) gives
    // codes 0: every code of such a block dequantizes to 0
    const float d = amax / kQmax;
    // q = rint(v / d) with the IEEE quotient.  The quotient is first taken as
    // v * rcp(d): its error is below |v/d| * 3 * 2^-24 <= 2.3e-5 (|v/d| <= 127),
    // so wherever that product lies at least 1e-4 from a half-integer it
    // rounds to the same integer as the correctly rounded quotient.  Within
    // that band (rare) and for tiny scales the IEEE division decides.
    const bool fast = d >= 0x1p-100f;
    const float rd = __builtin_amdgcn_rcpf(d);
    int q[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        float r = 0.0f;
        if (d != 0.0f) {
            r = v[i] * rd;
            if (!fast || fabsf(fabsf(r - rintf(r)) - 0.5f) < 1e-4f)
                r = v[i] / d;
            r = rintf(r);
        }
        r = fminf(fmaxf(r, kQmin), kQmax);
        q[i] = (int)r;
    }

    if (BITS == 4) {
        // byte 4t+i = code(4t+i) low nibble | code(16+4t+i) high nibble
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 4; i++)
            word |= (uint32_t)((q[i] & 0xF) | ((q[i + 4] & 0xF) << 4)) << (8 * i);
        *reinterpret_cast<uint32_t *>(codes + row * (k / 2) + b * 16 + 4 * t) = word;
    } else {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            lo |= (uint32_t)(q[i] & 0xFF) << (8 * i);
            hi |= (uint32_t)(q[i + 4] & 0xFF) << (8 * i);
        }
        uint8_t *dst = codes + row * k + b * 32;
        *reinterpret_cast<uint32_t *>(dst + 4 * t) = lo;
        *reinterpret_cast<uint32_t *>(dst + 16 + 4 * t) = hi;
    }
    if (t == 0)
        scales[row * nb + b] = d;
}

} // namespace
} // namespace bpg
