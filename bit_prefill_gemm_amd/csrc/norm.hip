// norm.hip -- RMSNorm with the residual's addition feeding the quantizer, and
// the decoding of codes (gfx950).
//
// "509 tokens a second of prompt: the Hadamard route ships", section "The
// rotation": the rotation runs inside the step that quantizes activations.
// What is quantized is, in a pre-norm block, the root-mean-square norm of the
// residual stream; this kernel adds the block's output to the stream, norms,
// rotates and quantizes a row in one pass, so the row is read once and the
// normed values never reach memory:
//   h_i = x_i + r_i          one fp32 addition, rounded to the stream's type;
//                            the norm is that of the stored value
//   s   = 1 / sqrt(sum h_i^2 / k + eps)   in fp64, rounded to fp32 once
//   v_i = (h_i * s) * g_i    two fp32 roundings
// then the rotation and quantization of quantize.hip on v, step by step.
// The squares of fp32 values are exact in fp64 and their sum is off by less
// than k 2^-53, so s does not depend on the order of the sum (but for about
// one row in 10^8, next to a rounding border) and the codes are those of a
// plain evaluation, bit for bit.  The fp64 sum is one instruction per value.
//
// One workgroup per row (grid-stride), a quad of lanes per 32-block, R blocks
// per quad held in registers between the sum and the codes.
//
// This file must be compiled with -ffp-contract=off (see quantize.hip).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "rotate.h"

namespace bpg {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// two fp32 -> bf16 bits, round to nearest even (NaN stays NaN)
__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const f32x2 f = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

// store the lane's 8 values of a block and return what was stored
__device__ __forceinline__ void store8(float *dst, int t, float (&v)[8])
{
    *reinterpret_cast<float4 *>(dst + 4 * t) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(dst + 16 + 4 * t) = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ void store8(uint16_t *dst, int t, float (&v)[8])
{
    const uint2 lo = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    const uint2 hi = make_uint2(bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
    *reinterpret_cast<uint2 *>(dst + 4 * t) = lo;
    *reinterpret_cast<uint2 *>(dst + 16 + 4 * t) = hi;
}

__device__ __forceinline__ void round_to(const float *, float (&)[8]) {}

__device__ __forceinline__ void round_to(const uint16_t *, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint32_t p = bf16_pair(v[i], v[i + 1]);
        v[i] = bf16_to_f32(p & 0xFFFFu);
        v[i + 1] = bf16_to_f32(p >> 16);
    }
}

template <int R>
__device__ __forceinline__ void rotate_rounds(float (&v)[R][8], int rot, int t, int lane)
{
    if (rot == 32) {
#pragma unroll
        for (int r = 0; r < R; r++)
            rotate_p<32>(v[r], t, lane);
    } else if (rot == 64) {
#pragma unroll
        for (int r = 0; r < R; r++)
            rotate_p<64>(v[r], t, lane);
    } else if (rot == 128) {
#pragma unroll
        for (int r = 0; r < R; r++)
            rotate_p<128>(v[r], t, lane);
    }
}

// Tx: type of x, Tr: type of the residual stream (float, or uint16_t = bf16
// bits); without a residual the stream is x.
template <typename Tx, typename Tr, int BITS, int R>
__global__ __launch_bounds__(1024) void norm_quantize_kernel(NormProblem p)
{
    __shared__ double partial[2][16];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int t = lane & 3;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x >> 6;
    const int quads = blockDim.x >> 2, qd = tid >> 2;
    const int nb = (int)(p.k / 32); // the host limits k to 2^16

    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x, parity ^= 1) {
        const Tx *x = static_cast<const Tx *>(p.x) + row * p.ldx;
        const Tr *res = static_cast<const Tr *>(p.residual) + row * p.ldr;
        float v[R][8], g[R][8];
#pragma unroll
        for (int r = 0; r < R; r++) {
            const int b = qd + r * quads;
#pragma unroll
            for (int i = 0; i < 8; i++)
                v[r][i] = 0.0f;
            if (b < nb)
                load8(x + b * 32, t, v[r]);
        }
        if (p.residual) {
            float a[R][8];
#pragma unroll
            for (int r = 0; r < R; r++) {
                const int b = qd + r * quads;
#pragma unroll
                for (int i = 0; i < 8; i++)
                    a[r][i] = 0.0f;
                if (b < nb)
                    load8(res + b * 32, t, a[r]);
            }
#pragma unroll
            for (int r = 0; r < R; r++) {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    v[r][i] = v[r][i] + a[r][i];
                round_to(res, v[r]);
            }
            if (p.h) {
                Tr *h = static_cast<Tr *>(p.h) + row * p.ldh;
#pragma unroll
                for (int r = 0; r < R; r++) {
                    const int b = qd + r * quads;
                    if (b < nb)
                        store8(h + b * 32, t, v[r]);
                }
            }
        }
        // the norm's weight (1 where there is none)
#pragma unroll
        for (int r = 0; r < R; r++) {
            const int b = qd + r * quads;
#pragma unroll
            for (int i = 0; i < 8; i++)
                g[r][i] = 1.0f;
            if (p.weight && b < nb) {
                if (p.weight_bf16)
                    load8(static_cast<const uint16_t *>(p.weight) + b * 32, t, g[r]);
                else
                    load8(static_cast<const float *>(p.weight) + b * 32, t, g[r]);
            }
        }

        // the sum of squares: lane, wave, workgroup, each in a fixed order
        double ss = 0.0;
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int i = 0; i < 8; i++)
                ss = __builtin_fma((double)v[r][i], (double)v[r][i], ss);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
            ss += __shfl_xor(ss, d);
        if (waves > 1) {
            // (two buffers: a wave may be one row ahead of the slowest reader)
            if (lane == 0)
                partial[parity][wave] = ss;
            __syncthreads();
            ss = 0.0;
            for (int w = 0; w < waves; w++)
                ss += partial[parity][w];
        }
        const float s = (float)(1.0 / sqrt(ss / (double)p.k + (double)p.eps));

#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                v[r][i] = v[r][i] * s;
                v[r][i] = v[r][i] * g[r][i];
            }
        rotate_rounds(v, p.rot, t, lane);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const int b = qd + r * quads;
            if (b < nb)
                quantize_block<BITS>(v[r], t, 0, row, b, p.k, nb, static_cast<uint8_t *>(p.codes),
                                     p.scales);
        }
    }
}

// One quad per block, grid-stride over the blocks: v = code * scale, rotated
// back (the Sylvester matrix is symmetric and, with its factor, its own
// inverse), rounded once to the output's type.  A span never straddles the
// end of the blocks, so its quads walk together.
template <typename Ty, int BITS>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint8_t *__restrict__ codes,
                                                         const float *__restrict__ scales,
                                                         int64_t k, int rot, int64_t nblk,
                                                         Ty *__restrict__ y, int64_t ldy)
{
    const int t = threadIdx.x & 3, lane = threadIdx.x & 63;
    const int64_t nb = k / 32;
    const int64_t stride = (int64_t)gridDim.x * 64;
    for (int64_t blk = (int64_t)blockIdx.x * 64 + (threadIdx.x >> 2); blk < nblk; blk += stride) {
        const int64_t row = blk / nb, b = blk - row * nb;
        const float d = scales[blk];
        float v[1][8];
        if constexpr (BITS == 4) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + blk * 16 + 4 * t);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[0][i] = (float)((int)(w << (28 - 8 * i)) >> 28) * d;
                v[0][i + 4] = (float)((int)(w << (24 - 8 * i)) >> 28) * d;
            }
        } else {
            const uint32_t lo = *reinterpret_cast<const uint32_t *>(codes + blk * 32 + 4 * t);
            const uint32_t hi = *reinterpret_cast<const uint32_t *>(codes + blk * 32 + 16 + 4 * t);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[0][i] = (float)((int)(lo << (24 - 8 * i)) >> 24) * d;
                v[0][i + 4] = (float)((int)(hi << (24 - 8 * i)) >> 24) * d;
            }
        }
        rotate_rounds(v, rot, t, lane);
        store8(y + row * ldy + b * 32, t, v[0]);
    }
}

template <typename Tx, typename Tr, int BITS>
hipError_t launch_norm_rounds(const NormProblem &p, hipStream_t stream)
{
    const int nb = (int)(p.k / 32);
    const int64_t rows = p.m < ((int64_t)1 << 20) ? p.m : (int64_t)1 << 20;
    const dim3 grid((unsigned)rows);
    auto threads = [&](int rounds) { return dim3((unsigned)(64 * ((nb + 16 * rounds - 1) / (16 * rounds)))); };
    if (nb <= 256)
        norm_quantize_kernel<Tx, Tr, BITS, 1><<<grid, threads(1), 0, stream>>>(p);
    else if (nb <= 512)
        norm_quantize_kernel<Tx, Tr, BITS, 2><<<grid, threads(2), 0, stream>>>(p);
    else if (nb <= 1024)
        norm_quantize_kernel<Tx, Tr, BITS, 4><<<grid, threads(4), 0, stream>>>(p);
    else
        norm_quantize_kernel<Tx, Tr, BITS, 8><<<grid, threads(8), 0, stream>>>(p);
    return hipGetLastError();
}

template <typename Tx, typename Tr>
hipError_t launch_norm_types(const NormProblem &p, hipStream_t stream)
{
    return p.act_bits == 4 ? launch_norm_rounds<Tx, Tr, 4>(p, stream)
                           : launch_norm_rounds<Tx, Tr, 8>(p, stream);
}

} // namespace

hipError_t launch_norm_quantize(const NormProblem &p, hipStream_t stream)
{
    if (p.m == 0)
        return hipSuccess;
    if (p.x_bf16)
        return p.residual_bf16 ? launch_norm_types<uint16_t, uint16_t>(p, stream)
                               : launch_norm_types<uint16_t, float>(p, stream);
    return p.residual_bf16 ? launch_norm_types<float, uint16_t>(p, stream)
                           : launch_norm_types<float, float>(p, stream);
}

hipError_t launch_dequantize(const void *codes, const float *scales, int act_bits, int rot,
                             int64_t m, int64_t k, void *y, bool y_bf16, int64_t ldy,
                             hipStream_t stream)
{
    const int64_t nblk = m * (k / 32);
    if (nblk == 0)
        return hipSuccess;
    const int64_t needed = (nblk + 63) / 64;
    const dim3 grid((unsigned)(needed < 8192 ? needed : 8192));
    const uint8_t *c = static_cast<const uint8_t *>(codes);
    if (y_bf16 && act_bits == 4)
        dequantize_kernel<uint16_t, 4><<<grid, 256, 0, stream>>>(c, scales, k, rot, nblk, static_cast<uint16_t *>(y), ldy);
    else if (y_bf16)
        dequantize_kernel<uint16_t, 8><<<grid, 256, 0, stream>>>(c, scales, k, rot, nblk, static_cast<uint16_t *>(y), ldy);
    else if (act_bits == 4)
        dequantize_kernel<float, 4><<<grid, 256, 0, stream>>>(c, scales, k, rot, nblk, static_cast<float *>(y), ldy);
    else
        dequantize_kernel<float, 8><<<grid, 256, 0, stream>>>(c, scales, k, rot, nblk, static_cast<float *>(y), ldy);
    return hipGetLastError();
}

} // namespace bpg
