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
// than k 2^-53 relative, so s depends on the order of the sum only where the
// exact value lies that close to a rounding border of fp32: at most k rows in
// 2^29 by that bound, some k^(1/2) in 2^29 with the usual cancelling of
// roundings.  The codes of all others are a plain evaluation's, bit for bit.
// The fp64 sum is a conversion and an FMA per value.
//
// A row belongs to a workgroup, a 32-block to a quad of lanes (lane t holds
// elements 8t..8t+7: one 16-byte load per 8 bf16 values), R blocks per quad
// between the sum and the codes: in registers up to R = 4 (32768 values), while
// R = 8 spills 96 to 144 of them.  What bounds it is memory (two reads, a write
// and the codes) as long as loads are always in flight, so the grid holds about
// the workgroups that fit the chip (see launch_norm_rounds); each walks several
// rows and, up to R = 2 (bf16 x and stream 3), issues the next row's loads
// before it reduces the current one.  From R = 4 on a block's loads also wait
// for the store of h before them, as h may be the residual.  A row of fewer
// than 16 blocks leaves lanes of its wave idle.
// Measured in graph replays (8-bit codes): 8192 x 5120 with H128, bf16 x and
// stream, 66 us for 299 MB (4.5 TB/s; a large copy reaches 5.07), 101 us before
// with a workgroup per row, 8-byte loads and a check per value; bf16 x into an
// fp32 stream 106 us (4.4 TB/s), both fp32 117 (4.7), fp32 without a residual
// 68 (3.2).  Long bf16 rows: 2000 x 28672 115 us (3.6 TB/s), 500 x 65536 122
// (1.9); narrow ones: 100000 x 256 49 us (3.7), 100000 x 64 43 (1.1).  With
// 4-bit codes 512 x 5120 takes 7.0 us (354 vector instructions per wave and
// row), one row 3.7 us (a launch is 1.9).
//
// This file must be compiled with -ffp-contract=off (see quantize.hip).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "between.h"
#include "rotate.h"

namespace bpg {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
// 16 bytes of rows that are 8-byte aligned (bf16, leading dimension a multiple of 4)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(8)));

// two fp32 -> bf16 bits, round to nearest even (NaN stays NaN)
__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const f32x2 f = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

// The lane's 8 values of a block as they sit in memory, T = float or uint16_t
// (bf16 bits).
template <typename T> struct Raw;

template <> struct Raw<uint16_t> {
    u32x4 w;
    __device__ __forceinline__ void load(const uint16_t *p) { w = *reinterpret_cast<const u32x4 *>(p); }
    __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<u32x4 *>(p) = w; }
    __device__ __forceinline__ float at(int i) const
    {
        return __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ void round(const float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; i++)
            w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    }
};

template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void store(float *p) const
    {
        *reinterpret_cast<float4 *>(p) = a;
        *reinterpret_cast<float4 *>(p + 4) = b;
    }
    __device__ __forceinline__ float at(int i) const
    {
        return i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w
             : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w;
    }
    __device__ __forceinline__ void round(const float (&v)[8])
    {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
};

constexpr int kRowRor8 = 0x128; // DPP row_ror:8: lane ^ 8 inside 16 lanes

// The rotation of quantize.hip with lane t of a quad holding elements
// 8t..8t+7: h = 1, 2, 4 inside the lane, 8 and 16 inside the quad (the lane
// with the bit clear is lower), 32 and 64 across the quads of a longer span.
template <int ROT>
__device__ __forceinline__ void rotate_lanes(float (&v)[8], int lane)
{
#pragma unroll
    for (int h = 1; h < 8; h *= 2)
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (!(i & h)) {
                const float a = v[i], b = v[i + h];
                v[i] = a + b;
                v[i + h] = a - b;
            }
    cross_stage<kQuadXor1>(v, (lane & 1) != 0);
    cross_stage<kQuadXor2>(v, (lane & 2) != 0);
    if constexpr (ROT >= 64)
        cross_quad_stage<kSwzXor4>(v, (lane & 4) != 0);
    if constexpr (ROT >= 128)
        cross_stage<kRowRor8>(v, (lane & 8) != 0);
    const float c = ROT == 64 ? 0.125f : __uint_as_float(ROT == 128 ? 0x3DB504F3u : 0x3E3504F3u);
#pragma unroll
    for (int i = 0; i < 8; i++)
        v[i] = v[i] * c;
}

template <int R>
__device__ __forceinline__ void rotate_rounds(float (&v)[R][8], int rot, int lane)
{
    if (rot == 32) {
#pragma unroll
        for (int r = 0; r < R; r++)
            rotate_lanes<32>(v[r], lane);
    } else if (rot == 64) {
#pragma unroll
        for (int r = 0; r < R; r++)
            rotate_lanes<64>(v[r], lane);
    } else if (rot == 128) {
#pragma unroll
        for (int r = 0; r < R; r++)
            rotate_lanes<128>(v[r], lane);
    }
}

// low bytes of a, b, c, d, first to last
__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d)
{
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(d), __float_as_uint(c), 0x04000c0cu);
    return lo | hi;
}

// Scale and codes of one block per quad, as quantize.hip defines them; the
// lane's part of the codes: 8 bytes, for 4-bit codes in lanes t = 0, 1 only
// (bytes 8t..8t+7 of the block).
template <int BITS>
__device__ __forceinline__ uint2 quantize_lanes(const float (&v)[8], float &d)
{
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++)
        amax = fmaxf(amax, fabsf(v[i]));
    amax = fmaxf(amax, quad_swap<kQuadXor1>(amax));
    amax = fmaxf(amax, quad_swap<kQuadXor2>(amax));
    constexpr float kQmax = BITS == 4 ? 7.0f : 127.0f;
    constexpr float kQmin = BITS == 4 ? -8.0f : -127.0f;
    d = amax / kQmax;
    // rint(v / d), taken as v * rcp(d) with one check per wave whether any
    // value lies within 1e-4 of a rounding midpoint (the product is within
    // 2.3e-5 of the quotient, |v / d| <= 127); then, or where d is too small for
    // the reciprocal, the IEEE quotient decides.  Adding 1.5 2^23 rounds to the
    // nearest integer (ties to even) and leaves it in the low bits.
    constexpr float kMagic = 12582912.0f;
    const float rd = d != 0.0f ? __builtin_amdgcn_rcpf(d) : 0.0f;
    float y[8];
    float off = d != 0.0f && !(d >= 0x1p-100f) ? 1.0f : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float q = v[i] * rd;
        y[i] = q + kMagic;
        off = fmaxf(off, fabsf(q - (y[i] - kMagic)));
    }
    if (__builtin_amdgcn_ballot_w64(off > 0.4999f) != 0) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float q = d != 0.0f ? v[i] / d : 0.0f;
            y[i] = fminf(fmaxf(q, kQmin), kQmax) + kMagic;
        }
    }
    uint2 w = make_uint2(low_bytes(y[0], y[1], y[2], y[3]), low_bytes(y[4], y[5], y[6], y[7]));
    if constexpr (BITS == 4) {
        // byte j = code j | code j + 16 << 4: the upper half of the block is with lane t ^ 2
        w.x &= 0x0F0F0F0Fu;
        w.y &= 0x0F0F0F0Fu;
        w.x |= (uint32_t)__builtin_amdgcn_mov_dpp((int)w.x, kQuadXor2, 0xF, 0xF, true) << 4;
        w.y |= (uint32_t)__builtin_amdgcn_mov_dpp((int)w.y, kQuadXor2, 0xF, 0xF, true) << 4;
    }
    return w;
}

// Sum over a row of 16 lanes, in lane 15 (row_shr steps), then over the rows
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

__device__ __forceinline__ double row16_sum(double v)
{
    v += dpp_f64<0x111, 0xF>(v);
    v += dpp_f64<0x112, 0xF>(v);
    v += dpp_f64<0x114, 0xF>(v);
    v += dpp_f64<0x118, 0xF>(v);
    return v;
}

__device__ __forceinline__ double lane_of(double v, int lane)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// 1 / sqrt(a), a > 0 normal: the hardware's estimate (2^-24) and one step of
// third order, within a few units of the 53rd bit
__device__ __forceinline__ double rsqrt_f64(double a)
{
    const double y = __builtin_amdgcn_rsq(a);
    const double e = __builtin_fma(-a * y, y, 1.0);
    return __builtin_fma(y * e, __builtin_fma(0.375, e, 0.5), y);
}

// Tx: type of x, Tr: type of the residual stream (float, or uint16_t = bf16
// bits); without a residual the stream is x.
template <typename Tx, typename Tr, int BITS, int R>
__global__ __launch_bounds__(1024) void norm_quantize_kernel(NormProblem p)
{
    // two buffers: a wave may be one row ahead of the slowest reader
    __shared__ double partial[2][16];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int t = lane & 3;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x >> 6;
    const int quads = blockDim.x >> 2, qd = tid >> 2;
    const int nb = (int)(p.k / 32); // the host limits k to 2^16
    const Tx *const x = static_cast<const Tx *>(p.x);
    const Tr *const res = static_cast<const Tr *>(p.residual);
    if (waves > 1 && tid < 32)
        partial[tid >> 4][tid & 15] = 0.0; // the waves that do not exist

    // The lane's part of block qd + r quads; quads past the row's end read its
    // first block instead and store nothing.  (Where h is the residual another
    // wave may store that block meanwhile; these quads' values reach nothing
    // but the wave's vote in quantize_lanes, whose two ways give the same codes.)
    int at[R];
    bool live[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int b = qd + r * quads;
        live[r] = b < nb;
        at[r] = (live[r] ? b : 0) * 32 + 8 * t;
    }
    // as far as the registers go, the next row's values are loaded a row ahead,
    // or a row's values all before the first is used
    constexpr bool ahead = R <= 2 || (R == 3 && sizeof(Tx) + sizeof(Tr) == 4);
    constexpr bool whole = R <= 3;
    Raw<Tx> rx[whole ? R : 1];
    Raw<Tr> rr[whole ? R : 1];
    auto load_row = [&](int64_t row) {
#pragma unroll
        for (int r = 0; r < R; r++)
            rx[r].load(x + row * p.ldx + at[r]);
        if (res) {
#pragma unroll
            for (int r = 0; r < R; r++)
                rr[r].load(res + row * p.ldr + at[r]);
        }
    };
    auto load_weight = [&](int r, float (&g)[8]) {
        if (!p.weight) {
#pragma unroll
            for (int i = 0; i < 8; i++)
                g[i] = 1.0f;
        } else if (p.weight_bf16) {
            Raw<uint16_t> w;
            w.load(static_cast<const uint16_t *>(p.weight) + at[r]);
#pragma unroll
            for (int i = 0; i < 8; i++)
                g[i] = w.at(i);
        } else {
            Raw<float> w;
            w.load(static_cast<const float *>(p.weight) + at[r]);
#pragma unroll
            for (int i = 0; i < 8; i++)
                g[i] = w.at(i);
        }
    };
    // and the weight stays in registers for all rows
    constexpr bool keep = R <= 2;
    float g[keep ? R : 1][8];
    if constexpr (ahead)
        load_row(blockIdx.x);
    if constexpr (keep) {
#pragma unroll
        for (int r = 0; r < R; r++)
            load_weight(r, g[r]);
    }
    if (waves > 1)
        __syncthreads(); // the zeros

    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x, parity ^= 1) {
        float v[R][8];
        double ss = 0.0;
        if constexpr (whole && !ahead)
            load_row(row);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const int q = whole ? r : 0;
            if constexpr (!whole) {
                rx[0].load(x + row * p.ldx + at[r]);
                if (res)
                    rr[0].load(res + row * p.ldr + at[r]);
            }
            if (res) {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    v[r][i] = rx[q].at(i) + rr[q].at(i);
                Raw<Tr> h;
                h.round(v[r]);
                if (p.h && live[r])
                    h.store(static_cast<Tr *>(p.h) + row * p.ldh + at[r]);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    v[r][i] = h.at(i);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    v[r][i] = rx[q].at(i);
            }
            double sb = 0.0;
#pragma unroll
            for (int i = 0; i < 8; i++)
                sb = __builtin_fma((double)v[r][i], (double)v[r][i], sb);
            ss += live[r] ? sb : 0.0;
        }
        if constexpr (ahead) {
            if (row + gridDim.x < p.m)
                load_row(row + gridDim.x);
        }

        // the sum: lanes, waves, each in a fixed order
        ss = row16_sum(ss);
        ss += dpp_f64<0x142, 0xA>(ss);
        ss += dpp_f64<0x143, 0xC>(ss);
        if (waves > 1) {
            if (lane == 63)
                partial[parity][wave] = ss;
            __syncthreads();
            ss = lane_of(row16_sum(partial[parity][lane & 15]), 15);
        } else {
            ss = lane_of(ss, 63);
        }
        const float s = (float)rsqrt_f64(__builtin_fma(ss, p.inv_k, (double)p.eps));

#pragma unroll
        for (int r = 0; r < R; r++) {
            if constexpr (!keep)
                load_weight(r, g[0]);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                v[r][i] = v[r][i] * s;
                v[r][i] = v[r][i] * g[keep ? r : 0][i];
            }
        }
        rotate_rounds(v, p.rot, lane);
#pragma unroll
        for (int r = 0; r < R; r++) {
            float d;
            const uint2 w = quantize_lanes<BITS>(v[r], d);
            if (!live[r])
                continue;
            const int64_t b = row * nb + qd + r * quads;
            uint8_t *const codes = static_cast<uint8_t *>(p.codes);
            if constexpr (BITS == 4) {
                if (t < 2)
                    *reinterpret_cast<uint2 *>(codes + b * 16 + 8 * t) = w;
            } else {
                *reinterpret_cast<uint2 *>(codes + b * 32 + 8 * t) = w;
            }
            if (t == 0)
                p.scales[b] = d;
        }
    }
}

// One quad per block, grid-stride over the blocks: v = code * scale, rotated
// back (the Sylvester matrix is symmetric and, with its factor, its own
// inverse), rounded once to the output's type.  A span never straddles the
// end of the blocks, so its quads walk together.
// Bound by memory: 8192 x 5120, 8-bit codes to bf16, 24 us for 131 MB
// (5.4 TB/s).
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
            // bytes 8 (t & 1) .. + 7 of the block: elements 8t.. in the low nibbles for t < 2,
            // in the high ones for t = 2, 3
            const uint2 c = *reinterpret_cast<const uint2 *>(codes + blk * 16 + 8 * (t & 1));
            const int up = t < 2 ? 4 : 0;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[0][i] = (float)((int)((c.x << up) << (24 - 8 * i)) >> 28) * d;
                v[0][i + 4] = (float)((int)((c.y << up) << (24 - 8 * i)) >> 28) * d;
            }
        } else {
            const uint2 c = *reinterpret_cast<const uint2 *>(codes + blk * 32 + 8 * t);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[0][i] = (float)((int)(c.x << (24 - 8 * i)) >> 24) * d;
                v[0][i + 4] = (float)((int)(c.y << (24 - 8 * i)) >> 24) * d;
            }
        }
        rotate_rounds(v, rot, lane);
        Raw<Ty> out;
        out.round(v[0]);
        out.store(y + row * ldy + b * 32 + 8 * t);
    }
}

constexpr int kCUs = 256;

template <typename Tx, typename Tr, int BITS>
hipError_t launch_norm_rounds(const NormProblem &p, hipStream_t stream)
{
    const int nb = (int)(p.k / 32);
    // per_cu: waves that a CU holds of the kernel by its registers.  The grid is
    // no more workgroups than fit at once; only of R = 2 with an fp32 x or stream
    // (100 to 104 registers: 16 waves, not the 20 that bf16 with 89 has) it may
    // be more, four where three fit at K = 5120: the rest waits for a place.
    auto launch = [&](auto kernel, int rounds, int per_cu) {
        const int waves = (nb + 16 * rounds - 1) / (16 * rounds);
        const int64_t most = (int64_t)kCUs * (per_cu / waves > 0 ? per_cu / waves : 1);
        const dim3 grid((unsigned)(p.m < most ? p.m : most));
        kernel<<<grid, dim3((unsigned)(64 * waves)), 0, stream>>>(p);
    };
    // One block per quad while every row has a workgroup at once (the shortest
    // chain from the loads to the stores); with more rows than that, two (half
    // the reductions and barriers a row), unless more lanes would idle.  A row of
    // fewer than 16 blocks takes a wave all the same.
    const int w1 = (nb + 15) / 16, w2 = (nb + 31) / 32;
    const bool once = w1 <= 16 && p.m <= (int64_t)kCUs * (32 / w1);
    if (w1 <= 16 && (once || 2 * w2 > w1))
        launch(norm_quantize_kernel<Tx, Tr, BITS, 1>, 1, 32);
    else if (nb <= 512)
        launch(norm_quantize_kernel<Tx, Tr, BITS, 2>, 2, 20);
    else if (nb <= 768)
        launch(norm_quantize_kernel<Tx, Tr, BITS, 3>, 3, 16);
    else if (nb <= 1024)
        launch(norm_quantize_kernel<Tx, Tr, BITS, 4>, 4, 16);
    else
        launch(norm_quantize_kernel<Tx, Tr, BITS, 8>, 8, 16);
    return hipGetLastError();
}

template <typename Tx, typename Tr>
hipError_t launch_norm_types(const NormProblem &p, hipStream_t stream)
{
    return p.act_bits == 4 ? launch_norm_rounds<Tx, Tr, 4>(p, stream)
                           : launch_norm_rounds<Tx, Tr, 8>(p, stream);
}

} // namespace

hipError_t launch_norm_quantize(const NormProblem &problem, hipStream_t stream)
{
    if (problem.m == 0)
        return hipSuccess;
    NormProblem p = problem;
    p.inv_k = 1.0 / (double)p.k;
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
