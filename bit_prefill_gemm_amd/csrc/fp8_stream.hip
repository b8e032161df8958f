// fp8_stream.hip -- products of e4m3 codes with few rows (gfx950).
//
//   y[m][n] = sum over blocks b of sx[m][b] sw[n / 128][b] * dot(x block, w block)
//
// and, gated, act(y_gate) * y_up.  All that is read once is w, so this is a
// stream of it: a workgroup makes 16 columns (16 of each matrix, gated) of all
// rows, and each of its eight waves takes a part of K, whose blocks it brings to
// a ring of its own in LDS by direct loads, two blocks on the way.  No wave waits
// for another before the end, where their sums are added in wave order.
//
// Bound by memory where there are many columns (rows x columns x K 1 x 17408 x
// 5120, 89 MB: 20.5 us, 4.4 TB/s; gated to codes 44 us, 4.0 TB/s) and by the time
// to fill and drain where there are few (1 x 5120 x 5120: 8.8 us, 3.0 TB/s; 1 x
// 1024 x 5120: 5.1 us).  With the weights in the last cache these take 16.6, 35.5,
// 5.5 and 3.8 us.  Blocks of K dealt to the waves in turn, straight to registers,
// took a microsecond more for the first and 14.2 instead of 8.7 for 16 x 5120 x
// 5120, where a load of x or w in the operands' shape keeps the load unit for 47
// clocks (fp8_lds.h).
#include "fp8.h"

#include "epilogue.h"
#include "fp8_lds.h"
#include "fp8_mma.h"

namespace bpg {
namespace {

constexpr int kWaves = 8;

// XL: loads of 8 rows of x per block, so 8 XL rows at most.
template <int XL, bool GATED> struct Ring {
    static constexpr int G = GATED ? 2 : 1, MT = (XL + 1) / 2;
    static constexpr int kLoads = 2 * G + XL;                // of 1 KiB, per block
    static constexpr int kSlot = 2048 * (G + MT), kDepth = 2; // blocks on the way
    static constexpr int kScales = 2 * 256 * MT;             // two times four blocks'
    static constexpr int kWave = kDepth * kSlot + kScales;
};

template <int XL, bool GATED, bool EXACT>
__global__ __launch_bounds__(64 * kWaves) void fp8_stream_kernel(const Fp8Problem p, bool vec)
{
    typedef Ring<XL, GATED> R;
    constexpr int G = R::G, MT = R::MT, D = R::kDepth;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kWaves * R::kWave];
    static_assert(G * MT * 1024 <= R::kWave);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t k = p.k;
    const int blocks = (int)fp8_blocks(k), per = (blocks + kWaves - 1) / kWaves;
    const int first = min(wave * per, blocks), end = min(first + per, blocks);

    const uint32_t base = lds_address(lds) + wave * R::kWave;
    const uint32_t piece = (uint32_t)((lane & 7) ^ (lane >> 3)) * 16;
    const uint32_t lane_at = (uint32_t)((lane >> 3) * k) + piece;
    const v4i w0 = buffer_of(p.w, n0, p.n, k, 16);
    const v4i w1 = GATED ? buffer_of(p.up, n0, p.n, k, 16) : w0;
    const v4i x = buffer_of(p.codes, 0, p.m, k, 8 * XL);
    const v4i xs = buffer_of(p.scales, 0, p.m, (int64_t)blocks * 4, 8 * XL);
    const uint32_t slane = (uint32_t)(lane * blocks) * 4;
    auto load = [&](int slot, int b) {
        const uint32_t to = base + slot * R::kSlot, at = (uint32_t)b * kFp8Block;
        // pieces past K, and blocks past this wave's: zeros
        const uint32_t l = b < end && at + piece < k ? lane_at : kPastBuffer;
#pragma unroll
        for (int u = 0; u < 2; u++) {
            load16(w0, to + 1024 * u, l, (uint32_t)(8 * u * k) + at);
            if constexpr (GATED)
                load16(w1, to + 2048 + 1024 * u, l, (uint32_t)(8 * u * k) + at);
        }
#pragma unroll
        for (int u = 0; u < XL; u++)
            load16(x, to + 2048 * G + 1024 * u, l, (uint32_t)(8 * u * k) + at);
    };
    auto load_scales = [&](int c) { // of the wave's blocks 4 c .. 4 c + 3
        load16_lanes((uint64_t)~0u >> (32 - 16 * MT), xs,
                     base + D * R::kSlot + (c & 1) * 256 * MT, slane, (uint32_t)(first + 4 * c) * 4);
    };
    const int64_t wb = n0 / kFp8Block * blocks;
    // scalar loads: vector ones would be counted with the direct loads
    typedef const __attribute__((address_space(4))) float *Scalars;
    const Scalars s0 = (Scalars)(p.w_scales + wb);
    const Scalars s1 = (Scalars)(GATED ? p.up_scales + wb : p.w_scales);
    float w_next[G];
    auto w_scales = [&](int b) {
        b = min(b, blocks - 1);
        w_next[0] = s0[b];
        if constexpr (GATED)
            w_next[1] = s1[b];
    };

    v4f acc[G][MT];
#pragma unroll
    for (int i = 0; i < G; i++)
#pragma unroll
        for (int j = 0; j < MT; j++)
            acc[i][j] = v4f{0, 0, 0, 0};
    const uint32_t lo = (uint32_t)(r * 128 + ((g ^ (r & 7)) * 16)), hi = lo ^ 64;
    auto block = [&](int slot, int b) {
        const uint32_t at = base + slot * R::kSlot, i = (uint32_t)(b - first);
        auto operand = [&](uint32_t tile) {
            return Operand<EXACT>(lds_read<v4i>(at + lo, tile), lds_read<v4i>(at + hi, tile));
        };
        float sw[G], sx[MT];
#pragma unroll
        for (int q = 0; q < G; q++)
            sw[q] = w_next[q];
        w_scales(b + 1);
        arrived<(D - 1) * R::kLoads>();
        Operand<EXACT> a[G], c[MT];
#pragma unroll
        for (int q = 0; q < G; q++)
            a[q] = operand(2048 * q);
#pragma unroll
        for (int j = 0; j < MT; j++) {
            c[j] = operand(2048 * (G + j));
            sx[j] = lds_read<float>(
                base + D * R::kSlot + (i / 4 & 1) * 256 * MT + (i & 3) * 4 + r * 16, 256 * j);
        }
        read_done();
        load(slot, b + D);
        if ((i & 3) == 0)
            load_scales((int)i / 4 + 1);
#pragma unroll
        for (int j = 0; j < MT; j++)
#pragma unroll
            for (int q = 0; q < G; q++)
                add_scaled(acc[q][j], dot(a[q], c[j]), sx[j] * sw[q]);
    };
    load_scales(0);
#pragma unroll
    for (int q = 0; q < D; q++)
        load(q, first + q);
    w_scales(first);
    static_assert(D == 2);
    int b = first;
    for (; b + 1 < end; b += 2) {
        block(0, b);
        block(1, b + 1);
    }
    if (b < end)
        block(0, b);
    arrived<0>();

    // ---- the waves' sums, in their order; this wave's LDS is its own until here
    const uint32_t mine = base + lane * 16;
#pragma unroll
    for (int i = 0; i < G; i++)
#pragma unroll
        for (int j = 0; j < MT; j++)
            lds_write(mine + 1024 * (i * MT + j), acc[i][j]);
    __syncthreads();
    if (wave >= MT)
        return;
    const int j = wave;
    v4f sum[G];
#pragma unroll
    for (int i = 0; i < G; i++) {
        const uint32_t at = lds_address(lds) + lane * 16 + 1024 * (i * MT + j);
        sum[i] = lds_read<v4f>(at, 0);
#pragma unroll
        for (int u = 1; u < kWaves; u++)
            sum[i] += lds_read<v4f>(at, u * R::kWave);
    }
    if constexpr (GATED) {
        float t[4] = {sum[0][0], sum[0][1], sum[0][2], sum[0][3]};
        ep_activate(p.act, t);
        sum[0] = v4f{t[0], t[1], t[2], t[3]} * sum[G - 1];
    }
    const int64_t row = 16 * j + r, n = n0 + 4 * g;
    if (row < p.m && n < p.n)
        store4(p.y, p.y_bf16, vec, row * p.ldy + n, (int)min((int64_t)4, p.n - n), sum[0]);
}

template <int XL, bool EXACT> hipError_t launch(const Fp8Problem &p, hipStream_t s)
{
    const dim3 grid((unsigned)((p.n + 15) / 16));
    const bool vec = vector_rows(p.y, p.ldy, p.y_bf16);
    if (p.up)
        fp8_stream_kernel<XL, true, EXACT><<<grid, 64 * kWaves, 0, s>>>(p, vec);
    else
        fp8_stream_kernel<XL, false, EXACT><<<grid, 64 * kWaves, 0, s>>>(p, vec);
    return hipGetLastError();
}

template <bool EXACT> hipError_t stream(const Fp8Problem &p, hipStream_t s)
{
    return p.m <= 8    ? launch<1, EXACT>(p, s)
           : p.m <= 16 ? launch<2, EXACT>(p, s)
                       : launch<4, EXACT>(p, s);
}

} // namespace

hipError_t launch_fp8_stream(const Fp8Problem &p, hipStream_t s)
{
    return p.exact ? stream<true>(p, s) : stream<false>(p, s);
}

} // namespace bpg
