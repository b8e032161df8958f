// fp8_stream.hip -- products of e4m3 codes whose operands go straight from
// memory to registers (gfx950).
//
//   y[m][n] = sum over blocks b of sx[m][b] sw[n / 128][b] * dot(x block, w block)
//
// and, gated, act(y_gate) * y_up.  A workgroup makes 16 columns of w (16 of
// each matrix, gated) by 16 MT rows of x; its eight waves take the blocks of K
// in turn and add their partial results through LDS, in wave order.
#include "fp8.h"

#include "epilogue.h"
#include "fp8_mma.h"

namespace bpg {
namespace {

constexpr int kWaves = 8;

template <int MT, bool GATED, bool EXACT>
__global__ __launch_bounds__(64 * kWaves) void fp8_stream_kernel(const Fp8Problem p, bool vec)
{
    constexpr int G = GATED ? 2 : 1;
    __shared__ v4f part[kWaves][G * MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * MT);
    const int64_t blocks = fp8_blocks(p.k);
    // rows past the end read the last one: their results are not stored
    const int64_t wr = min(n0 + r, p.n - 1);
    const uint8_t *w[G];
    const float *ws[G];
    w[0] = p.w + wr * p.k + 16 * g;
    ws[0] = p.w_scales + n0 / kFp8Block * blocks;
    if constexpr (GATED) {
        w[1] = p.up + wr * p.k + 16 * g;
        ws[1] = p.up_scales + n0 / kFp8Block * blocks;
    }
    const uint8_t *x[MT];
    const float *xs[MT];
#pragma unroll
    for (int j = 0; j < MT; j++) {
        const int64_t row = min(m0 + 16 * j + r, p.m - 1);
        x[j] = p.codes + row * p.k + 16 * g;
        xs[j] = p.scales + row * blocks;
    }
    v4f acc[G][MT];
#pragma unroll
    for (int i = 0; i < G; i++)
#pragma unroll
        for (int j = 0; j < MT; j++)
            acc[i][j] = v4f{0, 0, 0, 0};
    for (int64_t b = wave; b < blocks; b += kWaves) {
        const int64_t at = b * kFp8Block;
        // K is a multiple of 32, so 16 codes are all inside it or all outside
        const bool lo = at + 16 * g < p.k, hi = at + 64 + 16 * g < p.k;
        const v4i none{0, 0, 0, 0};
        auto operand = [&](const uint8_t *row) {
            return Operand<EXACT>(lo ? *reinterpret_cast<const v4i *>(row + at) : none,
                                  hi ? *reinterpret_cast<const v4i *>(row + at + 64) : none);
        };
        Operand<EXACT> a[G];
#pragma unroll
        for (int i = 0; i < G; i++)
            a[i] = operand(w[i]);
#pragma unroll
        for (int j = 0; j < MT; j++) {
            const Operand<EXACT> c = operand(x[j]);
            const float s = xs[j][b];
#pragma unroll
            for (int i = 0; i < G; i++)
                add_scaled(acc[i][j], dot(a[i], c), s * ws[i][b]);
        }
    }
#pragma unroll
    for (int i = 0; i < G; i++)
#pragma unroll
        for (int j = 0; j < MT; j++)
            part[wave][i * MT + j][lane] = acc[i][j];
    __syncthreads();
    for (int j = wave; j < MT; j += kWaves) {
        v4f sum[G];
#pragma unroll
        for (int i = 0; i < G; i++) {
            sum[i] = part[0][i * MT + j][lane];
#pragma unroll
            for (int u = 1; u < kWaves; u++)
                sum[i] += part[u][i * MT + j][lane];
        }
        if constexpr (GATED) {
            float t[4] = {sum[0][0], sum[0][1], sum[0][2], sum[0][3]};
            ep_activate(p.act, t);
            sum[0] = v4f{t[0], t[1], t[2], t[3]} * sum[G - 1];
        }
        const int64_t row = m0 + 16 * j + r, n = n0 + 4 * g;
        if (row < p.m && n < p.n)
            store4(p.y, p.y_bf16, vec, row * p.ldy + n, (int)min((int64_t)4, p.n - n), sum[0]);
    }
}

template <int MT, bool EXACT> hipError_t stream(const Fp8Problem &p, hipStream_t s)
{
    const dim3 grid((unsigned)((p.n + 15) / 16), (unsigned)((p.m + 16 * MT - 1) / (16 * MT)));
    const bool vec = vector_rows(p.y, p.ldy, p.y_bf16);
    if (p.up)
        fp8_stream_kernel<MT, true, EXACT><<<grid, 64 * kWaves, 0, s>>>(p, vec);
    else
        fp8_stream_kernel<MT, false, EXACT><<<grid, 64 * kWaves, 0, s>>>(p, vec);
    return hipGetLastError();
}

} // namespace

hipError_t launch_fp8_gemm(const Fp8Problem &p, hipStream_t s)
{
    if (p.m == 0)
        return hipSuccess;
    if (p.m > 64)
        return launch_fp8_tiles(p, s);
    if (p.m <= 16)
        return p.exact ? stream<1, true>(p, s) : stream<1, false>(p, s);
    if (p.m <= 32)
        return p.exact ? stream<2, true>(p, s) : stream<2, false>(p, s);
    return p.exact ? stream<4, true>(p, s) : stream<4, false>(p, s);
}

size_t fp8_gated_quantize_bytes(int64_t m, int64_t n, int64_t)
{
    return m > 64 ? 0 : (size_t)m * (size_t)n * sizeof(float);
}

hipError_t launch_fp8_gated_quantize(const Fp8Problem &p, uint8_t *codes, float *scales,
                                     void *workspace, hipStream_t s)
{
    if (p.m > 64)
        return launch_fp8_tile_codes(p, codes, scales, s);
    Fp8Problem values = p;
    values.y = workspace;
    values.ldy = p.n;
    const hipError_t e = launch_fp8_gemm(values, s);
    if (e != hipSuccess)
        return e;
    return launch_fp8_quantize(workspace, false, p.m, p.n, p.n, false, codes, scales, s);
}

} // namespace bpg
