// fp8_tile.hip -- products of e4m3 codes over LDS tiles, for many rows (gfx950).
#include "fp8.h"

#include "epilogue.h"
#include "fp8_mma.h"

namespace bpg {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

// A workgroup's tile: NW x MW waves, each of 16 NI columns of y (rows of the
// weights) by 16 MJ rows.  Gated, the first half of a wave's NI row tiles are
// rows of the gate and the second half the same rows of the up projection.
template <int NI_, int MJ_, int NW_, int MW_> struct Tile {
    static constexpr int NI = NI_, MJ = MJ_, NW = NW_, MW = MW_;
    static constexpr int kWaves = NW * MW;
    static constexpr int kRowsW = 16 * NI * NW, kRowsX = 16 * MJ * MW;
    static constexpr int kLoadsW = kRowsW / 8 / kWaves, kLoadsX = kRowsX / 8 / kWaves;
};

// Codes [rows][k] from `row` on, as a buffer whose reads past the last row
// give zeros; `most` rows at most.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const uint8_t *codes, int64_t row,
                                                          int64_t rows, int64_t k, int most)
{
    const int64_t left = max((int64_t)0, min(rows - row, (int64_t)most));
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(codes + min(row, rows - 1) * k), 0,
                                             (int)(left * k), 0x00020000);
}

// 8 rows of 128 codes to LDS.  The 16-byte pieces of a row are stored in the
// order piece ^ (row % 8), so that the 16 rows that a quarter wave reads at one
// piece lie in different banks.
__device__ __forceinline__ void load_rows(__amdgpu_buffer_rsrc_t from, uint8_t *to, uint32_t lane_at,
                                          uint32_t at)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void *)to, 16, (int)lane_at, (int)at, 0, 0);
}

template <class T, bool GATED, bool EXACT, bool QUANT>
__global__ __launch_bounds__(64 * T::kWaves, T::kWaves == 8 ? 2 : 2) void fp8_tile_kernel(
    const Fp8Problem p, uint8_t *out_codes, float *out_scales, bool vec)
{
    constexpr int NI = T::NI, MJ = T::MJ, G = GATED ? 2 : 1;
    constexpr int kCols = T::kRowsW / G;
    __shared__ __attribute__((aligned(16))) uint8_t lw0[T::kRowsW * 128], lx0[T::kRowsX * 128];
    __shared__ __attribute__((aligned(16))) uint8_t lw1[T::kRowsW * 128], lx1[T::kRowsX * 128];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave % T::NW, wm = wave / T::NW;
    const int r = lane & 15, g = lane >> 4;
    // ---- which tile: every XCD a stretch of them, in panels of eight row tiles
    const int mt = (int)((p.m + T::kRowsX - 1) / T::kRowsX), nt = (int)((p.n + kCols - 1) / kCols);
    int id = blockIdx.x;
    {
        const int total = mt * nt, per = total / 8, past = total % 8;
        const int xcd = id % 8, at = id / 8;
        id = xcd * per + min(xcd, past) + at;
    }
    const int panel = id / (8 * nt), first = panel * 8, height = min(8, mt - first);
    const int in = id - panel * 8 * nt;
    const int64_t m0 = (int64_t)(first + in % height) * T::kRowsX;
    const int64_t n0 = (int64_t)(in / height) * kCols;
    const int64_t k = p.k;
    const int blocks = (int)fp8_blocks(k);

    // ---- direct loads: lane l of an instruction brings piece l % 8 of row l / 8
    const uint32_t piece = (uint32_t)((lane & 7) ^ (lane >> 3)) * 16;
    const uint32_t lane_at = (uint32_t)((lane >> 3) * k) + piece;
    const __amdgpu_buffer_rsrc_t xs = rows_of(p.codes, m0, p.m, k, T::kRowsX);
    const __amdgpu_buffer_rsrc_t ws = rows_of(p.w, n0, p.n, k, kCols);
    const __amdgpu_buffer_rsrc_t us = GATED ? rows_of(p.up, n0, p.n, k, kCols) : ws;
    auto load = [&](uint8_t *lw, uint8_t *lx, int b) {
        const uint32_t at = (uint32_t)b * kFp8Block;
        // pieces past K are read from past the buffer: zeros
        const uint32_t l = at + piece < k ? lane_at : 0x80000000u;
#pragma unroll
        for (int u = 0; u < T::kLoadsX; u++) {
            const int i = wave + T::kWaves * u;
            load_rows(xs, lx + 1024 * i, l, (uint32_t)(8 * i * k) + at);
        }
#pragma unroll
        for (int u = 0; u < T::kLoadsW; u++) {
            const int i = wave + T::kWaves * u;
            if constexpr (GATED) {
                constexpr int kWaveRows = 16 * NI, kHalf = kWaveRows / 2;
                const int row = 8 * i, in_wave = row % kWaveRows;
                const int col = row / kWaveRows * kHalf + in_wave % kHalf;
                if (in_wave < kHalf)
                    load_rows(ws, lw + 1024 * i, l, (uint32_t)(col * k) + at);
                else
                    load_rows(us, lw + 1024 * i, l, (uint32_t)(col * k) + at);
            } else {
                load_rows(ws, lw + 1024 * i, l, (uint32_t)(8 * i * k) + at);
            }
        }
    };

    // ---- scales: one per lane and row tile of x, one per wave of the weights
    const __amdgpu_buffer_rsrc_t xscales = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<float *>(p.scales + m0 * blocks), 0,
        (int)(min(p.m - m0, (int64_t)T::kRowsX) * blocks * 4), 0x00020000);
    const uint32_t sx_at = (uint32_t)(16 * wm * MJ + r) * (uint32_t)blocks * 4;
    const int64_t wb = min((n0 + wn * (16 * NI / G)) / kFp8Block, fp8_blocks(p.n) - 1) * blocks;
    const float *sw[G];
    sw[0] = p.w_scales + wb;
    if constexpr (GATED)
        sw[1] = p.up_scales + wb;
    float sx[MJ], ws_now[G];
    auto load_scales = [&](int b) {
#pragma unroll
        for (int j = 0; j < MJ; j++)
            sx[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                xscales, (int)sx_at, (16 * j * blocks + b) * 4, 0));
#pragma unroll
        for (int q = 0; q < G; q++)
            ws_now[q] = sw[q][b];
    };

    float sv[G][MJ];
    auto make_scales = [&] {
#pragma unroll
        for (int j = 0; j < MJ; j++)
#pragma unroll
            for (int q = 0; q < G; q++)
                sv[q][j] = sx[j] * ws_now[q];
    };

    v4f acc[NI][MJ];
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
        for (int j = 0; j < MJ; j++)
            acc[i][j] = v4f{0, 0, 0, 0};

    const uint32_t lo = (uint32_t)(r * 128 + ((g ^ (r & 7)) * 16)), hi = lo ^ 64;
    const uint32_t wrow = (uint32_t)(wn * NI) * 2048, xrow = (uint32_t)(wm * MJ) * 2048;
    auto operand = [&](const uint8_t *base, uint32_t tile) {
        return Operand<EXACT>(*reinterpret_cast<const v4i *>(base + tile + lo),
                              *reinterpret_cast<const v4i *>(base + tile + hi));
    };
    // The additions of a tile follow its matrix instruction kLag tiles behind.
    constexpr int kLag = 3, kTiles = NI * MJ;
    auto compute = [&](const uint8_t *lw, const uint8_t *lx) {
        Operand<EXACT> x[MJ];
#pragma unroll
        for (int j = 0; j < MJ; j++)
            x[j] = operand(lx, xrow + 2048 * j);
        Operand<EXACT> w = operand(lw, wrow), next = w;
        v4f d[kLag + 1];
#pragma unroll
        for (int t = 0; t < kTiles + kLag; t++) {
            const int i = t / MJ, j = t % MJ;
            if (t < kTiles) {
                if (j == 0) {
                    w = next;
                    if (i + 1 < NI)
                        next = operand(lw, wrow + 2048 * (i + 1));
                }
                d[t % (kLag + 1)] = dot(w, x[j]);
            }
            if (t >= kLag) {
                const int o = t - kLag;
                add_scaled(acc[o / MJ][o % MJ], d[o % (kLag + 1)],
                           sv[GATED && o / MJ >= NI / 2 ? G - 1 : 0][o % MJ]);
            }
            if (j == MJ - 1)
                __builtin_amdgcn_sched_barrier(0);
        }
    };

    // Two blocks a round, one basic block: what is loaded past the last one is
    // zeros that nobody reads.
    load(lw0, lx0, 0);
    load_scales(0);
    int b = 0;
    for (; b + 1 < blocks; b += 2) {
        __syncthreads(); // block b is there, and nobody reads the other buffer any more
        make_scales();
        load(lw1, lx1, b + 1);
        load_scales(b + 1);
        compute(lw0, lx0);
        __syncthreads();
        make_scales();
        load(lw0, lx0, b + 2);
        load_scales(min(b + 2, blocks - 1));
        compute(lw1, lx1);
    }
    __syncthreads();
    if (b < blocks) {
        make_scales();
        compute(lw0, lx0);
    }

    // ---- results
    constexpr int NO = NI / G; // row tiles of results
    const int64_t col0 = n0 + wn * (16 * NO);
    if constexpr (GATED) {
#pragma unroll
        for (int i = 0; i < NO; i++)
#pragma unroll
            for (int j = 0; j < MJ; j++) {
                float t[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                ep_activate(p.act, t);
                acc[i][j] = v4f{t[0], t[1], t[2], t[3]} * acc[i + NO][j];
            }
    }
    if constexpr (QUANT) {
        // a block of 128 columns: the waves of a row tile share its maximum
        static_assert(!QUANT || kCols == 128);
        __syncthreads(); // the operands are no longer read
        uint32_t *top = reinterpret_cast<uint32_t *>(lx0);
        uint32_t mine[MJ];
#pragma unroll
        for (int j = 0; j < MJ; j++) {
            uint32_t a = 0;
#pragma unroll
            for (int i = 0; i < NO; i++)
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    if (col0 + 16 * i + 4 * g < p.n) // n is a multiple of 32
                        a = max(a, __float_as_uint(acc[i][j][q]) & 0x7fffffffu);
                }
            a = max(a, (uint32_t)__shfl_xor((int)a, 16));
            mine[j] = max(a, (uint32_t)__shfl_xor((int)a, 32));
            if (g == 0)
                top[wn * T::kRowsX + 16 * (wm * MJ + j) + r] = mine[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < MJ; j++) {
            const int line = 16 * (wm * MJ + j) + r;
            uint32_t a = mine[j];
#pragma unroll
            for (int o = 0; o < T::NW; o++)
                a = max(a, top[o * T::kRowsX + line]);
            const float d = __uint_as_float(a) / 448.0f;
            const float inv = d > 0.0f ? fminf(1.0f / d, 3.402823466e38f) : 0.0f;
            const int64_t row = m0 + line;
            if (row >= p.m)
                continue;
            if (wn == 0 && g == 0)
                out_scales[row * fp8_blocks(p.n) + n0 / kFp8Block] = d;
#pragma unroll
            for (int i = 0; i < NO; i++) {
                const v4f v = acc[i][j] * inv;
                int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
                c = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], c, true);
                const int64_t n = col0 + 16 * i + 4 * g;
                if (n < p.n)
                    *reinterpret_cast<int *>(out_codes + row * p.n + n) = c;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < MJ; j++) {
            const int64_t row = m0 + 16 * (wm * MJ + j) + r;
            if (row >= p.m)
                continue;
#pragma unroll
            for (int i = 0; i < NO; i++) {
                const int64_t n = col0 + 16 * i + 4 * g;
                if (n < p.n)
                    store4(p.y, p.y_bf16, vec, row * p.ldy + n, (int)min((int64_t)4, p.n - n),
                           acc[i][j]);
            }
        }
    }
}

typedef Tile<8, 4, 2, 4> Tile256; // 256 x 256, eight waves
typedef Tile<4, 4, 2, 2> Tile128; // 128 x 128, four waves

template <class T, bool GATED, bool EXACT, bool QUANT>
hipError_t launch_tile(const Fp8Problem &p, uint8_t *codes, float *scales, hipStream_t s)
{
    constexpr int kCols = T::kRowsW / (GATED ? 2 : 1);
    const int64_t tiles = (p.m + T::kRowsX - 1) / T::kRowsX * ((p.n + kCols - 1) / kCols);
    fp8_tile_kernel<T, GATED, EXACT, QUANT><<<(unsigned)tiles, 64 * T::kWaves, 0, s>>>(
        p, codes, scales, !QUANT && vector_rows(p.y, p.ldy, p.y_bf16));
    return hipGetLastError();
}

} // namespace

hipError_t launch_fp8_tile(const Fp8Problem &p, int size, hipStream_t s)
{
    if (p.exact)
        return p.up ? launch_tile<Tile128, true, true, false>(p, nullptr, nullptr, s)
                    : launch_tile<Tile128, false, true, false>(p, nullptr, nullptr, s);
    if (size == 256)
        return p.up ? launch_tile<Tile256, true, false, false>(p, nullptr, nullptr, s)
                    : launch_tile<Tile256, false, false, false>(p, nullptr, nullptr, s);
    return p.up ? launch_tile<Tile128, true, false, false>(p, nullptr, nullptr, s)
                : launch_tile<Tile128, false, false, false>(p, nullptr, nullptr, s);
}

hipError_t launch_fp8_tile_quantize(const Fp8Problem &p, uint8_t *codes, float *scales, hipStream_t s)
{
    return launch_tile<Tile256, true, false, true>(p, codes, scales, s);
}

} // namespace bpg
