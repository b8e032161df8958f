// fp8_tile.hip -- products of e4m3 codes over LDS tiles, for many rows (gfx950).
#include "fp8.h"

#include "epilogue.h"
#include "fp8_mma.h"

#include <type_traits>

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
};

// [rows][row_bytes] from `row` on, `most` rows at most, as a buffer: reads past
// its last row give zeros.
__device__ __forceinline__ v4i rows_of(const void *at, int64_t row, int64_t rows, int64_t row_bytes,
                                       int most)
{
    const int64_t first = min(row, rows - 1);
    const int64_t left = max((int64_t)0, min(rows - row, (int64_t)most));
    const uint64_t base = reinterpret_cast<uint64_t>(at) + (uint64_t)(first * row_bytes);
    return v4i{__builtin_amdgcn_readfirstlane((int)(uint32_t)base),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32)),
               __builtin_amdgcn_readfirstlane((int)(left * row_bytes)), 0x00020000};
}

// Direct loads of 16 or 4 bytes a lane, to LDS addresses to + 16 lane or
// to + 4 lane.  Written out so that the compiler, which cannot tell the stages
// of one LDS array apart, waits for none of them before a read: the waits are
// at the barriers (`arrived`).
__device__ __forceinline__ void load16(v4i from, uint32_t to, uint32_t lane_at, uint32_t at)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(to), "v"(lane_at), "s"(from), "s"(at)
                 : "memory");
}

__device__ __forceinline__ void load4(v4i from, uint32_t to, uint32_t lane_at, uint32_t at)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(to), "v"(lane_at), "s"(from), "s"(at)
                 : "memory");
}

// All direct loads of this wave but the last N are in LDS, its own LDS reads
// are done, and so are those of the other waves.
template <int N> __device__ __forceinline__ void arrived()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

template <class T, bool GATED, bool EXACT, bool QUANT>
__global__ __launch_bounds__(64 * T::kWaves, T::kWaves == 8 ? 2 : 2) void fp8_tile_kernel(
    const Fp8Problem p, uint8_t *out_codes, float *out_scales, bool vec)
{
    constexpr int NI = T::NI, MJ = T::MJ, G = GATED ? 2 : 1;
    constexpr int kCols = T::kRowsW / G;
    constexpr int kX = T::kRowsX * 128, kW = T::kRowsW * 128;
    constexpr int kStage = kX + kW + T::kRowsX * 4; // codes of x and w, scales of x
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];
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

    // ---- direct loads.  Lane l of an instruction brings a 16-byte piece of row
    //      l / 8: piece l % 8 of the row in LDS, which is piece (l % 8) ^ (l / 8)
    //      of the row in memory, so that the 16 rows that a quarter wave reads at
    //      one piece lie in different banks.
    const uint32_t base = (uint32_t) reinterpret_cast<uintptr_t>((lds_void *)lds);
    const uint32_t piece = (uint32_t)((lane & 7) ^ (lane >> 3)) * 16;
    const uint32_t lane_at = (uint32_t)((lane >> 3) * k) + piece;
    const v4i xs = rows_of(p.codes, m0, p.m, k, T::kRowsX);
    const v4i ws = rows_of(p.w, n0, p.n, k, kCols);
    const v4i us = GATED ? rows_of(p.up, n0, p.n, k, kCols) : ws;
    const v4i ss = rows_of(p.scales, m0, p.m, (int64_t)blocks * 4, T::kRowsX);
    const int sline = wave % (T::kRowsX / 64) * 64; // rows whose scales this wave brings
    const uint32_t slane = (uint32_t)((sline + lane) * blocks) * 4;
    // What a stage brings comes in two groups: x, the scales and each wave's
    // first half of w's row tiles; and their second half.
    constexpr int kLoadsX = T::kRowsX / 8 / T::kWaves, kLoadsW = T::kRowsW / 16 / T::kWaves;
    constexpr int kFirst = kLoadsX + 1 + kLoadsW, kSecond = kLoadsW;
    auto load_w = [&](uint32_t to, int b, uint32_t l, int half, int u) {
        constexpr int kHalf = 8 * NI, kParts = kHalf / 8; // rows and loads of a wave's half
        const int i = wave + T::kWaves * u, owner = i / kParts, row = i % kParts * 8;
        const int in = owner * 2 * kHalf + half * kHalf + row;
        const int col = GATED ? owner * kHalf + row : in;
        load16(GATED && half ? us : ws, to + kX + in * 128, l, (uint32_t)(col * k) + b * kFp8Block);
    };
    // pieces past K are read from past the buffer: zeros
    auto lane_from = [&](int b) {
        return (uint32_t)(b * kFp8Block) + piece < k ? lane_at : 0x80000000u;
    };
    auto load_first = [&](int b, int u) {
        const uint32_t to = base + (b & 1) * kStage, l = lane_from(b);
        if (u < kLoadsX) {
            const int i = wave + T::kWaves * u;
            load16(xs, to + 1024 * i, l, (uint32_t)(8 * i * k) + b * kFp8Block);
        } else if (u < kLoadsX + kLoadsW) {
            load_w(to, b, l, 0, u - kLoadsX);
        } else {
            load4(ss, to + kX + kW + 4 * sline, b < blocks ? slane : 0x80000000u, b * 4);
        }
    };
    auto load_second = [&](int b, int u) {
        load_w(base + (b & 1) * kStage, b, lane_from(b), 1, u);
    };

    // ---- scales of the weights: one per wave and block
    typedef const __attribute__((address_space(4))) float *Scalars;
    const int64_t wb = min((n0 + wn * (16 * NI / G)) / kFp8Block, fp8_blocks(p.n) - 1) * blocks;
    const Scalars sw = (Scalars)(p.w_scales + wb), su = (Scalars)(GATED ? p.up_scales + wb : nullptr);
    float w_scale[G], w_next[G];
    auto load_scalars = [&](int b) {
        b = min(b, blocks - 1);
        w_next[0] = sw[b];
        if constexpr (GATED)
            w_next[1] = su[b];
    };

    v4f acc[NI][MJ];
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
        for (int j = 0; j < MJ; j++)
            acc[i][j] = v4f{0, 0, 0, 0};

    const uint32_t lo = (uint32_t)(r * 128 + ((g ^ (r & 7)) * 16)), hi = lo ^ 64;
    const uint32_t x_lo = wm * MJ * 2048 + lo, x_hi = wm * MJ * 2048 + hi;
    const uint32_t w_lo = kX + wn * NI * 2048 + lo, w_hi = kX + wn * NI * 2048 + hi;
    const uint32_t s_at = kX + kW + (wm * MJ * 16 + r) * 4;
    Operand<EXACT> x[MJ], w, next;
    float sx[MJ], sv[MJ];
    auto read_w = [&](int stage, int i) {
        const uint8_t *at = lds + stage * kStage + 2048 * i;
        next = Operand<EXACT>(*reinterpret_cast<const v4i *>(at + w_lo),
                              *reinterpret_cast<const v4i *>(at + w_hi));
    };
    auto read_x = [&](int stage, int j) {
        const uint8_t *at = lds + stage * kStage + 2048 * j;
        x[j] = Operand<EXACT>(*reinterpret_cast<const v4i *>(at + x_lo),
                              *reinterpret_cast<const v4i *>(at + x_hi));
    };
    auto read_scales = [&](int stage) {
#pragma unroll
        for (int j = 0; j < MJ; j++)
            sx[j] = *reinterpret_cast<const float *>(lds + stage * kStage + s_at + 64 * j);
    };
    // The additions of a tile follow its matrix instruction kLag tiles behind,
    // into the next block's: the first ones add zeros.
    constexpr int kLag = 3, kRing = kLag + 1, kTiles = NI * MJ;
    static_assert(kTiles % kRing == 0);
    v4f d[kRing];
#pragma unroll
    for (int q = 0; q < kRing; q++)
        d[q] = v4f{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < MJ; j++)
        sv[j] = 0;
    auto additions = [&](int t) { // of tile t, or of the block before for t < 0
        const bool past = t < 0;
        t = past ? t + kTiles : t;
        const int i = t / MJ, j = t % MJ;
        if (!past && i == 0)
            sv[j] = sx[j] * w_scale[0];
        if (GATED && !past && i == NI / 2)
            sv[j] = sx[j] * w_scale[G - 1];
        add_scaled(acc[i][j], d[t % kRing], sv[j]);
    };

    // One block of K from stage b & 1.  x and the first row tile of w have been
    // read; on the way the other stage arrives and this one is loaded anew:
    //   before row tile NI/2 - 1: the second half of w is there, and x, the
    //     scales and the first half are read by everybody: block b + 2's follow;
    //   before the last row tile: the next block's x, scales and first half are
    //     there, and this one's second half is read by everybody.
    // Each load has about one and a half blocks' time to arrive.
    auto block = [&](auto stage_of, int b) {
        constexpr int stage = decltype(stage_of)::value;
        constexpr int kTurn = NI / 2 - 1, kLast = NI - 1;
        constexpr int kPerRow = (kFirst + kLast - kTurn - 1) / (kLast - kTurn);
#pragma unroll
        for (int i = 0; i < NI; i++) {
            if (i == kTurn || i == kLast)
                arrived<kFirst + kSecond>();
            w = next;
            if (i == 0) {
#pragma unroll
                for (int q = 0; q < G; q++)
                    w_scale[q] = w_next[q];
                load_scalars(b + 1);
            }
            if (i < kLast)
                read_w(stage, i + 1);
            else
                read_w(stage ^ 1, 0);
            if (i >= kTurn && i < kLast) {
#pragma unroll
                for (int u = (i - kTurn) * kPerRow; u < min((i - kTurn + 1) * kPerRow, kFirst); u++)
                    load_first(b + 2, u);
            }
            if (i == kLast) {
#pragma unroll
                for (int u = 0; u < kSecond; u++)
                    load_second(b + 2, u);
            }
#pragma unroll
            for (int j = 0; j < MJ; j++) {
                const int t = i * MJ + j;
                d[t % kRing] = dot(w, x[j]);
                additions(t - kLag);
                if (i == kLast)
                    read_x(stage ^ 1, j);
            }
            if (i == kLast)
                read_scales(stage ^ 1);
            if (!EXACT) {
#pragma unroll
                for (int j = 0; j < MJ; j++) {
                    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0); // a matrix instruction
                    __builtin_amdgcn_sched_group_barrier(0x2, 4, 0); // an earlier one's additions
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

#pragma unroll
    for (int u = 0; u < kFirst; u++)
        load_first(0, u);
#pragma unroll
    for (int u = 0; u < kSecond; u++)
        load_second(0, u);
#pragma unroll
    for (int u = 0; u < kFirst; u++)
        load_first(1, u);
    load_scalars(0);
    arrived<kFirst + kSecond>();
#pragma unroll
    for (int u = 0; u < kSecond; u++)
        load_second(1, u);
    read_w(0, 0);
#pragma unroll
    for (int j = 0; j < MJ; j++)
        read_x(0, j);
    read_scales(0);
    int b = 0;
    for (; b + 1 < blocks; b += 2) {
        block(std::integral_constant<int, 0>{}, b);
        block(std::integral_constant<int, 1>{}, b + 1);
    }
    if (b < blocks)
        block(std::integral_constant<int, 0>{}, b);
#pragma unroll
    for (int t = -kLag; t < 0; t++)
        additions(t);
    arrived<0>(); // loads past the last block write to LDS, too

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
        uint32_t *top = reinterpret_cast<uint32_t *>(lds);
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
