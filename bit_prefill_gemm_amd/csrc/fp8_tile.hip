// fp8_tile.hip -- products of e4m3 codes over LDS tiles, for many rows (gfx950).
#include "fp8.h"

#include "epilogue.h"
#include "fp8_lds.h"
#include "fp8_mma.h"

#include <cfloat>
#include <type_traits>

namespace bpg {
namespace {

typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// A workgroup's tile: NW x MW waves, each of 16 NI columns of y (rows of the
// weights) by 16 MJ rows.  Gated, the first half of a wave's NI row tiles are
// rows of the gate and the second half the same rows of the up projection.
// KS groups of such waves take a part of K each; S stages of one block of K are
// in LDS, and P waves of a group do nothing but load them (0: the others do).
//
// What the tiles reach (bf16 results, rows x columns x K, weights in the last
// cache): 256x256 2290 to 2380 TF at 8192 x 17408 x 5120 (614 to 637 us with the
// rest of the columns; the library's product of the same size under one scale for
// everything 2500 TF), 128x128 1210 TF at 512 x 5120 x 5120 (22.1 us, 160
// workgroups).  A block of 256x256 takes 2700 clocks of the matrix unit's 2048,
// one of 128x128 1080 of 512.  What bounds them is the vector unit beside the
// matrix unit: the block scales cost four additions per instruction, and while a
// matrix instruction reads its operands (16 clocks) no other one is issued, so
// that two waves of a SIMD need 37 clocks for 32 and one, alone, 45; the rest is
// barriers and the first and last block.  32 x 32 instructions (half the reads,
// but twice the registers per operand, so fewer of them in flight) took 663 us
// at the first size beside 614, and 22.9 at the second beside 22.5.
template <int NI_, int MJ_, int NW_, int MW_, int KS_, int S_, int P_ = 0>
struct Tile {
    static constexpr int NI = NI_, MJ = MJ_, NW = NW_, MW = MW_, KS = KS_, S = S_;
    static constexpr int P = P_; // loading waves of a group, 0: the others load
    static constexpr int kLoaders = P ? P : NW_ * MW_, kThreads = 64 * KS_ * (NW_ * MW_ + P_);
    static constexpr int kWaves = NW * MW; // of a group
    static constexpr int kRowsW = 16 * NI * NW, kRowsX = 16 * MJ * MW;
};

// What a tile's results are stored as.
enum Store { kBf16, kF32, kCodes };

template <class T, bool GATED, bool EXACT, Store STORE>
__global__ __launch_bounds__(T::kThreads, 2) void fp8_tile_kernel(
    const Fp8Problem p, int64_t col_first, int64_t cols, int k_each, uint8_t *out_codes,
    float *out_scales)
{
    constexpr int NI = T::NI, MJ = T::MJ, S = T::S, KS = T::KS, G = GATED ? 2 : 1;
    constexpr int kCols = T::kRowsW / G;
    constexpr int kX = T::kRowsX * 128, kW = T::kRowsW * 128;
    constexpr int kStage = kX + kW, kScales = T::kRowsX * 16; // four blocks' scales of x
    constexpr int kGroup = S * kStage + 2 * kScales;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[KS * kGroup];
    const int lane = threadIdx.x & 63;
    // the waves that multiply come first, then those that load (P of a group)
    const int number = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool loads = T::P > 0 && number >= T::kWaves * KS;
    const int wave = loads ? (number - T::kWaves * KS) % T::kLoaders : number % T::kWaves;
    const int group = loads ? (number - T::kWaves * KS) / T::kLoaders : number / T::kWaves;
    const int wn = wave % T::NW, wm = wave / T::NW;
    const int r = lane & 15, g = lane >> 4;
    // ---- which tile: every XCD a stretch of them, in panels of eight row tiles
    const int mt = (int)((p.m + T::kRowsX - 1) / T::kRowsX), nt = (int)((cols + kCols - 1) / kCols);
    int id = blockIdx.x;
    {
        const int total = mt * nt, per = total / 8, past = total % 8;
        const int xcd = id % 8, at = id / 8;
        id = xcd * per + min(xcd, past) + at;
    }
    const int panel = id / (8 * nt), first = panel * 8, height = min(8, mt - first);
    const int in = id - panel * 8 * nt;
    const int64_t m0 = (int64_t)(first + in % height) * T::kRowsX;
    const int64_t n0 = col_first + (int64_t)(in / height) * kCols;
    const int64_t k = p.k;
    const int blocks = (int)fp8_blocks(k);

    // ---- direct loads, eight rows an instruction (fp8_lds.h)
    const uint32_t base = lds_address(lds) + group * kGroup;
    const uint32_t piece = (uint32_t)((lane & 7) ^ (lane >> 3)) * 16;
    const uint32_t lane_at = (uint32_t)((lane >> 3) * k) + piece;
    const v4i xs = buffer_of(p.codes, m0, p.m, k, T::kRowsX);
    const v4i ws = buffer_of(p.w, n0, p.n, k, kCols);
    const v4i us = GATED ? buffer_of(p.up, n0, p.n, k, kCols) : ws;
    const v4i ss = buffer_of(p.scales, m0, p.m, (int64_t)blocks * 4, T::kRowsX);
    // scales: 64 rows of 16 bytes an instruction, every fourth block
    constexpr int kScaleWaves = T::kRowsX / 64;
    static_assert(kScaleWaves <= T::kLoaders);
    const uint32_t slane = (uint32_t)((64 * wave + lane) * blocks) * 4;
    // What a stage brings comes in two groups: x, the scales and each wave's
    // first half of w's row tiles; and their second half.
    constexpr int kLoadsX = T::kRowsX / 8 / T::kLoaders, kLoadsW = T::kRowsW / 16 / T::kLoaders;
    static_assert(kLoadsX * 8 * T::kLoaders == T::kRowsX && kLoadsW * 16 * T::kLoaders == T::kRowsW);
    constexpr int kFirst = kLoadsX + kLoadsW, kSecond = kLoadsW;
    // a group's block b is block b + before of K; blockIdx.y: which k_each blocks
    // of K the workgroup takes
    const int k_first = blockIdx.y * k_each, k_end = min(k_first + k_each, blocks);
    const int rounds = (k_end - k_first + KS - 1) / KS, before = k_first + group * rounds;
    auto at_of = [&](int b) { return (uint32_t)(b + before) * kFp8Block; };
    auto load_w = [&](uint32_t to, int b, uint32_t l, int half, int u) {
        constexpr int kHalf = 8 * NI, kParts = kHalf / 8; // rows and loads of a wave's half
        const int i = wave + T::kLoaders * u, owner = i / kParts, row = i % kParts * 8;
        const int in = owner * 2 * kHalf + half * kHalf + row;
        const int col = GATED ? owner * kHalf + row : in;
        load16(GATED && half ? us : ws, to + kX + in * 128, l, (uint32_t)(col * k) + at_of(b));
    };
    // pieces past K or past the workgroup's blocks are read from past the buffer: zeros
    auto lane_from = [&](int b) {
        return b + before < k_end && at_of(b) + piece < k ? lane_at : kPastBuffer;
    };
    auto load_first = [&](int stage, int b, int u) {
        const uint32_t to = base + stage * kStage, l = lane_from(b);
        if (u < kLoadsX) {
            const int i = wave + T::kLoaders * u;
            load16(xs, to + 1024 * i, l, (uint32_t)(8 * i * k) + at_of(b));
        } else {
            load_w(to, b, l, 0, u - kLoadsX);
        }
    };
    auto load_scales = [&](int b, bool now) { // of blocks b..b+3
        load16_lanes(now && wave < kScaleWaves ? ~(uint64_t)0 : 0, ss,
                     base + S * kStage + (b / 4 & 1) * kScales + 1024 * wave, slane,
                     (uint32_t)(b + before) * 4);
    };
    auto load_second = [&](int stage, int b, int u) {
        load_w(base + stage * kStage, b, lane_from(b), 1, u);
    };

    // ---- scales of the weights: one per wave and block, 64 blocks' at a time in
    //      the lanes of a register.  (As scalar loads they would share a counter
    //      with the LDS reads, which then could not be waited for one by one.)
    const int64_t wb = min((n0 + wn * (16 * NI / G)) / kFp8Block, fp8_blocks(p.n) - 1) * blocks;
    float w_lanes[G], w_scale[G];
    auto load_w_scales = [&](int b) {
        const int at = b + lane + before;
        w_lanes[0] = at < k_end ? p.w_scales[wb + at] : 0.0f;
        if constexpr (GATED)
            w_lanes[1] = at < k_end ? p.up_scales[wb + at] : 0.0f;
        // wait here, not where they are used: that is in the loop below, and the
        // wait would be for its direct loads too
#pragma unroll
        for (int q = 0; q < G; q++)
            asm volatile("" : "+v"(w_lanes[q]));
    };

    v4f acc[NI][MJ];
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
        for (int j = 0; j < MJ; j++)
            acc[i][j] = v4f{0, 0, 0, 0};

    // LDS addresses of this lane's operands, a register each per stage: the rest
    // of an address is a constant of the instruction
    const uint32_t lo = (uint32_t)(r * 128 + ((g ^ (r & 7)) * 16)), hi = lo ^ 64;
    uint32_t x_lo[S], x_hi[S], w_lo[S], w_hi[S];
#pragma unroll
    for (int q = 0; q < S; q++) {
        x_lo[q] = opaque(base + q * kStage + wm * MJ * 2048 + lo);
        x_hi[q] = opaque(base + q * kStage + wm * MJ * 2048 + hi);
        w_lo[q] = opaque(base + q * kStage + kX + wn * NI * 2048 + lo);
        w_hi[q] = opaque(base + q * kStage + kX + wn * NI * 2048 + hi);
    }
    const uint32_t s_at = opaque(base + S * kStage + (wm * MJ * 16 + r) * 16);
    // w's row tiles are read kAhead tiles before their use
    constexpr int kAhead = 2;
    constexpr int XS = T::P > 0 ? 2 : 1; // sets of x
    static_assert(T::P == 0 || S % 2 == 0);
    Operand<EXACT> x[XS][MJ], w[kAhead];
    float sx[MJ], sv[G][MJ];
    auto read_w = [&](int stage, int i) {
        w[i % kAhead] = Operand<EXACT>(lds_read<v4i>(w_lo[stage], 2048 * i),
                                       lds_read<v4i>(w_hi[stage], 2048 * i));
    };
    auto read_x = [&](int stage, int j) {
        x[stage % XS][j] = Operand<EXACT>(lds_read<v4i>(x_lo[stage], 2048 * j),
                                          lds_read<v4i>(x_hi[stage], 2048 * j));
    };
    auto read_scales = [&](int b) {
        const uint32_t at = s_at + (b / 4 & 1) * kScales + (b & 3) * 4;
#pragma unroll
        for (int j = 0; j < MJ; j++) {
            sx[j] = lds_read<float>(at, 256 * j);
            if (KS > 1) // blocks past the end: what lies there is no scale
                sx[j] = b + before < k_end ? sx[j] : 0.0f;
        }
    };
    // The additions of a tile follow its matrix instruction kLag tiles behind,
    // into the next block's: the first ones add zeros.  Row tile 0's, which take
    // the block's scales, are never left for the next block.
    constexpr int kTiles = NI * MJ, kRing = 4;
    constexpr int kLag = kRing - 1 < kTiles - MJ ? kRing - 1 : kTiles - MJ;
    static_assert(kTiles % kRing == 0);
    v4f d[kRing];
#pragma unroll
    for (int q = 0; q < kRing; q++)
        d[q] = v4f{0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < G; q++)
#pragma unroll
        for (int j = 0; j < MJ; j++)
            sv[q][j] = 0;
    auto additions = [&](int t) { // of tile t, or of the block before for t < 0
        const bool past = t < 0;
        t = past ? t + kTiles : t;
        const int i = t / MJ, j = t % MJ;
        if (!past && i == 0) {
#pragma unroll
            for (int q = 0; q < G; q++)
                sv[q][j] = sx[j] * w_scale[q];
        }
        add_scaled(acc[i][j], d[t % kRing], sv[i / (NI / G)][j]);
    };

    // One block of K from its stage.  x and the first kAhead row tiles of w have
    // been read; on the way the next stage arrives and, where these waves load,
    // this one is loaded anew:
    //   at row tile kTurn: the second half of w is there, and x, the scales and
    //     the first half are read by everybody: block b + S's follow;
    //   at row tile kLast: the next block's x, scales and first half are there,
    //     and this one's second half is read by everybody.
    // With two stages each load has about one and a half blocks' time to arrive.
    auto block = [&](auto stage_of, int b0, int b) {
        constexpr int stage = decltype(stage_of)::value, after = (stage + 1) % S;
        constexpr int kTurn = NI / 2 - kAhead, kLast = NI - kAhead;
        constexpr int kPerRow = (kFirst + kLast - kTurn - 1) / (kLast - kTurn);
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const Operand<EXACT> row = w[i % kAhead];
            if (i == 0) {
#pragma unroll
                for (int q = 0; q < G; q++)
                    w_scale[q] = __uint_as_float(
                        __builtin_amdgcn_readlane(__float_as_uint(w_lanes[q]), b - b0));
            }
            if (T::P == 0 && i == kTurn + 1)
                load_scales((b & ~3) + 4, (b & 3) == 0);
            if (T::P > 0 && i == NI - 1) {
#pragma unroll
                for (int j = 0; j < MJ; j++)
                    read_x(after, j);
            }
            if (T::P == 0 && i > kTurn && i <= kLast) {
#pragma unroll
                for (int u = (i - kTurn - 1) * kPerRow; u < min((i - kTurn) * kPerRow, kFirst); u++)
                    load_first(stage, b + S, u);
            }
            if (T::P == 0 && i == kLast + 1) {
#pragma unroll
                for (int u = 0; u < kSecond; u++)
                    load_second(stage, b + S, u);
            }
#pragma unroll
            for (int j = 0; j < MJ; j++) {
                const int t = i * MJ + j;
                d[t % kRing] = dot(row, x[stage % XS][j]);
                additions(t - kLag);
                if (T::P == 0 && i == NI - 1)
                    read_x(after, j);
            }
            if ((T::P == 0 && i == kTurn) || i == kLast) {
                __builtin_amdgcn_sched_barrier(0);
                arrived_all<(T::P > 0) ? 63 : (S - 1) * (kFirst + kSecond)>();
            }
            if (i < kLast)
                read_w(stage, i + kAhead);
            else
                read_w(after, i + kAhead - NI);
            if (i == NI - 1)
                read_scales(b + 1);
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

    // Waves of their own load, S - 1 blocks ahead: a wave that does both waits for
    // the load unit while it could multiply (64x128, 256 x 5120 x 5120: 17.9 us,
    // so 16.5).  One barrier a block, behind its last read of w: block b + 1 is
    // there, and block b's stage is free.
    if (loads) {
        constexpr int kAll = kFirst + kSecond;
        auto load_all = [&](int stage, int b) {
#pragma unroll
            for (int u = 0; u < kFirst; u++)
                load_first(stage, b, u);
#pragma unroll
            for (int u = 0; u < kSecond; u++)
                load_second(stage, b, u);
        };
        load_scales(0, true);
#pragma unroll
        for (int q = 0; q < S - 1; q++)
            load_all(q, q);
        arrived_all<(S - 2) * kAll>();
        for (int b = 0; b < rounds; b++) {
            load_scales((b & ~3) + 4, (b & 3) == 0);
            load_all((b + S - 1) % S, b + S - 1);
            arrived_all<(S - 2) * kAll>();
        }
        arrived_all<0>();
        if (KS > 1)
            __syncthreads();
        return;
    }
    if constexpr (T::P > 0) {
        arrived_all<63>();
    } else {
        load_scales(0, true);
#pragma unroll
        for (int q = 0; q < S; q++) {
#pragma unroll
            for (int u = 0; u < kFirst; u++)
                load_first(q, q, u);
            if (q == S - 1)
                arrived_all<(S - 1) * (kFirst + kSecond)>();
#pragma unroll
            for (int u = 0; u < kSecond; u++)
                load_second(q, q, u);
        }
    }
#pragma unroll
    for (int i = 0; i < kAhead; i++)
        read_w(0, i);
#pragma unroll
    for (int j = 0; j < MJ; j++)
        read_x(0, j);
    read_scales(0);
    constexpr int kChunk = 60; // a multiple of S
    for (int b0 = 0; b0 < rounds; b0 += kChunk) {
        load_w_scales(b0);
        const int end = min(b0 + kChunk, rounds);
        int b = b0;
        for (; b + S <= end; b += S) {
            block(std::integral_constant<int, 0>{}, b0, b);
            block(std::integral_constant<int, 1>{}, b0, b + 1);
            if constexpr (S > 2)
                block(std::integral_constant<int, 2 % S>{}, b0, b + 2);
            if constexpr (S > 3)
                block(std::integral_constant<int, 3 % S>{}, b0, b + 3);
        }
        if (b < end)
            block(std::integral_constant<int, 0>{}, b0, b);
        if (S > 2 && b + 1 < end)
            block(std::integral_constant<int, 1>{}, b0, b + 1);
        if (S > 3 && b + 2 < end)
            block(std::integral_constant<int, 2 % S>{}, b0, b + 2);
    }
#pragma unroll
    for (int t = -kLag; t < 0; t++)
        additions(t);
    arrived_all<0>(); // loads past the last block write to LDS, too

    // ---- the groups' sums, in their order
    if constexpr (KS > 1) {
        static_assert(KS == 1 || T::kWaves * NI * MJ * 1024 <= S * kStage);
        const uint32_t at = wave * (NI * MJ * 1024) + lane * 16;
        if (group > 0) {
#pragma unroll
            for (int t = 0; t < kTiles; t++)
                lds_write(base + at + 1024 * t, acc[t / MJ][t % MJ]);
        }
        __syncthreads();
        if (group > 0)
            return;
#pragma unroll
        for (int q = 1; q < KS; q++)
#pragma unroll
            for (int t = 0; t < kTiles; t++)
                acc[t / MJ][t % MJ] += lds_read<v4f>(base + q * kGroup + at + 1024 * t, 0);
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
    // Results go through this wave's own part of LDS, so that a store is 16 bytes
    // a lane of whole rows: straight from the registers it would be 32 bytes of
    // each of 16 rows.  The 16-byte pieces of a row are stored in the order
    // piece ^ row, as above.
    constexpr int kValue = STORE == kCodes ? 1 : STORE == kF32 ? 4 : 2, kPerPiece = 16 / kValue;
    constexpr int kRow = 16 * NO * kValue, kPieces = kRow / 16; // bytes, 16-byte pieces
    const uint32_t mine = base + wave * (16 * MJ * kRow);
    // (A part of K's sums of the largest tiles do not fit: 64 bytes of each row.)
    constexpr bool kFits = T::kWaves * 16 * MJ * kRow + 4 * T::NW * T::kRowsX <= kGroup;
    static_assert(kFits || STORE == kF32);
    auto put = [&](int i, int j, auto v) { // columns 16 i + 4 g .. + 3 of row 16 j + r
        const int line = 16 * j + r, at = (16 * i + 4 * g) * kValue;
        lds_write(mine + line * kRow + ((at / 16) ^ (line % kPieces)) * 16 + at % 16, v);
    };
    auto store = [&](void *y, int64_t ldy) {
        constexpr int kLines = 64 / kPieces; // rows per instruction
#pragma unroll
        for (int q = 0; q < 16 * MJ / kLines; q++) {
            const int line = q * kLines + lane / kPieces, c = lane % kPieces;
            const v4i v = lds_read<v4i>(mine + line * kRow + (c ^ (line % kPieces)) * 16, 0);
            const int64_t row = m0 + 16 * wm * MJ + line, n = col0 + c * kPerPiece;
            if (row >= p.m || n >= p.n)
                continue;
            uint8_t *to = static_cast<uint8_t *>(y) + (row * ldy + n) * kValue;
            if (n + kPerPiece <= p.n) {
                __builtin_memcpy(__builtin_assume_aligned(to, kValue), &v, 16);
            } else {
                const int left = (int)(p.n - n);
                for (int e = 0; e < left; e++) {
                    const uint32_t word = (uint32_t)v[e * kValue / 4] >> (8 * (e * kValue % 4));
                    if constexpr (kValue == 4)
                        reinterpret_cast<uint32_t *>(to)[e] = word;
                    else if constexpr (kValue == 2)
                        reinterpret_cast<uint16_t *>(to)[e] = (uint16_t)word;
                    else
                        to[e] = (uint8_t)word;
                }
            }
        }
    };
    if constexpr (STORE == kCodes) {
        // a block of 128 columns: the waves of a row tile share its maximum
        static_assert(STORE != kCodes || (kCols == 128 && KS == 1));
        const uint32_t tops = base + kGroup - 4 * T::NW * T::kRowsX;
        uint32_t top[MJ];
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
            top[j] = max(a, (uint32_t)__shfl_xor((int)a, 32));
            if (g == 0)
                lds_write(tops + 4 * (wn * T::kRowsX + 16 * (wm * MJ + j) + r), top[j]);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < MJ; j++) {
            const int line = 16 * (wm * MJ + j) + r;
#pragma unroll
            for (int o = 0; o < T::NW; o++)
                top[j] = max(top[j], lds_read<uint32_t>(tops + 4 * (o * T::kRowsX + line), 0));
            const float d = __uint_as_float(top[j]) / 448.0f;
            const float inv = d > 0.0f ? fminf(1.0f / d, FLT_MAX) : 0.0f;
            if (wn == 0 && g == 0 && m0 + line < p.m)
                out_scales[(m0 + line) * fp8_blocks(p.n) + n0 / kFp8Block] = d;
#pragma unroll
            for (int i = 0; i < NO; i++) {
                const v4f v = acc[i][j] * inv;
                int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
                put(i, j, __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], c, true));
            }
        }
        store(out_codes, p.n);
    } else if constexpr (!kFits) {
        float *y = static_cast<float *>(p.y) + blockIdx.y * (p.m * p.ldy);
#pragma unroll
        for (int j = 0; j < MJ; j++) {
            const int64_t line = m0 + 16 * (wm * MJ + j) + r;
#pragma unroll
            for (int i = 0; i < NO; i++) {
                const int64_t n = col0 + 16 * i + 4 * g; // p.ldy is n's next multiple of 4
                if (line < p.m && n < p.n)
                    *reinterpret_cast<v4f *>(y + line * p.ldy + n) = acc[i][j];
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < MJ; j++)
#pragma unroll
            for (int i = 0; i < NO; i++) {
                const v4f v = acc[i][j];
                if constexpr (STORE == kF32)
                    put(i, j, v);
                else
                    put(i, j, v2u{bf16_bits(v[0]) | bf16_bits(v[1]) << 16,
                                  bf16_bits(v[2]) | bf16_bits(v[3]) << 16});
            }
        store(static_cast<uint8_t *>(p.y) + blockIdx.y * (p.m * p.ldy * kValue), p.ldy);
    }
}

typedef Tile<8, 4, 2, 4, 1, 2> Tile256x256;
typedef Tile<4, 4, 2, 2, 1, 4, 4> Tile128x128;
typedef Tile<4, 4, 2, 2, 1, 2> Tile128x128Pair; // two workgroups a CU
typedef Tile<2, 2, 4, 2, 1, 4, 4> Tile64x128;
typedef Tile<2, 2, 2, 2, 2, 4, 2> Tile64x64; // two halves of K
typedef Tile<4, 4, 4, 1, 1, 3> Tile64x256;

template <class T, bool GATED, bool EXACT, Store STORE>
hipError_t launch_tile(const Fp8Problem &p, const Fp8Part &part, uint8_t *codes, float *scales,
                       hipStream_t s)
{
    constexpr int kCols = T::kRowsW / (GATED ? 2 : 1);
    const int64_t tiles =
        (p.m + T::kRowsX - 1) / T::kRowsX * ((part.cols + kCols - 1) / kCols);
    const int64_t blocks = fp8_blocks(p.k), splits = part.splits > 1 ? part.splits : 1;
    fp8_tile_kernel<T, GATED, EXACT, STORE>
        <<<dim3((unsigned)tiles, (unsigned)splits), T::kThreads, 0, s>>>(
            p, part.first, part.cols, (int)((blocks + splits - 1) / splits), codes, scales);
    return hipGetLastError();
}

template <class T, bool EXACT>
hipError_t launch_values(const Fp8Problem &p, const Fp8Part &part, hipStream_t s)
{
    constexpr Store STORE = EXACT ? kF32 : kBf16;
    return p.up ? launch_tile<T, true, EXACT, STORE>(p, part, nullptr, nullptr, s)
                : launch_tile<T, false, EXACT, STORE>(p, part, nullptr, nullptr, s);
}

// What a tile costs, in us on an MI355X: `fixed`, and per block of K with few
// tiles on the chip (`light`) and with as many as it holds at once (`full`,
// `slots` of them).  Fitted to 5120 x 5120 to 17408 x 5120 with 128 to 8192
// rows; products whose codes are widened take longer.  A head's 131072 columns of
// K = 5120 take 313, 323 and 600 us for 333, 512 and 1024 rows with them (1430,
// 2130 and 2290 TF), fp32 469, 622 and 1198; 64 rows 150 and 162 (4.5 TB/s).
struct Cost {
    int kernel, rows, cols, slots;
    float fixed, light, full;
};
constexpr Cost kFast[] = {
    {kFp8Tile256x256, 256, 256, 256, 5.0f, 1.24f, 1.60f},
    {kFp8Tile128x128Pair, 128, 128, 512, 3.5f, 0.52f, 1.05f},
    {kFp8Tile128x128, 128, 128, 256, 4.0f, 0.46f, 0.75f},
    {kFp8Tile64x128, 64, 128, 256, 3.0f, 0.36f, 0.46f},
    {kFp8Tile64x64, 64, 64, 256, 3.0f, 0.25f, 0.30f},
};
constexpr Cost kExact[] = {
    {kFp8Tile128x128Pair, 128, 128, 512, 3.5f, 1.20f, 1.75f},
    {kFp8Tile64x128, 64, 128, 256, 3.0f, 0.62f, 0.62f},
    {kFp8Tile64x64, 64, 64, 256, 3.0f, 0.38f, 0.36f},
};
// a gated product's codes: blocks of 128 columns, so tiles of 128 and 128 ...
constexpr Cost kToCodes[] = {
    {kFp8Tile256x256, 256, 256, 256, 5.0f, 1.24f, 1.60f},
    {kFp8Tile64x256, 64, 256, 256, 4.0f, 0.65f, 0.75f},
};
// ... or fp32 values in smaller ones, quantized by another launch
constexpr Cost kStaged[] = {
    {kFp8Tile64x128, 64, 128, 256, 3.0f, 0.36f, 0.46f},
    {kFp8Tile64x64, 64, 64, 256, 3.0f, 0.25f, 0.30f},
};
constexpr float kLaunch = 2.0f; // another launch behind one
constexpr int kMaxSplits = 16;  // parts of K

int64_t tiles_of(const Cost &c, int64_t m, int64_t cols, int g)
{
    const int64_t each = c.cols / g;
    return (m + c.rows - 1) / c.rows * ((cols + each - 1) / each);
}

float time_of(const Cost &c, int64_t tiles, int64_t blocks)
{
    const int64_t full = tiles / c.slots, rest = tiles % c.slots;
    float t = (float)full * (c.fixed + c.full * (float)blocks);
    if (rest > 0)
        t += c.fixed + (c.light + (c.full - c.light) * (float)rest / (float)c.slots) * (float)blocks;
    return t;
}

// The quickest of `costs` for `cols` columns, and its time.
template <int N>
float best_of(const Cost (&costs)[N], const Fp8Problem &p, int64_t cols, int *kernel)
{
    float best = 0;
    for (int i = 0; i < N; i++) {
        const float t = time_of(costs[i], tiles_of(costs[i], p.m, cols, p.up ? 2 : 1), fp8_blocks(p.k));
        if (i == 0 || t < best) {
            best = t;
            *kernel = costs[i].kernel;
        }
    }
    return best;
}

template <int N> float plan(const Cost (&costs)[N], const Fp8Problem &p, Fp8Plan *plan)
{
    *plan = Fp8Plan{};
    plan->part[0].cols = p.n;
    const float whole = best_of(costs, p, p.n, &plan->part[0].kernel);
    // The largest tiles (the first of the list) for as many columns as fill the
    // chip in whole rounds, and the quickest for the rest: 1024 x 17408 x 5120
    // gated is 2.1 rounds, 208 us as three and 192 us as two and a rest.
    const Cost &c = costs[0];
    const int64_t each = c.cols / (p.up ? 2 : 1), down = (p.m + c.rows - 1) / c.rows;
    const int64_t rounds = tiles_of(c, p.m, p.n, p.up ? 2 : 1) / c.slots;
    const int64_t cols = rounds * c.slots / down * each;
    if (cols > 0 && cols < p.n) {
        Fp8Plan split{};
        split.part[0] = {c.kernel, 0, cols};
        split.part[1] = {0, cols, p.n - cols};
        const float t = time_of(c, cols / each * down, fp8_blocks(p.k)) + kLaunch +
                        best_of(costs, p, p.n - cols, &split.part[1].kernel);
        if (t < whole) {
            *plan = split;
            return t;
        }
    }
    return whole;
}

// Tiles over a part of K each, where there are few of them: the sums are written
// and read again, at 5 TB/s.  In us, without and with: rows x columns x K
// 1024 x 5120 x 17408, 80 tiles of 256x256, 143 and 101; 64 x 5120 x 17408 35 and
// 25; 96 x 1024 x 16384 29 and 14; fp32 results 256 x 5120 x 17408 79 and 58.
// Replaces *plan where that is quicker than `best`.
template <int N>
void split_k(const Cost (&costs)[N], const Fp8Problem &p, float best, Fp8Plan *plan)
{
    const int64_t blocks = fp8_blocks(p.k);
    const float value = p.y_bf16 ? 2 : 4; // bytes of a result
    for (const Cost &c : costs) {
        // one 128x128 a CU, with its loads further ahead, is the quicker of the two
        // there: 520 x 5000 x 7808 33 us, two a CU 44
        if (c.kernel == kFp8Tile128x128Pair && !p.exact)
            continue;
        const int64_t tiles = tiles_of(c, p.m, p.n, 1);
        for (int splits = 2; splits <= kMaxSplits && tiles * splits <= 2 * c.slots; splits++) {
            const int64_t each = (blocks + splits - 1) / splits;
            if (each < 8)
                break;
            if ((splits - 1) * each >= blocks)
                continue; // the last would have none
            const float t = time_of(c, tiles * splits, each) + kLaunch +
                            (float)(p.m * p.n) * ((float)(8 * splits) + value) / 5e6f;
            if (t < best) {
                best = t;
                *plan = Fp8Plan{};
                plan->part[0] = {c.kernel, 0, p.n, splits};
            }
        }
    }
}

// columns of a row of a part's sums
int64_t sums_ld(int64_t n) { return (n + 3) / 4 * 4; }

// y = the splits' sums [splits][m][ld], in their order
template <bool BF16>
__global__ __launch_bounds__(256) void fp8_join_kernel(const float *sums, int splits, int64_t m,
                                                       int64_t n, int64_t ld, void *y, int64_t ldy)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= m * ld)
        return;
    v4f sum = *reinterpret_cast<const v4f *>(sums + i);
    for (int q = 1; q < splits; q++)
        sum += *reinterpret_cast<const v4f *>(sums + q * m * ld + i);
    const int64_t col = i % ld, at = i / ld * ldy + col;
    if constexpr (BF16) {
        uint16_t *to = static_cast<uint16_t *>(y) + at;
        const v2u v{bf16_bits(sum[0]) | bf16_bits(sum[1]) << 16,
                    bf16_bits(sum[2]) | bf16_bits(sum[3]) << 16};
        if (col + 4 <= n)
            __builtin_memcpy(__builtin_assume_aligned(to, 2), &v, 8);
        else
            for (int e = 0; e < (int)(n - col); e++)
                to[e] = (uint16_t)(v[e / 2] >> (16 * (e % 2)));
    } else {
        float *to = static_cast<float *>(y) + at;
        if (col + 4 <= n)
            __builtin_memcpy(__builtin_assume_aligned(to, 4), &sum, 16);
        else
            for (int e = 0; e < (int)(n - col); e++)
                to[e] = sum[e];
    }
}

hipError_t launch_part(const Fp8Problem &p, const Fp8Part &part, hipStream_t s)
{
    if (p.exact) {
        switch (part.kernel) {
        case kFp8Tile128x128Pair: return launch_values<Tile128x128Pair, true>(p, part, s);
        case kFp8Tile64x128: return launch_values<Tile64x128, true>(p, part, s);
        default: return launch_values<Tile64x64, true>(p, part, s);
        }
    }
    if (!p.y_bf16 && p.up) { // the values of a staged gated product
        return part.kernel == kFp8Tile64x128
                   ? launch_tile<Tile64x128, true, false, kF32>(p, part, nullptr, nullptr, s)
                   : launch_tile<Tile64x64, true, false, kF32>(p, part, nullptr, nullptr, s);
    }
    if (!p.y_bf16) { // the sums of parts of K
        switch (part.kernel) {
        case kFp8Tile256x256:
            return launch_tile<Tile256x256, false, false, kF32>(p, part, nullptr, nullptr, s);
        case kFp8Tile128x128:
            return launch_tile<Tile128x128, false, false, kF32>(p, part, nullptr, nullptr, s);
        case kFp8Tile64x128:
            return launch_tile<Tile64x128, false, false, kF32>(p, part, nullptr, nullptr, s);
        default: return launch_tile<Tile64x64, false, false, kF32>(p, part, nullptr, nullptr, s);
        }
    }
    switch (part.kernel) {
    case kFp8Tile256x256: return launch_values<Tile256x256, false>(p, part, s);
    case kFp8Tile128x128Pair: return launch_values<Tile128x128Pair, false>(p, part, s);
    case kFp8Tile128x128: return launch_values<Tile128x128, false>(p, part, s);
    case kFp8Tile64x128: return launch_values<Tile64x128, false>(p, part, s);
    default: return launch_values<Tile64x64, false>(p, part, s);
    }
}

// Few rows, and few enough columns for a workgroup per 16 of them, or a long K
// and 16 rows at most, which leave two workgroups a CU: otherwise workgroups that
// begin and end take longer than the weights.  In us, streamed and (in tiles),
// weights in the last cache where they fit, K = 5120 but where another is named:
//   8192 columns     1 row 8.8 (12.8), 16 8.9 (13.4), 32 12.2 (13.7);
//                    K = 160 16 rows 4.3 (5.3), 32 5.6 (5.4)
//   17408            1 to 16 rows 17 (17), fp32 17 (27), 32 rows 26 (18);
//                    K = 1024 16 rows 9.3 (6.5), fp32 9.3 (9.2), 1 row 7.5 (9.0)
//   49152            16 rows 38 (41), fp32 38 (49); K = 1024 18 (13)
//   131072           1 row 115 (121), 4 120 (122), 8 126 (119), 16 154 (120);
//                    fp32 113 (129), 119 (130), 124 (126), 155 (129);
//                    K = 160 16 rows 37 (11)
// A gated product of 16 rows at most always streams: its codes come from products
// added in fp32.
bool streams(const Fp8Problem &p)
{
    if (p.m <= kFp8StreamRows && p.n * (p.up ? 2 : 1) <= 8192)
        return true;
    if (p.m > 16 || p.up)
        return p.m <= 16;
    return fp8_blocks(p.k) >= (p.exact ? 8 : 32) && (p.n <= 49152 || p.m <= 4);
}

Fp8Plan streamed(const Fp8Problem &p)
{
    Fp8Plan plan{};
    plan.part[0] = {kFp8Stream, 0, p.n};
    return plan;
}

} // namespace

Fp8Plan plan_fp8_gemm(const Fp8Problem &p)
{
    if (p.m == 0)
        return Fp8Plan{};
    if (streams(p))
        return streamed(p);
    Fp8Plan values;
    const float whole = p.exact ? plan(kExact, p, &values) : plan(kFast, p, &values);
    if (p.up)
        return values;
    if (p.exact)
        split_k(kExact, p, whole, &values);
    else
        split_k(kFast, p, whole, &values);
    return values;
}

Fp8Plan plan_fp8_codes(const Fp8Problem &p)
{
    if (p.m == 0)
        return Fp8Plan{};
    Fp8Plan codes, values{};
    if (streams(p)) {
        values = streamed(p);
        values.staged = true;
        return values;
    }
    const float direct = plan(kToCodes, p, &codes);
    // the values are written and read by the quantizer's launch, at 4 TB/s
    values.staged = true;
    values.part[0].cols = p.n;
    const float staged = best_of(kStaged, p, p.n, &values.part[0].kernel) + kLaunch +
                         (float)(p.m * p.n) * (9.0f / 4e6f);
    return staged < direct ? values : codes;
}

const char *fp8_plan_name(const Fp8Plan &plan)
{
    static const char *const one[] = {"none",           "stream",      "tile 256x256",
                                      "tile 128x128 pair", "tile 128x128", "tile 64x128",
                                      "tile 64x64",     "tile 64x256"};
    // the first columns' kernel is the one with the largest tiles there
    static const char *const behind[] = {"",
                                         "",
                                         "tile 256x256, then tile 256x256",
                                         "tile 256x256, then tile 128x128 pair",
                                         "tile 256x256, then tile 128x128",
                                         "tile 256x256, then tile 64x128",
                                         "tile 256x256, then tile 64x64",
                                         "tile 256x256, then tile 64x256"};
    static const char *const pairs[] = {"",
                                        "",
                                        "",
                                        "tile 128x128 pair, then tile 128x128 pair",
                                        "",
                                        "tile 128x128 pair, then tile 64x128",
                                        "tile 128x128 pair, then tile 64x64",
                                        ""};
    const Fp8Part &first = plan.part[0], &rest = plan.part[1];
    if (rest.cols > 0)
        return (first.kernel == kFp8Tile256x256 ? behind : pairs)[rest.kernel];
    static const char *const parts[] = {"",
                                        "",
                                        "tile 256x256 over parts of K",
                                        "tile 128x128 pair over parts of K",
                                        "tile 128x128 over parts of K",
                                        "tile 64x128 over parts of K",
                                        "tile 64x64 over parts of K",
                                        ""};
    return (first.splits > 1 ? parts : one)[first.kernel];
}

namespace {

hipError_t launch_plan(const Fp8Problem &p, const Fp8Plan &plan, hipStream_t s)
{
    for (const Fp8Part &part : plan.part) {
        if (part.cols == 0)
            continue;
        const hipError_t e =
            part.kernel == kFp8Stream ? launch_fp8_stream(p, s) : launch_part(p, part, s);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace

size_t fp8_gemm_bytes(const Fp8Problem &p)
{
    const int64_t splits = plan_fp8_gemm(p).part[0].splits;
    return splits > 1 ? (size_t)(splits * p.m * sums_ld(p.n)) * sizeof(float) : 0;
}

hipError_t launch_fp8_gemm(const Fp8Problem &p, void *workspace, hipStream_t s)
{
    const Fp8Plan plan = plan_fp8_gemm(p);
    const int splits = plan.part[0].splits;
    if (splits < 2)
        return launch_plan(p, plan, s);
    Fp8Problem sums = p;
    sums.y = workspace;
    sums.ldy = sums_ld(p.n);
    sums.y_bf16 = false;
    const hipError_t e = launch_part(sums, plan.part[0], s);
    if (e != hipSuccess)
        return e;
    (p.y_bf16 ? fp8_join_kernel<true> : fp8_join_kernel<false>)<<<
        (unsigned)((p.m * sums.ldy / 4 + 255) / 256), 256, 0, s>>>(
        static_cast<const float *>(workspace), splits, p.m, p.n, sums.ldy, p.y, p.ldy);
    return hipGetLastError();
}

size_t fp8_gated_quantize_bytes(const Fp8Problem &p)
{
    return plan_fp8_codes(p).staged ? (size_t)p.m * (size_t)p.n * sizeof(float) : 0;
}

hipError_t launch_fp8_gated_quantize(const Fp8Problem &p, uint8_t *codes, float *scales,
                                     void *workspace, hipStream_t s)
{
    const Fp8Plan plan = plan_fp8_codes(p);
    if (plan.staged) {
        Fp8Problem values = p;
        values.y = workspace;
        values.ldy = p.n;
        // Few rows wait for memory, so their products may as well be added in fp32:
        // a value next to a border of e4m3 moves by a whole step if it is a little
        // off, and one row's down projection does not average that out.
        values.exact = plan.part[0].kernel == kFp8Stream;
        const hipError_t e = launch_plan(values, plan, s);
        if (e != hipSuccess)
            return e;
        return launch_fp8_quantize(workspace, false, p.m, p.n, p.n, false, codes, scales, s);
    }
    for (const Fp8Part &part : plan.part) {
        hipError_t e = hipSuccess;
        if (part.cols > 0 && part.kernel == kFp8Tile256x256)
            e = launch_tile<Tile256x256, true, false, kCodes>(p, part, codes, scales, s);
        else if (part.cols > 0)
            e = launch_tile<Tile64x256, true, false, kCodes>(p, part, codes, scales, s);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace bpg
