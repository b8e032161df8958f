// logprobs.hip -- log probabilities of given tokens, entropies and top
// alternatives of rows of logits (gfx950).
//
//   m = max l, R = sum e^(l - m) without one of the largest, T = sum (l - m) e^(l - m)
//   log p(t) = l_t - m - log1p(R),  entropy = log1p(R) - T / (1 + R)
//
// T <= 0 and R >= 0, so nothing cancels: where one token is nearly certain, its
// log probability and the entropy keep the digits of R and T.  The top
// alternatives are the largest logits, equal ones by the lowest id; a NaN counts
// as -inf there.  A row with a NaN or +inf, or of -inf only, has no distribution:
// NaN.
//
// One pass over the logits: a thread holds 16 at a time and has 16 more on the
// way, takes their maximum, rescales its sums to it and adds the 16 terms (in fp32
// among the 16, in fp64 from one 16 to the next).  These sums hold the largest
// logit's own term, with an error of fp32; where R is not well above it, the wave
// reads the logits of the thread that has the largest again and leaves it out.
//
// For the alternatives a thread leaves each 16's maximum in LDS.  The k-th
// largest of 64 (or 128) groups' maxima is then below or at the k-th largest
// logit, and few logits reach it (64 ln (64 / (64 - k)) on shuffled rows: 24 for
// k = 20), so only the 16s that do are read again.  A mask may leave fewer than k
// groups open: then the open logits and the lowest masked ids are taken.  Where
// many groups have the k-th maximum itself (a mask's finite value, rows of few
// values), or more than kCandidates logits reach it, the logits above it are
// taken and, in the order of their ids, as many equal ones as are missing.  With
// ten open logits and 20 alternatives 64 x 131072 takes 21 to 22 us and 1024 rows
// 59 to 61, as without a mask.  If too many are above it even so (thousands of
// open logits in fewer than k groups), the alternatives are found one scan of the
// part each.
//
// Few rows are split into parts of 8192 logits or more, a workgroup each, and
// another launch joins them.
//
// Bound by memory where there are many rows: 4096 x 131072 bf16, 1.07 GB, 200 us
// (5.4 TB/s; 195 to 215 with an alternative), fp32 2048 x 131072 186 us (5.8 TB/s).
// Few or short rows are bound by the chain of their steps: the sums over a
// workgroup, the k-th of the groups' maxima, the ranks, the join (1 x 131072 with
// 20 alternatives 12 us, 333 x 50001 with 5 18 us, a quarter of it masked 19, 16 x
// 262144 with 64 25 us).  Rows whose largest logit has nearly all of the
// probability read a thread's logits again: 333 x 50001 19 us, 4096 x 131072 207,
// 8192 x 1000 fp32 with 5 alternatives 23.6 instead of 21.
#include "fp8.h"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace bpg {
namespace {

constexpr int kEach = 16;  // logits a thread holds at once
constexpr int kSteps = 32; // of a workgroup, at most
constexpr int kCandidates = 1024;
constexpr int kMaxParts = 64;
constexpr float kLog2e = 1.44269504f; // log2 e to 2^-26

// Up to here m log2 e is at most 1 from the float next to it, which the sums are
// taken about; far beyond, 2^x of the largest logit itself would leave fp32.
constexpr float kFarRef = 16777216.0f;

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// What a thread has: sums of 2^x and x 2^x, x = l log2 e - ref.  The reference is
// m log2 e, or up to kFarRef the float next to it: x is then one FMA, with one
// rounding relative to x.
struct Sums {
    double ref;
    double s, t; // 0 where m is -inf; NaN with a NaN or +inf among them
    float m;     // the largest logit, -inf if there is none
};

// What a part of a row amounts to, x = (l - m) log2 e: sums of 2^x over all
// logits but one of the largest, and of x 2^x.
struct Part {
    double s, t; // as above
    float m;
};

// The largest logit's own term leaves up to ten roundings of 2^-24 in a thread's
// s (the sum of 16, the exponential, the reference): from here on that is 2^-18
// of the rest at most.
constexpr double kClose = 1.0 / 4;

// An order of the logits and their ids in one word: larger words are larger
// logits, or the lower id of equal ones.  No logit has word 0.
__device__ __forceinline__ uint64_t word_of(float v, uint32_t id)
{
    uint32_t u = __float_as_uint(v == v ? v + 0.0f : -INFINITY); // -0 becomes 0
    u = u & 0x80000000u ? ~u : u | 0x80000000u;
    return (uint64_t)u << 32 | (~id);
}

__device__ __forceinline__ float logit_of(uint64_t word)
{
    const uint32_t u = (uint32_t)(word >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ double reference(float m)
{
    return fabsf(m) < INFINITY ? (double)m * kLog2e : 0.0;
}

// a DPP move of both halves; lanes without a source keep `old`
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_double(double old, double v)
{
    const uint64_t o = __builtin_bit_cast(uint64_t, old), u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)o, (int)(uint32_t)u,
                                                              CTRL, ROWS, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(
        (int)(uint32_t)(o >> 32), (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// the sum over a wave, in its last lane: shifts by 1, 2, 4, 8 within 16 lanes,
// then the last lane of 16 to the next 16, of 32 to the next 32
__device__ __forceinline__ double sum_to_last(double v)
{
    v += dpp_double<0x111, 0xf>(0.0, v);
    v += dpp_double<0x112, 0xf>(0.0, v);
    v += dpp_double<0x114, 0xf>(0.0, v);
    v += dpp_double<0x118, 0xf>(0.0, v);
    v += dpp_double<0x142, 0xa>(0.0, v);
    v += dpp_double<0x143, 0xc>(0.0, v);
    return v;
}

template <int CTRL> __device__ __forceinline__ float max_dpp(float v)
{
    return fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
                        (int)__float_as_uint(v), (int)__float_as_uint(v), CTRL, 0xf, 0xf, false)));
}

// the maximum over a wave, in every lane
__device__ __forceinline__ float wave_max(float v)
{
    v = max_dpp<0x128>(v);
    v = max_dpp<0x124>(v);
    v = max_dpp<0x122>(v);
    v = max_dpp<0x121>(v);
    v = max_dpp<0x142>(v);
    v = max_dpp<0x143>(v);
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// sums about a maximum that is not smaller
__device__ __forceinline__ void rescale(Sums &p, float m, double ref)
{
    const double d = p.m == -INFINITY ? 0.0 : p.ref - ref;
    const double e = __builtin_amdgcn_exp2f((float)d);
    p.t = (p.t + d * p.s) * e;
    p.s *= e;
    p.m = m;
    p.ref = ref;
}

__device__ __forceinline__ double last_lane(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// the lanes' s and t as one part, in every lane
__device__ __forceinline__ Part over_lanes(double s, double t, float m)
{
    return Part{last_lane(sum_to_last(s)), last_lane(sum_to_last(t)), m};
}

// The threads of a wave as one part, in every lane.  again(lane, m, s, t): adds
// the terms of one lane's logits, without the largest, to s and t, each lane a
// share of them.
template <class F> __device__ __forceinline__ Part over_wave(Sums p, F &&again)
{
    const float m = wave_max(p.m);
    const int owner = __builtin_ctzll(__ballot(p.m == m)); // p.m is no NaN
    rescale(p, m, reference(m));
    const bool mine = (int)(threadIdx.x & 63) == owner && m > -INFINITY;
    const Part all = over_lanes(mine ? p.s - 1.0 : p.s, p.t, m);
    if (!(all.s < kClose) || m == -INFINITY)
        return all;
    double s = mine ? 0.0 : p.s, t = mine ? 0.0 : p.t;
    again(owner, m, s, t);
    return over_lanes(s, t, m);
}

// parts of one row in LDS as one, a lane each (64 at most), in every lane
__device__ __forceinline__ Part over_parts(const Part *parts, int count)
{
    Part p{0.0, 0.0, -INFINITY};
    const int lane = threadIdx.x & 63;
    if (lane < count)
        p = parts[lane];
    const float m = wave_max(p.m);
    const int owner = __builtin_ctzll(__ballot(p.m == m));
    if (lane != owner && p.m > -INFINITY) {
        const double d = ((double)p.m - m) * kLog2e, s = p.s + 1.0;
        const double e = __builtin_amdgcn_exp2f((float)d);
        p.t = (p.t + d * s) * e;
        p.s = s * e;
    }
    return over_lanes(p.s, p.t, m);
}

// Sixteen logits of a thread in a step: groups of one 16-byte load each, the
// threads' groups side by side.  Rows of more than one wave are loaded without a
// branch, so that loads of later steps can be on the way: a group that would
// pass the end is the last whole one instead, less what is not its own.
template <bool BF16, int THREADS> struct Step {
    static constexpr int kGroups = BF16 ? 2 : 4, kPer = kEach / kGroups;
    static constexpr bool kWhole = THREADS > 64; // of a row of kPer logits or more
    v4u raw[kGroups];
    static __device__ __forceinline__ int64_t id(int64_t at, int q, int thread)
    {
        return at + (int64_t)q * (THREADS * kPer) + thread * kPer;
    }
    // logit e of group q of the step that begins at `at`: is it the group's own?
    static __device__ __forceinline__ bool own(int64_t at, int q, int e, int64_t end)
    {
        return kWhole ? id_of(at, q, e, end) >= id(at, q, threadIdx.x) : id(at, q, threadIdx.x) + e < end;
    }
    static __device__ __forceinline__ int64_t id_of(int64_t at, int q, int e, int64_t end)
    {
        return (kWhole ? min(id(at, q, threadIdx.x), end - kPer) : id(at, q, threadIdx.x)) + e;
    }
    static __device__ __forceinline__ const uint8_t *address(const void *row, int64_t i)
    {
        return static_cast<const uint8_t *>(row) + i * (BF16 ? 2 : 4);
    }
    __device__ __forceinline__ void load(const void *row, int64_t at, int64_t end)
    {
#pragma unroll
        for (int q = 0; q < kGroups; q++) {
            const int64_t i = id_of(at, q, 0, end);
            if (kWhole || i + kPer <= end) {
                __builtin_memcpy(&raw[q], __builtin_assume_aligned(address(row, i), BF16 ? 2 : 4), 16);
                continue;
            }
#pragma unroll
            for (int e = 0; e < kPer; e++) {
                uint32_t v = BF16 ? 0xff80u : 0xff800000u; // -inf
                if (i + e < end)
                    v = BF16 ? *reinterpret_cast<const uint16_t *>(address(row, i + e))
                             : *reinterpret_cast<const uint32_t *>(address(row, i + e));
                if (BF16)
                    raw[q][e / 2] = e & 1 ? raw[q][e / 2] | v << 16 : v;
                else
                    raw[q][e] = v;
            }
        }
    }
    // -inf for those that are not the thread's own
    __device__ __forceinline__ void values(float (&v)[kEach], int64_t at, int64_t end) const
    {
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const uint32_t w = raw[i / kPer][BF16 ? i % kPer / 2 : i % kPer];
            v[i] = __uint_as_float(!BF16 ? w : i & 1 ? w & 0xffff0000u : w << 16);
        }
        if (kWhole && at + THREADS * kEach > end) {
#pragma unroll
            for (int i = 0; i < kEach; i++)
                v[i] = own(at, i / kPer, i % kPer, end) ? v[i] : -INFINITY;
        }
    }
};

template <bool BF16> __device__ __forceinline__ float logit(const void *row, int64_t i)
{
    return BF16 ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(row)[i] << 16)
                : static_cast<const float *>(row)[i];
}

// the next float above one that is not -inf; NaN above +inf
__device__ __forceinline__ float next_above(float v)
{
    const uint32_t u = __float_as_uint(v);
    return __uint_as_float(v == 0.0f ? 1u : u & 0x80000000u ? u - 1 : u + 1);
}

// the upper half of a float, rounded up
__device__ __forceinline__ uint16_t above(float v)
{
    const uint32_t u = __float_as_uint(v);
    return (uint16_t)((u & 0x80000000u ? u : u + 0xffffu) >> 16);
}

template <int N> __device__ __forceinline__ float sum_of(const float (&v)[N])
{
    float a[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; i++)
        a[i] = v[i] + v[i + N / 2];
    if constexpr (N == 2)
        return a[0];
    else
        return sum_of<N / 2>(a);
}

// The logit of row r's token, NaN for one outside the vocabulary.
struct Token {
    float logit;
    bool none; // a position without a token
};

template <bool BF16>
__device__ __forceinline__ Token token_of(const LogprobsProblem &p, int64_t r, const void *row)
{
    if (!p.tokens)
        return Token{NAN, true};
    const int64_t id = p.wide ? static_cast<const int64_t *>(p.tokens)[r]
                              : static_cast<const int32_t *>(p.tokens)[r];
    return Token{id < 0 || id >= p.vocab ? NAN : logit<BF16>(row, id), id < 0};
}

// log S, NaN for a row without a distribution
__device__ __forceinline__ double log_sum(const Part &all)
{
    return all.m == -INFINITY ? NAN : log1p(all.s);
}

__device__ __forceinline__ float log_probability(const Part &all, double log_s, float logit)
{
    return (float)((double)logit - all.m - log_s);
}

__device__ __forceinline__ void write_row(const LogprobsProblem &p, int64_t r, const Part &all, double log_s,
                                          Token token)
{
    if (p.entropy)
        p.entropy[r] = (float)(log_s - all.t / (1.0 + all.s) * (1.0 / kLog2e));
    if (p.tokens)
        p.logprobs[r] = token.none ? 0.0f : log_probability(all, log_s, token.logit);
}

template <bool BF16>
__device__ __forceinline__ const void *row_of(const LogprobsProblem &p, int64_t r)
{
    return static_cast<const uint8_t *>(p.logits) + r * p.ldl * (BF16 ? 2 : 4);
}

// Writes rank and word of the words among the k largest of `count` different
// ones, which begin at a multiple of 16 bytes and have room for eight more.
template <int THREADS, class F>
__device__ __forceinline__ void rank_words(uint64_t *words, int count, int k, F &&emit)
{
    typedef uint64_t Pair __attribute__((ext_vector_type(2)));
    if (threadIdx.x < 8)
        words[count + threadIdx.x] = 0; // below every logit
    if (THREADS > 64)
        __syncthreads();
    for (int i = threadIdx.x; i < count; i += THREADS) {
        const uint64_t mine = words[i];
        int rank = 0;
        for (int j = 0; j < count; j += 8) {
            Pair o[4];
#pragma unroll
            for (int u = 0; u < 4; u++)
                o[u] = *reinterpret_cast<const Pair *>(words + j + 2 * u);
#pragma unroll
            for (int u = 0; u < 4; u++)
                rank += (o[u][0] > mine) + (o[u][1] > mine);
        }
        if (rank < k)
            emit(rank, mine);
    }
}

// workgroup (row, part): logits [part * length, ...) of its row.  TOP: with
// alternatives.
template <bool BF16, bool TOP, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void logprobs_kernel(const LogprobsProblem p, int parts,
                                                              int64_t length, Part *out_parts,
                                                              uint64_t *out_words)
{
    constexpr int kThreads = 64 * WAVES, kStep = kThreads * kEach;
    typedef Step<BF16, kThreads> Logits;
    __shared__ Part wave_parts[WAVES];
    __shared__ uint16_t tops[TOP ? kSteps : 1][kThreads];
    __shared__ float groups[WAVES][64], reach;
    __shared__ __attribute__((aligned(16))) uint64_t words[TOP ? kCandidates + 8 : 1];
    __shared__ uint64_t best[WAVES];
    __shared__ int count, equals[WAVES];
    __shared__ bool many;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t r = blockIdx.x / parts, part = blockIdx.x % parts;
    const void *row = row_of<BF16>(p, r);
    const int64_t begin = part * length, end = min(begin + length, p.vocab);
    Token token{NAN, true};
    if (parts == 1 && threadIdx.x == 0)
        token = token_of<BF16>(p, r, row);

    // ---- the sums
    Sums mine{0.0, 0.0, 0.0, -INFINITY};
    int steps = 0;
    bool masked = false;
    auto step = [&](const Logits &now, int64_t at) {
        float v[kEach];
        now.values(v, at, end);
        float top = v[0];
#pragma unroll
        for (int i = 1; i < kEach; i++) // NaN is dropped
            top = fmaxf(top, v[i]);
        if (TOP)
            tops[steps][threadIdx.x] = above(top == top ? top : -INFINITY);
        const float m = fmaxf(mine.m, top);
        const float ref = m * kLog2e;
        float e[kEach], t[4] = {0, 0, 0, 0};
        double by = ref;
        bool again = masked; // logits of -inf or next to it
        if (!masked) { // x is -inf or NaN where it is, and x 2^x NaN
#pragma unroll
            for (int i = 0; i < kEach; i++) {
                const float x = __builtin_fmaf(v[i], kLog2e, -ref);
                e[i] = __builtin_amdgcn_exp2f(x);
                t[i % 4] = __builtin_fmaf(x, e[i], t[i % 4]);
            }
            again = __ballot(!(sum_of(t) > -FLT_MAX) || fabsf(ref) > kFarRef) != 0;
        }
        if (again) { // x held to -250 and above, where 2^x is 0; NaN stays
            by = reference(m);
            const float from = m == -INFINITY ? 0.0f : m;
            float low = v[0];
#pragma unroll
            for (int i = 0; i < kEach; i++) {
                low = fminf(low, v[i]);
                const float x = __builtin_elementwise_maximum((v[i] - from) * kLog2e, -250.0f);
                e[i] = __builtin_amdgcn_exp2f(x);
                t[i % 4] = __builtin_fmaf(x, e[i], i < 4 ? 0.0f : t[i % 4]);
            }
            masked = __ballot(!(low > -1e38f)) != 0; // the next 16 are likely to be, too
        }
        rescale(mine, m, by);
        mine.s += (double)sum_of(e);
        mine.t += (double)sum_of(t);
        steps++;
    };
    constexpr int kRing = WAVES > 1 ? 2 : 1; // steps in registers, all but one on the way
    Logits ring[kRing];
#pragma unroll
    for (int u = 0; u < kRing - 1; u++)
        ring[u].load(row, begin + u * kStep, end);
    for (int64_t at = begin; at < end; at += kRing * kStep) {
#pragma unroll
        for (int u = 0; u < kRing; u++) {
            const int64_t here = at + u * kStep;
            ring[(u + kRing - 1) % kRing].load(row, here + (kRing - 1) * kStep, end);
            if (here < end)
                step(ring[u], here);
        }
    }
    const float top = mine.m;
    Part all = over_wave(mine, [&](int from, float m, double &s, double &t) {
        const int thread = 64 * wave + from;
        for (int c = lane; c < steps * Logits::kGroups; c += 64) {
            const int64_t at = begin + (int64_t)(c / Logits::kGroups) * kStep;
            const int64_t i = Logits::id(at, c % Logits::kGroups, thread);
            for (int64_t e = i; e < min(i + Logits::kPer, end); e++) {
                const float l = logit<BF16>(row, e);
                if (l == m) // one of them, or s were 1 at least
                    continue;
                const float x = fmaxf((l - m) * kLog2e, -250.0f); // where 2^x is 0
                const float p = __builtin_amdgcn_exp2f(x);
                s += p;
                t += x * p;
            }
        }
    });
    if (WAVES > 1 && lane == 0)
        wave_parts[wave] = all;
    if (TOP) {
        groups[wave][lane] = top;
        if (threadIdx.x == 0)
            count = 0;
    }
    if (WAVES > 1)
        __syncthreads();
    // the first wave goes on; the others come back to read their logits again
    float least = 0;
    bool tied = false;
    double log_s = 0;
    if (wave == 0) {
        if (WAVES > 1)
            all = over_parts(wave_parts, WAVES);
        if (parts == 1)
            log_s = log_sum(all);
        if (threadIdx.x == 0) {
            if (parts == 1)
                write_row(p, r, all, log_s, token);
            else
                out_parts[blockIdx.x] = all;
        }
    }
    if constexpr (!TOP)
        return;

    // ---- the alternatives
    const int k = (int)min((int64_t)p.topk, end - begin);
    if (wave == 0) {
        // the smallest of the k largest of 64 groups' maxima, of 128 for many
        // alternatives: the lowest bits of a key give way to the group, which makes
        // the keys different
        auto key_of = [](float g, int group) {
            return (uint32_t)(word_of(g, 0) >> 32 & ~(uint64_t)127) | (uint32_t)group;
        };
        const int kinds = WAVES > 1 && k > 32 ? 2 : 1;
        float even = groups[0][lane], odd = -INFINITY;
#pragma unroll
        for (int w = 1; w < WAVES; w++) {
            if (kinds == 2 && w % 2)
                odd = fmaxf(odd, groups[w][lane]);
            else
                even = fmaxf(even, groups[w][lane]);
        }
        const uint32_t key = key_of(even, lane), other = key_of(odd, 64 + lane);
        int rank = 0, rank_other = 0;
#pragma unroll
        for (int i = 0; i < 64; i++)
            rank += (uint32_t)__builtin_amdgcn_readlane((int)key, i) > key;
        if (kinds == 2) {
#pragma unroll
            for (int i = 0; i < 64; i++) {
                const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)key, i);
                const uint32_t b = (uint32_t)__builtin_amdgcn_readlane((int)other, i);
                rank += b > key;
                rank_other += (a > other) + (b > other);
            }
        }
        float kth = rank < k ? even : INFINITY;
        if (kinds == 2 && rank_other < k)
            kth = fminf(kth, odd);
        least = -wave_max(-kth);
        tied = __popcll(__ballot(even == least)) + __popcll(__ballot(odd == least)) > 16;
        if (WAVES > 1 && threadIdx.x == 0) {
            reach = least;
            many = tied;
        }
    }
    if constexpr (WAVES > 1) {
        __syncthreads();
        least = reach;
        tied = many;
    }
    auto take = [&](float l, int64_t id) {
        const int slot = atomicAdd(&count, 1); // the order decides nothing
        if (slot < kCandidates)
            words[slot] = word_of(l, (uint32_t)id);
    };
    // With fewer than k open groups, `least` is -inf: the open logits, and of the
    // masked ones the first k.  Where many groups have `least` itself, or too many
    // logits reach it, those above it first.
    const bool masks = least == -INFINITY;
    float from = masks ? -FLT_MAX : tied ? next_above(least) : least;
    int found;
#pragma unroll 1
    for (;;) {
        if (top >= from) {
            for (int s = 0; s < steps; s++) {
                const int64_t at = begin + (int64_t)s * kStep;
                if (__uint_as_float((uint32_t)tops[s][threadIdx.x] << 16) < from)
                    continue;
                Logits again;
                again.load(row, at, end);
                float v[kEach];
                again.values(v, at, end); // -inf where not the thread's own
#pragma unroll
                for (int i = 0; i < kEach; i++)
                    if (v[i] >= from)
                        take(v[i], Logits::id_of(at, i / Logits::kPer, i % Logits::kPer, end));
            }
        }
        if (masks && (int)threadIdx.x < k && !(logit<BF16>(row, begin + threadIdx.x) > -INFINITY))
            take(-INFINITY, begin + threadIdx.x); // NaN is as masked
        __syncthreads();
        found = count;
        if (found <= kCandidates || from != least)
            break;
        __syncthreads();
        if (threadIdx.x == 0)
            count = 0;
        __syncthreads();
        from = next_above(least);
    }
    // then the equal ones in the order of their ids (everybody has the same found)
    for (int64_t at = begin; found < k && at < end; at += kThreads) {
        const int64_t id = at + threadIdx.x;
        const bool equal = id < end && logit<BF16>(row, id) == least;
        const uint64_t lanes = __ballot(equal);
        if (lane == 0)
            equals[wave] = __popcll(lanes);
        __syncthreads();
        int slot = found + __popcll(lanes & (((uint64_t)1 << lane) - 1));
#pragma unroll
        for (int w = 0; w < WAVES; w++) {
            slot += w < wave ? equals[w] : 0;
            found += equals[w];
        }
        if (equal && slot < k)
            words[slot] = word_of(least, (uint32_t)id);
        found = min(found, k);
        __syncthreads();
    }
    const bool few = found <= kCandidates;
    if (few && wave > 0)
        return;
    auto emit = [&](int rank, uint64_t word) {
        if (parts > 1) {
            out_words[(int64_t)blockIdx.x * p.topk + rank] = word;
            return;
        }
        p.ids[r * p.topk + rank] = (int32_t)(~(uint32_t)word);
        p.top[r * p.topk + rank] = log_probability(all, log_s, logit_of(word));
    };
    if (parts > 1 && (int)threadIdx.x >= k && (int)threadIdx.x < p.topk)
        out_words[(int64_t)blockIdx.x * p.topk + threadIdx.x] = 0; // none: below every logit
    if (few) {
        rank_words<64>(words, found, k, emit);
        return;
    }
    uint64_t last = ~(uint64_t)0;
    for (int j = 0; j < k; j++) {
        uint64_t next = 0;
        for (int64_t i = begin + threadIdx.x; i < end; i += kThreads) {
            const uint64_t w = word_of(logit<BF16>(row, i), (uint32_t)i);
            next = w < last ? larger(next, w) : next;
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1)
            next = larger(next, __shfl_xor(next, d));
        __syncthreads();
        if (lane == 0)
            best[wave] = next;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; w++)
            next = larger(next, best[w]);
        last = next;
        if (threadIdx.x == 0)
            emit(j, last);
    }
}

constexpr int kJoinThreads = 256;

template <bool BF16>
__global__ __launch_bounds__(kJoinThreads) void logprobs_join_kernel(const LogprobsProblem p, int parts,
                                                                     const Part *in_parts,
                                                                     const uint64_t *in_words)
{
    __shared__ __attribute__((aligned(16))) uint64_t words[kMaxParts * 64 + 8];
    __shared__ Part sums[kMaxParts];
    __shared__ uint64_t reach[2];
    __shared__ int count;
    const int64_t r = blockIdx.x;
    Token token{NAN, true};
    if (threadIdx.x == 0) {
        token = token_of<BF16>(p, r, row_of<BF16>(p, r));
        count = 0;
    }
    if ((int)threadIdx.x < parts)
        sums[threadIdx.x] = in_parts[r * parts + threadIdx.x];
    // Every part's words fall.  At least topk words are not below the largest
    // of the parts' last, nor below the smallest of their (topk / parts)-th.
    const int k = p.topk, each = (k + parts - 1) / parts;
    const uint64_t *in = in_words + r * parts * k;
    if (k > 0 && threadIdx.x < 64) {
        uint64_t last = 0, share = ~(uint64_t)0;
        for (int i = threadIdx.x; i < parts; i += 64) {
            last = larger(last, in[i * k + k - 1]);
            share = min(share, in[i * k + each - 1]);
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) {
            last = larger(last, __shfl_xor(last, d));
            share = min(share, (uint64_t)__shfl_xor(share, d));
        }
        if (threadIdx.x == 0)
            reach[0] = larger(larger(last, share), 1);
    }
    __syncthreads();
    const Part all = over_parts(sums, parts);
    const double log_s = log_sum(all);
    if (threadIdx.x == 0)
        write_row(p, r, all, log_s, token);
    if (k == 0)
        return;
    for (int i = threadIdx.x; i < parts * k; i += kJoinThreads) {
        const uint64_t w = in[i];
        if (w >= reach[0])
            words[atomicAdd(&count, 1)] = w; // the order decides nothing
    }
    __syncthreads();
    rank_words<kJoinThreads>(words, count, k, [&](int rank, uint64_t word) {
        p.ids[r * k + rank] = (int32_t)(~(uint32_t)word);
        p.top[r * k + rank] = log_probability(all, log_s, logit_of(word));
    });
}

// How a row is split: waves of a workgroup, and parts of `length` logits.  One
// part from half as many rows as CUs (256) on, else about 1024 workgroups; a
// part is a whole number of steps, 32 at most.  More rows gain nothing from parts,
// whose chains of steps and join cost what a fuller chip saves: bf16 with 5
// alternatives, in one part, (two) and (four), 129 x 50001 13.0 us (15.9, 17.8),
// 333 x 50001 18.7 (23.7, 28.8), 333 x 131072 27.5 (30.8, 34.7), 512 x 131072
// without alternatives 25.5 (27.8, 28.1); only 300 x 262144 fp32, 300 MB, 69 (66, 64).
struct Split {
    int waves, parts;
    int64_t length;
};

Split split_of(int64_t rows, int64_t vocab)
{
    Split s;
    s.waves = vocab <= 4096 ? 1 : vocab <= 131072 && rows > 512 ? 4 : 8;
    const int64_t step = 64 * s.waves * kEach, steps = (vocab + step - 1) / step;
    int64_t parts = rows > 128 ? 1 : (1024 + rows - 1) / (rows > 0 ? rows : 1);
    parts = std::min<int64_t>(std::min<int64_t>(parts, steps), kMaxParts);
    if (s.waves == 1)
        parts = 1;
    parts = std::max<int64_t>(parts, (steps + kSteps - 1) / kSteps);
    s.length = (steps + parts - 1) / parts * step;
    s.parts = (int)((vocab + s.length - 1) / s.length);
    return s;
}

template <bool BF16, bool TOP>
void launch_parts(const LogprobsProblem &p, const Split &s, Part *sums, uint64_t *words, hipStream_t stream)
{
    const unsigned grid = (unsigned)(p.rows * s.parts);
    if (s.waves == 1)
        logprobs_kernel<BF16, TOP, 1><<<grid, 64, 0, stream>>>(p, s.parts, s.length, sums, words);
    else if (s.waves == 4)
        logprobs_kernel<BF16, TOP, 4><<<grid, 256, 0, stream>>>(p, s.parts, s.length, sums, words);
    else
        logprobs_kernel<BF16, TOP, 8><<<grid, 512, 0, stream>>>(p, s.parts, s.length, sums, words);
}

hipError_t launch_rows(const LogprobsProblem &p, const Split &s, Part *sums, uint64_t *words,
                       hipStream_t stream)
{
    if (p.bf16 && p.topk > 0)
        launch_parts<true, true>(p, s, sums, words, stream);
    else if (p.bf16)
        launch_parts<true, false>(p, s, sums, words, stream);
    else if (p.topk > 0)
        launch_parts<false, true>(p, s, sums, words, stream);
    else
        launch_parts<false, false>(p, s, sums, words, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || s.parts == 1)
        return e;
    const unsigned grid = (unsigned)p.rows;
    if (p.bf16)
        logprobs_join_kernel<true><<<grid, kJoinThreads, 0, stream>>>(p, s.parts, sums, words);
    else
        logprobs_join_kernel<false><<<grid, kJoinThreads, 0, stream>>>(p, s.parts, sums, words);
    return hipGetLastError();
}

} // namespace

size_t logprobs_bytes(int64_t rows, int64_t vocab, int topk)
{
    const int64_t parts = split_of(rows, vocab).parts;
    return parts == 1 ? 0 : (size_t)(rows * parts) * (sizeof(Part) + (size_t)topk * sizeof(uint64_t));
}

hipError_t launch_logprobs(const LogprobsProblem &p, void *workspace, hipStream_t stream)
{
    if (p.rows == 0)
        return hipSuccess;
    const Split s = split_of(p.rows, p.vocab);
    Part *sums = static_cast<Part *>(workspace);
    uint64_t *words = reinterpret_cast<uint64_t *>(sums + p.rows * s.parts);
    // 2^22 workgroups a launch: a grid holds fewer than 2^32 threads
    const int64_t each = ((int64_t)1 << 22) / s.parts;
    for (int64_t r = 0; r < p.rows; r += each) {
        LogprobsProblem q = p;
        q.rows = std::min(p.rows - r, each);
        q.logits = static_cast<const uint8_t *>(p.logits) + r * p.ldl * (p.bf16 ? 2 : 4);
        if (p.tokens) {
            q.tokens = static_cast<const uint8_t *>(p.tokens) + r * (p.wide ? 8 : 4);
            q.logprobs = p.logprobs + r;
        }
        if (p.entropy)
            q.entropy = p.entropy + r;
        if (p.topk > 0) {
            q.ids = p.ids + r * p.topk;
            q.top = p.top + r * p.topk;
        }
        const hipError_t e = launch_rows(q, s, sums + r * s.parts, words + r * s.parts * p.topk, stream);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace bpg
