// logprobs.hip -- log probabilities of given tokens, entropies and top
// alternatives of rows of logits (gfx950).
//
//   m = max l, S = sum e^(l - m), T = sum (l - m) e^(l - m)
//   log p(t) = l_t - m - log S,  entropy = log S - T / S
//
// T <= 0 and S >= 1, so nothing cancels in the entropy.  The top alternatives
// are the largest logits, equal ones by the lowest id; a NaN counts as -inf
// there.  A row with a NaN or +inf, or of -inf only, has no distribution: NaN.
//
// One pass over the logits: a thread holds 16 at a time, takes their maximum,
// rescales its sums to it and adds the 16 terms (in fp32 among the 16, in fp64
// from one 16 to the next).  For the alternatives it leaves each 16's maximum in
// LDS.  The k-th largest of 64 groups' maxima is then below or at the k-th
// largest logit, and few logits reach it (64 ln (64 / (64 - k)) on shuffled
// rows: 24 for k = 20), so only the 16s that do are read again.  Where more than
// kCandidates reach it (rows of equal logits, or with fewer than k above -inf)
// the alternatives are found one scan of the part each.
//
// Few rows are split into parts of 8192 logits or more, a workgroup each, and
// another launch joins them.
#include "fp8.h"

#include <algorithm>
#include <cmath>

namespace bpg {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kEach = 16;                    // logits a thread holds at once
constexpr int kStep = kThreads * kEach;      // logits of a step of a workgroup
constexpr int kSteps = 32;                   // at most, per workgroup
constexpr int kCandidates = 1024;
constexpr int kMaxParts = 64;
constexpr float kLog2e = 1.44269504f;

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// What a part of a row amounts to.
struct Part {
    float m;      // the largest logit, -inf if there is none
    uint32_t odd; // a NaN or +inf among them
    double s, t;  // the sums, 0 where m is -inf
};

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

// e^d, d <= 0 or NaN (from -inf - -inf: no logit yet); 0 below -150
__device__ __forceinline__ float clamped(float d) { return fmaxf(d, -150.0f); }
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

__device__ __forceinline__ Part join(Part a, Part b)
{
    const float m = fmaxf(a.m, b.m);
    const float da = clamped(a.m - m), db = clamped(b.m - m);
    const double ea = exp_of(da), eb = exp_of(db);
    return Part{m, a.odd | b.odd, a.s * ea + b.s * eb,
                (a.t + da * a.s) * ea + (b.t + db * b.s) * eb};
}

__device__ __forceinline__ Part over_wave(Part p)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        Part o;
        o.m = __shfl_xor(p.m, d);
        o.odd = __shfl_xor(p.odd, d);
        o.s = __shfl_xor(p.s, d);
        o.t = __shfl_xor(p.t, d);
        p = join(p, o);
    }
    return p;
}

// Sixteen logits of a thread in a step: groups of one 16-byte load each, the
// threads' groups side by side.
template <bool BF16> struct Step {
    static constexpr int kGroups = BF16 ? 2 : 4, kPer = kEach / kGroups;
    v4u raw[kGroups];
    static __device__ __forceinline__ int64_t id(int64_t at, int q)
    {
        return at + (int64_t)q * (kThreads * kPer) + threadIdx.x * kPer;
    }
    static __device__ __forceinline__ const uint8_t *address(const void *row, int64_t i)
    {
        return static_cast<const uint8_t *>(row) + i * (BF16 ? 2 : 4);
    }
    // the step that begins at logit `at`; -inf past `end`
    __device__ __forceinline__ void load(const void *row, int64_t at, int64_t end)
    {
#pragma unroll
        for (int q = 0; q < kGroups; q++) {
            const int64_t i = id(at, q);
            if (i + kPer <= end) {
                __builtin_memcpy(&raw[q], __builtin_assume_aligned(address(row, i), BF16 ? 2 : 4), 16);
                continue;
            }
#pragma unroll
            for (int e = 0; e < kPer; e++) {
                uint32_t v = BF16 ? 0xff80u : 0xff800000u;
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
    __device__ __forceinline__ void values(float (&v)[kEach]) const
    {
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const uint32_t w = raw[i / kPer][BF16 ? i % kPer / 2 : i % kPer];
            v[i] = __uint_as_float(!BF16 ? w : i & 1 ? w & 0xffff0000u : w << 16);
        }
    }
};

template <bool BF16> __device__ __forceinline__ float logit(const void *row, int64_t i)
{
    return BF16 ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(row)[i] << 16)
                : static_cast<const float *>(row)[i];
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

__device__ __forceinline__ void write_row(const LogprobsProblem &p, int64_t r, const Part &all, Token token)
{
    const double log_s = all.odd || all.m == -INFINITY ? NAN : log(all.s);
    if (p.entropy)
        p.entropy[r] = (float)(log_s - all.t / all.s);
    if (p.tokens)
        p.logprobs[r] = token.none ? 0.0f : (float)((double)(token.logit - all.m) - log_s);
}

template <bool BF16>
__device__ __forceinline__ const void *row_of(const LogprobsProblem &p, int64_t r)
{
    return static_cast<const uint8_t *>(p.logits) + r * p.ldl * (BF16 ? 2 : 4);
}

__device__ __forceinline__ void write_top(const LogprobsProblem &p, int64_t at, uint64_t word, const Part &all)
{
    const double log_s = all.odd || all.m == -INFINITY ? NAN : log(all.s);
    p.ids[at] = (int32_t)(~(uint32_t)word);
    p.top[at] = (float)((double)(logit_of(word) - all.m) - log_s);
}

// rank < k of `count` different words: emit(rank, word)
template <int THREADS, class F>
__device__ __forceinline__ void rank_words(const uint64_t *words, int count, int k, F &&emit)
{
    for (int i = threadIdx.x; i < count; i += THREADS) {
        const uint64_t mine = words[i];
        int rank = 0;
        for (int j = 0; j < count; j++)
            rank += words[j] > mine;
        if (rank < k)
            emit(rank, mine);
    }
}

// workgroup (row, part): logits [part * length, ...) of its row.  TOP: with
// alternatives.
template <bool BF16, bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(const LogprobsProblem p, int parts,
                                                            int64_t length, Part *out_parts,
                                                            uint64_t *out_words)
{
    __shared__ Part wave_parts[kWaves];
    __shared__ uint16_t tops[TOP ? kSteps : 1][kThreads];
    __shared__ float groups[kWaves][64];
    __shared__ uint64_t words[TOP ? kCandidates : 1], best[kWaves];
    __shared__ int count;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r = blockIdx.x / parts, part = blockIdx.x % parts;
    const void *row = row_of<BF16>(p, r);
    const int64_t begin = part * length, end = min(begin + length, p.vocab);

    Token token{NAN, true};
    if (parts == 1 && threadIdx.x == 0)
        token = token_of<BF16>(p, r, row);

    // ---- the sums
    Part mine{-INFINITY, 0, 0.0, 0.0};
    Step<BF16> now, next;
    now.load(row, begin, end);
    int steps = 0;
    for (int64_t at = begin; at < end; at += kStep, steps++) {
        if (at + kStep < end)
            next.load(row, at + kStep, end);
        float v[kEach];
        now.values(v);
        float top = v[0];
        bool odd = false;
#pragma unroll
        for (int i = 1; i < kEach; i++)
            top = fmaxf(top, v[i]); // drops NaN
#pragma unroll
        for (int i = 0; i < kEach; i += 2)
            odd |= __builtin_isunordered(v[i], v[i + 1]);
        if (TOP)
            tops[steps][threadIdx.x] = above(top == top ? top : -INFINITY);
        const float m = fmaxf(mine.m, top), dm = clamped(mine.m - m);
        float e[kEach], t[kEach];
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const float d = clamped(v[i] - m);
            e[i] = exp_of(d);
            t[i] = d * e[i];
        }
        const double c = exp_of(dm);
        mine.t = (mine.t + dm * mine.s) * c + (double)sum_of(t);
        mine.s = mine.s * c + (double)sum_of(e);
        mine.m = m;
        mine.odd |= odd || top == INFINITY;
        now = next;
    }
    const float top = mine.m; // -inf: the sums are 0 (-inf - -inf is clamped)
    mine = over_wave(mine);
    if (lane == 0)
        wave_parts[wave] = mine;
    if (TOP) {
        groups[wave][lane] = top;
        if (threadIdx.x == 0)
            count = 0;
    }
    __syncthreads();
    Part all = wave_parts[0];
#pragma unroll
    for (int w = 1; w < kWaves; w++)
        all = join(all, wave_parts[w]);
    if (threadIdx.x == 0) {
        if (parts == 1)
            write_row(p, r, all, token);
        else
            out_parts[blockIdx.x] = all;
    }
    if constexpr (!TOP)
        return;

    // ---- the alternatives
    const int k = (int)min((int64_t)p.topk, end - begin);
    if (parts > 1 && (int)threadIdx.x >= k && (int)threadIdx.x < p.topk)
        out_words[(int64_t)blockIdx.x * p.topk + threadIdx.x] = 0; // none: below every logit
    auto emit = [&](int rank, uint64_t word) {
        if (parts == 1)
            write_top(p, r * p.topk + rank, word, all);
        else
            out_words[(int64_t)blockIdx.x * p.topk + rank] = word;
    };
    if (all.m == -INFINITY) { // the first ones
        if ((int)threadIdx.x < k)
            emit(threadIdx.x, word_of(-INFINITY, (uint32_t)(begin + threadIdx.x)));
        return;
    }
    // the k-th largest of 64 groups' maxima, in every wave
    float g = groups[0][lane];
#pragma unroll
    for (int w = 1; w < kWaves; w++)
        g = fmaxf(g, groups[w][lane]);
    int rank = 0;
#pragma unroll
    for (int i = 0; i < 64; i++) {
        const float o = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), i));
        rank += o > g || (o == g && i < lane);
    }
    const uint64_t which = __ballot(rank == k - 1);
    const float least =
        __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), __builtin_ctzll(which)));
    if (top >= least) {
        for (int s = 0; s < steps; s++) {
            const int64_t at = begin + (int64_t)s * kStep;
            if (__uint_as_float((uint32_t)tops[s][threadIdx.x] << 16) < least)
                continue;
            now.load(row, at, end);
            float v[kEach];
            now.values(v);
#pragma unroll
            for (int i = 0; i < kEach; i++) {
                const int64_t id = Step<BF16>::id(at, i / Step<BF16>::kPer) + i % Step<BF16>::kPer;
                const float l = v[i] == v[i] ? v[i] : -INFINITY;
                if (l >= least && id < end) {
                    const int slot = atomicAdd(&count, 1); // the order decides nothing
                    if (slot < kCandidates)
                        words[slot] = word_of(l, (uint32_t)id);
                }
            }
        }
    }
    __syncthreads();
    if (count <= kCandidates) {
        rank_words<kThreads>(words, count, k, emit);
        return;
    }
    uint64_t last = ~(uint64_t)0;
    for (int j = 0; j < k; j++) {
        uint64_t found = 0;
        for (int64_t i = begin + threadIdx.x; i < end; i += kThreads) {
            const uint64_t w = word_of(logit<BF16>(row, i), (uint32_t)i);
            found = w < last ? larger(found, w) : found;
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1)
            found = larger(found, __shfl_xor(found, d));
        __syncthreads();
        if (lane == 0)
            best[wave] = found;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; w++)
            found = larger(found, best[w]);
        last = found;
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
    __shared__ uint64_t words[kMaxParts * 64];
    const int64_t r = blockIdx.x;
    Part all = in_parts[r * parts];
    for (int i = 1; i < parts; i++)
        all = join(all, in_parts[r * parts + i]);
    if (threadIdx.x == 0)
        write_row(p, r, all, token_of<BF16>(p, r, row_of<BF16>(p, r)));
    const int count = parts * p.topk;
    for (int i = threadIdx.x; i < count; i += kJoinThreads)
        words[i] = in_words[r * count + i];
    __syncthreads();
    rank_words<kJoinThreads>(words, count, p.topk, [&](int rank, uint64_t word) {
        write_top(p, r * p.topk + rank, word, all);
    });
}

// Parts of a row: one where the rows fill the chip (256 CUs), else about 1024
// workgroups; a part is a whole number of steps, 32 at most.
int parts_of(int64_t rows, int64_t vocab, int64_t *length)
{
    const int64_t steps = (vocab + kStep - 1) / kStep;
    int64_t parts = rows > 128 ? 1 : (1024 + rows - 1) / (rows > 0 ? rows : 1);
    parts = std::min<int64_t>(std::min<int64_t>(parts, steps), kMaxParts);
    parts = std::max<int64_t>(parts, (steps + kSteps - 1) / kSteps);
    const int64_t each = (steps + parts - 1) / parts;
    *length = each * kStep;
    return (int)((vocab + *length - 1) / *length);
}

} // namespace

size_t logprobs_bytes(int64_t rows, int64_t vocab, int topk)
{
    int64_t length;
    const int parts = parts_of(rows, vocab, &length);
    return parts == 1 ? 0 : (size_t)rows * parts * (sizeof(Part) + (size_t)topk * sizeof(uint64_t));
}

hipError_t launch_logprobs(const LogprobsProblem &p, void *workspace, hipStream_t stream)
{
    if (p.rows == 0)
        return hipSuccess;
    int64_t length;
    const int parts = parts_of(p.rows, p.vocab, &length);
    Part *sums = static_cast<Part *>(workspace);
    uint64_t *words = reinterpret_cast<uint64_t *>(sums + p.rows * parts);
    const unsigned grid = (unsigned)(p.rows * parts);
#define BPG_LOGPROBS(BF16, TOP)                                                                    \
    logprobs_kernel<BF16, TOP><<<grid, kThreads, 0, stream>>>(p, parts, length, sums, words)
    if (p.bf16 && p.topk > 0)
        BPG_LOGPROBS(true, true);
    else if (p.bf16)
        BPG_LOGPROBS(true, false);
    else if (p.topk > 0)
        BPG_LOGPROBS(false, true);
    else
        BPG_LOGPROBS(false, false);
#undef BPG_LOGPROBS
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || parts == 1)
        return e;
    if (p.bf16)
        logprobs_join_kernel<true><<<(unsigned)p.rows, kJoinThreads, 0, stream>>>(p, parts, sums, words);
    else
        logprobs_join_kernel<false><<<(unsigned)p.rows, kJoinThreads, 0, stream>>>(p, parts, sums, words);
    return hipGetLastError();
}

} // namespace bpg
