// logprobs.hip -- log probabilities of given tokens, entropies and top
// alternatives of rows of logits (gfx950).
//
//   m = max l, S = sum e^(l - m), T = sum (l - m) e^(l - m)
//   log p(t) = l_t - m - log S,  entropy = log S - T / S
//
// T <= 0 and S >= 1, so nothing cancels in the entropy.  The top alternatives
// are the largest logits, equal ones by the lowest id; a NaN counts as -inf
// there.  A row with a NaN or +inf, or of -inf only, has no distribution: NaN.
#include "fp8.h"

#include <climits>
#include <cmath>

namespace bpg {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

template <bool BF16> __device__ __forceinline__ float logit(const void *row, int64_t i)
{
    return BF16 ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(row)[i] << 16)
                : static_cast<const float *>(row)[i];
}

// An order of the logits and their ids in one word: larger words are larger
// logits, or the lower id of equal ones.
__device__ __forceinline__ uint64_t rank_of(float v, uint32_t id)
{
    uint32_t u = __float_as_uint(v == v ? v + 0.0f : -INFINITY); // -0 becomes 0
    u = u & 0x80000000u ? ~u : u | 0x80000000u;
    return (uint64_t)u << 32 | (~id);
}

__device__ __forceinline__ float logit_of(uint64_t rank)
{
    const uint32_t u = (uint32_t)(rank >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

template <class T, class F> __device__ T over_group(T v, T *shared, F &&join)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        v = join(v, __shfl_xor(v, d));
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        shared[threadIdx.x >> 6] = v;
    __syncthreads();
    v = shared[0];
#pragma unroll
    for (int w = 1; w < kWaves; w++)
        v = join(v, shared[w]);
    return v;
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(const LogprobsProblem p)
{
    __shared__ uint64_t words[kWaves];
    __shared__ double sums[kWaves];
    const int64_t r = blockIdx.x;
    const void *row = BF16 ? (const void *)(static_cast<const uint16_t *>(p.logits) + r * p.ldl)
                           : (const void *)(static_cast<const float *>(p.logits) + r * p.ldl);
    const auto larger = [](uint64_t a, uint64_t b) { return a > b ? a : b; };
    const auto add = [](double a, double b) { return a + b; };
    uint64_t best = 0;
    double odd = 0;
    for (int64_t i = threadIdx.x; i < p.vocab; i += kThreads) {
        const float v = logit<BF16>(row, i);
        odd += !(v < INFINITY);
        best = larger(best, rank_of(v, (uint32_t)i));
    }
    best = over_group(best, words, larger);
    const float m = logit_of(best);
    const bool none = over_group(odd, sums, add) > 0 || m == -INFINITY;
    double s = 0, t = 0;
    for (int64_t i = threadIdx.x; i < p.vocab; i += kThreads) {
        const float d = logit<BF16>(row, i) - m, e = expf(d);
        s += e;
        t += e > 0 ? (double)(d * e) : 0.0;
    }
    s = over_group(s, sums, add);
    t = over_group(t, sums, add);
    const double log_s = none ? NAN : log(s);
    if (threadIdx.x == 0) {
        if (p.entropy)
            p.entropy[r] = (float)(log_s - t / s);
        if (p.tokens) {
            const int64_t id = p.wide ? static_cast<const int64_t *>(p.tokens)[r]
                                      : static_cast<const int32_t *>(p.tokens)[r];
            float l = id < 0 ? 0.0f : NAN;
            if (id >= 0 && id < p.vocab)
                l = (float)((double)(logit<BF16>(row, id) - m) - log_s);
            p.logprobs[r] = l;
        }
    }
    for (int j = 0; j < p.topk; j++) {
        if (j > 0) {
            uint64_t next = 0;
            for (int64_t i = threadIdx.x; i < p.vocab; i += kThreads) {
                const uint64_t w = rank_of(logit<BF16>(row, i), (uint32_t)i);
                next = w < best ? larger(next, w) : next;
            }
            best = over_group(next, words, larger);
        }
        if (threadIdx.x == 0) {
            p.ids[r * p.topk + j] = (int32_t)(~(uint32_t)best);
            p.top[r * p.topk + j] = (float)((double)(logit_of(best) - m) - log_s);
        }
    }
}

} // namespace

size_t logprobs_bytes(int64_t, int64_t, int) { return 0; }

hipError_t launch_logprobs(const LogprobsProblem &p, void *, hipStream_t stream)
{
    if (p.rows == 0)
        return hipSuccess;
    if (p.bf16)
        logprobs_kernel<true><<<(unsigned)p.rows, kThreads, 0, stream>>>(p);
    else
        logprobs_kernel<false><<<(unsigned)p.rows, kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

} // namespace bpg
