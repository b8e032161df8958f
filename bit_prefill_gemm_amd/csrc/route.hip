// route.hip -- routing of tokens to experts (gfx950).
//
// "Where the engine is going: HRX and the NPU", section "4-bit activations
// reach the MoE experts": the route covers the expert matmuls; the pages give
// no detail of the router, so the steps are this library's reading.  Per
// token, over the logits l_e of its E experts:
//   p_e = exp(l_e - max l) / sum exp(l - max l)   or   1 / (1 + exp(-l_e))
//   key_e = p_e + bias_e                          (the bias moves the choice only)
//   a group of experts scores its best key, or the sum of its two best keys;
//   the experts of the topk_groups best groups stay in the choice
//   the topk best keys, best first; ties go to the lowest index
//   w_j = p_j / sum p (if renormalised) * scale
// Scores, keys and sums are fp64: two keys are then told apart wherever their
// logits or biases differ, so the choice does not depend on how exp is
// rounded.  Softmax is monotone, so without a bias its choice compares the
// logits themselves.  A NaN logit counts as -inf (score 0), +inf as the
// largest fp32; a row of -inf only has scores 0 and weights 0.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace bpg {

namespace {

__device__ __forceinline__ float load_logit(const float *p, int i) { return p[i]; }
__device__ __forceinline__ float load_logit(const uint16_t *p, int i)
{
    return __uint_as_float((uint32_t)p[i] << 16);
}

__device__ __forceinline__ double max_f64(double a, double b) { return a > b ? a : b; }

__device__ __forceinline__ double wave_max(double v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v = max_f64(v, __shfl_xor(v, d));
    return v;
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ int wave_min(int v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v = min(v, __shfl_xor(v, d));
    return v;
}

constexpr int kTaken = 1 << 30; // above every expert index

// One wave per token; lane l holds experts l, l + 64, ..., NE of them.
template <typename T, int NE>
__global__ __launch_bounds__(256) void route_topk_kernel(RouteProblem p)
{
    const int lane = threadIdx.x & 63;
    const int64_t token = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (token >= p.tokens)
        return;
    const T *row = static_cast<const T *>(p.logits) + token * p.ldl;
    const int E = p.experts;
    float l[NE];
    double score[NE], key[NE];
    bool open[NE]; // in the choice
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NE; i++) {
        const int e = lane + 64 * i;
        open[i] = e < E;
        const float x = open[i] ? load_logit(row, e) : -INFINITY;
        l[i] = x != x ? -INFINITY : fminf(x, 0x1.fffffep127f);
        top = fmaxf(top, l[i]);
    }
    if (p.sigmoid) {
#pragma unroll
        for (int i = 0; i < NE; i++)
            score[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    } else {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
            top = fmaxf(top, __shfl_xor(top, d));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NE; i++) {
            score[i] = l[i] == -INFINITY ? 0.0 : exp((double)l[i] - (double)top);
            sum += score[i];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < NE; i++)
            score[i] = sum > 0.0 ? score[i] / sum : 0.0;
    }
#pragma unroll
    for (int i = 0; i < NE; i++) {
        const int e = lane + 64 * i;
        double k = p.sigmoid || p.bias || p.groups > 1 ? score[i] : (double)l[i];
        if (p.bias && e < E) {
            k = score[i] + (double)p.bias[e];
            k = k != k ? -INFINITY : k;
        }
        key[i] = k;
    }

    if (p.groups > 1) {
        const int size = E / p.groups;
        double gkey = -INFINITY; // lane g: the score of group g
        for (int g = 0; g < p.groups; g++) {
            double best = -INFINITY;
            int at = kTaken;
#pragma unroll
            for (int i = 0; i < NE; i++) {
                const int e = lane + 64 * i;
                if (e / size == g && e < E && (key[i] > best || at == kTaken)) {
                    best = key[i];
                    at = e;
                }
            }
            const double m = wave_max(at == kTaken ? -INFINITY : best);
            const int first = wave_min(at != kTaken && best == m ? at : kTaken);
            double s = m;
            if (p.pair) {
                double second = -INFINITY;
#pragma unroll
                for (int i = 0; i < NE; i++) {
                    const int e = lane + 64 * i;
                    if (e / size == g && e < E && e != first)
                        second = max_f64(second, key[i]);
                }
                s = m + wave_max(second);
            }
            if (lane == g)
                gkey = s;
        }
        uint64_t kept = 0;
        bool taken = lane >= p.groups;
        for (int j = 0; j < p.kept; j++) {
            const double m = wave_max(taken ? -INFINITY : gkey);
            const int g = wave_min(!taken && gkey == m ? lane : kTaken);
            if (lane == g)
                taken = true;
            if (g != kTaken)
                kept |= (uint64_t)1 << g;
        }
#pragma unroll
        for (int i = 0; i < NE; i++) {
            const int e = lane + 64 * i;
            open[i] = e < E && ((kept >> (e / size)) & 1);
        }
    }

    // lane j keeps choice j
    int chosen = 0;
    double weight = 0.0;
    for (int j = 0; j < p.topk; j++) {
        double best = -INFINITY, mine = 0.0;
        int at = kTaken;
#pragma unroll
        for (int i = 0; i < NE; i++)
            if (open[i] && (at == kTaken || key[i] > best)) {
                best = key[i];
                at = lane + 64 * i;
                mine = score[i];
            }
        const double m = wave_max(best);
        const int e = wave_min(at != kTaken && best == m ? at : kTaken);
        const double w = __shfl(mine, e & 63);
#pragma unroll
        for (int i = 0; i < NE; i++)
            if (lane + 64 * i == e)
                open[i] = false;
        if (lane == j) {
            chosen = e;
            weight = w;
        }
    }
    if (p.renormalize) {
        const double sum = wave_sum(weight);
        weight = sum > 0.0 ? weight / sum : 0.0;
    }
    if (lane < p.topk) {
        p.expert_of[token * p.topk + lane] = chosen;
        p.weights[token * p.topk + lane] = (float)(weight * (double)p.scale);
    }
}

template <typename T>
void launch_type(const RouteProblem &p, hipStream_t stream)
{
    const dim3 grid((unsigned)((p.tokens + 3) / 4));
    if (p.experts <= 64)
        route_topk_kernel<T, 1><<<grid, 256, 0, stream>>>(p);
    else if (p.experts <= 128)
        route_topk_kernel<T, 2><<<grid, 256, 0, stream>>>(p);
    else if (p.experts <= 256)
        route_topk_kernel<T, 4><<<grid, 256, 0, stream>>>(p);
    else
        route_topk_kernel<T, 8><<<grid, 256, 0, stream>>>(p);
}

} // namespace

hipError_t launch_route_topk(const RouteProblem &p, hipStream_t stream)
{
    if (p.tokens == 0)
        return hipSuccess;
    if (p.logits_bf16)
        launch_type<uint16_t>(p, stream);
    else
        launch_type<float>(p, stream);
    return hipGetLastError();
}

} // namespace bpg
