// epilogue.h -- bias, activation and residual applied to a dense product's
// fp32 results before the store (gfx950).  Internal; included by the dense
// product kernels, whose template argument EP selects the form with it.
//
//   y = act(v + bias[column]) + residual[row][column]
//
// each step in fp32, rounded once to the output's type at the store.  The
// kernels load a lane's residual values before they store its first result
// (the tiled 64 x 160 form those of a round of its reduction, four tiles and
// then one): the residual may be y itself, so a load after a store could not be
// moved ahead of it and would wait for it.  They are loaded as raw bits and
// converted where they are added, so that nothing waits for them before.
// 512 x 5120 x 5120 takes 39.4 us with a bf16 residual and 38.9 without; with
// the loads where the values are added 43.6.  With 8-bit codes (tiled) it takes
// 49.5 and 48.0.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bpg.h"
#include "internal.h"

namespace bpg {
namespace {

__device__ __forceinline__ float ep_load(const void *p, bool bf16, int64_t i)
{
    return bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16)
                : static_cast<const float *>(p)[i];
}

// the bits of residual value i, and their value
__device__ __forceinline__ uint32_t ep_raw(const Epilogue &ep, int64_t i)
{
    return ep.residual_bf16 ? (uint32_t) static_cast<const uint16_t *>(ep.residual)[i]
                            : static_cast<const uint32_t *>(ep.residual)[i];
}

__device__ __forceinline__ float ep_value(const Epilogue &ep, uint32_t raw)
{
    return __uint_as_float(ep.residual_bf16 ? raw << 16 : raw);
}

// e^x is 2^n 2^f (Cody and Waite's argument reduction: log2 e in two parts),
// n the nearest integer to x log2 e and f = x log2 e - n to 2^-24; x is held to
// +-150
__device__ __forceinline__ float ep_exp_parts(float x, float &f)
{
    const float u = fminf(fmaxf(x, -150.0f), 150.0f);
    const float n = rintf(u * 1.44269502f);
    f = __builtin_fmaf(u, 1.44269502f, -n);
    f = __builtin_fmaf(u, 1.92596299e-8f, f);
    return n;
}

// 1 / (1 + e^-x) within 8 2^-24 for x > -87: the parts of e^-x, the hardware's
// exp2 and reciprocal within an ulp each and the sum's rounding.  Below, e^-x
// overflows and the result falls to 0 (see ep_gated).  10 instructions; expf
// and a division took 40, 9 us of the 256 us of a 1024 x 5120 x 17408 product.
__device__ __forceinline__ float ep_sigmoid(float x)
{
    float f;
    const float n = ep_exp_parts(-x, f);
    const float e = ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
    return __builtin_amdgcn_rcpf(1.0f + e);
}

// v / (1 + e^-z), also where e^-z overflows: the denominator is then taken
// 2^-64 times.  Up to e^-z = 2^100 the steps are those of v * ep_sigmoid(z).
__device__ __forceinline__ float ep_gated_far(float v, float z)
{
    float f;
    const int n = (int)ep_exp_parts(-z, f);
    const int k = n > 100 ? 64 : 0;
    const float e = ldexpf(__builtin_amdgcn_exp2f(f), n - k);
    return ldexpf(v * __builtin_amdgcn_rcpf((n > 100 ? 0x1p-64f : 1.0f) + e), -k);
}

// v = v / (1 + e^-z(v)) for N values of a lane, down to subnormal results.
// `far`: above it e^-z stays below 2^100.  Values below it are rare, so the
// whole wave looks for them first (N / 2 instructions); the other values of
// such a wave get the same bits either way.
template <int N, class Z>
__device__ __forceinline__ void ep_gated(float (&v)[N], float far, Z &&z)
{
    float low = v[0];
#pragma unroll
    for (int i = 1; i < N; i++)
        low = fminf(low, v[i]);
    if (__builtin_amdgcn_ballot_w64(low < far) != 0) {
#pragma unroll
        for (int i = 0; i < N; i++)
            v[i] = ep_gated_far(v[i], z(v[i]));
        return;
    }
#pragma unroll
    for (int i = 0; i < N; i++)
        v[i] = v[i] * ep_sigmoid(z(v[i]));
}

// the activation of N values of a lane (act is uniform across the launch)
template <int N>
__device__ __forceinline__ void ep_activate(int act, float (&v)[N])
{
    switch (act) {
    case BPG_ACT_RELU:
#pragma unroll
        for (int i = 0; i < N; i++)
            v[i] = v[i] < 0.0f ? 0.0f : v[i];
        break;
    case BPG_ACT_SILU:
        ep_gated(v, -64.0f, [](float x) { return x; });
        break;
    case BPG_ACT_GELU:
        // x Phi(x) = x / 2 erfc(-x / sqrt 2): 1 + erf would cancel below zero
        // (4% off at -5, 0 from -6 on)
#pragma unroll
        for (int i = 0; i < N; i++)
            v[i] = 0.5f * v[i] * erfcf(v[i] * -0.70710678118654752f);
        break;
    case BPG_ACT_GELU_TANH:
        // 0.5 (1 + tanh u) = sigmoid(2 u), u = sqrt(2 / pi) (x + 0.044715 x^3); 2 u is -66.4 at -9
        ep_gated(v, -9.0f, [](float x) { return 1.5957691216057308f * (x + 0.044715f * x * x * x); });
        break;
    default: break;
    }
}

} // namespace
} // namespace bpg
