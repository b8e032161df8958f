// epilogue.h -- bias, activation and residual applied to a dense product's
// fp32 results before the store (gfx950).  Internal; included by the dense
// product kernels, whose template argument EP selects the form with it.
//
//   y = act(v + bias[column]) + residual[row][column]
//
// each step in fp32, rounded once to the output's type at the store.  The
// kernels load every residual value of a lane before they store its first
// result: the residual may be y itself, so a load after a store could not be
// moved ahead of it and would wait for it.  They are loaded as raw bits and
// converted where they are added, so that nothing waits for them before.
// 512 x 5120 x 5120 takes 39.4 us with a bf16 residual and 38.9 without; with
// the loads where the values are added 43.6.
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

// 1 / (1 + e^-x) within 8 2^-24: e^-x = 2^n 2^f with n the nearest integer to
// -x log2 e and f = -x log2 e - n to 2^-25 (log2 e in two parts), the
// hardware's exp2 and reciprocal within an ulp each.  Past +-150 the result is
// 0 or 1 whatever x is.  10 instructions; expf and a division took 40, 9 us of
// the 256 us of a 1024 x 5120 x 17408 product.
__device__ __forceinline__ float ep_sigmoid(float x)
{
    const float u = fminf(fmaxf(-x, -150.0f), 150.0f);
    const float n = rintf(u * 1.44269502f);
    float f = __builtin_fmaf(u, 1.44269502f, -n);
    f = __builtin_fmaf(u, 1.92596299e-8f, f);
    const float e = ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
    return __builtin_amdgcn_rcpf(1.0f + e);
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
#pragma unroll
        for (int i = 0; i < N; i++)
            v[i] = v[i] * ep_sigmoid(v[i]);
        break;
    case BPG_ACT_GELU:
        // x Phi(x) = x / 2 erfc(-x / sqrt 2): 1 + erf would cancel below zero
        // (4% off at -5, 0 from -6 on)
#pragma unroll
        for (int i = 0; i < N; i++)
            v[i] = 0.5f * v[i] * erfcf(v[i] * -0.70710678118654752f);
        break;
    case BPG_ACT_GELU_TANH:
        // 0.5 (1 + tanh u) = sigmoid(2 u), u = sqrt(2 / pi) (x + 0.044715 x^3)
#pragma unroll
        for (int i = 0; i < N; i++)
            v[i] = v[i] * ep_sigmoid(1.5957691216057308f * (v[i] + 0.044715f * v[i] * v[i] * v[i]));
        break;
    default: break;
    }
}

} // namespace
} // namespace bpg
