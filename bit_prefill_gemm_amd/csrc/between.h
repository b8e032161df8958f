// between.h -- launchers of the operators between the products (norm.hip,
// route.hip).  Not part of the public interface (see include/bpg.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bpg {

// RMSNorm of x (+ residual), rotation and quantization (norm.hip).
struct NormProblem {
    const void *x;        // [m][ldx], bf16 bits when x_bf16, else fp32
    const void *residual; // [m][ldr] or null, of the stream's type
    void *h;              // [m][ldh] or null: x + residual in the stream's type
    const void *weight;   // [k] or null
    void *codes;
    float *scales;
    int64_t m, k, ldx, ldr, ldh;
    float eps;
    double inv_k; // set by the launcher: 1 / k
    int act_bits, rot;
    bool x_bf16, residual_bf16, weight_bf16;
};
hipError_t launch_norm_quantize(const NormProblem &p, hipStream_t stream);
// The values of codes times scales, rotated back; y fp32 or bf16 bits [m][ldy].
hipError_t launch_dequantize(const void *codes, const float *scales, int act_bits, int rot,
                             int64_t m, int64_t k, void *y, bool y_bf16, int64_t ldy,
                             hipStream_t stream);

// Routing of tokens to experts (route.hip).
struct RouteProblem {
    const void *logits; // [tokens][ldl], bf16 bits when logits_bf16, else fp32
    const float *bias;  // [experts] or null
    int32_t *expert_of; // [tokens][topk]
    float *weights;     // [tokens][topk]
    int64_t tokens, ldl;
    int experts, topk, groups, kept;
    float scale;
    bool logits_bf16, sigmoid, pair, renormalize;
    uint32_t size_magic; // set by the launcher: ceil(2^20 / group size),
    int lanes_shift;     // and log2 of the lanes that share a group
};
hipError_t launch_route_topk(const RouteProblem &p, hipStream_t stream);

} // namespace bpg
