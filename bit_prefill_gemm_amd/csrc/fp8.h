// fp8.h -- launchers of the 8-bit floating-point route (fp8_quantize.hip,
// fp8_stream.hip, fp8_tile.hip) and of the log probabilities of tokens
// (logprobs.hip).  Not part of the public interface (see include/bpg.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bpg {

constexpr int kFp8Block = 128; // values under one scale

__host__ __device__ inline int64_t fp8_blocks(int64_t k)
{
    return (k + kFp8Block - 1) / kFp8Block;
}

// x [m][ldx] (fp32, or bf16 bits) to e4m3 codes [m][k] with a scale per block
// of 1 x 128 values, or of 128 x 128 (square).
hipError_t launch_fp8_quantize(const void *x, bool bf16, int64_t m, int64_t k, int64_t ldx,
                               bool square, void *codes, float *scales, hipStream_t stream);

// Products of e4m3 codes: y = x . w^T, or act(x . w^T) * (x . up^T) where `up`
// is set.
struct Fp8Problem {
    const uint8_t *codes;  // activations [m][k]
    const float *scales;   // [m][blocks of k]
    const uint8_t *w;      // [n][k]
    const float *w_scales; // [blocks of n][blocks of k]
    const uint8_t *up;     // the second matrix of a gated product, or null
    const float *up_scales;
    int64_t m, n, k;
    void *y;               // [m][ldy], bf16 bits when y_bf16, else fp32
    int64_t ldy;
    bool y_bf16;
    bool exact;            // products added in fp32 (fp8_mma.h)
    int act;               // bpg_activation (gated)
};
size_t fp8_gemm_bytes(const Fp8Problem &p); // of the workspace
hipError_t launch_fp8_gemm(const Fp8Problem &p, void *workspace, hipStream_t stream);
// The gated product (p.y, ldy, y_bf16 unused) as codes [m][n] and scales
// [m][blocks of n]; workspace: fp8_gated_quantize_bytes(p) bytes.
size_t fp8_gated_quantize_bytes(const Fp8Problem &p);
hipError_t launch_fp8_gated_quantize(const Fp8Problem &p, uint8_t *codes, float *scales,
                                     void *workspace, hipStream_t stream);

// Which kernels make which columns, from the shape alone (fp8_tile.hip); the
// launches above go by it.
enum Fp8Kernel {
    kFp8None = 0,
    kFp8Stream,          // few rows: each wave streams its part of K (fp8_stream.hip)
    kFp8Tile256x256,     // rows x columns (gated: columns of both matrices)
    kFp8Tile128x128Pair, // two workgroups a CU
    kFp8Tile128x128,     // one, with loads further ahead
    kFp8Tile64x128,
    kFp8Tile64x64,       // two halves of K a workgroup
    kFp8Tile64x256,      // a gated product's codes
};
struct Fp8Part {
    int kernel;
    int64_t first, cols;
    int splits; // parts of K, joined by another launch; 0 or 1: one
};
struct Fp8Plan {
    Fp8Part part[2]; // the second may have no columns
    bool staged;     // fp32 values in a workspace, quantized behind it
};
Fp8Plan plan_fp8_gemm(const Fp8Problem &p);
Fp8Plan plan_fp8_codes(const Fp8Problem &p);
const char *fp8_plan_name(const Fp8Plan &plan);

constexpr int kFp8StreamRows = 32; // at most
hipError_t launch_fp8_stream(const Fp8Problem &p, hipStream_t stream);

// Log probabilities, entropies and top alternatives of rows of logits.
struct LogprobsProblem {
    const void *logits;  // [rows][ldl], bf16 bits when bf16, else fp32
    const void *tokens;  // [rows] int32 or int64 (wide), or null
    float *logprobs;     // [rows], or null without tokens
    float *entropy;      // [rows]
    int32_t *ids;        // [rows][topk]
    float *top;          // [rows][topk]
    int64_t rows, vocab, ldl;
    int topk;
    bool bf16, wide;
};
size_t logprobs_bytes(int64_t rows, int64_t vocab, int topk);
hipError_t launch_logprobs(const LogprobsProblem &p, void *workspace, hipStream_t stream);

} // namespace bpg
