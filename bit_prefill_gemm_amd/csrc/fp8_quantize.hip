// fp8_quantize.hip -- activations and weights to e4m3 codes with a scale per
// block of 128 (gfx950).
//
//   a = max |x| over the block, d = a / 448, r = min(1 / d, FLT_MAX) (0 where
//   d is 0), code = e4m3(x r)
//
// both divisions IEEE, each step one fp32 rounding, the code to nearest even.
// 448 is the largest e4m3 value; x r is at most 448 (1 + 2^-22), which rounds
// to it.  A multiplication by r, not a division by d: a code may then differ
// from that of x / d where x / d is within an ulp of fp32 of a rounding border
// of e4m3, which is not further from x.
#include "fp8.h"

#include <algorithm>
#include <cfloat>

namespace bpg {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// eight values of a row; its address is a multiple of 8 bytes
template <bool BF16> struct Eight;

template <> struct Eight<true> {
    v4u raw;
    __device__ __forceinline__ void load(const void *x, int64_t i)
    {
        __builtin_memcpy(&raw, __builtin_assume_aligned(static_cast<const uint16_t *>(x) + i, 8), 16);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(raw[i] << 16);
            v[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u);
        }
    }
};

template <> struct Eight<false> {
    v4f lo, hi;
    __device__ __forceinline__ void load(const void *x, int64_t i)
    {
        const float *p = static_cast<const float *>(x) + i;
        lo = *reinterpret_cast<const v4f *>(p);
        hi = *reinterpret_cast<const v4f *>(p + 4);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = lo[i];
            v[4 + i] = hi[i];
        }
    }
};

// the largest magnitude as bits: a NaN is above every number
__device__ __forceinline__ uint32_t top_of(const float (&v)[8])
{
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; i++)
        a = max(a, __float_as_uint(v[i]) & 0x7fffffffu);
    return a;
}

template <int CTRL> __device__ __forceinline__ uint32_t max_dpp(uint32_t a)
{
    return max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, CTRL, 0xf, 0xf, true));
}

// the maximum over a row of 16 lanes, in each of them (rotations by 8, 4, 2, 1)
__device__ __forceinline__ uint32_t max16(uint32_t a)
{
    a = max_dpp<0x128>(a);
    a = max_dpp<0x124>(a);
    a = max_dpp<0x122>(a);
    return max_dpp<0x121>(a);
}

__device__ __forceinline__ float inverse(float d) { return d > 0.0f ? fminf(1.0f / d, FLT_MAX) : 0.0f; }

__device__ __forceinline__ v2u codes_of(const float (&v)[8], float r)
{
    v2u c;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * r, v[4 * i + 1] * r, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * r, v[4 * i + 3] * r, w, true);
        c[i] = (uint32_t)w;
    }
    return c;
}

// Blocks of 1 x 128: 16 lanes a block, eight values a lane, so that a wave
// reads and writes whole lines; blocks are numbered over all rows, which leaves
// no lane idle at any width.  Bound by memory: 8192 x 5120 bf16 (127 MB) 21 us,
// 6.0 TB/s, the outputs left in the last cache; a launch of its own for one row.
constexpr int kUnroll = 2;

template <bool BF16>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void *x, int64_t ldx, int64_t k,
                                                            uint32_t blocks, uint32_t begin,
                                                            uint32_t total, uint32_t magic,
                                                            int shift, uint8_t *codes,
                                                            float *scales)
{
    const uint32_t lane = threadIdx.x & 15;
    const uint32_t first = begin + blockIdx.x * (16 * kUnroll) + (threadIdx.x >> 4);
    Eight<BF16> in[kUnroll];
    uint32_t id[kUnroll], row[kUnroll], col[kUnroll];
    bool live[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
        id[u] = first + 16 * u;
        row[u] = (uint32_t)(((uint64_t)id[u] * magic) >> shift);
        col[u] = (id[u] - row[u] * blocks) * kFp8Block + 8 * lane;
        live[u] = id[u] < total && col[u] < k;
        in[u] = Eight<BF16>{};
        if (live[u])
            in[u].load(x, (int64_t)row[u] * ldx + col[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
        float v[8];
        in[u].values(v);
        const float d = __uint_as_float(max16(top_of(v))) / 448.0f;
        if (live[u]) {
            *reinterpret_cast<v2u *>(codes + (int64_t)row[u] * k + col[u]) = codes_of(v, inverse(d));
            if (lane == 0)
                scales[id[u]] = d;
        }
    }
}

// Blocks of 128 x 128: a workgroup a block, 64 values a thread in registers.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_square_kernel(const void *x, int64_t ldx, int64_t m,
                                                              int64_t k, uint8_t *codes,
                                                              float *scales)
{
    __shared__ uint32_t part[16];
    const int lane = threadIdx.x & 15, line = threadIdx.x >> 4;
    const int64_t row = (int64_t)blockIdx.y * kFp8Block + line;
    const int64_t col = (int64_t)blockIdx.x * kFp8Block + 8 * lane;
    Eight<BF16> in[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        in[i] = Eight<BF16>{};
        if (row + 16 * i < m && col < k)
            in[i].load(x, (row + 16 * i) * ldx + col);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        float v[8];
        in[i].values(v);
        top = max(top, top_of(v));
    }
    top = max16(top);
    if (lane == 0)
        part[line] = top;
    __syncthreads();
    const float d = __uint_as_float(max16(part[lane])) / 448.0f;
    const float r = inverse(d);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        float v[8];
        in[i].values(v);
        if (row + 16 * i < m && col < k)
            *reinterpret_cast<v2u *>(codes + (row + 16 * i) * k + col) = codes_of(v, r);
    }
    if (threadIdx.x == 0)
        scales[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = d;
}

} // namespace

hipError_t launch_fp8_quantize(const void *x, bool bf16, int64_t m, int64_t k, int64_t ldx,
                               bool square, void *codes, float *scales, hipStream_t stream)
{
    if (m == 0)
        return hipSuccess;
    const int64_t blocks = fp8_blocks(k);
    uint8_t *out = static_cast<uint8_t *>(codes);
    if (square) {
        const dim3 grid((unsigned)blocks, (unsigned)fp8_blocks(m));
        if (bf16)
            quantize_square_kernel<true><<<grid, 256, 0, stream>>>(x, ldx, m, k, out, scales);
        else
            quantize_square_kernel<false><<<grid, 256, 0, stream>>>(x, ldx, m, k, out, scales);
        return hipGetLastError();
    }
    // id / blocks as a multiplication, exact below 2^31
    const uint32_t total = (uint32_t)(m * blocks);
    int log2 = 0;
    while (((int64_t)1 << log2) < blocks)
        log2++;
    const uint32_t magic = (uint32_t)(((uint64_t)1 << (31 + log2)) / (uint64_t)blocks + 1);
    // 2^28 blocks a launch: a grid holds fewer than 2^32 threads
    for (int64_t begin = 0; begin < total; begin += 1 << 28) {
        const int64_t count = std::min((int64_t)total - begin, (int64_t)1 << 28);
        const unsigned grid = (unsigned)((count + 16 * kUnroll - 1) / (16 * kUnroll));
        (bf16 ? quantize_rows_kernel<true> : quantize_rows_kernel<false>)<<<grid, 256, 0, stream>>>(
            x, ldx, k, (uint32_t)blocks, (uint32_t)begin, total, magic, 31 + log2, out, scales);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace bpg
