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
// rounded.  Both scores are monotone, so without a bias the logits themselves
// are the keys.  A NaN logit counts as -inf (score 0), +inf as the largest
// fp32; a row of -inf only has softmax scores 0 and weights 0.
//
// One wave per token; lane l holds experts l, l + 64, ...  What bounds it is
// issue: fp64 exponentials of every expert and an arg-max per choice.  So the
// choice is first made on fp32 keys, whose error is bounded; wherever two keys
// that the choice has to tell apart lie closer than that bound, the wave makes
// it again on fp64 keys (choose).  Only the chosen
// experts' scores are then computed in fp64 (all of them for softmax weights
// that are not renormalised).  Measured (in a graph; an empty launch is 1.9
// us): 1 x 128, top-8 softmax 2.6 us; 512 x 128 3.1; 4099 x 256 bf16 in 8
// groups, sigmoid and bias 7.9 (675 vector and 345 scalar instructions a token,
// most of the scalar ones from the merge of a group's lanes, whose distance is a
// run-time value); 16384 x 512, top-10 softmax and bias 20.2, of
// which 690 vector instructions a token are 18.7.  With every score and key in
// fp64 and shuffles for the reductions these were 6.5, 7.3, 31.6 and 53.4 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "between.h"

namespace bpg {

namespace {

__device__ __forceinline__ float load_logit(const float *p, int i) { return p[i]; }
__device__ __forceinline__ float load_logit(const uint16_t *p, int i)
{
    return __uint_as_float((uint32_t)p[i] << 16);
}

// Lane l gets the value of lane l - 1, 2, 4, 8 of its row of 16 (row_shr), or
// of the last lane of the row (pair of rows) before it (row_bcast), 0 where
// there is none: after the six steps lane 63 has seen every lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}

constexpr int kShr1 = 0x111, kShr2 = 0x112, kShr4 = 0x114, kShr8 = 0x118;
constexpr int kBcast15 = 0x142, kBcast31 = 0x143;

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
    v = max(v, dpp_u32<kShr1, 0xF>(v));
    v = max(v, dpp_u32<kShr2, 0xF>(v));
    v = max(v, dpp_u32<kShr4, 0xF>(v));
    v = max(v, dpp_u32<kShr8, 0xF>(v));
    v = max(v, dpp_u32<kBcast15, 0xA>(v));
    v = max(v, dpp_u32<kBcast31, 0xC>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// the largest of 64-bit keys: by the upper words, then by the lower ones of
// the lanes that have the largest upper word
__device__ __forceinline__ uint64_t wave_max_key(uint64_t v)
{
    const uint32_t hi = wave_max_u32((uint32_t)(v >> 32));
    const uint32_t lo = wave_max_u32((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ uint32_t wave_max_key(uint32_t v) { return wave_max_u32(v); }

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint64_t lo = dpp_u32<CTRL, ROWS>((uint32_t)b), hi = dpp_u32<CTRL, ROWS>((uint32_t)(b >> 32));
    return __longlong_as_double((long long)(lo | (hi << 32)));
}

// lane i's value
__device__ __forceinline__ float read_lane(float v, int i)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i));
}

__device__ __forceinline__ double read_lane(double v, int i)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, i);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), i);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

__device__ __forceinline__ double wave_sum(double v)
{
    v += dpp_f64<kShr1, 0xF>(v);
    v += dpp_f64<kShr2, 0xF>(v);
    v += dpp_f64<kShr4, 0xF>(v);
    v += dpp_f64<kShr8, 0xF>(v);
    v += dpp_f64<kBcast15, 0xA>(v);
    v += dpp_f64<kBcast31, 0xC>(v);
    return read_lane(v, 63);
}

__device__ __forceinline__ float wave_sum(float v)
{
    v += __uint_as_float(dpp_u32<kShr1, 0xF>(__float_as_uint(v)));
    v += __uint_as_float(dpp_u32<kShr2, 0xF>(__float_as_uint(v)));
    v += __uint_as_float(dpp_u32<kShr4, 0xF>(__float_as_uint(v)));
    v += __uint_as_float(dpp_u32<kShr8, 0xF>(__float_as_uint(v)));
    v += __uint_as_float(dpp_u32<kBcast15, 0xA>(__float_as_uint(v)));
    v += __uint_as_float(dpp_u32<kBcast31, 0xC>(__float_as_uint(v)));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// A float or double as an unsigned integer of the same order, -0 as 0; every
// number is above 0, which stands for "not in the choice".
__device__ __forceinline__ uint32_t ordered(float f)
{
    const uint32_t b = __float_as_uint(f + 0.0f);
    return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ uint64_t ordered(double f)
{
    const uint64_t b = (uint64_t)__double_as_longlong(f + 0.0);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000u);
}

__device__ __forceinline__ float unordered(uint32_t u)
{
    return __uint_as_float(u ^ ((uint32_t)((int)~u >> 31) | 0x80000000u));
}

__device__ __forceinline__ double unordered(uint64_t u)
{
    return __longlong_as_double(
        (long long)(u ^ ((uint64_t)((int64_t)~u >> 63) | 0x8000000000000000u)));
}

__device__ __forceinline__ float largest(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double largest(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ float smallest(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smallest(double a, double b) { return fmin(a, b); }

// fp32 e^x within (2.5 |x| + 2) 2^-24 relative (0 below the normal numbers)
__device__ __forceinline__ float exp_fast(float x)
{
    return __builtin_amdgcn_exp2f(x * 1.44269504f);
}

// e / size for e < 512, with magic = ceil(2^20 / size)
__device__ __forceinline__ int group_of(const RouteProblem &p, int e)
{
    return (int)(((uint32_t)e * p.size_magic) >> 20);
}

// LDS written by lanes of this wave is read by others of it
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The topk largest of the wave's keys (0: not in the choice), largest first,
// ties to the lowest expert: lane j gets choice j.
template <int NE>
__device__ __forceinline__ void take_exact(uint64_t (&key)[NE], int topk, int lane, int &chosen)
{
    for (int j = 0; j < topk;) {
        uint64_t best = key[0];
#pragma unroll
        for (int i = 1; i < NE; i++)
            best = best > key[i] ? best : key[i];
        const uint64_t m = wave_max_key(best);
        if (m == 0)
            return; // nothing is left
#pragma unroll
        for (int i = 0; i < NE; i++) {
            uint64_t at = __ballot(key[i] == m);
            key[i] = key[i] == m ? 0 : key[i];
            for (; at != 0 && j < topk; at &= at - 1, j++)
                if (lane == j)
                    chosen = 64 * i + __builtin_ctzll(at);
        }
    }
}

// Sorts N values of a lane, largest first (Batcher's odd-even merge).
template <int N>
__device__ __forceinline__ void sort_lane(uint32_t (&v)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; i++)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t a = v[i + j], b = v[i + j + k];
                        v[i + j] = max(a, b);
                        v[i + j + k] = min(a, b);
                    }
}

// 1 / (1 + e^-l)
__device__ __forceinline__ double sigmoid_f64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }

// e^(l - top), 0 where l is -inf
__device__ __forceinline__ double exp_f64(float l, float top)
{
    return l == -INFINITY ? 0.0 : exp((double)l - (double)top);
}

// Over all experts: the sum of exp_f64.
template <int NE>
__device__ __forceinline__ double exp_sum(const float (&l)[NE], float top)
{
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NE; i++)
        sum += exp_f64(l[i], top);
    return wave_sum(sum);
}

// The same on fp32 keys.  Each lane sorts its keys once and the wave then
// takes the largest head, one pop a choice.  The lowest log2(NE) bits of a key
// give way to the key's place in its lane, upside down: the order of these
// words is that of the shortened keys, then of the experts.  It is that of the
// keys themselves wherever two consecutive words differ by more than both
// keys' tolerances, tol0 + tol1 (1 + |key|) where the keys are approximate and
// the shortened bits where they are exact.  Where some do not, more words are
// taken until one is clear of the rest, and the taken ones are ranked by their
// fp64 keys.  Returns false if 64 words were not enough for that.
//   ls: the logits by expert
template <int NE>
__device__ __forceinline__ bool take_fast(const RouteProblem &p, uint32_t (&key)[NE],
                                          const float (&l)[NE], float top, const float *ls,
                                          float tol0, int lane, int &chosen)
{
    const bool approximate = p.bias != nullptr;
    // one rounding of p + bias (half an ulp) and the shortened bits
    constexpr float tol1 = (2 + 2 * (NE - 1)) * 0x1p-24f;
#pragma unroll
    for (int i = 0; i < NE; i++)
        key[i] = (key[i] & ~(uint32_t)(NE - 1)) | (NE - 1 - i); // below NE: not in the choice
    sort_lane<NE>(key);
    uint32_t word = 0; // lane j keeps the word of choice j
    int from = 0;      // and its lane
    int count = 0;
    auto take = [&](int n) {
        for (; count < n; count++) {
            const uint32_t m = wave_max_u32(key[0]);
            const int w = __builtin_ctzll(__ballot(key[0] == m));
            if (lane == count) {
                word = m;
                from = w;
            }
            // (a select written as ?: over the array became an indexed one)
            const uint32_t pop = lane == w ? ~0u : 0u;
#pragma unroll
            for (int i = 0; i + 1 < NE; i++)
                key[i] = (pop & key[i + 1]) | (~pop & key[i]);
            key[NE - 1] &= ~pop;
        }
    };
    // bit j: words j and j + 1 are too close (a word below NE: nothing was left)
    auto too_close = [&]() -> uint64_t {
        const uint32_t next = (uint32_t)__shfl_down((int)word, 1);
        bool close;
        if (approximate) {
            // (a difference of infinities is NaN, which is not clear)
            const float k = unordered(word), k1 = unordered(next);
            close = !(k - k1 > 2.0f * (tol0 + tol1 * (1.0f + fabsf(k))));
        } else {
            close = (word ^ next) < NE;
        }
        return __ballot(close && next >= NE && lane + 1 < count);
    };
    auto expert = [&]() { return (NE - 1 - (int)(word & (NE - 1))) * 64 + from; };

    const bool whole = !approximate && (NE == 1 || p.logits_bf16); // the bits given were all equal
    take(p.topk < 64 && !whole ? p.topk + 1 : p.topk);
    chosen = expert();
    if (whole)
        return true;
    if (p.topk == 64)
        return false;
    uint64_t close = too_close();
    if (close == 0)
        return true;
    while ((close >> (count - 2)) & 1) {
        if (count == 64)
            return false;
        take(count + 1);
        close = too_close();
    }
    const int taken = __popcll(__ballot(word >= NE)); // of count: the experts may have run out
    const int e = lane < taken ? expert() : 0;
    double k = (double)ls[e];
    if (approximate) {
        double s;
        if (p.sigmoid) {
            s = sigmoid_f64(ls[e]);
        } else {
            const double sum = exp_sum<NE>(l, top); // 0 where every logit is -inf
            s = sum > 0.0 ? exp_f64(ls[e], top) / sum : 0.0;
        }
        k = fmax(s + (double)p.bias[e], -INFINITY);
    }
    int rank = 0;
    for (int i = 0; i < taken; i++) {
        const double ki = read_lane(k, i);
        const int ei = __builtin_amdgcn_readlane(e, i);
        rank += ki > k || (ki == k && ei < e);
    }
    chosen = __builtin_amdgcn_ds_permute(4 * (lane < taken ? rank : lane), e);
    return true;
}

// The value of lane ^ d inside every 2 d lanes, for lanes whose values are
// equal inside every d (d < 16 on the DPP path: a mirror is as good as the
// exchange then).
__device__ __forceinline__ float other_half(float v, int d)
{
    const int b = __float_as_int(v);
    switch (d) {
    case 1: return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0xB1, 0xF, 0xF, true));  // quad_perm 1,0,3,2
    case 2: return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0x4E, 0xF, 0xF, true));  // quad_perm 2,3,0,1
    case 4: return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0x141, 0xF, 0xF, true)); // row_half_mirror
    case 8: return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0x140, 0xF, 0xF, true)); // row_mirror
    default: return __shfl_xor(v, d);
    }
}

__device__ __forceinline__ double other_half(double v, int d) { return __shfl_xor(v, d); }

// The choice of a token.  V = double: on fp64 keys, always made.  V = float:
// on fp32 keys; false where they are too close to tell.  The fp32 scores are
// within (35 + 2.5 |x|) 2^-24 p for softmax (x = l - max l; the sum of the
// exponentials is off by less than 31 2^-24: their own errors weighted by p,
// where the mean of |x| is at most ln 512, and 13 additions), and |x| p is at
// most 0.37 max p; for sigmoid within (1 - p) (2.5 |l| + 2) 2^-24 + 3 2^-24 of
// p, and |l| p (1 - p) is below 0.23.  tol0 holds that: 40 2^-24 max p, and
// 5 2^-24.  A sum of two scores without a bias is within 2^-16 of itself.
//   ls: the logits by expert; scratch: E values of V
template <int NE, typename V>
__device__ __forceinline__ bool choose(const RouteProblem &p, const float (&l)[NE], float top,
                                       const float (&bias)[NE], const float *ls, V *scratch,
                                       int lane, int &chosen)
{
    typedef decltype(ordered(V(0))) K;
    constexpr bool fast = sizeof(V) == 4;
    const int E = p.experts;
    const bool grouped = p.groups > p.kept; // every group is kept otherwise
    const bool scores = p.bias || (grouped && p.pair);
    K key[NE];
    V score[NE]; // p, with a bias the key
    float tol0 = 0.0f;
    if (scores) {
        if (p.sigmoid) {
#pragma unroll
            for (int i = 0; i < NE; i++) {
                if constexpr (fast)
                    score[i] = __builtin_amdgcn_rcpf(1.0f + exp_fast(-l[i]));
                else
                    score[i] = sigmoid_f64(l[i]);
            }
            tol0 = 5 * 0x1p-24f;
        } else {
            V sum = 0;
            // (a row of -inf only: 0 instead of the difference of infinities)
            const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int i = 0; i < NE; i++) {
                if constexpr (fast)
                    score[i] = exp_fast(l[i] - base);
                else
                    score[i] = exp_f64(l[i], top);
                sum += score[i];
            }
            sum = wave_sum(sum);
            const V r = sum > V(0) ? V(1) / sum : V(0);
#pragma unroll
            for (int i = 0; i < NE; i++)
                score[i] = score[i] * r;
            tol0 = 40 * 0x1p-24f * (float)r; // the largest score is r
        }
    }
#pragma unroll
    for (int i = 0; i < NE; i++) {
        V k = l[i];
        if (p.bias) {
            k = score[i] + (V)bias[i];
            k = largest(k, -(V)INFINITY); // NaN to -inf
            score[i] = k;
        }
        key[i] = lane + 64 * i < E ? ordered(k) : 0;
    }

    if (grouped) {
        const int size = E / p.groups;
#pragma unroll
        for (int i = 0; i < NE; i++)
            if (lane + 64 * i < E)
                scratch[lane + 64 * i] = p.pair ? score[i] : unordered(key[i]);
        wave_fence();
        // `per` lanes per group, a power of two, each over every per-th of its experts
        const int shift = p.lanes_shift, per = 1 << shift;
        const int g = lane >> shift, sub = lane & (per - 1);
        V a = -INFINITY, b = -INFINITY;
        if (g < p.groups) {
#pragma unroll 4
            for (int q = sub; q < size; q += per) {
                const V v = scratch[g * size + q];
                b = largest(b, smallest(a, v));
                a = largest(a, v);
            }
        }
        wave_fence();
        for (int d = 1; d < per; d <<= 1) {
            const V a2 = other_half(a, d), b2 = other_half(b, d);
            b = largest(smallest(a, a2), largest(b, b2));
            a = largest(a, a2);
        }
        V gs = largest(p.pair ? a + b : a, -(V)INFINITY); // NaN (+inf and -inf) to -inf
        // a group's rank: how many score more, or as much and come first
        int rank = 0;
        for (int o = 0; o < p.groups; o++) {
            const V so = read_lane(gs, o << shift);
            rank += so > gs || (so == gs && o < g);
        }
        const bool first = sub == 0 && g < p.groups;
        if (fast && scores) {
            const V last = read_lane(gs, __builtin_ctzll(__ballot(first && rank == p.kept - 1)));
            const V next = read_lane(gs, __builtin_ctzll(__ballot(first && rank == p.kept)));
            V tol = V(0x1p-16f) * last + V(0x1p-100f);
            if (p.bias) {
                V big = 0; // the largest finite key bounds the error of a sum of two
#pragma unroll
                for (int i = 0; i < NE; i++)
                    if (lane + 64 * i < E && fabs(score[i]) < (V)INFINITY)
                        big = largest(big, (V)fabs(score[i]));
                big = unordered(wave_max_key(ordered(big)));
                tol = V(2) * ((V)tol0 + V(0x1p-22f) * (V(1) + big));
            }
            if (!(last - next > V(2) * tol)) // (nor are infinities told apart)
                return false;
        }
        const uint64_t kept = __ballot(first && rank < p.kept);
#pragma unroll
        for (int i = 0; i < NE; i++)
            key[i] = (kept >> ((group_of(p, lane + 64 * i) << shift) & 63)) & 1 ? key[i] : 0;
    }
    if constexpr (fast) {
        return take_fast<NE>(p, key, l, top, ls, tol0, lane, chosen);
    } else {
        take_exact<NE>(key, p.topk, lane, chosen);
        return true;
    }
}

constexpr int kWaves = 4; // tokens per workgroup

template <typename T, int NE>
__global__ __launch_bounds__(64 * kWaves) void route_topk_kernel(RouteProblem p)
{
    __shared__ float logits[kWaves][64 * NE];
    __shared__ double scratch[kWaves][64 * NE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t token = (int64_t)blockIdx.x * kWaves + wave;
    if (token >= p.tokens)
        return; // uniform across the wave; no workgroup barrier follows
    const T *row = static_cast<const T *>(p.logits) + token * p.ldl;
    float *ls = logits[wave];
    const int E = p.experts;
    float l[NE], bias[NE];
    // (unmasked loads: lanes past the last expert read that one)
#pragma unroll
    for (int i = 0; i < NE; i++)
        l[i] = load_logit(row, min(lane + 64 * i, E - 1));
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < NE; i++)
            bias[i] = p.bias[min(lane + 64 * i, E - 1)];
    }
#pragma unroll
    for (int i = 0; i < NE; i++)
        l[i] = lane + 64 * i < E ? l[i] : -INFINITY;
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NE; i++) {
        l[i] = fminf(fmaxf(l[i], -INFINITY), 0x1.fffffep127f); // NaN to -inf
        best = max(best, ordered(l[i]));
    }
    const float top = unordered(wave_max_u32(best));
#pragma unroll
    for (int i = 0; i < NE; i++)
        ls[lane + 64 * i] = l[i];
    wave_fence();
    int chosen = 0; // lane j keeps choice j
    if (!choose<NE, float>(p, l, top, bias, ls, reinterpret_cast<float *>(scratch[wave]), lane,
                           chosen))
        choose<NE, double>(p, l, top, bias, ls, scratch[wave], lane, chosen);

    // the chosen experts' scores, in fp64
    const float lc = ls[lane < p.topk ? chosen : 0];
    double w;
    w = p.sigmoid ? sigmoid_f64(lc) : exp_f64(lc, top);
    if (p.renormalize || !p.sigmoid) {
        const double sum = p.renormalize ? wave_sum(lane < p.topk ? w : 0.0) : exp_sum<NE>(l, top);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (lane < p.topk) {
        p.expert_of[token * p.topk + lane] = chosen;
        p.weights[token * p.topk + lane] = (float)(w * (double)p.scale);
    }
}

template <typename T>
void launch_type(const RouteProblem &p, hipStream_t stream)
{
    const dim3 grid((unsigned)((p.tokens + kWaves - 1) / kWaves));
    if (p.experts <= 64)
        route_topk_kernel<T, 1><<<grid, 64 * kWaves, 0, stream>>>(p);
    else if (p.experts <= 128)
        route_topk_kernel<T, 2><<<grid, 64 * kWaves, 0, stream>>>(p);
    else if (p.experts <= 256)
        route_topk_kernel<T, 4><<<grid, 64 * kWaves, 0, stream>>>(p);
    else
        route_topk_kernel<T, 8><<<grid, 64 * kWaves, 0, stream>>>(p);
}

} // namespace

hipError_t launch_route_topk(const RouteProblem &problem, hipStream_t stream)
{
    if (problem.tokens == 0)
        return hipSuccess;
    RouteProblem p = problem;
    const int size = p.experts / p.groups;
    p.size_magic = (uint32_t)(((1 << 20) + size - 1) / size);
    p.lanes_shift = 0;
    while ((p.groups << (p.lanes_shift + 1)) <= 64)
        p.lanes_shift++;
    if (p.logits_bf16)
        launch_type<uint16_t>(p, stream);
    else
        launch_type<float>(p, stream);
    return hipGetLastError();
}

} // namespace bpg
