// Routing of tokens to experts: the n_used best of n_expert logits per token, with
// weights, for the expert products.
//
// A row has a warp, or half of one where it has few experts; as many warps as are resident go from row to row with
// the next one's logits on their way (16384 rows on 4864 warps are 3.4 each, so that some have 4 and others 3). A lane
// holds a run of neighbouring experts in registers, so that a row is
// read once and no block waits for another. It sorts its own keys (a network of minima and maxima, without the
// experts) into a list in shared memory; then the best of all lanes are taken one a round, by one
// reduction over the lists' heads and a ballot: of equal heads the lowest lane's, which are the lowest
// experts'. Lane i keeps the i-th key and its lane, and finds the expert by the key among that lane's. The weights
// are computed for the chosen alone. A group whose experts are those of whole lanes has its highest keys at
// its lanes' heads.
//
// Keys with a bias (and sums of two keys) are sums of rounded numbers: two of them that
// are close in 32 bits may be in the other order. Where neighbours in the ranking, or the groups on both sides of
// the choice, are closer than twice their error, the keys that may matter (or all, where these are more
// than 32) are computed in 64 bits and ranked again; with random logits that is one row in some hundreds.
// That code is kept short rather than unrolled: it is not in the SM's instruction cache when it is
// needed, and one such row lengthened the kernel by 18 us while all of the row was ranked again by unrolled code.
//
// Error of the difference of two keys, S the row's largest score, n the experts of a lane. A term
// exp(x - m) has 2^-22 of ex2.approx, and t 2^-22.9 of its argument, a difference t that is
// rounded, times log2 e rounded: at most 0.37 2^-22.9 S as t e^-t <= 0.37. A softmax's sum is off by
// (n + 5) 2^-24 of itself beside that, by which the difference of two scores changes, S at most. Together below
// (n + 29) 2^-24 S. A sigmoid: 2^-24 by ex2 (s (1 - s) <= 1/4), 2^-25.5 by its argument, 2^-23 by
// the reciprocal, 2^-24 by 1 + e: 2^-21 for two. s + bias rounds by 2^-24 of the key. The margins below
// are twice these.
//
// What of this reaches the weights: without norm a softmax's sum with the errors above; with norm nothing, they are made of expf, a
// sum of n_used and divisions.
//
// The margin of a row follows the largest finite |bias| of all experts. One that masks by -1e9 and not by -inf makes every row
// go through all candidates and be ranked in 64 bits: the same experts, but the case below takes 600 us instead of 18.5.
//
// What bounds it: instructions. 16384 rows of 256 experts, the best 8 of 4 groups of 8 by sigmoid + bias: 18.5 us
// (17.8 MB: 2.7 us at the copy rate), 811 instructions a row at two thirds of the issue rate; 52 us with keys searched
// in registers in every round, 45 with lists of keys and experts sorted together. Without groups and bias 11.6.
#include <algorithm>

#include "q2_0_device.cuh"
#include "q2_0_internal.h"

namespace q2 {

namespace {

constexpr int kWarps = 4;           // of a block
constexpr int kTwoExperts = 160;    // most experts of a row that has half a warp
static_assert(kTwoExperts <= 16 * 16, "");
constexpr int kTwoTokens = 8;       // and least rows an SM
constexpr float kMax = 3.402823466e38f;

__device__ __forceinline__ bool masks(float v) { return !(v > -INFINITY); }

// The warp's largest (no NaN).
__device__ __forceinline__ float max_of(float v) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}
// exp and 1 / x within a few units, for keys
__device__ __forceinline__ float exp_near(float v) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * 1.44269504f));
    return e;
}
__device__ __forceinline__ float reciprocal_near(float v) {
    float e;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
    return e;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Group of expert e < 1024 for groups of `size` (>= 1): exact, as e * size < 2^22.
__device__ __forceinline__ int group_of(int e, uint32_t inv) { return int((uint32_t(e) * inv) >> 22); }

// A group's score of its two highest keys: the highest, or half the sum of both (a sum of two may be beyond f32; without
// a second one, -inf, half the first).
template <typename T>
__device__ __forceinline__ T group_score(T a, T b, bool two) {
    return two ? T(0.5) * a + (b > T(-INFINITY) ? T(0.5) * b : T(0)) : a;
}

// The groups that are chosen from, as a mask: g's sum of its `top` highest keys (in `key`, this
// warp's copy of the row) is among the n_group_used highest. T float or double. *near is set
// where two scores that the choice parts are closer than `margin`.
template <typename T>
__device__ uint32_t best_groups(const T *key, const q2_0_router &r, int top, T margin, bool *near) {
    const int lane = threadIdx.x & 31;
    const int size = r.n_expert / r.n_group;
    int sub = 1;  // lanes of a group
    while (sub * 2 * r.n_group <= 32) sub *= 2;
    const int g = lane / sub, s = lane % sub;
    T a = T(-INFINITY), b = T(-INFINITY);  // the two highest
    if (g < r.n_group) {
        // (each group starts at another place, so that lanes meet different banks)
        const int n = (size - s + sub - 1) / sub;
        int i = n > 0 ? g % n : 0;
        for (int c = 0; c < n; ++c) {
            const T v = key[g * size + s + i * sub];
            if (v > a) {
                b = a;
                a = v;
            } else if (v > b) {
                b = v;
            }
            if (++i == n) i = 0;
        }
    }
    for (int o = 1; o < sub; o <<= 1) {
        const T a2 = __shfl_xor_sync(~0u, a, o), b2 = __shfl_xor_sync(~0u, b, o);
        if (a2 > a) {
            b = a > b2 ? a : b2;
            a = a2;
        } else {
            b = b > a2 ? b : a2;
        }
    }
    const T score = group_score(a, b, top == 2);
    int rank = 0;
    for (int h = 0; h < r.n_group; ++h) {
        const T other = __shfl_sync(~0u, score, h * sub);
        rank += other > score || (other == score && h < g);
    }
    const bool mine = g < r.n_group && s == 0;
    const bool in = mine && rank < r.n_group_used;
    // the lowest of the chosen and the highest of the others
    T lo = in ? score : T(INFINITY), hi = mine && !in ? score : T(-INFINITY);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const T l2 = __shfl_xor_sync(~0u, lo, o), h2 = __shfl_xor_sync(~0u, hi, o);
        lo = l2 < lo ? l2 : lo;
        hi = h2 > hi ? h2 : hi;
    }
    *near = hi > T(-INFINITY) && lo - hi < margin;
    uint32_t set = 0;
    const uint32_t votes = __ballot_sync(~0u, in);
    for (int h = 0; h < r.n_group; ++h) set |= ((votes >> (h * sub)) & 1u) << h;
    return set;
}

// Order of doubles as whole numbers above 0 (no NaN).
__device__ __forceinline__ uint64_t ordered(double v) {
    const int64_t b = __double_as_longlong(v + 0.0);  // (-0 is 0)
    return uint64_t(b ^ (b >> 63 | int64_t(1) << 63));
}

// A key in 64 bits (-inf: masked). `scores`: of scores, otherwise the logit; m, z: a softmax's
// largest logit and sum.
__device__ __noinline__ double key64(const float *x, const q2_0_router &r, int e, bool scores, double m, double z) {
    const float xe = x[e], be = r.bias ? r.bias[e] : 0.0f;
    if (masks(xe) || masks(be)) return -INFINITY;
    const double v = fminf(xe, kMax);
    if (!scores) return v;
    const bool softmax = r.score == Q2_0_SCORE_SOFTMAX;
    const double t = exp(softmax ? v - m : -v);
    return (softmax ? t : 1.0) / (softmax ? z : 1.0 + t) + double(fminf(be, kMax));
}
// A softmax's largest logit and sum in 64 bits.
__device__ __noinline__ void sum64(const float *x, const q2_0_router &r, int lane, double &m, double &z) {
    float mf = -kMax;
    for (int e = lane; e < r.n_expert; e += 32)
        if (!masks(x[e])) mf = fmaxf(mf, fminf(x[e], kMax));
    m = max_of(mf);
    z = 0;
#pragma unroll 2
    for (int e = lane; e < r.n_expert; e += 32)
        if (!masks(x[e])) z += exp(double(fminf(x[e], kMax)) - m);
    z = warp_sum(z);
}

// The whole row again with keys in 64 bits: lane i returns the i-th expert. `key` is the warp's
// place for n_expert doubles. Few rows come here, to code that is not in the SM's cache: it is short rather than
// unrolled.
__device__ __noinline__ int rank64(const float *x, const q2_0_router &r, int lane, double *key) {
    const bool grouped = r.n_group_used < r.n_group, sums = grouped && r.group_top == 2;
    const int size = r.n_expert / r.n_group;
    // without a bias the logits rank (scores may round to the same value), but for sums of two scores
    bool scores = r.bias || sums;
    double m = 0, z = 1;
    if (scores && r.score == Q2_0_SCORE_SOFTMAX) sum64(x, r, lane, m, z);
    __syncwarp();
#pragma unroll 1
    for (int e = lane; e < r.n_expert; e += 32) key[e] = key64(x, r, e, scores, m, z);
    uint32_t set = ~0u;
    if (grouped) {
        __syncwarp();
        bool near;
        set = best_groups<double>(key, r, r.group_top, 0.0, &near);
        __syncwarp();
        if (!r.bias && sums)
#pragma unroll 1
            for (int e = lane; e < r.n_expert; e += 32) key[e] = key64(x, r, e, false, m, z);
    }
    // ranked as whole numbers of the same order (0: taken, or of another group), by the lanes that hold them
    uint64_t *const o = reinterpret_cast<uint64_t *>(key);
#pragma unroll 1
    for (int e = lane; e < r.n_expert; e += 32) o[e] = (set >> (grouped ? e / size : 0)) & 1u ? ordered(key[e]) : 0;
    int mine = 0;
#pragma unroll 1
    for (int i = 0; i < r.n_used; ++i) {
        uint64_t best = 0;
        int at = lane;
#pragma unroll 1
        for (int e = lane; e < r.n_expert; e += 32)
            if (o[e] > best) {
                best = o[e];
                at = e;
            }
        const uint32_t hi = __reduce_max_sync(~0u, uint32_t(best >> 32));
        const uint32_t lo = __reduce_max_sync(~0u, uint32_t(best >> 32) == hi ? uint32_t(best) : 0u);
        const int e = int(__reduce_min_sync(~0u, best == (uint64_t(hi) << 32 | lo) ? unsigned(at) : ~0u));
        if (i == lane) mine = e;
        if ((e & 31) == lane) o[e] = 0;
    }
    return mine;
}

// n candidates in 64 bits, lane i < n having expert e: the n_used best of them, in their order. `slot` is
// the warp's place for 32 numbers.
__device__ __noinline__ int rank64_of(const float *x, const q2_0_router &r, int lane, int n, int e, int *slot) {
    double m = 0, z = 1;
    if (r.score == Q2_0_SCORE_SOFTMAX) sum64(x, r, lane, m, z);
    const uint64_t o = lane < n ? ordered(key64(x, r, e, true, m, z)) : 0;
    int rank = 0;
#pragma unroll 1
    for (int h = 0; h < n; ++h) {
        const uint64_t other = __shfl_sync(~0u, o, h);
        const int other_e = __shfl_sync(~0u, e, h);
        rank += other > o || (other == o && other_e < e);
    }
    __syncwarp();
    slot[lane] = e;  // (ranks are all different; were they not, what stands here is an expert)
    __syncwarp();
    if (lane < n) slot[rank] = e;
    __syncwarp();
    return slot[lane < n ? lane : 0];
}

// ---------------------------------------------------------------------------
// A row has kW lanes of a warp: all 32, or 16, so that a warp goes through two rows at once.
// ---------------------------------------------------------------------------
// The largest of a row's lanes (no NaN).
template <int kW>
__device__ __forceinline__ float row_max(float v) {
    if constexpr (kW == 32) {
        return max_of(v);
    } else {
#pragma unroll
        for (int o = kW / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
        return v;
    }
}
template <int kW>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = kW / 2; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}
// A vote of the row's lanes, its first lane's in bit 0.
template <int kW>
__device__ __forceinline__ uint32_t row_votes(bool is) {
    const uint32_t votes = __ballot_sync(~0u, is);
    if constexpr (kW == 32) return votes;
    return votes >> (threadIdx.x & 32 - kW) & ((1u << (kW & 31)) - 1);
}

// Whether the lane's group (of `lanes` lanes of its row) is one of the n_group_used best, by scores in 64 bits.
// Of a lane's `have` keys (or logits, without a bias) in their order and sorted, those from `least` on (a key)
// may be among the group's highest. x: the lane's row; m, z: its softmax's largest logit and sum.
template <int kW>
__device__ __noinline__ bool among_best64(const float *x, const q2_0_router &r, int lanes, const float *key, int have,
                                          const float *sorted, int n, float least, double m, double z) {
    const int in_row = threadIdx.x & (kW - 1), row_lane = threadIdx.x & 32 - kW;
    double a = -INFINITY, b = -INFINITY;
    const int e0 = in_row * ((r.n_expert + kW - 1) / kW);
    __syncwarp();  // (the lists have been written)
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const float k = sorted[kW * i];
        // without a bias sorted[] are logits, in their scores' order: the first two are the highest
        const bool may = k > -INFINITY && (r.bias ? k >= least : i < 2);
        if (!__any_sync(~0u, may)) break;
        if (!may) continue;
        int before = 0, e = e0;  // of equal keys the next one
        for (int j = 0; j < i; ++j) before += sorted[kW * j] == k;
#pragma unroll 1
        for (int j = 0; j < have; ++j)
            if (key[j] == k && before-- == 0) e = e0 + j;
        const double d = key64(x, r, e, true, m, z);
        if (d > a) {
            b = a;
            a = d;
        } else if (d > b) {
            b = d;
        }
    }
    __syncwarp();
    for (int o = 1; o < lanes; o <<= 1) {
        const double a2 = __shfl_xor_sync(~0u, a, o), b2 = __shfl_xor_sync(~0u, b, o);
        if (a2 > a) {
            b = a > b2 ? a : b2;
            a = a2;
        } else {
            b = b > a2 ? b : a2;
        }
    }
    const double score = r.group_top == 2 && b > -INFINITY ? a + b : a;
    const int g = in_row / lanes;
    int rank = 0;
    for (int h = 0; h < r.n_group; ++h) {
        const double other = __shfl_sync(~0u, score, row_lane + h * lanes);
        rank += other > score || (other == score && h < g);
    }
    return rank < r.n_group_used && g < r.n_group;
}

// Descending, by Batcher's odd-even merging.
template <int kE, int kP = 1, int kK = 1>
__device__ __forceinline__ void sort_descending(float (&v)[kE]) {
    if constexpr (kP < kE) {
#pragma unroll
        for (int a = kK % kP; a + kK < kE; ++a)
            if ((a - kK % kP) % (2 * kK) < kK && a / (2 * kP) == (a + kK) / (2 * kP)) {
                const float hi = fmaxf(v[a], v[a + kK]);
                v[a + kK] = fminf(v[a], v[a + kK]);
                v[a] = hi;
            }
        if constexpr (kK > 1)
            sort_descending<kE, kP, kK / 2>(v);
        else
            sort_descending<kE, 2 * kP, 2 * kP>(v);
    }
}

// Blocks of an SM. (Half a warp a row, 128 experts: 6 blocks 7.6 us, 8 8.0; a warp a row, 256: 6 20.8, 8 18.3.)
template <int kW, int kE>
constexpr int kResident = kE <= 8 ? (kW == 32 ? 8 : 6) : kE == 16 ? 6 : 4;

// Floats in shared memory of a row: its keys, its lists, -inf behind them, and what a lane looks at beyond
// that (a value it does not use) when its list has come to the end.
template <int kW, int kE>
constexpr int kFloats = kW * (2 * kE + 3);

template <int kW, int kE, bool kBias, bool kGrouped>
__global__ void __launch_bounds__(kWarps * 32, kResident<kW, kE>) route_kernel(
    const __grid_constant__ q2_0_router r, const float *logits, int64_t stride, int64_t n_tokens, int32_t *ids,
    float *weights, int wide) {
    constexpr int kRows = 32 / kW;  // of a warp
    extern __shared__ __align__(16) float lists[];  // of each row: keys by expert [kW kE], sorted in lanes [kE + 3][kW]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, in_row = lane & (kW - 1), row = lane / kW;
    float *const warp_s = lists + warp * (kRows * kFloats<kW, kE>);
    float *const key_s = warp_s + row * kFloats<kW, kE>, *const sorted_s = key_s + kW * kE + in_row;
    sorted_s[kW * kE] = -INFINITY;
    const bool softmax = r.score == Q2_0_SCORE_SOFTMAX;
    const bool sums = kGrouped && r.group_top == 2;  // of two scores
    const int size = kGrouped ? r.n_expert / r.n_group : r.n_expert;
    const int per = (r.n_expert + kW - 1) / kW, e0 = in_row * per;
    const int have = max(0, min(per, r.n_expert - e0));  // experts of this lane
    // lanes of a group, if its experts are those of whole lanes and they are a power of two
    int lanes = kGrouped ? size / per : 0;
    if (lanes * per != size || (lanes & (lanes - 1))) lanes = 0;
    const int shift = lanes ? __ffs(lanes) - 1 : 0;
    float bias[kE], most = 0.0f;
#pragma unroll
    for (int j = 0; j < kE; ++j) {
        bias[j] = 0.0f;
        if (kBias && j < have) bias[j] = fminf(fmaxf(r.bias[e0 + j], -INFINITY), kMax);
        if (bias[j] > -INFINITY) most = fmaxf(most, fabsf(bias[j]));
    }
    most = max_of(most);
    auto load = [&](const float *x, float (&v)[kE]) {
        if (wide) {
            if constexpr (kE >= 4) {
#pragma unroll
                for (int j = 0; j < kE; j += 4) {
                    float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                    if (j < have) f = *reinterpret_cast<const float4 *>(x + e0 + j);
                    v[j] = f.x;
                    v[j + 1] = f.y;
                    v[j + 2] = f.z;
                    v[j + 3] = f.w;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < kE; ++j) v[j] = j < have ? x[e0 + j] : -INFINITY;
        }
    };
    const int64_t step = int64_t(gridDim.x) * kWarps * kRows;
    int64_t t0 = (int64_t(blockIdx.x) * kWarps + warp) * kRows;  // the warp's first row
    auto row_of = [&](int64_t t, int h) { return logits + min(t + h, n_tokens - 1) * stride; };  // (a last row may be there twice)
    const uint32_t below = (1u << in_row) - 1;
    float ahead[kE];  // the next row's logits, on their way
    if (t0 < n_tokens) load(row_of(t0, row), ahead);
    for (; t0 < n_tokens; t0 += step) {
        const float *x = row_of(t0, row);
        float v[kE];
#pragma unroll
        for (int j = 0; j < kE; ++j) v[j] = ahead[j];
        if (t0 + step < n_tokens) load(row_of(t0 + step, row), ahead);
#pragma unroll
        for (int j = 0; j < kE; ++j) v[j] = fminf(fmaxf(v[j], -INFINITY), kMax);  // (NaN: -inf)
        // a softmax's sum, where scores of their own are needed
        float m = 0.0f, z = 0.0f;
        if (softmax && (kBias || !r.norm || sums)) {
            m = -INFINITY;
#pragma unroll
            for (int j = 0; j < kE; ++j) m = fmaxf(m, v[j]);
            m = fmaxf(row_max<kW>(m), -kMax);
#pragma unroll
            for (int j = 0; j < kE; ++j) z += exp_near(v[j] - m);
            z = row_sum<kW>(z);
        }
        const float inv_z = reciprocal_near(z);
        auto near_score = [&](float y) { return softmax ? exp_near(y - m) * inv_z : reciprocal_near(1.0f + exp_near(-y)); };
        if (kBias && softmax) {
#pragma unroll
            for (int j = 0; j < kE; ++j) v[j] = v[j] > -INFINITY ? fmaf(exp_near(v[j] - m), inv_z, bias[j]) : -INFINITY;
        } else if (kBias) {
#pragma unroll
            for (int j = 0; j < kE; ++j)
                v[j] = v[j] > -INFINITY ? reciprocal_near(1.0f + exp_near(-v[j])) + bias[j] : -INFINITY;
        }
        float margin = 0.0f;
        if (kBias || sums) margin = softmax ? float(per + 32) * 0x1p-23f * inv_z : 0x1p-20f;
        if (kBias) margin += 0x1p-22f * (1.0f + most);
        const float group_margin = r.group_top == 2 ? margin : 2.0f * margin;  // (of half a sum of two: half of two keys')
        bool full = false, in = true;  // full: the whole row has to be ranked in 64 bits
        if (kGrouped && !lanes) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kE; ++j)
                if (j < have) key_s[e0 + j] = kBias || !sums || v[j] == -INFINITY ? v[j] : near_score(v[j]);
            __syncwarp();
            uint32_t set = 0;
#pragma unroll 1
            for (int h = 0; h < kRows; ++h) {
                bool near;
                const uint32_t s = best_groups<float>(warp_s + h * kFloats<kW, kE>, r, r.group_top,
                                                      __shfl_sync(~0u, group_margin, h * kW), &near);
                if (h == row) {
                    set = s;
                    full = near;
                }
            }
            const uint32_t inv = ((1u << 22) + size - 1) / size;
#pragma unroll
            for (int j = 0; j < kE; ++j)
                if (!((set >> (group_of(e0 + j, inv) & 31)) & 1u)) v[j] = -INFINITY;
        }
        __syncwarp();
        if (wide) {
            if constexpr (kE >= 4) {
#pragma unroll
                for (int j = 0; j < kE; j += 4)
                    if (j < have)
                        *reinterpret_cast<float4 *>(key_s + e0 + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kE; ++j)
                if (j < have) key_s[e0 + j] = v[j];
        }
        sort_descending<kE>(v);
#pragma unroll
        for (int j = 0; j < kE; ++j) sorted_s[kW * j] = v[j];
        if (kGrouped && lanes) {
            float a = v[0], b = kE > 1 ? v[kE > 1 ? 1 : 0] : -INFINITY;  // the two highest
            if (!kBias && sums) {
                a = a > -INFINITY ? near_score(a) : a;
                b = b > -INFINITY ? near_score(b) : b;
            }
            for (int o = 1; o < lanes; o <<= 1) {
                const float a2 = __shfl_xor_sync(~0u, a, o), b2 = __shfl_xor_sync(~0u, b, o);
                b = fmaxf(fmaxf(b, b2), fminf(a, a2));
                a = fmaxf(a, a2);
            }
            const float score = group_score(a, b, r.group_top == 2);
            const int g = in_row >> shift;
            float left = g < r.n_group ? score : -INFINITY, lowest = 0.0f;
            in = false;
            for (int h = 0; h < r.n_group_used; ++h) {
                lowest = row_max<kW>(left);
                if ((__ffs(row_votes<kW>(left == lowest)) - 1) >> shift == g) {
                    in = true;
                    left = -INFINITY;
                }
            }
            full = lowest == -INFINITY;  // groups of masked experts alone: which are taken is seen to below
            const float highest = row_max<kW>(left);
            const bool near = margin > 0.0f && highest > -INFINITY && lowest - highest < group_margin;
            if (__any_sync(~0u, near)) {
                double m64 = 0, z64 = 1;
                if (softmax)
#pragma unroll 1
                    for (int h = 0; h < kRows; ++h) {
                        double mh, zh;
                        sum64(row_of(t0, h), r, lane, mh, zh);
                        if (h == row) {
                            m64 = mh;
                            z64 = zh;
                        }
                    }
                const bool best = among_best64<kW>(x, r, lanes, key_s + e0, have, sorted_s, kE,
                                                   (r.group_top == 2 && b > -INFINITY ? b : a) - margin, m64, z64);
                if (near) in = best;
            }
        }
        __syncwarp();
        // the best n_used, and one more to see how close it is: of the lanes whose lists are headed
        // by the highest key the first one's, and in a lane its experts of that key in their order
        float head = in ? v[0] : -INFINITY, mine_key = -INFINITY, top = 0.0f;
        const float *at = sorted_s + kW;
        float next = in ? *at : -INFINITY;
        uint32_t mine_votes = 0;
        auto take = [&](int i, bool go) {  // go: the row takes one
            top = row_max<kW>(head);
            const bool is = head == top;
            const uint32_t votes = row_votes<kW>(is);
            // (nothing is taken from lists that have come to the end; a warp's only row stops there instead)
            const bool first = is && go && (kW == 32 || top > -INFINITY) && !(votes & below), mine = i == in_row && go;
            mine_key = mine ? top : mine_key;
            mine_votes = mine ? votes : mine_votes;
            head = first ? next : head;
            at += first ? kW : 0;
            next = *at;
        };
        for (int i = 0; i < r.n_used && (kW < 32 || top > -INFINITY); ++i) take(i, true);
        full |= !(top > -INFINITY);  // too few are not masked
        int taken = r.n_used;
        if (kBias) {
            const float least = top - margin;
            float behind = row_max<kW>(head);
            // others that may be among the best: candidates of the lanes behind
            while (true) {
                const bool go = behind > least && taken < kW && !full;
                if (!__any_sync(~0u, go)) break;
                take(taken, go);
                taken += go;
                behind = row_max<kW>(head);
            }
            full |= behind > least;
        }
        // the expert: in its lane the one with as many of the same key before it as were taken before it
        const int from = max(0, __ffs(mine_votes) - 1), up_from = __shfl_up_sync(~0u, from, 1);
        const float up_key = __shfl_up_sync(~0u, mine_key, 1);
        const bool behind_one = in_row && in_row < taken;
        const uint32_t same = row_votes<kW>(behind_one && up_from == from && up_key == mine_key);
        int mine = 0;
        const float *of = key_s + from * per;
        if (!__any_sync(~0u, same)) {
#pragma unroll
            for (int j = kE - 1; j >= 0; --j)
                if (j < per && of[j] == mine_key) mine = j;
        } else {
            int left = __clz(~(same << (31 - in_row)));
            for (int j = 0; j < per; ++j)
                if (of[j] == mine_key && left-- == 0) mine = j;
        }
        mine = min(mine + from * per, r.n_expert - 1);  // (of lanes that took none: any)
        {
            const bool close = kBias && row_votes<kW>(behind_one && up_key - mine_key < margin);
            if (__any_sync(~0u, full || close)) {
#pragma unroll 1
                for (int h = 0; h < kRows; ++h) {
                    const bool all = __shfl_sync(~0u, full, h * kW), some = __shfl_sync(~0u, close, h * kW);
                    if (!all && !some) continue;
                    float *const place = warp_s + h * kFloats<kW, kE>;
                    const int n = __shfl_sync(~0u, taken, h * kW), e = __shfl_sync(~0u, mine, h * kW + in_row);
                    int got = all ? rank64(row_of(t0, h), r, lane, reinterpret_cast<double *>(place))
                                  : rank64_of(row_of(t0, h), r, lane, n, e, reinterpret_cast<int *>(place));
                    got = __shfl_sync(~0u, got, in_row);
                    if (h == row) mine = got;
                }
            }
        }
        // weights of the chosen
        float y = -INFINITY;
        if (in_row < r.n_used) {
            const float b = kBias ? r.bias[mine] : 0.0f;
            y = x[mine];
            y = masks(y) || masks(b) ? -INFINITY : fminf(y, kMax);
        }
        float w = 0.0f;
        const float small = expf(-fabsf(y));  // sigmoid(y) = 1 / (1 + small), or small / (1 + small) for y < 0
        if (!r.norm) {
            if (y > -INFINITY) w = softmax ? expf(y - m) / z : (y < 0.0f ? small : 1.0f) / (1.0f + small);
        } else {
            // relative to the largest, so that no sum of scores is 0 or loses bits
            const float highest = row_max<kW>(y);
            w = y < 0.0f ? small : 1.0f;
            if (softmax || highest < 0.0f) w = expf(y - highest);
            if (!softmax) w = __fdividef(w, 1.0f + small);  // (a divisor in [1, 2]: within 2^-22)
            if (!(y > -INFINITY)) w = 0.0f;
            const float sum = row_sum<kW>(w);
            if (sum > 0.0f) w /= sum;
        }
        if (in_row < r.n_used && t0 + row < n_tokens) {
            ids[(t0 + row) * r.n_used + in_row] = mine;
            weights[(t0 + row) * r.n_used + in_row] = w * r.scale;
        }
    }
}

template <int kW, int kE>
cudaError_t launch(const q2_0_router &r, const float *logits, int64_t stride, int64_t n_tokens, int32_t *ids,
                   float *weights, cudaStream_t s) {
    const int per = (r.n_expert + kW - 1) / kW;
    const bool wide = per % 4 == 0 && r.n_expert % 4 == 0 && stride % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15u) == 0;
    // as many warps as are resident at once: each goes through rows, with the bias in registers
    constexpr int kRows = 32 / kW;
    const int64_t blocks = std::min<int64_t>((n_tokens + kWarps * kRows - 1) / (kWarps * kRows),
                                             int64_t(sm_count()) * kResident<kW, kE>);
    const bool grouped = r.n_group_used < r.n_group;
    auto *const kernel = r.bias ? (grouped ? route_kernel<kW, kE, true, true> : route_kernel<kW, kE, true, false>)
                                : (grouped ? route_kernel<kW, kE, false, true> : route_kernel<kW, kE, false, false>);
    kernel<<<unsigned(blocks), kWarps * 32, kWarps * kRows * kFloats<kW, kE> * sizeof(float), s>>>(
        r, logits, stride, n_tokens, ids, weights, wide);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route(const q2_0_router &r, const float *logits, int64_t stride, int64_t n_tokens, int32_t *ids,
                         float *weights, cudaStream_t s) {
    // Two rows a warp where there are rows for all SMs: fewer instructions a row, but more registers and longer chains.
    // us of 16384 rows, one row a warp / two: 64 experts, best 8 8.6 / 6.8; 128 9.3 / 7.6; 160, 6 of 3 groups of 8
    // 14.7 / 11.8; 256 11.6 / 12.5 (with groups and bias 18.4 / 19.5); 512, best 10 18.3 / 29.7
    const bool two = r.n_used <= 16 && r.n_expert <= kTwoExperts && r.n_group <= 16 && n_tokens >= kTwoTokens * int64_t(sm_count());
    const int per_lane = two ? (r.n_expert + 15) / 16 : (r.n_expert + 31) / 32;
#define LAUNCH(e) \
    if (per_lane <= e) return two ? launch<16, e>(r, logits, stride, n_tokens, ids, weights, s) : launch<32, e>(r, logits, stride, n_tokens, ids, weights, s)
    LAUNCH(1);
    LAUNCH(2);
    LAUNCH(4);
    LAUNCH(8);
    LAUNCH(16);
#undef LAUNCH
    // (kTwoExperts are 10 a lane of half a warp)
    return launch<32, 32>(r, logits, stride, n_tokens, ids, weights, s);
}

}  // namespace q2
