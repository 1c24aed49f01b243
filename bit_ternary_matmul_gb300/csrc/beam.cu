// q2_0_beam_select: the n best continuations of each group of beams over the
// vocabulary, by running score + log-softmax of the logits.
//
// A beam's order by score is its order by logit, so one pass over the logits
// finds both what the log-softmax needs (running maximum and sum of
// exponentials) and the only candidates that can be selected: each beam's n
// best. Pass 1 does so per chunk of a row, pass 2 joins a group's chunks. The
// logits are read once from memory: 4 bytes, one exponential and a comparison
// each. Nothing depends on the order in which blocks run.
#include <float.h>

#include <algorithm>

#include "q2_0_device.cuh"
#include "q2_0_internal.h"

namespace q2 {

namespace {

constexpr int kThreads1 = 256;
constexpr int kPiece = 16 * kThreads1;         // logits of a piece
constexpr int kBlocks1 = 4;                    // blocks per SM
constexpr int kThreads2 = 512;
constexpr int kCap1 = 512;                     // survivors held in shared memory
constexpr int kCap2 = 1024;
constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.44269504f;
constexpr float kHuge = 1e30f;                 // maxima beyond it take the long way

// Bits that order as the floats do (x not NaN, no -0): above 0 for x > -inf.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// A candidate of a row: larger logit first, then lower token. 0: none.
__device__ __forceinline__ uint64_t cand_key(float x, uint32_t token) {
    return uint64_t(ordered(x)) << 32 | (0xFFFFFFFFu - token);
}

// The n-th largest (1..32) of the lanes' values.
__device__ __forceinline__ float warp_nth(float v, int n) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const float o = __shfl_xor_sync(0xffffffffu, v, j);
            const bool up = ((lane & k) == 0) == ((lane & j) == 0);  // the lower lane of a pair keeps the larger
            v = up ? fmaxf(v, o) : fminf(v, o);
        }
    return __shfl_sync(0xffffffffu, v, n - 1);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct Work {
    // [rows][chunks] (R, s): the chunk's sum of exponentials is s 2^R, R a whole number;
    // or, where its maximum is beyond kHuge, (m, -s): s e^m
    float2 *sums;
    uint64_t *keys;  // [rows][chunks][n_out], best first, 0 where there are no more
    int chunks, steps;  // pieces of a chunk
};

// Two f32 operations in one instruction.
union Pair {
    float2 f;
    unsigned long long u;
};
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    Pair x{a}, y{b}, z{c}, d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.u) : "l"(x.u), "l"(y.u), "l"(z.u));
    return d.f;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    Pair x{a}, y{b}, d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(x.u), "l"(y.u));
    return d.f;
}

// Pass 1: one block per (chunk, row). A chunk is up to `steps` pieces of 4096 logits,
// 16 to a thread; the next piece is loaded while one is worked on. A thread keeps the
// sum of its own elements, of 2^(x log2(e) - R) with R a whole number, so that the
// exponent is one fused multiply-add, rounded near 0, and R ln 2 can be added to
// the logarithm without loss later.
// The first piece gives the threshold that leaves few candidates: in each warp the
// n-th largest of the lanes' maxima, the largest of those over the warps; at least
// n values of the chunk reach it. Its survivors are ranked by counting, and the
// n-th of them is the threshold from then on. Too many survivors (later pieces with
// larger values, or ties): the chunk is read again with the largest of its pieces'
// thresholds, and if that does not help, n times for a maximum each.
// The long ways are also taken by chunks with a maximum beyond kHuge or a NaN (seen
// in the sum), which counts as -inf there.
__global__ void __launch_bounds__(kThreads1, kBlocks1)
    select_chunk_kernel(const SelectArgs a, const Work w) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t row = blockIdx.y;
    const int chunk = blockIdx.x;
    if (a.done && a.done[row]) return;
    __shared__ float s_m[8], s_s[8], s_t[8], s_thr;
    __shared__ __align__(16) uint64_t s_key[kCap1];
    __shared__ int s_n;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) s_n = 0;
    // The row in 16-byte blocks: block b holds elements 4 b - off .. + 3.
    const float *p = a.logits + row * a.stride;
    const int off = int((reinterpret_cast<uintptr_t>(p) >> 2) & 3);
    const int V = int(a.n_vocab);
    const int p0 = chunk * w.steps, p1 = min(p0 + w.steps, (V + off + kPiece - 1) / kPiece);
    using Values = float[16];
    auto load = [&](int piece, Values &x) {
        const int first = piece * kPiece + 4 * tid - off;  // element of x[0]
        if ((piece > 0 || off == 0) && (piece + 1) * kPiece - off <= V) {
            const float4 *p4 = reinterpret_cast<const float4 *>(p + first);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4 *>(x + 4 * i) = __ldcs(p4 + i * kThreads1);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = first + 4 * i * kThreads1;
                if (e >= 0 && e + 4 <= V) {
                    *reinterpret_cast<float4 *>(x + 4 * i) =
                        __ldcs(reinterpret_cast<const float4 *>(p + e));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[4 * i + j] = e + j >= 0 && e + j < V ? p[e + j] : kNegInf;
                }
            }
        }
    };
    auto key_of = [&](int piece, int i, float v) {
        return cand_key(fminf(v, FLT_MAX) + 0.0f,
                        uint32_t(piece * kPiece + 4 * (tid + (i / 4) * kThreads1) - off + i % 4));
    };
    auto maximum = [](const Values &x) {  // (NaN is passed over)
        float tm = kNegInf;
#pragma unroll
        for (int i = 0; i < 16; ++i) tm = fmaxf(tm, x[i]);
        return tm;
    };
    auto threshold = [&](float tm) {  // called by all threads
        const float t = warp_nth(tm, a.n_out);
        __syncthreads();
        if (lane == 0) s_t[warp] = t;
        __syncthreads();
        float v = -FLT_MAX;
#pragma unroll
        for (int i = 0; i < 8; ++i) v = fmaxf(v, s_t[i]);
        return v;
    };
    float thr = -FLT_MAX;
    auto collect = [&](int piece, float tm, const Values &x) {
        if (tm < thr) return;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (x[i] >= thr) {
                const int at = atomicAdd(&s_n, 1);
                if (at < kCap1) s_key[at] = key_of(piece, i, x[i]);
            }
    };
    auto rank_of = [&](uint64_t k, int n) {
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) rank += s_key[j] > k;
        return rank;
    };
    float most = kNegInf, R = -kHuge, sum = 0.0f;
    auto work = [&](int piece, const Values &x) {
        const float tm = maximum(x);
        most = fmaxf(most, tm);
        // A thread whose maximum is below -kHuge adds nothing to a chunk whose maximum is
        // above; a maximum above kHuge: what comes out here is not used.
        if (tm > -kHuge && tm * kLog2e > R) {
            const float Rn = ceilf(tm * kLog2e);
            sum *= ex2(R - Rn);
            R = Rn;
        }
        const float r = R > -kHuge ? -R : 0.0f;
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float2 e = fma2(make_float2(x[i], x[i + 1]), make_float2(kLog2e, kLog2e), make_float2(r, r));
            s = add2(s, make_float2(ex2(e.x), ex2(e.y)));
        }
        sum += s.x + s.y;
        // (a piece in which little may be chosen gives no threshold: the next one does)
        if (piece == p0 || thr <= -FLT_MAX) {
            thr = threshold(tm);
            collect(piece, tm, x);
            if (piece + 1 < p1) {
                if (tid == 0) s_thr = thr;
                __syncthreads();
                const int n = s_n;
                if (n <= kCap1)
                    for (int i = tid; i < n; i += kThreads1) {
                        const uint64_t k = s_key[i];
                        if (rank_of(k, n) == a.n_out - 1) s_thr = unordered(uint32_t(k >> 32));
                    }
                __syncthreads();
                thr = s_thr;
            }
        } else {
            collect(piece, tm, x);
        }
    };
    Values x, y;
    if (p0 < p1) load(p0, x);
    for (int piece = p0; piece < p1; piece += 2) {
        if (piece + 1 < p1) load(piece + 1, y);
        work(piece, x);
        if (piece + 2 < p1) load(piece + 2, x);
        if (piece + 1 < p1) work(piece + 1, y);
    }
    const float wm = warp_max(most);
    const float wr = warp_max(R);
    sum = warp_sum(sum * ex2(R - wr));
    __syncthreads();
    if (lane == 0) {
        s_m[warp] = wm;
        s_t[warp] = wr;
        s_s[warp] = sum;
    }
    __syncthreads();
    float m = s_m[0];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m = fmaxf(m, s_m[i]);
        nan |= s_s[i] != s_s[i];
    }
    const int64_t rec = row * w.chunks + chunk;
    if (!nan && (m == kNegInf || fabsf(m) < kHuge)) {
        if (warp == 7) {
            const float Rw = lane < 8 ? s_t[lane] : -kHuge;
            const float top = warp_max(Rw);
            const float s = warp_sum(Rw > -kHuge ? s_s[lane & 7] * ex2(Rw - top) : 0.0f);
            if (lane == 0) w.sums[rec] = make_float2(top > -kHuge ? top : kNegInf, s);
        }
    } else {
        m = fminf(m, FLT_MAX);
        const bool whole = fabsf(m) < kHuge;  // only NaN brought it here: the first kind
        const float c = whole ? ceilf(m * kLog2e) : m;
        sum = 0.0f;
        for (int piece = p0; piece < p1; ++piece) {
            load(piece, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float v = fminf(fmaxf(x[i], kNegInf), FLT_MAX);
                sum += whole ? ex2(fmaf(v, kLog2e, -c)) : m == kNegInf ? 0.0f : ex2((v - c) * kLog2e);
            }
        }
        sum = warp_sum(sum);
        __syncthreads();
        if (lane == 0) s_s[warp] = sum;
        __syncthreads();
        if (tid == 0) {
            for (int i = 1; i < 8; ++i) sum += s_s[i];
            w.sums[rec] = make_float2(c, whole || m == kNegInf ? sum : -sum);
        }
    }
    __syncthreads();
    uint64_t *out = w.keys + rec * a.n_out;
    int n = s_n;
    if (n > kCap1) {
        for (int piece = p0; piece < p1; ++piece) {
            load(piece, x);
            thr = fmaxf(thr, threshold(maximum(x)));
        }
        if (tid == 0) s_n = 0;
        __syncthreads();
        for (int piece = p0; piece < p1; ++piece) {
            load(piece, x);
            collect(piece, maximum(x), x);
        }
        __syncthreads();
        n = s_n;
    }
    if (n <= kCap1) {
        // of many, first thin out again: the threshold of the survivors themselves
        if (n > 64) {
            float v[kCap1 / kThreads1], best = kNegInf;
#pragma unroll
            for (int j = 0; j < kCap1 / kThreads1; ++j) {
                const int i = tid + j * kThreads1;
                v[j] = i < n ? unordered(uint32_t(s_key[i] >> 32)) : kNegInf;
                best = fmaxf(best, v[j]);
            }
            const float least = threshold(best);
            uint64_t k[kCap1 / kThreads1];
#pragma unroll
            for (int j = 0; j < kCap1 / kThreads1; ++j)
                k[j] = v[j] >= least ? s_key[tid + j * kThreads1] : 0;
            if (tid == 0) s_n = 0;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kCap1 / kThreads1; ++j)
                if (k[j]) s_key[atomicAdd(&s_n, 1)] = k[j];
            __syncthreads();
            n = s_n;
        }
        for (int i = tid; i < n; i += kThreads1) {
            const uint64_t k = s_key[i];
            const int rank = rank_of(k, n);
            if (rank < a.n_out) out[rank] = k;
        }
        for (int i = n + tid; i < a.n_out; i += kThreads1) out[i] = 0;
        return;
    }
    uint64_t last = ~0ull;
    for (int r = 0; r < a.n_out; ++r) {
        uint64_t best = 0;
        for (int piece = p0; piece < p1; ++piece) {
            load(piece, x);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (x[i] >= thr) {
                    const uint64_t k = key_of(piece, i, x[i]);
                    if (k < last && k > best) best = k;
                }
        }
        for (int o = 16; o; o >>= 1) {
            const uint64_t v = __shfl_xor_sync(0xffffffffu, best, o);
            best = v > best ? v : best;
        }
        __syncthreads();
        if (lane == 0) s_key[warp] = best;
        __syncthreads();
        best = s_key[0];
        for (int i = 1; i < 8; ++i) best = s_key[i] > best ? s_key[i] : best;
        if (tid == 0) out[r] = best;
        last = best;
    }
}

// log of a row's sum from its chunks' (one warp). Sums of the two kinds differ so
// much that those of one kind alone count.
__device__ __forceinline__ float row_lse(const float2 *sums, int C) {
    const int lane = threadIdx.x & 31;
    const float2 none = make_float2(kNegInf, 0.0f);
    const float2 mine = lane < C ? __ldcg(sums + lane) : none;
    float R = kNegInf, m = kNegInf;  // the largest 2^R, the largest e^m
    for (int i = lane; i < C; i += 32) {
        const float2 c = i == lane ? mine : __ldcg(sums + i);
        if (c.y >= 0.0f)
            R = fmaxf(R, c.x);
        else
            m = fmaxf(m, c.x);
    }
    R = warp_max(R);
    m = warp_max(m);
    float s = 0.0f;
    if (m > 0.0f || (R == kNegInf && m > kNegInf)) {
        for (int i = lane; i < C; i += 32) {
            const float2 c = __ldcg(sums + i);
            if (c.y < 0.0f) s -= c.y * ex2((c.x - m) * kLog2e);
        }
        return m + logf(warp_sum(s));
    }
    if (R == kNegInf) return kNegInf;
    for (int i = lane; i < C; i += 32) {
        const float2 c = i == lane ? mine : __ldcg(sums + i);
        if (c.y > 0.0f) s += c.y * ex2(c.x - R);
    }
    s = warp_sum(s);
    // ln 2 in two parts, the first of 10 bits: its product with R is exact
    return fmaf(R, 0.693359375f, fmaf(R, -2.12194440e-4f, logf(s)));
}

// A continuation in a group's order: score, then lower beam, then the row's order.
struct Cand {
    uint32_t score;  // ordered bits, 0: none
    uint32_t beam;
    uint64_t key;
    __device__ __forceinline__ bool before(const Cand &o) const {
        if (score != o.score) return score > o.score;
        if (beam != o.beam) return beam < o.beam;
        return key > o.key;
    }
};

// Pass 2: one block per group. Every row's chunks are joined to the log of its sum.
// A chunk's candidates are in order, so the chunks' first ones give the threshold
// as the lanes' maxima do in pass 1, and each list is read only as far as it
// reaches it. The survivors are ranked as in pass 1.
__global__ void __launch_bounds__(kThreads2) select_group_kernel(const SelectArgs a, const Work w) {
    __shared__ float s_base[64], s_lse[64];
    __shared__ float s_t[kThreads2 / 32];
    __shared__ Cand s_c[kCap2];
    __shared__ int s_n;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row0 = int64_t(blockIdx.x) * a.n_beams;
    const int W = a.n_beams, C = w.chunks, n_out = a.n_out;
    if (tid == 0) s_n = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int b = warp; b < W; b += kThreads2 / 32) {
        const bool done = a.done && a.done[row0 + b];
        const float lse = done ? 0.0f : row_lse(w.sums + (row0 + b) * C, C);
        if (lane == 0) {
            s_lse[b] = lse;
            s_base[b] = a.score[row0 + b];
        }
    }
    __syncthreads();
    const int lists = W * C, per_beam = C * n_out, total = W * per_beam;
    const unsigned long long *keys =
        reinterpret_cast<const unsigned long long *>(w.keys) + row0 * per_beam;
    // candidate i < total of the chunks, i - total the beam of a finished one
    auto get = [&](int i, Cand &c) {
        c.score = 0;
        float s;
        if (i < total) {
            const int b = i / per_beam;
            if (a.done && a.done[row0 + b]) return;
            c.key = __ldcg(keys + i);
            if (!c.key) return;
            c.beam = uint32_t(b);
            s = s_base[b] + (unordered(uint32_t(c.key >> 32)) - s_lse[b]);
        } else {
            const int b = i - total;
            if (!a.done || !a.done[row0 + b]) return;
            c.beam = uint32_t(b);
            c.key = 1;
            s = s_base[b];
        }
        if (s > kNegInf) c.score = ordered(s + 0.0f);
    };
    uint32_t best = 0;
    for (int i = tid; i < lists + W; i += kThreads2) {
        Cand c;
        get(i < lists ? i * n_out : total + i - lists, c);
        best = max(best, c.score);
    }
    // no candidate counts as -inf, below every score
    const float t = warp_nth(best ? unordered(best) : kNegInf, n_out);
    if (lane == 0) s_t[warp] = t;
    __syncthreads();
    float thr = s_t[0];
#pragma unroll
    for (int i = 1; i < kThreads2 / 32; ++i) thr = fmaxf(thr, s_t[i]);
    const uint32_t least = thr > kNegInf ? ordered(thr) : 1u;
    for (int i = tid; i < lists + W; i += kThreads2) {
        const int from = i < lists ? i * n_out : total + i - lists;
        const int n = i < lists ? n_out : 1;
        for (int r = 0; r < n; ++r) {
            Cand c;
            get(from + r, c);
            if (c.score < least) break;
            const int at = atomicAdd(&s_n, 1);
            if (at < kCap2) s_c[at] = c;
        }
    }
    __syncthreads();
    const int n = s_n;
    float *so = a.score_out + int64_t(blockIdx.x) * n_out;
    int32_t *po = a.parent + int64_t(blockIdx.x) * n_out;
    int32_t *to = a.token + int64_t(blockIdx.x) * n_out;
    auto put = [&](int r, const Cand &c) {
        so[r] = c.score ? unordered(c.score) : kNegInf;
        po[r] = c.score ? int32_t(c.beam) : 0;
        to[r] = !c.score ? -1
                : a.done && a.done[row0 + c.beam]
                    ? a.done_token
                    : int32_t(0xFFFFFFFFu - uint32_t(c.key & 0xFFFFFFFFu));
    };
    if (n <= kCap2) {
        for (int i = tid; i < n; i += kThreads2) {
            const Cand c = s_c[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += s_c[j].before(c);
            if (rank < n_out) put(rank, c);
        }
        for (int i = n + tid; i < n_out; i += kThreads2) put(i, Cand{0, 0, 0});
        return;
    }
    Cand last{0xFFFFFFFFu, 0, ~0ull};  // before every candidate
    for (int r = 0; r < n_out; ++r) {
        Cand c{0, 0, 0};
        for (int i = tid; i < total + W; i += kThreads2) {
            Cand o;
            get(i, o);
            if (o.score && last.before(o) && o.before(c)) c = o;
        }
        for (int o = 16; o; o >>= 1) {
            Cand v;
            v.score = __shfl_xor_sync(0xffffffffu, c.score, o);
            v.beam = __shfl_xor_sync(0xffffffffu, c.beam, o);
            v.key = __shfl_xor_sync(0xffffffffu, c.key, o);
            if (v.before(c)) c = v;
        }
        __syncthreads();
        if (lane == 0) s_c[warp] = c;
        __syncthreads();
        c = s_c[0];
        for (int i = 1; i < kThreads2 / 32; ++i)
            if (s_c[i].before(c)) c = s_c[i];
        if (tid == 0) put(r, c);
        last = c;
        if (!c.score) {  // no more
            for (int i = r + 1 + tid; i < n_out; i += kThreads2) put(i, c);
            break;
        }
    }
}

// Chunks of a row: the number with which the blocks, kBlocks1 per SM at a time, are done
// first, a block costing its pieces and about 4 pieces' time of its own.
int chunks_of(size_t rows, int pieces) {
    const size_t at_once = size_t(kBlocks1) * std::max(1, sm_count());
    int best = 1;
    size_t best_cost = ~size_t(0);
    for (int c = 1; c <= pieces && rows * c <= 4 * at_once + rows; ++c) {
        const size_t waves = (rows * c + at_once - 1) / at_once;
        const size_t cost = waves * size_t((pieces + c - 1) / c + 4);
        if (cost < best_cost) {
            best_cost = cost;
            best = c;
        }
    }
    return best;
}
int pieces_of(int64_t n_vocab) {  // up to 3 elements lie before the first
    return int((n_vocab + 3 + kPiece - 1) / kPiece);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

size_t select_workspace_bytes(int64_t n_groups, int n_beams, int64_t n_vocab, int n_out) {
    const size_t recs = size_t(n_groups) * n_beams * pieces_of(n_vocab);  // the most chunks
    return align256(recs * sizeof(float2)) + align256(recs * n_out * sizeof(uint64_t));
}

cudaError_t select_run(const SelectArgs &a, void *ws, cudaStream_t s) {
    const size_t rows = size_t(a.n_groups) * a.n_beams;
    const int pieces = pieces_of(a.n_vocab);
    Work w;
    w.chunks = chunks_of(rows, pieces);
    w.steps = (pieces + w.chunks - 1) / w.chunks;
    w.sums = static_cast<float2 *>(ws);
    w.keys = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) +
                                          align256(rows * w.chunks * sizeof(float2)));
    const dim3 grid(unsigned(w.chunks), unsigned(rows));
    select_chunk_kernel<<<grid, kThreads1, 0, s>>>(a, w);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // The second pass starts while the first drains, and waits for it.
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(unsigned(a.n_groups));
    cfg.blockDim = dim3(kThreads2);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_group_kernel, a, w);
}

}  // namespace q2
