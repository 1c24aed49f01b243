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
constexpr int kVec = 4;                        // float4 per thread
constexpr int kChunkVec = kThreads1 * kVec;    // float4 per chunk
constexpr int kThreads2 = 512;
constexpr int kCap1 = 512;                     // survivors held in shared memory
constexpr int kCap2 = 1024;
constexpr float kNegInf = -INFINITY;

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

// exp(d) for d <= 0, exp(-inf) = 0
__device__ __forceinline__ float exp_neg(float d) { return exp2f(d * 1.44269504f); }

// What a logit counts as: NaN as -inf, +inf as the largest finite value, -0 as 0.
__device__ __forceinline__ float clean(float x) {
    return x != x ? kNegInf : fminf(x, FLT_MAX) + 0.0f;
}

struct Work {
    float2 *ms;      // [rows][chunks] maximum and sum of exponentials
    uint64_t *keys;  // [rows][chunks][n_out], best first, 0 where there are no more
    int chunks;
};

// Pass 1: one block per (chunk, row). The threshold that leaves few candidates:
// in each warp the n-th largest of the lanes' maxima, the largest of those over
// the warps; at least n values of the chunk reach it. The survivors are ranked by
// counting. Where ties make too many of them, n rounds of a block maximum.
__global__ void __launch_bounds__(kThreads1) select_chunk_kernel(const SelectArgs a, const Work w) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t row = blockIdx.y;
    const int chunk = blockIdx.x;
    if (a.done && a.done[row]) return;
    __shared__ float s_m[8], s_s[8], s_t[8];
    __shared__ uint64_t s_key[kCap1];
    __shared__ int s_n;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) s_n = 0;
    // The row in 16-byte blocks: block b holds elements 4 b - off .. + 3.
    const float *p = a.logits + row * a.stride;
    const int off = int((reinterpret_cast<uintptr_t>(p) >> 2) & 3);
    const float4 *p4 = reinterpret_cast<const float4 *>(p - off);
    const int V = int(a.n_vocab);
    float x[4 * kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int b = chunk * kChunkVec + i * kThreads1 + tid;
        const int e = 4 * b - off;
        if (e >= 0 && e + 4 <= V) {
            const float4 f = __ldcs(p4 + b);
            x[4 * i] = clean(f.x);
            x[4 * i + 1] = clean(f.y);
            x[4 * i + 2] = clean(f.z);
            x[4 * i + 3] = clean(f.w);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[4 * i + j] = e + j >= 0 && e + j < V ? clean(p[e + j]) : kNegInf;
        }
    }
    float tm = x[0];
#pragma unroll
    for (int i = 1; i < 4 * kVec; ++i) tm = fmaxf(tm, x[i]);
    const float t = warp_nth(tm, a.n_out);
    const float wm = warp_max(tm);
    const float ref = wm == kNegInf ? 0.0f : wm;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4 * kVec; ++i) sum += exp_neg(x[i] - ref);
    sum = warp_sum(sum);
    if (lane == 0) {
        s_m[warp] = wm;
        s_s[warp] = sum;
        s_t[warp] = t;
    }
    __syncthreads();
    float thr = s_t[0], m = s_m[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        thr = fmaxf(thr, s_t[i]);
        m = fmaxf(m, s_m[i]);
    }
    thr = fmaxf(thr, -FLT_MAX);
    if (tm >= thr) {
#pragma unroll
        for (int i = 0; i < 4 * kVec; ++i)
            if (x[i] >= thr) {
                const int at = atomicAdd(&s_n, 1);
                const int e = 4 * (chunk * kChunkVec + (i / 4) * kThreads1 + tid) - off + i % 4;
                if (at < kCap1) s_key[at] = cand_key(x[i], uint32_t(e));
            }
    }
    __syncthreads();
    const int64_t rec = row * w.chunks + chunk;
    if (tid == 0) {
        float s = 0.0f;
        for (int i = 0; i < 8; ++i)
            if (s_m[i] > kNegInf) s += s_s[i] * exp_neg(s_m[i] - m);
        w.ms[rec] = make_float2(m, s);
    }
    uint64_t *out = w.keys + rec * a.n_out;
    const int n = s_n;
    if (n <= kCap1) {
        for (int i = tid; i < n; i += kThreads1) {
            const uint64_t k = s_key[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += s_key[j] > k;
            if (rank < a.n_out) out[rank] = k;
        }
        for (int i = n + tid; i < a.n_out; i += kThreads1) out[i] = 0;
        return;
    }
    uint64_t last = ~0ull;
    for (int r = 0; r < a.n_out; ++r) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < 4 * kVec; ++i)
            if (x[i] >= thr) {
                const int e = 4 * (chunk * kChunkVec + (i / 4) * kThreads1 + tid) - off + i % 4;
                const uint64_t k = cand_key(x[i], uint32_t(e));
                if (k < last && k > best) best = k;
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

// Pass 2: one block per group. Every row's chunks are joined to its log of the
// sum, then the chunks' candidates are thinned and ranked as in pass 1.
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
        const float2 *ms = w.ms + (row0 + b) * C;
        float m = kNegInf, s = 0.0f;
        if (!done) {
            for (int i = lane; i < C; i += 32) m = fmaxf(m, ms[i].x);
            m = warp_max(m);
            for (int i = lane; i < C; i += 32)
                if (ms[i].x > kNegInf) s += ms[i].y * exp_neg(ms[i].x - m);
            s = warp_sum(s);
        }
        if (lane == 0) {
            s_lse[b] = m + logf(s);
            s_base[b] = a.score[row0 + b];
        }
    }
    __syncthreads();
    const int per_beam = C * n_out;
    const int total = W * per_beam;
    const uint64_t *keys = w.keys + row0 * per_beam;
    // candidate i < total of the chunks, i - total the beam of a finished one
    auto get = [&](int i, Cand &c) {
        c.score = 0;
        float s;
        if (i < total) {
            const int b = i / per_beam;
            if (a.done && a.done[row0 + b]) return;
            c.key = __ldcg(reinterpret_cast<const unsigned long long *>(keys) + i);
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
    for (int i = tid; i < total + W; i += kThreads2) {
        Cand c;
        get(i, c);
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
    for (int i = tid; i < total + W; i += kThreads2) {
        Cand c;
        get(i, c);
        if (c.score >= least) {
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

int chunks_of(int64_t n_vocab) {
    return int(((n_vocab + 3 + 3) / 4 + kChunkVec - 1) / kChunkVec);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

size_t select_workspace_bytes(int64_t n_groups, int n_beams, int64_t n_vocab, int n_out) {
    const size_t recs = size_t(n_groups) * n_beams * chunks_of(n_vocab);
    return align256(recs * sizeof(float2)) + align256(recs * n_out * sizeof(uint64_t));
}

cudaError_t select_run(const SelectArgs &a, void *ws, cudaStream_t s) {
    Work w;
    w.chunks = chunks_of(a.n_vocab);
    const size_t rows = size_t(a.n_groups) * a.n_beams;
    w.ms = static_cast<float2 *>(ws);
    w.keys = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) +
                                          align256(rows * w.chunks * sizeof(float2)));
    select_chunk_kernel<<<dim3(unsigned(w.chunks), unsigned(rows)), kThreads1, 0, s>>>(a, w);
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
