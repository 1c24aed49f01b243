// q2_0_beam_select: the n best continuations of each group of beams over the
// vocabulary, by running score + log-softmax of the logits.
//
// A beam's order by score is its order by logit, so one pass over the logits
// finds both what the log-softmax needs (running maximum and sum of
// exponentials) and the only candidates that can be selected: each beam's n
// best. Pass 1 does so per chunk of a row, pass 2 joins a group's chunks. The
// logits are read once from memory: 4 bytes, one exponential and a comparison
// each. Nothing depends on the order in which blocks run.
//
// Measured on one GB300 (device time; 151936 logits a row, 6.7 TB/s copy): 4 rows
// 8.3 us, 64 rows 19, 256 rows 39 (156 MB: 23 at the copy rate), 800 rows 89
// (5.4 TB/s). At 256 rows, profiled with cold caches, pass 1 takes 36 us (memory
// 51 % busy) and pass 2 9.8. What is over the copy rate is put down to the rankings of
// each chunk's first and last piece, in which a block does not stream, and to pass 2;
// their shares were not measured apart.
#include <float.h>

#include <algorithm>
#include <mutex>

#include "q2_0_device.cuh"
#include "q2_0_internal.h"

namespace q2 {

namespace {

constexpr int kThreads1 = 256;
constexpr int kPiece = 16 * kThreads1;         // logits of a piece
constexpr int kBlocks1 = 3;                    // blocks per SM
constexpr int kStages = 3;                     // pieces in shared memory
constexpr int kSmem1 = kStages * kPiece * 4;
constexpr int kThreads2 = 512;
constexpr int kCap1 = 512;                     // survivors held in shared memory
constexpr int kCap2 = 1024;
constexpr int kSms = 152;
constexpr int kMaxLists = 2432;                // chunks of a call that cuts rows at all
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
    int chunks, steps;  // of a row, pieces of a chunk
};

// A value that at least n (1..32) of the block's values reach, cheaply: the smallest of the
// maxima of 1, 2, 4 .. 32 >= n groups, a thread's group being its lane modulo their
// number. v is a thread's maximum, s_t holds a float per thread. Called by all threads.
template <int kWarps>
__device__ __forceinline__ float reached_by(float v, int n, float *s_t) {
    const int groups = n <= 1 ? 1 : 1 << (32 - __clz(n - 1));
    const int lane = threadIdx.x & 31;
    __syncthreads();
    s_t[threadIdx.x] = v;
    __syncthreads();
    float r = s_t[lane];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) r = fmaxf(r, s_t[32 * i + lane]);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, r, o);
        r = o >= groups ? fmaxf(r, w) : fminf(r, w);
    }
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

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

// A row in 16-byte blocks: block b holds elements 4 b - off .. + 3.
struct Row {
    const float *p;
    int off, V;
    __device__ __forceinline__ bool inside(int piece) const {  // all of its blocks lie in the row
        return (piece > 0 || off == 0) && (piece + 1) * kPiece - off <= V;
    }
    // element i of a thread's 16 of a piece
    __device__ __forceinline__ int element(int piece, int i) const {
        return piece * kPiece + 4 * (int(threadIdx.x) + (i / 4) * kThreads1) - off + i % 4;
    }
    __device__ __forceinline__ void load(int piece, float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int e = element(piece, i);
            if (e >= 0 && e + 4 <= V) {
                *reinterpret_cast<float4 *>(x + i) = __ldcs(reinterpret_cast<const float4 *>(p + e));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i + j] = e + j >= 0 && e + j < V ? p[e + j] : kNegInf;
            }
        }
    }
};

// The n_out best values so far, in order, in key[0, kept); what is appended lies behind.
struct Best {
    uint64_t key[kCap1];
    uint64_t top[8];
    float t[kThreads1];
    int n, kept;
    float lo;  // what a value has to reach to enter
};

__device__ __forceinline__ void append(Best &b, const Row &row, int piece, const float (&x)[16],
                                       const float (&part)[4], float from) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
        if (part[g] >= from) {
#pragma unroll
            for (int i = 4 * g; i < 4 * g + 4; ++i)
                if (x[i] >= from) {
                    const int at = atomicAdd(&b.n, 1);
                    if (at < kCap1)
                        b.key[at] = cand_key(fminf(x[i], FLT_MAX) + 0.0f, uint32_t(row.element(piece, i)));
                }
        }
}
// The maxima of a thread's four float4 (NaN is passed over).
__device__ __forceinline__ float maxima(const float (&x)[16], float (&part)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        part[i] = max3(max3(x[4 * i], x[4 * i + 1], x[4 * i + 2]), x[4 * i + 3], kNegInf);
    return max3(fmaxf(part[0], part[1]), part[2], part[3]);
}

// After the list was written. All threads.
__device__ __forceinline__ void listed(Best &b, int n, int n_out) {
    __syncthreads();
    if (threadIdx.x == 0) {
        b.n = b.kept = n;
        if (n == n_out) b.lo = unordered(uint32_t(b.key[n - 1] >> 32) + 1u);
    }
    __syncthreads();
}

// key[0, n) into the list, n <= kCap1, by counting. All threads, after a barrier.
__device__ __noinline__ void rank_list(Best &b, int n_out) {
    const int tid = threadIdx.x;
    constexpr int kPer = kCap1 / kThreads1;
    int n = b.n;
    uint64_t k[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) k[j] = tid + j * kThreads1 < n ? b.key[tid + j * kThreads1] : 0;
    if (n > 64) {  // cut them first, as a piece is
        float most = kNegInf;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (k[j]) most = fmaxf(most, unordered(uint32_t(k[j] >> 32)));
        const float t = reached_by<kThreads1 / 32>(most, n_out, b.t);
        if (tid == 0) b.n = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (k[j] && unordered(uint32_t(k[j] >> 32)) >= t) b.key[atomicAdd(&b.n, 1)] = k[j];
        __syncthreads();
        n = b.n;
#pragma unroll
        for (int j = 0; j < kPer; ++j) k[j] = tid + j * kThreads1 < n ? b.key[tid + j * kThreads1] : 0;
    }
    int at[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        at[j] = n_out;
        if (k[j]) {
            at[j] = 0;
#pragma unroll 8
            for (int i = 0; i < n; ++i) at[j] += b.key[i] > k[j];
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (at[j] < n_out) b.key[at[j]] = k[j];
    listed(b, min(n, n_out), n_out);
}

// Pieces [from, to] into the list one by one, each cut by a value that n_out of its
// values reach; `stage` holds piece `to`, the others are read again. All threads, after
// a barrier; the list is whole and what lies behind it is forgotten.
__device__ __noinline__ void settle(Best &b, const Row row, int n_out, int from, int to,
                                    const float4 *stage) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) b.n = b.kept;
    for (int q = from; q <= to; ++q) {
        float x[16], part[4];
        if (q < to) {
            row.load(q, x);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<float4 *>(x + 4 * i) = stage[tid + i * kThreads1];
        }
        const float most = maxima(x, part);
        const float lo = b.lo;
        const float t = fmaxf(reached_by<kThreads1 / 32>(most, n_out, b.t), lo);
        append(b, row, q, x, part, t);
        __syncthreads();
        if (b.n <= kCap1) {
            rank_list(b, n_out);
            continue;
        }
        // ties: the list and the piece, n_out times for the best one after the last
        uint64_t last = ~0ull, mine = tid < b.kept ? b.key[tid] : 0, put = 0;
#pragma unroll 1
        for (int n = 0; n < n_out; ++n) {
            uint64_t best = mine < last ? mine : 0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (x[i] >= lo) {
                    const uint64_t k =
                        cand_key(fminf(x[i], FLT_MAX) + 0.0f, uint32_t(row.element(q, i)));
                    if (k < last && k > best) best = k;
                }
            for (int o = 16; o; o >>= 1) {
                const uint64_t v = __shfl_xor_sync(0xffffffffu, best, o);
                best = v > best ? v : best;
            }
            __syncthreads();
            if (lane == 0) b.top[warp] = best;
            __syncthreads();
            for (int i = 0; i < 8; ++i) best = b.top[i] > best ? b.top[i] : best;
            if (tid == n) put = best;
            last = best;
        }
        if (tid < n_out) b.key[tid] = put;
        listed(b, n_out, n_out);  // there were more than kCap1
    }
}

// Pass 1: one block per (chunk, row). A chunk is up to `steps` pieces of 4096 logits,
// 16 to a thread, copied to shared memory kStages - 1 pieces ahead; each thread reads
// only what it copied, so that no barrier is needed.
// Sum: a thread keeps that of its own elements, of 2^(x log2(e) - R) with R a whole
// number, so that the exponent is one fused multiply-add, rounded near 0, and
// R ln 2 can be added to the logarithm without loss later. A chunk with a maximum
// beyond kHuge or a NaN (seen in the sum; counts as -inf) is summed again with care.
// Best n: the list of the n best so far lies in order (Best). A value that is not
// above the list's last cannot enter it (tokens come in order, and the lower one
// wins a tie), so from the second piece on few do. They are appended without a
// barrier, and ranked into the list, by counting, after 8 pieces, 64 and so on.
// The first piece is cut by a value that n of its values reach (reached_by). Where more
// come than it has room for, the pieces since the last ranking are gone through again one
// by one with that cut, and where ties defeat it, n rounds of a block maximum serve.
__global__ void __launch_bounds__(kThreads1, kBlocks1)
    select_chunk_kernel(const SelectArgs a, const Work w) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t row_i = blockIdx.y;
    const int chunk = blockIdx.x;
    if (a.done && a.done[row_i]) return;
    __shared__ float s_m[8], s_s[8], s_r[8];
    __shared__ Best best;
    extern __shared__ float4 s_x[];  // [kStages][4][kThreads1]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        best.n = best.kept = 0;
        best.lo = -FLT_MAX;
    }
    Row row;
    row.p = a.logits + row_i * a.stride;
    row.off = int((reinterpret_cast<uintptr_t>(row.p) >> 2) & 3);
    row.V = int(a.n_vocab);
    const int n_out = a.n_out;
    const int p0 = chunk * w.steps, p1 = min(p0 + w.steps, (row.V + row.off + kPiece - 1) / kPiece);
    // pieces before i1 are whole, but maybe the row's first
    const int i1 = p1 > p0 && row.inside(p1 - 1) ? p1 : p1 - 1;
    const float *g = row.p + row.element(p0, 0);
    int in = 0, at = 0, next = p0;  // stages, piece to fetch
    auto fetch = [&]() {
        float4 *d = s_x + in * (4 * kThreads1) + tid;
        if (next < i1 && (next > 0 || row.off == 0)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 smem_addr(d + i * kThreads1)),
                             "l"(g + 4 * i * kThreads1)
                             : "memory");
        } else if (next < p1) {
            float v[16];
            row.load(next, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i * kThreads1] = *reinterpret_cast<float4 *>(v + 4 * i);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        g += kPiece;
        ++next;
        in = in == kStages - 1 ? 0 : in + 1;
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) fetch();
    float most = kNegInf, R = -kHuge, sum = 0.0f, lo = -FLT_MAX;
    bool whole = false;  // the list has n_out values
    int ranked = p0, due = p0 + 8;  // pieces before `ranked` are in the list; the next ranking's place
#pragma unroll 1
    for (int piece = p0; piece < p1; ++piece) {
        fetch();
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        const float4 *stage = s_x + at * (4 * kThreads1);
        at = at == kStages - 1 ? 0 : at + 1;
        float x[16], part[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float4 *>(x + 4 * i) = stage[tid + i * kThreads1];
        const float tm = maxima(x, part);
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
        if (whole) {
            if (tm >= lo) append(best, row, piece, x, part, lo);
            if (piece + 1 < due && piece + 1 < p1) continue;
            due = p0 + 8 * (piece + 1 - p0);
        }
        __syncthreads();
        if (whole && best.n <= kCap1) {
            rank_list(best, n_out);
        } else {
            __syncthreads();
            settle(best, row, n_out, ranked, piece, stage);
        }
        ranked = piece + 1;
        whole = best.kept == n_out;
        lo = best.lo;
    }
    const float wm = warp_max(most);
    const float wr = warp_max(R);
    sum = warp_sum(sum * ex2(R - wr));
    if (lane == 0) {
        s_m[warp] = wm;
        s_r[warp] = wr;
        s_s[warp] = sum;
    }
    __syncthreads();
    const int64_t rec = row_i * w.chunks + chunk;
    if (tid < n_out) w.keys[rec * n_out + tid] = tid < best.kept ? best.key[tid] : 0;
    float m = s_m[0];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m = fmaxf(m, s_m[i]);
        nan |= s_s[i] != s_s[i];
    }
    if (!nan && (m == kNegInf || fabsf(m) < kHuge)) {
        if (warp == 7) {
            const float Rw = lane < 8 ? s_r[lane] : -kHuge;
            const float top = warp_max(Rw);
            const float s = warp_sum(Rw > -kHuge ? s_s[lane & 7] * ex2(Rw - top) : 0.0f);
            if (lane == 0) w.sums[rec] = make_float2(top > -kHuge ? top : kNegInf, s);
        }
        return;
    }
    m = fminf(m, FLT_MAX);
    const bool plain = fabsf(m) < kHuge;  // only NaN brought it here: the first kind
    const float c = plain ? ceilf(m * kLog2e) : m;
    sum = 0.0f;
    for (int piece = p0; piece < p1; ++piece) {
        float x[16];
        row.load(piece, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float v = fminf(fmaxf(x[i], kNegInf), FLT_MAX);
            sum += plain ? ex2(fmaf(v, kLog2e, -c)) : m == kNegInf ? 0.0f : ex2((v - c) * kLog2e);
        }
    }
    sum = warp_sum(sum);
    __syncthreads();
    if (lane == 0) s_s[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < 8; ++i) sum += s_s[i];
        w.sums[rec] = make_float2(c, plain || m == kNegInf ? sum : -sum);
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
// A chunk's candidates are in order, so the chunks' first ones give a threshold, and only chunks whose first reaches it are looked
// at further. The survivors are thinned and ranked as in pass 1. The loads of a
// step are all in flight together: what this kernel costs is their latency.
__global__ void __launch_bounds__(kThreads2) select_group_kernel(const SelectArgs a, const Work w) {
    __shared__ float s_base[64], s_lse[64];
    __shared__ uint8_t s_done[64];
    __shared__ uint32_t s_head[kMaxLists];  // the chunks' first scores
    __shared__ float s_t[kThreads2];
    __shared__ Cand s_c[kCap2];
    __shared__ int s_n;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row0 = int64_t(blockIdx.x) * a.n_beams;
    const int W = a.n_beams, C = w.chunks, n_out = a.n_out;
    // the call's inputs: complete before the first pass began
    if (tid < W) {
        s_base[tid] = a.score[row0 + tid];
        s_done[tid] = a.done && a.done[row0 + tid];
    }
    if (tid == 0) s_n = 0;
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lists = W * C, per_beam = C * n_out, total = W * per_beam;
    const unsigned long long *keys =
        reinterpret_cast<const unsigned long long *>(w.keys) + row0 * per_beam;
    const uint64_t head = tid < lists && !s_done[tid / C] ? __ldcg(keys + tid * n_out) : 0;
    for (int b = warp; b < W; b += kThreads2 / 32) {
        const float lse = s_done[b] ? 0.0f : row_lse(w.sums + (row0 + b) * C, C);
        if (lane == 0) s_lse[b] = lse;
    }
    __syncthreads();
    auto of = [&](int b, uint64_t key) {  // a chunk's candidate, or none
        Cand c{0, uint32_t(b), key};
        if (key) {
            const float s = s_base[b] + (unordered(uint32_t(key >> 32)) - s_lse[b]);
            if (s > kNegInf) c.score = ordered(s + 0.0f);
        }
        return c;
    };
    // candidate i < total of the chunks, i - total the beam of a finished one
    auto get = [&](int i) {
        if (i < total) {
            const int b = i / per_beam;
            return of(b, s_done[b] ? 0 : __ldcg(keys + i));
        }
        Cand c{0, uint32_t(i - total), 1};
        if (s_done[c.beam] && s_base[c.beam] > kNegInf) c.score = ordered(s_base[c.beam] + 0.0f);
        return c;
    };
    auto threshold = [&](uint32_t best) {  // called by all threads; no candidate: below every score
        const float v = reached_by<kThreads2 / 32>(best ? unordered(best) : kNegInf, n_out, s_t);
        return v > kNegInf ? ordered(v) : 1u;
    };
    uint32_t best = 0;
    for (int i = tid; i < lists; i += kThreads2) {
        const Cand c = i == tid ? of(i / C, head) : get(i * n_out);
        s_head[i] = c.score;
        best = max(best, c.score);
    }
    if (tid < W) best = max(best, get(total + tid).score);
    const uint32_t least = threshold(best);
    auto keep = [&](const Cand &c) {
        if (c.score < least) return;
        const int at = atomicAdd(&s_n, 1);
        if (at < kCap2) s_c[at] = c;
    };
    for (int i0 = tid; i0 < total; i0 += 4 * kThreads2) {
        uint64_t k[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * kThreads2;
            k[j] = i < total && s_head[i / n_out] >= least ? __ldcg(keys + i) : 0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (k[j]) keep(of((i0 + j * kThreads2) / per_beam, k[j]));
    }
    if (tid < W) keep(get(total + tid));
    __syncthreads();
    int n = s_n;
    float *so = a.score_out + int64_t(blockIdx.x) * n_out;
    int32_t *po = a.parent + int64_t(blockIdx.x) * n_out;
    int32_t *to = a.token + int64_t(blockIdx.x) * n_out;
    auto put = [&](int r, const Cand &c) {
        so[r] = c.score ? unordered(c.score) : kNegInf;
        po[r] = c.score ? int32_t(c.beam) : 0;
        to[r] = !c.score         ? -1
                : s_done[c.beam] ? a.done_token
                                 : int32_t(0xFFFFFFFFu - uint32_t(c.key & 0xFFFFFFFFu));
    };
    if (n <= kCap2) {
        if (n > 64) {
            const Cand none{0, 0, 0};
            Cand c[kCap2 / kThreads2];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < kCap2 / kThreads2; ++j) {
                const int i = tid + j * kThreads2;
                c[j] = i < n ? s_c[i] : none;
                top = max(top, c[j].score);
            }
            const uint32_t more = threshold(top);
            if (tid == 0) s_n = 0;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kCap2 / kThreads2; ++j)
                if (c[j].score >= more) s_c[atomicAdd(&s_n, 1)] = c[j];
            __syncthreads();
            n = s_n;
        }
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
            const Cand o = get(i);
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

int pieces_of(int64_t n_vocab) {  // up to 3 elements lie before the first
    return int((n_vocab + 3 + kPiece - 1) / kPiece);
}

std::mutex g_mu;
bool g_attr[64];

cudaError_t ensure_attr() {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(g_mu);
    if (dev < 64 && g_attr[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(select_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem1);
    if (e == cudaSuccess && dev < 64) g_attr[dev] = true;
    return e;
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Chunks of a row: the number with the least time, in units of a piece's share of the
// memory rate of an SM (0.37 us): a block's own time is about 16 units and 2 a piece, in
// waves of kBlocks1 per SM, and the busiest SM's pieces have to be read. Measured at
// 151936 logits, 8 chosen, the rule's choice first: 4 rows in 38 chunks 8.5 us, in 19 9.0, in 8
// 11.1; 64 rows in 7 19.4, in 4 20.5, in 8 22.9, in 1 27.6; 256 rows in 3 40.4, in 1 38.4, in 2 44.1, in 7
// 47.7 (16 chosen: in 3 45.5, in 1 41.0). So at 256 rows it misses the best by 5 to 11 %; how many
// are chosen is not in it.
int chunks_of(size_t rows, int pieces) {
    int best = 1;
    size_t best_cost = ~size_t(0);
    for (int c = 1; c <= pieces && (c == 1 || rows * c <= kMaxLists); ++c) {
        const size_t n = rows * c, per = size_t((pieces + c - 1) / c);
        const size_t waves = (n + kBlocks1 * kSms - 1) / (kBlocks1 * kSms);
        const size_t cost = waves * (16 + 2 * per) + (n + kSms - 1) / kSms * per;
        if (cost < best_cost) {
            best_cost = cost;
            best = c;
        }
    }
    return best;
}

}  // namespace

size_t select_workspace_bytes(int64_t n_groups, int n_beams, int64_t n_vocab, int n_out) {
    const size_t rows = size_t(n_groups) * n_beams;
    const size_t recs = rows * chunks_of(rows, pieces_of(n_vocab));
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
    cudaError_t e = ensure_attr();
    if (e != cudaSuccess) return e;
    select_chunk_kernel<<<dim3(unsigned(w.chunks), unsigned(rows)), kThreads1, kSmem1, s>>>(a, w);
    e = cudaGetLastError();
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
