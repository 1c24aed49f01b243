// Verification of drafted tokens: which drafts of a sequence stand, and the token drawn
// behind them from what the target model's probabilities leave.
//
// One cluster of blocks per sequence. Only one row of probabilities is drawn from, so
// every block first finds out which: a draft costs two single reads. The row is cut
// into as many runs as the cluster has warps, and each warp sums its run; the sums go to all
// blocks' shared memory. The block that holds the run in which the running sum passes
// r * total cuts that run among its warps again, and the warp with the place finds it. The row is
// read once, a run of it three times, and nothing depends on the order in which blocks come.
//
// Sums are pairs of floats, the sum and what it lost (two-sum: 6 additions a value, two values at once by
// the packed f32x2 forms): one addition in f64 would take 64 times an f32 one's share of the SM. A pair's second
// part, up to j 2^-24 of the sum after j additions, is rounded to 2^-24 of itself at each: (n^2 + n) / 2 units of 2^-48 of the
// sum over n additions at worst. So n is 16 before a pair is added to that of all such windows, which is settled (136 units,
// 33 for the addition and 3 for each window before it; with n = 64 it would be 2080, more than 2^-37). A warp's sum takes
// 38 units, the running sums over the runs, the parts of one and its tokens 511 and 3 for each 8192 tokens: together with
// the windows' (half of a run's error goes into the total as well) below 2^-38 + n_vocab 2^-58 of the total where a running
// sum is compared with r * total.
//
// Measured in a CUDA graph, inputs beyond L2, 151936 tokens: 4 drafts of 1 sequence 8.5 us (1.2 MB: the bytes take 0.2, a
// sequence of dependent reads, barriers and prefix sums the rest: 1000 tokens take 5.8), up to 5 of 64 16.1 (58 MB at
// 3.6 TB/s; the copy rate would give 8.6); without the drafts' probabilities 7.8 and 14.7. Inputs in L2: 6.6 and 12.8.
// Windows of 64 additions instead of 16, which lose more than 2^-38, take 0.6 % less; merged and settled pair by pair 1 % more.
// Values read singly and sums in f64 took 19.0 and 38.7.
#include <algorithm>
#include <mutex>

#include "q2_0_cluster.cuh"
#include "q2_0_internal.h"

namespace q2 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kRuns = kMaxCluster * kWarps;
constexpr int kFlush = 2;   // times 16 values that two pairs take before they are added to another
constexpr int kResident = 4;      // blocks of an SM
constexpr int kMinBlock = 2048;  // values of a block, and where SMs have several
constexpr int kMinShare = 8000;
constexpr int kHeld = 4;    // values a lane holds in the end

struct Pair {
    float h, l;
};
__device__ __forceinline__ Pair settled(float s, float e) {  // |s| >= |e|
    const float h = __fadd_rn(s, e);
    return {h, __fsub_rn(e, __fsub_rn(h, s))};
}
__device__ __forceinline__ void add(Pair &p, float w) {  // (not settled)
    const float s = __fadd_rn(p.h, w), b = __fsub_rn(s, p.h);
    p.l = __fadd_rn(p.l, __fadd_rn(__fsub_rn(p.h, __fsub_rn(s, b)), __fsub_rn(w, b)));
    p.h = s;
}
// (Not settled either: the second part may be some units of the first, which costs it as many roundings, and the
// next addition need not wait for it.)
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    const float l = __fadd_rn(a.l, b.l);
    a.l = 0.0f;
    add(a, b.h);
    a.l = __fadd_rn(a.l, l);
    return a;
}
__device__ __forceinline__ Pair settled(Pair a) { return settled(a.h, a.l); }
// Of settled pairs.
__device__ __forceinline__ bool operator>(Pair a, Pair b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }
__device__ __forceinline__ Pair operator*(float r, Pair a) {
    const float h = __fmul_rn(r, a.h);
    return settled(h, __fmaf_rn(r, a.l, __fmaf_rn(r, a.h, -h)));
}
__device__ __forceinline__ Pair shuffle(Pair a, int lane) { return {__shfl_sync(~0u, a.h, lane), __shfl_sync(~0u, a.l, lane)}; }
__device__ __forceinline__ Pair warp_sum(Pair a) {
#pragma unroll
    for (int o = 16; o; o >>= 1) a = a + Pair{__shfl_xor_sync(~0u, a.h, o), __shfl_xor_sync(~0u, a.l, o)};
    return a;
}
__device__ __forceinline__ Pair warp_scan(Pair a, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair b = a + Pair{__shfl_up_sync(~0u, a.h, o), __shfl_up_sync(~0u, a.l, o)};
        if (lane >= o) a = b;
    }
    return a;
}
__device__ __forceinline__ Pair before(Pair a, int lane) {  // the lane's before it, of an inclusive scan
    const Pair b = {__shfl_up_sync(~0u, a.h, 1), __shfl_up_sync(~0u, a.l, 1)};
    return lane ? b : Pair{0.0f, 0.0f};
}

// Two floats at once.
__device__ __forceinline__ uint64_t pack(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ float2 unpack(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
struct Pair2 {  // two pairs
    uint64_t h, l;
    __device__ __forceinline__ Pair sum() const {
        const float2 a = unpack(h), b = unpack(l);
        return Pair{a.x, b.x} + Pair{a.y, b.y};
    }
};
__device__ __forceinline__ void add(Pair2 &p, uint64_t w) {
    const uint64_t s = add2(p.h, w), b = sub2(s, p.h);
    p.l = add2(p.l, add2(sub2(p.h, sub2(s, b)), sub2(w, b)));
    p.h = s;
}
// A window's pairs go to those of all windows, which are settled again.
__device__ __forceinline__ void flush(Pair2 &all, Pair2 &p) {
    const uint64_t s = add2(all.h, p.h), b = sub2(s, all.h);
    const uint64_t l = add2(add2(sub2(all.h, sub2(s, b)), sub2(p.h, b)), add2(all.l, p.l));
    all.h = add2(s, l);
    all.l = sub2(l, sub2(all.h, s));
    p = {0, 0};
}

// What counts as a probability: not a negative one or NaN.
__device__ __forceinline__ float clean(float p) { return fmaxf(p, 0.0f); }

// What a token is drawn from: row p, less row q (null: nothing), without token `out` (-1: none).
struct Row {
    const float *p, *q;
    int out;
    __device__ __forceinline__ float weight(float pv, float qv, int v) const {
        const float w = clean(pv);
        if (q) return clean(w - clean(qv));
        return v == out ? 0.0f : w;
    }
    __device__ __forceinline__ float operator[](int v) const { return weight(p[v], q ? q[v] : 0.0f, v); }
};

// Sum of a warp's run [v0, v1). `wide`: p + v0 and q + v0 are 16-byte aligned (v1 may be anything). A lane has
// 16 values of each row on their way at a time.
template <bool kQ>
__device__ __forceinline__ Pair run_sum(const Row &row, int v0, int v1, bool wide, int lane) {
    int v = v0;
    auto take = [&](Pair2 &s, float4 p, float4 q, int out) {  // out: where row.out is among them
        p = make_float4(clean(p.x), clean(p.y), clean(p.z), clean(p.w));
        if (kQ) {
            const float2 x = unpack(sub2(pack(p.x, p.y), pack(clean(q.x), clean(q.y))));
            const float2 y = unpack(sub2(pack(p.z, p.w), pack(clean(q.z), clean(q.w))));
            p = make_float4(clean(x.x), clean(x.y), clean(y.x), clean(y.y));
        } else {
            p = make_float4(out == 0 ? 0.0f : p.x, out == 1 ? 0.0f : p.y, out == 2 ? 0.0f : p.z, out == 3 ? 0.0f : p.w);
        }
        add(s, pack(p.x, p.y));
        add(s, pack(p.z, p.w));
    };
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    Pair2 sum = {0, 0}, s = {0, 0};
    int taken = 0;
    if (wide) {
        const int whole = v0 + (v1 - v0) / 4 * 4;
        for (; v < whole; v += 512) {
            float4 p[4], q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = v + 128 * k + 4 * lane;
                p[k] = at < whole ? *reinterpret_cast<const float4 *>(row.p + at) : zero;
                if (kQ) q[k] = at < whole ? *reinterpret_cast<const float4 *>(row.q + at) : zero;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) take(s, p[k], kQ ? q[k] : zero, row.out - (v + 128 * k + 4 * lane));
            if (++taken % kFlush == 0) flush(sum, s);
        }
        v = whole;
    }
    for (; v < v1; v += 512) {
        float p[16], q[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int at = v + 32 * k + lane;
            p[k] = at < v1 ? row.p[at] : 0.0f;
            if (kQ) q[k] = at < v1 ? row.q[at] : 0.0f;
            if (!kQ && at == row.out) p[k] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 16; k += 4)
            take(s, make_float4(p[k], p[k + 1], p[k + 2], p[k + 3]), kQ ? make_float4(q[k], q[k + 1], q[k + 2], q[k + 3]) : zero, -1);
        if (++taken % kFlush == 0) flush(sum, s);
    }
    flush(sum, s);
    return settled(warp_sum(settled(sum.sum())));
}
__device__ __forceinline__ Pair run_sum(const Row &row, int v0, int v1, bool wide, int lane) {
    return row.q ? run_sum<true>(row, v0, v1, wide, lane) : run_sum<false>(row, v0, v1, wide, lane);
}

// Of n <= 32 kEach sums in shared memory, whose running sums start at `base`: the first that is not 0 and takes it
// beyond `limit`, or the last that is not 0; base becomes the running sum before it. -1 if all are 0. With kAll the
// limit is r times all of them.
template <int kEach, bool kAll = false>
__device__ int pick(const Pair *sums, int n, Pair &limit, Pair &base, int lane, float r = 0.0f) {
    Pair s[kEach], all = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int i = lane * kEach + k;
        s[k] = i < n ? sums[i] : Pair{0.0f, 0.0f};
        all = all + s[k];
    }
    all = warp_scan(all, lane);
    if constexpr (kAll) limit = r * settled(shuffle(all, 31));
    Pair c = base + before(all, lane), from_hit = c, from_last = c;
    int hit = -1, last = -1;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const Pair next = c + s[k];
        if (s[k].h > 0.0f) {
            last = lane * kEach + k;
            from_last = c;
            if (hit < 0 && settled(next) > limit) {
                hit = last;
                from_hit = c;
            }
        }
        c = next;
    }
    const unsigned hits = __ballot_sync(~0u, hit >= 0), some = __ballot_sync(~0u, last >= 0);
    if (!some) return -1;
    const int by = hits ? __ffs(hits) - 1 : 31 - __clz(some);
    base = settled(shuffle(hits ? from_hit : from_last, by));
    return __shfl_sync(~0u, hits ? hit : last, by);
}

struct VerifyArgs {
    const float *target, *draft;
    int64_t target_stride, draft_stride;
    const int32_t *tokens, *count;
    const float *rand;
    int n_draft, n_vocab;
    int32_t *accepted, *token;
    unsigned long long *err;
};

__global__ void __launch_bounds__(kThreads, kResident) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ Pair sums[kRuns];  // the runs'
    __shared__ Pair parts[kWarps];
    __shared__ int stand_s, run_s;
    __shared__ Pair base_s, limit_s;
    const int64_t b = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int runs = int(size) * kWarps;
    const int32_t *tok = a.tokens + b * a.n_draft;
    const float *u = a.rand + b * (a.n_draft + 1);
    // (shared memory of a block that has started alone may be written: waited for below)
    cluster_arrive();
    // ---- how many drafts stand (-1: a bad argument); each block finds out by itself
    const int n = a.count ? a.count[b] : a.n_draft;
    if (warp == 0) {
        bool bad = n < 0 || n > a.n_draft;
        int stand = n;
        for (int i0 = 0; !bad && i0 < n; i0 += 32) {
            const int i = i0 + lane;
            bool stands = true, in = true;
            if (i < n) {
                const int d = tok[i];
                in = d >= 0 && d < a.n_vocab;
                if (in) {
                    const float p = clean(a.target[(b * (a.n_draft + 1) + i) * a.target_stride + d]);
                    const float q = a.draft ? clean(a.draft[(b * a.n_draft + i) * a.draft_stride + d]) : 1.0f;
                    stands = __fmul_rn(u[i], q) < p;
                }
            }
            bad = __any_sync(~0u, !in);
            const unsigned no = __ballot_sync(~0u, !stands);
            if (no && stand == n) stand = i0 + __ffs(no) - 1;
        }
        if (lane == 0) stand_s = bad ? -1 : stand;
    }
    __syncthreads();
    const int stand = stand_s;
    if (stand < 0) {  // (all blocks of the cluster come to the same)
        if (rank == 0 && threadIdx.x == 0) record_error(a.err, Q2_0_DEVERR_BAD_ID, b);
        __syncwarp();  // (the cluster's barrier takes a warp's lanes together)
        cluster_wait();
        return;
    }
    const float *p = a.target + (b * (a.n_draft + 1) + stand) * a.target_stride;
    Row row{p, nullptr, -1};
    if (stand < n && a.draft) row.q = a.draft + (b * a.n_draft + stand) * a.draft_stride;
    if (stand < n && !a.draft) row.out = tok[stand];
    // runs begin where both rows are aligned, if they are alike
    const int odd = int(reinterpret_cast<uintptr_t>(p) >> 2) & 3;
    bool wide = !row.q || (int(reinterpret_cast<uintptr_t>(row.q) >> 2) & 3) == odd;
    const int len = ((a.n_vocab + 3 + runs - 1) / runs + 3) / 4 * 4;
    auto begin = [&](int i) { return int(max(int64_t(0), min(int64_t(i) * len - odd, int64_t(a.n_vocab)))); };
    Pair limit, base = {0.0f, 0.0f};
    for (bool first = true;; first = false) {
        const int i = int(rank) * kWarps + warp;
        // (the first run of a row that is not aligned begins before it)
        const Pair sum = run_sum(row, begin(i), begin(i + 1), wide && (i || !odd), lane);
        if (first) cluster_wait();
        if (lane < int(size)) store_cluster(&sums[i], uint32_t(lane), sum);
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (warp == 0) {
            const int at = pick<kRuns / 32, true>(sums, runs, limit, base, lane, u[a.n_draft]);
            if (lane == 0) {
                run_s = at;
                base_s = base;
                limit_s = limit;
            }
        }
        __syncthreads();
        if (run_s >= 0 || !first || (!row.q && row.out < 0)) break;
        // nothing is left: drawn from p, after all have seen so
        cluster_arrive();
        cluster_wait();
        row = Row{p, nullptr, -1};
        wide = true;
    }
    const int run = run_s;
    if (rank == 0) {
        int32_t *out = a.token + b * (a.n_draft + 1);
        for (int i = threadIdx.x; i <= a.n_draft; i += kThreads)
            if (i != stand || run < 0) out[i] = i < stand ? tok[i] : -1;
        if (threadIdx.x == 0) a.accepted[b] = stand;
    }
    if (run < 0 || run / kWarps != int(rank)) return;
    // ---- the run is this block's: cut again, and the warp with the place finds it
    base = base_s;
    limit = limit_s;
    const int v0 = begin(run), v1 = begin(run + 1), each = (v1 - v0 + kWarps - 1) / kWarps;
    const Pair part = run_sum(row, min(v0 + warp * each, v1), min(v0 + (warp + 1) * each, v1), false, lane);
    if (lane == 0) parts[warp] = part;
    __syncthreads();
    if (pick<1>(parts, kWarps, limit, base, lane) != warp) return;
    const int w1 = min(v0 + (warp + 1) * each, v1);
    int found = -1;
    for (int w0 = v0 + warp * each; w0 < w1; w0 += 32 * kHeld) {
        float w[kHeld];
        Pair s = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int v = w0 + lane * kHeld + k;
            w[k] = v < w1 ? row[v] : 0.0f;
            s = s + Pair{w[k], 0.0f};
        }
        s = warp_scan(s, lane);
        Pair c = base + before(s, lane);
        base = settled(base + shuffle(s, 31));
        int hit = -1, last = -1;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            c = c + Pair{w[k], 0.0f};
            if (w[k] > 0.0f) {
                last = k;
                if (hit < 0 && settled(c) > limit) hit = k;
            }
        }
        const unsigned hits = __ballot_sync(~0u, hit >= 0), some = __ballot_sync(~0u, last >= 0);
        if (some) {
            const int by = hits ? __ffs(hits) - 1 : 31 - __clz(some);
            found = w0 + by * kHeld + __shfl_sync(~0u, hits ? hit : last, by);
        }
        if (hits) break;
    }
    if (lane == 0) a.token[b * (a.n_draft + 1) + stand] = found;
}

std::mutex g_mu;
int g_cluster[64];  // blocks that a cluster may have, of a device

// Clusters of more than 8 blocks are asked for, and had where the GPU has room for one.
cudaError_t max_cluster(int *blocks) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(g_mu);
    if (dev < 64 && g_cluster[dev]) {
        *blocks = g_cluster[dev];
        return cudaSuccess;
    }
    e = cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cluster_fits(verify_kernel, kThreads, 0, kMaxCluster, blocks);
    if (e == cudaSuccess && dev < 64) g_cluster[dev] = *blocks;
    return e;
}

}  // namespace

cudaError_t launch_verify(const float *target, int64_t target_stride, const float *draft, int64_t draft_stride,
                          const int32_t *tokens, const int32_t *count, const float *rand, int64_t n_seq, int n_draft,
                          int64_t n_vocab, int32_t *accepted, int32_t *token, unsigned long long *err, cudaStream_t s) {
    const VerifyArgs a = {target, draft,   target_stride, draft_stride, tokens, count,
                          rand,   n_draft, int(n_vocab),  accepted,     token,  err};
    // Blocks of a cluster, of 256 threads: as many as are resident together, if each has enough to read. us of 1 / 16 /
    // 64 / 150 sequences, 3 drafts, 151936 tokens, four calls' inputs in turn (from 64 on beyond L2): 1 block
    // 24.4 / 34.2 / 48.9 / 52.9, 4 11.8 / 13.4 /
    // 20.4 / 36.7, 8 8.1 / 9.4 / 17.3 / 35.1, 16 6.9 / 9.0 / 25.4 / 49.0; of 32003 tokens 2 7.2 / 8.5 / 8.7, 4 6.4 / 6.8 / 7.6,
    // 8 6.2 / 6.3 / 8.2; of 1000: 64 sequences 1 block 6.4, 8 7.8. (512 threads: 64 sequences 17.6, one 7.6.)
    int most = 1;
    const cudaError_t e = max_cluster(&most);
    if (e != cudaSuccess) return e;
    const int64_t sms = sm_count();
    int64_t blocks = 1;
    auto good = [&](int64_t c) {
        return n_vocab >= c * kMinBlock &&
               (c * n_seq <= sms || (c * n_seq <= kResident * sms && n_vocab >= c * kMinShare));
    };
    while (blocks < most && good(2 * blocks)) blocks *= 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(blocks);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(unsigned(blocks), unsigned(n_seq));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel, a);
}

}  // namespace q2
