// Decode attention over a paged cache for sequences that share prefixes
// (q2_0_attn_plan_*).
//
// Work. The keys of one (kv head, prefix of a group) serve all the group's query
// heads of that kv head: rows = sequences x heads per kv head of one product. The
// own tokens of a sequence serve its heads per kv head. Both are cut into tiles of
// 128 keys, and the flat list of all tiles is dealt to one persistent block per SM
// in equal, contiguous shares (a block's run of tiles of one (prefix | sequence,
// kv head) is a segment). Every segment leaves an unnormalised output, reference
// and sum per row; a second kernel joins the segments of each query row.
//
// Products. Keys are the M of the first product and head elements the M of the
// second, so that the tensor core's 128 rows are always full and the few query
// rows are its N:
//   S^T [128 keys][N] = K Q^T,   O^T [dim][N] += V^T P^T
// K, Q and V are read from shared memory as TMA lays them down (K-major, K-major,
// MN-major, 128-byte swizzle); P is written by the softmax warps as the second
// product's MN-major B: a thread owns a key, and writes 16 bytes for each 8 rows.
//
// Softmax. p = 2^(s - ref + 7), ref a row's reference in log2 units: the maximum of
// the segment's first tile, raised to the running maximum only when a score
// passes it by more than 8 (then the output and sums so far are scaled down). Any
// ref gives the same quotient; this one keeps p below 2^15 (f16's largest is 2^16)
// and its rounding relative (normal f16) down to 2^-21 of the reference's weight,
// and spares most tiles a reduction over their keys. Sums of p stay in registers,
// one per (thread = key of the tile, row), and are reduced once per segment.
#include <cuda_bf16.h>

#include <algorithm>
#include <new>
#include <type_traits>

#include "q2_0_device.cuh"
#include "q2_0_internal.h"
#include "q2_0_tcgen05.cuh"

namespace q2 {

namespace {

constexpr int kTile = 128;     // keys per tile
constexpr int kThreads = 224;  // warps: 0 K/V copies, 1 MMA, 2-5 softmax, 6 Q copies
constexpr int kSoftThreads = 128;
constexpr int kTag = 300;      // waits' tags: 301..
constexpr float kLift = 7.0f;  // p = 2^(s - ref + kLift)
constexpr float kSlack = 8.0f; // how far a score may pass the reference

// Tile sizes of a variant: NCAP is the most query rows of a product.
template <int NCAP, int D>
struct Cfg {
    static constexpr int kStageBytes = kTile * D * 2;
    static constexpr int kHalves = D / 64;
    static constexpr int kQBufs = NCAP <= 64 ? 2 : 1;
    static constexpr int kPBufs = NCAP <= 32 ? 2 : 1;
    static constexpr int kQBytes = NCAP * D * 2;
    static constexpr int kPBytes = NCAP * kTile * 2;
    // what is left of 227 KB after Q, P and about 4 KB of small things
    static constexpr int kStages =
        (227 * 1024 - 5120 - kQBufs * kQBytes - kPBufs * kPBytes) / kStageBytes;
    static constexpr int kTmemCols = NCAP == 32 ? 128 : NCAP == 64 ? 256 : 512;
    static constexpr int kOCol = 2 * NCAP;  // S buffers at 0 and NCAP
    static constexpr int kBars = 2 * kStages + 2 * kQBufs + 4 + 2 * kPBufs + 1;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kQBufs * kQBytes +
                                 kPBufs * kPBytes + NCAP * 4 * 6 + kBars * 8 + 128;
    static_assert(kStages >= 4 && kSmem <= 227 * 1024, "shared memory");
};

struct AttnArgs {
    CUtensorMap k_map, v_map;   // [layers * pages * n_kv * page][dim], box {64, min(page, 128)}
    CUtensorMap qp_map, qs_map; // [seqs][n_q][dim], box {64, share, spb} and {64, share, 1}
    void *out;
    const int32_t *prefix_table, *prefix_len, *table, *len;
    int64_t prefix_width, width, n_pages;
    int n_groups, n_seq, n_q, n_kv, share;
    int spb, row_blocks;  // sequences of a row block of a prefix, row blocks
    int page_shift, dim;
    int row0;             // the layer's first row / (n_kv * page): layer * n_pages
    float scale_log2;     // scale * log2(e)
    // scratch
    long long *start;      // [groups + seqs + 1] first tile of each owner
    float *p_out, *s_out;  // segments' outputs: prefix [slot][NCAP][dim], own [slot][share][dim]
    float2 *p_ml, *s_ml;   // their (reference, sum): [slot][NCAP], [slot][share]
    int grid;
    unsigned long long *err;
};

// An owner of tiles: a group's prefix (o < n_groups) or a sequence.
__device__ __forceinline__ int owner_len(const AttnArgs &a, int o, bool record = false) {
    const bool pre = o < a.n_groups;
    if (pre && a.prefix_width == 0) return 0;
    const int n = pre ? a.prefix_len[o] : a.len[o - a.n_groups];
    const int most = int((pre ? a.prefix_width : a.width) << a.page_shift);
    if (n >= 0 && n <= most) return n;
    if (record)
        record_error(a.err, Q2_0_DEVERR_BAD_ID,
                     pre ? (long long)a.n_groups * a.n_seq + o : o - a.n_groups);
    return n < 0 ? 0 : most;
}
__device__ __forceinline__ int owner_items(const AttnArgs &a, int o) {
    return o < a.n_groups ? a.n_kv * a.row_blocks : a.n_kv;
}

// T tiles in shares over G <= T blocks (none is empty, so that a tile run's segments are
// those of consecutive blocks).
__device__ __forceinline__ int sharers(long long T, int grid) { return T < grid ? int(T) : grid; }
__host__ __device__ inline long long share_begin(long long c, long long T, int G) { return T * c / G; }
// the block that tile t belongs to
__host__ __device__ inline int share_owner(long long t, long long T, int G) {
    return int(((t + 1) * G + T - 1) / T) - 1;
}

// A block's run of tiles of one item.
struct Segment {
    int owner, item;   // item of the owner: head (own tokens) or head * row_blocks + row block
    int head, block;
    int t0, n;         // its tiles
    int len;           // the owner's keys
    int rows, N;       // query rows, and the product's N
};

// Goes over a block's segments; every role does so by itself.
struct Walk {
    int owner, len, nt;
    long long off, left;
    __device__ __forceinline__ bool next(const AttnArgs &a, Segment &s) {
        if (left <= 0) return false;
        while (nt == 0) {  // terminates: left > 0 tiles lie ahead
            ++owner;
            off = 0;
            len = owner_len(a, owner);
            nt = (len + kTile - 1) / kTile;
        }
        s.owner = owner;
        s.item = int(off / nt);
        s.t0 = int(off - (long long)s.item * nt);
        s.n = int(left < nt - s.t0 ? left : nt - s.t0);
        s.len = len;
        if (owner < a.n_groups) {
            s.head = s.item / a.row_blocks;
            s.block = s.item - s.head * a.row_blocks;
            const int seqs = a.n_seq - s.block * a.spb;
            s.rows = (seqs < a.spb ? seqs : a.spb) * a.share;
        } else {
            s.head = s.item;
            s.block = 0;
            s.rows = a.share;
        }
        s.N = s.rows <= 16 ? 16 : (s.rows + 31) & ~31;
        off += s.n;
        left -= s.n;
        if (off == (long long)nt * owner_items(a, owner)) nt = 0;
        return true;
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool BF>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    if (BF)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Over the lanes of the warp, for W = 32 or 16 values each: lane l gets the maximum
// (sum) of value l % W.
template <int W, bool kMax>
__device__ __forceinline__ float across(float (&v)[W]) {
    const int lane = threadIdx.x & 31;
    if (W == 16) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float o = __shfl_xor_sync(0xffffffffu, v[i], 16);
            v[i] = kMax ? fmaxf(v[i], o) : v[i] + o;
        }
    }
#pragma unroll
    for (int h = W / 2; h; h >>= 1) {
        const bool hi = lane & h;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float keep = hi ? v[i + h] : v[i], send = hi ? v[i] : v[i + h];
            const float o = __shfl_xor_sync(0xffffffffu, send, h);
            v[i] = kMax ? fmaxf(keep, o) : keep + o;
        }
    }
    return v[0];
}

template <int W>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[W]) {
    uint32_t r[W];
    if constexpr (W == 32) {
        tmem_ld32(addr, r);
    } else {
        tmem_ld16(addr, r);
        tmem_wait_ld();
    }
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = __uint_as_float(r[i]);
}
template <int W>
__device__ __forceinline__ void tmem_store(uint32_t addr, const float (&v)[W]) {
    uint32_t r[W];
#pragma unroll
    for (int i = 0; i < W; ++i) r[i] = __float_as_uint(v[i]);
    if constexpr (W == 32)
        tmem_st32(addr, r);
    else
        tmem_st16(addr, r);
    tmem_wait_st();
}

// Barrier of the softmax warps.
__device__ __forceinline__ void soft_sync() {
    asm volatile("bar.sync 1, 128;" ::: "memory");
}
__device__ __forceinline__ bool soft_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, 2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(v))
        : "memory");
    return r != 0;
}

// Calls f over the columns [0, N) in pieces: 16 wide if N = 16, else 32 (f is
// instantiated for both; c is a compile-time constant after unrolling).
template <int NCAP, typename F>
__device__ __forceinline__ void columns(int N, F f) {
    if (N == 16) {
        f(std::integral_constant<int, 16>{}, std::integral_constant<int, 0>{});
        return;
    }
    f(std::integral_constant<int, 32>{}, std::integral_constant<int, 0>{});
    if constexpr (NCAP > 32)
        if (N > 32) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 32>{});
    if constexpr (NCAP > 64) {
        if (N > 64) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 64>{});
        if (N > 96) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 96>{});
    }
}

template <int NCAP, int D, bool BF>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ AttnArgs a) {
    using C = Cfg<NCAP, D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem;
    uint8_t *q_s = ring + C::kStages * C::kStageBytes;
    uint8_t *p_s = q_s + C::kQBufs * C::kQBytes;
    float *nref_s = reinterpret_cast<float *>(p_s + C::kPBufs * C::kPBytes);  // kLift - ref
    float *alpha_s = nref_s + NCAP;
    float *red_s = alpha_s + NCAP;  // [4][NCAP]
    uint64_t *bars = reinterpret_cast<uint64_t *>(red_s + 4 * NCAP);
    uint64_t *kv_full = bars, *kv_empty = kv_full + C::kStages;
    uint64_t *q_full = kv_empty + C::kStages, *q_empty = q_full + C::kQBufs;
    uint64_t *s_full = q_empty + C::kQBufs, *s_empty = s_full + 2;
    uint64_t *p_full = s_empty + 2, *p_empty = p_full + C::kPBufs;
    uint64_t *o_full = p_empty + C::kPBufs;
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(o_full + 1);
    __shared__ long long sum_s[kThreads / 32];
    __shared__ int first_owner_s;
    __shared__ long long first_off_s;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < C::kQBufs; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 4);
        }
        for (int i = 0; i < C::kPBufs; ++i) {
            mbar_init(&p_full[i], 4);
            mbar_init(&p_empty[i], 1);
        }
        mbar_init(o_full, 1);
        fence_barrier_init();
        prefetch_tensormap(&a.k_map);
        prefetch_tensormap(&a.v_map);
        prefetch_tensormap(&a.qp_map);
        prefetch_tensormap(&a.qs_map);
    }
    if (warp == 1) {
        tmem_alloc(tmem_ptr, C::kTmemCols);
        tmem_relinquish();
    }
    // rows that no copy fills are zero or an earlier segment's
    for (int i = tid; i < C::kQBufs * C::kQBytes / 16; i += kThreads)
        reinterpret_cast<uint4 *>(q_s)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the tile list: each thread sums a run of owners, then finds the block's first tile
    const int owners = a.n_groups + a.n_groups * a.n_seq;
    const int per = (owners + kThreads - 1) / kThreads;
    const int o0 = min(tid * per, owners), o1 = min(o0 + per, owners);
    long long mine = 0;
    for (int o = o0; o < o1; ++o)
        mine += (long long)((owner_len(a, o, blockIdx.x == 0) + kTile - 1) / kTile) * owner_items(a, o);
    long long scan = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += v;
    }
    if (lane == 31) sum_s[warp] = scan;
    __syncthreads();
    long long before = scan - mine, T = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sum_s[w];
        T += sum_s[w];
    }
    const int G = sharers(T, gridDim.x);
    const bool has = int(blockIdx.x) < G;
    const long long begin = has ? share_begin(blockIdx.x, T, G) : T;
    const long long end = has ? share_begin(blockIdx.x + 1, T, G) : T;
    if (blockIdx.x == 0 || (begin >= before && begin < before + mine)) {
        long long at = before;
        for (int o = o0; o < o1; ++o) {
            const long long n =
                (long long)((owner_len(a, o) + kTile - 1) / kTile) * owner_items(a, o);
            if (blockIdx.x == 0) a.start[o] = at;
            if (begin >= at && begin < at + n) {
                first_owner_s = o;
                first_off_s = begin - at;
            }
            at += n;
        }
        if (blockIdx.x == 0 && tid == 0) a.start[owners] = T;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_ptr;

    Walk walk;
    walk.left = end - begin;
    if (walk.left > 0) {
        walk.owner = first_owner_s;
        walk.off = first_off_s;
        walk.len = owner_len(a, walk.owner);
        walk.nt = (walk.len + kTile - 1) / kTile;
    }
    Segment s;

    if (warp == 0) {
        // ------------------------------ K and V copies ------------------------------
        const int page = 1 << a.page_shift;
        const int box = page < kTile ? page : kTile;
        const int box_bytes = box * 128;
        int st = 0;
        uint32_t ph = 0;
        bool ok = true;
        while (ok && walk.next(a, s)) {
            const bool pre = s.owner < a.n_groups;
            const int64_t who = pre ? s.owner : s.owner - a.n_groups;
            const int32_t *row = pre ? a.prefix_table + who * a.prefix_width : a.table + who * a.width;
            for (int t = s.t0; t < s.t0 + s.n; ++t) {
                const int left = s.len - t * kTile;
                const int n = ((left < kTile ? left : kTile) + box - 1) / box;  // boxes with keys
                // lane l copies box l / kHalves, columns 64 * (l % kHalves)
                const int b = lane / C::kHalves, half = lane % C::kHalves;
                int at = 0;
                if (b < n) {
                    const int key = t * kTile + b * box;
                    int id = row[key >> a.page_shift];
                    if (id < 0 || id >= a.n_pages) {
                        record_error(a.err, Q2_0_DEVERR_BAD_ID,
                                     pre ? (long long)a.n_groups * a.n_seq + who : who);
                        id = 0;
                    }
                    at = (((a.row0 + id) * a.n_kv + s.head) << a.page_shift) + (key & (page - 1));
                }
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[st], ph ^ 1u, a.err, kTag + 1, true));
                    if (!ok) break;
                    if (lane == 0)
                        mbar_arrive_expect_tx(&kv_full[st], uint32_t(n * C::kHalves * box_bytes));
                    __syncwarp();
                    if (b < n)
                        tma_load_2d(ring + st * C::kStageBytes + half * (kTile * 128) + b * box_bytes,
                                    kv ? &a.v_map : &a.k_map, half * 64, at, &kv_full[st]);
                    if (++st == C::kStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
            }
        }
        if (!ok)  // let the copies in flight land (bounded)
            for (int k = 0; k < C::kStages; ++k) {
                if (--st < 0) {
                    st = C::kStages - 1;
                    ph ^= 1u;
                }
                mbar_wait(&kv_full[st], ph, a.err, kTag + 2);
            }
    } else if (warp == 6) {
        // --------------------------------- Q copies ---------------------------------
        for (int n = 0; walk.next(a, s); ++n) {
            const int qb = n % C::kQBufs, use = n / C::kQBufs;
            if (use > 0 && !__all_sync(0xffffffffu, mbar_wait(&q_empty[qb], uint32_t(use - 1) & 1u, a.err,
                                                              kTag + 3, true)))
                break;
            if (lane == 0) {
                const bool pre = s.owner < a.n_groups;
                const int rows = (pre ? a.spb : 1) * a.share;  // of the box
                const int seq = pre ? s.owner * a.n_seq + s.block * a.spb : s.owner - a.n_groups;
                mbar_arrive_expect_tx(&q_full[qb], uint32_t(rows * D * 2));
                for (int h = 0; h < C::kHalves; ++h)
                    tma_load_3d(q_s + qb * C::kQBytes + h * (NCAP * 128), pre ? &a.qp_map : &a.qs_map,
                                h * 64, s.head * a.share, seq, &q_full[qb]);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        // ------------------------------------ MMA ------------------------------------
        const uint32_t types = (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u);
        const bool leader = elect_one();
        int st = 0, seg = 0;
        uint32_t ph = 0;
        int n = 0;  // tiles so far
        bool ok = true;
        // the second product of the tile before: it is issued after the next tile's first
        bool pend = false, p_first = false, p_last = false;
        int p_st = 0, p_steps = 0, p_n = 0, p_N = 0;
        uint32_t p_ph = 0;
        auto second = [&]() {
            const int pb = p_n % C::kPBufs;
            const uint32_t use = uint32_t(p_n / C::kPBufs);
            const bool got = mbar_wait2(&kv_full[p_st], p_ph, kTag + 4, &p_full[pb], use & 1u, kTag + 5,
                                        a.err, kWaitLimitNs);
            if (!__all_sync(0xffffffffu, got)) return false;
            tc_fence_after();
            if (leader) {
                // A = V^T: MN-major; dim 64 reads its one half twice (lanes 64.. are not used)
                const uint32_t idesc = types | (1u << 15) | (1u << 16) | (uint32_t(p_N >> 3) << 17) |
                                       (uint32_t(kTile >> 4) << 24);
                const uint32_t va = smem_addr(ring + p_st * C::kStageBytes);
                const uint32_t pa = smem_addr(p_s + pb * C::kPBytes);
                for (int ks = 0; ks < p_steps; ++ks)
                    tc_mma_f16_ss(tmem + C::kOCol,
                                  smem_desc(va + ks * 2048, C::kHalves == 2 ? kTile * 128 : 0, 1024, 2),
                                  smem_desc(pa + ks * 256, 128, kTile * 16, 0), idesc,
                                  !p_first || ks > 0);
                tc_commit(&kv_empty[p_st]);
                tc_commit(&p_empty[pb]);
                if (p_last) tc_commit(o_full);
            }
            __syncwarp();
            pend = false;
            return true;
        };
        for (; ok && walk.next(a, s); ++seg) {
            if (C::kQBufs == 1 && pend && !second()) {
                ok = false;
                break;
            }
            const int qb = seg % C::kQBufs;
            if (!__all_sync(0xffffffffu,
                            mbar_wait(&q_full[qb], uint32_t(seg / C::kQBufs) & 1u, a.err, kTag + 6))) {
                ok = false;
                break;
            }
            const uint32_t idesc =
                types | (uint32_t(s.N >> 3) << 17) | (uint32_t(kTile >> 4) << 24);
            const uint32_t qa = smem_addr(q_s + qb * C::kQBytes);
            for (int i = 0; i < s.n; ++i, ++n) {
                const int sb = n & 1;
                const uint32_t use = uint32_t(n >> 1);
                bool got = mbar_wait(&kv_full[st], ph, a.err, kTag + 7);
                if (use > 0) got = got && mbar_wait(&s_empty[sb], (use - 1) & 1u, a.err, kTag + 8);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (leader) {
                    const uint32_t ka = smem_addr(ring + st * C::kStageBytes);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        tc_mma_f16_ss(tmem + sb * NCAP,
                                      sw128_desc(ka + (ks / 4) * (kTile * 128) + (ks % 4) * 32),
                                      sw128_desc(qa + (ks / 4) * (NCAP * 128) + (ks % 4) * 32), idesc,
                                      ks > 0);
                    tc_commit(&kv_empty[st]);
                    tc_commit(&s_full[sb]);
                    if (i == s.n - 1) tc_commit(&q_empty[qb]);
                }
                __syncwarp();
                if (++st == C::kStages) {
                    st = 0;
                    ph ^= 1u;
                }
                if (pend && !second()) {
                    ok = false;
                    break;
                }
                const int keys = s.len - (s.t0 + i) * kTile;
                pend = true;
                p_first = i == 0;
                p_last = i == s.n - 1;
                p_steps = keys >= kTile ? kTile / 16 : (keys + 15) / 16;
                p_st = st;
                p_ph = ph;
                p_n = n;
                p_N = s.N;
                if (++st == C::kStages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
        }
        if (ok && pend) ok = second();
        if (!ok && leader) {
            // the products in flight end before tensor memory is freed (bounded)
            tc_commit(o_full);
        }
    } else {
        // ---------------------------------- softmax ----------------------------------
        // Thread = key `key` of the tile, or element `key` of the head in the output.
        const int quarter = warp & 3;
        const int key = quarter * 32 + lane;
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        const float c = a.scale_log2;
        float l[NCAP];
        int n = 0;         // tiles so far
        int st = 1;        // the ring stage of the tile's V
        uint32_t ph = 0;
        // A warp whose wait timed out waits no more: it goes through the motions, so that
        // the barriers of the softmax warps stay matched, and its results mean nothing.
        bool dead = false;
        auto wait = [&](uint64_t *bar, uint32_t parity, int tag) {
            if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, a.err, tag));
        };
        for (int seg = 0; walk.next(a, s); ++seg) {
            const int N = s.N;
#pragma unroll
            for (int i = 0; i < NCAP; ++i) l[i] = 0.0f;
            for (int i = 0; i < s.n; ++i, ++n) {
                const int sb = n & 1, pb = n % C::kPBufs;
                const int keys = s.len - (s.t0 + i) * kTile;  // valid ones of this tile, if < 128
                const bool in = key < keys;
                const uint32_t sa = tmem + lanes + sb * NCAP;
                wait(&s_full[sb], uint32_t(n >> 1), kTag + 9);
                tc_fence_after();
                bool raise = i == 0;
                if (!raise) {
                    float most = -INFINITY;
                    columns<NCAP>(N, [&](auto w, auto c0) {
                        constexpr int W = w, C0 = c0;
                        float v[W];
                        tmem_load<W>(sa + C0, v);
#pragma unroll
                        for (int j = 0; j < W; j += 4) {
                            const float4 r = *reinterpret_cast<const float4 *>(nref_s + C0 + j);
                            most = fmaxf(most, fmaxf(fmaxf(fmaf(v[j], c, r.x), fmaf(v[j + 1], c, r.y)),
                                                     fmaxf(fmaf(v[j + 2], c, r.z), fmaf(v[j + 3], c, r.w))));
                        }
                    });
                    raise = soft_any(in && most > kSlack + kLift);
                }
                if (raise) {
                    // the rows' maxima over the tile, and with them new references
                    columns<NCAP>(N, [&](auto w, auto c0) {
                        constexpr int W = w, C0 = c0;
                        float v[W];
                        tmem_load<W>(sa + C0, v);
#pragma unroll
                        for (int j = 0; j < W; ++j) v[j] = in ? v[j] * c : -INFINITY;
                        const float m = across<W, true>(v);
                        if (lane < W) red_s[quarter * NCAP + C0 + lane] = m;
                    });
                    soft_sync();
                    if (key < N) {
                        const float old = i == 0 ? -INFINITY : kLift - nref_s[key];
                        float m = fmaxf(fmaxf(red_s[key], red_s[NCAP + key]),
                                        fmaxf(red_s[2 * NCAP + key], red_s[3 * NCAP + key]));
                        // no key counts (scores of -inf): any finite reference does
                        m = fmaxf(fmaxf(m, old), -1e30f);
                        alpha_s[key] = ex2(old - m);
                        nref_s[key] = kLift - m;
                    }
                    soft_sync();
                    if (i > 0) {
                        wait(&p_empty[(n - 1) % C::kPBufs], uint32_t((n - 1) / C::kPBufs), kTag + 10);
                        tc_fence_after();
                        columns<NCAP>(N, [&](auto w, auto c0) {
                            constexpr int W = w, C0 = c0;
                            float v[W];
                            tmem_load<W>(tmem + lanes + C::kOCol + C0, v);
#pragma unroll
                            for (int j = 0; j < W; ++j) {
                                const float f = alpha_s[C0 + j];
                                v[j] *= f;
                                l[C0 + j] *= f;
                            }
                            tmem_store<W>(tmem + lanes + C::kOCol + C0, v);
                        });
                    }
                }
                if (n >= C::kPBufs) wait(&p_empty[pb], uint32_t(n / C::kPBufs - 1), kTag + 11);
                uint8_t *ps = p_s + pb * C::kPBytes + key * 16;
                columns<NCAP>(N, [&](auto w, auto c0) {
                    constexpr int W = w, C0 = c0;
                    float v[W];
                    tmem_load<W>(sa + C0, v);
#pragma unroll
                    for (int j = 0; j < W; j += 4) {
                        const float4 r = *reinterpret_cast<const float4 *>(nref_s + C0 + j);
                        v[j] = ex2(fmaf(v[j], c, r.x));
                        v[j + 1] = ex2(fmaf(v[j + 1], c, r.y));
                        v[j + 2] = ex2(fmaf(v[j + 2], c, r.z));
                        v[j + 3] = ex2(fmaf(v[j + 3], c, r.w));
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        v[j] = in ? v[j] : 0.0f;
                        l[C0 + j] += v[j];
                    }
#pragma unroll
                    for (int j = 0; j < W; j += 8)
                        *reinterpret_cast<uint4 *>(ps + ((C0 + j) / 8) * (kTile * 16)) =
                            make_uint4(pack<BF>(v[j], v[j + 1]), pack<BF>(v[j + 2], v[j + 3]),
                                       pack<BF>(v[j + 4], v[j + 5]), pack<BF>(v[j + 6], v[j + 7]));
                });
                if (keys < kTile && (keys & 15)) {
                    // places past the last key up to the product's 16: whatever V holds there,
                    // 0 times it has to be 0
                    wait(&kv_full[st], ph, kTag + 12);
                    const int n0 = 16 - (keys & 15);
                    for (int x = key; x < n0 * C::kHalves * 8; x += kSoftThreads) {
                        const int piece = x & 7, r = (x >> 3) / C::kHalves, h = (x >> 3) % C::kHalves;
                        *reinterpret_cast<uint4 *>(ring + st * C::kStageBytes + h * (kTile * 128) +
                                                   (keys + r) * 128 + piece * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s_empty[sb]);
                    mbar_arrive(&p_full[pb]);
                }
                st += 2;
                if (st >= C::kStages) {
                    st -= C::kStages;
                    ph ^= 1u;
                }
            }
            // ---- the segment's output, references and sums
            const bool pre = s.owner < a.n_groups;
            const int64_t slot =
                (pre ? int64_t(s.owner) * a.n_kv * a.row_blocks : int64_t(s.owner - a.n_groups) * a.n_kv) +
                s.item + blockIdx.x;
            const int64_t stride = pre ? NCAP : a.share;
            float *out = (pre ? a.p_out : a.s_out) + slot * stride * D;
            float2 *ml = (pre ? a.p_ml : a.s_ml) + slot * stride;
            columns<NCAP>(N, [&](auto w, auto c0) {
                constexpr int W = w, C0 = c0;
                float v[W];
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] = l[C0 + j];
                const float t = across<W, false>(v);
                if (lane < W) red_s[quarter * NCAP + C0 + lane] = t;
            });
            soft_sync();
            if (key < s.rows)
                ml[key] = make_float2(kLift - nref_s[key],
                                      (red_s[key] + red_s[NCAP + key]) +
                                          (red_s[2 * NCAP + key] + red_s[3 * NCAP + key]));
            wait(o_full, uint32_t(seg), kTag + 13);
            tc_fence_after();
            columns<NCAP>(N, [&](auto w, auto c0) {
                constexpr int W = w, C0 = c0;
                float v[W];
                tmem_load<W>(tmem + lanes + C::kOCol + C0, v);
                if (key < D) {
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        if (C0 + j < s.rows) out[(C0 + j) * D + key] = v[j];
                }
            });
            tc_fence_before();
            soft_sync();  // nref_s and red_s are free again
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Joins the segments of each query row: one warp per row, one block per (sequence,
// kv head).
template <int D, bool BF>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnArgs a, int ncap) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.x, head = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = b / a.n_seq, in_group = b - group * a.n_seq;
    const long long T = a.start[a.n_groups + a.n_groups * a.n_seq];
    // the segments of the prefix's item and of the sequence's: slots [c0, c1] of each
    int c0[2], c1[2];
    int64_t slot[2];
    const int block = in_group / a.spb;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int o = w ? a.n_groups + b : group;
        const int items = w ? a.n_kv : a.n_kv * a.row_blocks;
        const int item = w ? head : head * a.row_blocks + block;
        const long long s0 = a.start[o];
        const long long nt = (a.start[o + 1] - s0) / items;
        c0[w] = 0;
        c1[w] = -1;
        if (nt > 0) {
            c0[w] = share_owner(s0 + item * nt, T, sharers(T, a.grid));
            c1[w] = share_owner(s0 + item * nt + nt - 1, T, sharers(T, a.grid));
        }
        slot[w] = (w ? int64_t(b) * a.n_kv : int64_t(group) * a.n_kv * a.row_blocks) + item;
    }
    const int np = c1[0] - c0[0] + 1, n = np + c1[1] - c0[1] + 1;
    constexpr int E = D / 32;  // elements per lane
    for (int r = warp; r < a.share; r += 4) {
        const int pr = (in_group - block * a.spb) * a.share + r;  // row in the prefix's item
        auto at = [&](int i) {  // segment i's row: index into (out, ml) of its region
            return i < np ? (slot[0] + c0[0] + i) * ncap + pr : (slot[1] + c0[1] + i - np) * a.share + r;
        };
        float m = -INFINITY;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, (i < np ? a.p_ml : a.s_ml)[at(i)].x);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float acc[E], l = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const int64_t x = at(i);
            const float2 ml = (i < np ? a.p_ml : a.s_ml)[x];
            const float *o = (i < np ? a.p_out : a.s_out) + x * D + lane * E;
            const float w = ex2(ml.x - m);
            l += w * ml.y;
            if (E == 4) {
                const float4 v = *reinterpret_cast<const float4 *>(o);
                acc[0] += w * v.x;
                acc[1] += w * v.y;
                acc[E - 2] += w * v.z;
                acc[E - 1] += w * v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2 *>(o);
                acc[0] += w * v.x;
                acc[1] += w * v.y;
            }
        }
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // (NaN stays NaN)
        uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) +
                                                     (int64_t(b) * a.n_q + head * a.share + r) * D +
                                                     lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) dst[e / 2] = pack<BF>(acc[e] * inv, acc[e + 1] * inv);
    }
}

}  // namespace
}  // namespace q2

struct q2_0_attn_plan {
    q2::AttnArgs args;
    int ncap, dim, n_layers, device;
    bool bf;
    int64_t n_pages;
    void *scratch;
};

namespace q2 {

namespace {

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

using Kernel = void (*)(AttnArgs);
struct Variant {
    Kernel fn;
    int smem;
};
template <int NCAP, int D, bool BF>
Variant variant() {
    return {attn_kernel<NCAP, D, BF>, Cfg<NCAP, D>::kSmem};
}
template <int NCAP>
Variant variant_n(int dim, bool bf) {
    if (dim == 64) return bf ? variant<NCAP, 64, true>() : variant<NCAP, 64, false>();
    return bf ? variant<NCAP, 128, true>() : variant<NCAP, 128, false>();
}
Variant variant_of(int ncap, int dim, bool bf) {
    if (ncap == 32) return variant_n<32>(dim, bf);
    if (ncap == 64) return variant_n<64>(dim, bf);
    return variant_n<128>(dim, bf);
}

}  // namespace

int attn_plan_create(const q2_0_attn_desc &d, q2_0_attn_plan **plan) {
    unsigned long long *err = error_word_ptr();
    const int sms = sm_count();
    if (!err || sms < 1) return Q2_0_ECUDA;
    q2_0_attn_plan *p = new (std::nothrow) q2_0_attn_plan;
    if (!p) return Q2_0_ECUDA;
    const q2_0_kv_cache &c = d.cache;
    AttnArgs &a = p->args;
    a.out = d.out;
    a.prefix_table = d.prefix_table;
    a.prefix_len = d.prefix_len;
    a.table = d.table;
    a.len = d.len;
    a.prefix_width = d.prefix_width;
    a.width = d.width;
    a.n_pages = c.n_pages;
    a.n_groups = int(d.n_groups);
    a.n_seq = int(d.n_seq);
    a.n_q = d.n_q;
    a.n_kv = c.n_kv;
    a.share = d.n_q / c.n_kv;
    a.page_shift = log2_of(c.page);
    a.dim = c.dim;
    a.row0 = 0;
    a.scale_log2 = d.scale * 1.44269504f;
    a.grid = sms;
    a.err = err;
    // the smallest product that holds a prefix's rows: 32, 64 or 128 at a time
    const int64_t rows = d.prefix_width ? d.n_seq * a.share : a.share;
    p->ncap = rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    a.spb = int(std::min<int64_t>(d.n_seq, p->ncap / a.share));
    a.row_blocks = d.prefix_width ? (a.n_seq + a.spb - 1) / a.spb : 1;
    p->dim = c.dim;
    p->n_layers = c.n_layers;
    p->n_pages = c.n_pages;
    p->bf = c.type == Q2_0_TYPE_BF16;
    const CUtensorMapDataType ty =
        p->bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const uint64_t rows_all = uint64_t(c.n_layers) * c.n_pages * c.n_kv * c.page;
    const uint64_t row_bytes = uint64_t(c.dim) * 2;
    const uint64_t seqs = uint64_t(d.n_groups) * d.n_seq;
    const uint64_t qdims[3] = {uint64_t(c.dim), uint64_t(d.n_q), seqs};
    const uint64_t qstr[2] = {row_bytes, row_bytes * d.n_q};
    const uint32_t box_p[3] = {64, uint32_t(a.share), uint32_t(a.spb)};
    const uint32_t box_s[3] = {64, uint32_t(a.share), 1};
    const uint32_t key_box = uint32_t(std::min(c.page, kTile));
    bool ok = encode_tmap_2d(&a.k_map, ty, c.k, c.dim, rows_all, row_bytes, 64, key_box,
                             CU_TENSOR_MAP_SWIZZLE_128B) &&
              encode_tmap_2d(&a.v_map, ty, c.v, c.dim, rows_all, row_bytes, 64, key_box,
                             CU_TENSOR_MAP_SWIZZLE_128B) &&
              encode_tmap_3d(&a.qp_map, ty, d.q, qdims, qstr, box_p, CU_TENSOR_MAP_SWIZZLE_128B) &&
              encode_tmap_3d(&a.qs_map, ty, d.q, qdims, qstr, box_s, CU_TENSOR_MAP_SWIZZLE_128B);
    // A segment's slot is its item's number plus its block's: both never fall from one
    // segment to the next, and one of them rises.
    const size_t p_slots = d.prefix_width ? size_t(a.n_groups) * a.n_kv * a.row_blocks + sms : 0;
    const size_t s_slots = size_t(seqs) * a.n_kv + sms;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += align256(bytes);
        return o;
    };
    const size_t o_start = take((size_t(a.n_groups) + seqs + 1) * 8);
    const size_t o_p = take(p_slots * p->ncap * c.dim * 4), o_s = take(s_slots * a.share * c.dim * 4);
    const size_t o_pml = take(p_slots * p->ncap * 8), o_sml = take(s_slots * a.share * 8);
    p->scratch = nullptr;
    if (ok) ok = cudaMalloc(&p->scratch, at) == cudaSuccess;
    const Variant v = variant_of(p->ncap, p->dim, p->bf);
    if (ok)
        ok = cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem) ==
             cudaSuccess;
    if (!ok) {
        if (p->scratch) cudaFree(p->scratch);
        delete p;
        return Q2_0_ECUDA;
    }
    char *base = static_cast<char *>(p->scratch);
    a.start = reinterpret_cast<long long *>(base + o_start);
    a.p_out = reinterpret_cast<float *>(base + o_p);
    a.s_out = reinterpret_cast<float *>(base + o_s);
    a.p_ml = reinterpret_cast<float2 *>(base + o_pml);
    a.s_ml = reinterpret_cast<float2 *>(base + o_sml);
    *plan = p;
    return Q2_0_OK;
}

int attn_plan_execute(const q2_0_attn_plan *p, int layer, cudaStream_t s) {
    AttnArgs a = p->args;
    a.row0 = int(layer * p->n_pages);
    const Variant v = variant_of(p->ncap, p->dim, p->bf);
    // Each launch may be set up while the one before it drains; both wait for its
    // results (griddepcontrol.wait) before they read anything.
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(unsigned(a.grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = size_t(v.smem);
    cudaError_t e = cudaLaunchKernelEx(&cfg, v.fn, a);
    if (e != cudaSuccess) return cuda_status(e);
    cfg.gridDim = dim3(unsigned(a.n_groups * a.n_seq), unsigned(a.n_kv));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    auto *join = p->dim == 64 ? (p->bf ? attn_join_kernel<64, true> : attn_join_kernel<64, false>)
                              : (p->bf ? attn_join_kernel<128, true> : attn_join_kernel<128, false>);
    return cuda_status(cudaLaunchKernelEx(&cfg, join, a, p->ncap));
}

int attn_plan_launches(const q2_0_attn_plan *) { return 2; }

int attn_plan_layers(const q2_0_attn_plan *p) { return p->n_layers; }

void attn_plan_destroy(q2_0_attn_plan *p) {
    cudaFree(p->scratch);
    delete p;
}

}  // namespace q2
