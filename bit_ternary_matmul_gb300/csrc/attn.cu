// Decode attention over a paged cache for sequences that share prefixes
// (q2_0_attn_plan_*).
//
// Work. The keys of one (kv head, prefix of a group) serve all the group's query
// heads of that kv head: rows = sequences x heads per kv head of one product. The own
// tokens of a sequence serve its heads per kv head. Both are cut into tiles of 128
// keys, and the flat list of all tiles is dealt to one persistent block per SM in
// contiguous shares of equal cost (a block's run of tiles of one (prefix | sequence,
// kv head, row block) is a segment). Segments leave unnormalised outputs, references
// and sums per row; a last kernel joins those of each query row.
//
// Softmax. p = 2^(s - ref + 7), ref a row's reference in log2 units: the maximum of
// the first tile, raised to the running maximum only when a score passes it by more
// than 8 (then the output and sums so far are scaled down). Any ref gives the same
// quotient; this one keeps p below 2^15 (f16's largest is 2^16) and its rounding
// relative (normal f16) down to 2^-21 of the reference's weight, and spares most tiles
// the scaling. Scores, sums and outputs are f32; p is rounded to the cache's type to be
// the second product's operand.
//
// Two kernels, by the rows of a product:
//   Up to 64 (attn_kernel): keys are the M of the first product and head elements the
//   M of the second, so that the tensor core's 128 rows are full and the few query
//   rows are its N:  S^T [128 keys][N] = K Q^T,  O^T [dim][N] += V^T P^T.
//   K, Q and V are read from shared memory as TMA lays them down (K-major, K-major,
//   MN-major, 128-byte swizzle); P is written by the softmax warps as the second
//   product's MN-major B: a thread owns a key, and writes 16 bytes for each 8 rows.
//   Two groups of four warps take turns at the tiles, each with scores, weights,
//   references, sums and output of its own (two records per segment): a tile's chain of
//   steps, about 1300 clocks, is longer than half of what its 64 KB take to arrive.
//   More (attn_rows_kernel, prefixes only): query rows are the M of both products,
//   S [128 rows][128 keys] = Q K^T,  O [128][dim] += P V, with up to 256 rows to a tile
//   in shared memory. A thread owns a row, so that references and sums are its own,
//   and P stays in tensor memory, over the scores. With keys as M these products would
//   read 128 KB and write 32 KB of shared memory per 128 rows, 1800 clocks of its
//   bandwidth with the copies; here 64 KB per 128 rows and P not at all.
//
// Measured on one GB300 (device time of an execute, in a graph; floors at its 6.7 TB/s
// copy): 4 beams, 517 shared and 37 own tokens, 16 / 8 heads of 128: 11.3 us (latency:
// clocks read in an earlier version gave 2 us to the deal and 3 to 5 more to the first
// scores). 8 beams, 50021 + 200, 32 / 8 heads of 128: 44.4 us, floor 31.6 (the same clocks:
// first scores 6 to 8 us after the deal, with all blocks' first tiles in flight). 4 x 16
// sequences, up to 4099 + 1500, 16 heads of 64: 55.8 us, floor 37.4 (the same clocks: about
// 4000 to end a segment, 1200 to 1700 of work a tile). 64 sequences, 131072 + up to 3000,
// 32 / 8 heads of 128: 190 us, floor 139. Profiled one by one with cold caches,
// attn_rows_kernel takes 123 us of it (tensor pipe 48 % busy, memory 56 %: neither is full)
// and attn_kernel 72 (memory 74 %).
#include <cuda_bf16.h>
#include <float.h>

#include <algorithm>
#include <atomic>
#include <new>
#include <type_traits>

#include "q2_0_attn.cuh"
#include "q2_0_internal.h"

namespace q2 {

namespace {

constexpr int kTile = 128;     // keys per tile
constexpr int kThreads = 384;  // 4 warps that copy and multiply, 8 of softmax
// Registers: launched with 168 per thread, 64512 in all; the first four warps leave some (kRegsFew)
// to the softmax warps (kRegsMany). A spilled register costs more here than elsewhere: shared
// memory leaves the first-level cache next to nothing.
constexpr bool regs_fit(int few, int many) { return 128 * few + 256 * many == 384 * 168; }
constexpr int kTag = 300;      // waits' tags: 301..
constexpr float kLift = 7.0f;  // p = 2^(s - ref + kLift)
constexpr float kSlack = 8.0f; // how far a score may pass the reference
constexpr float kFused = 1.6e7f; // references up to which a score is scaled and reduced by it in one operation
// Cost of a tile, and of a segment beside its tiles, for the shares. Measured (four groups of
// sixteen, 4099 shared and up to 1500 own tokens, dim 64): 4 of an item 64.0 us, 8 59.3, 14 55.3,
// 20 55.9, 28 59.3; 8 beams on 50021 tokens of dim 128 43.6 to 44.2 with any of them.
constexpr int kTileCost = 4, kItemCost = 14;

// Sizes of a variant of attn_kernel: NCAP, 32 or 64, is the most query rows of a product.
template <int NCAP, int D>
struct Cfg {
    static constexpr int kRegsFew = NCAP == 32 ? 136 : 88, kRegsMany = NCAP == 32 ? 184 : 208;
    static_assert(regs_fit(kRegsFew, kRegsMany), "registers");
    static constexpr int kStageBytes = kTile * D * 2;
    static constexpr int kHalves = D / 64;
    static constexpr int kQBufs = NCAP <= 32 ? 2 : 1;
    static constexpr int kQBytes = NCAP * D * 2;
    static constexpr int kPBytes = NCAP * kTile * 2;
    static constexpr int kRefs = 2 * 6 * NCAP;  // floats
    // references, barriers, the tile list's 12 + 2 sums
    static constexpr int kSmall = kRefs * 4 + 448;
    // K and V have stages of their own, half of the ring each. (Their consumers are different warps;
    // in a shared stage one could be a whole phase ahead of the other, which a wait by parity
    // does not see.) A fifth stage of NCAP = 64, D = 128, given to either, was slower (60 against
    // 55.5 us for 64 rows and 50021 keys).
    static constexpr int kStages =
        (227 * 1024 - kSmall - kQBufs * kQBytes - 2 * kPBytes) / kStageBytes / 2 * 2;
    static constexpr int kK = kStages / 2, kV = kK;
    static constexpr int kTmemCols = 4 * NCAP;
    static constexpr int kOCol = 2 * NCAP;  // S buffers at 0 and NCAP, O at 2 NCAP and 3 NCAP
    static constexpr int kSmem = kSmall + kStages * kStageBytes + kQBufs * kQBytes + 2 * kPBytes;
    static constexpr int kBars = 2 * kStages + 2 * kQBufs + 10;
    static_assert(kStages >= 4 && kSmem <= 227 * 1024, "shared memory");
    static_assert((kBars + 1 + kThreads / 32 + 2) * 8 <= 448, "barriers and sums");
};

// Sizes of attn_rows_kernel: kRows, 128 or 256, query rows of D.
template <int ROWS, int D>
struct RowsCfg {
    static constexpr int kRows = ROWS;
    static constexpr int kRegsFew = 120, kRegsMany = 192;
    static_assert(regs_fit(kRegsFew, kRegsMany), "registers");
    static constexpr int kStageBytes = kTile * D * 2;
    static constexpr int kHalves = D / 64;
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kSmall = 512;
    static constexpr int kStages = (227 * 1024 - kSmall - kQBytes) / kStageBytes;
    static constexpr int kK = kStages / 2, kV = kStages - kK;  // as above
    static constexpr int kOCol = 256;  // S (and P) at 0 and 128, O at 256 and 384
    static constexpr int kSmem = kSmall + kStages * kStageBytes + kQBytes;
    static constexpr int kBars = 2 * kStages + 2 + 8;
    static_assert(kStages >= 4 && kSmem <= 227 * 1024, "shared memory");
    static_assert((kBars + 1 + kThreads / 32 + 2) * 8 <= kSmall, "barriers and sums");
};

struct AttnArgs {
    CUtensorMap k_map, v_map;   // [layers * pages * n_kv * page][dim], box {64, min(page, 128)}
    CUtensorMap qp_map, qs_map; // [seqs][n_q][dim], box {64, share, spb} and {64, share, 1}
    void *out;
    const int32_t *prefix_table, *prefix_len, *table, *len;
    int64_t prefix_width, width, n_pages;
    int n_groups, n_seq, n_q, n_kv, share;
    int spb, row_blocks;  // sequences of a row block of a prefix, row blocks
    int page_shift;
    int own0, own1;       // the launch's owners
    int row0;             // the layer's first row / (n_kv * page): layer * n_pages
    float scale_log2;     // scale * log2(e)
    // scratch
    int2 *p_item, *s_item; // items' records: the first one, how many (of items with keys)
    float *p_out, *s_out;  // records' outputs: prefix [rec][NCAP or 128][dim], own [rec][share][dim]
    float2 *p_ml, *s_ml;   // their (reference - kLift, sum), a row each; sum 0: nothing
    int grid;
    unsigned long long *err;
    int stall;  // test hook (q2_0_test_stall_attention): > 0: copies of K end stall - 1 tiles' units into a block's share
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

// T units in shares over G blocks, none smaller than a tile, so that a tile run's segments
// are those of consecutive blocks. An item of nt tiles has kItemCost + nt * kTileCost units;
// a tile belongs to the block that its first unit falls to.
__device__ __forceinline__ int sharers(long long T, int grid) {
    return int(T / kTileCost < grid ? T / kTileCost : grid);
}
__device__ __forceinline__ long long share_begin(long long c, long long T, int G) { return T * c / G; }
// the block that unit t belongs to
__device__ __forceinline__ int share_owner(long long t, long long T, int G) {
    return int(((t + 1) * G + T - 1) / T) - 1;
}
// (a length may come within kTile of 2^31)
__device__ __forceinline__ int tiles_of(int len) { return int((uint32_t(len) + kTile - 1) / kTile); }
__device__ __forceinline__ long long item_units(int nt) {
    return nt ? kItemCost + (long long)nt * kTileCost : 0;
}

// A block's run of tiles of one item.
struct Segment {
    int owner, item;   // item of the owner: head (own tokens) or head * row_blocks + row block
    int head, block;
    int t0, n;         // its tiles
    int len;           // the owner's keys
    int rows, N;       // query rows, and the product's N
    long long at;      // the item's first unit
};

// Goes over a block's segments; every role does so by itself.
struct Walk {
    int owner, len, nt;
    int item, head, block, unit;  // place: unit of the item
    long long at, end;            // unit of all, the end of the block's share
    __device__ __forceinline__ void start(const AttnArgs &a, int o, long long off) {
        owner = o;
        len = owner_len(a, o);
        nt = tiles_of(len);
        const long long units = item_units(nt);
        item = int(off / units);
        unit = int(off - item * units);
        head = o < a.n_groups ? item / a.row_blocks : item;
        block = o < a.n_groups ? item - head * a.row_blocks : 0;
    }
    __device__ __forceinline__ bool next(const AttnArgs &a, Segment &s) {
        while (at < end) {
            while (nt == 0) {  // terminates: units lie ahead
                ++owner;
                item = head = block = unit = 0;
                len = owner_len(a, owner);
                nt = tiles_of(len);
            }
            const int units = int(item_units(nt));
            const int n = int(end - at < units - unit ? end - at : units - unit);
            s.at = at - unit;
            at += n;
            const bool pre = owner < a.n_groups;
            // tiles whose first unit lies in [unit, unit + n)
            s.t0 = unit <= kItemCost ? 0 : (unit - kItemCost + kTileCost - 1) / kTileCost;
            const int t1 = unit + n <= kItemCost ? 0 : (unit + n - kItemCost + kTileCost - 1) / kTileCost;
            s.n = t1 - s.t0;
            s.owner = owner;
            s.len = len;
            s.item = item;
            s.head = head;
            s.block = block;
            const int seqs = a.n_seq - block * a.spb;
            s.rows = pre ? (seqs < a.spb ? seqs : a.spb) * a.share : a.share;
            s.N = s.rows <= 16 ? 16 : (s.rows + 31) & ~31;
            unit += n;
            if (unit == units) {
                unit = 0;
                ++item;
                if (!pre || ++block == a.row_blocks) {
                    block = 0;
                    if (++head == a.n_kv) nt = 0;
                }
            }
            if (s.n) return true;
        }
        return false;
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

__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
// Two f32 operations in one instruction.
union Pair {
    float2 f;
    unsigned long long u;
};
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    Pair p{x}, q{y}, r{z}, d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.u) : "l"(p.u), "l"(q.u), "l"(r.u));
    return d.f;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    Pair p{x}, q{y}, d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(p.u), "l"(q.u));
    return d.f;
}

// Over the lanes of the warp, for W = 32 or 16 values each: lane l gets the maximum
// (sum) of value l % W.
template <int W, bool kMax>
__device__ __forceinline__ float across(float *v) {
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
// The same for a row of W = 16, 32 or 64 values, into dst[0, W).
template <int W, bool kMax>
__device__ __forceinline__ void across_to(float (&v)[W], float *dst) {
    const int lane = threadIdx.x & 31;
    if constexpr (W == 16) {
        const float t = across<16, kMax>(v);
        if (lane < 16) dst[lane] = t;
    } else {
#pragma unroll
        for (int c = 0; c < W; c += 32) dst[c + lane] = across<32, kMax>(v + c);
    }
}

// W = 16, 32 or 64 columns of the warp's lanes of tensor memory.
template <int W>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[W]) {
    uint32_t r[W];
    if constexpr (W == 16) {
        tmem_ld16(addr, r);
    } else {
#pragma unroll
        for (int c = 0; c < W; c += 32) tmem_ld32_issue(addr + c, r + c);
    }
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = __uint_as_float(r[i]);
}
template <int W>
__device__ __forceinline__ void tmem_store(uint32_t addr, const float (&v)[W]) {
    constexpr int P = W < 32 ? W : 32;
#pragma unroll
    for (int c = 0; c < W; c += P) {
        uint32_t r[P];
#pragma unroll
        for (int i = 0; i < P; ++i) r[i] = __float_as_uint(v[c + i]);
        if constexpr (P == 32)
            tmem_st32(addr + c, r);
        else
            tmem_st16(addr + c, r);
    }
    tmem_wait_st();
}

// Barriers of a softmax group.
__device__ __forceinline__ void group_sync(int w) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + 2 * w) : "memory");
}
__device__ __forceinline__ bool group_any(int w, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(v)), "r"(2 + 2 * w)
        : "memory");
    return r != 0;
}

// f(W) with the number of columns as a constant: 16, 32 or 64.
template <int COLS, typename F>
__device__ __forceinline__ void with_columns(int cols, F f) {
    if (cols == 16) {
        f(std::integral_constant<int, 16>{});
    } else if (COLS == 32 || cols == 32) {
        f(std::integral_constant<int, 32>{});
    } else {
        if constexpr (COLS == 64) f(std::integral_constant<int, 64>{});
    }
}

// From a stage of a ring of kN to the next.
template <int kN>
__device__ __forceinline__ void next_stage(int &st, uint32_t &ph) {
    if (++st == kN) {
        st = 0;
        ph ^= 1u;
    }
}

// Deals the launch's tiles: the block's share [begin, end) of all T units, over G blocks,
// and the owner in which it begins. Each thread sums a run of owners. All threads; sum_s
// holds kThreads / 32 + 1; the last one (the place in the owner) and *first_s are there
// after the block's next barrier.
struct Deal {
    long long T, begin, end;
    int G;
};
__device__ __forceinline__ Deal deal(const AttnArgs &a, long long *sum_s, int *first_s) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int owners = a.own1 - a.own0;
    const int per = (owners + kThreads - 1) / kThreads;
    const int o0 = a.own0 + min(tid * per, owners), o1 = min(o0 + per, a.own1);
    long long mine = 0;
    for (int o = o0; o < o1; ++o)
        mine += item_units(tiles_of(owner_len(a, o, blockIdx.x == 0))) * owner_items(a, o);
    long long scan = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += v;
    }
    if (lane == 31) sum_s[warp] = scan;
    __syncthreads();
    long long before = scan - mine, T = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const long long v = sum_s[w];
        if (w < warp) before += v;
        T += v;
    }
    const int G = sharers(T, gridDim.x);
    const bool has = int(blockIdx.x) < G;
    const long long begin = has ? share_begin(blockIdx.x, T, G) : T;
    const long long end = has ? share_begin(blockIdx.x + 1, T, G) : T;
    if (begin < end && begin >= before && begin < before + mine) {
        long long at = before;
        for (int o = o0; o < o1; ++o) {
            const long long n =
                o1 - o0 == 1 ? mine : item_units(tiles_of(owner_len(a, o))) * owner_items(a, o);
            if (begin >= at && begin < at + n) {
                *first_s = o;
                sum_s[kThreads / 32] = begin - at;
            }
            at += n;
        }
    }
    return {T, begin, end, G};
}

// The warp's copies of K or V of the block's tiles, into their ring. K and V have a
// warp each: with short pages the issue of a tile's copies takes
// longer than they do.
template <int D>
__device__ __forceinline__ void copy_tiles(const AttnArgs &a, Walk walk, const CUtensorMap *map, int stages,
                                           uint8_t *ring, uint64_t *kv_full, uint64_t *kv_empty) {
    constexpr int kHalves = D / 64, kStageBytes = kTile * D * 2;
    const int lane = threadIdx.x & 31;
    Segment s;
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
        // page ids, a lane each, in batches of 32 pages, the next batch ahead of its use
        const int pages = (s.len + page - 1) >> a.page_shift;
        int base = s.t0 * kTile >> a.page_shift;
        auto ids_from = [&](int p) { return p + lane < pages ? row[p + lane] : 0; };
        int ids = ids_from(base), more = ids_from(base + 32);
        auto checked = [&](int id) {
            if (id >= 0 && id < a.n_pages) return id;
            record_error(a.err, Q2_0_DEVERR_BAD_ID, pre ? (long long)a.n_groups * a.n_seq + who : who);
            return 0;
        };
        ids = checked(ids);
        for (int t = s.t0; t < s.t0 + s.n; ++t) {
            const int left = s.len - t * kTile;
            const int n = ((left < kTile ? left : kTile) + box - 1) / box;  // boxes with keys
            // lane l copies box l / kHalves, columns 64 * (l % kHalves)
            const int b = lane / kHalves, half = lane % kHalves;
            const int key = t * kTile + (b < n ? b : 0) * box;
            if ((t * kTile >> a.page_shift) >= base + 32) {  // (a tile's pages lie in one batch)
                base += 32;
                ids = checked(more);
                more = ids_from(base + 32);
            }
            const int id = __shfl_sync(0xffffffffu, ids, (key >> a.page_shift) - base);
            const int at = (((a.row0 + id) * a.n_kv + s.head) << a.page_shift) + (key & (page - 1));
            ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[st], ph ^ 1u, a.err, kTag + 1, true));
            if (!ok) break;
            if (lane == 0)
                mbar_arrive_expect_tx(&kv_full[st], uint32_t(n * kHalves * box_bytes));
            __syncwarp();
            if (b < n)
                tma_load_2d(ring + st * kStageBytes + half * (kTile * 128) + b * box_bytes, map,
                            half * 64, at, &kv_full[st]);
            if (++st == stages) {
                st = 0;
                ph ^= 1u;
            }
        }
    }
    if (!ok)  // let the copies in flight land (bounded)
        for (int k = 0; k < stages; ++k) {
            if (--st < 0) {
                st = stages - 1;
                ph ^= 1u;
            }
            mbar_wait(&kv_full[st], ph, a.err, kTag + 2);
        }
}

// The item whose first tile is this segment's: where its records are, for the join.
__device__ __forceinline__ void note_item(const AttnArgs &a, const Segment &s, const Deal &d) {
    const bool pre = s.owner < a.n_groups;
    const long long i =
        (pre ? (long long)s.owner * a.n_kv * a.row_blocks : (long long)(s.owner - a.n_groups) * a.n_kv) +
        s.item;
    const int last = share_owner(s.at + item_units(tiles_of(s.len)) - kTileCost, d.T, d.G);
    (pre ? a.p_item : a.s_item)[i] =
        make_int2(int((i + blockIdx.x) * 2), (last - int(blockIdx.x) + 1) * 2);
}
// The segment's first record (it has two).
__device__ __forceinline__ int64_t record_of(const AttnArgs &a, const Segment &s) {
    const int64_t i = s.owner < a.n_groups ? int64_t(s.owner) * a.n_kv * a.row_blocks
                                           : int64_t(s.owner - a.n_groups) * a.n_kv;
    return 2 * (i + s.item + blockIdx.x);
}

template <int NCAP, int D, bool BF>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ AttnArgs a) {
    using C = Cfg<NCAP, D>;
    extern __shared__ __align__(1024) uint8_t ring[];  // all of the block's shared memory
    if (smem_addr(ring) & 1023u) {  // the swizzle counts on it; the 1024-byte alignment is asked for above
        if (threadIdx.x == 0) record_error(a.err, Q2_0_DEVERR_TIMEOUT, kTag);
        return;
    }
    uint8_t *q_s = ring + C::kStages * C::kStageBytes;
    uint8_t *p_s = q_s + C::kQBufs * C::kQBytes;
    float *ref_s = reinterpret_cast<float *>(p_s + 2 * C::kPBytes);  // [group's 6 NCAP]
    uint64_t *bars = reinterpret_cast<uint64_t *>(ref_s + C::kRefs);
    uint8_t *v_ring = ring + C::kK * C::kStageBytes;
    uint64_t *k_full = bars, *k_empty = k_full + C::kK;
    uint64_t *v_full = k_empty + C::kK, *v_empty = v_full + C::kV;
    uint64_t *q_full = v_empty + C::kV, *q_empty = q_full + C::kQBufs;
    uint64_t *s_full = q_empty + C::kQBufs, *s_empty = s_full + 2;
    uint64_t *p_full = s_empty + 2, *p_empty = p_full + 2;
    uint64_t *o_full = p_empty + 2;
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(o_full + 2);
    int *first_s = reinterpret_cast<int *>(tmem_ptr + 1);  // the block's first owner
    long long *sum_s = reinterpret_cast<long long *>(o_full + 2 + 1);  // [warps], the place in the owner

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2 * C::kStages; ++i) mbar_init(&k_full[i], 1);  // the four rings of barriers
        for (int i = 0; i < C::kQBufs; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 4);
            mbar_init(&p_full[i], 4);
            mbar_init(&p_empty[i], 1);
            mbar_init(&o_full[i], 1);
        }
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
    // Behind attn_rows_kernel (own0 > 0) this launch begins when all blocks of that one have seen
    // the call's inputs complete, runs beside its last blocks, and waits for it before it ends.
    if (a.own0 == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    const Deal dealt = deal(a, sum_s, first_s);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_ptr;

    Walk walk;
    walk.at = dealt.begin;
    walk.end = dealt.end;
    if (walk.at < walk.end) walk.start(a, *first_s, sum_s[kThreads / 32]);
    Segment s;
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsFew));
    if (warp == 0 || warp == 2) {
        // ------------------------- K (warp 0) and V (warp 2) copies -------------------------
        if (warp == 0 && a.stall) walk.end = min(walk.end, walk.at + (a.stall - 1) * kTileCost);
        copy_tiles<D>(a, walk, warp ? &a.v_map : &a.k_map, warp ? C::kV : C::kK, warp ? v_ring : ring,
                      warp ? v_full : k_full, warp ? v_empty : k_empty);
    } else if (warp == 1) {
        // ----------------------- Q copies and the first products -----------------------
        const bool leader = elect_one();
        int st = 0, seg = 0;
        uint32_t ph = 0;
        int n = 0;  // tiles so far
        int loads = 0;  // of Q so far
        bool ok = true;
        // the segment's Q, into buffer seg % kQBufs
        auto load_q = [&](const Segment &q, int i) {
            const int qb = i % C::kQBufs, use = i / C::kQBufs;
            if (use > 0 && !__all_sync(0xffffffffu, mbar_wait_spin(&q_empty[qb], uint32_t(use - 1) & 1u,
                                                                   a.err, kTag + 3)))
                return false;
            if (leader) {
                const bool pre = q.owner < a.n_groups;
                const int rows = (pre ? a.spb : 1) * a.share;  // of the box
                const int seq = pre ? q.owner * a.n_seq + q.block * a.spb : q.owner - a.n_groups;
                mbar_arrive_expect_tx(&q_full[qb], uint32_t(rows * D * 2));
                for (int h = 0; h < C::kHalves; ++h)
                    tma_load_3d(q_s + qb * C::kQBytes + h * (NCAP * 128), pre ? &a.qp_map : &a.qs_map,
                                h * 64, q.head * a.share, seq, &q_full[qb]);
            }
            ++loads;
            __syncwarp();
            return true;
        };
        Segment ahead;
        bool more = walk.next(a, ahead);
        if (more) ok = load_q(ahead, 0);
        for (; ok && more; ++seg) {
            s = ahead;
            more = walk.next(a, ahead);
            if (C::kQBufs == 2 && more && !(ok = load_q(ahead, seg + 1))) break;
            const int qb = seg % C::kQBufs;
            ok = __all_sync(0xffffffffu, mbar_wait_spin(&q_full[qb], uint32_t(seg / C::kQBufs) & 1u, a.err,
                                                        kTag + 6));
            const uint32_t idesc = (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) |
                                   (uint32_t(s.N >> 3) << 17) | (uint32_t(kTile >> 4) << 24);
            const uint64_t qa = sw128_desc(smem_addr(q_s + qb * C::kQBytes));
            for (int i = 0; ok && i < s.n; ++i, ++n) {
                const int sb = n & 1;
                const uint32_t use = uint32_t(n >> 1);
                bool got = use == 0 || mbar_wait_spin(&s_empty[sb], (use - 1) & 1u, a.err, kTag + 8);
                got = got && mbar_wait_spin(&k_full[st], ph, a.err, kTag + 7);
                ok = __all_sync(0xffffffffu, got);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint64_t ka = sw128_desc(smem_addr(ring + st * C::kStageBytes));
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        tc_mma_f16_ss(tmem + sb * NCAP, ka + (ks / 4) * (kTile * 8) + (ks % 4) * 2,
                                      qa + (ks / 4) * (NCAP * 8) + (ks % 4) * 2, idesc, ks > 0);
                    tc_commit(&s_full[sb]);
                    tc_commit(&k_empty[st]);
                    if (i == s.n - 1) tc_commit(&q_empty[qb]);
                }
                __syncwarp();
                next_stage<C::kK>(st, ph);
            }
            if (C::kQBufs == 1 && ok && more) ok = load_q(ahead, seg + 1);
        }
        if (!ok)  // let the copies in flight land (bounded)
            for (int i = max(0, loads - C::kQBufs); i < loads; ++i)
                mbar_wait(&q_full[i % C::kQBufs], uint32_t(i / C::kQBufs) & 1u, a.err, kTag + 2);
    } else if (warp == 3) {
        // ------------------------------- the second products -------------------------------
        const bool leader = elect_one();
        int st = 0;
        uint32_t ph = 0;
        int n = 0;  // tiles so far
        bool ok = true;
        while (ok && walk.next(a, s)) {
            // A = V^T: MN-major; dim 64 reads its one half twice (lanes 64.. are not used)
            const uint32_t idesc = (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | (1u << 15) | (1u << 16) |
                                   (uint32_t(s.N >> 3) << 17) | (uint32_t(kTile >> 4) << 24);
            if (s.t0 == 0 && leader) note_item(a, s, dealt);
            for (int i = 0; i < s.n; ++i, ++n) {
                const int pb = n & 1;
                const int keys = s.len - (s.t0 + i) * kTile;
                const bool got = mbar_wait_spin(&v_full[st], ph, a.err, kTag + 4) &&
                                 mbar_wait_spin(&p_full[pb], uint32_t(n >> 1) & 1u, a.err, kTag + 5);
                ok = __all_sync(0xffffffffu, got);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint64_t va = smem_desc(smem_addr(v_ring + st * C::kStageBytes),
                                                  C::kHalves == 2 ? kTile * 128 : 0, 1024, 2);
                    const uint64_t pa = smem_desc(smem_addr(p_s + pb * C::kPBytes), 128, kTile * 16, 0);
                    const uint32_t o = tmem + C::kOCol + pb * NCAP;
                    const bool add = i >= 2;  // not its output's first
                    // (descriptor addresses count 16 bytes: 16 keys are 2048 bytes of V and 256 of P)
                    if (keys > kTile - 16) {
#pragma unroll
                        for (int ks = 0; ks < kTile / 16; ++ks)
                            tc_mma_f16_ss(o, va + ks * 128, pa + ks * 16, idesc, add || ks > 0);
                    } else {
                        for (int ks = 0; ks < (keys + 15) / 16; ++ks)
                            tc_mma_f16_ss(o, va + ks * 128, pa + ks * 16, idesc, add || ks > 0);
                    }
                    tc_commit(&p_empty[pb]);
                    tc_commit(&v_empty[st]);
                    if (i >= s.n - 2) tc_commit(&o_full[pb]);
                }
                __syncwarp();
                next_stage<C::kV>(st, ph);
            }
        }
        // the products in flight end before tensor memory is freed: the softmax warps' wait for this
        // one runs out after them
        if (!ok && leader) tc_commit(&o_full[0]);
    } else if (warp >= 4) {
        // ---------------------------------- softmax ----------------------------------
        // Thread = key `key` of the tile, or element `key` of the head in the output.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsMany));
        const int w = warp >= 8;  // group
        const int quarter = warp & 3;
        const int key = quarter * 32 + lane;
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        const float2 scale = make_float2(a.scale_log2, a.scale_log2);
        // A reference is a rounded product of a score and the scale. A score scaled and reduced by it in one
        // fused operation is off it by that rounding, half a unit at most up to kFused; beyond (finite, if
        // absurd, scores) the largest weights could overflow or vanish, so that every tile goes the way
        // of a raise, where the products are rounded by themselves as the reference is.
        bool far = false;
        // of the group's rows: kLift - ref, the factors of a raise, and the four warps' [4][NCAP] to be
        // reduced. (The factors have floats of their own: after a raise in a segment's last tile no
        // barrier lies between a warp that still reads them and one that writes its sums to red_s.)
        float *nref_s = ref_s + w * 6 * NCAP;
        float *alpha_s = nref_s + NCAP;
        float *red_s = alpha_s + NCAP;
        const uint32_t o_col = tmem + lanes + C::kOCol + w * NCAP;
        float2 l[NCAP / 2];
        int n = 0;         // tiles so far
        int segs = 0;      // the group's segments so far
        int st = 0;        // the stage of the tile's V
        uint32_t ph = 0;
        // A warp whose wait timed out waits no more: it goes through the motions, so that
        // the barriers of the softmax warps stay matched, and its results mean nothing.
        bool dead = false;
        auto wait = [&](uint64_t *bar, int use, int tag) {
            if (!dead)
                dead = !__all_sync(0xffffffffu, mbar_wait_spin(bar, uint32_t(use) & 1u, a.err, tag));
        };
        // The output of a segment is read when the group's next weights are ready (or at the end): by
        // then its products are done. With 64 columns there are no registers for that.
        constexpr bool kDefer = NCAP == 32;
        float *o_out = nullptr;
        int o_rows = 0, o_cols = 0;
        auto flush = [&]() {
            if (!o_out) return;
            wait(&o_full[w], segs++, kTag + 13);
            tc_fence_after();
            if (quarter * 32 < D)
                with_columns<NCAP>(o_cols, [&](auto columns) {
                    constexpr int W = columns;
                    float v[W];
                    tmem_load<W>(o_col, v);
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        if (j < o_rows) o_out[j * D + key] = v[j];
                });
            tc_fence_before();
            o_out = nullptr;
        };
        while (walk.next(a, s)) {
            bool fresh = true;  // no tile of this segment yet
            for (int i = 0; i < s.n; ++i, ++n) {
                const int v_st = st;
                const uint32_t v_ph = ph;
                next_stage<C::kV>(st, ph);
                if ((n & 1) != w) continue;
                // (the group's buffers of scores, weights and outputs are number w)
                const int keys = s.len - (s.t0 + i) * kTile;  // valid ones of this tile, if < 128
                wait(&s_full[w], n >> 1, kTag + 9);
                tc_fence_after();
                with_columns<NCAP>(s.N, [&](auto columns) {
                    constexpr int W = columns;
                    const bool in = key < keys;
                    const uint32_t sa = tmem + lanes + w * NCAP;
                    float v[W];
                    auto exponents = [&](auto fused) {
                        auto scaled = [&](float2 x, float2 r) {
                            return fused ? fma2(x, scale, r) : add2(fma2(x, scale, make_float2(0.0f, 0.0f)), r);
                        };
#pragma unroll
                        for (int j = 0; j < W; j += 4) {
                            const float4 r = *reinterpret_cast<const float4 *>(nref_s + j);
                            *reinterpret_cast<float2 *>(v + j) =
                                scaled(make_float2(v[j], v[j + 1]), make_float2(r.x, r.y));
                            *reinterpret_cast<float2 *>(v + j + 2) =
                                scaled(make_float2(v[j + 2], v[j + 3]), make_float2(r.z, r.w));
                        }
                        if (keys < kTile) {
#pragma unroll
                            for (int j = 0; j < W; ++j) v[j] = in ? v[j] : -INFINITY;
                        }
                    };
                    tmem_load<W>(sa, v);
                    bool raise = fresh;
                    if (!raise) {
                        exponents(std::true_type{});
                        float most = v[0];
#pragma unroll
                        for (int j = 1; j < W - 1; j += 2) most = max3(most, v[j], v[j + 1]);
                        raise = group_any(w, far || fmaxf(most, v[W - 1]) > kSlack + kLift);
                        if (raise) tmem_load<W>(sa, v);
                    }
                    if (raise) {
                        // the rows' maxima over the tile, and with them new references
#pragma unroll
                        for (int j = 0; j < W; ++j) v[j] = in ? v[j] * scale.x : -INFINITY;
                        across_to<W, true>(v, red_s + quarter * NCAP);
                        group_sync(w);
                        bool beyond = false;
                        if (key < W) {
                            const float m = fmaxf(fmaxf(red_s[key], red_s[NCAP + key]),
                                                  fmaxf(red_s[2 * NCAP + key], red_s[3 * NCAP + key]));
                            const float old = fresh ? INFINITY : nref_s[key];
                            // no key counts (scores of -inf): any finite reference does
                            const float now = fminf(kLift - fmaxf(m, -FLT_MAX), old);
                            alpha_s[key] = ex2(now - old);
                            nref_s[key] = now;
                            beyond = fabsf(now) > kFused;
                        }
                        far = group_any(w, beyond);
                        if (fresh) {
#pragma unroll
                            for (int j = 0; j < NCAP / 2; ++j) l[j] = make_float2(0.0f, 0.0f);
                        } else {
                            // the products into this output so far are done
                            wait(&p_empty[w], (n >> 1) - 1, kTag + 14);
                            tc_fence_after();
                            tmem_load<W>(o_col, v);
#pragma unroll
                            for (int j = 0; j < W; j += 2) {
                                const float2 f = *reinterpret_cast<const float2 *>(alpha_s + j);
                                v[j] *= f.x;
                                v[j + 1] *= f.y;
                                l[j / 2].x *= f.x;
                                l[j / 2].y *= f.y;
                            }
                            tmem_store<W>(o_col, v);
                        }
                        tmem_load<W>(sa, v);
                        exponents(std::false_type{});
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_empty[w]);
                    if (kDefer && fresh) flush();
                    if (n >= 2) wait(&p_empty[w], (n >> 1) - 1, kTag + 10);
                    uint8_t *ps = p_s + w * C::kPBytes + key * 16;
#pragma unroll
                    for (int j = 0; j < W; j += 8) {
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            v[j + e] = ex2(v[j + e]);
                            v[j + e + 1] = ex2(v[j + e + 1]);
                            l[(j + e) / 2] = add2(l[(j + e) / 2], make_float2(v[j + e], v[j + e + 1]));
                        }
                        *reinterpret_cast<uint4 *>(ps + (j / 8) * (kTile * 16)) =
                            make_uint4(pack<BF>(v[j], v[j + 1]), pack<BF>(v[j + 2], v[j + 3]),
                                       pack<BF>(v[j + 4], v[j + 5]), pack<BF>(v[j + 6], v[j + 7]));
                    }
                });
                if (keys < kTile && (keys & 15)) {
                    // places past the last key up to the product's 16: whatever V holds there,
                    // 0 times it has to be 0
                    wait(&v_full[v_st], int(v_ph), kTag + 12);
                    const int n0 = 16 - (keys & 15);
                    for (int x = key; x < n0 * C::kHalves * 8; x += 128) {
                        const int piece = x & 7, r = (x >> 3) / C::kHalves, h = (x >> 3) % C::kHalves;
                        *reinterpret_cast<uint4 *>(v_ring + v_st * C::kStageBytes + h * (kTile * 128) +
                                                   (keys + r) * 128 + piece * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[w]);
                fresh = false;
            }
            // ---- the segment's output, references and sums
            const bool pre = s.owner < a.n_groups;
            const int64_t at = (record_of(a, s) + w) * (pre ? NCAP : a.share);
            float *out = (pre ? a.p_out : a.s_out) + at * D;
            float2 *ml = (pre ? a.p_ml : a.s_ml) + at;
            const int rows = s.rows;
            if (fresh) {  // the other group had the only tile
                if (key < rows) ml[key] = make_float2(-FLT_MAX, 0.0f);
                continue;
            }
            with_columns<NCAP>(s.N, [&](auto columns) {
                constexpr int W = columns;
                float v[W];
#pragma unroll
                for (int j = 0; j < W; j += 2) {
                    v[j] = l[j / 2].x;
                    v[j + 1] = l[j / 2].y;
                }
                across_to<W, false>(v, red_s + quarter * NCAP);
                group_sync(w);
                if (key < rows)
                    ml[key] = make_float2(-nref_s[key],
                                          (red_s[key] + red_s[NCAP + key]) +
                                              (red_s[2 * NCAP + key] + red_s[3 * NCAP + key]));
                group_sync(w);  // nref_s and red_s are free again
            });
            o_out = out;
            o_rows = rows;
            o_cols = s.N;
            if (!kDefer) flush();
        }
        flush();
    }
    if (a.own0) asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Prefixes with more than 64 query rows: see the top of the file. Of a row block of up to 256
// rows, softmax group w has rows 128 w .. 127 + 128 w of every tile where there are more than
// 128 ("both"); otherwise the two groups take turns at the tiles.
// S_w and P_w share 128 columns of tensor memory, so a group's next scores wait for its second
// product; the other group's softmax fills that time, and the weights are handed over in
// halves of 64 keys. (Scores in halves, too, would cost more than they save: a product of N =
// 64 reads as much of Q from shared memory as one of 128, and takes as long.) A product step holds its issuing warp
// about as long as it runs, so that the two kinds have a warp each.
template <int ROWS, int D, bool BF>
__global__ void __launch_bounds__(kThreads, 1) attn_rows_kernel(const __grid_constant__ AttnArgs a) {
    using C = RowsCfg<ROWS, D>;
    extern __shared__ __align__(1024) uint8_t ring[];  // all of the block's shared memory
    if (smem_addr(ring) & 1023u) {  // the swizzle counts on it
        if (threadIdx.x == 0) record_error(a.err, Q2_0_DEVERR_TIMEOUT, kTag);
        return;
    }
    uint8_t *q_s = ring + C::kStages * C::kStageBytes;
    uint8_t *v_ring = ring + C::kK * C::kStageBytes;
    uint64_t *k_full = reinterpret_cast<uint64_t *>(q_s + C::kQBytes), *k_empty = k_full + C::kK;
    uint64_t *v_full = k_empty + C::kK, *v_empty = v_full + C::kV;
    uint64_t *q_full = v_empty + C::kV, *q_empty = q_full + 1;
    uint64_t *s_full = q_empty + 1, *p_full = s_full + 2, *o_done = p_full + 4;  // p_full: 2 w + half
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(o_done + 2);
    int *first_s = reinterpret_cast<int *>(tmem_ptr + 1);
    long long *sum_s = reinterpret_cast<long long *>(o_done + 3);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2 * C::kStages; ++i) mbar_init(&k_full[i], 1);  // the four rings of barriers
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], 4);
            mbar_init(&p_full[2 * i + 1], 4);
            mbar_init(&o_done[i], 1);
        }
        fence_barrier_init();
        prefetch_tensormap(&a.k_map);
        prefetch_tensormap(&a.v_map);
        prefetch_tensormap(&a.qp_map);
    }
    if (warp == 1) {
        tmem_alloc(tmem_ptr, 512);
        tmem_relinquish();
    }
    // rows that no copy fills are zero or an earlier segment's
    for (int i = tid; i < C::kQBytes / 16; i += kThreads)
        reinterpret_cast<uint4 *>(q_s)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Deal dealt = deal(a, sum_s, first_s);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_ptr;
    Walk walk;
    walk.at = dealt.begin;
    walk.end = dealt.end;
    if (walk.at < walk.end) walk.start(a, *first_s, sum_s[kThreads / 32]);
    Segment s;

    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsFew));
    if (warp == 0 || warp == 2) {
        if (warp == 0 && a.stall) walk.end = min(walk.end, walk.at + (a.stall - 1) * kTileCost);
        copy_tiles<D>(a, walk, warp ? &a.v_map : &a.k_map, warp ? C::kV : C::kK, warp ? v_ring : ring,
                      warp ? v_full : k_full, warp ? v_empty : k_empty);
    } else if (warp == 1) {
        // ----------------------- Q copies and the first products -----------------------
        const bool leader = elect_one();
        int st = 0, seg = 0;
        uint32_t ph = 0;
        int count[2] = {0, 0};  // the groups' tiles so far
        int loads = 0;          // of Q so far
        bool ok = true;
        const uint32_t idesc = (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | (uint32_t(kTile >> 3) << 17) |
                               (uint32_t(128 >> 4) << 24);
        for (; ok && walk.next(a, s); ++seg) {
            if (s.t0 == 0 && leader) note_item(a, s, dealt);
            if (seg > 0)
                ok = __all_sync(0xffffffffu, mbar_wait_spin(q_empty, uint32_t(seg - 1) & 1u, a.err, kTag + 3));
            if (!ok) break;
            if (leader) {
                mbar_arrive_expect_tx(q_full, uint32_t(a.spb * a.share * D * 2));
                for (int h = 0; h < C::kHalves; ++h)
                    tma_load_3d(q_s + h * (C::kRows * 128), &a.qp_map, h * 64, s.head * a.share,
                                s.owner * a.n_seq + s.block * a.spb, q_full);
            }
            ++loads;
            __syncwarp();
            ok = __all_sync(0xffffffffu, mbar_wait_spin(q_full, uint32_t(seg) & 1u, a.err, kTag + 6));
            const bool both = ROWS > 128 && s.rows > 128;
            for (int i = 0; ok && i < s.n; ++i) {
                ok = __all_sync(0xffffffffu, mbar_wait_spin(&k_full[st], ph, a.err, kTag + 7));
                const uint64_t ka = sw128_desc(smem_addr(ring + st * C::kStageBytes));
                const int w0 = both ? 0 : i & 1, w1 = both ? 1 : i & 1;
                for (int w = w0; ok && w <= w1; ++w) {
                    // the scores' place held the weights of the group's tile before
                    if (count[w] > 0)
                        ok = __all_sync(0xffffffffu, mbar_wait_spin(&o_done[w], uint32_t(count[w] - 1) & 1u,
                                                                    a.err, kTag + 8));
                    if (!ok) break;
                    ++count[w];
                    tc_fence_after();
                    if (leader) {
                        const uint64_t qa = sw128_desc(smem_addr(q_s + (both ? w : 0) * (128 * 128)));
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
                            tc_mma_f16_ss(tmem + w * 128, qa + (ks / 4) * (C::kRows * 8) + (ks % 4) * 2,
                                          ka + (ks / 4) * (kTile * 8) + (ks % 4) * 2, idesc, ks > 0);
                        tc_commit(&s_full[w]);
                        if (w == w1) tc_commit(&k_empty[st]);
                        if (w == w1 && i == s.n - 1) tc_commit(q_empty);
                    }
                    __syncwarp();
                }
                next_stage<C::kK>(st, ph);
            }
        }
        if (!ok && loads > 0)  // let the copies in flight land (bounded)
            mbar_wait(q_full, uint32_t(loads - 1) & 1u, a.err, kTag + 2);
    } else if (warp == 3) {
        // ------------------------------- the second products -------------------------------
        const bool leader = elect_one();
        int st = 0;
        uint32_t ph = 0;
        int count[2] = {0, 0};
        bool ok = true;
        // B = V: MN-major
        const uint32_t idesc = (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | (1u << 16) |
                               (uint32_t(D >> 3) << 17) | (uint32_t(128 >> 4) << 24);
        while (ok && walk.next(a, s)) {
            const bool both = ROWS > 128 && s.rows > 128;
            for (int i = 0; ok && i < s.n; ++i) {
                const int keys = s.len - (s.t0 + i) * kTile;
                const int steps = keys >= kTile ? kTile / 16 : (keys + 15) / 16;
                const int w0 = both ? 0 : i & 1, w1 = both ? 1 : i & 1;
                ok = __all_sync(0xffffffffu, mbar_wait_spin(&v_full[st], ph, a.err, kTag + 4));
                const uint64_t va = smem_desc(smem_addr(v_ring + st * C::kStageBytes),
                                              C::kHalves == 2 ? kTile * 128 : 0, 1024, 2);
                const bool add = i >= (both ? 1 : 2);  // not the output's first
                for (int w = w0; ok && w <= w1; ++w) {
                    for (int hf = 0; ok && hf < 2; ++hf) {
                        ok = __all_sync(0xffffffffu, mbar_wait_spin(&p_full[2 * w + hf], uint32_t(count[w]) & 1u,
                                                                    a.err, kTag + 5));
                        if (!ok) break;
                        tc_fence_after();
                        if (leader) {
                            // (16 keys are 8 columns of P, and 2048 bytes of V: 128 units of the address)
                            for (int ks = 4 * hf; ks < min(4 * hf + 4, steps); ++ks)
                                tc_mma_f16_ta(tmem + C::kOCol + w * 128, tmem + w * 128 + ks * 8, va + ks * 128,
                                              idesc, add || ks > 0);
                            if (hf) tc_commit(&o_done[w]);
                            if (hf && w == w1) tc_commit(&v_empty[st]);
                        }
                        __syncwarp();
                    }
                    ++count[w];
                }
                next_stage<C::kV>(st, ph);
            }
        }
        // the products in flight end before tensor memory is freed: the softmax warps' wait for this
        // one runs out after them
        if (!ok && leader) tc_commit(&o_done[0]);
    } else if (warp >= 4) {
        // ---------------------------------- softmax: thread = row ----------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsMany));
        const int w = warp >= 8;  // group
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        const uint32_t s_col = tmem + lanes + w * 128, o_col = tmem + lanes + C::kOCol + w * 128;
        const float2 scale = make_float2(a.scale_log2, a.scale_log2);
        int done = 0;  // the group's tiles so far
        int st = 0;    // the stage of the tile's V
        uint32_t ph = 0;
        bool dead = false;  // as in attn_kernel
        auto wait = [&](uint64_t *bar, int use, int tag) {
            if (!dead)
                dead = !__all_sync(0xffffffffu, mbar_wait_spin(bar, uint32_t(use) & 1u, a.err, tag));
        };
        while (walk.next(a, s)) {
            const bool both = ROWS > 128 && s.rows > 128;
            float nref = 0.0f, l = 0.0f;  // kLift - ref, sum
            bool fresh = true;
            for (int i = 0; i < s.n; ++i) {
                const int v_st = st;
                const uint32_t v_ph = ph;
                next_stage<C::kV>(st, ph);
                if (!both && (i & 1) != w) continue;
                const int keys = s.len - (s.t0 + i) * kTile;  // valid ones of this tile, if < 128
                wait(&s_full[w], done, kTag + 9);
                tc_fence_after();
                float v[kTile];
                {
                    uint32_t r[kTile];
#pragma unroll
                    for (int c = 0; c < kTile; c += 32) tmem_ld32_issue(s_col + c, r + c);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < kTile; j += 2)
                        *reinterpret_cast<float2 *>(v + j) =
                            fma2(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), scale,
                                 make_float2(0.0f, 0.0f));
                }
                if (keys < kTile) {
#pragma unroll
                    for (int j = 0; j < kTile; ++j) v[j] = j < keys ? v[j] : -INFINITY;
                }
                float most[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    most[e] = v[e];
#pragma unroll
                    for (int j = 4; j < kTile - 4; j += 8) most[e] = max3(most[e], v[j + e], v[j + 4 + e]);
                    most[e] = fmaxf(most[e], v[kTile - 4 + e]);
                }
                most[0] = fmaxf(max3(most[0], most[1], most[2]), most[3]);
                const bool raise = fresh || most[0] + nref > kSlack + kLift;
                if (__any_sync(0xffffffffu, raise)) {
                    // no key counts (scores of -inf): any finite reference does
                    const float now = kLift - fmaxf(most[0], -FLT_MAX);
                    const float next = fresh ? now : raise ? fminf(now, nref) : nref;
                    const float f = fresh ? 0.0f : ex2(next - nref);
                    nref = next;
                    l *= f;
                    if (!fresh) {  // the products into this output so far are done
                        wait(&o_done[w], done - 1, kTag + 14);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            float o[16];
                            tmem_load<16>(o_col + c, o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] *= f;
                            tmem_store<16>(o_col + c, o);
                        }
                    }
                }
                if (keys < kTile && (keys & 15) && (!both || w == 0)) {
                    // places past the last key up to the product's 16: whatever V holds there,
                    // 0 times it has to be 0
                    wait(&v_full[v_st], int(v_ph), kTag + 12);
                    const int n0 = 16 - (keys & 15);
                    for (int x = row; x < n0 * C::kHalves * 8; x += 128) {
                        const int piece = x & 7, r = (x >> 3) / C::kHalves, h = (x >> 3) % C::kHalves;
                        *reinterpret_cast<uint4 *>(v_ring + v_st * C::kStageBytes + h * (kTile * 128) +
                                                   (keys + r) * 128 + piece * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                const float2 off = make_float2(nref, nref);
#pragma unroll
                for (int c = 0; c < kTile; c += 64) {
                    uint32_t p[32];
#pragma unroll
                    for (int j = 0; j < 64; j += 2) {
                        float2 e = add2(make_float2(v[c + j], v[c + j + 1]), off);
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        sum[j / 2 & 1] = add2(sum[j / 2 & 1], e);
                        p[j / 2] = pack<BF>(e.x, e.y);
                    }
                    tmem_st32(s_col + c / 2, p);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * w + c / 64]);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                fresh = false;
                ++done;
            }
            // ---- the segment's output, reference and sum
            const int rows = both ? s.rows - 128 * w : s.rows;  // of the group
            const int64_t at = (record_of(a, s) + w) * 128 + row;
            if (row < rows) a.p_ml[at] = fresh ? make_float2(-FLT_MAX, 0.0f) : make_float2(-nref, l);
            if (fresh) continue;
            wait(&o_done[w], done - 1, kTag + 13);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_load<32>(o_col + c, o);
                if (row < rows) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8)  // whole sectors: lanes' rows lie apart
                        asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(
                                         a.p_out + at * D + c + j),
                                     "f"(o[j]), "f"(o[j + 1]), "f"(o[j + 2]), "f"(o[j + 3]), "f"(o[j + 4]),
                                     "f"(o[j + 5]), "f"(o[j + 6]), "f"(o[j + 7])
                                     : "memory");
                }
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the records of each query row: `split` warps of a block to a row, each with every
// split-th record; their sums meet in shared memory.
template <int D, bool BF>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnArgs a, int ncap,
                                                        int split, int by_rows) {
    constexpr int E = D / 32;  // elements per lane
    __shared__ float s_m[8], s_l[8];
    __shared__ float s_o[8][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % split;
    const int row = int(blockIdx.x) * (8 / split) + warp / split;  // sequence * n_q + head
    const bool live = row < a.n_groups * a.n_seq * a.n_q;
    const int b = live ? row / a.n_q : 0, h = row - b * a.n_q;
    const int head = h / a.share, r = h - head * a.share;
    const int group = b / a.n_seq, in_group = b - group * a.n_seq;
    const int block = a.prefix_width ? in_group / a.spb : 0;
    const int pr = (in_group - block * a.spb) * a.share + r;  // row in the prefix's item
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float acc[E], l = 0.0f, m = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    if (live) {
        const int plen = owner_len(a, group), slen = owner_len(a, a.n_groups + b);
        int2 pi = make_int2(0, 0), si = make_int2(0, 0);
        if (plen) pi = __ldcg(a.p_item + (int64_t(group) * a.n_kv + head) * a.row_blocks + block);
        if (slen) si = __ldcg(a.s_item + int64_t(b) * a.n_kv + head);
        // of a prefix block of more than 128 rows, a segment's two records are those of different rows
        const int seqs = min(a.spb, a.n_seq - block * a.spb);
        const bool both = by_rows && seqs * a.share > 128;
        const int pstep = both ? 2 : 1, prow = both ? pr & 127 : pr;
        if (both) {
            pi.x += pr >> 7;
            pi.y >>= 1;
        }
        const int np = pi.y, n = np + si.y;
        // 32 records at a time: lane i has the i-th's reference and sum
        for (int i0 = part; i0 < n; i0 += 32 * split) {
            const int i = i0 + lane * split;
            float2 ml = make_float2(-INFINITY, 0.0f);
            const float *o = nullptr;
            if (i < n) {
                const int64_t x = i < np ? (int64_t(pi.x) + i * pstep) * ncap + prow
                                         : (int64_t(si.x) + i - np) * a.share + r;
                ml = __ldcg((i < np ? a.p_ml : a.s_ml) + x);
                o = (i < np ? a.p_out : a.s_out) + x * D;
            }
            float top = ml.x;
#pragma unroll
            for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            top = fmaxf(top, m);
            const float keep = ex2(m - top), mine = ml.y != 0.0f ? ex2(ml.x - top) : 0.0f;
            m = top;
            float sum = mine * ml.y;
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            l = l * keep + sum;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= keep;
            // a record without a sum has no output either
            const unsigned long long ptr = reinterpret_cast<unsigned long long>(ml.y != 0.0f ? o : nullptr);
            const int count = min(32, (n - i0 + split - 1) / split);
            for (int j0 = 0; j0 < count; j0 += 8) {  // eight loads in flight
                float f[8], q[8][E];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    f[j] = __shfl_sync(0xffffffffu, mine, j0 + j);
                    const float *oj =
                        reinterpret_cast<const float *>(__shfl_sync(0xffffffffu, ptr, j0 + j));
#pragma unroll
                    for (int e = 0; e < E; ++e) q[j][e] = 0.0f;
                    if (oj) {
                        if constexpr (E == 4)
                            *reinterpret_cast<float4 *>(q[j]) =
                                __ldcg(reinterpret_cast<const float4 *>(oj) + lane);
                        else
                            *reinterpret_cast<float2 *>(q[j]) =
                                __ldcg(reinterpret_cast<const float2 *>(oj) + lane);
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += f[j] * q[j][e];
            }
        }
    }
    if (split > 1) {
        if (lane == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
        __syncthreads();
        if (part) return;
        for (int j = 1; j < split; ++j) m = fmaxf(m, s_m[warp + j]);
        const float m0 = m == -INFINITY ? 0.0f : m;
        l = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
        for (int j = 0; j < split; ++j) {
            const float f = ex2(s_m[warp + j] - m0);
            l += f * s_l[warp + j];
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += f * s_o[warp + j][lane * E + e];
        }
    }
    if (!live) return;
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // (NaN stays NaN)
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + int64_t(row) * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack<BF>(acc[e] * inv, acc[e + 1] * inv);
}

}  // namespace
}  // namespace q2

struct q2_0_attn_plan {
    q2::AttnArgs args;
    int ncap, dim, n_layers;
    int by_rows;  // prefixes by attn_rows_kernel with so many rows at a time, or 0
    bool bf;
    int64_t n_pages;
    void *scratch;
};

namespace q2 {

namespace {

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Test hook (q2_0_test_stall_attention): 1 + the tiles of the next execute's stall on a device, or 0.
std::atomic<int> g_stall[64];

int take_stall() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || g_stall[dev] == 0) return 0;
    return g_stall[dev].exchange(0);
}

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
    return ncap == 32 ? variant_n<32>(dim, bf) : variant_n<64>(dim, bf);
}
template <int ROWS, int D, bool BF>
Variant rows_variant() {
    return {attn_rows_kernel<ROWS, D, BF>, RowsCfg<ROWS, D>::kSmem};
}
template <int ROWS>
Variant rows_variant_n(int dim, bool bf) {
    if (dim == 64) return bf ? rows_variant<ROWS, 64, true>() : rows_variant<ROWS, 64, false>();
    return bf ? rows_variant<ROWS, 128, true>() : rows_variant<ROWS, 128, false>();
}
Variant rows_variant_of(int rows, int dim, bool bf) {
    return rows == 128 ? rows_variant_n<128>(dim, bf) : rows_variant_n<256>(dim, bf);
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
    a.row0 = 0;
    a.scale_log2 = d.scale * 1.44269504f;
    a.grid = sms;
    a.err = err;
    a.stall = 0;
    // More than 64 rows to a prefix: 128 or 256 at a time by attn_rows_kernel. Lengths are not known here,
    // so that rows alone decide. Measured with 8 kv heads of 128 on 4099 and on 50021 keys (us), blocks of 64
    // rows by attn_kernel against attn_rows_kernel: 48 rows 19 and 54 against 25 and 58, 64 rows 20 and 55
    // against 26 and 59, 96 rows 23 and 76 against 30 and 63, 128 rows 26 and 65 against 32 and 65; heads of
    // 64: 64 rows 19 and 45 against 23 and 47, 96 rows 22 and 60 against 25 and 50, 128 rows 25 and 61 against 25
    // and 51. Above 128 rows, 128 at a time against 256: 160 rows 33 and 96 against 33 and 72, heads of 64 28 and 66
    // against 29 and 65; up to 128 rows the smaller tile is ahead by 0 to 2 %.
    const int64_t rows = d.prefix_width ? d.n_seq * a.share : a.share;
    p->by_rows = !d.prefix_width || rows <= 64 ? 0 : rows <= 128 ? 128 : 256;
    p->ncap = (p->by_rows ? a.share : rows) <= 32 ? 32 : 64;
    a.spb = int(std::min<int64_t>(d.n_seq, (p->by_rows ? p->by_rows : p->ncap) / a.share));
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
    const size_t o_pi = take(size_t(a.n_groups) * a.n_kv * a.row_blocks * 8);
    const size_t o_si = take(size_t(seqs) * a.n_kv * 8);
    const size_t p_rows = 2 * p_slots * (p->by_rows ? 128 : p->ncap), s_rows = 2 * s_slots * a.share;
    const size_t o_p = take(p_rows * c.dim * 4), o_s = take(s_rows * c.dim * 4);
    const size_t o_pml = take(p_rows * 8), o_sml = take(s_rows * 8);
    p->scratch = nullptr;
    if (ok) ok = cudaMalloc(&p->scratch, at) == cudaSuccess;
    // An execute whose waits ran out may leave items without their records' places: the join then
    // finds none or an earlier execute's, never what lay in this memory before.
    if (ok) ok = cudaMemset(p->scratch, 0, o_p) == cudaSuccess && cudaStreamSynchronize(nullptr) == cudaSuccess;
    const Variant v = variant_of(p->ncap, p->dim, p->bf);
    if (ok)
        ok = cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem) ==
             cudaSuccess;
    const Variant vr = rows_variant_of(p->by_rows, p->dim, p->bf);
    if (ok && p->by_rows)
        ok = cudaFuncSetAttribute(vr.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, vr.smem) ==
             cudaSuccess;
    if (!ok) {
        if (p->scratch) cudaFree(p->scratch);
        delete p;
        return Q2_0_ECUDA;
    }
    char *base = static_cast<char *>(p->scratch);
    a.p_item = reinterpret_cast<int2 *>(base + o_pi);
    a.s_item = reinterpret_cast<int2 *>(base + o_si);
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
    a.stall = take_stall();
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
    cudaError_t e;
    const int owners = a.n_groups + a.n_groups * a.n_seq;
    a.own0 = 0;
    a.own1 = owners;
    if (p->by_rows) {
        const Variant vr = rows_variant_of(p->by_rows, p->dim, p->bf);
        a.own1 = a.n_groups;
        cfg.dynamicSmemBytes = size_t(vr.smem);
        e = cudaLaunchKernelEx(&cfg, vr.fn, a);
        if (e != cudaSuccess) return cuda_status(e);
        a.own0 = a.n_groups;
        a.own1 = owners;
    }
    cfg.dynamicSmemBytes = size_t(v.smem);
    e = cudaLaunchKernelEx(&cfg, v.fn, a);
    if (e != cudaSuccess) return cuda_status(e);
    // few rows have many records each: more warps to a row
    const int64_t rows = int64_t(a.n_groups) * a.n_seq * a.n_q;
    const int split = rows <= 2 * a.grid ? 8 : rows <= 4 * a.grid ? 4 : rows <= 8 * a.grid ? 2 : 1;
    cfg.gridDim = dim3(unsigned((rows * split + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    auto *join = p->dim == 64 ? (p->bf ? attn_join_kernel<64, true> : attn_join_kernel<64, false>)
                              : (p->bf ? attn_join_kernel<128, true> : attn_join_kernel<128, false>);
    return cuda_status(cudaLaunchKernelEx(&cfg, join, a, p->by_rows ? 128 : p->ncap, split, p->by_rows > 128));
}

int attn_plan_launches(const q2_0_attn_plan *p) { return p->by_rows ? 3 : 2; }

int attn_plan_layers(const q2_0_attn_plan *p) { return p->n_layers; }

void attn_plan_destroy(q2_0_attn_plan *p) {
    cudaFree(p->scratch);
    delete p;
}

}  // namespace q2

// Test hook: the next execute on the current device stops copying keys about `tiles` tiles into
// each block's share, so that the waits for them run out.
extern "C" int q2_0_test_stall_attention(int tiles) {
    int dev = 0;
    if (tiles < 0 || tiles > (1 << 20)) return Q2_0_EINVAL;
    if (cudaGetDevice(&dev) != cudaSuccess) return q2::reported(Q2_0_ECUDA);
    if (dev < 0 || dev >= 64) return Q2_0_EUNSUPPORTED;
    q2::g_stall[dev] = tiles + 1;
    return Q2_0_OK;
}
