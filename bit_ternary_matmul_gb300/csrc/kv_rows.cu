// The pages of a paged key/value cache: copies, rows that share pages (fork), rows that grow, shrink
// and part (resize), and pages moved to the front (compact).
//
// Counts and tables are a few bytes a page, and what has to be decided about them is a chain: what is given
// back, which pages are then free, which row gets which. (So a page that is given back may be written in the same
// call.) One cluster of blocks goes through the chain, with the cluster's barrier between its steps, so that it is one launch and no block waits for one that may not
// have started. The tokens that move, the bulk of the bytes, are copied by a launch of the whole GPU
// behind it, from a list that the cluster leaves.
//
// Nothing depends on the order of atomics: counts are sums, the lowest row is a minimum, and
// free pages go to rows by their ranks.
#include <algorithm>
#include <mutex>

#include "q2_0_cluster.cuh"
#include "q2_0_internal.h"

namespace q2 {

namespace {

// ---------------------------------------------------------------------------
// Copying pages. What is copied of a page in one layer of keys or values is cut into parts; a warp takes
// a part at a time, and has kPerLane 16-byte vectors a lane on their way. Of pages so short that
// this is more than one layer's, it takes keys and values of a layer at once.
// Bound by memory: 150 pages of 64 tokens in 36 layers (2.83 GB) 425 us, the copy rate's time (423); 30000 pages of 2 KB a
// layer to scattered places (0.98 GB) 160 of a compaction's 170 us, where the rate would give 147: one layer's at a time
// took 205, 4 vectors a lane 212 (and 434 for the long pages). What is done in one turn of all warps is cut into as many
// parts as there are warps: half pages of 24 rows 8 us, in parts of 256 vectors 11.
// ---------------------------------------------------------------------------
constexpr int kPerLane = 8;
constexpr int kPart = 32 * kPerLane;
constexpr int kCopyThreads = 256;
constexpr int kCopyBlocks = 4;  // of an SM (copy_kernel; of move_kernel's, with 76 registers a thread, three are there at once, and
                                // the fourth goes through its share behind them)

struct CopyArgs {
    uint4 *k, *v;
    int64_t n_pages;
    int n_layers, n_kv, page, vec;  // vec: vectors of a token's head
    const int32_t *src, *dst, *count;
    int64_t n;            // copies, or
    const int32_t *n_at;  // where their number is
    bool check;           // ids and counts come from the caller
    unsigned long long *err;
};

// Parts of a page in a layer: of kPart vectors; four times that where each warp takes many; and where all is done
// in about one turn, as many as there are warps for, so that it is one.
__device__ __forceinline__ int parts_of(int page_vec, int64_t items, int64_t warps) {
    const int fine = (page_vec + kPart - 1) / kPart;
    const int64_t all = items * fine;
    if (all > 16 * warps) return (fine + 3) / 4;
    if (all > 2 * warps) return fine;
    return int(max(int64_t(1), min(int64_t(fine), warps / items)));
}

__device__ __forceinline__ void copy_pages(const CopyArgs &a, int64_t warp, int64_t warps) {
    const int lane = threadIdx.x & 31;
    const int64_t n = a.n_at ? *a.n_at : a.n;
    if (!n) return;
    const int page_vec = a.n_kv * a.page * a.vec;  // < 2^29
    const int layers2 = 2 * a.n_layers;            // keys and values of a layer in turn
    const bool two = page_vec <= kPart / 2;        // items at once: of two neighbouring layers2
    const int64_t items = two ? n * a.n_layers : n * layers2;
    const int per = two ? a.n_layers : layers2;
    const int parts = parts_of(page_vec, items, warps);
    for (int64_t t = warp; t < items * parts; t += warps) {
        const int64_t item = t / parts, i = item / per;
        const int part = int(t - item * parts), l = int(item - i * per);
        const int64_t from = a.src[i], to = a.dst[i];
        const int count = a.count ? a.count[i] : a.page;
        if (a.check) {
            if (from < 0) continue;
            if (from >= a.n_pages || to < 0 || to >= a.n_pages || count < 0 || count > a.page) {
                if (l == 0 && part == 0 && lane == 0) record_error(a.err, Q2_0_DEVERR_BAD_ID, i);
                continue;
            }
            if (from == to) continue;
        }
        const uint32_t head = uint32_t(count * a.vec);  // vectors of a head that are copied: contiguous
        const uint32_t skip = uint32_t((a.page - count) * a.vec);
        const uint32_t total = head * uint32_t(a.n_kv);
        if (two) {
            const int64_t at_layer = int64_t(l) * a.n_pages * page_vec;
            uint4 x[kPerLane];
            uint32_t at[kPerLane / 2];
#pragma unroll
            for (int u = 0; u < kPerLane / 2; ++u) {
                at[u] = lane + 32 * u;
                if (at[u] < total) {
                    if (skip) at[u] += at[u] / head * skip;
                    x[2 * u] = a.k[at_layer + from * page_vec + at[u]];
                    x[2 * u + 1] = a.v[at_layer + from * page_vec + at[u]];
                } else {
                    at[u] = ~0u;
                }
            }
#pragma unroll
            for (int u = 0; u < kPerLane / 2; ++u)
                if (at[u] != ~0u) {
                    a.k[at_layer + to * page_vec + at[u]] = x[2 * u];
                    a.v[at_layer + to * page_vec + at[u]] = x[2 * u + 1];
                }
            continue;
        }
        uint4 *c = (l & 1 ? a.v : a.k) + int64_t(l >> 1) * a.n_pages * page_vec;
        const uint4 *s = c + from * page_vec;
        uint4 *d = c + to * page_vec;
        const uint32_t end = uint32_t(uint64_t(total) * (part + 1) / parts);
        for (uint32_t at0 = uint32_t(uint64_t(total) * part / parts) + lane; at0 < end; at0 += kPart) {
            uint4 x[kPerLane];
            uint32_t at[kPerLane];
#pragma unroll
            for (int u = 0; u < kPerLane; ++u) {
                at[u] = at0 + 32 * u;
                if (at[u] < end) {
                    if (skip) at[u] += at[u] / head * skip;
                    x[u] = s[at[u]];
                } else {
                    at[u] = ~0u;
                }
            }
#pragma unroll
            for (int u = 0; u < kPerLane; ++u)
                if (at[u] != ~0u) d[at[u]] = x[u];
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads, kCopyBlocks) copy_kernel(const __grid_constant__ CopyArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warps = kCopyThreads / 32;
    copy_pages(a, int64_t(blockIdx.x) * warps + (threadIdx.x >> 5), int64_t(gridDim.x) * warps);
}

// ---------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------
struct Rows {
    int32_t *refs, *table, *len;
    int64_t n_pages, n_rows, width;
    int page_shift;
    unsigned long long *err;
    __device__ __forceinline__ int64_t pages(int n) const { return (int64_t(n) + (1 << page_shift) - 1) >> page_shift; }
    __device__ __forceinline__ bool valid_len(int n) const { return n >= 0 && n <= (width << page_shift); }
};

// rows_out where it is not the rows themselves
struct MoveArgs {
    const int32_t *from[3];
    int32_t *to[3];
    int64_t n[3];
};
// Thread i0's share of `step` threads'.
__device__ __forceinline__ void move_rows(const MoveArgs &a, int64_t i0, int64_t step) {
#pragma unroll
    for (int w = 0; w < 3; ++w) {
        const bool vec = ((reinterpret_cast<uintptr_t>(a.from[w]) | reinterpret_cast<uintptr_t>(a.to[w])) & 15u) == 0;
        const int64_t n4 = vec ? a.n[w] / 4 : 0;
        for (int64_t i = i0; i < n4; i += step)
            reinterpret_cast<uint4 *>(a.to[w])[i] = reinterpret_cast<const uint4 *>(a.from[w])[i];
        for (int64_t i = 4 * n4 + i0; i < a.n[w]; i += step) a.to[w][i] = a.from[w][i];
    }
}
__global__ void __launch_bounds__(256) rows_move_kernel(const __grid_constant__ MoveArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    move_rows(a, int64_t(blockIdx.x) * blockDim.x + threadIdx.x, int64_t(gridDim.x) * blockDim.x);
}

// ---- fork: one block per child ------------------------------------------------
// 192 children of rows of up to 2048 pages, with the arrays moved apart first: 6.6 us (5.3 MB, 0.8 at the copy rate): two
// launches and four dependent reads, then 327000 additions at L2. 256 threads that read a row twice took 7.9.
constexpr int kForkThreads = 512;
constexpr int kForkHeld = 8;
struct ForkArgs {
    Rows r;
    const int32_t *parent, *child;
    int n;
};
__global__ void __launch_bounds__(kForkThreads) fork_kernel(const __grid_constant__ ForkArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Rows &r = a.r;
    const int j = blockIdx.x;
    const int64_t p = a.parent[j], c = a.child[j];
    // a row that is named twice, or goes on itself, is not written
    int again = 0;
    for (int i = threadIdx.x; i < a.n; i += kForkThreads)
        again |= (i < j && a.child[i] == c) || a.child[i] == p || a.parent[i] == c;
    bool bad = p < 0 || p >= r.n_rows || c < 0 || c >= r.n_rows;
    const int len = bad ? 0 : r.len[p];
    bad = bad || !r.valid_len(len) || r.len[c] != 0;
    const int64_t n = bad ? 0 : r.pages(len);
    const int32_t *from = r.table + p * r.width;
    int32_t *to = r.table + c * r.width;
    // kForkHeld pages a thread at a time; of a row that has no more they stay in registers
    int32_t held[kForkHeld];
    constexpr int kTurn = kForkHeld * kForkThreads;
    auto load = [&](int64_t i) {
#pragma unroll
        for (int u = 0; u < kForkHeld; ++u) {
            const int64_t at = i + u * kForkThreads + threadIdx.x;
            held[u] = at < n ? from[at] : 0;
        }
    };
    int out = 0;
    for (int64_t i = 0; i < n; i += kTurn) {
        load(i);
#pragma unroll
        for (int u = 0; u < kForkHeld; ++u) out |= held[u] < 0 || held[u] >= r.n_pages;
    }
    // (after this barrier too, so that no thread writes a length that another still reads)
    if (__syncthreads_or(again | out | int(bad))) {
        if (threadIdx.x == 0) record_error(r.err, Q2_0_DEVERR_BAD_ID, j);
        return;
    }
    for (int64_t i = 0; i < n; i += kTurn) {
        if (n > kTurn) load(i);
#pragma unroll
        for (int u = 0; u < kForkHeld; ++u) {
            const int64_t at = i + u * kForkThreads + threadIdx.x;
            if (at < n) {
                to[at] = held[u];
                atomicAdd(&r.refs[held[u]], 1);
            }
        }
    }
    if (threadIdx.x == 0) r.len[c] = len;
}

// Few forks of short rows, with the arrays moved apart: one block does all, in one launch.
constexpr int kForkFew = 64;
constexpr int kForkInts = 16384;  // of the arrays
constexpr int kForkBlock = 1024;
__global__ void __launch_bounds__(kForkBlock) fork_few_kernel(const __grid_constant__ ForkArgs a, const Rows in,
                                                               const __grid_constant__ MoveArgs m) {
    __shared__ int len_s[kForkFew];  // of the parent, or -1: refused
    const Rows &r = a.r;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int j = warp; j < a.n; j += kForkBlock / 32) {
        const int64_t p = a.parent[j], c = a.child[j];
        bool bad = p < 0 || p >= r.n_rows || c < 0 || c >= r.n_rows;
        for (int i = lane; i < a.n; i += 32) bad |= (i < j && a.child[i] == c) || a.child[i] == p || a.parent[i] == c;
        bad = __any_sync(~0u, bad);
        const int len = bad ? -1 : in.len[p];
        bad = bad || !r.valid_len(len) || in.len[c] != 0;
        const int64_t n = bad ? 0 : r.pages(len);
        bool out = false;
        for (int64_t i = lane; i < n; i += 32) {
            const int32_t page = in.table[p * r.width + i];
            out |= page < 0 || page >= r.n_pages;
        }
        bad = __any_sync(~0u, bad || out);
        if (lane == 0) {
            len_s[j] = bad ? -1 : len;
            if (bad) record_error(r.err, Q2_0_DEVERR_BAD_ID, j);
        }
    }
    move_rows(m, threadIdx.x, kForkBlock);
    __syncthreads();
    for (int j = warp; j < a.n; j += kForkBlock / 32) {
        const int len = len_s[j];
        if (len < 0) continue;
        const int64_t p = a.parent[j], c = a.child[j], n = r.pages(len);
        for (int64_t i = lane; i < n; i += 32) {
            const int32_t page = in.table[p * r.width + i];
            r.table[c * r.width + i] = page;
            atomicAdd(&r.refs[page], 1);
        }
        if (lane == 0) r.len[c] = len;
    }
}

// ---- the cluster's steps ------------------------------------------------------
constexpr int kMaxBlocks = 16;
constexpr int kMaxThreads = 1024;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kBits = 2048;          // words of a block's bitmap of pages: 2^16 pages
// More new or given back pages of a row than kManyPages are the whole block's work, of kManyRows rows of a block; others are their
// warp's. us of a call, a row's warp alone / its block: 1 row of 131072 tokens in pages of 16 18.5 / 8.0, of 500000
// 62 / 21, 16 rows of 20000 12.7 / 11.6.
constexpr int kManyPages = 512;
constexpr int kManyRows = 16;
constexpr int kMoveEach = 8;         // numbers of the rows that a thread moves apart itself (345000 on 16384 threads: 17.4 us
                                     // against 16.6 with a launch of their own; 613 on 512: 13.1 against 14.3)
constexpr int kStateBytes = 96 << 10;  // shared memory for the states of a block's rows

// The barrier of all blocks of the cluster; of one block alone its own, which orders what its threads
// read and write at less cost.
__device__ __forceinline__ void sync_all() {
    if (cluster_size() == 1)
        __syncthreads();
    else
        cluster_sync();
}

// Sums of pages, kept at kMany where they are more (a cache has fewer than 2^27 pages, so that kMany are never served).
constexpr int kMany = 1 << 28;
__device__ __forceinline__ int plus(int a, int b) { return min(a + b, kMany); }
__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v = plus(v, u);
    }
    return v;
}

// Running sums over the warps of the cluster, of kN numbers at once.
template <int kN>
struct Scan {
    int64_t block[(kN + 1) / 2 * kMaxBlocks];  // two sums each
    int warp[kN][kMaxWarps];
};
// In: a warp's sums (the same in all its lanes). Out: those of all warps before it, and of all. A barrier of the cluster.
template <int kN>
__device__ __forceinline__ void scan_warps(Scan<kN> &s, int (&v)[kN], int (&total)[kN]) {
    static_assert(kN <= 2, "");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int rank = int(cluster_rank()), size = int(cluster_size());
#pragma unroll
    for (int k = 0; k < kN; ++k)
        if (lane == 0) s.warp[k][warp] = v[k];
    __syncthreads();
    int all[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        const int upto = warp_scan(lane < warps ? s.warp[k][lane] : 0, lane), before = __shfl_up_sync(~0u, upto, 1);
        v[k] = __shfl_sync(~0u, lane ? before : 0, warp);
        all[k] = __shfl_sync(~0u, upto, 31);
    }
    if (size == 1) {
#pragma unroll
        for (int k = 0; k < kN; ++k) total[k] = all[k];
        return;
    }
    if (warp == 0 && lane < size) store_cluster(&s.block[rank], uint32_t(lane), int64_t(uint64_t(uint32_t(all[1])) << 32 | uint32_t(all[0])));
    cluster_sync();
    const int64_t mine = lane < size ? s.block[lane] : 0;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        const int b = int(k ? mine >> 32 : mine), upto = warp_scan(b, lane), before = __shfl_up_sync(~0u, upto, 1);
        v[k] = plus(v[k], __shfl_sync(~0u, lane ? before : 0, rank));
        total[k] = __shfl_sync(~0u, upto, 31);
    }
}

// The pages of a warp: a run of whole words of 32, as bits (is(refs)) in shared memory where they fit.
struct PageBits {
    const int32_t *refs;
    int64_t page0, page1;
    uint32_t *bits;  // of page0 on; null: read again
    bool live;       // the bits are of live pages (refs > 0), otherwise of free ones (0)
    __device__ __forceinline__ bool is(int32_t n) const { return live ? n > 0 : n == 0; }
    __device__ __forceinline__ uint32_t word(int64_t p, int lane) const {  // of pages p .. p + 31
        if (bits) return bits[(p - page0) >> 5];
        return __ballot_sync(~0u, p + lane < page1 && is(__ldcg(refs + p + lane)));
    }
    // how many there are; keeps the bits. Four words' loads at a time.
    __device__ __forceinline__ int count(int lane) {
        int n = 0;
        for (int64_t p = page0; p < page1; p += 128) {
            int32_t v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = p + 32 * u + lane < page1 ? __ldcg(refs + p + 32 * u + lane) : -1;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t w = __ballot_sync(~0u, is(v[u]));
                n += __popc(w);
                if (bits && lane == u && p + 32 * u < page1) bits[((p - page0) >> 5) + u] = w;
            }
        }
        __syncwarp();
        return n;
    }
};
__device__ __forceinline__ PageBits pages_of_warp(const Rows &r, int64_t warp, int64_t warps, uint32_t *block_bits, bool live) {
    const int64_t each = ((r.n_pages + warps - 1 >> __ffs(int(warps)) - 1) + 31) / 32 * 32;  // (warps: a power of two)
    PageBits b;
    b.refs = r.refs;
    b.page0 = min(warp * each, r.n_pages);
    b.page1 = min(b.page0 + each, r.n_pages);
    b.bits = each / 32 * (blockDim.x >> 5) <= kBits ? block_bits + (threadIdx.x >> 5) * (each / 32) : nullptr;
    b.live = live;
    return b;
}

// A row before and after.
struct RowState {
    int len, to;
    int last;   // the last page that is kept, if it is filled in part; -1
    int need;   // 4 * pages needed + kParts or kKeeps
    int first;  // its first page among those taken
    int many;   // kManyBack or kManyNew: the block gives its pages back, or hands them out, together
};
constexpr int kManyBack = 1, kManyNew = 2;
constexpr int kParts = 1;  // one of the pages is for a copy of the last one
constexpr int kKeeps = 2;  // the last page is shared, but the others that end in it leave it
constexpr int kNoRow = 1 << 30;

struct ResizeArgs {
    Rows r, in;     // the rows after, and before the call
    MoveArgs move;  // what of them is moved apart first, if that is little
    const int32_t *new_len;
    // workspace
    int32_t *ends, *lowest, *highest;  // [n_pages]: rows that end in a page, the first and last of them
    int32_t *free_list;                // [n_pages]
    RowState *states;                  // [n_rows], or null: they are in shared memory
    int32_t *src, *dst, *count;        // [n_rows]: copies
    int32_t *n_copies;
    int32_t *unserved;                 // the first row that gets no pages
};

// Each warp has a run of neighbouring rows through all steps, dealt evenly to the blocks, their states in shared memory. Bound by latency: four barriers,
// and in each step two or three dependent reads at L2. In place and with the copies' launch behind it 5.5 us for 32 rows on
// 400 pages (one block), 9.9 for 256 rows on 100000; 512 rows of which 77 end give back 20700 pages: 16.6 with
// the arrays moved apart (3.4 MB); with states read again from memory in each step and sums in 64 bits 29.4.
__global__ void __launch_bounds__(kMaxThreads, 1) resize_kernel(const __grid_constant__ ResizeArgs a) {
    extern __shared__ __align__(16) RowState states_s[];  // of the block's rows
    __shared__ Scan<2> scan_s;
    __shared__ uint32_t bits_s[kBits];
    __shared__ int n_many_s, many_s[kManyRows];  // rows of the block, from its first one on
    const Rows &r = a.r;
    const int lane = threadIdx.x & 31, shift = r.page_shift;
    const int64_t block_warps = blockDim.x >> 5, warps = cluster_size() * block_warps;
    const int64_t warp = cluster_rank() * block_warps + (threadIdx.x >> 5);
    const int log_warps = __ffs(int(warps)) - 1;  // (a power of two)
    const int64_t row0 = warp * r.n_rows >> log_warps, row1 = (warp + 1) * r.n_rows >> log_warps;
    const int64_t block_row0 = cluster_rank() * block_warps * r.n_rows >> log_warps;
    RowState *const block_st = a.states ? a.states + block_row0 : states_s, *const st = block_st + (row0 - block_row0);
    if (threadIdx.x == 0) n_many_s = 0;
    __syncthreads();  // (while the launch before ends)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 0 && lane == 0) {
        *a.n_copies = 0;
        *a.unserved = kNoRow;
    }
    // ---- 1. the rows, and the places of pages that they end in
    for (int64_t row = row0 + lane; row < row1; row += 32) {
        RowState s;
        s.len = a.in.len[row];
        s.to = a.new_len[row];
        s.last = -1;
        s.need = 0;
        s.first = 0;
        s.many = 0;
        bool ok = r.valid_len(s.len) && r.valid_len(s.to);
        const int kept = min(s.len, s.to);
        if (ok && (kept & ((1 << shift) - 1))) {
            s.last = a.in.table[row * r.width + (kept >> shift)];
            ok = s.last >= 0 && s.last < r.n_pages;
            if (ok) {
                a.ends[s.last] = 0;
                a.lowest[s.last] = kNoRow;
                a.highest[s.last] = -1;
            }
        }
        if (!ok) {  // left as it is
            record_error(r.err, Q2_0_DEVERR_BAD_ID, row);
            s.to = s.len;
            s.last = -1;
        }
        const int64_t more = r.pages(s.to) - r.pages(s.len);
        if (more > kManyPages || -more > kManyPages) {
            const int at = atomicAdd(&n_many_s, 1);
            if (at < kManyRows) {
                many_s[at] = int(row - block_row0);
                s.many = more > 0 ? kManyNew : kManyBack;
            }
        }
        st[row - row0] = s;
    }
    if (a.move.n[0] + a.move.n[1] + a.move.n[2]) move_rows(a.move, warp * 32 + lane, warps * 32);
    sync_all();
    // ---- 2. who ends where; pages given back
    for (int64_t row = row0 + lane; row < row1; row += 32) {
        const RowState &s = st[row - row0];
        if (s.last >= 0) {
            atomicAdd(&a.ends[s.last], 1);
            atomicMin(&a.lowest[s.last], int(row));
            atomicMax(&a.highest[s.last], int(row));
        }
    }
    // a row's places from `i` on, a warp's eight words of them every `step`
    auto give_back = [&](int64_t row, const RowState &s, int64_t i, int64_t step) {
        const int64_t have = r.pages(s.len);
        int32_t *t = r.table + row * r.width;
        for (i += r.pages(s.to) + lane; i < have; i += step) {
            int32_t page[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) page[u] = i + 32 * u < have ? t[i + 32 * u] : 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (i + 32 * u >= have) break;
                t[i + 32 * u] = -1;
                if (page[u] >= 0 && page[u] < r.n_pages)
                    atomicSub(&r.refs[page[u]], 1);
                else
                    record_error(r.err, Q2_0_DEVERR_BAD_ID, row);
            }
        }
    };
    for (int64_t b = row0; b < row1; b += 32) {
        bool gives = false;
        if (b + lane < row1) {
            const RowState &s = st[b + lane - row0];
            gives = !s.many && r.pages(s.to) < r.pages(s.len);
        }
        for (uint32_t rest = __ballot_sync(~0u, gives); rest; rest &= rest - 1) {
            const int64_t of = b + __ffs(rest) - 1;
            give_back(of, st[of - row0], 0, 256);
        }
    }
    // (the pieces of all such rows are dealt to the warps in turn)
    const int n_many = min(n_many_s, kManyRows);
    auto together = [&](int what, auto &&f) {
        int64_t dealt = 0;
        for (int k = 0; k < n_many; ++k) {
            const RowState &s = block_st[many_s[k]];
            if (s.many != what) continue;
            const int64_t first = ((threadIdx.x >> 5) + block_warps - dealt) & (block_warps - 1);
            f(block_row0 + many_s[k], s, first * 256, block_warps * 256);
            const int64_t more = r.pages(s.to) - r.pages(s.len);
            dealt = dealt + ((more < 0 ? -more : more) + 255) / 256 & (block_warps - 1);
        }
    };
    if (n_many) together(kManyBack, give_back);
    sync_all();
    // ---- 3. what each row needs, and how many pages are free
    PageBits free = pages_of_warp(r, warp, warps, bits_s, false);
    int sum = 0;
    for (int64_t b = row0; b < row1; b += 32) {
        const int64_t row = b + lane;
        int need = 0;
        if (row < row1) {
            RowState &s = st[row - row0];
            int how = 0;
            if (s.last >= 0) {
                const int held = __ldcg(r.refs + s.last), ends = __ldcg(a.ends + s.last), low = __ldcg(a.lowest + s.last);
                if (held > 1) how = ends == held && low == row ? kKeeps : kParts;
            }
            need = int(max(r.pages(s.to) - r.pages(s.len), int64_t(0))) + (how == kParts);
            s.need = need * 4 + how;
        }
        const int upto = warp_scan(need, lane), before = __shfl_up_sync(~0u, upto, 1);
        if (row < row1) st[row - row0].first = plus(sum, lane ? before : 0);
        sum = plus(sum, __shfl_sync(~0u, upto, 31));
    }
    int base[2] = {free.count(lane), sum}, total[2];
    scan_warps(scan_s, base, total);
    const int total_free = total[0], taken = min(total[0], total[1]);
    for (int64_t row = row0 + lane; row < row1; row += 32) {
        RowState &s = st[row - row0];
        s.first = plus(base[1], s.first);
        if (s.need >> 2 && s.first + (s.need >> 2) > total_free) atomicMin(a.unserved, int(row));
    }
    // ---- 4. the free pages in order, as many as are needed
    int rank = base[0];
    for (int64_t p = free.page0; p < free.page1 && rank < taken; p += 32) {
        const uint32_t w = free.word(p, lane);
        const int at = rank + __popc(w & ((1u << lane) - 1));
        if ((w >> lane & 1) && at < taken) a.free_list[at] = int32_t(p + lane);
        rank += __popc(w);
    }
    sync_all();
    // ---- 5. rows take theirs
    const int unserved = total[1] > total_free ? __ldcg(a.unserved) : kNoRow;
    // a row that would keep its page does not where one that was to leave it could not: that one may have more tokens in it
    auto gets_none = [&](int64_t row, const RowState &s) {
        return ((s.need >> 2) && row >= unserved) ||
               ((s.need & kKeeps) && unserved < kNoRow && __ldcg(a.highest + s.last) >= unserved);
    };
    // a row's new pages from the i-th on, a warp's eight words of them every `step`
    auto hand_out = [&](int64_t row, const RowState &s, int64_t i, int64_t step) {
        const int64_t have = r.pages(s.len), more = r.pages(s.to) - have;
        const int32_t *from = a.free_list + s.first + (s.need & kParts);
        int32_t *t = r.table + row * r.width + have;
        for (i += lane; i < more; i += step) {
            int32_t page[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) page[u] = i + 32 * u < more ? __ldcg(from + i + 32 * u) : 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (i + 32 * u >= more) break;
                t[i + 32 * u] = page[u];
                r.refs[page[u]] = 1;
            }
        }
    };
    for (int64_t b = row0; b < row1; b += 32) {
        const int64_t row = b + lane;
        bool grows = false;
        if (row < row1) {
            const RowState &s = st[row - row0];
            const int kept = min(s.len, s.to);
            int32_t *t = r.table + row * r.width;
            if (gets_none(row, s)) {
                r.len[row] = kept;
                record_error(r.err, Q2_0_DEVERR_NO_PAGES, row);
            } else {
                r.len[row] = s.to;
                if (s.need & kParts) {
                    const int32_t page = __ldcg(a.free_list + s.first);
                    t[kept >> shift] = page;
                    r.refs[page] = 1;
                    atomicSub(&r.refs[s.last], 1);
                    const int i = atomicAdd(a.n_copies, 1);
                    a.src[i] = s.last;
                    a.dst[i] = page;
                    a.count[i] = kept & ((1 << shift) - 1);
                }
                const int64_t have = r.pages(s.len), more = r.pages(s.to) - have;
                // few new pages are the lane's own work, more the warp's, many the block's
                grows = more > 4 && !s.many;
                if (more <= 4)
                    for (int64_t i = 0; i < more; ++i) {
                        const int32_t page = __ldcg(a.free_list + s.first + (s.need & kParts) + i);
                        t[have + i] = page;
                        r.refs[page] = 1;
                    }
            }
        }
        for (uint32_t rest = __ballot_sync(~0u, grows); rest; rest &= rest - 1) {
            const int64_t of = b + __ffs(rest) - 1;
            hand_out(of, st[of - row0], 0, 256);
        }
    }
    if (n_many) together(kManyNew, [&](int64_t row, const RowState &s, int64_t i, int64_t step) {
        if (!gets_none(row, s)) hand_out(row, s, i, step);
    });
}

// Compaction: ranks of live and free pages, from bitmaps of the counts. 120000 pages take about 8 us, the tables and the
// list of moves are gone through by the launch that moves the pages.
struct CompactArgs {
    Rows r, in;  // the rows after, and before the call
    int32_t *place, *live;
    int32_t *src, *dst, *n_moves;  // workspace: [n_pages], [n_pages], [1]
    int32_t *rank;                 // [n_pages]: a moved page's place in the list of moves
};

__global__ void __launch_bounds__(kMaxThreads, 1) compact_kernel(const __grid_constant__ CompactArgs a) {
    __shared__ Scan<1> scan_s;
    __shared__ uint32_t bits_s[kBits];
    const int lane = threadIdx.x & 31;
    const int64_t block_warps = blockDim.x >> 5, warps = cluster_size() * block_warps;
    const int64_t warp = cluster_rank() * block_warps + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    cluster_arrive();  // (the sums below go to blocks that have started)
    // ---- how many pages are live
    PageBits pages = pages_of_warp(a.in, warp, warps, bits_s, true);
    int base[1] = {pages.count(lane)}, total[1];
    cluster_wait();
    scan_warps(scan_s, base, total);
    const int64_t live = total[0];
    int64_t before = base[0];
    if (warp == 0 && lane == 0) {
        *a.live = int32_t(live);
        if (live == 0) *a.n_moves = 0;
    }
    // ---- ranks: of the free places below `live` upwards, of the live pages above it downwards
    for (int64_t p0 = pages.page0; p0 < pages.page1; p0 += 32) {
        const int64_t p = p0 + lane;
        const uint32_t w = pages.word(p0, lane);
        const bool in = p < pages.page1, is = w >> lane & 1;
        const int64_t at = before + __popc(w & ((1u << lane) - 1));  // live pages below p
        if (in && (p < live || !is)) a.place[p] = is ? int32_t(p) : -1;
        if (in && p < live && !is) a.dst[p - at] = int32_t(p);
        if (is && p >= live) {
            a.src[live - 1 - at] = int32_t(p);
            a.rank[p] = int32_t(live - 1 - at);
        }
        if (in && p == live - 1) *a.n_moves = int32_t(live - at - is);
        before += __popc(w);
    }
}

// The counts and tables follow, in place or to arrays apart, and the pages move.
__global__ void __launch_bounds__(kCopyThreads) move_kernel(const __grid_constant__ CompactArgs a,
                                                            const __grid_constant__ CopyArgs c) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Rows &r = a.r, &in = a.in;
    const int warps = kCopyThreads / 32;
    const int64_t warp = int64_t(blockIdx.x) * warps + (threadIdx.x >> 5), all = int64_t(gridDim.x) * warps;
    const int lane = threadIdx.x & 31;
    const int64_t moves = *a.n_moves, live = *a.live;
    for (int64_t i = warp * 32 + lane; i < moves; i += all * 32) {
        const int32_t s = a.src[i], d = a.dst[i];
        a.place[s] = d;
        r.refs[d] = in.refs[s];
        r.refs[s] = 0;
    }
    const bool refs_apart = r.refs != in.refs, table_apart = r.table != in.table, len_apart = r.len != in.len;
    if (refs_apart)  // (of places below `live` that are free the moves have written the counts)
        for (int64_t p = warp * 32 + lane; p < r.n_pages; p += all * 32) {
            const int32_t n = in.refs[p];
            if (p >= live) {
                if (n <= 0) r.refs[p] = n;
            } else if (n > 0) {
                r.refs[p] = n;
            }
        }
    // 128 places of a row a warp
    const int64_t runs = (r.width + 127) / 128;
    for (int64_t k = warp; k < r.n_rows * runs; k += all) {
        const int64_t row = k / runs, i0 = (k - row * runs) * 128 + lane;
        const int len = in.len[row];
        int64_t n = r.pages(len);
        if (!r.valid_len(len)) {
            if (lane == 0) record_error(r.err, Q2_0_DEVERR_BAD_ID, row);
            n = 0;
        }
        if (len_apart && i0 == 0) r.len[row] = len;
        const int64_t end = table_apart ? r.width : n;
        if (i0 - lane >= end) continue;
        const int32_t *from = in.table + row * r.width;
        int32_t *to = r.table + row * r.width;
        int32_t p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) p[u] = i0 + 32 * u < end ? from[i0 + 32 * u] : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = i0 + 32 * u;
            int32_t now = p[u];
            if (i < n) {
                if (now < 0 || now >= r.n_pages) {
                    record_error(r.err, Q2_0_DEVERR_BAD_ID, row);
                } else if (now >= live) {
                    // (a page that no count holds has no rank: what stands there is checked against the list)
                    const int64_t m = a.rank[now];
                    if (m >= 0 && m < moves && a.src[m] == now) now = a.dst[m];
                }
            }
            if (i < end && (table_apart || now != p[u])) to[i] = now;
        }
    }
    copy_pages(c, warp, all);
}

// ---------------------------------------------------------------------------
CopyArgs copy_args(const q2_0_kv_cache &c, unsigned long long *err) {
    CopyArgs a = {};
    a.k = static_cast<uint4 *>(c.k);
    a.v = static_cast<uint4 *>(c.v);
    a.n_pages = c.n_pages;
    a.n_layers = c.n_layers;
    a.n_kv = c.n_kv;
    a.page = c.page;
    a.vec = c.dim / 8;
    a.err = err;
    return a;
}

// Blocks for copies of up to n pages: no more than fit the GPU at once, nor than have a part each.
unsigned copy_grid(const q2_0_kv_cache &c, int64_t n) {
    const int64_t full = int64_t(c.n_kv) * c.page * (c.dim / 8) * 2 * c.n_layers;
    const int64_t most = int64_t(sm_count()) * kCopyBlocks;
    if (n >= most * kCopyThreads) return unsigned(most);
    return unsigned(std::max<int64_t>(1, std::min(most, (n * full + kCopyThreads * kPerLane - 1) / (kCopyThreads * kPerLane))));
}

Rows rows_of(const q2_0_kv_cache &c, const q2_0_kv_rows &r, unsigned long long *err) {
    return Rows{r.refs, r.table, r.len, c.n_pages, r.n_rows, r.width, log2_of(c.page), err};
}

// Launches a kernel that may begin while the one before it on the stream still runs (it waits itself), as one
// cluster if `cluster`.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, bool cluster, cudaStream_t s,
                          const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = grid;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.dynamicSmemBytes = smem;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// What is moved apart: nothing of an array that stays in its place.
MoveArgs move_args(const q2_0_kv_cache &c, const q2_0_kv_rows &r, const q2_0_kv_rows &to) {
    MoveArgs m = {{r.refs, r.table, r.len}, {to.refs, to.table, to.len}, {c.n_pages, r.n_rows * r.width, r.n_rows}};
    for (int i = 0; i < 3; ++i)
        if (m.from[i] == m.to[i]) m.n[i] = 0;
    return m;
}
int64_t ints_of(const MoveArgs &m) { return m.n[0] + m.n[1] + m.n[2]; }

// A launch of its own for it.
cudaError_t launch_move(const MoveArgs &m, cudaStream_t s) {
    const int64_t most = std::max(m.n[0], std::max(m.n[1], m.n[2]));
    if (!most) return cudaSuccess;
    const int64_t blocks = std::min<int64_t>(int64_t(sm_count()) * 4, (most / 4 + 255) / 256 + 1);
    rows_move_kernel<<<unsigned(blocks), 256, 0, s>>>(m);
    return cudaGetLastError();
}

std::mutex g_mu;
int g_cluster[64];  // blocks that a cluster may have, of a device

// Clusters of more than 8 blocks are asked for, and had where the GPU has room for one; resize_kernel's shared memory too.
cudaError_t max_cluster(int *blocks) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(g_mu);
    if (dev < 64 && g_cluster[dev]) {
        *blocks = g_cluster[dev];
        return cudaSuccess;
    }
    e = cudaFuncSetAttribute(resize_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(compact_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStateBytes);
    if (e == cudaSuccess) e = cluster_fits(resize_kernel, kMaxThreads, kStateBytes, kMaxBlocks, blocks);
    if (e == cudaSuccess && dev < 64) g_cluster[dev] = *blocks;
    return e;
}

// Blocks of the cluster and their threads: one block where what it goes through is little, as its barrier costs less than the
// cluster's, and fewer threads, whose barriers cost less too, up to a middling size. us in place, one block of 512 / 16 of
// 512 / 16 of 1024 threads: lengths of 32 rows on 400 pages 5.5 / 7.2 / 8.6, on 2000 5.8 / 7.1 / 8.4, on 8000 8.0 / 7.4 /
// 8.8, of 256 rows on 2000 10.6 / 7.6 / 9.0, on 100000 43 / 9.6 / 9.9, of the 512 rows above - / 17.4 / 16.4; compaction
// without moves of 400 pages 3.3 / 4.0 / 4.3, 2000 4.3 / 4.4 / 5.0, 8000 7.8 / 4.4 / 5.1, 100000 84 / 7.9 / 7.8.
constexpr int kAloneRows = 64, kAlonePages = 4096, kAloneCompact = 2048;
constexpr int kFewPages = 65536, kFewRows = 4096;
cudaError_t cluster_shape(bool alone, bool few, int *blocks, int *threads) {
    const cudaError_t e = max_cluster(blocks);
    if (alone) *blocks = 1;
    *threads = alone || few ? kMaxThreads / 2 : kMaxThreads;
    return e;
}

int64_t up(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_kv_copy(const q2_0_kv_cache &c, const int32_t *src, const int32_t *dst, const int32_t *count,
                           int64_t n, unsigned long long *err, cudaStream_t s) {
    CopyArgs a = copy_args(c, err);
    a.src = src;
    a.dst = dst;
    a.count = count;
    a.n = n;
    a.check = true;
    copy_kernel<<<copy_grid(c, n), kCopyThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_fork(const q2_0_kv_cache &c, const q2_0_kv_rows &r, const int32_t *parent, const int32_t *child,
                           int64_t n, const q2_0_kv_rows &out, unsigned long long *err, cudaStream_t s) {
    const MoveArgs m = move_args(c, r, out);
    const ForkArgs a = {rows_of(c, out, err), parent, child, int(n)};
    if (ints_of(m) && ints_of(m) <= kForkInts && n <= kForkFew) {
        fork_few_kernel<<<1, kForkBlock, 0, s>>>(a, rows_of(c, r, err), m);
        return cudaGetLastError();
    }
    const cudaError_t e = launch_move(m, s);
    if (e != cudaSuccess || n == 0) return e;
    return launch_behind(fork_kernel, unsigned(n), kForkThreads, 0, false, s, a);
}

size_t resize_workspace_bytes(int64_t n_pages, int64_t n_rows) {
    return size_t(4 * up(n_pages * 4) + up(n_rows * int64_t(sizeof(RowState))) + 3 * up(n_rows * 4) + 256);
}

cudaError_t resize_run(const q2_0_kv_cache &c, const q2_0_kv_rows &r, const int32_t *new_len, const q2_0_kv_rows &out,
                       void *ws, unsigned long long *err, cudaStream_t s) {
    ResizeArgs a = {};
    a.r = rows_of(c, out, err);
    a.in = rows_of(c, r, err);
    a.new_len = new_len;
    char *p = static_cast<char *>(ws);
    auto take = [&](int64_t bytes) {
        char *q = p;
        p += up(bytes);
        return q;
    };
    a.ends = reinterpret_cast<int32_t *>(take(c.n_pages * 4));
    a.lowest = reinterpret_cast<int32_t *>(take(c.n_pages * 4));
    a.highest = reinterpret_cast<int32_t *>(take(c.n_pages * 4));
    a.free_list = reinterpret_cast<int32_t *>(take(c.n_pages * 4));
    a.states = reinterpret_cast<RowState *>(take(r.n_rows * int64_t(sizeof(RowState))));
    a.src = reinterpret_cast<int32_t *>(take(r.n_rows * 4));
    a.dst = reinterpret_cast<int32_t *>(take(r.n_rows * 4));
    a.count = reinterpret_cast<int32_t *>(take(r.n_rows * 4));
    a.n_copies = reinterpret_cast<int32_t *>(take(8));
    a.unserved = a.n_copies + 1;
    int blocks, threads;
    cudaError_t e = cluster_shape(r.n_rows <= kAloneRows && c.n_pages <= kAlonePages, c.n_pages <= kFewPages && r.n_rows <= kFewRows,
                      &blocks, &threads);
    if (e != cudaSuccess) return e;
    a.move = move_args(c, r, out);
    if (ints_of(a.move) > int64_t(kMoveEach) * blocks * threads) {
        e = launch_move(a.move, s);
        if (e != cudaSuccess) return e;
        for (int64_t &n : a.move.n) n = 0;
    }
    int64_t smem = (r.n_rows / blocks + 1) * int64_t(sizeof(RowState));
    if (smem <= kStateBytes)
        a.states = nullptr;
    else
        smem = 0;
    e = launch_behind(resize_kernel, unsigned(blocks), unsigned(threads), size_t(smem), true, s, a);
    if (e != cudaSuccess) return e;
    CopyArgs k = copy_args(c, err);
    k.src = a.src;
    k.dst = a.dst;
    k.count = a.count;
    k.n_at = a.n_copies;
    return launch_behind(copy_kernel, copy_grid(c, std::min(r.n_rows, c.n_pages)), kCopyThreads, 0, false, s, k);
}

size_t compact_workspace_bytes(int64_t n_pages) { return size_t(3 * up(n_pages * 4) + 256); }

cudaError_t compact_run(const q2_0_kv_cache &c, const q2_0_kv_rows &r, const q2_0_kv_rows &out, int32_t *place,
                        int32_t *live, void *ws, unsigned long long *err, cudaStream_t s) {
    CompactArgs a = {};
    a.r = rows_of(c, out, err);
    a.in = rows_of(c, r, err);
    a.place = place;
    a.live = live;
    char *p = static_cast<char *>(ws);
    a.src = reinterpret_cast<int32_t *>(p);
    a.dst = reinterpret_cast<int32_t *>(p + up(c.n_pages * 4));
    a.rank = reinterpret_cast<int32_t *>(p + 2 * up(c.n_pages * 4));
    a.n_moves = reinterpret_cast<int32_t *>(p + 3 * up(c.n_pages * 4));
    int blocks, threads;
    cudaError_t e = cluster_shape(c.n_pages <= kAloneCompact, c.n_pages <= kFewPages, &blocks, &threads);
    if (e != cudaSuccess) return e;
    e = launch_behind(compact_kernel, unsigned(blocks), unsigned(threads), 0, true, s, a);
    if (e != cudaSuccess) return e;
    CopyArgs k = copy_args(c, err);
    k.src = a.src;
    k.dst = a.dst;
    k.n_at = a.n_moves;
    // (a fourth block of each SM runs behind the other three: see kCopyBlocks)
    return launch_behind(move_kernel, unsigned(sm_count() * kCopyBlocks), kCopyThreads, 0, false, s, a, k);
}

}  // namespace q2
