// Paged key/value cache: q2_0_kv_append (position rotation of q and k, k and v
// stored in their pages) and q2_0_beam_reorder (page tables follow the beams'
// parents, a shared last page is copied).
//
// Both are bound by memory: append reads 4 bytes and writes 2 per value, reorder
// reads and writes 2. Measured on one GB300 against its 6.7 TB/s copy: 16384 tokens of
// 32 + 8 + 8 heads of 128 (613 MB) appended in 94.3 us, 6.5 TB/s; 8 tokens of 16 + 8 + 8
// heads in 2.5 us; the last pages of 128 beams in 36 layers reordered in 87.8 us (profiled
// cold: 84, memory 69 % busy), of 8 beams in 28 layers in 4.3 us.
#include <cuda_bf16.h>

#include "q2_0_device.cuh"
#include "q2_0_internal.h"

namespace q2 {

namespace {

// Two f32 rounded (to nearest even, once) to two values of the cache's type.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

struct AppendArgs {
    const float *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *pos, *slot, *seq, *table;
    const float *rope;
    void *q_out, *k_cache, *v_cache;  // of the layer
    int64_t n_seq, width, n_pos, n_pages;
    int n_q, n_kv, dim, rot, pairs;
    int page_shift;
    unsigned long long *err;
};

// A token's page, looked up once per block: >= 0, or -1: store nothing of k and
// v, or -2: an index is out of range.
__device__ __forceinline__ int64_t token_page(const AppendArgs &a, int64_t t, int slot) {
    if (a.rot && (a.pos[t] < 0 || a.pos[t] >= a.n_pos)) return -2;
    if (slot < 0) return -1;
    const int64_t sq = a.seq ? a.seq[t] : t;
    const int64_t col = slot >> a.page_shift;
    if (sq < 0 || sq >= a.n_seq || col >= a.width) return -2;
    const int64_t p = a.table[sq * a.width + col];
    return p < 0 || p >= a.n_pages ? -2 : p;
}

// One block per token. A thread owns a unit of 16 elements of a head, the same
// unit of every head it visits, so that the unit's cosines and sines are loaded
// once: two spans of 8 at (i, i + rot/2), i = 8u, of a rotating unit of HALVES, of
// 16 neighbours otherwise. Loads are float4, stores 16 bytes; the inputs are read
// once (streaming loads).
template <typename T>
__global__ void __launch_bounds__(128) append_kernel(const __grid_constant__ AppendArgs a) {
    const int64_t t = blockIdx.x;
    const int units = a.dim / 16;
    const int u = threadIdx.x % units;
    const int heads = a.n_q + 2 * a.n_kv;
    const int step = 128 / units;
    const int slot = a.slot[t];
    const int64_t page = token_page(a, t, slot);
    if (page == -2) {
        if (threadIdx.x == 0) record_error(a.err, Q2_0_DEVERR_BAD_ID, t);
        return;
    }
    const bool turns = u < a.rot / 16;
    int e0 = 16 * u, e1 = 16 * u + 8;
    if (turns && !a.pairs) {
        e0 = 8 * u;
        e1 = e0 + a.rot / 2;
    }
    float c[8], s[8];
    if (turns) {
        const float *r = a.rope + int64_t(a.pos[t]) * a.rot + 8 * u;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            *reinterpret_cast<float4 *>(c + i) = __ldg(reinterpret_cast<const float4 *>(r + i));
            *reinterpret_cast<float4 *>(s + i) =
                __ldg(reinterpret_cast<const float4 *>(r + a.rot / 2 + i));
        }
    }
    const int in_page = slot & ((1 << a.page_shift) - 1);
    for (int h = threadIdx.x / units; h < heads; h += step) {
        const float *src;
        T *dst;
        const int hk = h - a.n_q;
        if (hk < 0) {
            src = a.q + t * a.q_stride + int64_t(h) * a.dim;
            dst = static_cast<T *>(a.q_out) + (t * a.n_q + h) * a.dim;
        } else {
            if (page < 0) break;
            const bool is_v = hk >= a.n_kv;
            const int g = is_v ? hk - a.n_kv : hk;
            src = (is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + int64_t(g) * a.dim;
            dst = static_cast<T *>(is_v ? a.v_cache : a.k_cache) +
                  ((((page * a.n_kv + g) << a.page_shift) + in_page) * a.dim);
        }
        float x[8], y[8];
        *reinterpret_cast<float4 *>(x) = __ldcs(reinterpret_cast<const float4 *>(src + e0));
        *reinterpret_cast<float4 *>(x + 4) = __ldcs(reinterpret_cast<const float4 *>(src + e0 + 4));
        *reinterpret_cast<float4 *>(y) = __ldcs(reinterpret_cast<const float4 *>(src + e1));
        *reinterpret_cast<float4 *>(y + 4) = __ldcs(reinterpret_cast<const float4 *>(src + e1 + 4));
        if (turns && hk < a.n_kv) {
            if (a.pairs) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p0 = x[2 * i], p1 = x[2 * i + 1], r0 = y[2 * i], r1 = y[2 * i + 1];
                    x[2 * i] = p0 * c[i] - p1 * s[i];
                    x[2 * i + 1] = p0 * s[i] + p1 * c[i];
                    y[2 * i] = r0 * c[i + 4] - r1 * s[i + 4];
                    y[2 * i + 1] = r0 * s[i + 4] + r1 * c[i + 4];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p0 = x[i], p1 = y[i];
                    x[i] = p0 * c[i] - p1 * s[i];
                    y[i] = p0 * s[i] + p1 * c[i];
                }
            }
        }
        *reinterpret_cast<uint4 *>(dst + e0) =
            make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]),
                       pack2<T>(x[6], x[7]));
        *reinterpret_cast<uint4 *>(dst + e1) =
            make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]),
                       pack2<T>(y[6], y[7]));
    }
}

// The same for rows that are not 16-byte aligned and rotations that do not come
// in units of 16: one thread per element.
template <typename T>
__global__ void __launch_bounds__(128) append_any_kernel(const __grid_constant__ AppendArgs a) {
    const int64_t t = blockIdx.x;
    const int heads = a.n_q + 2 * a.n_kv;
    const int slot = a.slot[t];
    const int64_t page = token_page(a, t, slot);
    if (page == -2) {
        if (threadIdx.x == 0) record_error(a.err, Q2_0_DEVERR_BAD_ID, t);
        return;
    }
    const int in_page = slot & ((1 << a.page_shift) - 1);
    const int half = a.rot / 2;
    const float *r = a.rot ? a.rope + int64_t(a.pos[t]) * a.rot : nullptr;
    for (int i = threadIdx.x; i < heads * a.dim; i += 128) {
        const int h = i / a.dim, e = i % a.dim;
        const int hk = h - a.n_q;
        const float *src;
        T *dst;
        if (hk < 0) {
            src = a.q + t * a.q_stride + int64_t(h) * a.dim;
            dst = static_cast<T *>(a.q_out) + (t * a.n_q + h) * a.dim;
        } else {
            if (page < 0) break;
            const bool is_v = hk >= a.n_kv;
            const int g = is_v ? hk - a.n_kv : hk;
            src = (is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + int64_t(g) * a.dim;
            dst = static_cast<T *>(is_v ? a.v_cache : a.k_cache) +
                  ((((page * a.n_kv + g) << a.page_shift) + in_page) * a.dim);
        }
        float val = src[e];
        if (e < a.rot && hk < a.n_kv) {
            const int j = a.pairs ? e >> 1 : (e < half ? e : e - half);
            const bool second = a.pairs ? (e & 1) : e >= half;
            const float mate = src[a.pairs ? (e ^ 1) : (second ? e - half : e + half)];
            const float c = r[j], s = r[half + j];
            val = second ? mate * s + val * c : val * c - mate * s;
        }
        const uint32_t bits = pack2<T>(val, 0.0f);
        reinterpret_cast<uint16_t *>(dst)[e] = uint16_t(bits & 0xFFFFu);
    }
}

// 16-byte pieces a thread has in flight when a page is copied. The last pages of 128 beams in 36
// layers: 1 105 us, 2 94, 4 87.7, 8 87.6; of 8 beams in 28 layers: 5.1, 4.7, 4.5, 4.2.
constexpr int kCopies = 8;

// One block per (beam, layer): the blocks of layer 0 write the beam's table row,
// every block copies its layer's share of the last page where one is copied.
__global__ void __launch_bounds__(256) reorder_kernel(const __grid_constant__ ReorderArgs a) {
    const int64_t j = blockIdx.x;
    const int64_t g0 = j / a.n_beams * a.n_beams;
    const int me = int(j - g0);
    const int p = a.parent[j];
    const int layer = blockIdx.y;
    if (p < 0 || p >= a.n_beams) {
        if (layer == 0 && threadIdx.x == 0) record_error(a.err, Q2_0_DEVERR_BAD_ID, j);
        return;
    }
    const int64_t src = g0 + p;
    const int len = a.len[src];
    const int last = len >> a.page_shift;
    const int fill = len & ((1 << a.page_shift) - 1);
    if (len < 0 || last > a.width || (last == a.width && fill)) {
        if (layer == 0 && threadIdx.x == 0) record_error(a.err, Q2_0_DEVERR_BAD_ID, j);
        return;
    }
    // a lower beam of the same parent keeps the page
    int again = 0;
    for (int i = threadIdx.x; i < me; i += blockDim.x) again |= a.parent[g0 + i] == p;
    again = __syncthreads_or(again);
    const bool copies = fill && again;
    const bool takes = last < a.width && (copies || !fill);
    const int32_t *row = a.table + src * a.width;
    const int64_t to = takes ? a.fresh[j] : 0, from = copies ? row[last] : 0;
    if (copies && (to < 0 || to >= a.n_pages || from < 0 || from >= a.n_pages)) {
        if (layer == 0 && threadIdx.x == 0) record_error(a.err, Q2_0_DEVERR_BAD_ID, j);
        return;
    }
    if (layer == 0) {
        for (int64_t i = threadIdx.x; i < a.width; i += blockDim.x)
            a.table_out[j * a.width + i] = takes && i == last ? int32_t(to) : row[i];
        if (threadIdx.x == 0) {
            a.len_out[j] = len;
            a.used[j] = takes;
        }
    }
    if (!copies) return;
    const int vec = a.dim / 8;  // 16-byte pieces of a token
    const int64_t page_vec = int64_t(a.n_kv) * vec << a.page_shift;
    const int n = fill * vec;   // of a head's filled places: contiguous
    const int head_vec = vec << a.page_shift;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint4 *c = static_cast<uint4 *>(w ? a.v : a.k) + int64_t(layer) * a.n_pages * page_vec;
        const uint4 *s = c + from * page_vec;
        uint4 *d = c + to * page_vec;
        const int total = n * a.n_kv, step = int(blockDim.x);
        // kCopies loads in flight a thread, then their stores: the pages differ, which the compiler
        // cannot know, and one at a time leaves memory waiting
        for (int i0 = threadIdx.x; i0 < total; i0 += kCopies * step) {
            uint4 x[kCopies];
            int at[kCopies];
#pragma unroll
            for (int u = 0; u < kCopies; ++u) {
                const int i = i0 + u * step;
                if (i < total) {
                    const int h = i / n;
                    at[u] = h * head_vec + i - h * n;
                    x[u] = s[at[u]];
                }
            }
#pragma unroll
            for (int u = 0; u < kCopies; ++u)
                if (i0 + u * step < total) d[at[u]] = x[u];
        }
    }
}

template <typename T>
cudaError_t launch_append_t(const AppendArgs &a, int64_t n_tokens, bool vec, cudaStream_t s) {
    if (vec)
        append_kernel<T><<<dim3(unsigned(n_tokens)), 128, 0, s>>>(a);
    else
        append_any_kernel<T><<<dim3(unsigned(n_tokens)), 128, 0, s>>>(a);
    return cudaGetLastError();
}

// (a null pointer counts as aligned)
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

int log2_of(int page) {
    int s = 0;
    while ((1 << s) < page) ++s;
    return s;
}

cudaError_t launch_append(const q2_0_kv_cache &c, int layer, const float *q, int64_t q_stride,
                          const float *k, int64_t k_stride, const float *v, int64_t v_stride,
                          int64_t n_tokens, int n_q, const int32_t *pos, const int32_t *slot,
                          const int32_t *seq, const int32_t *table, int64_t n_seq, int64_t width,
                          const float *rope, int64_t n_pos, int rot, int style, void *q_out,
                          unsigned long long *err, cudaStream_t s) {
    const int64_t layer_bytes = c.n_pages * c.n_kv * c.page * int64_t(c.dim) * 2;
    AppendArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.pos = pos;
    a.slot = slot;
    a.seq = seq;
    a.table = table;
    a.rope = rope;
    a.q_out = q_out;
    a.k_cache = static_cast<char *>(c.k) + layer * layer_bytes;
    a.v_cache = static_cast<char *>(c.v) + layer * layer_bytes;
    a.n_seq = n_seq;
    a.width = width;
    a.n_pos = n_pos;
    a.n_pages = c.n_pages;
    a.n_q = n_q;
    a.n_kv = c.n_kv;
    a.dim = c.dim;
    a.rot = rot;
    a.pairs = style == Q2_0_ROPE_PAIRS;
    a.page_shift = log2_of(c.page);
    a.err = err;
    const bool vec = rot % 16 == 0 && aligned16(rope) && aligned16(k) && aligned16(v) && k_stride % 4 == 0 &&
                     v_stride % 4 == 0 &&
                     (n_q == 0 || (aligned16(q) && q_stride % 4 == 0 && aligned16(q_out)));
    return c.type == Q2_0_TYPE_F16 ? launch_append_t<__half>(a, n_tokens, vec, s)
                                   : launch_append_t<__nv_bfloat16>(a, n_tokens, vec, s);
}

cudaError_t launch_reorder(const ReorderArgs &a, int64_t n, int n_layers, cudaStream_t s) {
    reorder_kernel<<<dim3(unsigned(n), unsigned(n_layers)), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace q2
