// Decode attention over a paged cache for sequences that share prefixes
// (q2_0_attn_plan_*).
//
// One block per (sequence, query head): tiles of 128 keys, one thread per key
// for the scores, one per output element for the sums, with the running maximum
// and sum of the softmax in f32.
#include <cuda_bf16.h>

#include <new>

#include "q2_0_device.cuh"
#include "q2_0_internal.h"

namespace q2 {

namespace {

constexpr int kTile = 128;

struct AttnArgs {
    const void *k, *v;  // of the layer
    const void *q;
    void *out;
    const int32_t *prefix_table, *prefix_len, *table, *len;
    int64_t prefix_width, width, n_pages;
    int n_groups, n_seq, n_q, n_kv, page_shift;
    float scale_log2;  // scale * log2(e)
    unsigned long long *err;
};

__device__ __forceinline__ float up(__half x) { return __half2float(x); }
__device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T down(float x);
template <>
__device__ __forceinline__ __half down<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 down<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

template <typename T, int D>
__global__ void __launch_bounds__(128) attn_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ float s_q[D], s_p[kTile], s_r[4];
    __shared__ int s_page[kTile];
    const int b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    const int hk = h / (a.n_q / a.n_kv);
    const int group = b / a.n_seq;
    const T *q = static_cast<const T *>(a.q) + (int64_t(b) * a.n_q + h) * D;
    if (tid < D) s_q[tid] = up(q[tid]) * a.scale_log2;
    const T *K = static_cast<const T *>(a.k);
    const T *V = static_cast<const T *>(a.v);
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int part = 0; part < 2; ++part) {
        const int64_t width = part ? a.width : a.prefix_width;
        const int32_t *row = part ? a.table + b * width : a.prefix_table + group * width;
        int64_t n = part ? a.len[b] : (width ? a.prefix_len[group] : 0);
        const int64_t most = width << a.page_shift;
        if (n < 0 || n > most) {
            if (tid == 0 && h == 0)
                record_error(a.err, Q2_0_DEVERR_BAD_ID, part ? b : a.n_groups * a.n_seq + group);
            n = n < 0 ? 0 : most;
        }
        for (int64_t t0 = 0; t0 < n; t0 += kTile) {
            __syncthreads();
            const int64_t t = t0 + tid;
            float s = -INFINITY;
            if (t < n) {
                int page = row[t >> a.page_shift];
                if (page < 0 || page >= a.n_pages) {
                    record_error(a.err, Q2_0_DEVERR_BAD_ID, part ? b : a.n_groups * a.n_seq + group);
                    page = 0;
                }
                s_page[tid] = page;
                const T *kr = K + ((((int64_t(page) * a.n_kv + hk) << a.page_shift) +
                                    (t & ((1 << a.page_shift) - 1))) * D);
                s = 0.0f;
#pragma unroll 8
                for (int e = 0; e < D; ++e) s += s_q[e] * up(kr[e]);
            }
            float tm = s;
            for (int x = 16; x; x >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, x));
            if ((tid & 31) == 0) s_r[tid >> 5] = tm;
            __syncthreads();
            const float mn = fmaxf(m, fmaxf(fmaxf(s_r[0], s_r[1]), fmaxf(s_r[2], s_r[3])));
            const float ref = mn == -INFINITY ? 0.0f : mn;
            const float p = exp2f(s - ref);
            const float keep = exp2f(m - ref);
            m = mn;
            s_p[tid] = p;
            __syncthreads();
            float ts = p;
            for (int x = 16; x; x >>= 1) ts += __shfl_xor_sync(0xffffffffu, ts, x);
            if ((tid & 31) == 0) s_r[tid >> 5] = ts;
            __syncthreads();
            l = l * keep + (s_r[0] + s_r[1] + s_r[2] + s_r[3]);
            if (tid < D) {
                o *= keep;
                const int cnt = n - t0 < kTile ? int(n - t0) : kTile;
                for (int i = 0; i < cnt; ++i) {
                    const int64_t at = (((int64_t(s_page[i]) * a.n_kv + hk) << a.page_shift) +
                                        ((t0 + i) & ((1 << a.page_shift) - 1))) * D;
                    o += s_p[i] * up(V[at + tid]);
                }
            }
        }
    }
    if (tid < D)
        static_cast<T *>(a.out)[(int64_t(b) * a.n_q + h) * D + tid] = down<T>(l > 0.0f ? o / l : 0.0f);
}

}  // namespace
}  // namespace q2

struct q2_0_attn_plan {
    q2::AttnArgs args;
    q2_0_kv_cache cache;
};

namespace q2 {

int attn_plan_create(const q2_0_attn_desc &d, q2_0_attn_plan **plan) {
    unsigned long long *err = error_word_ptr();
    if (!err) return Q2_0_ECUDA;
    q2_0_attn_plan *p = new (std::nothrow) q2_0_attn_plan;
    if (!p) return Q2_0_ECUDA;
    p->cache = d.cache;
    AttnArgs &a = p->args;
    a.q = d.q;
    a.out = d.out;
    a.prefix_table = d.prefix_table;
    a.prefix_len = d.prefix_len;
    a.table = d.table;
    a.len = d.len;
    a.prefix_width = d.prefix_width;
    a.width = d.width;
    a.n_pages = d.cache.n_pages;
    a.n_groups = int(d.n_groups);
    a.n_seq = int(d.n_seq);
    a.n_q = d.n_q;
    a.n_kv = d.cache.n_kv;
    a.page_shift = log2_of(d.cache.page);
    a.scale_log2 = d.scale * 1.44269504f;
    a.err = err;
    *plan = p;
    return Q2_0_OK;
}

int attn_plan_execute(const q2_0_attn_plan *p, int layer, cudaStream_t s) {
    AttnArgs a = p->args;
    const q2_0_kv_cache &c = p->cache;
    const int64_t layer_bytes = c.n_pages * c.n_kv * c.page * int64_t(c.dim) * 2;
    a.k = static_cast<const char *>(c.k) + layer * layer_bytes;
    a.v = static_cast<const char *>(c.v) + layer * layer_bytes;
    const dim3 grid(unsigned(a.n_groups * a.n_seq), unsigned(a.n_q));
    if (c.type == Q2_0_TYPE_F16) {
        if (c.dim == 64)
            attn_kernel<__half, 64><<<grid, 128, 0, s>>>(a);
        else
            attn_kernel<__half, 128><<<grid, 128, 0, s>>>(a);
    } else {
        if (c.dim == 64)
            attn_kernel<__nv_bfloat16, 64><<<grid, 128, 0, s>>>(a);
        else
            attn_kernel<__nv_bfloat16, 128><<<grid, 128, 0, s>>>(a);
    }
    return cuda_status(cudaGetLastError());
}

int attn_plan_launches(const q2_0_attn_plan *) { return 1; }

int attn_plan_layers(const q2_0_attn_plan *p) { return p->cache.n_layers; }

void attn_plan_destroy(q2_0_attn_plan *p) { delete p; }

}  // namespace q2
