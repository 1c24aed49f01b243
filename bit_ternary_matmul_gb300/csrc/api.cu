// C-ABI entry points of libq2_0: argument validation, device checks, scratch
// handling and the device error word. Kernels live in the other .cu files.
#include <math.h>

#include <mutex>

#include "q2_0_device.cuh"
#include "q2_0_internal.h"

namespace q2 {

// Per-device error word (first error wins until q2_0_get_error clears it).
__device__ unsigned long long g_error_word[2];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_dev_state[kMaxDevices];  // 0 unknown, 1 ok, 2 unsupported
int g_sm_count[kMaxDevices];
unsigned long long *g_err_ptr[kMaxDevices];

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

EncodeTiledFn get_encode() {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
    return g_encode;
}

}  // namespace

int check_device(int *device_out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return Q2_0_ECUDA;
    if (device_out) *device_out = dev;
    if (dev < 0 || dev >= kMaxDevices) return Q2_0_EUNSUPPORTED;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (g_dev_state[dev] == 1) return Q2_0_OK;
        if (g_dev_state[dev] == 2) return Q2_0_EUNSUPPORTED;
    }
    cudaDeviceProp p;
    if (cudaGetDeviceProperties(&p, dev) != cudaSuccess) return Q2_0_ECUDA;
    std::lock_guard<std::mutex> lk(g_mu);
    g_dev_state[dev] = (p.major == 10 && p.minor == 3) ? 1 : 2;
    g_sm_count[dev] = p.multiProcessorCount;
    return g_dev_state[dev] == 1 ? Q2_0_OK : Q2_0_EUNSUPPORTED;
}

int sm_count() {
    int dev = 0;
    if (check_device(&dev) != Q2_0_OK) return 0;
    std::lock_guard<std::mutex> lk(g_mu);
    return g_sm_count[dev];
}

unsigned long long *error_word_ptr() {
    int dev = 0;
    if (check_device(&dev) != Q2_0_OK) return nullptr;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_err_ptr[dev]) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_error_word) != cudaSuccess) return nullptr;
        g_err_ptr[dev] = static_cast<unsigned long long *>(p);
    }
    return g_err_ptr[dev];
}

bool encode_tmap_2d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t dim0,
                    uint64_t dim1, uint64_t stride1_bytes, uint32_t box0, uint32_t box1,
                    CUtensorMapSwizzle swizzle) {
    EncodeTiledFn f = get_encode();
    if (!f) return false;
    cuuint64_t dims[2] = {dim0, dim1};
    cuuint64_t strides[1] = {stride1_bytes};
    cuuint32_t box[2] = {box0, box1};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = f(map, dtype, 2, const_cast<void *>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

bool encode_tmap_3d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base,
                    const uint64_t (&dims)[3], const uint64_t (&strides_bytes)[2],
                    const uint32_t (&box)[3], CUtensorMapSwizzle swizzle) {
    EncodeTiledFn f = get_encode();
    if (!f) return false;
    cuuint64_t d[3] = {dims[0], dims[1], dims[2]};
    cuuint64_t st[2] = {strides_bytes[0], strides_bytes[1]};
    cuuint32_t b[3] = {box[0], box[1], box[2]};
    cuuint32_t estr[3] = {1, 1, 1};
    return f(map, dtype, 3, const_cast<void *>(base), d, st, b, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace q2

using namespace q2;

namespace {

inline cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }

inline bool valid_k(int64_t K) { return K >= 64 && K % 64 == 0 && K <= (int64_t(1) << 30); }

// Stream-ordered scratch from the device's default memory pool.
struct PoolScratch {
    void *ptr = nullptr;
    cudaStream_t s = nullptr;
    int alloc(size_t bytes, cudaStream_t st) {
        s = st;
        if (bytes == 0) return Q2_0_OK;
        return cuda_status(cudaMallocAsync(&ptr, bytes, st));
    }
    int release() {
        if (!ptr) return Q2_0_OK;
        cudaError_t e = cudaFreeAsync(ptr, s);
        ptr = nullptr;
        return cuda_status(e);
    }
};

}  // namespace

extern "C" {

const char *q2_0_version(void) { return "q2_0-gb300 0.1.0 (sm_103a)"; }

int q2_0_device_check(void) { return check_device(nullptr); }

size_t q2_0_mul_mat_vec_workspace_size(int64_t K, int ncols) {
    if (!valid_k(K) || ncols < 1 || ncols > 8) return 0;
    return matvec_workspace_bytes(K, ncols);
}

int q2_0_mul_mat_vec_ws(const void *w, const float *x, float *y, int64_t N, int64_t K, int ncols,
                        void *workspace, size_t workspace_bytes, void *stream) {
    if (!w || !x || !y || N < 1 || N > (int64_t(1) << 31) - 1 || !valid_k(K) || ncols < 1 ||
        ncols > 8)
        return Q2_0_EINVAL;
    size_t need = matvec_workspace_bytes(K, ncols);
    if (workspace_bytes < need || (need && !workspace) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    return matvec_run(static_cast<const uint8_t *>(w), x, kXF32, y, N, K, ncols, workspace,
                      workspace_bytes, as_stream(stream));
}

}  // extern "C"

namespace {

int mul_mat_vec_pool(const void *w, const void *x, int xtype, float *y, int64_t N, int64_t K,
                     int ncols, void *stream) {
    if (!w || !x || !y || N < 1 || N > (int64_t(1) << 31) - 1 || !valid_k(K) || ncols < 1 ||
        ncols > 8)
        return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    size_t need = matvec_workspace_bytes(K, ncols);
    PoolScratch ws;
    st = ws.alloc(need, as_stream(stream));
    if (st != Q2_0_OK) return st;
    st = matvec_run(static_cast<const uint8_t *>(w), x, xtype, y, N, K, ncols, ws.ptr, need,
                    as_stream(stream));
    int st2 = ws.release();
    return st != Q2_0_OK ? st : st2;
}

int mul_mat_impl(const void *w, const void *x, int xtype, float *y, int64_t N, int64_t K,
                 int64_t M, int prec, void *workspace, size_t workspace_bytes, void *stream) {
    if (!w || !x || !y || N < 1 || M < 1 || N > (int64_t(1) << 31) - 1 ||
        M > (int64_t(1) << 31) - 1 || !valid_k(K) ||
        (prec != Q2_0_PREC_F16_SPLIT && prec != Q2_0_PREC_F16))
        return Q2_0_EINVAL;
    size_t need = gemm_workspace_bytes(M, N, K, prec);
    if (workspace && (workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    if (workspace || need == 0)
        return gemm_run(static_cast<const uint8_t *>(w), x, xtype, y, N, K, M, prec, workspace,
                        workspace_bytes, as_stream(stream));
    PoolScratch ws;
    st = ws.alloc(need, as_stream(stream));
    if (st != Q2_0_OK) return st;
    st = gemm_run(static_cast<const uint8_t *>(w), x, xtype, y, N, K, M, prec, ws.ptr, need,
                  as_stream(stream));
    int st2 = ws.release();
    return st != Q2_0_OK ? st : st2;
}

}  // namespace

extern "C" {

int q2_0_mul_mat_vec(const void *w, const float *x, float *y, int64_t N, int64_t K, int ncols,
                     void *stream) {
    return mul_mat_vec_pool(w, x, kXF32, y, N, K, ncols, stream);
}

int q2_0_mul_mat_vec_f16(const void *w, const void *x, float *y, int64_t N, int64_t K, int ncols,
                         void *stream) {
    return mul_mat_vec_pool(w, x, kXF16, y, N, K, ncols, stream);
}

int q2_0_mv_plan_create(const q2_0_mv_desc *descs, int n_desc, int ncols, q2_0_mv_plan **plan) {
    if (!plan) return Q2_0_EINVAL;
    *plan = nullptr;
    if (!descs || n_desc < 1 || ncols < 1 || ncols > 8) return Q2_0_EINVAL;
    for (int i = 0; i < n_desc; ++i) {
        const q2_0_mv_desc &d = descs[i];
        if (!d.w || !d.x || !d.y || d.N < 1 || d.N > (int64_t(1) << 31) - 1 || !valid_k(d.K))
            return Q2_0_EINVAL;
    }
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    return reported(mv_plan_create(descs, n_desc, ncols, plan));
}

int q2_0_mv_plan_execute(const q2_0_mv_plan *plan, void *stream) {
    if (!plan) return Q2_0_EINVAL;
    return mv_plan_execute(plan, as_stream(stream));
}

int q2_0_mv_plan_launches(const q2_0_mv_plan *plan) { return plan ? mv_plan_launches(plan) : 0; }

void q2_0_mv_plan_destroy(q2_0_mv_plan *plan) {
    if (plan) mv_plan_destroy(plan);
}

size_t q2_0_mul_mat_workspace_size(int64_t M, int64_t N, int64_t K, int prec) {
    if (M < 1 || N < 1 || !valid_k(K) || (prec != Q2_0_PREC_F16_SPLIT && prec != Q2_0_PREC_F16))
        return 0;
    return gemm_workspace_bytes(M, N, K, prec);
}

int q2_0_mul_mat(const void *w, const float *x, float *y, int64_t N, int64_t K, int64_t M, int prec,
                 void *workspace, size_t workspace_bytes, void *stream) {
    return mul_mat_impl(w, x, kXF32, y, N, K, M, prec, workspace, workspace_bytes, stream);
}

int q2_0_mul_mat_f16(const void *w, const void *x, float *y, int64_t N, int64_t K, int64_t M,
                     void *workspace, size_t workspace_bytes, void *stream) {
    return mul_mat_impl(w, x, kXF16, y, N, K, M, Q2_0_PREC_F16, workspace, workspace_bytes, stream);
}

int q2_0_mm_plan_create(const q2_0_mm_desc *descs, int n_desc, int prec, q2_0_mm_plan **plan) {
    if (!plan) return Q2_0_EINVAL;
    *plan = nullptr;
    if (!descs || n_desc < 1 || (prec != Q2_0_PREC_F16_SPLIT && prec != Q2_0_PREC_F16))
        return Q2_0_EINVAL;
    for (int i = 0; i < n_desc; ++i) {
        const q2_0_mm_desc &d = descs[i];
        if (!d.w || !d.x || !d.y || d.N < 1 || d.M < 1 || d.N > (int64_t(1) << 31) - 1 ||
            d.M > (int64_t(1) << 31) - 1 || !valid_k(d.K))
            return Q2_0_EINVAL;
    }
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    return reported(mm_plan_create(descs, n_desc, prec, plan));
}

int q2_0_mm_plan_execute(const q2_0_mm_plan *plan, void *stream) {
    if (!plan) return Q2_0_EINVAL;
    return mm_plan_execute(plan, as_stream(stream));
}

int q2_0_mm_plan_launches(const q2_0_mm_plan *plan) { return plan ? mm_plan_launches(plan) : 0; }

void q2_0_mm_plan_destroy(q2_0_mm_plan *plan) {
    if (plan) mm_plan_destroy(plan);
}

size_t q2_0_split_bytes(int64_t N, int64_t K) {
    if (N < 1 || N > (int64_t(1) << 31) - 1 || !valid_k(K)) return 0;
    return soa_bytes(N, K);
}

int q2_0_split_layout(const void *w, void *dst, int64_t N, int64_t K, void *stream) {
    if (!w || !dst || N < 1 || N > (int64_t(1) << 31) - 1 || !valid_k(K)) return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    return cuda_status(launch_soa_move(static_cast<const uint8_t *>(w), static_cast<uint8_t *>(dst),
                                       N, K, true, as_stream(stream)));
}

int q2_0_join_layout(const void *src, void *w, int64_t N, int64_t K, void *stream) {
    if (!src || !w || N < 1 || N > (int64_t(1) << 31) - 1 || !valid_k(K)) return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    return cuda_status(launch_soa_move(static_cast<const uint8_t *>(src), static_cast<uint8_t *>(w),
                                       N, K, false, as_stream(stream)));
}

int q2_0_mul_mat_vec_split(const void *w, const float *x, float *y, int64_t N, int64_t K,
                           int ncols, void *stream) {
    if (!w || !x || !y || N < 1 || N > (int64_t(1) << 31) - 1 || !valid_k(K) || ncols < 1 ||
        ncols > 8)
        return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    const size_t need = ncols == 1 ? matvec_workspace_bytes(K, 1) : 0;
    PoolScratch ws;
    st = ws.alloc(need, as_stream(stream));
    if (st != Q2_0_OK) return st;
    st = matvec_split_run(static_cast<const uint8_t *>(w), x, y, N, K, ncols, ws.ptr, need,
                          as_stream(stream));
    int st2 = ws.release();
    return st != Q2_0_OK ? st : st2;
}

int q2_0_g128_mul_mat_vec(const void *w, const float *x, float *y, int64_t N, int64_t K, int ncols,
                         void *stream) {
    if (!w || !x || !y || N < 1 || N > (int64_t(1) << 31) - 1 || K < 128 || K % 128 != 0 ||
        K > (int64_t(1) << 30) || ncols < 1 || ncols > 8)
        return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    const size_t need = matvec_g128_workspace_bytes(K, ncols);
    PoolScratch ws;
    st = ws.alloc(need, as_stream(stream));
    if (st != Q2_0_OK) return st;
    st = matvec_g128_run(static_cast<const uint8_t *>(w), x, y, N, K, ncols, ws.ptr, need,
                         as_stream(stream));
    int st2 = ws.release();
    return st != Q2_0_OK ? st : st2;
}

// Expert mat-vec shapes: n_expert * N rows must fit a tensor-map coordinate,
// and the activation vectors a grid dimension.
static bool valid_moe(int64_t n_expert, int64_t N, int64_t K, int64_t n_x, int64_t n_used,
                      int64_t n_tokens) {
    return n_expert >= 1 && N >= 1 && valid_k(K) && n_used >= 1 && n_tokens >= 0 &&
           (n_x == 1 || n_x == n_used) && n_expert * N <= (int64_t(1) << 31) - 1 &&
           n_tokens * n_x <= 65535 && n_tokens * n_used <= 65535;
}

size_t q2_0_mul_mat_id_workspace_size(int64_t K, int64_t n_tokens, int64_t n_x) {
    if (!valid_k(K) || n_tokens < 0 || n_x < 1) return 0;
    return matvec_moe_workspace_bytes(K, n_tokens * n_x);
}

int q2_0_mul_mat_id(const void *w, int64_t n_expert, int64_t N, int64_t K, const float *x,
                    int64_t n_x, const int32_t *ids, int64_t n_used, int64_t n_tokens, float *y,
                    void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_moe(n_expert, N, K, n_x, n_used, n_tokens)) return Q2_0_EINVAL;
    if (n_tokens == 0) return Q2_0_OK;
    if (!w || !x || !ids || !y) return Q2_0_EINVAL;
    const size_t need = matvec_moe_workspace_bytes(K, n_tokens * n_x);
    if (matvec_fast_path_ok(w, K) &&
        (workspace_bytes < need || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    return matvec_moe_run(static_cast<const uint8_t *>(w), n_expert, N, K, x, n_x, ids, n_used,
                          n_tokens, y, workspace, workspace_bytes, as_stream(stream));
}

int q2_0_get_rows(const void *table, int64_t n_rows, int64_t K, const int32_t *ids, int64_t n_ids,
                  float *out, void *stream) {
    if (n_ids < 0 || n_rows < 1 || !valid_k(K)) return Q2_0_EINVAL;
    if (n_ids == 0) return Q2_0_OK;
    if (!table || !ids || !out || n_ids > (int64_t(1) << 31) - 1) return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    unsigned long long *err = error_word_ptr();
    if (!err) return Q2_0_ECUDA;
    return cuda_status(launch_get_rows(static_cast<const uint8_t *>(table), n_rows, K, ids, n_ids,
                                       out, err, as_stream(stream)));
}

int q2_0_quantize_ref(const float *src, void *dst, int64_t nrows, int64_t K, void *stream) {
    if (!src || !dst || nrows < 1 || !valid_k(K) || nrows > (int64_t(1) << 31) - 1)
        return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    return cuda_status(launch_quantize(src, static_cast<uint8_t *>(dst), nrows, K,
                                       as_stream(stream)));
}

// A cache struct a call may use: shapes, types, alignment, rows of `dim` elements that
// a 32-bit tensor-map coordinate reaches, and pages whose pieces 32 bits count.
static bool valid_cache(const q2_0_kv_cache *c) {
    if (!c || !c->k || !c->v || c->n_pages < 1 || c->n_layers < 1 || c->n_kv < 1 ||
        c->n_kv > (1 << 16))
        return false;
    if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15u) return false;
    if (c->dim != 64 && c->dim != 128) return false;
    if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1))) return false;
    if (c->type != Q2_0_TYPE_F16 && c->type != Q2_0_TYPE_BF16) return false;
    const int64_t most = (int64_t(1) << 31) - 1;
    return c->n_pages <= most && c->n_kv <= most / c->page &&
           c->n_layers <= most / (int64_t(c->n_kv) * c->page) &&
           c->n_pages <= most / (int64_t(c->n_layers) * c->n_kv * c->page);
}

int q2_0_kv_append(const q2_0_kv_cache *cache, int layer, const float *q, int64_t q_stride,
                   const float *k, int64_t k_stride, const float *v, int64_t v_stride,
                   int64_t n_tokens, int n_q, const int32_t *pos, const int32_t *slot,
                   const int32_t *seq, const int32_t *table, int64_t n_seq, int64_t width,
                   const float *rope, int64_t n_pos, int rot, int style, void *q_out,
                   void *stream) {
    if (!valid_cache(cache) || layer < 0 || layer >= cache->n_layers || n_tokens < 0 ||
        n_tokens > (int64_t(1) << 31) - 1 || n_q < 0 || n_q > (1 << 16) || rot < 0 || rot > cache->dim || rot % 2 ||
        (style != Q2_0_ROPE_HALVES && style != Q2_0_ROPE_PAIRS))
        return Q2_0_EINVAL;
    if (n_tokens == 0) return Q2_0_OK;
    if (!k || !v || !slot || !table || n_seq < 1 || width < 1 || (!seq && n_tokens > n_seq) ||
        (n_q && (!q || !q_out || q_stride < int64_t(n_q) * cache->dim)) ||
        k_stride < int64_t(cache->n_kv) * cache->dim ||
        v_stride < int64_t(cache->n_kv) * cache->dim || (rot && (!rope || !pos || n_pos < 1)))
        return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    unsigned long long *err = error_word_ptr();
    if (!err) return Q2_0_ECUDA;
    return cuda_status(launch_append(*cache, layer, q, q_stride, k, k_stride, v, v_stride, n_tokens,
                                     n_q, pos, slot, seq, table, n_seq, width, rope, n_pos, rot,
                                     style, q_out, err, as_stream(stream)));
}

int q2_0_attn_plan_create(const q2_0_attn_desc *d, q2_0_attn_plan **plan) {
    if (!plan) return Q2_0_EINVAL;
    *plan = nullptr;
    if (!d || !valid_cache(&d->cache) || !d->q || !d->out || !d->table || !d->len ||
        ((reinterpret_cast<uintptr_t>(d->q) | reinterpret_cast<uintptr_t>(d->out)) & 15u) ||
        d->n_groups < 1 || d->n_seq < 1 || d->n_groups > 65535 || d->n_seq > 65535 ||
        d->n_groups * d->n_seq > 65535 || d->n_q < 1 || d->n_q > 65535 ||
        d->n_q % d->cache.n_kv || d->n_q / d->cache.n_kv > 64 ||
        d->n_groups * d->n_seq * d->n_q > (int64_t(1) << 28) || d->width < 1 ||
        d->prefix_width < 0 || (d->prefix_width && (!d->prefix_table || !d->prefix_len)) ||
        !(d->scale > -INFINITY && d->scale < INFINITY))
        return Q2_0_EINVAL;
    // a sequence's tokens are counted in 32 bits
    const int64_t most = ((int64_t(1) << 31) - 1) / d->cache.page - 1;
    if (d->width > most || d->prefix_width > most) return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    return reported(attn_plan_create(*d, plan));
}

int q2_0_attn_plan_execute(const q2_0_attn_plan *plan, int layer, void *stream) {
    if (!plan || layer < 0 || layer >= attn_plan_layers(plan)) return Q2_0_EINVAL;
    return attn_plan_execute(plan, layer, as_stream(stream));
}

int q2_0_attn_plan_launches(const q2_0_attn_plan *plan) {
    return plan ? attn_plan_launches(plan) : 0;
}

void q2_0_attn_plan_destroy(q2_0_attn_plan *plan) {
    if (plan) attn_plan_destroy(plan);
}

static bool valid_select(int64_t n_groups, int n_beams, int64_t n_vocab, int n_out) {
    return n_groups >= 0 && n_beams >= 1 && n_beams <= 64 && n_groups <= 65535 / n_beams &&
           n_vocab >= 1 && n_vocab < (int64_t(1) << 31) - (1 << 16) && n_out >= 1 && n_out <= 32;
}

size_t q2_0_beam_select_workspace_size(int64_t n_groups, int n_beams, int64_t n_vocab, int n_out) {
    if (!valid_select(n_groups, n_beams, n_vocab, n_out)) return 0;
    return select_workspace_bytes(n_groups, n_beams, n_vocab, n_out);
}

int q2_0_beam_select(const float *logits, int64_t stride, const float *score, const uint8_t *done,
                     int done_token, int64_t n_groups, int n_beams, int64_t n_vocab, int n_out,
                     float *score_out, int32_t *parent, int32_t *token, void *workspace,
                     size_t workspace_bytes, void *stream) {
    if (!valid_select(n_groups, n_beams, n_vocab, n_out) || stride < n_vocab) return Q2_0_EINVAL;
    if (n_groups == 0) return Q2_0_OK;
    if (!logits || !score || !score_out || !parent || !token) return Q2_0_EINVAL;
    const size_t need = select_workspace_bytes(n_groups, n_beams, n_vocab, n_out);
    if (workspace && (workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    const SelectArgs a = {logits,  stride,  score, done,      done_token, n_groups,
                          n_vocab, n_beams, n_out, score_out, parent,     token};
    if (workspace) return cuda_status(select_run(a, workspace, as_stream(stream)));
    PoolScratch ws;
    st = ws.alloc(need, as_stream(stream));
    if (st != Q2_0_OK) return st;
    st = cuda_status(select_run(a, ws.ptr, as_stream(stream)));
    int st2 = ws.release();
    return st != Q2_0_OK ? st : st2;
}

int q2_0_beam_reorder(const q2_0_kv_cache *cache, const int32_t *parent, int64_t n_groups,
                      int n_beams, const int32_t *table, const int32_t *len, int64_t width,
                      const int32_t *fresh, int32_t *table_out, int32_t *len_out, int32_t *used,
                      void *stream) {
    if (!valid_cache(cache) || n_groups < 0 || n_beams < 1 || n_beams > 1024 || width < 1 ||
        width > ((int64_t(1) << 31) - 1) / cache->page || cache->n_layers > 65535 ||
        n_groups > ((int64_t(1) << 31) - 1) / n_beams)
        return Q2_0_EINVAL;
    if (n_groups == 0) return Q2_0_OK;
    if (!parent || !table || !len || !fresh || !table_out || !len_out || !used) return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    unsigned long long *err = error_word_ptr();
    if (!err) return Q2_0_ECUDA;
    const ReorderArgs a = {cache->k, cache->v, cache->n_pages, cache->n_kv, log2_of(cache->page),
                           cache->dim, parent, table, len, fresh, table_out, len_out, used, width,
                           n_beams, err};
    return cuda_status(launch_reorder(a, n_groups * n_beams, cache->n_layers, as_stream(stream)));
}

static bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    if (!a || !b || !a_bytes || !b_bytes) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + uintptr_t(b_bytes) && y < x + uintptr_t(a_bytes);
}
// Bytes from the first of `rows` rows of n floats, `stride` apart, to the end of the last one.
static int64_t rows_bytes(int64_t rows, int64_t stride, int64_t n) {
    const int64_t most = int64_t(1) << 62;
    if (rows < 1) return 0;
    if (rows > 1 && stride > (most / 4 - n) / (rows - 1)) return most;
    return ((rows - 1) * stride + n) * 4;
}

int q2_0_moe_route(const q2_0_router *r, const float *logits, int64_t stride, int64_t n_tokens, int32_t *ids,
                   float *weights, void *stream) {
    if (!r || r->n_expert < 1 || r->n_expert > 1024 || r->n_used < 1 || r->n_used > 32 ||
        (r->score != Q2_0_SCORE_SOFTMAX && r->score != Q2_0_SCORE_SIGMOID) || r->n_group < 1 || r->n_group > 32 ||
        r->n_expert % r->n_group || r->n_group_used < 1 || r->n_group_used > r->n_group ||
        r->n_used > r->n_group_used * (r->n_expert / r->n_group) || (r->group_top != 1 && r->group_top != 2) ||
        !(r->scale > -INFINITY && r->scale < INFINITY) || stride < r->n_expert || n_tokens < 0 ||
        n_tokens > (int64_t(1) << 31) - 1)
        return Q2_0_EINVAL;
    if (n_tokens == 0) return Q2_0_OK;
    if (!logits || !ids || !weights) return Q2_0_EINVAL;
    const int64_t in = rows_bytes(n_tokens, stride, r->n_expert), out = n_tokens * r->n_used * 4;
    if (overlap(ids, out, weights, out)) return Q2_0_EINVAL;
    for (const void *p : {static_cast<const void *>(ids), static_cast<const void *>(weights)})
        if (overlap(p, out, logits, in) || overlap(p, out, r->bias, r->n_expert * int64_t(4))) return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    return cuda_status(launch_route(*r, logits, stride, n_tokens, ids, weights, as_stream(stream)));
}

int q2_0_draft_verify(const float *target, int64_t target_stride, const float *draft, int64_t draft_stride,
                      const int32_t *tokens, const int32_t *count, const float *rand, int64_t n_seq, int n_draft,
                      int64_t n_vocab, int32_t *accepted, int32_t *token, void *stream) {
    if (n_seq < 0 || n_seq > 65535 || n_draft < 0 || n_draft > 1024 || n_vocab < 1 ||
        n_vocab >= (int64_t(1) << 31) - (1 << 16) || target_stride < n_vocab || (draft && draft_stride < n_vocab))
        return Q2_0_EINVAL;
    if (n_seq == 0) return Q2_0_OK;
    if (!target || !rand || !accepted || !token || (n_draft && !tokens)) return Q2_0_EINVAL;
    // (the blocks of a sequence's cluster read the inputs each for itself, and have to come to the same)
    const int64_t drafts = n_seq * n_draft, all = drafts + n_seq;
    if (overlap(accepted, n_seq * 4, token, all * 4)) return Q2_0_EINVAL;
    for (int i = 0; i < 2; ++i) {
        const void *p = i ? token : accepted;
        const int64_t n = i ? all * 4 : n_seq * 4;
        if (overlap(p, n, target, rows_bytes(all, target_stride, n_vocab)) ||
            overlap(p, n, draft, rows_bytes(drafts, draft_stride, n_vocab)) || overlap(p, n, tokens, drafts * 4) ||
            overlap(p, n, count, n_seq * 4) || overlap(p, n, rand, all * 4))
            return Q2_0_EINVAL;
    }
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    unsigned long long *err = error_word_ptr();
    if (!err) return Q2_0_ECUDA;
    return cuda_status(launch_verify(target, target_stride, n_draft ? draft : nullptr, draft_stride, tokens, count, rand,
                                     n_seq, n_draft, n_vocab, accepted, token, err, as_stream(stream)));
}

// Rows of a valid cache, and where their outcome goes: each array itself, or one apart from all of `r` and from the others of
// the outcome. (What is read of the arrays is checked once: it must not change while a call is at work.)
static bool valid_rows(const q2_0_kv_cache *c, const q2_0_kv_rows *r, const q2_0_kv_rows *out) {
    if (!r || !r->refs || !r->table || !r->len || r->n_rows < 1 || r->n_rows > (1 << 20) || r->width < 1 ||
        r->width > ((int64_t(1) << 31) - 1) / c->page)
        return false;
    if (!out) out = r;
    if (!out->refs || !out->table || !out->len || out->n_rows != r->n_rows || out->width != r->width) return false;
    const int64_t bytes[3] = {c->n_pages * 4, r->n_rows * r->width * 4, r->n_rows * 4};
    const int32_t *const from[3] = {r->refs, r->table, r->len}, *const to[3] = {out->refs, out->table, out->len};
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 3; ++j) {
            if (i == j && from[i] == to[i]) continue;
            if (overlap(to[i], bytes[i], from[j], bytes[j])) return false;
            if (i < j && (overlap(from[i], bytes[i], from[j], bytes[j]) || overlap(to[i], bytes[i], to[j], bytes[j]))) return false;
        }
    return true;
}
// An input or output of `bytes` beside the rows that a call writes.
static bool apart(const void *p, int64_t bytes, const q2_0_kv_cache *c, const q2_0_kv_rows &out) {
    return !overlap(p, bytes, out.refs, c->n_pages * 4) && !overlap(p, bytes, out.table, out.n_rows * out.width * 4) &&
           !overlap(p, bytes, out.len, out.n_rows * 4);
}
// Whether an array of `bytes` shares memory with the cache's pages.
static bool in_cache(const void *p, int64_t bytes, const q2_0_kv_cache *c) {
    const int64_t cache = c->n_pages * c->n_layers * c->n_kv * c->page * c->dim * 2;
    return overlap(p, bytes, c->k, cache) || overlap(p, bytes, c->v, cache);
}
// A workspace that a call on rows can take: large enough, aligned, beside the rows and the cache.
static bool valid_rows_workspace(const void *ws, size_t bytes, size_t need, const q2_0_kv_cache *c, const q2_0_kv_rows &r,
                                 const q2_0_kv_rows &out) {
    if (!ws) return true;
    const int64_t n = int64_t(need);
    return bytes >= need && !(reinterpret_cast<uintptr_t>(ws) & 255u) && apart(ws, n, c, r) && apart(ws, n, c, out) &&
           !in_cache(ws, n, c);
}

int q2_0_kv_copy(const q2_0_kv_cache *cache, const int32_t *src, const int32_t *dst, const int32_t *count, int64_t n,
                 void *stream) {
    if (!valid_cache(cache) || n < 0 || n > (int64_t(1) << 31) - 1) return Q2_0_EINVAL;
    if (n == 0) return Q2_0_OK;
    if (!src || !dst || in_cache(src, n * 4, cache) || in_cache(dst, n * 4, cache) || in_cache(count, n * 4, cache))
        return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    unsigned long long *err = error_word_ptr();
    if (!err) return Q2_0_ECUDA;
    return cuda_status(launch_kv_copy(*cache, src, dst, count, n, err, as_stream(stream)));
}

int q2_0_kv_fork(const q2_0_kv_cache *cache, const q2_0_kv_rows *rows, const int32_t *parent, const int32_t *child,
                 int64_t n, const q2_0_kv_rows *rows_out, void *stream) {
    if (!valid_cache(cache) || !valid_rows(cache, rows, rows_out) || n < 0 || n > 4096 || (n && (!parent || !child)))
        return Q2_0_EINVAL;
    const q2_0_kv_rows &out = rows_out ? *rows_out : *rows;
    if (n && (!apart(parent, n * 4, cache, out) || !apart(child, n * 4, cache, out))) return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    unsigned long long *err = error_word_ptr();
    if (!err) return Q2_0_ECUDA;
    return cuda_status(launch_kv_fork(*cache, *rows, parent, child, n, out, err, as_stream(stream)));
}

size_t q2_0_kv_resize_workspace_size(int64_t n_pages, int64_t n_rows) {
    if (n_pages < 1 || n_pages > (int64_t(1) << 31) - 1 || n_rows < 1 || n_rows > (1 << 20)) return 0;
    return resize_workspace_bytes(n_pages, n_rows);
}

int q2_0_kv_resize(const q2_0_kv_cache *cache, const q2_0_kv_rows *rows, const int32_t *new_len,
                   const q2_0_kv_rows *rows_out, void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_cache(cache) || !valid_rows(cache, rows, rows_out) || !new_len) return Q2_0_EINVAL;
    const q2_0_kv_rows &out = rows_out ? *rows_out : *rows;
    // (the lengths themselves, in place, are read before they are written)
    if (!(new_len == rows->len && out.len == rows->len) &&
        (!apart(new_len, rows->n_rows * 4, cache, out) || in_cache(new_len, rows->n_rows * 4, cache)))
        return Q2_0_EINVAL;
    const size_t need = resize_workspace_bytes(cache->n_pages, rows->n_rows);
    if (!valid_rows_workspace(workspace, workspace_bytes, need, cache, *rows, out) ||
        overlap(workspace, int64_t(need), new_len, rows->n_rows * 4))
        return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    unsigned long long *err = error_word_ptr();
    if (!err) return Q2_0_ECUDA;
    PoolScratch ws;
    if (!workspace) {
        st = ws.alloc(need, as_stream(stream));
        if (st != Q2_0_OK) return st;
    }
    st = cuda_status(resize_run(*cache, *rows, new_len, out, workspace ? workspace : ws.ptr, err, as_stream(stream)));
    int st2 = ws.release();
    return st != Q2_0_OK ? st : st2;
}

size_t q2_0_kv_compact_workspace_size(int64_t n_pages, int64_t n_rows) {
    if (n_pages < 1 || n_pages > (int64_t(1) << 31) - 1 || n_rows < 1 || n_rows > (1 << 20)) return 0;
    return compact_workspace_bytes(n_pages);
}

int q2_0_kv_compact(const q2_0_kv_cache *cache, const q2_0_kv_rows *rows, const q2_0_kv_rows *rows_out, int32_t *place,
                    int32_t *live, void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_cache(cache) || !valid_rows(cache, rows, rows_out) || !place || !live) return Q2_0_EINVAL;
    const q2_0_kv_rows &out = rows_out ? *rows_out : *rows;
    for (const q2_0_kv_rows *r : {rows, &out})
        if (!apart(place, cache->n_pages * 4, cache, *r) || !apart(live, 4, cache, *r)) return Q2_0_EINVAL;
    if (overlap(place, cache->n_pages * 4, live, 4) || in_cache(place, cache->n_pages * 4, cache) || in_cache(live, 4, cache))
        return Q2_0_EINVAL;
    const size_t need = compact_workspace_bytes(cache->n_pages);
    if (!valid_rows_workspace(workspace, workspace_bytes, need, cache, *rows, out) ||
        overlap(workspace, int64_t(need), place, cache->n_pages * 4) ||
        overlap(workspace, int64_t(need), live, 4))
        return Q2_0_EINVAL;
    int st = check_device(nullptr);
    if (st != Q2_0_OK) return st;
    unsigned long long *err = error_word_ptr();
    if (!err) return Q2_0_ECUDA;
    PoolScratch ws;
    if (!workspace) {
        st = ws.alloc(need, as_stream(stream));
        if (st != Q2_0_OK) return st;
    }
    st = cuda_status(compact_run(*cache, *rows, out, place, live, workspace ? workspace : ws.ptr, err,
                                 as_stream(stream)));
    int st2 = ws.release();
    return st != Q2_0_OK ? st : st2;
}

int q2_0_get_error(void *stream, int64_t *info) {
    if (check_device(nullptr) != Q2_0_OK) return -1;
    cudaStream_t s = as_stream(stream);
    unsigned long long host[2] = {0, 0};
    const unsigned long long zero[2] = {0, 0};
    if (cudaStreamSynchronize(s) != cudaSuccess) return -1;
    if (cudaMemcpyFromSymbolAsync(host, g_error_word, sizeof(host), 0, cudaMemcpyDeviceToHost, s) !=
        cudaSuccess)
        return -1;
    if (cudaMemcpyToSymbolAsync(g_error_word, zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s) !=
        cudaSuccess)
        return -1;
    if (cudaStreamSynchronize(s) != cudaSuccess) return -1;
    if (info) *info = static_cast<int64_t>(host[1]);
    return static_cast<int>(host[0]);
}

}  // extern "C"
