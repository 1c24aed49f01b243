/*
 * q2_0.h — C ABI of the GB300 (sm_103a) Q2_0 dequantize-fused matmul library.
 *
 * Q2_0 format. Sources: "WebGPU: add Q2_0 support" (bisque.today write-up of
 * llama.cpp PR 30914), format paragraph; "Llama.cpp umí dvoubitový Q2_0 i na
 * kartách NVIDIA" (aisvetem.cz), section "Osmnáct bajtů na čtyřiašedesát vah".
 *   A block packs 64 weights into 18 bytes: a little-endian IEEE fp16 scale d at
 *   byte 0, then four little-endian u32 words at bytes 2, 6, 10, 14. Element
 *   16*w + i of the block is the code q = (word_w >> 2i) & 3, and decodes to
 *   (q - 1) * d: codes 0/1/2/3 give -d / 0 / +d / +2d (3 is reserved by the
 *   format but decoded by the same rule).
 *   A weight matrix W has N rows of K weights (K a multiple of 64) stored as
 *   N * K/64 consecutive blocks, row-major: block b of row n is at byte offset
 *   (n * K/64 + b) * 18. No alignment is required of W.
 *
 * Activations and outputs follow ggml's mul_mat(src0 = W, src1 = X):
 *   X is F32 [C][K] row-major (C = ncols or M), Y is F32 [C][N] row-major,
 *   Y[c][n] = sum_k W[n][k] * X[c][k].
 *
 * Conventions for every call:
 *   - All pointers are device pointers owned by the caller, unless stated.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream). Calls are
 *     asynchronous on it; nothing synchronises the host except
 *     q2_0_get_error().
 *   - The calls act on the device current to the calling thread. That device
 *     must be compute capability 10.3 (GB300); otherwise Q2_0_EUNSUPPORTED.
 *   - Argument errors return Q2_0_EINVAL before anything is launched. A failed
 *     launch or runtime call returns Q2_0_ECUDA. No exception crosses the ABI.
 *     There is no CPU fallback: every result is computed by a CUDA kernel.
 *   - Data-dependent errors found by a kernel (an id out of range in get_rows,
 *     a pipeline wait that timed out) are recorded in a per-device error word;
 *     q2_0_get_error() reads and clears it.
 */
#ifndef Q2_0_H
#define Q2_0_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define Q2_0_BLOCK_WEIGHTS 64
#define Q2_0_BLOCK_BYTES 18

typedef enum q2_0_status {
    Q2_0_OK = 0,
    Q2_0_EINVAL = 1,       /* bad argument; nothing was launched */
    Q2_0_ECUDA = 2,        /* a CUDA runtime call or kernel launch failed */
    Q2_0_EUNSUPPORTED = 3, /* the current device is not compute capability 10.3 */
    Q2_0_EDEVICE = 4,      /* a kernel recorded an error: see q2_0_get_error() */
    Q2_0_ENOSPACE = 5      /* q2_0_mul_mat_vec_noalloc: the call needs more scratch than
                              Q2_0_NOALLOC_SCRATCH_BYTES; nothing was launched */
} q2_0_status;

/* Device error codes (first error wins until cleared). */
#define Q2_0_DEVERR_NONE 0
#define Q2_0_DEVERR_BAD_ID 1  /* get_rows / mul_mat_id: ids[info] out of range; cache calls: see there */
#define Q2_0_DEVERR_TIMEOUT 2 /* a pipeline wait gave up; info = kernel tag */
#define Q2_0_DEVERR_NO_PAGES 3 /* kv_resize: row info got none of the pages that it needs */

/* GEMM activation precision. F32 activations are used by the tensor cores as
 * fp16 operands (the weights (q-1)*d are exact in fp16). Each token row is first
 * scaled by an exact power of two that puts its largest |x| in [2^14, 2^15), and
 * the f32 result is scaled back, so any finite x is in range:
 *   Q2_0_PREC_F16_SPLIT: x = hi + lo with hi = fp16(x), lo = fp16(x - hi); two
 *     tensor-core products. Each element x is held to within 2^-22 |x| + 2^-39 M
 *     (M its row's largest |x|): 22 bits of its own value down to 2^-18 M;
 *     tolerance |y - exact| <= 1e-5 * sum|w*x| + 1e-7. The products are exact; the f32 accumulation over K/16 tensor-core
 *     steps adds rounding that is far below that in practice, but whose
 *     worst-case bound grows as (K/16) * 2^-24 * sum|w*x|.
 *   Q2_0_PREC_F16: x rounded once to fp16, within 2^-11 |x| + 2^-39 M.
 *     Tolerance <= 4e-3 * sum|w*x|.
 * Precondition of both: finite x, and |2d| <= 65504 (so that (q-1)*d is finite
 * in fp16). */
typedef enum q2_0_prec { Q2_0_PREC_F16_SPLIT = 0, Q2_0_PREC_F16 = 1 } q2_0_prec;

/* Library version string (static storage). */
const char *q2_0_version(void);

/* Checks that the current device is a compute capability 10.3 GPU.
 * Returns Q2_0_OK, Q2_0_EUNSUPPORTED or Q2_0_ECUDA. */
int q2_0_device_check(void);

/*
 * q2_0_mul_mat_vec — decode mat-vec, Y[c][n] = sum_k W[n][k] X[c][k].
 * Source: the mat-vec kernel of "WebGPU: add Q2_0 support" (each block's codes
 * are multiplied by the activations and the scale d is applied once per block
 * sum).
 *   w      N x K Q2_0 matrix (N*K/64*18 bytes), any alignment.
 *   x      F32 [ncols][K].   y  F32 [ncols][N] (written, not accumulated).
 *   N >= 1, K >= 64 with K % 64 == 0, 1 <= ncols <= 8.
 * Precision (finite x; M_b = the largest |x| of the activation block of 64
 * that holds element k; the tensor-core paths have K % 512 == 0 and w 16-byte
 * aligned, other shapes run f32 on CUDA cores):
 *   ncols 1 and 2, tensor cores (fp4): each element of x is represented to
 *     within 2^-33 M_b; zero weights contribute exactly nothing; the rest is
 *     f32 rounding: |y - exact| <= 2^-33 sum_k |W[n][k]| M_b + 2^-20 sum_k |W X|;
 *   ncols 3..8, tensor cores (e4m3): each element keeps 20 bits of its own value,
 *     with a floor of 2^-33 M_b: |y - exact| <= 2^-33 sum_k |W[n][k]| M_b +
 *     2^-17 sum_k |W X|;
 *   CUDA cores: f32 products and sums, |y - exact| <= 2^-17 sum_k |W X| for
 *     K <= 65536.
 * The tensor-core paths meet the tolerance |y - exact| <= 1e-5 *
 * sum_k |W[n][k] X[c][k]| + 1e-7 unless, weighted by |W|, the activations sit
 * on average more than ~2e4 times below the largest element of their own block
 * of 64.
 * Scratch: the call takes q2_0_mul_mat_vec_workspace_size(K, ncols) bytes of
 * stream-ordered memory from the device's default memory pool
 * (cudaMallocAsync/cudaFreeAsync on `stream`); use q2_0_mul_mat_vec_ws to
 * supply it instead.
 */
int q2_0_mul_mat_vec(const void *w, const float *x, float *y, int64_t N, int64_t K, int ncols,
                     void *stream);

/*
 * q2_0_mul_mat_vec_f16 — q2_0_mul_mat_vec with F16 (IEEE binary16)
 * activations x [ncols][K], any alignment; y F32. The pages' WebGPU port
 * supports F32 activations only and lists F16 ones as missing ("WebGPU: add
 * Q2_0 support", limitations paragraph); this is that variant. Each fp16
 * value is read exactly, so the F32 precision statement applies with x read
 * as the exact fp16 values. Scratch as q2_0_mul_mat_vec (default memory pool).
 */
int q2_0_mul_mat_vec_f16(const void *w, const void *x, float *y, int64_t N, int64_t K, int ncols,
                         void *stream);

/* Scratch bytes q2_0_mul_mat_vec_ws needs for (K, ncols); 0 on bad arguments. */
size_t q2_0_mul_mat_vec_workspace_size(int64_t K, int ncols);

/* As q2_0_mul_mat_vec, with caller-owned scratch `workspace` (device memory,
 * 256-byte aligned, at least workspace_size bytes; contents are overwritten and
 * must not be used by other work in flight). */
int q2_0_mul_mat_vec_ws(const void *w, const float *x, float *y, int64_t N, int64_t K, int ncols,
                        void *workspace, size_t workspace_bytes, void *stream);

/*
 * q2_0_mul_mat_vec_noalloc — q2_0_mul_mat_vec for callers that cannot allocate
 * device memory at call time. (The Q2_0 pages have no counterpart: this is a
 * deployment variant of the decode mat-vec above, with the same arguments and
 * the same result and error bound.)
 *   Who needs it: an inference server or framework that reserves all of HBM
 *   for its own allocator leaves nothing for cudaMalloc or the default memory
 *   pool, and a latency-critical decode loop should not call an allocator at
 *   all. This call allocates nothing: its scratch (the prepared activation
 *   fragments) lives in a static device array of Q2_0_NOALLOC_SCRATCH_BYTES
 *   that every GPU which loads the library holds until the process exits.
 *   Limit: shapes on the tensor-core path (K % 512 == 0 and w 16-byte
 *   aligned) need q2_0_mul_mat_vec_workspace_size(K, ncols) bytes of scratch;
 *   if that exceeds Q2_0_NOALLOC_SCRATCH_BYTES the call returns Q2_0_ENOSPACE
 *   and launches nothing (1 MiB covers K up to 126,976 for ncols = 1, 63,488
 *   for ncols 2..3, 31,744 for ncols 4..6 and 21,504 for ncols 7..8). Other
 *   shapes run the CUDA-core kernel, which needs no scratch, at any K.
 *   Set-up: the first call on a device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current and keeps it for the life
 *   of the process; make that first call before any stream capture, and do not
 *   call the entry point again after a cudaDeviceReset of that device (the
 *   kept address belongs to the context the reset destroyed).
 *   Sharing: every call uses the same array and leaves its contents behind.
 *   Each call rewrites all of the scratch it reads, so nothing needs clearing,
 *   but calls whose executions overlap on the GPU (e.g. on two streams) race
 *   on the array: serialise them.
 */
#define Q2_0_NOALLOC_SCRATCH_BYTES ((size_t)1 << 20)
int q2_0_mul_mat_vec_noalloc(const void *w, const float *x, float *y, int64_t N, int64_t K,
                             int ncols, void *stream);

/*
 * Batched decode mat-vec: many independent (W, x, y) products, e.g. all the
 * projections of one decoder step, run by one persistent launch with a static,
 * cost-balanced schedule of row tiles over the GPU's SMs.
 * q2_0_mv_plan_create records the descriptors (the pointers are kept, not the
 * data), encodes per-matrix TMA descriptors, builds the schedule and allocates
 * the plan's device memory and scratch. q2_0_mv_plan_execute launches the work
 * on `stream` (two kernels: activation preparation, then the mat-vecs); it
 * allocates nothing and may be captured in a CUDA graph. Each descriptor
 * obeys q2_0_mul_mat_vec's rules; all share ncols.
 */
typedef struct q2_0_mv_desc {
    const void *w; /* N x K Q2_0 matrix */
    const float *x; /* F32 [ncols][K] */
    float *y;       /* F32 [ncols][N] */
    int64_t N;
    int64_t K;
} q2_0_mv_desc;

typedef struct q2_0_mv_plan q2_0_mv_plan;

int q2_0_mv_plan_create(const q2_0_mv_desc *descs, int n_desc, int ncols, q2_0_mv_plan **plan);
int q2_0_mv_plan_execute(const q2_0_mv_plan *plan, void *stream);
/* Number of kernel launches one execute performs. */
int q2_0_mv_plan_launches(const q2_0_mv_plan *plan);
void q2_0_mv_plan_destroy(q2_0_mv_plan *plan);

/*
 * q2_0_mul_mat — prefill GEMM, Y[m][n] = sum_k W[n][k] X[m][k], M tokens.
 * Source: the tiled matrix multiply of "WebGPU: add Q2_0 support" (codes are
 * unpacked into shared memory as half precision before the product).
 *   w      N x K Q2_0 matrix.  x  F32 [M][K].  y  F32 [M][N] (written).
 *   N, M >= 1, K >= 64 with K % 64 == 0. prec is a q2_0_prec.
 * workspace: device memory of at least q2_0_mul_mat_workspace_size(M, N, K,
 * prec) bytes, 256-byte aligned, or NULL to take it from the device's default
 * memory pool on `stream` (stream-ordered).
 */
size_t q2_0_mul_mat_workspace_size(int64_t M, int64_t N, int64_t K, int prec);
int q2_0_mul_mat(const void *w, const float *x, float *y, int64_t N, int64_t K, int64_t M, int prec,
                 void *workspace, size_t workspace_bytes, void *stream);

/*
 * q2_0_mul_mat_f16 — q2_0_mul_mat with F16 activations x [M][K] (the missing
 * F16 path of the same limitations paragraph). fp16 x is already an exact fp16
 * tensor-core operand, so one product per weight suffices and the bound is
 * |y - exact| <= 1e-5 * sum_k |W[n][k] X[m][k]| + 1e-7 with X the fp16 values.
 * workspace: at least q2_0_mul_mat_workspace_size(M, N, K, Q2_0_PREC_F16)
 * bytes, 256-byte aligned, or NULL for the default memory pool. Fast path:
 * K % 512 == 0, w and x 16-byte aligned; otherwise a CUDA-core kernel.
 */
int q2_0_mul_mat_f16(const void *w, const void *x, float *y, int64_t N, int64_t K, int64_t M,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * Grouped prefill GEMM: several independent products Y = W X^T (e.g. the
 * gate and up projections of one layer, which read the same X) run as one
 * launch of the tensor-core kernel over the pooled output tiles, with one
 * activation prepass and one stream-K reduction for all of them.
 * q2_0_mm_plan_create records the descriptors (the pointers are kept, not the
 * data), prepares each distinct activation matrix once (descriptors with the
 * same x, M and K share it), encodes the TMA descriptors and allocates the
 * plan's device memory: per distinct X, the fp16 hi (and lo) copies and the
 * row exponents; the stream-K partial tiles (2 x 128 KB per SM). Each
 * descriptor obeys q2_0_mul_mat's rules and its bound; all share prec. A
 * descriptor outside the fast path (K % 512 != 0, w or x not 16-byte aligned)
 * runs the CUDA-core kernel inside execute. q2_0_mm_plan_execute launches the
 * work on `stream` (the prepass, one launch per 8 distinct X; the tensor-core
 * kernel; the reduction; one launch per CUDA-core descriptor); it allocates
 * nothing and may be captured in a CUDA graph. Each execute reads the
 * current contents of every w and x and writes every y, so the caller may
 * refill x between executes. Products must not write to memory that another
 * product of the same plan reads or writes, and two executes of one plan must
 * not overlap on the GPU (they share the plan's scratch).
 * Ownership: the plan belongs to the device current at creation; execute it
 * on a stream of that device. q2_0_mm_plan_destroy frees its device memory;
 * call it after the last execute has completed.
 * Errors: Q2_0_EINVAL for a null pointer, n_desc < 1, N or M outside
 * [1, 2^31), K not a multiple of 64 in [64, 2^30] or an unknown prec;
 * Q2_0_EUNSUPPORTED for a device that is not compute capability 10.3;
 * Q2_0_ECUDA when an allocation, a copy or a TMA descriptor fails.
 */
typedef struct q2_0_mm_desc {
    const void *w;  /* N x K Q2_0 matrix */
    const float *x; /* F32 [M][K] */
    float *y;       /* F32 [M][N] */
    int64_t N;
    int64_t K;
    int64_t M;
} q2_0_mm_desc;

typedef struct q2_0_mm_plan q2_0_mm_plan;

int q2_0_mm_plan_create(const q2_0_mm_desc *descs, int n_desc, int prec, q2_0_mm_plan **plan);
int q2_0_mm_plan_execute(const q2_0_mm_plan *plan, void *stream);
/* Number of kernel launches one execute performs. */
int q2_0_mm_plan_launches(const q2_0_mm_plan *plan);
void q2_0_mm_plan_destroy(q2_0_mm_plan *plan);

/*
 * Split layout — scales and codes in separate arrays, as the loader in
 * "kopitiam_runtime::gpu_offload" (section "Why the weight has to stay
 * quantized") splits a block format's scales from its quants. For an N x K
 * Q2_0 matrix with nb = K/64 blocks per row, the split buffer holds
 *   qs[n][b][16]  the 16 code bytes of block (n, b), row-major, then, from
 *                 byte round_up(N * nb * 16, 256),
 *   d[n][b]       its fp16 scale (2 bytes, little-endian), row-major;
 * q2_0_split_bytes(N, K) bytes in all. The code and scale rules are the
 * 18-byte block's. The split is a load-time option; q2_0_mul_mat_vec_split
 * computes what q2_0_mul_mat_vec computes on the 18-byte layout.
 *   q2_0_split_layout  18-byte blocks w -> split buffer dst (bit-exact move).
 *   q2_0_join_layout   split buffer src -> 18-byte blocks w (its inverse).
 *   q2_0_mul_mat_vec_split  y = W x with W in the split layout; same bound as
 *       q2_0_mul_mat_vec. Fast path (fp4 tensor cores): ncols 1, K % 512 == 0,
 *       the buffer 16-byte aligned; otherwise a CUDA-core kernel. Scratch is
 *       stream-ordered, from the default memory pool.
 * Returns 0 from q2_0_split_bytes and Q2_0_EINVAL from the others for N < 1,
 * N >= 2^31 or K not a positive multiple of 64. Device pointers, owned by the
 * caller.
 */
size_t q2_0_split_bytes(int64_t N, int64_t K);
int q2_0_split_layout(const void *w, void *dst, int64_t N, int64_t K, void *stream);
int q2_0_join_layout(const void *src, void *w, int64_t N, int64_t K, void *stream);
int q2_0_mul_mat_vec_split(const void *w, const float *x, float *y, int64_t N, int64_t K,
                           int ncols, void *stream);

/*
 * q2_0_mul_mat_id — expert mat-vec of a mixture-of-experts layer (ggml
 * mul_mat_id; the limitations paragraph of "WebGPU: add Q2_0 support" names
 * MUL_MAT_ID as not ported).
 *   w    n_expert Q2_0 matrices of N x K, one after another (expert e starts
 *        at byte e * N * K/64 * 18).
 *   x    F32 [n_tokens][n_x][K]: n_x = 1 (one vector per token, shared by its
 *        experts) or n_x = n_used (one vector per slot).
 *   ids  int32 [n_tokens][n_used], expert of each slot.
 *   y    F32 [n_tokens][n_used][N]:
 *        y[t][i][n] = sum_k W_{ids[t][i]}[n][k] * x[t][n_x == 1 ? 0 : i][k].
 * Bound: |y - exact| <= 1e-5 * sum_k |W x| + 1e-7, as q2_0_mul_mat_vec.
 * workspace: at least q2_0_mul_mat_id_workspace_size(K, n_tokens, n_x) bytes,
 * 256-byte aligned (the size is 0, and NULL allowed, off the fast path).
 * Fast path: K % 512 == 0 and w 16-byte aligned; otherwise a CUDA-core kernel.
 * Limits: n_expert * N < 2^31, n_tokens * n_used and n_tokens * n_x <= 65535.
 * An id outside [0, n_expert) leaves its slot's output unwritten and records
 * Q2_0_DEVERR_BAD_ID with info = the slot index t * n_used + i.
 * n_tokens == 0 is a no-op. All pointers are device memory owned by the caller.
 */
size_t q2_0_mul_mat_id_workspace_size(int64_t K, int64_t n_tokens, int64_t n_x);
int q2_0_mul_mat_id(const void *w, int64_t n_expert, int64_t N, int64_t K, const float *x,
                    int64_t n_x, const int32_t *ids, int64_t n_used, int64_t n_tokens, float *y,
                    void *workspace, size_t workspace_bytes, void *stream);

/*
 * q2_0_get_rows — gather rows of a Q2_0 table into F32, bit-exact.
 * Source: the get-rows shader of "WebGPU: add Q2_0 support" (copies rows of a
 * Q2_0 tensor out, 64 floats per block).
 *   table  n_rows x K Q2_0 matrix.  ids  int32 [n_ids] (repeats allowed).
 *   out    F32 [n_ids][K]: out[r][k] = f32(q - 1) * f32(d), the IEEE product
 *          (signed zeros kept).
 * An id outside [0, n_rows) leaves its output row unwritten and records
 * Q2_0_DEVERR_BAD_ID with info = its position r. n_ids == 0 is a no-op.
 */
int q2_0_get_rows(const void *table, int64_t n_rows, int64_t K, const int32_t *ids, int64_t n_ids,
                  float *out, void *stream);

/*
 * Group-128 Q2_0: 34-byte blocks of 128 weights (fp16 d, then eight
 * little-endian words of sixteen 2-bit codes; element 16w+i in bits 2i..2i+1
 * of word w; code q -> (q - 1) * d). Source: "Llama.cpp umí dvoubitový Q2_0 i
 * na kartách NVIDIA" (aisvetem.cz), "Šest procent, o která se vedl spor" (34
 * bytes per 128 weights) and its closing section (Q2_0.gguf files without the
 * _g64 suffix use this packing). The pages fix only the size; the word layout
 * is the 64-weight block's, extended. K % 128 == 0 for all three calls.
 *
 * q2_0_g128_to_g64 — exact repack: src is an nrows x K group-128 matrix
 * (nrows*K/128*34 bytes), dst (nrows*K/64*18 bytes, written) the same matrix in
 * the 64-weight layout: block i becomes blocks 2i and 2i+1 with i's scale and
 * its code bytes 0..15 and 16..31. Every q2_0_* call then applies to dst.
 */
int q2_0_g128_to_g64(const void *src, void *dst, int64_t nrows, int64_t K, void *stream);

/* q2_0_g128_get_rows — as q2_0_get_rows over a group-128 table, bit-exact. */
int q2_0_g128_get_rows(const void *table, int64_t n_rows, int64_t K, const int32_t *ids,
                      int64_t n_ids, float *out, void *stream);

/* q2_0_g128_mul_mat_vec — as q2_0_mul_mat_vec over a group-128 matrix, for
 * callers that keep the 128-weight packing. ncols = 1 with K % 1024 == 0 and w
 * 16-byte aligned runs the fp4 tensor-core kernel directly on the 34-byte
 * blocks (one 272-byte box per row and 1024 weights; activations scaled per
 * 128 elements), with scratch of 1024 + K/1024 * 8320 bytes (256-aligned) from
 * the device's default memory pool on `stream`; its bound is the ncols = 1 one
 * with M_b the largest |x| of the 128-element block. Other shapes run on CUDA
 * cores (f32, the same error bound as the CUDA-core mat-vec) without scratch. */
int q2_0_g128_mul_mat_vec(const void *w, const float *x, float *y, int64_t N, int64_t K, int ncols,
                         void *stream);

/*
 * q2_0_quantize_ref — the reference quantizer, bit-exact.
 * Source: "Llama.cpp umí dvoubitový Q2_0 i na kartách NVIDIA" (aisvetem.cz),
 * section "Na běžný model to není": the block's largest |w| is the scale and
 * each weight is rounded to the nearest of the four levels.
 *   src  F32 [nrows][K] (finite).  dst  nrows x K Q2_0 matrix (written).
 * Per block: amax = max |w|; d = fp16(amax) rounded to nearest even; code 2 if
 * 2w >= amax, code 0 if 2w <= -amax, else code 1 (ties away from zero; the
 * decisions use the unrounded amax); amax == 0 gives d = 0 and code 1.
 */
int q2_0_quantize_ref(const float *src, void *dst, int64_t nrows, int64_t K, void *stream);

/* ---- decode step on a paged key/value cache ---------------------------------
 * The operators between a decoder's products: rotated keys and values appended
 * to a paged cache, attention of sequences that share a prefix, and a beam
 * search's selection and reordering on the same pages. (The Q2_0 pages have no
 * counterpart; these calls take the F32 outputs of the mat-vec and GEMM calls
 * and give F16 or BF16 activations.)
 */

/* Element type of a cache and of the activations that go with it. */
typedef enum q2_0_type { Q2_0_TYPE_F16 = 0, Q2_0_TYPE_BF16 = 1 } q2_0_type;

/* Which elements of a head a position turns together, rot of them in all:
 * HALVES (i, i + rot/2), PAIRS (2i, 2i + 1), i < rot/2. Elements from rot on
 * are left as they are. */
typedef enum q2_0_rope { Q2_0_ROPE_HALVES = 0, Q2_0_ROPE_PAIRS = 1 } q2_0_rope;

/*
 * A paged key/value cache: two device arrays of the same layout,
 * [n_layers][n_pages][n_kv][page][dim], owned by the caller. A page holds
 * `page` tokens of every kv head of one layer; a sequence's tokens lie in the
 * pages that its row of a page table names, token t in page table[t / page] at
 * place t % page (the same page ids in every layer). The struct is read during
 * the call (or plan_create) it is given to and not kept.
 *   k, v 16-byte aligned; dim 64 or 128; page 16, 32, 64, 128 or 256; type a
 *   q2_0_type; n_kv <= 65536, n_layers * n_pages * n_kv * page < 2^31 (byte offsets are 64-bit).
 */
typedef struct q2_0_kv_cache {
    void *k;
    void *v;
    int64_t n_pages;
    int n_layers;
    int n_kv;
    int page;
    int dim;
    int type;
} q2_0_kv_cache;

/*
 * q2_0_kv_append — rotates q and k by their tokens' positions, and stores k and
 * v in one layer of the cache.
 *   q, k, v   F32, token t's heads [n_q or n_kv][dim] at q + t * q_stride (strides
 *             in floats, >= heads * dim; so the three may be slices of one
 *             product's rows). n_q <= 65536; q and q_out may be NULL with n_q = 0.
 *   pos       int32 [n_tokens], the row of `rope` that turns the token.
 *   slot      int32 [n_tokens], the token's place in its sequence's row of
 *             `table`; a negative slot stores nothing (padding), q is still
 *             written.
 *   seq       int32 [n_tokens], the row of `table` [n_seq][width] of the
 *             token's sequence; NULL: token t belongs to row t (n_tokens <= n_seq).
 *   rope      F32 [n_pos][rot]: the cosines of the rot/2 angles of a position,
 *             then their sines. rot even, 0..dim; rot = 0: nothing turns, and
 *             rope and pos may be NULL.
 *   q_out     [n_tokens][n_q][dim] in the cache's type.
 * (a, b) -> (a c - b s, a s + b c) in f32, each rounded once to the cache's
 * type. No two tokens of a call may name the same place. A position, sequence,
 * table column or page id that is out of range stores nothing of its token
 * (q_out, k and v stay unwritten) and records Q2_0_DEVERR_BAD_ID with info = t.
 * n_tokens == 0 is a no-op.
 */
int q2_0_kv_append(const q2_0_kv_cache *cache, int layer, const float *q, int64_t q_stride,
                   const float *k, int64_t k_stride, const float *v, int64_t v_stride,
                   int64_t n_tokens, int n_q, const int32_t *pos, const int32_t *slot,
                   const int32_t *seq, const int32_t *table, int64_t n_seq, int64_t width,
                   const float *rope, int64_t n_pos, int rot, int style, void *q_out,
                   void *stream);

/*
 * Decode attention of n_groups * n_seq sequences, one query token each, over a
 * paged cache. The sequences of a group (b / n_seq) share a prefix, whose keys
 * and values are read once for all of them; each goes on with tokens of its own:
 *   out[b][h] = sum_t softmax_t(scale * q[b][h] . k_t) v_t, t over the first
 *   prefix_len[b / n_seq] tokens of the group's prefix_table row, then over the
 *   first len[b] tokens of b's table row; query head h reads kv head
 *   h / (n_q / n_kv). Where both lengths are 0 the output is 0. A prefix need
 *   not end with a page: the places past a length are never used, whatever
 *   they hold.
 *   q, out    [n_groups * n_seq][n_q][dim] in the cache's type, 16-byte aligned;
 *             n_q a multiple of n_kv, <= 65535, n_q / n_kv <= 64; n_groups * n_seq <= 65535,
 *             n_groups * n_seq * n_q <= 2^28.
 *   prefix_table int32 [n_groups][prefix_width], prefix_len int32 [n_groups]:
 *             both NULL with prefix_width = 0 where nothing is shared.
 *   table     int32 [n_groups * n_seq][width], len int32 [n_groups * n_seq].
 *   Tables and lengths are read at each execute: a decode loop updates them on
 *   the device, and one captured execute serves all its steps.
 * Precision: scores, softmax sums and output sums are f32; each weight
 * exp(score - reference) enters its product with v rounded to the cache's type
 * (2^-11 or 2^-8 of itself; an F16 weight below 2^-21 of its row's largest by
 * 2^-32 of that at most, F16 having a fixed spacing there), and so is the output: it is
 * within u (sum p|v| + |out|), F16: + 2^-32 sum |v|, and f32 rounding of the exact
 * one, u that rounding, p the softmax weights and the sums over the row's keys. Scores
 * have to be finite in f32; BF16 values of v above 2^90 may overflow on the way.
 * A length outside [0, width * page] is taken as the nearer bound, and a page
 * id outside [0, n_pages) as page 0; both record Q2_0_DEVERR_BAD_ID with info =
 * the sequence (or n_groups * n_seq + the group).
 * q2_0_attn_plan_create keeps the pointers, encodes the TMA descriptors and
 * allocates the plan's scratch; q2_0_attn_plan_execute runs one layer on
 * `stream` (two launches: the attention and the join of its parts; three where a
 * prefix is shared by more than 64 query heads of a kv head), allocates nothing and may be captured in a CUDA graph. The plan
 * belongs to the device current at creation; executes of one plan must not
 * overlap on the GPU (they share its scratch). Destroy it after the last
 * execute has completed.
 */
typedef struct q2_0_attn_desc {
    q2_0_kv_cache cache;
    const void *q;
    void *out;
    int64_t n_groups;
    int64_t n_seq; /* sequences of a group */
    int n_q;
    float scale;
    const int32_t *prefix_table;
    const int32_t *prefix_len;
    int64_t prefix_width;
    const int32_t *table;
    const int32_t *len;
    int64_t width;
} q2_0_attn_desc;

typedef struct q2_0_attn_plan q2_0_attn_plan;

int q2_0_attn_plan_create(const q2_0_attn_desc *desc, q2_0_attn_plan **plan);
int q2_0_attn_plan_execute(const q2_0_attn_plan *plan, int layer, void *stream);
/* Number of kernel launches one execute performs. */
int q2_0_attn_plan_launches(const q2_0_attn_plan *plan);
void q2_0_attn_plan_destroy(q2_0_attn_plan *plan);

/*
 * q2_0_beam_select — the selection step of a beam search: of each group's
 * n_beams * n_vocab continuations, the n_out with the highest scores.
 *   logits    F32, row (group, beam) at logits + (group * n_beams + beam) *
 *             stride, n_vocab values (stride >= n_vocab, in floats). -inf and
 *             NaN: the token may not be chosen and has no weight. +inf counts
 *             as the largest finite value.
 *   score     F32 [n_groups][n_beams], the beams' sums of log probabilities;
 *             a beam of score -inf (or NaN) is not continued.
 *   done      uint8 [n_groups][n_beams] or NULL: a finished beam (non-zero) has
 *             one continuation, token done_token at its own score.
 * A continuation's score is score + (x - lse) in f32, lse = m + log(sum exp(x -
 * m)) of its row. Order: higher score first; among equals the lower beam, then
 * the larger logit, then the lower token.
 *   score_out, parent, token   F32, int32, int32 [n_groups][n_out]. Where fewer
 *             than n_out continuations are possible the rest have score -inf,
 *             parent 0 and token -1. They must not overlap the inputs.
 *   1 <= n_beams <= 64, 1 <= n_out <= 32, 1 <= n_vocab < 2^31 - 2^16,
 *   n_groups * n_beams <= 65535. n_groups == 0 is a no-op.
 * workspace: at least q2_0_beam_select_workspace_size(...) bytes of device
 * memory, 256-byte aligned, or NULL to take it from the device's default memory
 * pool on `stream`.
 */
size_t q2_0_beam_select_workspace_size(int64_t n_groups, int n_beams, int64_t n_vocab, int n_out);
int q2_0_beam_select(const float *logits, int64_t stride, const float *score, const uint8_t *done,
                     int done_token, int64_t n_groups, int n_beams, int64_t n_vocab, int n_out,
                     float *score_out, int32_t *parent, int32_t *token, void *workspace,
                     size_t workspace_bytes, void *stream);

/*
 * q2_0_beam_reorder — the page tables follow the selection. New beam j of a
 * group goes on from the group's old beam p = parent[j]:
 *   table_out[j] = table[p], len_out[j] = len[p], and the page that the next
 *   token goes to becomes j's own: where len is a multiple of the page size,
 *   table_out[j][len / page] = fresh[j] (if that column exists); otherwise the
 *   first child of p keeps p's last page, and each further one gets fresh[j] with
 *   the first len % page tokens of that page copied, in all layers. Full pages
 *   are shared. used[j] = 1 where fresh[j] went into the table, else 0.
 *   parent int32 [n_groups][n_beams] (index in the group); table, table_out
 *   int32 [n_groups * n_beams][width]; len, len_out, fresh, used int32
 *   [n_groups * n_beams]. Inputs and outputs must not overlap; the pages in
 *   fresh are distinct and named by no row of table; a beam's last, partly
 *   filled page is in no other row.
 * A parent, a length (outside [0, width * page]) or a page id of a copy that is
 * out of range leaves beam j's outputs unwritten, copies nothing and records
 * Q2_0_DEVERR_BAD_ID with info = j. n_groups == 0 is a no-op;
 * n_beams <= 1024, n_groups * n_beams < 2^31.
 */
int q2_0_beam_reorder(const q2_0_kv_cache *cache, const int32_t *parent, int64_t n_groups,
                      int n_beams, const int32_t *table, const int32_t *len, int64_t width,
                      const int32_t *fresh, int32_t *table_out, int32_t *len_out, int32_t *used,
                      void *stream);

/* ---- steps of a serving loop around the products ------------------------------
 * Which experts a token goes to, which drafted tokens stand, and what becomes of
 * the pages of the cache above. (The Q2_0 pages have no counterpart.)
 */

/* How a router's logits become scores. */
typedef enum q2_0_score { Q2_0_SCORE_SOFTMAX = 0, Q2_0_SCORE_SIGMOID = 1 } q2_0_score;

/*
 * q2_0_moe_route — the experts of each token, as q2_0_mul_mat_id takes them (up to
 * 65535 slots a call; a prompt of more in several), and their weights.
 *   s = softmax(x) over the n_expert logits, or sigmoid(x); key = s + bias.
 *   With n_group_used < n_group the experts are n_group runs of n_expert / n_group;
 *   a group's score is the sum of its group_top (1 or 2) highest keys, and only the
 *   n_group_used groups of the highest scores are chosen from.
 *   ids[t] are the n_used experts of the highest keys, highest first; weights[t]
 *   their s (without the bias), divided by their sum if norm, times scale.
 * Equal keys and equal groups: the lower index first. Without a bias the logits
 * are compared in the keys' place (scores grow with them, and may round to the
 * same value); keys with a bias, and sums of two, are compared in 64 bits where
 * 32 do not decide.
 * A logit of -inf or NaN, or a bias of either, masks its expert: it adds nothing
 * to its group, comes after all others, by index, and has weight 0 (so that ids
 * are always n_used different experts). +inf counts as the largest finite value.
 * (A large finite bias in a mask's place, as -1e9, makes every row take many times
 * as long.)
 *   logits   F32, token t's row at logits + t * stride (stride >= n_expert).
 *   ids      int32 [n_tokens][n_used].   weights  F32 [n_tokens][n_used]. They must
 *            not overlap the inputs or each other.
 *   bias     F32 [n_expert] or NULL; read at each call.
 *   1 <= n_expert <= 1024, 1 <= n_used <= 32, n_group a divisor of n_expert,
 *   1 <= n_group <= 32, 1 <= n_group_used <= n_group, n_used <= n_group_used *
 *   (n_expert / n_group), scale finite, n_tokens < 2^31. n_tokens == 0 is a no-op.
 * Weights are within 2^-17 of themselves, and scale * 2^-126 where a score is that small.
 */
typedef struct q2_0_router {
    int n_expert;
    int n_used;
    int score; /* q2_0_score */
    int n_group;
    int n_group_used;
    int group_top;
    int norm;
    float scale;
    const float *bias;
} q2_0_router;

int q2_0_moe_route(const q2_0_router *router, const float *logits, int64_t stride, int64_t n_tokens,
                   int32_t *ids, float *weights, void *stream);

/*
 * q2_0_draft_verify — which of a sequence's drafted tokens the target model keeps,
 * and the token that follows them.
 *   target  F32 probabilities of the target model, row (b, i) at target + (b *
 *           (n_draft + 1) + i) * target_stride: of the token that draft i of
 *           sequence b proposes; the last of a sequence's rows that is used is that
 *           of the token behind its last draft.
 *   draft   the draft model's, row (b, i) at draft + (b * n_draft + i) *
 *           draft_stride; NULL: the drafts were certain (a greedy model, a lookup).
 *   tokens  int32 [n_seq][n_draft].   count  int32 [n_seq], the drafts of each
 *           sequence (0..n_draft), or NULL: n_draft of each.
 *   rand    F32 [n_seq][n_draft + 1], from [0, 1): the i-th decides on draft i, the
 *           last one draws the token.
 * Draft i stands if all before it do and rand_i q(d) < p(d) (one f32 product; q = 1
 * without draft). accepted[b] = a drafts stand. The next token is drawn from w =
 * max(p - q, 0) (f32) of row a if draft a was rejected (without draft: p with the
 * rejected token left out), else from w = p of row count[b]: the first token with
 * w > 0 whose running sum exceeds r * total, r the last number of rand; the last
 * token with w > 0 if none does. Where all w are 0 it is drawn from p; where that
 * is all 0 too it is -1. Running sums are held, and compared with r * total, to
 * within 2^-38 + n_vocab * 2^-58 of the total, and 2^-149. A negative probability and
 * NaN count as 0; rows need not sum to 1, but their sums have to be finite in f32
 * (otherwise any token of the row, or -1, is drawn).
 *   accepted int32 [n_seq].   token  int32 [n_seq][n_draft + 1]: the drafts that
 *   stand, the next token, then -1. They must not overlap the inputs or
 *   each other.
 * A count outside 0..n_draft, or a drafted token outside the vocabulary among a
 * sequence's drafts, leaves its outputs unwritten and records Q2_0_DEVERR_BAD_ID
 * with info = b.
 *   0 <= n_draft <= 1024, 1 <= n_vocab < 2^31 - 2^16, strides >= n_vocab, n_seq <=
 *   65535. With n_draft == 0 tokens and draft may be NULL. n_seq == 0 is a no-op.
 */
int q2_0_draft_verify(const float *target, int64_t target_stride, const float *draft,
                      int64_t draft_stride, const int32_t *tokens, const int32_t *count,
                      const float *rand, int64_t n_seq, int n_draft, int64_t n_vocab,
                      int32_t *accepted, int32_t *token, void *stream);

/*
 * Rows of pages: the sequences of a cache, with counts of who holds a page.
 *   refs   int32 [n_pages]: how many places of the table name the page; 0: free.
 *   table  int32 [n_rows][width]; row r holds the pages of its first
 *          ceil(len[r] / page) places, the others are not read.
 *   len    int32 [n_rows], tokens.
 * Table and len are as q2_0_attn_plan_create and q2_0_kv_append take them. Pages
 * that other arrays name as well (a shared prefix's table) are held by a row of
 * their own. The struct is read during the call and not kept; the calls below keep
 * refs true to the table.
 *   1 <= n_rows <= 2^20, 1 <= width, width * page < 2^31.
 * rows_out is where a call leaves its outcome: NULL or the same arrays, in place; or
 * other arrays of the same sizes that overlap nothing (each of the three by itself),
 * e.g. while attention in flight still reads the old ones, and what their rows hold
 * in the cache: q2_0_kv_fork writes no page, q2_0_kv_compact only pages that were
 * free. q2_0_kv_resize also writes pages that are given back in it: attention on old
 * rows that give pages back has to end before the call, on others it may go on until
 * something is appended.
 * The three arrays must not overlap one another, and a call's other arrays and its
 * workspace not those that it writes, nor, but for the arrays of q2_0_kv_fork, the
 * cache's pages: Q2_0_EINVAL. Rows must not lie in the cache's pages either (that is
 * not checked). The calls below must not overlap one another on the GPU
 * where they have rows, pages or a workspace in common.
 */
typedef struct q2_0_kv_rows {
    int32_t *refs;
    int32_t *table;
    int32_t *len;
    int64_t n_rows;
    int64_t width;
} q2_0_kv_rows;

/*
 * q2_0_kv_copy — copies pages src[i] to pages dst[i], in all layers, keys and
 * values: their first count[i] tokens (NULL: all of them).
 *   src, dst, count  int32 [n]. A page may be copied to several, but must be the
 *   destination of one copy at most, and not a source as well. A negative src[i]
 *   copies nothing (padding). The arrays must not lie in the cache's pages.
 * A page id outside [0, n_pages) or a count outside [0, page] copies nothing and
 * records Q2_0_DEVERR_BAD_ID with info = i. n == 0 is a no-op; n < 2^31.
 */
int q2_0_kv_copy(const q2_0_kv_cache *cache, const int32_t *src, const int32_t *dst,
                 const int32_t *count, int64_t n, void *stream);

/*
 * q2_0_kv_fork — row child[j] goes on from row parent[j]: it has its length and
 * holds the same pages, a partly filled last one too (q2_0_kv_resize parts them
 * before a row writes there). Nothing is copied in the cache.
 *   parent, child  int32 [n], n <= 4096.
 * A child has to be an empty row (len 0); of those that name the same one the lowest
 * j has it. A j that names another one's parent as its child, or another's child as its
 * parent, or a row, a length (outside [0, width * page]) or a page id of the parent
 * out of range, changes nothing, as one without a child does, and records
 * Q2_0_DEVERR_BAD_ID with info = j. n == 0 changes nothing (rows_out is written).
 */
int q2_0_kv_fork(const q2_0_kv_cache *cache, const q2_0_kv_rows *rows, const int32_t *parent,
                 const int32_t *child, int64_t n, const q2_0_kv_rows *rows_out, void *stream);

/*
 * q2_0_kv_resize — gives each row the length new_len[r], and the pages for it.
 * Rows that shrink (to 0: end) give back the pages behind their new length, -1 in
 * the table. Rows that grow get pages, and a row whose last kept page (that of
 * token min(len, new_len)) is filled in part and held by others too gets a page of
 * its own in its place, with the filled places copied in all layers; where all
 * holders of such a page end in it, the lowest row keeps it. Nothing else is written
 * to the cache.
 * Pages given back count as free. The lowest free pages are taken in the order of
 * the rows; of a row's pages that of the copied one comes first. A row whose pages
 * would reach behind the last free one gets none (nor do later rows that need one,
 * nor the row that was to keep the last page of one of these): its length is min(len,
 * new_len), its last page stays shared, nothing may be appended to it, and
 * Q2_0_DEVERR_NO_PAGES is recorded with info = a row of that kind; a later call may
 * serve it.
 * A length outside [0, width * page] or a partly filled last page outside
 * [0, n_pages) leaves its row as it is and records Q2_0_DEVERR_BAD_ID with info = r,
 * and so does a page given back that is out of range (it is dropped).
 *   new_len  int32 [n_rows]; in place it may be len itself (last pages are parted, no
 *            length changes).
 * workspace: at least q2_0_kv_resize_workspace_size(n_pages, n_rows) bytes, 256-byte
 * aligned, or NULL to take it from the device's default memory pool on `stream`.
 */
size_t q2_0_kv_resize_workspace_size(int64_t n_pages, int64_t n_rows);
int q2_0_kv_resize(const q2_0_kv_cache *cache, const q2_0_kv_rows *rows, const int32_t *new_len,
                   const q2_0_kv_rows *rows_out, void *workspace, size_t workspace_bytes,
                   void *stream);

/*
 * q2_0_kv_compact — moves pages so that the live ones (refs > 0) are the first: with
 * n of them, the highest page goes to the lowest free place below n, the next one
 * to the next, until all lie below n, in all layers; refs and table follow.
 *   place  int32 [n_pages], written: where each page of before is now, -1 for free
 *          ones (for tables of the caller's own).
 *   live   int32 [1], written: n. Neither may lie in the cache's pages.
 * A length outside [0, width * page] leaves its row's table as it is, and a page id
 * outside [0, n_pages) its place; both record Q2_0_DEVERR_BAD_ID with info = the row.
 * workspace: at least q2_0_kv_compact_workspace_size(n_pages, n_rows) bytes, 256-byte
 * aligned, or NULL to take it from the device's default memory pool on `stream`.
 */
size_t q2_0_kv_compact_workspace_size(int64_t n_pages, int64_t n_rows);
int q2_0_kv_compact(const q2_0_kv_cache *cache, const q2_0_kv_rows *rows,
                    const q2_0_kv_rows *rows_out, int32_t *place, int32_t *live, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * q2_0_get_error — synchronises `stream`, then reads and clears the current
 * device's error word. Returns a Q2_0_DEVERR_* code; *info (if not NULL)
 * receives its detail. Returns -1 if the read itself failed.
 */
int q2_0_get_error(void *stream, int64_t *info);

/*
 * q2_0_test_inject_stall — TEST ONLY: exercises the bounded pipeline waits.
 * (No counterpart on the pages: the failure-detection path of this library.)
 * The next fp4 mat-vec launch on the current device (ncols 1 or 2 on the
 * tensor-core path: q2_0_mul_mat_vec, _ws, _noalloc, _f16, a plan; ncols 1:
 * _split or q2_0_mul_mat_id) stops feeding its pipeline before pipeline stage `stage`
 * of each CTA (0 = the first), and every pipeline wait of that launch gives up
 * after wait_limit_ns instead of about one second. The consumers' waits on
 * the missing stage then run out: the kernel records Q2_0_DEVERR_TIMEOUT with
 * info 111 (the wait for a stage's copies), lets the copies it issued land,
 * frees its tensor memory and returns; its outputs are incomplete. Later
 * launches are unaffected. Returns Q2_0_EINVAL for stage < 0 or a limit of 0
 * or above 10 s.
 */
int q2_0_test_inject_stall(int stage, uint64_t wait_limit_ns);

/*
 * q2_0_test_stall_attention — TEST ONLY, the same for attention: each block of the
 * next q2_0_attn_plan_execute on the current device stops copying keys about
 * `tiles` tiles into its share (0: at once), 0 <= tiles <= 2^20. The waits for them
 * run out after their usual second, Q2_0_DEVERR_TIMEOUT is recorded with info 301 to
 * 314, and the outputs are incomplete.
 */
int q2_0_test_stall_attention(int tiles);

#ifdef __cplusplus
}
#endif

#endif /* Q2_0_H */
