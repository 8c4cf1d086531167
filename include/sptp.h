/*
 * sptp.h -- C ABI of the GB300 (sm_103a) SP-TP FFN boundary library (libsptp.so).
 *
 * The library computes the sequence-parallel tensor-parallel (SP-TP) FFN
 * sub-layer boundary of a Megatron-style transformer with the P tensor-parallel
 * shards held as P buffers on ONE GPU, and a Delayed-TP stack of FFN sub-layers.
 *
 * Sources (web pages, by title and section):
 *   [A] "[Feature] Async Tensor Parallelism for Archon Engine",
 *       "TP Communication Is on Activations, Not Weights" and "Potential
 *       Solution" (chunked all-gather + matmul; the boundary reduce-scatter ->
 *       residual add + RMSNorm -> all-gather; norm(all_gather(x)) ==
 *       all_gather(norm(x))).
 *   [B] "Affinity-Aware Sharding for Delayed Tensor Parallelism", Abstract
 *       (Delayed TP; contiguous neuron sharding).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers on the current CUDA device,
 *     row-major and densely packed unless stated.  The caller owns every
 *     buffer; the library allocates no memory and keeps no data between calls.
 *   - Element type is given by `dtype` (sptp_dtype): SPTP_BF16 (compute in
 *     fp32, store bf16; tcgen05 tensor-core GEMMs) or SPTP_FP32 (fp32
 *     throughout; CUDA-core GEMMs).  `gamma` and all weights use the same type.
 *   - Weights use the [out][in] layout: W1g, W1u are [F][d], W2 is [d][F].
 *     Shard p owns neurons F_p = [p*F/P, (p+1)*F/P): rows F_p of W1g/W1u and
 *     columns F_p of W2 ([B], contiguous layout).
 *   - Work is enqueued asynchronously on `cuda_stream` (a cudaStream_t; NULL
 *     is the legacy default stream).  Nothing is synchronised.
 *   - Errors are returned as negative sptp_status codes; argument errors are
 *     detected before any CUDA call, so an error leaves all buffers untouched.
 *     SPTP_ERR_CUDA reports a launch failure.  A device-side wait that runs
 *     out (see sptp_read_device_status) is reported through the workspace.
 *   - Shape rules: M >= 0 (M == 0 is a no-op that returns SPTP_OK; the
 *     activation pointers may then be NULL), d >= 8,
 *     d % 8 == 0, d <= 16384; F > 0, F % P == 0, (F/P) % 8 == 0;
 *     1 <= P <= 8.  (Multiples of 8 keep every row 16-byte aligned.)
 *   - Pointers must be 16-byte aligned.
 */
#ifndef SPTP_H
#define SPTP_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* In C++ the enums get int as their underlying type, so that every int a C
 * caller passes is a valid value (and is rejected by the checks below rather
 * than being undefined). */
#ifdef __cplusplus
#define SPTP_ENUM_INT : int
#else
#define SPTP_ENUM_INT
#endif

/* Element type of activations, gamma and weights. */
typedef enum sptp_dtype_e SPTP_ENUM_INT { SPTP_BF16 = 0, SPTP_FP32 = 1 } sptp_dtype;

typedef enum sptp_status_e SPTP_ENUM_INT {
    SPTP_OK = 0,
    SPTP_ERR_NULL = -1,          /* a required pointer is NULL */
    SPTP_ERR_SHAPE = -2,         /* a size or divisibility rule is violated */
    SPTP_ERR_DTYPE = -3,         /* dtype is not an sptp_dtype */
    SPTP_ERR_WORKSPACE = -4,     /* ws_bytes smaller than the *_workspace_size query */
    SPTP_ERR_CUDA = -5,          /* a CUDA runtime call or kernel launch failed */
    SPTP_ERR_TIMEOUT = -6,       /* a bounded device-side wait ran out */
    SPTP_ERR_UNIMPLEMENTED = -7, /* the requested variant does not exist for this entry point and
                                    dtype, or this device cannot run its launch */
    SPTP_ERR_ALIAS = -8,         /* an output overlaps an input it must not overlap */
    SPTP_ERR_TOO_LARGE = -9,     /* the problem needs more scratch than the library's static array */
    SPTP_ERR_DEVICE = -10,       /* current device is not compute capability 10.3 */
    SPTP_ERR_BOUNDS = -11        /* bounds-checked builds only: a kernel computed an index or address
                                    outside its buffer and skipped the access */
} sptp_status;

/*
 * sptp_variant -- how a boundary call is split into launches.  Every
 * variant computes the same outputs; they differ in how the partial sum +
 * residual + RMSNorm rows reach the GEMMs.  SPTP_VARIANT_AUTO is the
 * library's default for the entry point and dtype; any other value runs
 * exactly that variant or returns SPTP_ERR_UNIMPLEMENTED (nothing enqueued)
 * where it does not exist or this device cannot co-schedule its launch.
 *   PAIR    (sptp_ffn_forward, sptp_attn_qkv_forward; bf16 and fp32) the
 *           prologue kernel over all M rows, then the GEMM launches (bf16:
 *           tcgen05 CTA-pair GEMMs; fp32: CUDA-core GEMMs).  The default.
 *   CHAIN   (sptp_ffn_forward, bf16) the prologue kernel, then ONE persistent
 *           launch running every gate/up tile and then every down tile; a
 *           down tile starts as soon as the gate/up tiles of its rows are
 *           stored.
 *   FUSED   (sptp_ffn_forward, sptp_attn_qkv_forward, dtp_ffn_stack_forward;
 *           bf16) ONE persistent launch: prologue warps produce the normed
 *           rows in sequence order, 256-row block by block, and the GEMM tiles
 *           consume each block as soon as it is published (the chunked
 *           all-gather + matmul of [A] "Potential Solution", literally).  The
 *           default of dtp_ffn_stack_forward for bf16.
 *   LAYERS  (dtp_ffn_stack_forward) a prologue launch and two GEMM launches
 *           per module.  The default for fp32, and for bf16 where FUSED
 *           cannot be launched.
 */
typedef enum sptp_variant_e SPTP_ENUM_INT {
    SPTP_VARIANT_AUTO = 0,
    SPTP_VARIANT_PAIR = 1,
    SPTP_VARIANT_CHAIN = 2,
    SPTP_VARIANT_FUSED = 3,
    SPTP_VARIANT_LAYERS = 4
} sptp_variant;

/* Bytes at the start of every workspace holding the device status words. */
#define SPTP_WS_HEADER_BYTES 4096

/* Workspace bytes needed by sptp_ffn_forward for these sizes (0 on bad args).
 * Layout: header | y [M][d] normed activations | s [P][M][F/P] SwiGLU output. */
size_t sptp_ffn_workspace_size(int M, int d, int F, int P, int chunks, sptp_dtype dtype);

/*
 * sptp_ffn_forward -- one SP-TP FFN sub-layer boundary ([A] "Potential
 * Solution", sub-layer boundary overlap; intra-layer chunked all-gather +
 * matmul).  For every token row t:
 *     r       = sum_{p=0}^{P-1} partials[p][t]      (reduce-scatter arithmetic)
 *     h       = x[t] + r                            (residual add)
 *     y       = h * gamma / sqrt(mean_j h_j^2 + eps) (RMSNorm)
 *   and for every shard p (chunk c of y, rows [c*M/chunks, (c+1)*M/chunks),
 *   is gathered to all shards; on one GPU the gather is the identity):
 *     s_p     = silu(y W1g[F_p]^T) * (y W1u[F_p]^T)  (column-parallel, SwiGLU)
 *     out[p]  = s_p W2[:, F_p]^T                    (row-parallel partial)
 *
 *   x         [M][d]    residual stream in
 *   partials  [P][M][d] the previous sub-layer's row-parallel partials
 *   gamma     [d]       RMSNorm scale
 *   W1g, W1u  [F][d]    gate / up projections;  W2 [d][F] down projection
 *   chunks    number of sequence chunks of the all-gather; M % chunks == 0,
 *             chunks % P == 0.  Chunk c is rows [c*M/chunks, (c+1)*M/chunks)
 *             and belongs to shard floor(c*P/chunks).  With
 *             SPTP_VARIANT_FUSED the gate/up tiles read a chunk's rows of y as
 *             soon as every row of the chunk is produced; the PAIR and CHAIN
 *             variants produce every chunk before the GEMMs start, so for
 *             them chunks changes nothing but the validation.
 *   out       [P][M][d] the next sub-layer's P partials (not reduced).  Must
 *             not overlap any input or the workspace.
 *   resid_out [M][d]    h, the new residual stream; may be NULL (not written)
 *             and may be exactly x (in place).
 *   workspace at least sptp_ffn_workspace_size(...) bytes, 256-byte aligned.
 * Numerics (bf16): sums, norm and SwiGLU in fp32; h, y, s and out are each
 * rounded once to bf16 (round to nearest even).  Every variant gives the same
 * bits.
 * sptp_ffn_forward runs SPTP_VARIANT_AUTO; sptp_ffn_forward_ex runs the
 * variant it is given (PAIR, CHAIN or FUSED; see sptp_variant).
 */
int sptp_ffn_forward(const void* x, const void* partials, const void* gamma,
                     const void* W1g, const void* W1u, const void* W2,
                     int M, int d, int F, int P, int chunks, float eps, sptp_dtype dtype,
                     void* out, void* resid_out,
                     void* workspace, size_t ws_bytes, void* cuda_stream);
int sptp_ffn_forward_ex(const void* x, const void* partials, const void* gamma,
                        const void* W1g, const void* W1u, const void* W2,
                        int M, int d, int F, int P, int chunks, float eps, sptp_dtype dtype,
                        void* out, void* resid_out,
                        void* workspace, size_t ws_bytes, void* cuda_stream, sptp_variant variant);

/* Workspace bytes needed by dtp_ffn_stack_forward (0 on bad args).
 * Layout: header | y [P][M][d] | s [P][M][F/P] | pending ring [S][P][M][d],
 * S = min(delta + 1, L). */
size_t dtp_ffn_stack_workspace_size(int M, int d, int F, int P, int L, int delta, sptp_dtype dtype);

/*
 * dtp_ffn_stack_forward -- a Delayed-TP stack of L FFN sub-layers ([B],
 * Abstract).  Shard p keeps its own residual stream x_p = x_shards[p].
 * Module l on shard p computes o_p^(l) = FFN_l,p(RMSNorm_l(x_p)) with shard
 * p's neurons; shard p adds o_p^(l) to x_p at once, and another shard q's
 * o_q^(l) reaches x_p `delta` modules later (before module l + 1 + delta).
 * delta == 0 is standard TP.  After module L-1 each shard adds its own last
 * partial and the partials arriving then; `flush` != 0 also adds every
 * other-shard partial still pending.
 *
 *   x_shards [P][M][d]  in/out residual streams (updated in place)
 *   gamma    [L][d];  W1g, W1u [L][F][d];  W2 [L][d][F]
 *   delta >= 0; L >= 1; 1 + (P-1)*min(L, delta+1) <= 64.
 * Numerics (bf16): each stream update is summed in fp32 (own partial first,
 * then other shards in ascending shard order, then x_p) and rounded to bf16.
 * dtp_ffn_stack_forward runs SPTP_VARIANT_AUTO (FUSED for bf16 where the
 * device can run it, else LAYERS); dtp_ffn_stack_forward_ex runs the variant
 * it is given (FUSED or LAYERS).
 */
int dtp_ffn_stack_forward(void* x_shards, const void* gamma,
                          const void* W1g, const void* W1u, const void* W2,
                          int M, int d, int F, int P, int L, int delta, int flush,
                          float eps, sptp_dtype dtype,
                          void* workspace, size_t ws_bytes, void* cuda_stream);
int dtp_ffn_stack_forward_ex(void* x_shards, const void* gamma,
                             const void* W1g, const void* W1u, const void* W2,
                             int M, int d, int F, int P, int L, int delta, int flush,
                             float eps, sptp_dtype dtype,
                             void* workspace, size_t ws_bytes, void* cuda_stream, sptp_variant variant);

/* ---- Step-level entry points (the same kernels the two calls above use). ---- */

/*
 * sptp_prologue -- steps 1-3 of the boundary ([A] "Potential Solution"):
 * h = x + sum_p partials[p]; y = RMSNorm(h) * gamma.  h_out may be NULL or x.
 * y_out [M][d] must not overlap the inputs.
 */
int sptp_prologue(const void* x, const void* partials, const void* gamma,
                  int M, int d, int P, float eps, sptp_dtype dtype,
                  void* h_out, void* y_out, void* cuda_stream);

/*
 * sptp_gateup_swiglu -- column-parallel gate/up GEMM with the SwiGLU epilogue
 * for every shard ([A] "Potential Solution"): s[p] = silu(y W1g[F_p]^T) *
 * (y W1u[F_p]^T), s_out laid out [P][M][F/P].  workspace: at least
 * SPTP_WS_HEADER_BYTES (status words).
 */
int sptp_gateup_swiglu(const void* y, const void* W1g, const void* W1u,
                       int M, int d, int F, int P, sptp_dtype dtype, void* s_out,
                       void* workspace, size_t ws_bytes, void* cuda_stream);

/*
 * sptp_down_proj -- row-parallel down GEMM per shard ([A] "Potential
 * Solution"): out[p] = s[p] W2[:, F_p]^T with s [P][M][F/P], out [P][M][d].
 * Also the row-parallel output projection of an attention sub-layer (s = the
 * per-shard attention output, W2 = Wo [d][F]).  workspace: at least
 * SPTP_WS_HEADER_BYTES.
 */
int sptp_down_proj(const void* s, const void* W2, int M, int d, int F, int P, sptp_dtype dtype,
                   void* out, void* workspace, size_t ws_bytes, void* cuda_stream);

/* Workspace bytes needed by sptp_attn_qkv_forward (0 on bad args).
 * Layout: header | y [M][d]. */
size_t sptp_attn_qkv_workspace_size(int M, int d, int N, int P, int chunks, sptp_dtype dtype);

/*
 * sptp_attn_qkv_forward -- the sub-layer boundary in front of an attention
 * sub-layer ([A] "Potential Solution": 4 boundaries per block, between the
 * attention and FFN sub-layers both ways).  Steps 1-3 as in
 * sptp_ffn_forward (partial sum, residual add, RMSNorm), the (identity)
 * chunked gather, then each shard's column-parallel QKV projection:
 *     qkv_out[p] = y Wqkv[p*N/P .. (p+1)*N/P)^T
 *   Wqkv      [N][d]: shard p owns rows [p*N/P, (p+1)*N/P) (its heads' q, k
 *             and v rows, arranged by the caller); N % P == 0, (N/P) % 8 == 0
 *   qkv_out   [P][M][N/P]; resid_out, chunks, eps, dtype, workspace and the
 *   shape rules as in sptp_ffn_forward.
 * The row-parallel output projection after attention, which yields the next
 * P partials, is sptp_down_proj with F = the attention width (attn [P][M][F/P],
 * Wo [d][F]).
 * sptp_attn_qkv_forward runs SPTP_VARIANT_AUTO (PAIR); sptp_attn_qkv_forward_ex
 * runs the variant it is given (PAIR, or FUSED for bf16).
 */
int sptp_attn_qkv_forward(const void* x, const void* partials, const void* gamma, const void* Wqkv,
                          int M, int d, int N, int P, int chunks, float eps, sptp_dtype dtype,
                          void* qkv_out, void* resid_out,
                          void* workspace, size_t ws_bytes, void* cuda_stream);
int sptp_attn_qkv_forward_ex(const void* x, const void* partials, const void* gamma, const void* Wqkv,
                             int M, int d, int N, int P, int chunks, float eps, sptp_dtype dtype,
                             void* qkv_out, void* resid_out,
                             void* workspace, size_t ws_bytes, void* cuda_stream, sptp_variant variant);

/*
 * sptp_permute_ffn_neurons -- executes a neuron-permutation shard map for
 * Delayed TP ([B], Abstract: the dense model is permuted before it is
 * sharded; with delayed partials, which neurons share a device changes the
 * model).  For every module l and new neuron i, new neuron i is old neuron
 * perm[l][i]:
 *     W1g_out[l][i][:] = W1g[l][perm[l][i]][:],  W1u_out likewise,
 *     W2_out[l][:][i]  = W2[l][:][perm[l][i]].
 * Contiguous sharding of the outputs (dtp_ffn_stack_forward) then gives
 * shard p the old neurons perm[l][F_p].
 *   W1g, W1u [L][F][d];  W2 [L][d][F];  perm: DEVICE int32 [L][F], meant to
 *   be a permutation of 0..F-1 per module.  An entry outside [0, F) is
 *   recorded as SPTP_ERR_SHAPE in the workspace status words (see
 *   sptp_read_device_status) and its outputs are zero-filled.
 *   Outputs must not overlap the inputs or each other.  F*sizeof(dtype) <=
 *   200 KiB.  workspace: at least SPTP_WS_HEADER_BYTES.
 */
int sptp_permute_ffn_neurons(const void* W1g, const void* W1u, const void* W2, const int* perm,
                             int L, int d, int F, sptp_dtype dtype,
                             void* W1g_out, void* W1u_out, void* W2_out,
                             void* workspace, size_t ws_bytes, void* cuda_stream);

/* ---- fp8 (E4M3) linear layers ------------------------------------------------
 * [A] "Additional Information" names fp8 (MXFP8) linear layers inside
 * tensor-parallel blocks; the pages fix no scaling recipe.  This library's
 * reading: every linear quantises its bf16 input row-wise (rows along the
 * GEMM's reduction axis) to OCP E4M3 with a power-of-two scale, and its GEMM
 * accumulates in fp32 on tcgen05 (kind::f8f6f4) and dequantises in the
 * epilogue.  A power-of-two scale makes a * 2^-e exact, so the codes depend on
 * the bf16 values alone.
 */

/*
 * sptp_quantize_rows_e4m3 -- row-wise E4M3 quantisation of a bf16 [R][K]:
 *     e_r      = least integer >= -126 with max_k |a[r][k]| <= 448 * 2^e_r
 *     q[r][k]  = RNE_E4M3(a[r][k] * 2^-e_r)       (E4M3 bytes, [R][K])
 *     scale[r] = 2^e_r                            (fp32, [R])
 * The weights of sptp_ffn_forward_fp8 are quantised with it once: W1g and
 * W1u as [F][d] (R = F, K = d: one scale per neuron) and W2 as [d*P][F/P]
 * (R = d*P, K = F/P: one scale per output feature n and shard p, at index
 * n*P + p -- shard p quantises its own slice).
 *   R >= 0 (0 is a no-op), K > 0, K % 16 == 0; a and q 16-byte aligned,
 *   scale 4-byte aligned; q and scale must not overlap a or each other.
 *   Inputs must be finite (non-finite values are outside the contract).
 */
int sptp_quantize_rows_e4m3(const void* a, long long R, int K, void* q, float* scale,
                            void* cuda_stream);

/* Workspace bytes needed by sptp_ffn_forward_fp8 (0 on bad args).  Layout:
 * header | y bf16 [M][d] | qy [M][d] | sy [M] | s bf16 [P][M][F/P] |
 * qs [P][M][F/P] | ss [P][M], each part 256-byte aligned. */
size_t sptp_ffn_fp8_workspace_size(int M, int d, int F, int P, int chunks);

/*
 * sptp_ffn_forward_fp8 -- sptp_ffn_forward with fp8 linear layers (bf16
 * activations in and out).  Steps 1-3 as there (fp32 partial sum, residual
 * add, RMSNorm); y is the bf16 activation; then for every shard p:
 *     qy, sy = quantize_rows(y)                    (over d, one scale per token)
 *     a      = (qy qW1g[F_p]^T) * sy[t] * sW1g[n]   b likewise with W1u
 *     s_p    = bf16(silu(a) * b)
 *     qs, ss = quantize_rows(s_p)                  (over F/P, per token and shard)
 *     out[p] = bf16((qs qW2[:, F_p]^T) * ss[p][t] * sW2[n*P + p])
 *   x, partials, gamma, out, resid_out, chunks, eps: as in sptp_ffn_forward
 *   (bf16).  qW1g, qW1u [F][d] E4M3 with sW1g, sW1u [F] fp32; qW2 [d][F]
 *   E4M3 with sW2 [d][P] fp32: the outputs of sptp_quantize_rows_e4m3 above.
 *   Shape rules of sptp_ffn_forward plus d % 16 == 0 and (F/P) % 16 == 0.
 */
int sptp_ffn_forward_fp8(const void* x, const void* partials, const void* gamma,
                         const void* qW1g, const float* sW1g, const void* qW1u, const float* sW1u,
                         const void* qW2, const float* sW2,
                         int M, int d, int F, int P, int chunks, float eps,
                         void* out, void* resid_out,
                         void* workspace, size_t ws_bytes, void* cuda_stream);

/*
 * sptp_prologue_e4m3 -- steps 1-3 with the gate/up linear's quantisation of y
 * fused (one launch where a row's sources fit the kernel's shared-memory
 * ring; otherwise y is stored to y_work and quantised by a second launch):
 * h = x + sum_p partials[p]; y = bf16(RMSNorm(h) * gamma); q_out [M][d] and
 * scale_out [M] as sptp_quantize_rows_e4m3(y).  bf16 only; h_out may be NULL
 * or x; y_work [M][d] bf16 scratch (contents undefined afterwards); d % 16 == 0.
 */
int sptp_prologue_e4m3(const void* x, const void* partials, const void* gamma,
                       int M, int d, int P, float eps,
                       void* h_out, void* y_work, void* q_out, float* scale_out, void* cuda_stream);

/* The two fp8 GEMMs of sptp_ffn_forward_fp8 as separate launches:
 *   sptp_gateup_swiglu_e4m3: s_out [P][M][F/P] bf16 from qy [M][d], sy [M].
 *   sptp_down_proj_e4m3: out [P][M][d] bf16 from qs [P][M][F/P], ss [P][M].
 * Weights and scales as in sptp_ffn_forward_fp8; workspace: at least
 * SPTP_WS_HEADER_BYTES (status words). */
int sptp_gateup_swiglu_e4m3(const void* qy, const float* sy, const void* qW1g, const float* sW1g,
                            const void* qW1u, const float* sW1u, int M, int d, int F, int P,
                            void* s_out, void* workspace, size_t ws_bytes, void* cuda_stream);
int sptp_down_proj_e4m3(const void* qs, const float* ss, const void* qW2, const float* sW2,
                        int M, int d, int F, int P, void* out,
                        void* workspace, size_t ws_bytes, void* cuda_stream);

/* ---- Between the QKV projection and the output projection -------------------
 * sptp_attn_qkv_forward leaves every shard's q, k and v rows, sptp_down_proj
 * takes every shard's attention output; the calls below are the sub-layer
 * between them: rotary positions, a paged key-value cache, and the attention
 * of one new token per sequence over it.  The pages name the attention
 * sub-layer ([A] "Potential Solution") and leave its inside open.
 *
 * A shard's row of qkv_out holds its Hq query heads, then its Hkv key heads,
 * then its Hkv value heads, D elements each (N/P = (Hq + 2 Hkv) D): Hq and Hkv
 * count one shard's heads.  Query head h reads key/value head h / (Hq/Hkv).
 *
 * The cache: k_cache and v_cache [P][num_pages][Hkv][page_size][D], allocated
 * by the caller.  page_table [B][max_pages] (int32) names the pages of each
 * sequence, the same in every shard's pool: key j of sequence b is row
 * j % page_size of page page_table[b][j / page_size].  Only entries that a
 * call reaches are read.
 *   kv_type  SPTP_KV_SAME: elements of `dtype`; k_scale and v_scale unused.
 *            SPTP_KV_E4M3 (dtype SPTP_BF16): E4M3 codes, and k_scale, v_scale
 *            [P][num_pages][Hkv][page_size] fp32: a head's row of D elements
 *            quantised as by sptp_quantize_rows_e4m3.
 *   Shape rules of all of them: 1 <= P <= 8; D % 8 == 0 (E4M3: % 16),
 *   8 <= D <= 256; Hq % Hkv == 0; P * (Hq + 2 Hkv) < 2^24; M, B < 2^30;
 *   page_size % 16 == 0; max_pages * page_size < 2^30; P * num_pages * Hkv *
 *   page_size < 2^31.  M == 0 or B == 0 enqueues nothing.
 *   int32 arrays are 4-byte aligned, `turns` 8-byte, all others 16-byte.
 * Calls that may overlap on the GPU need a workspace each; calls in one stream,
 * or replays of graphs one after another, may share it.  Appends and attention
 * on one cache are ordered by the caller, as on any buffer.
 */

/* Element type of a key-value cache. */
typedef enum sptp_kv_type_e SPTP_ENUM_INT { SPTP_KV_SAME = 0, SPTP_KV_E4M3 = 1 } sptp_kv_type;

/*
 * sptp_rope_scaling -- how the frequencies f_i = theta^(-2i/rot) are changed
 * for contexts `factor` times as long as the model was trained on.
 *   NONE    f_i
 *   LINEAR  f_i / factor
 *   NTK     f_i of the base theta * factor^(rot/(rot-2))
 *   PARTS   c f_i + (1 - c) f_i / factor, c = clamp((r_i - alpha)/(beta - alpha), 0, 1)
 *           with r_i = orig_len * f_i / (2 pi), the turns that the pair makes
 *           over the original length: fast pairs are kept, slow ones scaled.
 */
typedef enum sptp_rope_scaling_e SPTP_ENUM_INT {
    SPTP_ROPE_NONE = 0,
    SPTP_ROPE_LINEAR = 1,
    SPTP_ROPE_NTK = 2,
    SPTP_ROPE_PARTS = 3
} sptp_rope_scaling;

/*
 * sptp_rope_turns -- the frequency table of the rotation, made once per model
 * on the HOST (no CUDA call): turns[i] = round(2^64 f_i / (2 pi)), i < rot/2,
 * in HOST memory; the caller copies it to the device.  A frequency in turns
 * per position, as a 64-bit binary fraction, makes position * turns (mod
 * 2^64) the angle without rounding, however far the position.
 *   rot % 16 == 0, 16 <= rot <= 256; theta > 1; factor >= 1 (ignored for
 *   NONE); PARTS: orig_len > 0 and beta > alpha (ignored for the others).
 *   SPTP_ERR_SHAPE otherwise, SPTP_ERR_UNIMPLEMENTED for another scaling.
 */
int sptp_rope_turns(int rot, double theta, sptp_rope_scaling scaling, double factor, double orig_len,
                    double alpha, double beta, unsigned long long* turns);

/*
 * sptp_rope -- rotary positions of the first Hr of H heads of every row:
 *     (a, b) -> gain * (a cos t - b sin t, a sin t + b cos t),
 *     t = 2 pi * positions[m] * turns[i] / 2^64
 *   for the pairs i < rot/2 of a head's first rot elements: elements (i,
 *   i + rot/2), or (2i, 2i + 1) if `interleaved`.  The other elements and
 *   heads are copied.  transpose != 0 applies the transposed matrix (t -> -t,
 *   the same gain): the gradient of the rotation with respect to x.
 *   x, out    [P][M][H][D]; out may be exactly x (then only rotated elements
 *             are written) and must not overlap it otherwise.
 *   positions [M] int32, any value, the same for every shard.
 *   turns     DEVICE [rot/2], from sptp_rope_turns.  rot % 16 == 0,
 *             16 <= rot <= D; 1 <= Hr <= H; P * H < 2^24.
 *   gain      finite: the attention factor of a scaled context (0.1 ln(factor)
 *             + 1 is usual with PARTS), or 1.
 * Numerics: angles to 2^-25 of a turn, products in fp32, rounded once.
 */
int sptp_rope(const void* x, const int* positions, const unsigned long long* turns,
              int P, int M, int H, int Hr, int D, int rot, int interleaved, int transpose, float gain,
              sptp_dtype dtype, void* out, void* cuda_stream);

/*
 * sptp_rope_append_kv -- the QKV rows of M new tokens, of any mix of
 * sequences: q rotated to q_out, k rotated and stored in the cache, v stored
 * in the cache.
 *   qkv       [P][M][(Hq + 2 Hkv) D], sptp_attn_qkv_forward's qkv_out
 *   positions [M] int32: a token's position, for the rotation and its slot
 *   seq_ids   [M] int32: its row of page_table; < 0 marks a padding row:
 *             nothing is stored for it, its row of q_out is left as it was
 *   rot       as in sptp_rope, or 0: no rotation, turns unused
 *   q_out     [P][M][Hq][D].  q_out and the cache must not overlap an input,
 *             the workspace or each other.
 * A token whose sequence is >= B, whose position is outside [0, max_pages *
 * page_size) or whose page is outside [0, num_pages) is recorded as
 * SPTP_ERR_SHAPE in the workspace status words; its k and v are not stored
 * (its q is).  What two tokens with one sequence and position leave in their
 * slot is not defined (it may be parts of both).  workspace: at least
 * SPTP_WS_HEADER_BYTES, 256-byte aligned.  E4M3: k is rounded to bf16, then
 * quantised; non-finite rows are outside the contract.
 */
int sptp_rope_append_kv(const void* qkv, const int* positions, const int* seq_ids, const int* page_table,
                        const unsigned long long* turns, int P, int M, int Hq, int Hkv, int D, int rot,
                        int interleaved, float gain, int B, int max_pages, int num_pages, int page_size,
                        sptp_dtype dtype, sptp_kv_type kv_type, void* q_out, void* k_cache, void* v_cache,
                        float* k_scale, float* v_scale, void* workspace, size_t ws_bytes, void* cuda_stream);

/* Workspace bytes needed by sptp_paged_attn_decode (0 on bad args). */
size_t sptp_paged_attn_workspace_size(int P, int B, int Hq, int Hkv, int D);

/*
 * sptp_paged_attn_decode -- attention of one token per sequence over its
 * cached keys and values:
 *     s_j = scale * q . k_j,  lse = ln sum_j e^s_j,  out = sum_j e^(s_j - lse) v_j
 *   over j < seq_lens[b], and j >= seq_lens[b] - window if window > 0.
 *   q         [P][B][Hq][D] (sptp_rope_append_kv's q_out for one token each)
 *   seq_lens  [B] int32: keys in the cache, the new token's included.  0
 *             gives a row of zeros and lse -inf.
 *   out       [P][B][Hq D], the row-parallel operand of sptp_down_proj
 *   lse       [P][B][Hq] fp32, or NULL
 *   out and lse must not overlap an input, the workspace or each other.
 * The work is split over the length as well, evenly over the SMs whatever the
 * lengths, and the parts of a row are joined in a fixed order: equal inputs
 * give equal bits.  A row's result does not depend on what the cache holds
 * behind its length or before its window.
 * A length outside [0, max_pages * page_size] is cut to it, a page outside
 * [0, num_pages) counts as zero keys and values; both are recorded as
 * SPTP_ERR_SHAPE in the workspace status words.  workspace: at least
 * sptp_paged_attn_workspace_size(...), 256-byte aligned.
 * Numerics: scores, softmax statistics and sums in fp32; out is rounded once.
 * Weights are rounded for their product with v on the tensor cores:
 *   bf16  e^(s_j - m) to bf16 (2^-8), m the largest score so far
 *   E4M3  e^(s_j) times v's scale to fp16 (2^-11), relative to the largest such
 *         product so far, whose score may be far below the largest; below
 *         2^-38 of it: 0.  Codes are exact in fp16, and so is q but for elements
 *         below 2^-31 of its row's largest (held to 2^-39 of that).  The scales
 *         of v are positive.
 *   fp32  not rounded.
 */
int sptp_paged_attn_decode(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, const int* page_table, const int* seq_lens, int P, int B,
                           int Hq, int Hkv, int D, int max_pages, int num_pages, int page_size, int window,
                           float scale, sptp_dtype dtype, sptp_kv_type kv_type, void* out, float* lse,
                           void* workspace, size_t ws_bytes, void* cuda_stream);

/*
 * What a model may make of the scores before the softmax, in
 * sptp_paged_attn_prompt and sptp_paged_attn_decode_ex:
 *     s_j = cap tanh(scale q . k_j / cap) - slope |pos - j|
 *   for a row at position pos of its sequence and key j.
 *   cap     0: none (s_j = scale q . k_j - ..); else 1e-30 <= cap <= 1e30
 *   slopes  fp32 [P][Hq], one per query head of every shard, any sign, |slope| < 2e38;
 *           NULL: none
 * Numerics: tanh to 2^-22 of the cap, or of the score below an eighth of it
 * (prompts' attention in bf16, caps up to 128: of the cap); distances exact below
 * 2^24, a bias to 2^-23 of itself (prompts' attention in bf16, slopes up to 1: or 2^-17).
 */

/* Workspace bytes needed by sptp_paged_attn_prompt (0 on bad args). */
size_t sptp_paged_attn_prompt_workspace_size(int P, int M, int B, int Hq, int Hkv, int D);

/* Arguments of sptp_paged_attn_prompt. */
typedef struct sptp_paged_attn_prompt_args_s {
    const void *q, *k_cache, *v_cache, *k_scale, *v_scale, *page_table, *seq_lens, *row_starts, *prefix_lens, *slopes;
    void *out, *lse, *workspace, *cuda_stream;
    size_t ws_bytes;
    int P, M, B, Hq, Hkv, D, max_pages, num_pages, page_size, window, dtype, kv_type;
    float scale, cap;
} sptp_paged_attn_prompt_args;

/*
 * sptp_paged_attn_prompt -- attention of many new rows per sequence over their
 * cached keys and values: whole prompts, pieces of prompts behind what is
 * cached already, proposed tokens to be checked at once.  The rows of B
 * sequences are packed; a row sees keys of its own sequence only:
 *     lse = ln sum_j e^s_j,  out = sum_j e^(s_j - lse) v_j
 *   over lo <= j < hi:  pos = seq_lens[b] - n_b + r for row r of the sequence's
 *   n_b rows;  hi = pos + 1, or prefix_lens[b] where that is more (a prefix that
 *   rows see beyond their own position);  lo = pos + 1 - window if window > 0
 *   and that is positive, else 0 (a window cuts the prefix, too).
 *   q           [P][M][Hq][D] (sptp_rope_append_kv's q_out)
 *   row_starts  [B + 1] int32: sequence b's rows are row_starts[b] ..
 *               row_starts[b+1] - 1, ascending, 0 <= .. <= M.  Other rows of out
 *               and lse (padding) are left as they were
 *   seq_lens    [B] int32: keys in the cache, the new rows' included
 *   prefix_lens [B] int32, cut to [0, seq_lens[b]]; NULL: no prefixes
 *   cap, slopes as above
 *   out         [P][M][Hq D], the row-parallel operand of sptp_down_proj
 *   lse         [P][M][Hq] fp32, or NULL
 *   out and lse must not overlap an input, the workspace or each other.
 *   M < 2^30, and the shape rules above.  M == 0 or B == 0 enqueues nothing.
 * The work is split over rows, heads and keys, evenly over the SMs whatever the
 * lengths; the parts of a row are joined in a fixed order: equal inputs give
 * equal bits.  What the cache holds outside the keys that a sequence's rows see
 * does not matter, and neither does, for a row, what lies at keys that it does not
 * see.  (E4M3: a code that is no number counts as 480.)
 * Recorded as SPTP_ERR_SHAPE in the workspace status words, for any sequence: a row start outside
 * [0, M] or below the one before it (the rows concerned are undefined); a length
 * outside [0, max_pages * page_size] (cut to it); more rows than keys (the rows
 * before position 0 see nothing: zeros, lse -inf); a page outside [0, num_pages)
 * among the keys that are seen (zero keys and values).  workspace: at least
 * sptp_paged_attn_prompt_workspace_size(...), 256-byte aligned.
 * Numerics: scores, softmax statistics and sums in fp32, out rounded once.  bf16
 * and E4M3 caches: products on the tensor cores, weights rounded to bf16 (2^-8) and
 * taken relative to a base within 2^16 of the largest (2^-110 of it and less: 0; values
 * of v have to be below 2^111 over a row's keys), E4M3 keys and values (code times a
 * power of two) exact in bf16.  fp32: nothing rounded.
 */
int sptp_paged_attn_prompt(const sptp_paged_attn_prompt_args* args);

/* Arguments of the calls below: those of the three calls above, pointers first. */
typedef struct sptp_rope_args_s {
    const void *x, *positions, *turns;
    void *out, *cuda_stream;
    int P, M, H, Hr, D, rot, interleaved, transpose, dtype;
    float gain;
} sptp_rope_args;
typedef struct sptp_rope_append_kv_args_s {
    const void *qkv, *positions, *seq_ids, *page_table, *turns;
    void *q_out, *k_cache, *v_cache, *k_scale, *v_scale, *workspace, *cuda_stream;
    size_t ws_bytes;
    int P, M, Hq, Hkv, D, rot, interleaved, B, max_pages, num_pages, page_size, dtype, kv_type;
    float gain;
} sptp_rope_append_kv_args;
typedef struct sptp_paged_attn_decode_args_s {
    const void *q, *k_cache, *v_cache, *k_scale, *v_scale, *page_table, *seq_lens;
    void *out, *lse, *workspace, *cuda_stream;
    size_t ws_bytes;
    int P, B, Hq, Hkv, D, max_pages, num_pages, page_size, window, dtype, kv_type;
    float scale;
} sptp_paged_attn_decode_args;

/*
 * sptp_rope_packed, sptp_rope_append_kv_packed, sptp_paged_attn_decode_packed
 * -- the three calls above with their arguments in one block of memory (host;
 * read during the call), for callers whose calls cost by the argument: from
 * Python, 28 arguments take 2.2 us to convert and a block 0.7.  Same checks,
 * results and errors; SPTP_ERR_NULL for a NULL block.
 */
int sptp_rope_packed(const sptp_rope_args* args);
int sptp_rope_append_kv_packed(const sptp_rope_append_kv_args* args);
int sptp_paged_attn_decode_packed(const sptp_paged_attn_decode_args* args);

/*
 * sptp_paged_attn_decode_ex -- sptp_paged_attn_decode with scores as in
 * sptp_paged_attn_prompt: pos = seq_lens[b] - 1.  cap 0 and slopes NULL: the
 * same call.  slopes must not overlap an output; 4-byte aligned.
 */
int sptp_paged_attn_decode_ex(const sptp_paged_attn_decode_args* args, float cap, const float* slopes);

/* Workspace bytes needed by sptp_lora (0 on bad args). */
size_t sptp_lora_workspace_size(int P, int M, int K, int N, int R, int rowwise);

/*
 * sptp_lora -- low-rank adapters of many requests at once beside a shared
 * projection: every row of a batch names the adapter of its request,
 *     out[p][m] = base[p][m] + gains[a] * B_a (A_a x_m),  a = ids[m]
 *   added to what the projection itself gave (base).
 *   rowwise == 0: a column-parallel projection (sptp_attn_qkv_forward's qkv_out;
 *            x is then its normed rows, which it leaves in its workspace behind
 *            the header)
 *     x      [M][K], the same for every shard
 *     base, out [P][M][N/P]: shard p has rows [p N/P, (p+1) N/P) of B_a
 *   rowwise != 0: a row-parallel projection (sptp_down_proj's out, with x its s)
 *     x      [P][M][K/P]: shard p has columns [p K/P, (p+1) K/P) of A_a
 *     base, out [P][M][N]: each shard's partial gets its part of the sum
 *   A       [adapters][R][K];  B [adapters][N][R];  gains fp32 [adapters], or
 *           NULL for 1
 *   ids     [M] int32, in any order; < 0: no adapter, out[p][m] = base[p][m]
 *   out may be exactly base, and must not overlap any input otherwise.
 * 8 <= R <= 128, R % 8 == 0; K, N <= 2^20, multiples of 8, the split one of 8 P;
 * adapters >= 0.  An id >= adapters is recorded as SPTP_ERR_SHAPE in the
 * workspace status words, and its row treated as one without adapter.  What other
 * rows and their adapters hold does not reach a row (how many adapters its
 * neighbours name may change the order of its sums); equal calls give equal bits.
 * M == 0 enqueues nothing.  workspace: at least
 * sptp_lora_workspace_size(...), 256-byte aligned.
 * Numerics: A_a x summed in fp32, and kept to 2^-16 of itself for its product
 * with B_a (bf16; in fp32 not rounded), sums in fp32, out rounded once.  Infinities are
 * those of the formula.
 */
int sptp_lora(const void* x, const void* A, const void* B, const int* ids, const float* gains, int P, int M, int K, int N,
              int R, int adapters, int rowwise, sptp_dtype dtype, const void* base, void* out, void* workspace,
              size_t ws_bytes, void* cuda_stream);

/*
 * sptp_lora_ex -- sptp_lora next to the projection's own call.
 *   status_workspace  the workspace whose status words record an id >= adapters,
 *                     unless they hold an error already (a row without one
 *                     writes nothing there); NULL: workspace
 *   check_only        nonzero: the status of the call's arguments, nothing
 *                     enqueued (needs no GPU), so that a projection need not
 *                     be started whose adapters are refused
 */
int sptp_lora_ex(const void* x, const void* A, const void* B, const int* ids, const float* gains, int P, int M, int K, int N,
                 int R, int adapters, int rowwise, sptp_dtype dtype, const void* base, void* out, void* workspace,
                 size_t ws_bytes, void* cuda_stream, void* status_workspace, int check_only);

/*
 * sptp_read_device_status -- synchronises `cuda_stream` and returns the
 * status the kernels recorded in the workspace header since the last call
 * that reset it (every entry point above resets it when it starts, unless it
 * has no rows and enqueues nothing):
 * SPTP_OK; SPTP_ERR_TIMEOUT if a bounded device-side wait ran out (the
 * kernels then stop early and their outputs are undefined); or
 * SPTP_ERR_SHAPE if sptp_permute_ffn_neurons met an index outside [0, F), or
 * a call on a paged cache an index, a page or a length outside its range
 * (a wait that ran out in the attention is reported in place of it).  No
 * counterpart on the pages: this is the library's own failure detection.
 */
int sptp_read_device_status(const void* workspace, void* cuda_stream);

/*
 * sptp_wait_selftest -- enqueues a one-CTA kernel that waits on a flag in the
 * workspace header that nothing sets and on an mbarrier that never completes,
 * each with the bounded wait the GEMM kernels use and a limit of `limit_ns`
 * nanoseconds; both waits give up and record SPTP_ERR_TIMEOUT.  If
 * `preset_flag` != 0 the flag is set first and the flag wait succeeds.  Used to
 * test failure detection without hanging the GPU.  No counterpart on the pages.
 */
int sptp_wait_selftest(void* workspace, size_t ws_bytes, unsigned long long limit_ns,
                       int preset_flag, void* cuda_stream);

/*
 * sptp_paged_attn_wait_selftest -- sptp_paged_attn_decode with an arrival
 * withheld in the first of its two CTAs (D <= 128), so that bounded waits of
 * limit_ns run out in it: of tile withhold_full of that CTA's share, which is
 * not loaded, or of the stage that tile withhold_empty is not given back from.
 * One of the two is -1.  If the CTA has such a tile (and, for withhold_empty,
 * more tiles than stages after it), SPTP_ERR_TIMEOUT is recorded, whatever else
 * is, and out and lse are undefined.  No counterpart on the pages.
 */
int sptp_paged_attn_wait_selftest(const sptp_paged_attn_decode_args* args, int withhold_full, int withhold_empty,
                                  unsigned long long limit_ns);

/*
 * sptp_paged_attn_prompt_wait_selftest -- sptp_paged_attn_prompt (bf16 activations,
 * 64 < D <= 128, no cap, no slopes, scale > 0) on two CTAs, the first of which never
 * loads tile withhold_full of its share (K and V tiles in turn), so that bounded
 * waits of limit_ns run out in it: SPTP_ERR_TIMEOUT is recorded if it has such a
 * tile, and out and lse are then undefined.  No counterpart on the pages.
 */
int sptp_paged_attn_prompt_wait_selftest(const sptp_paged_attn_prompt_args* args, int withhold_full,
                                         unsigned long long limit_ns);

/* Bytes of the static device scratch array used by sptp_ffn_forward_noalloc. */
#define SPTP_NOALLOC_SCRATCH_BYTES (64u << 20)

/*
 * sptp_ffn_forward_noalloc -- sptp_ffn_forward for callers that cannot
 * allocate device memory (for example a plugin inside a host framework that
 * owns every device allocation, or a serving loop that must not call
 * cudaMalloc because it can synchronise the device).  The pages describe no
 * such entry point; it exists for those callers.
 *   - Arguments, results and errors are those of sptp_ffn_forward (variant
 *     AUTO), without the workspace.  The caller still passes every input and
 *     output.  The arguments are checked first, in the same order and with
 *     the same codes; then the size limit; then the device.
 *   - Scratch is a library-owned 256-byte aligned __device__ array of
 *     SPTP_NOALLOC_SCRATCH_BYTES (64 MiB) that every GPU loading the library
 *     holds until the process exits.  Problems whose
 *     sptp_ffn_workspace_size(...) exceeds it return SPTP_ERR_TOO_LARGE
 *     before any CUDA call (bf16, d=4096, F=14336: up to about 1800 tokens).
 *   - No cudaMalloc, cudaFree or other allocating call is made.  The array's
 *     device address is looked up (cudaGetSymbolAddress) on the first call in
 *     each device context, with that device current; make that first call
 *     before any stream capture.
 *   - Every call shares the one array, so calls whose work overlaps on the
 *     GPU (different streams, or different host threads) race and give wrong
 *     results; serialise them.  The array keeps the last call's contents; the
 *     status words are cleared at the start of each call.
 */
int sptp_ffn_forward_noalloc(const void* x, const void* partials, const void* gamma,
                             const void* W1g, const void* W1u, const void* W2,
                             int M, int d, int F, int P, int chunks, float eps, sptp_dtype dtype,
                             void* out, void* resid_out, void* cuda_stream);

/*
 * Failure detection of the no-allocation forward, whose status words live in
 * the library's static array rather than in a caller workspace.
 *   sptp_noalloc_read_device_status: as sptp_read_device_status, for the
 *     last sptp_ffn_forward_noalloc on the current device (synchronises
 *     `cuda_stream`).
 *   sptp_noalloc_wait_selftest: as sptp_wait_selftest, with the static
 *     array's status words.
 * No counterpart on the pages.
 */
int sptp_noalloc_read_device_status(void* cuda_stream);
int sptp_noalloc_wait_selftest(unsigned long long limit_ns, int preset_flag, void* cuda_stream);

/* Human-readable text of a status code (static storage). */
const char* sptp_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* SPTP_H */
