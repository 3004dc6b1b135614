/*
 * h3a.h -- C ABI of the B200 (sm_100a) attention core for H3-style video DiTs.
 *
 * One DiT self-attention core per call sequence:
 *   h3a_qk_norm_rope  fused QK-RMSNorm + 3D RoPE over Q and K
 *   h3a_route         blockwise KV-block router (pool -> fp32 scores -> top-k)
 *   h3a_attention     bidirectional attention, dense or over routed KV blocks
 * and, for the text model that conditions it, the prompt side (conventions of
 * its own further down):
 *   h3a_residual_rmsnorm  residual addition + RMS norm, to 16 or 8 bits
 *   h3a_rope              one-dimensional rotary positions
 *   h3a_packed_attention  causal attention over packed prompts and caches
 *
 * Conventions shared by every call
 *   - Tensors are bf16 (raw 16-bit words), laid out [B, N, heads, head_dim]
 *     with head_dim contiguous and element strides given by h3a_qkv_desc.
 *     Token n of the (T, H, W) grid is n = (t*H + h)*W + w.
 *   - head_dim must be 96 (hidden 5376 / 56 heads); the router and attention
 *     also take 128 (SubBlock's stated head size; the same hidden width as
 *     42 heads), the prologue does not (its 3D RoPE layout is defined for 96
 *     channels).  block must be 128.
 *   - All pointers are DEVICE pointers owned by the caller, 16-byte aligned;
 *     strides are multiples of 8 elements (16 bytes).  The library never
 *     allocates or frees device memory per call; the router's scratch is a
 *     caller workspace sized by h3a_route_workspace_size.  Its only device
 *     state is static: the status word below and the fixed scratch array of
 *     h3a_route_noalloc, both resident on every GPU that loads the library.
 *   - Calls are asynchronous on the caller's stream.  A status other than
 *     H3A_OK means nothing was launched, except H3A_ERR_CUDA, returned when a
 *     launch itself failed.  Device-side failures (a bounded pipeline wait that
 *     expired) are latched in a per-device status word and reported by
 *     h3a_last_device_error.
 *   - Thread safety: calls may be issued from several host threads.  A call
 *     writes only its arguments, except for two pieces of shared device state:
 *     kernels OR timeouts into the per-device status word (taken atomically by
 *     h3a_last_device_error), and h3a_route_noalloc works in one scratch array
 *     per device, so its calls race when they overlap on the GPU.
 */
#ifndef H3A_H_
#define H3A_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* h3a_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum {
    H3A_OK = 0,
    H3A_ERR_INVALID_ARG = 1, /* null/misaligned pointer, inconsistent sizes, bad sparsity */
    H3A_ERR_UNSUPPORTED = 2, /* head_dim not supported by the call, block != 128, sizes beyond int32 range */
    H3A_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed (see h3a_last_cuda_error_string) */
    H3A_ERR_TIMEOUT = 4,     /* a bounded device-side wait expired; results are undefined */
    H3A_ERR_WORKSPACE = 5    /* a workspace is null or too small */
} h3a_status;

/* Token grid of one clip latent: N = T*H*W tokens. */
typedef struct {
    int32_t T, H, W;
} h3a_grid;

/* Shape and element strides of a [B, N, heads, head_dim] bf16 tensor.
 * Q, K, V and O of one call share this descriptor. */
typedef struct {
    int32_t B, N, heads, head_dim;
    int64_t stride_b, stride_n, stride_h; /* in elements; head_dim is contiguous */
} h3a_qkv_desc;

/* Fused QK-RMSNorm + 3D RoPE.
 * Source: news.cocoloop.cn MiniMax-H3 SGLang report, section "Erst drei
 * übereinandergelegte Beschleunigungsebenen" (QK-RMSNorm with 3D RoPE fused
 * into one kernel, result unchanged); 3D multimodal RoPE and the 96-wide heads
 * from the 52hbtv.com H3-Image page, section 二, model table.
 * For every token n and head h of Q (and of K):
 *   y = x / sqrt(mean(x^2) + eps) * gamma        (over the head's 96 channels)
 *   then channels [0,32) turn with t, [32,64) with h, [64,96) with w: the pair
 *   (32a+2j, 32a+2j+1) rotates by pos_a * theta^(-2j/32), j = 0..15;
 *   computed in fp32, rounded once to bf16 (round to nearest even).
 * q, k      : input tensors (device, bf16, layout d).
 * gamma_q/k : fp32 [96] gains (device).
 * q_out/k_out: outputs (device, layout d); may equal q/k (in place), must not
 *             otherwise overlap them.
 * Errors: INVALID_ARG if any pointer is null or misaligned, T*H*W != N, or
 * eps < 0; UNSUPPORTED if head_dim != 96. */
h3a_status h3a_qk_norm_rope(const void* q, const void* k, const h3a_qkv_desc* d,
                            const float* gamma_q, const float* gamma_k, h3a_grid grid,
                            double theta, float eps, void* q_out, void* k_out,
                            h3a_stream_t stream);

/* Number of KV blocks kept per query block for a given sparsity:
 * k = clamp(ceil((1 - sparsity) * nkv - 1e-9), 1, nkv).
 * Returns -1 if sparsity is outside [0, 1) or nkv < 1. */
int64_t h3a_route_k(int64_t nkv, double sparsity);

/* h3a_qk_norm_rope with the RMSNorm spanning the token's whole hidden state:
 * the other reading of "QK-RMSNorm" on the same page (fused-operator
 * paragraph).  For every token n of Q (and of K):
 *   r = 1 / sqrt(mean over all heads x 96 channels of x^2 + eps)
 *   y[h, c] = x[h, c] * r * gamma[h * 96 + c], then the per-head 3D RoPE of
 *   h3a_qk_norm_rope; fp32 arithmetic, one rounding to bf16.
 * gamma_q/k : fp32 [heads * 96] gains (device, 16-byte aligned).
 * Other arguments, layouts and errors: as h3a_qk_norm_rope, and UNSUPPORTED
 * for more than 74 heads or B * N >= 2^31 (one CTA per token holds the
 * token's rows). */
h3a_status h3a_qk_fullnorm_rope(const void* q, const void* k, const h3a_qkv_desc* d,
                                const float* gamma_q, const float* gamma_k, h3a_grid grid,
                                double theta, float eps, void* q_out, void* k_out,
                                h3a_stream_t stream);

/* Sparsity to use at a denoising step: the router prunes KV blocks from the
 * first_sparse_step-th step on (news.cocoloop.cn MiniMax-H3 SGLang report,
 * SubBlock paragraph: from the 10th step), steps counted from 1.  Returns
 * `sparsity` when step >= first_sparse_step, 0.0 (dense attention) before,
 * and -1.0 if step < 1, first_sparse_step < 1 or sparsity is outside [0, 1).
 * Host only; no device work. */
double h3a_step_sparsity(int32_t step, int32_t first_sparse_step, double sparsity);

/* Bytes of device workspace h3a_route needs for the fp32 block means,
 * nblk = ceil(N / block), head_dim 96 or 128: Q's as [B, heads, nblk,
 * head_dim], then, from the next 256-byte boundary, K's channel-major as
 * [B, heads, head_dim, nblk rounded up to 4], each part rounded up to 256
 * bytes.  Returns INVALID_ARG/UNSUPPORTED for bad descriptors. */
h3a_status h3a_route_workspace_size(const h3a_qkv_desc* d, int32_t block, size_t* bytes);

/* Blockwise KV-block router.
 * Source: news.cocoloop.cn MiniMax-H3 SGLang report, SubBlock paragraph of
 * section "Erst drei übereinandergelegte Beschleunigungsebenen" (a blockwise
 * sparse router prunes the KV blocks, sparsity 0.75 or 0.80); pooling,
 * scoring and selection as fixed by the problem statement:
 *   qbar_i, kbar_j = fp32 means of the 128-token blocks (the tail block over
 *   its real length), score S_ij = (qbar_i . kbar_j) / sqrt(head_dim) in fp32,
 *   per (b, h, i) keep the k highest scores, ties to the lower j.
 * q, k       : prologue outputs (device, bf16, layout d).
 * block_idx  : device int32 [B, heads, nblk, k], each row ascending.
 * k_out      : host; receives k (may be NULL).
 * workspace  : device, at least h3a_route_workspace_size bytes, 16-B aligned.
 * Errors: INVALID_ARG for null pointers or sparsity outside [0, 1);
 * UNSUPPORTED for block != 128, head_dim other than 96 / 128, more key blocks
 * than the score kernel holds (each of its CTAs keeps 8 query blocks' fp32
 * scores against every key block in 200 KB of shared memory: ceil(N / 128)
 * <= 6,048 at head_dim 96, 6,016 at 128) or B * heads > 65,535; WORKSPACE if
 * the workspace is null or ws_bytes is too small.  Nothing is launched when a
 * check fails. */
h3a_status h3a_route(const void* q, const void* k, const h3a_qkv_desc* d, double sparsity,
                     int32_t block, int32_t* block_idx, int64_t* k_out, void* workspace,
                     size_t ws_bytes, h3a_stream_t stream);

/* h3a_qk_norm_rope that also pools its outputs for the router, so that
 * h3a_route_pooled can skip reading Q and K back from device memory.
 * Source: the fused prologue of h3a_qk_norm_rope and the block pooling of
 * h3a_route (news.cocoloop.cn MiniMax-H3 SGLang report: fused QK-RMSNorm +
 * 3D RoPE in section "Erst drei übereinandergelegte Beschleunigungsebenen",
 * SubBlock's blockwise router in the same section).
 * Writes q_out / k_out exactly as h3a_qk_norm_rope does, and into workspace
 * the fp32 means, over each 128-token block (the tail block over its real
 * length), of the rounded outputs: the same bytes h3a_route's pooling leaves
 * in its workspace (the layout h3a_route_workspace_size describes), bit for
 * bit.
 * workspace : device, at least h3a_route_workspace_size(d, 128) bytes,
 *             16-B aligned, owned by the caller; it must not overlap q, k,
 *             q_out or k_out.
 * Other arguments, layouts and errors: as h3a_qk_norm_rope; WORKSPACE if the
 * workspace is null, misaligned or too small; UNSUPPORTED if B > 65535.  Q
 * and K stream through shared memory with TMA; a bounded pipeline wait that
 * expired is reported by h3a_last_device_error (H3A_ERR_TIMEOUT). */
h3a_status h3a_qk_norm_rope_pool(const void* q, const void* k, const h3a_qkv_desc* d,
                                 const float* gamma_q, const float* gamma_k, h3a_grid grid,
                                 double theta, float eps, void* q_out, void* k_out,
                                 void* workspace, size_t ws_bytes, h3a_stream_t stream);

/* The scoring and top-k half of h3a_route, from block means that
 * h3a_qk_norm_rope_pool left in the workspace (same source and rule as
 * h3a_route).  d describes the Q/K tensors that were pooled; block_idx,
 * k_out and the result are those of h3a_route on the prologue's outputs.
 * The workspace is only read.  Errors: as h3a_route, and UNSUPPORTED for a
 * head_dim other than 96 (the prologue's only width). */
h3a_status h3a_route_pooled(const h3a_qkv_desc* d, double sparsity, int32_t block,
                            int32_t* block_idx, int64_t* k_out, const void* workspace,
                            size_t ws_bytes, h3a_stream_t stream);

/* Gated residual followed by the AdaLN update, one pass over device memory.
 * Source: news.cocoloop.cn MiniMax-H3 SGLang report, section "Erst drei
 * übereinandergelegte Beschleunigungsebenen", fused-operator paragraph (the
 * AdaLN update and the gated residual path fused like QK-RMSNorm + 3D RoPE,
 * no result changed); the page gives no formulas, these are the DiT block's.
 * For batch b and token row r of width C:
 *   h = x + gate[b] * f, rounded once to bf16 (f == NULL: h = x)
 *   y = (h - mean(h)) / sqrt(var(h) + eps) * (1 + scale[b]) + shift[b]
 *   (LayerNorm without affine, statistics over the C channels of the rounded
 *   h, fp32 arithmetic, y rounded once to bf16).
 * x, f        : device bf16 [B, rows, width], contiguous; f may be NULL.
 * gate, shift, scale: device fp32 [B, width] (gate only read when f != NULL).
 * h_out       : device bf16 [B, rows, width], written when f != NULL (then
 *               required; may equal x); ignored when f == NULL.
 * y_out       : device bf16 [B, rows, width]; must not overlap x, f or h_out.
 * All pointers 16-byte aligned.
 * Errors: INVALID_ARG for null/misaligned pointers, width not a positive
 * multiple of 8, eps < 0; UNSUPPORTED for width > 14336 or B*rows >= 2^31. */
h3a_status h3a_residual_adaln(const void* x, const void* f, const float* gate, const float* shift,
                              const float* scale, int32_t B, int64_t rows, int32_t width, float eps,
                              void* h_out, void* y_out, h3a_stream_t stream);

/* SwiGLU activation: out = silu(a) * b = a / (1 + exp(-a)) * b.
 * Source: the same fused-operator paragraph (the SwiGLU activation).
 * in  : device bf16 [rows, 2 * ffn_width], contiguous; each row is a (the
 *       first ffn_width channels) followed by b.
 * out : device bf16 [rows, ffn_width], contiguous; must not overlap in.
 * fp32 arithmetic, one rounding to bf16.  Both pointers 16-byte aligned.
 * Errors: INVALID_ARG for null/misaligned pointers or ffn_width not a
 * positive multiple of 8. */
h3a_status h3a_swiglu(const void* in, int64_t rows, int32_t ffn_width, void* out, h3a_stream_t stream);

/* Device workspace h3a_residual_diff needs: 32 KB (partial sums). */
#define H3A_RESIDUAL_DIFF_WORKSPACE_BYTES ((size_t)32768)

/* The Cache-DiT reuse decision between two denoising steps.
 * Source: news.cocoloop.cn MiniMax-H3 SGLang report, Cache-DiT paragraph
 * after the fused-operator one (results are reused between adjacent steps
 * when a residual-difference threshold allows: 0.04 conservative, 0.08 in
 * stride mode); read as the relative L1 difference
 *   rel = sum_i |cur_i - prev_i| / sum_i |prev_i|
 * (0 if both are zero, +inf if only prev is), reuse = rel < threshold.
 * cur, prev : device bf16 arrays of n values (n a positive multiple of 8),
 *             16-byte aligned.
 * workspace : device, >= H3A_RESIDUAL_DIFF_WORKSPACE_BYTES, 16-B aligned.
 * rel_out   : device fp64 scalar; reuse_out: device int32 scalar or NULL.
 * Sums: each 8 values in fp32, then fp64 in a fixed order (deterministic);
 * rel agrees with an fp64 sum to about 1e-7 relative, so a decision can only
 * differ from an exact one for rel within that band of the threshold.
 * Errors: INVALID_ARG for null/misaligned pointers, n not a positive multiple
 * of 8, threshold < 0 or NaN; WORKSPACE if the workspace is null or small. */
h3a_status h3a_residual_diff(const void* cur, const void* prev, int64_t n, double threshold,
                             void* workspace, size_t ws_bytes, double* rel_out, int32_t* reuse_out,
                             h3a_stream_t stream);

/* Capacity of the scratch built into h3a_route_noalloc: 64 MiB.  The router
 * keeps two fp32 block means of head_dim values per (batch, head, block) (the
 * layout h3a_route_workspace_size gives), so it holds about
 * B * heads * ceil(N / 128) <= 64 MiB / (8 * head_dim) blocks: some 87,000 at
 * head_dim 96 (e.g. 56 heads of a 124,992-token clip), 65,000 at 128; a shape
 * whose workspace size exceeds 64 MiB is refused. */
#define H3A_ROUTE_NOALLOC_MAX_BYTES ((size_t)64 << 20)

/* h3a_route for callers that cannot allocate device memory (no counterpart on
 * the pages).  Some callers have no allocator at hand where they route -- an
 * embedding runtime that hands out none after start-up, code inside a host
 * callback or another allocator's critical section, a serving loop with a
 * fixed memory budget -- so this variant takes no workspace: its scratch is a
 * file-scope device array of H3A_ROUTE_NOALLOC_MAX_BYTES that every GPU
 * loading the library holds until process exit.  It calls no cudaMalloc,
 * cudaFree or other allocating routine.  Arguments and results are those of
 * h3a_route.
 * The first call on a device resolves the array's device address for that
 * device (cudaGetSymbolAddress with the device current): make that first call
 * before any stream capture.  Every call shares the one array and overwrites
 * what it reads, so nothing needs clearing, but calls whose executions overlap
 * on the GPU (other streams, other host threads) race on it.
 * Errors: those of h3a_route; H3A_ERR_WORKSPACE when the shape needs more than
 * H3A_ROUTE_NOALLOC_MAX_BYTES of scratch (h3a_route_workspace_size bytes);
 * H3A_ERR_CUDA if the set-up fails. */
h3a_status h3a_route_noalloc(const void* q, const void* k, const h3a_qkv_desc* d, double sparsity,
                             int32_t block, int32_t* block_idx, int64_t* k_out, h3a_stream_t stream);

/* Bidirectional attention O = softmax(scale * Q K^T) V per (b, head).
 * Source: dense lossless path of the news.cocoloop.cn MiniMax-H3 SGLang
 * report (opening quote: no approximation; SSIM 1.0000) and its SubBlock
 * sparse attention (same page; "Ein paar Grenzen": long non-causal
 * attention, BF16).
 * block_idx == NULL: dense, every query attends to all N keys.
 * block_idx != NULL: device int32 [B, heads, nblk, k_blocks] routed lists
 *   (ascending, distinct, in [0, nblk)); the queries of block i attend exactly
 *   to the tokens of the KV blocks listed for (b, h, i), softmax renormalised
 *   over them.
 * scale: logit scale; 0 selects 1/sqrt(head_dim).
 * o: output (device, bf16, layout d), must not overlap q, k or v.
 * Tensor-core path: TMA tiles, tcgen05.mma with TMEM accumulators, fp32
 * online softmax, one rounding of O to bf16.
 * Errors: INVALID_ARG for null/misaligned pointers or k_blocks outside
 * [1, nblk] in sparse mode; UNSUPPORTED for head_dim other than 96 / 128,
 * block != 128, or N >= 2^31. */
h3a_status h3a_attention(const void* q, const void* k, const void* v, const h3a_qkv_desc* d,
                         const int32_t* block_idx, int32_t k_blocks, int32_t block, float scale,
                         void* o, h3a_stream_t stream);

/* ---- Prompt side: the conditioning text model's operators ------------------
 * Rows are tokens of packed prompts (sequences behind one another, no
 * padding); elements are bf16 or fp16, named by an h3a_dtype.  Pointers are
 * 16-byte aligned and strides multiples of 8 elements unless said otherwise. */

typedef enum { H3A_BF16 = 0, H3A_FP16 = 1 } h3a_dtype;

/* A [tokens, heads, head_dim] tensor read and its counterpart written, both
 * with head_dim contiguous and element strides of their own (a slice of a
 * fused QKV buffer is one). */
typedef struct {
    int32_t heads, head_dim;
    int64_t stride_n, stride_h;         /* of the input */
    int64_t out_stride_n, out_stride_h; /* of the output */
} h3a_heads_desc;

#define H3A_ROPE_MAX_PAIRS 128

/* Rotary frequencies of one model, made once on the host by
 * h3a_rope_plan_scaled or h3a_rope_plan_from and passed to every h3a_rope
 * call (read during the call only). */
typedef struct {
    int32_t pairs;                      /* rotated channels / 2 */
    int32_t interleaved;                /* pair j is channels (2j, 2j+1), else (j, j + pairs) */
    float amplitude;                    /* factor on the rotated channels */
    int32_t reserved;
    uint64_t turns[H3A_ROPE_MAX_PAIRS]; /* turns per position, modulo 1, in units of 2^-64 */
} h3a_rope_plan;

/* How h3a_rope_plan_scaled stretches theta^(-2j/rotary_dim) for contexts
 * longer than the model was trained on, by `factor` s:
 *   H3A_ROPE_PLAIN   not at all
 *   H3A_ROPE_LINEAR  every frequency / s
 *   H3A_ROPE_BASE    theta * s^(R / (R - 2)), R = rotary_dim: the slowest pair
 *                    turns s times slower, the fastest as before
 *   H3A_ROPE_PARTS   by n, the turns a pair makes over original_length: with
 *                    w = clamp((n - low_turns) / (high_turns - low_turns), 0, 1)
 *                    the frequency becomes f * (w + (1 - w) / s) */
typedef enum { H3A_ROPE_PLAIN = 0, H3A_ROPE_LINEAR = 1, H3A_ROPE_BASE = 2, H3A_ROPE_PARTS = 3 } h3a_rope_scaling;

/* Fills *plan.  Host only.  rotary_dim: even, 2 .. 256.  original_length,
 * low_turns and high_turns are read for H3A_ROPE_PARTS only.
 * Errors: INVALID_ARG for a null plan, an odd or non-positive rotary_dim,
 * theta <= 0, factor <= 0, an unknown scaling, original_length < 1 or
 * high_turns <= low_turns with H3A_ROPE_PARTS, or a value that is not finite (the
 * amplitude in fp32, the stretched base, the frequencies); UNSUPPORTED for
 * rotary_dim > 256. */
h3a_status h3a_rope_plan_scaled(int32_t rotary_dim, int32_t interleaved, double theta, h3a_rope_scaling scaling,
                                double factor, int64_t original_length, double low_turns, double high_turns,
                                double amplitude, h3a_rope_plan* plan);

/* Fills *plan from rotary_dim / 2 frequencies in radians per position (host
 * array), for scalings the call above does not name.  Errors: as above. */
h3a_status h3a_rope_plan_from(int32_t rotary_dim, int32_t interleaved, const double* frequencies, double amplitude,
                              h3a_rope_plan* plan);

/* One-dimensional rotary positions over q and, unless k is NULL, k.
 * For every token n, head and pair j with channels (a, b):
 *   angle = 2 pi * frac(positions[n] * turns[j])
 *   a' = amplitude * (a cos - b sin), b' = amplitude * (a sin + b cos),
 * with the angle negated when `inverse` is nonzero (which undoes a rotation of
 * amplitude 1 and is the rotation's transpose); channels past the rotated ones
 * pass through unchanged.  The angle's turn is exact for any int32 position
 * (64-bit fixed point, modulo 1), cos and sin are fp32, one rounding to the
 * element type.
 * q, k        : device, layouts dq and dk; q_out and k_out: device.  An output
 *               may be its own input with the same strides (in place) and must
 *               not overlap anything else.
 * positions   : device int32 [tokens], 4-byte aligned.
 * Errors: INVALID_ARG for null or misaligned pointers, tokens < 0, heads < 1,
 * head_dim < rotary_dim, head_dim or a stride no multiple of 8, a stride
 * smaller than what it steps over or a plan not made by the calls above;
 * UNSUPPORTED for head_dim > 512, tokens >= 2^31 or more than 32,768 heads in
 * all. */
h3a_status h3a_rope(const void* q, void* q_out, const h3a_heads_desc* dq, const void* k, void* k_out,
                    const h3a_heads_desc* dk, h3a_dtype dtype, const int32_t* positions, int64_t tokens,
                    const h3a_rope_plan* plan, int32_t inverse, h3a_stream_t stream);

/* What h3a_residual_rmsnorm writes as y: the element type of x, or e4m3 (8
 * bits) with one fp32 scale a row or a group of 128 channels. */
typedef enum { H3A_SCALES_NONE = 0, H3A_SCALES_ROW = 1, H3A_SCALES_GROUP = 2 } h3a_scales;
#define H3A_SCALE_GROUP 128

/* The residual's addition and the root-mean-square norm, one pass over device
 * memory (the prompt side's counterpart of h3a_residual_adaln).  For every row:
 *   h = x + f, rounded once to the element type (f == NULL: h = x)
 *   y = h / sqrt(mean(h^2) + eps) * gamma     (statistics of the rounded h, fp32:
 *       the sum of h^2 has to stay in fp32's range.  Beyond it, |h| of about 1e17, y
 *       is 0; with eps = 0 and all |h| under about 1e-19 y loses its accuracy, and
 *       under 1e-23 it is infinite or NaN)
 * H3A_SCALES_NONE: y rounded once to the element type.  Otherwise, per row or
 * per group of 128 channels (the last group may be shorter):
 *   scale = max(max|y|, 2^-100) / 448, y8 = e4m3(y / scale) (nearest even),
 * so that y8 * scale stands for y; a NaN makes its scale NaN.  Both divisions are
 * products with the fp32 reciprocal, so scale and y / scale are within a few
 * roundings of 2^-24 of the quotients, and a y / scale that close to the middle
 * between two codes may take either.
 * x, f, h_out : device, [rows, width] with row strides; f may be NULL.  h_out
 *               is written when f != NULL (then required; may be x or f with
 *               the same stride).
 * gamma       : device fp32 [width].
 * y_out       : device [rows, width] of the element type or of bytes, row
 *               stride y_stride in its own elements; overlaps nothing else.
 * scales_out  : device fp32 [rows] or [rows, ceil(width / 128)], 4-byte
 *               aligned, NULL with H3A_SCALES_NONE.
 * Errors: INVALID_ARG for null or misaligned pointers, rows < 0, width or a
 * stride no positive multiple of 8, a stride below width, eps < 0 or NaN, an
 * unknown dtype or scales; UNSUPPORTED for width > 16384 or rows >= 2^31. */
h3a_status h3a_residual_rmsnorm(const void* x, int64_t x_stride, const void* f, int64_t f_stride, const float* gamma,
                                int64_t rows, int32_t width, h3a_dtype dtype, float eps, h3a_scales scales,
                                void* h_out, int64_t h_stride, void* y_out, int64_t y_stride, float* scales_out,
                                h3a_stream_t stream);

/* Shapes of one h3a_packed_attention call.  q and o are [total_q, heads,
 * head_dim], k and v [total_k, kv_heads, head_dim], head_dim contiguous. */
typedef struct {
    h3a_dtype dtype;
    int32_t seqs, heads, kv_heads, head_dim;
    int64_t total_q, total_k;           /* rows of the tensors */
    int64_t max_q, max_k;               /* no sequence has more queries / keys (max_k: see below) */
    int64_t q_stride_n, q_stride_h, k_stride_n, k_stride_h, v_stride_n, v_stride_h, o_stride_n, o_stride_h;
    int32_t causal;
    float scale;                        /* logit scale; 0 selects 1 / sqrt(head_dim) */
} h3a_packed_desc;

/* Bytes of device workspace h3a_packed_attention needs for this descriptor: 0
 * when no sequence's keys are cut into parts, else the parts' fp32 rows and
 * log-sum-exps (a few MB for single tokens over caches; for prompts and pieces
 * of them, one row for each part, query and head).  It goes by the descriptor
 * alone, so a workspace for the largest shapes of a program serves the whole
 * range only if it is asked for each of them.  Errors: those of
 * h3a_packed_attention that concern the descriptor. */
h3a_status h3a_packed_attention_workspace_size(const h3a_packed_desc* d, size_t* bytes);

/* Attention over packed sequences with grouped heads, causal or not: whole
 * prompts, pieces of prompts behind cached ones and single tokens over caches.
 * Sequence s has the queries starts_q[s] .. starts_q[s+1]-1 and the keys
 * starts_k[s] .. starts_k[s]+lk-1 with lk = lengths_k[s], or starts_k[s+1] -
 * starts_k[s] when lengths_k is NULL (with lengths_k, a cache of fixed capacity
 * per sequence, rows behind lk are never used).  Head h reads kv head
 * h / (heads / kv_heads).  Query i of lq attends key j < lk, and when causal
 * only j <= i + lk - lq (the last query sees every key):
 *   o_i = sum_j softmax_j(scale * q_i . k_j) v_j,  lse_i = ln sum_j exp(scale * q_i . k_j)
 * A query without keys (lk = 0, or causal and i + lk < lq) gets o = 0 and
 * lse = -inf.  What a query does not attend has no influence on it, NaN and
 * infinities included.  Rows of o and lse outside every sequence are left as
 * they were.
 * starts_q, starts_k: device int32 [seqs + 1], ascending (with lengths_k,
 * starts_k in any order, its last entry unused, and sequences may share keys);
 * lengths_k: device int32 [seqs] or NULL.  Values that do not fit total_q / total_k are cut to
 * them (no access outside the tensors).
 * max_q bounds the sequences' queries (rows past it are left as they were);
 * max_k only decides how keys are cut into parts, so a wrong one costs time, not
 * correctness.
 * o         : device, overlaps nothing else.
 * lse       : device fp32 [total_q, heads], contiguous, or NULL.
 * workspace : device, h3a_packed_attention_workspace_size bytes, 16-byte
 *             aligned; NULL when that is 0.  It needs no preparation and holds
 *             nothing from call to call; calls that may overlap on the GPU
 *             (captured ones too) need workspaces of their own.
 * QK^T and PV run on the tensor cores with fp32 accumulation; logits, maxima
 * and sums are fp32; P is rounded to the element type for PV; o is rounded
 * once.
 * Errors: INVALID_ARG for null or misaligned pointers, seqs < 1, heads no
 * positive multiple of kv_heads, negative sizes, max_q or max_k < 0, a stride no
 * multiple of 8 or smaller than what it steps over, an unknown dtype, a scale
 * that is negative or, times log2 e, not finite in fp32; UNSUPPORTED for
 * head_dim other than 64 / 96 / 128, more than 128 heads to a kv head, total_q,
 * total_k or total_q * heads >= 2^31, strides of 2^39 elements, or a grid beyond
 * 2^31 blocks; WORKSPACE if it is null, misaligned or too small.  A bounded
 * device-side wait that expired is reported by
 * h3a_last_device_error. */
h3a_status h3a_packed_attention(const void* q, const void* k, const void* v, const h3a_packed_desc* d,
                                const int32_t* starts_q, const int32_t* starts_k, const int32_t* lengths_k, void* o,
                                float* lse, void* workspace, size_t ws_bytes, h3a_stream_t stream);

/* Human-readable name of a status. Never NULL. */
const char* h3a_status_string(h3a_status s);

/* Text of the last CUDA error seen by the calling host thread ("" if none). */
const char* h3a_last_cuda_error_string(void);

/* Takes the current device's status word: after everything already queued
 * on `stream`, one atomic exchange reads the word and clears it, then the call
 * synchronises `stream` and returns H3A_OK, or H3A_ERR_TIMEOUT if a bounded
 * device wait expired since the word was last taken.  The word is shared by
 * every stream of the device: a timeout raised by a kernel on another stream is
 * reported to exactly one caller -- this one if that kernel had already raised
 * it, else a later one; it is never lost, and never reported twice.  Readers
 * in one process are serialised.  H3A_ERR_CUDA if the launch, the copy or the
 * synchronisation failed. */
h3a_status h3a_last_device_error(h3a_stream_t stream);

/* Self-check of the bounded-wait path (no counterpart on the pages): launches
 * one CTA that waits on a barrier nothing ever completes, with a limit of
 * `limit_us` microseconds, then synchronises.  Returns H3A_ERR_TIMEOUT when
 * the limit expired and was reported through the status word (the expected
 * result), H3A_OK if it was not, H3A_ERR_CUDA on a CUDA failure.  Clears the
 * status word afterwards. */
h3a_status h3a_selftest_wait_timeout(uint32_t limit_us, h3a_stream_t stream);

/* Self-check of the tensor-core building blocks used by h3a_attention (no
 * counterpart on the pages): one CTA loads a 128x96 tile A and a 128x96 tile
 * B (bf16, row-major, device) with TMA, computes S = A B^T (fp32 [128,128])
 * with tcgen05.mma into tensor memory, rounds S to bf16 into tensor memory and
 * computes R = bf16(S) C (fp32 [128,96]) with C = B read as a [128 kv, 96]
 * MN-major operand.  Writes S and R (device fp32).  For diagnosing a new
 * toolkit or driver. */
h3a_status h3a_selftest_mma(const void* a, const void* b, float* s_out, float* r_out,
                            h3a_stream_t stream);

/* Self-check of the exponential of the attention softmax (no counterpart on
 * the pages): y[i] = 2^x[i] for n device floats, by the instruction the
 * softmax evaluates every exponential with (ex2.approx.ftz.f32, in the log2
 * domain).  Asynchronous on `stream`.  INVALID_ARG for n < 0 or null /
 * misaligned pointers. */
h3a_status h3a_selftest_exp2(const float* x, float* y, int32_t n, h3a_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* H3A_H_ */
