/*
 * bq.h -- C ABI of the block-quantized MoE gather-qmm library for GB300
 * (sm_103a).  Plain pointers and sizes only; no C++ or framework types.
 *
 * Pages cited below (titles as they appear on each page):
 *   [iron]      "feat(gguf,dsv4): GGUF block-dequant + DSv4 kernel surface (WIP)",
 *               thewafflehaus/iron PR #9
 *   [butter]    "Everything Bagel 2", thewafflehaus/butter PR #10
 *   [slimserve] "metal: DSV4 M1 Ultra prefill/decode campaign", QuixiAI/SlimServe PR #2
 *   [vllm]      "WIP: metaltile shim -- Qwen3.6 mt_qmm_mma / mt_moe_gather dispatch",
 *               TheTom/vllm-swift PR #22
 *
 * Conventions for every entry point
 * ---------------------------------
 *  - Pointers marked "device" must point to device memory the caller
 *    allocated and owns; the library never allocates or frees in these
 *    calls and keeps no pointer after a call returns.  Caller-owned
 *    scratch ("workspace") lets a loop reuse one buffer ([butter], the
 *    two-pass decode note: scratch buffers are caller-owned so a decode
 *    loop can amortise them).
 *  - Every call is asynchronous on `stream` (NULL = the legacy default
 *    stream) and does no host synchronisation, except bq_device_status.
 *    Inputs must stay valid until the stream reaches the call.
 *  - Preconditions are checked on the host before any launch ([butter]:
 *    wrapper preconditions with a clear message; [slimserve]: host-checked
 *    TORCH_CHECK contracts).  A failing check returns a status != BQ_OK
 *    and launches nothing; bq_last_error() then holds a message.
 *  - Errors found on the device (an expert id out of range, a bounded
 *    wait that ran out) never trap: the kernel records a code in a
 *    per-device status word and skips the bad element.  Read and clear it
 *    with bq_device_status().
 *  - Pointers must be 16-byte aligned unless stated otherwise.
 */
#ifndef BQ_H
#define BQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream. */
typedef struct CUstream_st* bq_stream_t;

typedef enum {
    BQ_OK = 0,
    BQ_ERR_NULL = 1,       /* a required pointer is NULL                     */
    BQ_ERR_SHAPE = 2,      /* a size is out of range or not divisible        */
    BQ_ERR_ALIGN = 3,      /* a pointer is not aligned as required           */
    BQ_ERR_FORMAT = 4,     /* unknown or mismatched weight format            */
    BQ_ERR_WORKSPACE = 5,  /* workspace pointer NULL or too small            */
    BQ_ERR_CUDA = 6,       /* a CUDA runtime call or launch failed           */
    BQ_ERR_DEVICE = 7,     /* the device status word was set (see below)     */
    BQ_ERR_ARCH = 8        /* current device is not a compute-capability 10.3 GPU */
} bq_status;

/* Codes written to the device status word. */
enum {
    BQ_DEV_OK = 0,
    BQ_DEV_BAD_EXPERT_ID = 1,   /* a routed expert id was outside [0, E)        */
    BQ_DEV_WAIT_TIMEOUT = 2,    /* a bounded mbarrier / flag wait ran out       */
    BQ_DEV_SCALE_RANGE = 3,     /* a block scale the device path cannot represent
                                   met bq_repack_mxfp4 / bq_repack_fp8_b128       */
    BQ_DEV_BAD_ROW = 4          /* a sorted row number outside [-1, T*k) or an
                                   offset list that is not ascending in [0, rows] */
};

/* Element types of plain (unquantised) rows. */
typedef enum {
    BQ_DT_F32 = 0,
    BQ_DT_F16 = 1,
    BQ_DT_BF16 = 2
} bq_dtype;

typedef enum {
    BQ_FMT_Q8_0 = 1,      /* GGUF Q8_0: 32-value blocks, fp16 d + 32 int8 ([iron] kernel 1) */
    BQ_FMT_Q2_K = 2,      /* GGUF Q2_K: 256-value super-blocks of 84 bytes ([iron] kernel 2) */
    BQ_FMT_INT4_G64 = 3,  /* MLX int4 affine, 8 codes per u32, fp16 scale+bias per 64 ([butter]) */
    BQ_FMT_MXFP4 = 4,     /* OCP MX FP4: 32 e2m1 codes + one E8M0 exponent per block ([iron]) */
    BQ_FMT_FP8_B128 = 5   /* FP8 e4m3 bytes, one fp32 scale per 128 x 128 block ([iron]) */
} bq_format;

/*
 * A quantised weight resident on the device in the library's tile-major
 * layout (built by bq_repack_*).  The matrix stack is [n_mats][n][k]:
 * n_mats experts (1 for a dense weight), n output rows, k input columns;
 * row r of matrix e computes output feature r.  `data` is one device
 * buffer of bq_qweight_bytes() bytes, 256-byte aligned, owned by the
 * caller.  swiglu = 1 marks a fused gate/up weight (rows [0, n/2) gate,
 * [n/2, n) up) stored in the interleaved order the SwiGLU epilogue reads.
 *
 * Layout (informative): for each matrix, 128-row tile and K-slab, one
 * contiguous slab of bytes holding 64 quant bytes per row followed by the
 * slab's scale fields.  K-slab width: Q8_0 and FP8 64, Q2_K 256, int4 and
 * MXFP4 128 values.  Bytes per weight equal the on-disk format's (34/32,
 * 84/256, 9/16, 17/32), and for FP8 1 + 16/8192.
 */
typedef struct {
    int32_t fmt;      /* bq_format */
    int32_t n_mats;
    int32_t n;        /* multiple of 128 */
    int32_t k;        /* multiple of 256 (Q2_K), 128 (int4, MXFP4, FP8) or 64 (Q8_0) */
    int32_t swiglu;   /* 0 or 1 */
    int32_t reserved;
    void* data;       /* device */
} bq_qweight;

/* Human-readable name of a status code (static storage). */
const char* bq_status_string(bq_status s);

/* Message of the last failing call on this host thread ("" if none). */
const char* bq_last_error(void);

/*
 * Synchronises `stream`, then reads and clears the current device's status
 * word.  *code receives BQ_DEV_OK or the first device error code recorded
 * since the last read.  Returns BQ_ERR_DEVICE if a code was set.
 */
bq_status bq_device_status(bq_stream_t stream, int32_t* code);

/* ------------------------------------------------------------------ S1, S2
 * Standalone GGUF block dequantisation to fp32 ([iron] kernels 1 and 2).
 *   Q8_0: out[32b + i] = sext8(qs[i]) * d,  sext8(u) = u >= 128 ? u - 256 : u
 *   Q2_K: for value v of super-block b, sub-block j = v/16:
 *         out[256b + v] = (d * sc_j) * q_v - dmin * m_j,
 *         sc_j = scales[j] & 15, m_j = scales[j] >> 4,
 *         q_v = (qs[32*(v/128) + v%32] >> 2*((v/32)%4)) & 3
 * blocks: device, n_blocks on-disk blocks back to back (34 or 84 bytes
 *         each; Q8_0: d then qs; Q2_K: scales[16], qs[64], d, dmin).
 * out:    device fp32 [n_blocks * 32] or [n_blocks * 256].
 * Every product and difference is evaluated in fp32 round-to-nearest with
 * no contraction, in the order written above.
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE (n_blocks < 0), BQ_ERR_ALIGN, BQ_ERR_CUDA.
 * n_blocks == 0 is a no-op.
 */
bq_status bq_gguf_dequant_q8_0(const void* blocks, int64_t n_blocks, float* out,
                               bq_stream_t stream);
bq_status bq_gguf_dequant_q2_k(const void* blocks, int64_t n_blocks, float* out,
                               bq_stream_t stream);

/*
 * Standalone MXFP4 block dequantisation to fp32 ([iron]: DeepSeek V4-Flash
 * MXFP4 experts, OCP MX v1.0 block of 17 bytes per 32 values).  Block b is
 * one E8M0 exponent byte e followed by 16 code bytes; code byte i holds
 * value 2i in its low nibble and value 2i + 1 in its high nibble.
 *   out[32b + v] = lut[code_v] * 2^(e - 127),
 *   lut = {0, 0.5, 1, 1.5, 2, 3, 4, 6, -0, -0.5, -1, -1.5, -2, -3, -4, -6}
 * and e = 255 gives NaN for every value of the block (the only NaN of the
 * format).  Every output is the exact value in fp32 (e = 0 gives fp32
 * subnormals), except magnitudes of 2^128 and above (e >= 253), which
 * overflow to +-inf as fp32 rounding gives.
 * blocks: device, n_blocks blocks of 17 bytes back to back.
 * out:    device fp32 [n_blocks * 32].
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE (n_blocks < 0), BQ_ERR_ALIGN, BQ_ERR_CUDA.
 * n_blocks == 0 is a no-op.
 */
bq_status bq_dequant_mxfp4(const void* blocks, int64_t n_blocks, float* out, bq_stream_t stream);

/*
 * Standalone FP8 block dequantisation to fp32 ([iron]: DeepSeek V3 / V4
 * FP8 e4m3 weights with per-(128 x 128)-block fp32 scales):
 *   out[i][j] = e4m3(weight[i][j]) * scales[i / 128][j / 128]
 * e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits, largest 448,
 * 0x7F / 0xFF NaN, no infinities.  The product is one fp32 multiply
 * (round to nearest even, subnormals kept), so it is the fp32 rounding of
 * the exact product.
 * weight: device uint8 [n][k] row-major; scales: device fp32
 * [ceil(n/128)][ceil(k/128)] row-major (4-byte aligned); out: device fp32
 * [n][k].  n, k >= 0 (any values; a partial last block uses its scale).
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE (n or k < 0), BQ_ERR_ALIGN, BQ_ERR_CUDA.
 * n * k == 0 is a no-op.
 */
bq_status bq_dequant_fp8_b128(const void* weight, const float* scales, int64_t n, int64_t k,
                              float* out, bq_stream_t stream);

/* ------------------------------------------------------------------ S0
 * Load-time repack of on-disk blocks into the device layout ([iron]:
 * CPU-side decomposition of each block into separate GPU tensors;
 * [slimserve]: load-time q2_K SoA repack).  Runs on the device.
 * bq_qweight_bytes: bytes `data` must hold (0 if the shape is invalid).
 * Sources (device):
 *   Q8_0: blocks [n_mats][n][k/32] x 34 bytes
 *   Q2_K: blocks [n_mats][n][k/256] x 84 bytes
 *   int4: words [n_mats][n][k/8] u32 (value 8w+i in bits 4i..4i+3),
 *         scales and biases [n_mats][n][k/64] fp16 (passed as uint16 bits)
 *   MXFP4: blocks [n_mats][n][k/32] x 17 bytes (as bq_dequant_mxfp4; any
 *         alignment)
 *   FP8:  weight bytes [n_mats][n][k] e4m3 (any alignment), scales fp32
 *         [n_mats][n/128][k/128] (4-byte aligned)
 * dst->fmt/n_mats/n/k/swiglu/data must be filled in by the caller.
 * Errors: BQ_ERR_NULL, BQ_ERR_FORMAT, BQ_ERR_SHAPE, BQ_ERR_ALIGN, BQ_ERR_CUDA.
 *
 * MXFP4 on the device: the matmul kernels turn each value into the fp16
 * rounding of lut[code] * 2^(e - 127), which they can form exactly for
 * e <= 128 (for e <= 88 that rounding is 0) and for e = 255 (NaN).  Blocks
 * with e in 129..254 (block scales of 4 and above) are stored unchanged but set
 * BQ_DEV_SCALE_RANGE on the device; matmuls over them give +-inf or NaN.
 *
 * FP8 on the device: each block scale s is stored as the fp16 rounding of
 * 256 * s; a weight enters the matmul as the fp16 rounding of
 * e4m3 * fp16(256 s), and the factor 2^-8 is applied exactly to the fp32
 * accumulators.  Relative error per weight <= 2^-11 + 2^-11 (against 2^-12
 * for a single rounding of the exact product).  Scales with 448 * 256 * |s|
 * above 65504 (|s| > 0.571, block values above 256) or NaN set
 * BQ_DEV_SCALE_RANGE; matmuls over them give +-inf or NaN.  A fused gate/up
 * FP8 weight needs n/2 to be a multiple of 128 (each half has its own
 * scale rows).
 */
size_t bq_qweight_bytes(int32_t fmt, int32_t n_mats, int32_t n, int32_t k);
bq_status bq_repack_q8_0(const void* blocks, const bq_qweight* dst, bq_stream_t stream);
bq_status bq_repack_q2_k(const void* blocks, const bq_qweight* dst, bq_stream_t stream);
bq_status bq_repack_int4(const uint32_t* words, const uint16_t* scales,
                         const uint16_t* biases, const bq_qweight* dst,
                         bq_stream_t stream);
bq_status bq_repack_mxfp4(const void* blocks, const bq_qweight* dst, bq_stream_t stream);
bq_status bq_repack_fp8_b128(const void* weight, const float* scales, const bq_qweight* dst,
                             bq_stream_t stream);

/* ------------------------------------------------------------------ S3, S4
 * Dense qmm: Y[m][r] = sum_k X[m][k] * W[r][k] with W the dequantised
 * weight (matrix 0 of w, swiglu must be 0), fp32 accumulation
 * ([vllm]: mt_qmm_mma, dense activations x 4-bit weights; [butter]:
 * dequantGemmDynamicM; [slimserve]: qc_mmvq batch 2-8 qgemv and the q8_0
 * qgemm).  Weights are dequantised in registers to fp16; products are
 * accumulated in fp32.  Up to 32 rows (Q8_0, FP8) or 64 rows (the other
 * formats) run the GEMV (mma.sync fragments, 8 rows per CTA); more rows the
 * tensor-core (tcgen05) GEMM.
 * x: device fp16 [m][k] row-major (uint16 bits), k = w->k.
 * y: device fp32 [m][w->n] row-major.
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE (m < 0), BQ_ERR_FORMAT, BQ_ERR_ALIGN,
 * BQ_ERR_CUDA.  m == 0 is a no-op.
 */
bq_status bq_qmm(const uint16_t* x, int32_t m, const bq_qweight* w, float* y,
                 bq_stream_t stream);

/* ------------------------------------------------------------------ S5
 * Router top-k ([butter]: moeRouterTopK, logits -> top-k u32 indices and
 * weights summing to 1; [slimserve]: router contract E <= 1024, k <= 8).
 * z[t][e] = logits[t][e] + bias[e] (fp32; bias may be NULL).  ids[t][j]
 * = the j-th largest z of row t (ties: lower e first); weights[t][j] =
 * exp(z_j - z_0) / sum_i exp(z_i - z_0) over the k selected (fp32).
 * logits: device fp32 [T][E]; bias: device fp32 [E] or NULL;
 * ids: device int32 [T][k]; weights: device fp32 [T][k].
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE (T < 0, E < 1 or > 1024, k < 1 or
 * > min(8, E)), BQ_ERR_ALIGN (4-byte alignment suffices here), BQ_ERR_CUDA.
 */
bq_status bq_moe_route(const float* logits, const float* bias, int32_t T, int32_t E,
                       int32_t k, int32_t* ids, float* weights, bq_stream_t stream);

/* Router scoring rules (S5 variants). */
typedef enum {
    /* bq_moe_route above: bias added to the logits, softmax over the selected */
    BQ_SCORE_SOFTMAX = 0,
    /* [butter] LFM2-MoE "softmax-then-bias" ("Everything Bagel 2", the LFM2
     * family paragraph and the aura-port merge note): p = softmax(logits)
     * over all E; select the k largest p[e] + bias[e]; weights = the
     * selected unbiased p, renormalised to sum to 1 (the page does not say
     * which probabilities the weights take; this is the reading used) */
    BQ_SCORE_SOFTMAX_THEN_BIAS = 1,
    /* [iron] DeepSeek V4 scoring: s = sqrt(softplus(logit)) with softplus(x) =
     * max(x, 0) + log1p(exp(-|x|)); select the k largest s[e] + bias[e]
     * (aux-loss-free bias); weights = the selected unbiased s times `scale`
     * (the routed scaling factor), not renormalised */
    BQ_SCORE_SQRTSOFTPLUS = 2
} bq_scoring;

/*
 * Router top-k under a scoring rule.  Same layouts, ordering (descending
 * selection key, ties to the lower e) and errors as bq_moe_route, plus
 * BQ_ERR_SHAPE for an unknown `scoring`.  `scale` is used by
 * BQ_SCORE_SQRTSOFTPLUS only.  For BQ_SCORE_SOFTMAX the result equals
 * bq_moe_route.  Keys of the two other rules are computed in fp32 with
 * expf / log1pf / sqrtf, so where two keys differ by a rounding error the
 * choice between them may differ from an exact evaluation.
 */
bq_status bq_moe_route_scored(const float* logits, const float* bias, int32_t T, int32_t E,
                              int32_t k, int32_t scoring, float scale, int32_t* ids,
                              float* weights, bq_stream_t stream);

/* ------------------------------------------------------------------ S6, S7
 * Expert histogram, exclusive scan and deterministic token permutation
 * (the per-expert work queue of [slimserve] qc_moe_mm_map0 and the
 * gathered layout of [vllm] mt_moe_gather_qmm).  With f = t*k + j:
 *   counts[e]      = #{f : ids[f] == e}
 *   offsets[e]     = sum_{e' < e} counts[e'],  offsets[E] = T*k
 *   perm[r]        = the f listed by (ids[f], f) ascending
 *   perm_token[r]  = perm[r] / k,  perm_slot[r] = perm[r] % k,  inv[perm[r]] = r
 * ids: device int32 [T*k]; counts: device int32 [E]; offsets [E+1];
 * perm_token, perm_slot, inv: device int32 [T*k].  workspace: device,
 * >= bq_moe_permute_workspace_bytes(T, k, E) bytes.
 * Out-of-range ids set BQ_DEV_BAD_EXPERT_ID on the device and are
 * excluded from every output (their perm entries are not written).
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE, BQ_ERR_WORKSPACE, BQ_ERR_ALIGN, BQ_ERR_CUDA.
 */
size_t bq_moe_permute_workspace_bytes(int32_t T, int32_t k, int32_t E);
bq_status bq_moe_permute(const int32_t* ids, int32_t T, int32_t k, int32_t E,
                         int32_t* counts, int32_t* offsets, int32_t* perm_token,
                         int32_t* perm_slot, int32_t* inv, void* workspace,
                         size_t workspace_bytes, bq_stream_t stream);

/*
 * Allocation-free variant of bq_moe_permute (no counterpart on the pages;
 * an addition of this library).  For callers that cannot provide a
 * workspace -- e.g. code whose device memory is entirely owned by another
 * allocator, or a latency-critical loop where cudaMalloc must not be called
 * (it can fail there or synchronise the device).  Same arguments and
 * outputs as bq_moe_permute minus the workspace: the chunk histograms live
 * in a fixed 256 KiB device array built into the library, held on every GPU
 * that loads it until the process exits.
 *  - Limit: ceil(T*k / 256) * E <= 65536 (e.g. T*k <= 16384 for E = 1024,
 *    T*k <= 65536 for E = 256); larger requests return BQ_ERR_SHAPE and
 *    launch nothing.
 *  - The first call on a device looks up the array's address on that
 *    device; make it before any stream capture.
 *  - All calls share the array.  Calls whose kernels overlap on the GPU
 *    race on it; order them (one stream, or events).  Nothing needs to be
 *    cleared between calls: every scratch value read is written first.
 *  - Calls no cudaMalloc, cudaFree or allocating routine.
 * Errors: as bq_moe_permute, with BQ_ERR_SHAPE for the size limit.
 */
bq_status bq_moe_permute_noalloc(const int32_t* ids, int32_t T, int32_t k, int32_t E,
                                 int32_t* counts, int32_t* offsets, int32_t* perm_token,
                                 int32_t* perm_slot, int32_t* inv, bq_stream_t stream);

/* ------------------------------------------------------------------ S5..S13
 * One MoE layer: route -> permute -> grouped gate/up GEMM with SwiGLU ->
 * grouped down GEMM scaled by the gate weight -> combine, plus an
 * optional always-on shared expert added with weight 1.
 *   y[t] = sum_j g[t][j] * W_d[e_tj] (silu(W_g[e_tj] x_t) * (W_u[e_tj] x_t))
 *          (+ W_ds (silu(W_gs x_t) * (W_us x_t)))
 * ([vllm]: mt_moe_gather_qmm_mma_int4_bm{16,64}; [slimserve]: tiled MoE
 * prefill GEMM and sum-folded q2_K down projection; [butter]: GPU router,
 * expert-indexed gemv with no host readback, swiglu, scalarFMA combine.)
 * Token counts up to 32 take the GEMV path (gather-qgemv over each
 * expert's tokens, 8 rows per pass); larger ones the tensor-core grouped
 * GEMM, except that where the experts average fewer than 64 tokens the
 * experts holding at most 8 take the GEMV beside it.  Intermediates:
 * gathered activations and the SwiGLU output are fp16, expert outputs fp32.
 *
 * desc: host struct.  w_gate_up: n_mats = E, n = 2*inter, k = hidden,
 *   swiglu = 1.  w_down: n_mats = E, n = hidden, k = inter, swiglu = 0.
 *   shared_gate_up / shared_down: NULL, or dense weights (n_mats = 1) of
 *   the shared expert, with its own intermediate size.
 * x: device fp16 [T][hidden]; router_logits: device fp32 [T][E];
 * logit_bias: device fp32 [E] or NULL; how it and the logits become the
 * routing is set by desc->scoring (bq_scoring; BQ_SCORE_SOFTMAX adds the bias
 * before selection and weighting) and desc->route_scale (the routed scaling
 * factor of BQ_SCORE_SQRTSOFTPLUS); y: device fp32 [T][hidden].
 * workspace: device, >= bq_moe_workspace_bytes(desc) bytes, 256-aligned
 * (the query returns 0 for a descriptor it cannot size: bad T, E or k, or a
 * weight of unknown format or invalid shape).
 * Errors: as above, plus BQ_ERR_FORMAT if the weights' shapes disagree
 * with the descriptor.
 */
typedef struct {
    int32_t T;
    int32_t hidden;
    int32_t inter;
    int32_t n_experts;   /* E, 1..1024 */
    int32_t topk;        /* 1..min(8, E) */
    int32_t scoring;     /* bq_scoring (0 = BQ_SCORE_SOFTMAX) */
    bq_qweight w_gate_up;
    bq_qweight w_down;
    const bq_qweight* shared_gate_up;  /* host pointer or NULL */
    const bq_qweight* shared_down;     /* host pointer or NULL */
    float route_scale;   /* routed scaling factor (BQ_SCORE_SQRTSOFTPLUS) */
    int32_t reserved;
} bq_moe_desc;

size_t bq_moe_workspace_bytes(const bq_moe_desc* desc);
bq_status bq_moe_gather_qmm(const bq_moe_desc* desc, const uint16_t* x,
                            const float* router_logits, const float* logit_bias,
                            float* y, void* workspace, size_t workspace_bytes,
                            bq_stream_t stream);

/* ------------------------------------------------------------------ RMSNorm, fused
 * RMSNorm and RMSNorm fused with the quantised matmul behind it ([butter]:
 * rmsNormQgemvInt4Fast, the final norm fused with the int4 GEMV; the
 * mt_rms_norm row kernels).  For each row r of length H:
 *   x[r] = gamma * h[r] / sqrt(mean(h[r]^2) + eps)
 * computed in fp32 (1/sqrt by rsqrtf; each value (h * gamma) * inv, then
 * rounded to fp16).  Both entry points compute inv and x identically, so x
 * from bq_rmsnorm_qmm equals bq_rmsnorm's bit for bit.
 * h, x: device fp16 [T][H] row-major; gamma: device fp16 [H]; H a multiple
 * of 8; eps finite and >= 0.
 * bq_rmsnorm_qmm: y[r] = W x[r] (fp32 [m][w->n]) for a plain weight w
 * (n_mats 1, swiglu 0, k = H).  m <= 8 runs one norm-fused GEMV kernel
 * (x_out may be NULL; if set it receives x); larger m runs the norm kernel
 * into x_out (then required) and the tensor-core GEMM.
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE, BQ_ERR_FORMAT, BQ_ERR_ALIGN, BQ_ERR_CUDA.
 * T == 0 / m == 0 is a no-op.
 */
bq_status bq_rmsnorm(const uint16_t* h, int32_t T, int32_t H, const uint16_t* gamma, float eps,
                     uint16_t* x, bq_stream_t stream);
bq_status bq_rmsnorm_qmm(const uint16_t* h, int32_t m, const uint16_t* gamma, float eps,
                         const bq_qweight* w, uint16_t* x_out, float* y, bq_stream_t stream);

/*
 * One MoE layer from the hidden states: x = RMSNorm(hidden) (as above),
 * router_logits = W_router x (fp32; `router` a plain weight with n =
 * n_experts, k = hidden, n_experts a multiple of 128), then exactly
 * bq_moe_gather_qmm(desc, x, router_logits, logit_bias, y, ...).  x and the
 * logits live in the workspace.  workspace: device, >=
 * bq_moe_hidden_workspace_bytes(desc) bytes, 256-byte aligned.
 * Errors: as bq_moe_gather_qmm and bq_rmsnorm_qmm.
 */
size_t bq_moe_hidden_workspace_bytes(const bq_moe_desc* desc);
bq_status bq_moe_gather_qmm_hidden(const bq_moe_desc* desc, const bq_qweight* router,
                                   const uint16_t* hidden, const uint16_t* gamma, float eps,
                                   const float* logit_bias, float* y, void* workspace,
                                   size_t workspace_bytes, bq_stream_t stream);

/* ------------------------------------------------------------------ rows by expert
 * Moving activation rows into expert order and back, with their gradients.
 * inv (device int32 [T][k], from bq_moe_permute) names the sorted row of
 * each pair (t, j): a number in [0, T*k), each at most once, or -1 for a
 * pair that was dropped.  Sorted matrices have T*k rows; rows that no pair
 * names are not touched.  An entry outside [-1, T*k) sets BQ_DEV_BAD_ROW
 * and counts as dropped.  All sums are fp32, in slot order j = 0..k-1, so
 * results do not change from run to run; the result is rounded once to
 * `dtype` (bq_dtype, the type of every row matrix of the call).
 *   bq_moe_dispatch           xs[inv[t][j]] = x[t]
 *   bq_moe_dispatch_backward  dx[t] = sum_j dxs[inv[t][j]]
 *   bq_moe_combine            y[t] = sum_j weights[t][j] * ys[inv[t][j]]
 *                             (accumulate = 1: y[t] += the sum, added last)
 *   bq_moe_combine_backward   dys[inv[t][j]] = weights[t][j] * dy[t]
 *                             dweights[t][j] = sum_h dy[t][h] * ys[inv[t][j]][h]
 *                             (0 for a dropped pair).  Either output may be
 *                             NULL and is then not computed; ys is read only
 *                             for dweights (else it may be NULL), weights
 *                             only for dys (else it may be NULL).
 * A dropped pair contributes nothing to a sum: its weight is not read as a
 * factor, so a NaN there does no harm.  A zero weight multiplies like any
 * other (0 * inf is NaN).
 * Row matrices: device, H elements per row, rows ld* elements apart
 * (ld* >= H), H and ld* such that rows start on 16-byte boundaries;
 * weights, dweights: device fp32 [T][k], 4-byte aligned, as inv.  k in
 * 1..8.  Outputs must not overlap inputs (bq_moe_combine's y with
 * accumulate is the one matrix that is read and written).
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE, BQ_ERR_FORMAT (unknown dtype),
 * BQ_ERR_ALIGN, BQ_ERR_CUDA.  T == 0 is a no-op.
 */
bq_status bq_moe_dispatch(const void* x, int32_t dtype, int32_t T, int32_t H, int64_t ldx,
                          const int32_t* inv, int32_t k, void* xs, int64_t ldxs,
                          bq_stream_t stream);
bq_status bq_moe_dispatch_backward(const void* dxs, int32_t dtype, int32_t T, int32_t H,
                                   int64_t ldxs, const int32_t* inv, int32_t k, void* dx,
                                   int64_t ldx, bq_stream_t stream);
bq_status bq_moe_combine(const void* ys, int32_t dtype, int32_t T, int32_t H, int64_t ldys,
                         const int32_t* inv, const float* weights, int32_t k,
                         int32_t accumulate, void* y, int64_t ldy, bq_stream_t stream);
bq_status bq_moe_combine_backward(const void* dy, int64_t lddy, const void* ys, int64_t ldys,
                                  int32_t dtype, int32_t T, int32_t H, const int32_t* inv,
                                  const float* weights, int32_t k, void* dys, int64_t lddys,
                                  float* dweights, bq_stream_t stream);

/* ------------------------------------------------------------------ FP8 rows
 * Quantises rows to FP8 e4m3 with one fp32 scale per 128 values of a row
 * (the activation side of the 128 x 128 block-scaled FP8 weights).  For the
 * values v of a group (the last group of a row may be shorter):
 *   amax  = max |v|
 *   scale = max(amax / 448, 2^-126)              (fp32, rounded once)
 *   code  = e4m3(448 * v / max(amax, 448 * 2^-126)), half to even
 * The quotient is rounded to e4m3 as if it were exact, so codes are the
 * same on every machine.  A group holding a NaN gets NaN codes and a NaN
 * scale; one holding an infinity gets the scale +inf, NaN codes where the
 * value is infinite and 0 elsewhere.  Neither is hidden: a product over
 * such a row gives NaN.
 * x: device rows of k elements of `dtype`, ldx elements apart; k a multiple
 * of 16, rows on 16-byte boundaries.  q: device uint8 [rows][k].  scales:
 * device fp32 [rows][ceil(k/128)].
 * n_rows: NULL, or a device int32: only the first min(*n_rows, rows) rows
 * are read and written (for sorted rows: &offsets[E]).
 *
 * bq_moe_dispatch_fp8_b128 quantises row t of x and writes its codes and
 * scales to the rows inv[t][j] of q [T*k][H] and scales [T*k][ceil(H/128)]:
 * bq_moe_dispatch and bq_quant_fp8_b128 in one pass over x, with the same
 * results and the same conditions on inv.
 * Errors: as above.  No rows: a no-op.
 */
bq_status bq_quant_fp8_b128(const void* x, int32_t dtype, int32_t rows, int32_t k, int64_t ldx,
                            const int32_t* n_rows, uint8_t* q, float* scales,
                            bq_stream_t stream);
bq_status bq_moe_dispatch_fp8_b128(const void* x, int32_t dtype, int32_t T, int32_t H,
                                   int64_t ldx, const int32_t* inv, int32_t k, uint8_t* q,
                                   float* scales, bq_stream_t stream);

/* ------------------------------------------------------------------ FP8 x FP8 products
 * Products of FP8 rows (as bq_quant_fp8_b128 writes them) with FP8 weights
 * of one scale per 128 x 128 block (as bq_dequant_fp8_b128 reads them; no
 * repack):
 *   y[r][c] = sum_b xscales[r][b] * wscales[c/128][b]
 *                   * sum_{i in block b of 128} e4m3(x[r][i]) * e4m3(w[c][i])
 * Products and sums in fp32; the result is rounded once to `ydtype`
 * (bq_dtype).  A block's two scales are multiplied first, in fp32, and their
 * product then meets the block's sum.  The scales may be of any size, but
 * their product should be zero or a normal number: where it is below 2^-126
 * the block's term is off by up to 2^-125 (rows of the smallest scale that
 * bq_quant_fp8_b128 gives, 2^-126, hold values below 2^-117; zeros stay
 * zeros); from 2^128 on the term is infinite, or NaN where the block's sum
 * is 0.  NaN codes, NaN and infinite scales propagate.
 * swiglu = 1: w holds n/2 gate rows, then n/2 up rows (n a multiple of 256);
 * y has n/2 columns, silu(gate) * up with silu(g) = g / (1 + exp(-g)).
 *
 * bq_mm_fp8_b128: one weight w [n][k], x [m][k].
 * bq_moe_mm_fp8_b128: rows sorted by expert: rows [offsets[e],
 * offsets[e + 1]) of x take matrix e of w [E][n][k] (offsets: device int32
 * [E + 1], as bq_moe_permute writes it).  Rows outside [offsets[0],
 * offsets[E]) are not written.  Offsets that descend or leave [0, rows] set
 * BQ_DEV_BAD_ROW; the experts concerned are skipped (where ranges overlap,
 * experts behind them may be skipped too).
 *
 * x: device uint8 [rows][k]; xscales: device fp32 [rows][ceil(k/128)];
 * w: device uint8 [E][n][k]; wscales: device fp32 [E][ceil(n/128)]
 * [ceil(k/128)]; y: device rows of n (swiglu: n/2) elements of `ydtype`,
 * ldy elements apart.  k a multiple of 16 (a short last block is fine),
 * n >= 1 of any value (without swiglu), rows, n and k at most 2^31 - 256,
 * E * n <= 2^31 - 1, E <= 1024.  x, w 16-byte aligned; scales and offsets
 * 4-byte aligned; y aligned to its element.
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE, BQ_ERR_FORMAT, BQ_ERR_ALIGN,
 * BQ_ERR_CUDA.  No rows: a no-op.
 */
bq_status bq_mm_fp8_b128(const uint8_t* x, const float* xscales, int32_t m, const uint8_t* w,
                         const float* wscales, int32_t n, int32_t k, int32_t swiglu, void* y,
                         int32_t ydtype, int64_t ldy, bq_stream_t stream);
bq_status bq_moe_mm_fp8_b128(const uint8_t* x, const float* xscales, int32_t rows,
                             const int32_t* offsets, int32_t E, const uint8_t* w,
                             const float* wscales, int32_t n, int32_t k, int32_t swiglu, void* y,
                             int32_t ydtype, int64_t ldy, bq_stream_t stream);

/*
 * The same products with an end of their own, in the same pass:
 *   y[r][c] = scale * act(product[r][c] + bias[c]) + residual[r][c]
 * act: bq_activation; BQ_ACT_SWIGLU as swiglu = 1 above (its bias has n values,
 * gate then up).  bias: device fp32 [n], of bq_moe_mm_fp8_b128_epilogue [E][n]
 * (a row takes its expert's), or NULL.  residual: device rows of y's type and
 * columns, ldr elements apart, aligned to the element, or NULL; it may be y
 * itself (then with ldr = ldy) but not overlap it otherwise.  All of it in fp32
 * before the one rounding to `ydtype`.  epi: host struct, read during the call.
 * NaN of the product, bias or residual propagates through every activation.
 * Exponentials and reciprocals are the special-function unit's: of its exact
 * value, silu (also in SwiGLU; without an end that takes expf, so that the two may
 * differ in their last places) is off by (16 + 2.2 |v|) 2^-24, gelu by
 * (24 + 1.1 v^2) 2^-24, gelu_tanh by (16 + 8 |w|) 2^-24, w = 1.6 (v + 0.045 v^3);
 * results below 2^-119 may become 0.
 * Errors: as above, plus BQ_ERR_SHAPE (unknown activation, ldr below the columns).
 */
typedef enum {
    BQ_ACT_NONE = 0,
    BQ_ACT_SWIGLU = 1,
    BQ_ACT_SILU = 2,        /* v / (1 + exp(-v)) */
    BQ_ACT_GELU = 3,        /* v * Phi(v), the normal distribution's Phi */
    BQ_ACT_GELU_TANH = 4,   /* v / 2 * (1 + tanh(sqrt(2 / pi) * (v + 0.044715 v^3))) */
    BQ_ACT_RELU = 5,        /* max(v, 0) */
    BQ_ACT_RELU2 = 6        /* max(v, 0)^2 */
} bq_activation;

typedef struct {
    int32_t act;
    float scale;
    const float* bias;
    const void* residual;
    int64_t ldr;
} bq_epilogue;

bq_status bq_mm_fp8_b128_epilogue(const uint8_t* x, const float* xscales, int32_t m,
                                  const uint8_t* w, const float* wscales, int32_t n, int32_t k,
                                  const bq_epilogue* epi, void* y, int32_t ydtype, int64_t ldy,
                                  bq_stream_t stream);
bq_status bq_moe_mm_fp8_b128_epilogue(const uint8_t* x, const float* xscales, int32_t rows,
                                      const int32_t* offsets, int32_t E, const uint8_t* w,
                                      const float* wscales, int32_t n, int32_t k,
                                      const bq_epilogue* epi, void* y, int32_t ydtype, int64_t ldy,
                                      bq_stream_t stream);

/* ------------------------------------------------------------------ block to block
 * The way out of a block and into the next, in one pass over the rows ([butter]:
 * sigmoidScalarFMAResidual, the gated residual; gatedMixerNormMany).  With
 * n(v) = v / sqrt(mean(v^2) + eps) and, per row t,
 *   b     = post_gain * n(y), or y where post_gain is NULL
 *   g     = the gate, its sigmoid (gate_sigmoid = 1), or 1 (BQ_GATE_NONE)
 *   h_out = residual_scale * h + scale * g * b
 *   x     = gain * n(h_out)                      (not computed where x is NULL)
 * Everything is computed in fp32 and rounded once to the output's type; x comes
 * from h_out before that rounding.  A gate's sigmoid is off by (16 + 2.2 |v|) 2^-24
 * of its value, and 0 where that is below 2^-126.
 *
 * bq_residual_norm_backward: with dh_out and dx the gradients of h_out and x
 * (either may be NULL: none; then what only it needs, gain, may be NULL too),
 * r = 1 / sqrt(mean(h_out^2) + eps), s the same of y, all sums in fp32:
 *   G     = dh_out + r * gain * dx - h_out * r^3 * mean(gain * dx * h_out)
 *   D     = scale * G,      dh = residual_scale * G
 *   dy    = s * post_gain * D * g - y * s^3 * mean(post_gain * D * g * y), or D * g
 *   dgate = D * b (times g * (1 - g) under a sigmoid), summed over what the gate is shared by
 *   dgain = sum_t dx * h_out * r,   dpost_gain = sum_t D * g * y * s
 * h_out is the forward pass's output (read only where dx is given).  dgain,
 * dpost_gain: fp32 [H]; dgate: fp32 [T] or [H], for a gate per value rows of the
 * gate's type.  Each of the three may be NULL (not computed).  Sums over rows
 * have a fixed order: results do not change from run to run.
 *
 * y, h, h_out, x and their gradients: device rows of H elements of y_dtype (y,
 * dy), h_dtype (h, h_out, dh_out, dh) or x_dtype (x, dx), ld* elements apart.
 * H a multiple of 8, at most 16384; rows start and end on 16-byte boundaries and
 * lie less than 2^35 bytes apart.
 * gain, post_gain: gain_dtype [H], 16-byte aligned.  gate: gate_dtype, [T]
 * (aligned to its element), [H] (16-byte aligned) or rows like y.  Outputs must
 * not overlap inputs, but h_out may be h, and dh may be dh_out.
 * workspace of the backward pass: device, at least
 * bq_residual_norm_backward_workspace_bytes(T, H) bytes, 16-byte aligned; needed
 * only for dgain, dpost_gain and the dgate of a gate per channel.  Calls that may
 * overlap on the GPU (other streams, other captured graphs) need one each.
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE, BQ_ERR_FORMAT (an unknown type), BQ_ERR_ALIGN,
 * BQ_ERR_WORKSPACE, BQ_ERR_CUDA.  T == 0: a no-op, but sums over rows become 0.
 */
typedef enum {
    BQ_GATE_NONE = 0,
    BQ_GATE_TOKEN = 1,     /* [T]: a factor per row, as a shared expert's gate */
    BQ_GATE_CHANNEL = 2,   /* [H]: a factor per column, as a layer scale */
    BQ_GATE_FULL = 3       /* [T][H] */
} bq_gate;

typedef struct {
    int32_t T, H;
    int32_t y_dtype, h_dtype, x_dtype, gain_dtype, gate_dtype;   /* bq_dtype */
    int32_t gate_kind;       /* bq_gate */
    int32_t gate_sigmoid;    /* 0 or 1 */
    float scale, residual_scale, eps;
    const void* gain;        /* device, of the norm that gives x */
    const void* post_gain;   /* device, of the norm of y; NULL: none */
    const void* gate;        /* device */
    int64_t ldgate;          /* BQ_GATE_FULL */
} bq_residual_norm_desc;

bq_status bq_residual_norm(const bq_residual_norm_desc* desc, const void* y, int64_t ldy,
                           const void* h, int64_t ldh, void* h_out, int64_t ldho, void* x,
                           int64_t ldx, bq_stream_t stream);
size_t bq_residual_norm_backward_workspace_bytes(int32_t T, int32_t H);
bq_status bq_residual_norm_backward(const bq_residual_norm_desc* desc, const void* y, int64_t ldy,
                                    const void* h_out, int64_t ldho, const void* dh_out,
                                    int64_t lddho, const void* dx, int64_t lddx, void* dy,
                                    int64_t lddy, void* dh, int64_t lddh, float* dgain,
                                    float* dpost_gain, void* dgate, int64_t lddgate,
                                    void* workspace, size_t workspace_bytes, bq_stream_t stream);

/* ------------------------------------------------------------------ router training
 * Per-expert counts, mean probabilities, the balance loss and the z-loss of a
 * router's logits, over one batch or over the sequences of it.  Rows
 * [seq_offsets[s], seq_offsets[s + 1]) are sequence s (device int32 [S + 1],
 * ascending in [0, T]); rows before the first and behind the last are not read.
 * seq_offsets NULL: S = 1, all T rows.  z = logits + bias under
 * BQ_SCORE_SOFTMAX; under the other rules the bias only selects, so bias must
 * be NULL and z = logits.
 *   p[t]         = softmax(z[t]), under BQ_SCORE_SQRTSOFTPLUS score / sum of scores
 *   counts[s][e] = pairs (t, j) of the sequence with ids[t][j] = e
 *   probs[s][e]  = mean of p[t][e] over its n_s rows (0 for an empty sequence)
 *   losses[0]    = mean over the sequences that have rows of
 *                  sum_e E * counts[s][e] / (k * n_s) * probs[s][e]
 *   losses[1]    = mean over all rows of sequences of logsumexp(z[t])^2
 * A row of -inf only has probabilities 0 and adds 0 to losses[1]; NaN and +inf
 * propagate.  Probabilities of other rows add up to 1 however far below 0 their
 * logits are; those below 2^-110 may become 0.  Exponentials and logarithms are the
 * special-function unit's: a probability is off by (2 max |z| + 160) 2^-24 of itself
 * at most.  An id outside [0, E) sets BQ_DEV_BAD_EXPERT_ID and counts nowhere.
 * Offsets that descend or leave [0, T] set BQ_DEV_BAD_ROW; what such a call
 * returns is undefined.  Sums are fp32 in a fixed order.
 *
 * bq_moe_route_backward: the gradient with respect to the logits of what
 * bq_moe_route(_scored) returned, given dweights (fp32 [T][k], as
 * bq_moe_combine_backward writes them; NULL: none), and of the two losses,
 * given dlosses (device fp32 [2]; NULL: none) and the counts of the forward
 * call; selection and counts are constants.
 *   softmax rules:  dlogits[ids[j]] += w_j * (dweights_j - sum_i w_i dweights_i), w over the k selected
 *   score rule:     dlogits[ids[j]] += scale * dweights_j * score'(z)
 * (selected logits that are all -inf bring none)
 * ids are read only with dweights; those outside [0, E) set
 * BQ_DEV_BAD_EXPERT_ID and are left out of the k.  dlogits: device [T][E] of
 * `dtype`, computed in fp32 and rounded once; rows that belong to no sequence
 * are left as they were.  dbias: fp32 [E], the sum of the gradient over the
 * rows written (BQ_SCORE_SOFTMAX only), or NULL; it alone needs the workspace.
 *
 * logits: device fp32 [T][E]; ids int32 [T][k]; counts int32 [S][E]; probs fp32
 * [S][E]; losses fp32 [2]; all 4-byte aligned, dlogits to its element.  T at
 * most 2^31 - 65 and T * k below 2^31, E in 1..1024, k in 1..min(8, E), S in 1..65536.  workspace: device, 256-byte
 * aligned, at least bq_moe_balance_workspace_bytes(T, E, S) or
 * bq_moe_route_backward_workspace_bytes(T, E) bytes (0: invalid sizes); nothing in
 * it is read before it is written.  Calls that may overlap on the GPU (other
 * streams, other captured graphs) need one each.
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE, BQ_ERR_FORMAT, BQ_ERR_ALIGN,
 * BQ_ERR_WORKSPACE, BQ_ERR_CUDA.  T == 0: counts, probs, losses and dbias become 0.
 */
size_t bq_moe_balance_workspace_bytes(int32_t T, int32_t E, int32_t S);
bq_status bq_moe_balance_loss(const float* logits, const float* bias, int32_t T, int32_t E,
                              const int32_t* ids, int32_t k, int32_t scoring,
                              const int32_t* seq_offsets, int32_t S, int32_t* counts, float* probs,
                              float* losses, void* workspace, size_t workspace_bytes,
                              bq_stream_t stream);
size_t bq_moe_route_backward_workspace_bytes(int32_t T, int32_t E);
bq_status bq_moe_route_backward(const float* logits, const float* bias, int32_t T, int32_t E,
                                const int32_t* ids, int32_t k, int32_t scoring, float scale,
                                const float* dweights, const int32_t* counts,
                                const float* dlosses, const int32_t* seq_offsets, int32_t S,
                                void* dlogits, int32_t dtype, float* dbias, void* workspace,
                                size_t workspace_bytes, bq_stream_t stream);

/* ------------------------------------------------------------------ observability
 * Stage timing: while set, every bq_moe_gather_qmm call on this host thread
 * records `start` (a cudaEvent_t) on its stream immediately before the
 * kernels of `stage` and `stop` immediately after them.  Passing NULL
 * events clears the stage.  Events are owned by the caller.  This exists so
 * that a benchmark can time one stage of a layer call with CUDA events on
 * the stream the stage runs on; it adds two event records per stage.
 * Errors: BQ_ERR_SHAPE (unknown stage).
 */
typedef enum {
    BQ_STAGE_ROUTE_PERMUTE = 0,  /* route, histogram, scan, placement, segment list, tile list and
                                    the gather of the activation rows (tensor-core path) */
    BQ_STAGE_GATE_UP = 1,        /* routed gate/up GEMM (or GEMV) with SwiGLU */
    BQ_STAGE_DOWN = 2,           /* routed down GEMM scaled by the gate weight */
    BQ_STAGE_SHARED = 3,         /* shared expert (gate/up + down) */
    BQ_STAGE_COMBINE = 4,        /* gate-weighted combine */
    BQ_STAGE_NORM_ROUTER = 5,    /* RMSNorm + router matmul (bq_moe_gather_qmm_hidden) */
    BQ_STAGE_COUNT = 6
} bq_stage;
bq_status bq_set_stage_events(int32_t stage, void* start_event, void* stop_event);

/* Number of kernels this library has launched in this process (all threads). */
uint64_t bq_launch_count(void);

/*
 * Test hook for the bounded waits of the tensor-core kernels (the failure
 * detection path; the pages have no counterpart).  Every barrier wait in
 * such a kernel gives up after a time limit, sets BQ_DEV_WAIT_TIMEOUT in the
 * device status word, lets its own copies in flight land, frees its TMEM
 * and returns.  Normally nothing makes a wait run out.  While set, GEMM
 * launches (bq_qmm above the GEMV range, the prefill MoE layer, the FP8
 * products) take
 * `wait_limit_ns` as that limit (1 ms .. 2 s; 0 restores the 2 s default)
 * and, if `skip_weight_copies` is 1, their weight producer issues no copies,
 * so the waits for weights run out: the call then returns BQ_OK, its output
 * is undefined and bq_device_status reports BQ_DEV_WAIT_TIMEOUT.  3: the same,
 * but of an FP8 product whose K is split over a cluster only the odd parts
 * issue none; no part of a split then writes y.  Process wide, for tests
 * only; call bq_test_set_wait_probe(0, 0) to restore.
 * Errors: BQ_ERR_SHAPE (argument outside the ranges above).
 */
bq_status bq_test_set_wait_probe(int32_t skip_weight_copies, uint64_t wait_limit_ns);

#ifdef __cplusplus
}
#endif
#endif /* BQ_H */
