/*
 * moe_decode.h - C ABI of the GB300 small-M MoE decode layer library
 * (libmoe_decode.so, sm_103a).
 *
 * The layer, for M = 1..16 tokens (batch-1 decode and speculative verify):
 *   logits = x Wg^T                      router gate matvec, bf16 weight
 *   p = softmax(logits) (or sigmoid(logits)); S = top-k(p + bias);
 *   w = routed_scale * p_S / sum p_S
 *   y_t = sum_j w_tj * E_{S_tj}(x_t) + E_shared(x_t)
 *   E(x) = W2 (silu(W1 x) * (W3 x)),   silu(g) = g / (1 + e^-g)
 * "Chasing the Batch-1 Floor: Ling-3.0-flash Speculative Decode on
 * Blackwell" (lmsys.org): sections "The model" (512-expert MoE), "PDL:
 * stacking the latency floors of small kernels" (router chain norm -> gate
 * matvec -> top-k; MoE chain up-GEMM -> activation -> down-GEMM -> combine;
 * fp32 combine with one final cast), "Two fusions and a retune" (SwiGLU in
 * the up-GEMM epilogue), "bf16 router gate and lm_head"; "3 ways to boost MoE
 * inference on NVIDIA DGX Spark": "Model and baseline configuration" (8 of 512
 * routed experts plus one shared expert, hidden 2560) and "Optimization 1"
 * (MXFP4 expert weights).
 *
 * Conventions for every entry point:
 *  - Pointers named as device pointers must be memory the GPU can address,
 *    owned by the caller, 16-byte aligned: normally HBM. The tokens x and
 *    the outputs y, idx_out, w_out may also be pinned host memory (on a
 *    coherent CPU-GPU link the kernel then reads and writes it directly,
 *    with no separate copy). The library allocates and frees nothing.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *    default stream) and never synchronise, except moe_read_status.
 *  - Return value: MOE_OK (0), or a negative MOE_E* code. A negative code
 *    from argument checking means nothing was launched. MOE_ECUDA means a
 *    CUDA call failed (cudaGetLastError is then cleared).
 *  - Conditions found on the device (an expert index out of range passed to
 *    moe_ffn, a bounded wait that ran out) do not fault: they are written to
 *    a status word inside the workspace; read it with moe_read_status.
 *  - A workspace (`ws`, `ws_bytes` >= moe_workspace_bytes(shape, M)) holds
 *    the router logits (each tagged with its call), the SwiGLU activations
 *    (for one-token bf16 layers also tagged with the call, with a 16-bit tag
 *    that repeats every 65,535 calls: calls of several shapes that share a
 *    workspace should be re-initialised at least that often), a call counter
 *    and the grid-barrier counters. Zero it once with moe_workspace_init
 *    before its first use; every call leaves it ready for the next. Calls
 *    that share a workspace must be ordered on one stream (or otherwise
 *    serialised).
 *
 * Layouts (row-major; nn.Linear [out, in], contiguous along the reduction
 * dimension):
 *   x      bf16 [M, H]           the (already normalised) layer input
 *   Wg     bf16 [E, H]
 *   w1, w3 bf16 [E, I, H]        gate and up projections of routed experts
 *   w2     bf16 [E, H, I]        down projections
 *   MXFP4 routed experts (wfmt = 1): w1, w3 u8 [E, I, H/2], s1, s3 u8
 *     [E, I, H/32]; w2 u8 [E, H, I/2], s2 u8 [E, H, I/32]. Codes are e2m1,
 *     element 2j in the low nibble of byte j; scales are e8m0 (2^(s-127)),
 *     one per 32 consecutive elements of a row.
 *   FP8 routed experts (wfmt = 2): w1, w3 u8 [E, I, H], s1, s3 fp32
 *     [E, I, H/128]; w2 u8 [E, H, I], s2 fp32 [E, H, I/128] (the s pointers
 *     of moe_weights then point at fp32 values). Codes are OCP e4m3; a weight
 *     is e4m3(code) * scale, one scale per 128 consecutive elements of a row
 *     ("Chasing the Batch-1 Floor", "Where the time goes now": FP8 block-128
 *     experts; a 128 x 128 tile scale repeats over its 128 rows).
 *   ws1, ws3 bf16 [Is, H]; ws2 bf16 [H, Is]   shared expert (always bf16)
 *   idx    int32 [M, k]  selected experts, by descending logit (ties: lower
 *                        index first)
 *   w      fp32  [M, k]  renormalised routing weights, same order
 *   y      bf16  [M, H]
 */
#ifndef MOE_DECODE_H
#define MOE_DECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- codes */
#define MOE_OK 0
#define MOE_EINVAL (-1)      /* null pointer or unknown flag/option */
#define MOE_ESHAPE (-2)      /* shape outside what the kernels support */
#define MOE_EM (-3)          /* M outside [1, 16] */
#define MOE_EWORKSPACE (-4)  /* workspace missing or smaller than required */
#define MOE_EALIGN (-5)      /* a pointer is not 16-byte aligned */
#define MOE_ECUDA (-6)       /* a CUDA runtime call failed */
#define MOE_ENODEVICE (-7)   /* no usable CUDA device */
#define MOE_ESCRATCH (-8)    /* moe_decode_layer_static_scratch: the shape
                                and M need more than
                                MOE_STATIC_SCRATCH_BYTES of scratch */
/* written by the device into the workspace status word */
#define MOE_EDEVICE_BAD_INDEX (-100) /* moe_ffn got an index outside [0, E);
                                        that (token, slot) was skipped */
#define MOE_EDEVICE_OVERFLOW (-102)  /* moe_paged_plan: more new tokens than
                                        slot_map holds, a request longer
                                        than its row of the block table, or
                                        the free list ran out; the tokens
                                        concerned got slot -1 */
#define MOE_ETIMEOUT (-101)          /* a bounded device wait ran out; the
                                        call's outputs are incomplete and the
                                        workspace must be re-initialised:
                                        until then every call on it refuses
                                        to run and reports MOE_ETIMEOUT */

/* flags of moe_decode_layer */
#define MOE_F_NO_PDL 1u                /* launch without programmatic
                                          dependent launch */
#define MOE_F_RESET_SCRATCH 2u         /* moe_decode_layer_static_scratch
                                          only: zero the static scratch
                                          before the launch */
#define MOE_F_DEBUG_FORCE_TIMEOUT 256u /* test hook: the routing step waits
                                          for router logits of a call that
                                          never comes, so the wait runs out
                                          and reports MOE_ETIMEOUT */

/* options of moe_set_option */
#define MOE_OPT_GRID_CTAS 1       /* CTAs of the persistent grid; 0 = one per
                                     SM (default). Values above the SM count
                                     are rejected. */
#define MOE_OPT_WAIT_TIMEOUT_NS 2 /* budget of each bounded device wait in
                                     ns (default 1e9) */
#define MOE_OPT_TRACE_BUFFER 3    /* diagnostic: device address of a uint64
                                     buffer of at least 16 x (grid CTAs)
                                     entries; each CTA writes the global timer
                                     (ns) at its phase boundaries into its 16
                                     entries. 0 (default) disables it. */
#define MOE_OPT_DEBUG_HOLD_BACK 4 /* test hook: 1 keeps the first keys (or
                                     their scores) of each CTA of
                                     moe_paged_attention from coming, so that
                                     its waits run out and report MOE_ETIMEOUT.
                                     0 (default) disables it. */

typedef struct moe_shape {
    int32_t hidden;       /* H: multiple of 256 (bf16) or 512 (MXFP4, FP8), <= 8192 */
    int32_t n_experts;    /* E: 1..1024 */
    int32_t top_k;        /* k: 1..min(16, E) */
    int32_t inter;        /* I: multiple of 64 (FP8: 128), at most 4096 */
    int32_t shared_inter; /* Is: 0 (no shared expert) or a multiple of 64, <= 4096 */
    int32_t wfmt;         /* routed expert weights: 0 = bf16, 1 = MXFP4, 2 = FP8 e4m3 */
    /* router configuration ("Chasing the Batch-1 Floor", "PDL: stacking the
     * latency floors of small kernels": the top-k step reads a selection
     * bias). Zero-initialised fields give the plain softmax router. */
    int32_t scoring;          /* 0: softmax over all E; 1: sigmoid of each logit */
    float routed_scale;       /* routing weights are multiplied by this (<= 0: 1) */
    const float* router_bias; /* NULL, or fp32 [E] (device) added to the scores
                                 to select the top k only; the weights use
                                 the unbiased scores, renormalised */
    /* layer input and output ("PDL: stacking the latency floors of small
     * kernels": the router chain starts with the norm; the residual add
     * closes the layer). Zero-initialised fields: x is taken as given. */
    const void* norm_weight;  /* NULL, or bf16 [H] (device, 16-byte aligned):
                                 the input is the residual stream h and the
                                 layer runs on x = bf16(h / sqrt(mean(h^2) +
                                 eps) * norm_weight) */
    float norm_eps;           /* RMSNorm epsilon (<= 0: 1e-6) */
    int32_t residual;         /* 1: y = input + MoE(x), added in fp32 before
                                 the single bf16 cast (moe_ffn and
                                 moe_decode_layer) */
} moe_shape;

typedef struct moe_weights {
    const void* w1;     /* routed gate projection  (device) */
    const void* w3;     /* routed up projection    (device) */
    const void* w2;     /* routed down projection  (device) */
    const uint8_t* s1;  /* MXFP4 (u8) or FP8 (fp32) scales of w1, w3, w2; NULL for bf16 */
    const uint8_t* s3;
    const uint8_t* s2;
    const void* ws1;    /* shared expert, bf16; NULL when Is == 0 */
    const void* ws3;
    const void* ws2;
    /* Optional copies of the down projections transposed: w2t bf16 [E, I, H]
     * (w2t[e, i, :] = w2[e, :, i]) and ws2t bf16 [Is, H] (NULL when Is == 0),
     * made once at weight load with moe_transpose_down. When both are given
     * (bf16 experts, H <= 5376), one-token moe_decode_layer calls split the down
     * projection along I: the CTA that computes rows i of an expert's SwiGLU
     * activation also streams rows i of w2t and keeps a partial output, and
     * one fixed-order sum of the partials closes the layer, so no grid
     * barrier separates the gate/up and down projections ("Chasing the
     * Batch-1 Floor", "Two fusions and a retune": expert weights re-laid
     * once at load time for the decode kernel). Other calls ignore them. */
    const void* w2t;
    const void* ws2t;
} moe_weights;

/* Bytes of workspace a call with this shape and M needs. 0 for a shape or M
 * the library rejects. At M = 1 this includes the split-K layer's partial
 * outputs (MOE_MAX_GRID x H fp32). */
#define MOE_MAX_GRID 256
size_t moe_workspace_bytes(const moe_shape* shape, int M);

/* Zeroes the whole workspace (device, ws_bytes) on `stream`; needed once
 * before the first call and after a call reported MOE_ETIMEOUT. */
int moe_workspace_init(void* ws, size_t ws_bytes, void* stream);

/* Router alone: logits = x Wg^T in fp32, softmax, top-k, renormalised
 * weights. x bf16 [M,H], Wg bf16 [E,H] (device); idx int32 [M,k] and
 * w fp32 [M,k] (device) receive the routing. */
int moe_route(const void* x, int M, const void* Wg, const moe_shape* shape,
              int32_t* idx, float* w, void* ws, size_t ws_bytes, void* stream);

/* Expert FFN with the routing given: y = sum_j w[t,j] E_{idx[t,j]}(x_t)
 * + E_shared(x_t), gate/up + SwiGLU + down + combine; each touched expert's
 * weights are read from HBM once whatever M is. idx/w (device) as returned
 * by moe_route; an idx entry may repeat within a token (its weights then
 * add). An entry outside [0, E) is skipped and reported through the status
 * word. y bf16 [M,H] (device). */
int moe_ffn(const void* x, int M, const int32_t* idx, const float* w,
            const moe_weights* weights, const moe_shape* shape, void* y,
            void* ws, size_t ws_bytes, void* stream);

/* The whole layer in one persistent launch: router, top-k, gate/up +
 * SwiGLU, down + combine, shared expert. idx_out / w_out (device) may be
 * NULL. y bf16 [M,H] (device). flags: MOE_F_*. The result is deterministic:
 * every output element is accumulated in a fixed order, so it does not
 * depend on scheduling, PDL or the run. */
int moe_decode_layer(const void* x, int M, const void* Wg,
                     const moe_weights* weights, const moe_shape* shape,
                     int32_t* idx_out, float* w_out, void* y, void* ws,
                     size_t ws_bytes, uint32_t flags, void* stream);

/* Size of the library's static device scratch (512 KiB: a Ling-3.0-flash
 * shaped layer needs 255 KiB at M = 16). */
#define MOE_STATIC_SCRATCH_BYTES 524288u

/* moe_decode_layer without a caller workspace. The papers the library
 * follows have no counterpart of this entry point: it serves callers that
 * cannot hand over a workspace. The same kernel, launch configuration and
 * arithmetic as moe_decode_layer (so the same outputs, bit for bit), but the
 * workspace is a fixed array of MOE_STATIC_SCRATCH_BYTES in the library's
 * own device memory (one per device, created when the module loads). The
 * call allocates and frees nothing. Every call looks the array's device
 * address up again (cudaGetSymbolAddress, which allocates nothing); the
 * first call on a device, and the first after a device reset moved the
 * array, zeroes it on `stream`.
 *  - Returns MOE_ESCRATCH, before touching the device, when the shape and M
 *    need more than MOE_STATIC_SCRATCH_BYTES of workspace
 *    (moe_workspace_bytes > MOE_STATIC_SCRATCH_BYTES).
 *  - All calls on a device share the one scratch: they must be ordered on
 *    one stream (or otherwise serialised), also against other threads.
 *  - flags: MOE_F_NO_PDL, MOE_F_DEBUG_FORCE_TIMEOUT, MOE_F_RESET_SCRATCH
 *    (zeroes the scratch before the launch).
 *  - The transposed down projections (w2t, ws2t) are not used: one-token
 *    calls take the same path as moe_decode_layer without them.
 *  - Failure detection: the device status word lives in the scratch; read it
 *    with moe_static_scratch_status. After MOE_ETIMEOUT every later call
 *    refuses to run (it reports MOE_ETIMEOUT again and leaves its outputs
 *    unwritten) until one is made with MOE_F_RESET_SCRATCH.
 * Other arguments, layouts and errors as moe_decode_layer. */
int moe_decode_layer_static_scratch(const void* x, int M, const void* Wg,
                                    const moe_weights* weights,
                                    const moe_shape* shape, int32_t* idx_out,
                                    float* w_out, void* y, uint32_t flags,
                                    void* stream);

/* Synchronises `stream`, then copies the device status word of this
 * device's static scratch (moe_decode_layer_static_scratch) to *dev_status:
 * MOE_OK or a device code. Allocates nothing; not for the hot path. */
int moe_static_scratch_status(void* stream, int32_t* dev_status);

/* ------------------------------------------------------------ output layer
 * Output layer (lm_head) GEMV for M = 1..16 tokens: logits fp32 [M, V] =
 * x bf16 [M, H] . W^T. "Chasing the Batch-1 Floor: Ling-3.0-flash
 * Speculative Decode on Blackwell", "bf16 router gate and lm_head"; "3 ways
 * to boost MoE inference on NVIDIA DGX Spark", "Optimization 2: Online FP8
 * LM head quantization" (157,184 x 2,560 for the model).
 *  wfmt 0: W bf16 [V, H] (H a multiple of 8), w_scale unused (may be NULL).
 *  wfmt 2: W FP8 e4m3 codes [V, H] (H a multiple of 16) and w_scale fp32 [V],
 *          one scale per row: W[v, h] = e4m3(code) * w_scale[v] (see
 *          moe_fp8_quantize with block = H). Activations stay bf16.
 * H <= 8192. Every weight byte is read once per call. ws: a device buffer of
 * at least MOE_LM_HEAD_WORKSPACE_BYTES (status word; zero it once with
 * moe_workspace_init; moe_read_status reads it). flags: MOE_F_NO_PDL. One
 * launch; errors as for the layer calls. */
#define MOE_LM_HEAD_WORKSPACE_BYTES 1024u
int moe_lm_head(const void* x, int M, const void* W, const float* w_scale,
                int V, int H, int wfmt, float* logits, void* ws,
                size_t ws_bytes, uint32_t flags, void* stream);

/* FP8 e4m3 quantisation of bf16 rows [rows, K] with one fp32 scale per
 * block of `block` consecutive elements of a row (block a multiple of 32
 * dividing K): scale = amax(block) / 448 (1 for an all-zero block), code =
 * the e4m3 value nearest to w / scale (ties to even, saturating). codes u8
 * [rows, K], scales fp32 [rows, K / block] (all device). Not on the hot
 * path: it prepares weights for moe_lm_head. */
int moe_fp8_quantize(const void* w, int64_t rows, int K, int block,
                     uint8_t* codes, float* scales, void* stream);

/* Decodes e4m3 rows with the kernels' conversion: out fp32 [rows, K] =
 * e4m3(code) * scale[row, col / block] (all device). */
int moe_fp8_dequant(const uint8_t* codes, const float* scales, int64_t rows,
                    int K, int block, float* out, void* stream);

/* Transposed copy of down projections for the split-K one-token layer:
 * w2 bf16 [n, H, I] -> w2t bf16 [n, I, H] with w2t[e, i, h] = w2[e, h, i]
 * (n = E for the routed experts, n = 1 and I = Is for the shared expert).
 * Both device, not overlapping. Not on the hot path: run it once when the
 * weights are loaded. */
int moe_transpose_down(const void* w2, int64_t n, int H, int I, void* w2t,
                       void* stream);

/* ------------------------------------------------------------- paged step
 * The operators around the layer in one decode, speculative-verify or
 * chunked-prompt step of B requests: places in a paged KV cache for the
 * step's new tokens, the write of their keys and values, their attention
 * over the cache, and the choice of tokens from the output layer's logits.
 * "Chasing the Batch-1 Floor", "The shape of a batch-1 step"; "DSpark in
 * SGLang", "Verify modes" (verify blocks of variable length).
 *
 * A step's tokens lie packed, request after request: request b's new tokens
 * are rows q_start[b] .. q_start[b + 1] - 1 of the token arrays. Rows from
 * q_start[B] on are padding (a step captured in a graph at a fixed T). The
 * lengths are device data: nothing here reads them on the host.
 *
 * Device conditions go to the status word of ws (at least
 * MOE_PAGED_WORKSPACE_BYTES, zeroed once with moe_workspace_init). */
#define MOE_PAGED_WORKSPACE_BYTES 1024u
#define MOE_PAGED_MAX_REQUESTS 4096

/* A paged KV cache: n_blocks blocks (pages) of block_size tokens. Element
 * (block i, token j, head h, d) of K lies at k + i * k_block_stride + j *
 * k_token_stride + h * k_head_stride + d (elements), and of V alike, so both
 * [block][token][head][d] and [block][head][token][d] layouts, and K and V
 * interleaved in one buffer, are described by their strides. */
typedef struct moe_kv_cache {
    void* k;
    void* v;
    int32_t dtype;      /* 0 bf16, 1 fp16 (queries and outputs alike) */
    int32_t n_blocks;   /* n_blocks * block_size <= 2^31 - 1 */
    int32_t block_size; /* a multiple of 8, at most 1024 */
    int32_t kv_heads;   /* 1..256 */
    int32_t head_dim;   /* 64 or 128 */
    int64_t k_block_stride, k_token_stride, k_head_stride; /* multiples of 8, */
    int64_t v_block_stride, v_token_stride, v_head_stride; /* at least head_dim */
} moe_kv_cache;

/* Block tables and slot maps of a step from its requests' lengths.
 * ctx_lens, new_lens int32 [B]: tokens already in the cache, new tokens.
 * Request b holds ceil(ctx_lens[b] / block_size) blocks, listed in
 * block_tables [B, max_blocks]; it needs ceil((ctx + new) / block_size). The
 * missing ones are taken from free_list [n_free] in request order, starting
 * at *free_head (0 when free_head is NULL), and written into block_tables.
 * Outputs: q_start [B + 1], seq_lens [B] = ctx + new, taken [1] (blocks
 * taken; the next step's head is *free_head + *taken) and for each of T
 * token rows slot_map [T] (block * block_size + offset, -1 for padding) and
 * positions [T] (position in its request, -1 for padding; may be NULL). The
 * call writes the same results when repeated on the same inputs.
 * B <= MOE_PAGED_MAX_REQUESTS. Outputs must not overlap inputs.
 * A negative length, an old block id below 0 or a slot beyond 2^31 - 1
 * reports MOE_EDEVICE_BAD_INDEX (the length counts as 0, the token gets slot
 * -1); running out of room reports MOE_EDEVICE_OVERFLOW. */
int moe_paged_plan(const int32_t* ctx_lens, const int32_t* new_lens, int B, const int32_t* free_list, int n_free,
                   const int32_t* free_head, int32_t* block_tables, int max_blocks, int block_size,
                   int32_t* q_start, int32_t* seq_lens, int32_t* slot_map, int32_t* positions, int T,
                   int32_t* taken, void* ws, size_t ws_bytes, void* stream);

/* Writes T tokens' keys and values into the cache: token t's head h, at
 * k_new + t * k_token_stride + h * k_head_stride (elements; multiples of 8,
 * so that slices of a fused projection's output do), goes to slot
 * slot_map[t]. Slot -1 is skipped; a slot outside the cache is skipped and
 * reported (MOE_EDEVICE_BAD_INDEX). Slots of one call must differ. */
int moe_paged_append(const void* k_new, int64_t k_token_stride, int64_t k_head_stride, const void* v_new,
                     int64_t v_token_stride, int64_t v_head_stride, int T, const int32_t* slot_map,
                     const moe_kv_cache* cache, void* ws, size_t ws_bytes, void* stream);

/* Attention of the step's new tokens over the paged cache, which already
 * holds their keys and values. q [T, q_heads, head_dim] by its strides
 * (elements, multiples of 8), q_heads a multiple of kv_heads (at most 32
 * times), T * q_heads / kv_heads < 2^28; query head h reads kv head h / (q_heads / kv_heads). Row t of
 * request b sits at position p = seq_lens[b] - (q_start[b + 1] -
 * q_start[b]) + t - q_start[b] and sees the keys j <= p, with window > 0
 * only those with j > p - window:
 *   out[t, h] = sum_j softmax_j(scale q . k_j) v_j     [T, q_heads, head_dim], contiguous
 *   lse[t, h] = ln sum_j exp(scale q . k_j)            fp32 [T, q_heads], may be NULL
 * A row that sees no key (p < 0) and padding rows get out = 0, lse = -inf.
 * Products are summed in fp32, the softmax weights rounded once to the
 * cache's type for the second product. Pages that hold no visible key are
 * not read (their table entries may be anything), and what lies in a page
 * beyond the visible keys may be anything, NaN included. A row that sees a NaN
 * score is NaN, in lse too; a value that is NaN or infinite may also reach the
 * request's rows that do not see it yet (as 0 * NaN). A visible key whose
 * page is not in [0, n_blocks), or beyond max_blocks, is reported
 * (MOE_EDEVICE_BAD_INDEX) and that request's outputs are unspecified. A
 * request with a negative length, or whose rows q_start does not place within
 * [0, T] in ascending order (moe_paged_plan with more new tokens than T), is
 * reported alike and its rows are not written, nor are padding rows where it is
 * the last one. Rows that q_start gives to two requests, or to one and to the
 * padding, are unspecified.
 * scale <= 0 takes 1 / sqrt(head_dim). block_tables int32 [B, max_blocks].
 * ws: moe_paged_attention_workspace_bytes(q_heads, cache). One workspace serves
 * any of the paged step's calls, one after another (moe_paged_attention8 and
 * other caches and heads too), if it has the largest of the sizes that they ask
 * for. The result is deterministic. */
size_t moe_paged_attention_workspace_bytes(int q_heads, const moe_kv_cache* cache);
int moe_paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int T, int q_heads,
                        const moe_kv_cache* cache, const int32_t* block_tables, int max_blocks,
                        const int32_t* q_start, const int32_t* seq_lens, int B, float scale, int window, void* out,
                        float* lse, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------- trees of drafted tokens
 * A step may verify a tree of drafted tokens of each request instead of a
 * chain: its new tokens lie packed and in the cache as ever (token i of request
 * b in the slot of position ctx + i), and parents [T] names for each the one
 * that it continues, by its place among the request's new tokens, -1 for the
 * token before all of them. A token comes after its parent. A request of more
 * than MOE_TREE_MAX_TOKENS new tokens (a prompt's chunk in the same step) is no
 * tree: its parents are not read.
 * moe_tree_plan gives for each token row the mask of the new tokens that it
 * sees (bit i: token i; its own path up to the root) and its position, ctx
 * plus its depth (positions may be NULL). Rows that are no tree's get all
 * bits and consecutive positions, padding rows (from q_start[B] on) 0 and -1.
 * q_start and seq_lens as moe_paged_plan gives them. A parent outside
 * [-1, i) counts as -1 and is reported (MOE_EDEVICE_BAD_INDEX); so is a
 * request that q_start or seq_lens place wrongly, whose rows are not written (nor
 * padding rows, where q_start places the last one so). */
#define MOE_TREE_MAX_TOKENS 64
int moe_tree_plan(const int32_t* parents, const int32_t* q_start, const int32_t* seq_lens, int B, int T, uint64_t* masks,
                  int32_t* positions, void* ws, size_t ws_bytes, void* stream);

/* moe_paged_attention without a window, in which a row sees of its request's
 * new tokens those whose bits are set in masks [T] (as from moe_tree_plan, or
 * any others; bits of tokens after its own count as 0, those of requests of
 * more than MOE_TREE_MAX_TOKENS new tokens are not read), and all tokens before
 * them. A row that sees nothing gets out = 0, lse = -inf. To go on with an
 * accepted path, read its slots (moe_paged_read) and append them to the
 * consecutive ones. */
int moe_paged_tree_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int T, int q_heads,
                             const moe_kv_cache* cache, const int32_t* block_tables, int max_blocks,
                             const int32_t* q_start, const int32_t* seq_lens, const uint64_t* masks, int B, float scale,
                             void* out, float* lse, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------- rotary positions
 * The first rotary_dim of a head's dimensions turn with the token's position
 * p, two at a time: pair i (i < rotary_dim / 2) is (x_i, x_(i + rotary_dim/2)),
 * or, interleaved, (x_2i, x_(2i+1)), and with the angle a = p f_i
 *   y_first = scale (x_first cos a - x_second sin a)
 *   y_second = scale (x_first sin a + x_second cos a)
 * in fp32, rounded once. The other dimensions are copied. Frequencies are held
 * as turns: f_i / (2 pi), its whole part dropped, in units of 2^-64 turns. p
 * times that is exact modulo one turn in 64-bit integers, of which the upper 32
 * bits are taken. moe_rope_table's turns are off by less than one unit, so the
 * angle is as good at position 2^31 - 1 as at 1, to 2^-32 turns; moe_rope_turns
 * is as good as its numbers of 64 bits, 2^-52 of a frequency, times p. */
typedef struct moe_rope_angles {
    const uint64_t* turns; /* device, [rotary_dim / 2] */
    int32_t rotary_dim;    /* a multiple of 16, at most the head's dimensions */
    int32_t interleaved;   /* 0 or 1 */
    float scale;           /* of the rotated values (1: none) */
} moe_rope_angles;

/* How frequencies base^(-2i / rotary_dim) are changed for contexts `factor`
 * times the `context` that a model was made for:
 *  LINEAR  f / factor
 *  NTK     base * factor^(rotary_dim / (rotary_dim - 2)) in place of base
 *  YARN    pairs that turn more than `high` times in `context` keep f, those
 *          of less than `low` turns get f / factor, between them by a ramp
 *          over the pair's number; scale = 0.1 ln(factor) + 1 (factor > 1)
 *  BANDS   the same borders, the ramp over the number of turns; scale 1 */
#define MOE_ROPE_NONE 0
#define MOE_ROPE_LINEAR 1
#define MOE_ROPE_NTK 2
#define MOE_ROPE_YARN 3
#define MOE_ROPE_BANDS 4
/* Fills turns (host, [rotary_dim / 2]) and *scale (host) for these settings;
 * computed on the host, once when a model is loaded. base > 1,
 * factor > 0; context >= 1 for YARN and BANDS, with low < high (low <= 0: 1,
 * high <= 0: 32 for YARN, 4 for BANDS). Settings whose base or frequencies are no
 * finite numbers of 64 bits are refused (MOE_EINVAL), with nothing written. */
int moe_rope_table(int rotary_dim, double base, int scaling, double factor, int context, double low, double high,
                   uint64_t* turns, float* scale);
/* turns [n] (host) of any frequencies [n] in radians a position (host). */
int moe_rope_turns(const double* radians, int n, uint64_t* turns);

/* Rotates T tokens' queries q [T, q_heads, head_dim] and keys k [T, kv_heads,
 * head_dim] (k NULL: queries alone), each by its strides (elements, multiples
 * of 8), into q_out and k_out by theirs (at least head_dim). An output may be
 * its input (with its strides); otherwise outputs overlap nothing. dtype 0
 * bf16, 1 fp16; head_dim a multiple of 16, at most 512; heads <= 1024.
 * positions int32 [T] as moe_paged_plan or moe_tree_plan gives them: rows at a
 * negative one are padding and stay as they are in the outputs. */
int moe_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out, int64_t q_out_token_stride,
             int64_t q_out_head_stride, int q_heads, const void* k, int64_t k_token_stride, int64_t k_head_stride,
             void* k_out, int64_t k_out_token_stride, int64_t k_out_head_stride, int kv_heads, int T, int head_dim,
             int dtype, const int32_t* positions, const moe_rope_angles* angles, void* stream);

/* moe_rope and moe_paged_append in one launch, with their results bit for bit:
 * rotates q into q_out, and writes the rotated keys and the values as they are
 * to the cache's slots. q NULL (q_heads 0): keys and values alone. A row at a
 * negative position is padding: nothing of it is written. A row with slot -1
 * writes no keys and values; a slot outside the cache is skipped and reported
 * (MOE_EDEVICE_BAD_INDEX). All of the cache's dtype. ws as for
 * moe_paged_append. */
int moe_paged_rope_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                          int64_t q_out_token_stride, int64_t q_out_head_stride, int q_heads, const void* k_new,
                          int64_t k_token_stride, int64_t k_head_stride, const void* v_new, int64_t v_token_stride,
                          int64_t v_head_stride, int T, const int32_t* positions, const int32_t* slot_map,
                          const moe_rope_angles* angles, const moe_kv_cache* cache, void* ws, size_t ws_bytes,
                          void* stream);

/* ------------------------------------------------- cache of 8-bit values
 * A paged cache whose keys and values are e4m3 codes with one power of two for
 * each token and head, an e8m0 byte: value = e4m3(code) * 2^(byte - 127). As
 * written by the append calls: for the head_dim values x of a token's head the
 * byte is that of the least exponent e >= -127 with max |x| <= 448 * 2^e, and a
 * code is the e4m3 number nearest to x * 2^-e (ties to even; no value is cut
 * off, and a power of two adds no rounding of its own), but values of which the
 * nearest is the first one beyond their type (above 61,440 in fp16, above 240 *
 * 2^120 in bf16) are held as 240 * 2^e. A head in which some value is not finite
 * gets the byte 255: all its values are NaN. Writing again what was read back, in
 * the type that it was written in, gives the same values.
 * Codes by strides as in moe_kv_cache, in bytes, multiples of 16. Scales
 * [n_blocks, kv_heads, block_size], contiguous, 16-byte aligned. block_size a
 * multiple of 16, at most 1024; the other limits as in moe_kv_cache. */
typedef struct moe_kv_cache8 {
    void* k;
    void* v;
    uint8_t* k_scale;
    uint8_t* v_scale;
    int32_t n_blocks;
    int32_t block_size;
    int32_t kv_heads;
    int32_t head_dim;
    int64_t k_block_stride, k_token_stride, k_head_stride;
    int64_t v_block_stride, v_token_stride, v_head_stride;
} moe_kv_cache8;

/* moe_paged_append into such a cache, from bf16 (dtype 0) or fp16 (1). */
int moe_paged_append8(const void* k_new, int64_t k_token_stride, int64_t k_head_stride, const void* v_new,
                      int64_t v_token_stride, int64_t v_head_stride, int T, int dtype, const int32_t* slot_map,
                      const moe_kv_cache8* cache, void* ws, size_t ws_bytes, void* stream);

/* moe_paged_rope_append into such a cache: a rotated key is rounded to dtype
 * and then quantised, as by moe_rope and moe_paged_append8. */
int moe_paged_rope_append8(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                           int64_t q_out_token_stride, int64_t q_out_head_stride, int q_heads, const void* k_new,
                           int64_t k_token_stride, int64_t k_head_stride, const void* v_new, int64_t v_token_stride,
                           int64_t v_head_stride, int T, int dtype, const int32_t* positions, const int32_t* slot_map,
                           const moe_rope_angles* angles, const moe_kv_cache8* cache, void* ws, size_t ws_bytes,
                           void* stream);

/* moe_paged_attention over such a cache, of bf16 (dtype 0) or fp16 (1) queries
 * and outputs, in one launch; masks [T] of trees as for
 * moe_paged_tree_attention, or NULL (with masks window is 0). What it says of
 * scale, window, out, lse, padding, pages and bad tables holds here. Codes and
 * powers of two are exact, queries are held in fp16 times a power of two of
 * their row's own (exact down to 2^-28 of the row's largest; any finite size, by
 * scales up to 4,096), keys whose power of two is below 2^-102 (none of them above
 * 2^-93) may count as 0, and next to queries of 2^117 / scale and more those of
 * 2^97 and more as infinite, products are summed in fp32, and the softmax weights times the values' powers of two are
 * rounded once to fp16, relative to the row's largest such weight. A key whose
 * byte is 255 gives the rows that see it NaN, and may give NaN to the request's
 * rows that do not see it yet. A request of any length is taken 32 rows (tokens
 * times the heads that share a kv head) at a time: beyond some 256 rows it is
 * faster to read its context back (moe_paged_read8) into a 16-bit cache for
 * moe_paged_attention. An output beyond its type's largest value is infinite. ws: moe_paged_attention8_workspace_bytes. */
size_t moe_paged_attention8_workspace_bytes(int q_heads, const moe_kv_cache8* cache);
int moe_paged_attention8(const void* q, int64_t q_token_stride, int64_t q_head_stride, int T, int q_heads, int dtype,
                         const moe_kv_cache8* cache, const int32_t* block_tables, int max_blocks, const int32_t* q_start,
                         const int32_t* seq_lens, const uint64_t* masks, int B, float scale, int window, void* out,
                         float* lse, void* ws, size_t ws_bytes, void* stream);

/* Reads T slots back: k_out, v_out [T, kv_heads, head_dim] by their strides
 * (elements, multiples of 8, at least head_dim) get the keys and values of
 * slot_map [T]. Slot -1 leaves its row as it is; a slot outside the cache too,
 * and is reported (MOE_EDEVICE_BAD_INDEX). A slot may be read more than once.
 * moe_paged_read copies the cache's own dtype; moe_paged_read8 gives bf16
 * (dtype 0, exact but below 2^-126) or fp16 (1: rounded once, infinite above
 * 65504). Uses: the context of a prompt chunk into a 16-bit cache that
 * moe_paged_attention's many-row kernel reads; an accepted path of a tree,
 * read from its slots and appended to the consecutive ones. */
int moe_paged_read(const moe_kv_cache* cache, const int32_t* slot_map, int T, void* k_out, int64_t k_token_stride,
                   int64_t k_head_stride, void* v_out, int64_t v_token_stride, int64_t v_head_stride, void* ws,
                   size_t ws_bytes, void* stream);
int moe_paged_read8(const moe_kv_cache8* cache, const int32_t* slot_map, int T, int dtype, void* k_out,
                    int64_t k_token_stride, int64_t k_head_stride, void* v_out, int64_t v_token_stride,
                    int64_t v_head_stride, void* ws, size_t ws_bytes, void* stream);

/* One token from each of M rows of logits [M, V] (row_stride elements from
 * row to row; dtype 0: fp32, as moe_lm_head writes, 1: bf16), each with its
 * own settings (device arrays [M], NULL: off for every row):
 *   w_i = exp((l_i - max l) / temperature); order: l descending, index ascending
 *   kept: the first top_k (top_k <= 0: all), of those the shortest run whose
 *         mass reaches top_p of theirs (top_p >= 1: all; at least one), of
 *         those the ones with w_i >= min_p (<= 0: all; above 1 counts as 1)
 *   token = the lowest index at which the kept tokens' cumulated mass, in
 *           index order, exceeds u * (their total mass)
 * temperature <= 0 (or NaN) takes the largest logit's lowest index;
 * temperature NULL is 1; a NaN top_p or min_p is off. u fp32 [M] in [0, 1)
 * (clamped to it, NaN: 0). A NaN logit counts as -inf; +inf shares all the
 * mass. Masses are summed in 64-bit
 * fixed point, so the result does not depend on any order; each is off by some
 * 2^-22 of itself and a unit of 2^-42, so where a mass meets min_p, or a sum
 * top_p or u, more closely than that, either side may be taken. token int32 [M]
 * (-1 for a row without any logit above -inf), prob fp32 [M] or NULL: the
 * token's share of the kept mass (0 with token -1). A token whose w_i is below
 * 2^-41 has no part in any of it; temperatures below 1.4e-30 count as that.
 * V <= MOE_SAMPLE_MAX_VOCAB, any M >= 1; logits aligned to their type. */
#define MOE_SAMPLE_MAX_VOCAB 720896
int moe_sample(const void* logits, int dtype, int M, int V, int64_t row_stride, const float* u,
               const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
               int32_t* token, float* prob, void* stream);

/* Synchronises `stream`, then copies the device status word of `ws` to
 * *dev_status (MOE_OK or a device code above). Not for the hot path. */
int moe_read_status(const void* ws, void* stream, int32_t* dev_status);

/* Static description of a MOE_* code. */
const char* moe_status_str(int code);

/* Dequantises MXFP4 rows with the decode the kernels use: out fp32
 * [rows, K] = e2m1(code) * 2^(scale - 127). codes u8 [rows, K/2], scales
 * u8 [rows, K/32], out (all device); K a multiple of 32. */
int moe_mxfp4_dequant(const uint8_t* codes, const uint8_t* scales,
                      int64_t rows, int K, float* out, void* stream);

/* Process-wide tuning and test options (MOE_OPT_*). Not thread-safe with
 * concurrent calls. */
int moe_set_option(int option, int64_t value);

/* Number of kernel launches the most recent launching call on this thread
 * made (1 for moe_decode_layer / moe_route / moe_ffn). */
int moe_last_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_DECODE_H */
