/*
 * qdq.h -- C ABI of libqdq: dequantisation and fused dequant-GEMV over
 * block-quantised weights, in hand-written CUDA for sm_103a (GB300).
 *
 * Block formats (all little-endian, see the per-type notes below):
 *   QDQ_Q4_K  GGUF Q4_K, 144 bytes per 256 weights ("S21 The Capstone: picoLM,
 *             in Python", section 2 K-quants): fp16 d, fp16 dmin, 12 bytes of
 *             packed 6-bit scales and mins (one pair per 32-weight sub-block),
 *             128 nibble bytes. w = d*sc*q - dmin*mn.
 *   QDQ_Q6_K  GGUF Q6_K, 210 bytes per 256 weights ("PicoLM Q6_K quantisation
 *             bug", block_q6_K struct): ql[128] low 4 bits, qh[64] high 2 bits,
 *             int8 scales[16] (one per 16 weights), fp16 d. w = d*sc*(q6-32).
 *             The ql/qh bit placement follows the ggml layout.
 *   QDQ_Q8_0  PETIT q8_0, 36 bytes per 32 weights ("PETIT", How the pieces
 *             match): fp32 scale d, 32 int8 q. w = d*q. (Not ggml's q8_0, whose
 *             scale is fp16.)
 *   QDQ_Q4_0  PETIT q4_0, 18 bytes per 32 weights (same section): fp16 scale d,
 *             16 bytes; byte i holds weight i (low nibble) and weight i+16 (high
 *             nibble). w = (q-8)*d.
 *   More GGUF formats. The pages name eight GGUF formats and give Q2_K's size
 *   (84 bytes per 256 weights, "S21 The Capstone: picoLM, in Python", section
 *   2); the layouts follow the published ggml block layouts:
 *   QDQ_Q5_0       22 bytes per 32: fp16 d; qh (4 bytes, little-endian word, bit
 *                  i = fifth bit of weight i); 16 nibble bytes as q4_0.
 *                  w = (q-16)*d, q = nibble | bit << 4.
 *   QDQ_Q5_1       24 bytes per 32: fp16 d, fp16 m, qh, 16 nibble bytes.
 *                  w = q*d + m.
 *   QDQ_Q8_0_GGML  34 bytes per 32: fp16 d, 32 int8. w = q*d.
 *   QDQ_Q2_K       84 bytes per 256: 16 bytes of (scale | min << 4) per 16
 *                  weights, 64 bytes of 2-bit quants (weight 128n + 32j + l: bits
 *                  2j..2j+1 of byte 32n + l, pair 8n + 2j + l/16), fp16 d, fp16
 *                  dmin. w = d*sc*q - dmin*mn.
 *   QDQ_Q5_K       176 bytes per 256: fp16 d, fp16 dmin, the 12 scale/min bytes
 *                  of Q4_K (same packing), qh[32], qs[128]. Weight 64c + 32h + l:
 *                  low four bits in the low (h = 0) or high (h = 1) nibble of
 *                  qs[32c + l], fifth bit at bit 2c + h of qh[l]; sub-block 2c + h.
 *                  w = d*sc*q - dmin*mn, q in 0..31.
 *   QDQ_Q3_K       110 bytes per 256: hmask[32], qs[64], 12 bytes of sixteen
 *                  6-bit scales, fp16 d. Weight 128n + 32j + l: bits 2j..2j+1 of
 *                  qs[32n + l], minus 4 unless bit 4n + j of hmask[l] is set;
 *                  scale s = 8n + 2j + l/16 keeps its low four bits in byte s
 *                  (s < 8, low nibble) or s - 8 (high nibble), its top two at
 *                  bit 2(s/4) of byte 8 + s%4. w = d*(scale - 32)*q.
 *   These six are decoded by qdq_dequant and multiplied by qdq_gemv (a
 *   separate exact-per-weight kernel, any batch); groups and plans take the
 *   main four only (QDQ_ERR_TYPE).
 *
 * Conventions for every call:
 *   - Pointers named W, blocks, x, y, out are DEVICE pointers (cudaMalloc'd or
 *     managed) on the current device, 16-byte aligned. A host pointer gives
 *     QDQ_ERR_PTR, a misaligned one QDQ_ERR_ALIGN, a NULL one QDQ_ERR_PTR.
 *   - A weight matrix is rows x cols (out x in, "PETIT": weights stored out x in,
 *     a projection is one gemv), row-major, each row cols/QK whole blocks.
 *     cols must be a multiple of the block's weight count QK (the caller pads,
 *     as PETIT's exporter does), else QDQ_ERR_SHAPE.
 *   - x is [batch][cols] fp32 and y is [batch][rows] fp32, both contiguous. y is
 *     overwritten, never accumulated into.
 *   - rows == 0 or n == 0 is a no-op returning QDQ_OK.
 *   - Calls are asynchronous on `stream` (0 = the legacy default stream). Launch
 *     failures return QDQ_ERR_CUDA. A device-side failure (a bounded wait that
 *     ran out) is recorded in a per-device status word, read back by
 *     qdq_get_device_status(). Nothing aborts, traps or exits.
 *   - The caller owns every buffer. Besides plans, models and paged caches (below),
 *     the library keeps no device allocations: only a status word in module memory
 *     per device.
 *   - Calls on different streams may run concurrently. Only sm_103 (GB300)
 *     devices are accepted; others give QDQ_ERR_DEVICE.
 */
#ifndef QDQ_H
#define QDQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *qdq_stream_t; /* == cudaStream_t */

enum qdq_type {
    QDQ_Q4_0 = 1, QDQ_Q8_0 = 2, QDQ_Q4_K = 3, QDQ_Q6_K = 4,
    /* More GGUF formats (see the notes below the main four): */
    QDQ_Q5_0 = 5, QDQ_Q5_1 = 6, QDQ_Q8_0_GGML = 7, QDQ_Q2_K = 8, QDQ_Q5_K = 9, QDQ_Q3_K = 10
};

enum qdq_status {
    QDQ_OK = 0,
    QDQ_ERR_TYPE = -1,     /* unknown block type */
    QDQ_ERR_SHAPE = -2,    /* negative size, cols or n not a multiple of QK, batch < 1, row too wide */
    QDQ_ERR_ALIGN = -3,    /* a pointer not 16-byte aligned */
    QDQ_ERR_PTR = -4,      /* NULL or host pointer */
    QDQ_ERR_CUDA = -5,     /* a CUDA runtime call or kernel launch failed */
    QDQ_ERR_TIMEOUT = -6,  /* a device-side bounded wait ran out (from qdq_get_device_status) */
    QDQ_ERR_DEVICE = -7,   /* current device is not sm_103 */
    QDQ_ERR_LIMIT = -8,    /* more GEMVs or levels than a plan supports */
    QDQ_ERR_FORMAT = -9,   /* a malformed or truncated GGUF file */
    QDQ_ERR_NOT_FOUND = -10, /* no such GGUF metadata key */
    QDQ_ERR_BOUNDS = -11     /* debug builds (-DQDQ_DEBUG) only: a device-side index or
                                alignment check failed and the access was skipped
                                (from qdq_get_device_status) */
};

/* Bytes per block and weights per block of a type; -1 for an unknown type. */
int qdq_block_bytes(int type);
int qdq_block_weights(int type);

/* Static text for a status code. */
const char *qdq_status_string(int status);

/* ---------------------------------------------------------------------------
 * qdq_dequant: out[i] = w_i for i < n, the fp32 value of each weight.
 * Cited: "S21 The Capstone: picoLM, in Python", section 2 (dequantize_q4_K:
 * raw blocks + count n -> n floats); "PicoLM Q6_K quantisation bug"
 * (dequantize_row_q6_K); "PETIT", What makes it fast & small.
 * `blocks` holds n/QK consecutive blocks; `out` holds n floats. Each value is
 * evaluated in the pages' order with IEEE fp32 round-to-nearest and no fused
 * multiply-add, so the result is bit-for-bit that of a plain CPU decoder.
 * n must be a multiple of QK (QDQ_ERR_SHAPE).
 * qdq_dequant runs on the legacy default stream, qdq_dequant_async on `stream`.
 * ------------------------------------------------------------------------- */
int qdq_dequant(int type, const void *blocks, int64_t n, float *out_f32);
int qdq_dequant_async(int type, const void *blocks, int64_t n, float *out_f32,
                      qdq_stream_t stream);

/* ---------------------------------------------------------------------------
 * qdq_gemv: y[b][r] = sum_c w[r][c] * x[b][c] for b < batch, r < rows,
 * with dequantisation fused into the dot product: only the quantised bytes of W
 * cross the memory bus ("S21 The Capstone: picoLM, in Python", section 3,
 * fused dequant + dot; picoLM's matmul(out, x, W, n, d, type); PETIT gemv_q8 /
 * gemv_q4 / gemm).
 * Accumulation is fp32. Against the exact (double) sum y_ref the result meets
 * |y - y_ref| <= 1e-5 * sum_c |w[r][c] x[b][c]| + 1e-7 for finite inputs.
 * Batch 1..4 (1..3 for q8_0 and q4_0) runs the streaming
 * CUDA-core kernel (each decoded weight meets every batch column); larger
 * batches the tensor-core path (exact integer quants x bf16-split x on tcgen05,
 * scales applied per group in fp32). Any row width is accepted (wide rows are
 * split into column chunks inside the streaming kernel). Neither path allocates
 * memory: the tensor-core kernel splits x into its bf16 operand in shared memory.
 * ------------------------------------------------------------------------- */
int qdq_gemv(int type, const void *W, int64_t rows, int64_t cols, const float *x, float *y,
             int batch, qdq_stream_t stream);

/* One GEMV of a group or plan. */
typedef struct qdq_gemv_desc {
    int32_t type;
    int32_t reserved;
    const void *W;
    int64_t rows;
    int64_t cols;
    const float *x; /* [batch][cols] */
    float *y;       /* [batch][rows] */
} qdq_gemv_desc;

/* Up to 8 independent GEMVs with a common batch, in one launch (for instance
 * q, k and v of one layer, which may mix Q4_K and Q6_K). Same rules as
 * qdq_gemv for each; batch must be <= 8. */
int qdq_gemv_group(const qdq_gemv_desc *descs, int n, int batch, qdq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Plans: a whole decode step's GEMVs in one persistent launch.
 * ("S21 The Capstone: picoLM, in Python", section 4: model_forward runs, per
 * layer, the q/k/v, output, gate/up and down projections, then the output head.)
 * descs[i] belongs to dependency level level[i]; levels must be non-decreasing
 * from 0. All GEMVs of level k complete (their y written and visible) before any
 * GEMV of level k+1 reads its x; weight bytes of later levels may be fetched
 * earlier, since weights never depend on earlier outputs. batch <= 8; at most
 * 192 GEMVs and 128 levels (QDQ_ERR_LIMIT). The plan copies the descriptors
 * (not the buffers they point to, which must stay valid while the plan is run)
 * and allocates one small device array of level counters; destroy frees it.
 * Runs of one plan must not overlap on the GPU. If qdq_get_device_status()
 * reports QDQ_ERR_TIMEOUT after a run, call qdq_plan_reset() before the next.
 * ------------------------------------------------------------------------- */
typedef struct qdq_plan qdq_plan;
int qdq_plan_create(const qdq_gemv_desc *descs, const int *level, int n, int batch,
                    qdq_plan **plan_out);

/* ---------------------------------------------------------------------------
 * Step glue fused into a plan's GEMVs ("S21 The Capstone: picoLM, in Python",
 * section 4, model_forward: rmsnorm before the q/k/v and gate/up projections,
 * SwiGLU between gate/up and down, residual additions after the output and down
 * projections, and the output head whose largest logit greedy decoding takes;
 * "PETIT", What makes it fast & small: RMSNorm + SwiGLU Llama block).
 * opts[i] applies to descs[i]:
 *   x_op  QDQ_X_PLAIN    the GEMV reads x as given.
 *         QDQ_X_RMSNORM  it reads x / sqrt(mean(x^2) + eps) * norm_w (the mean
 *                        over the cols entries of each batch column), computed
 *                        while x is staged; norm_w is [cols] fp32.
 *         QDQ_X_SWIGLU   it reads silu(x) * x2 with silu(g) = g / (1 + exp(-g));
 *                        x is the gate output, x2 the up output, both
 *                        [batch][cols].
 *         QDQ_X_MUL      it reads x * x2 elementwise (x2 [cols]; batch 1): with
 *                        a gate GEMV stored through QDQ_Y_SILU, the same SwiGLU
 *                        product with silu evaluated once per element instead
 *                        of once per CTA that stages it.
 *   y_op  QDQ_Y_STORE    y = W x' (as qdq_gemv).
 *         QDQ_Y_ADD      y += W x' (a residual addition; y must not be read by
 *                        another GEMV of the same level).
 *         QDQ_Y_SILU     y = silu(W x'), the same silu as QDQ_X_SWIGLU's. Batch
 *                        1 and cols <= 4096 (a row's sum is complete in one
 *                        store).
 *   argmax  NULL, or a device int64: after the run it holds the index of the
 *           largest y of this GEMV (the smallest such index on ties). At most
 *           one GEMV of a plan, in its last level, batch 1, cols <= 8192.
 * GEMVs of one level that read the same x must use the same x_op, x2, norm_w
 * and eps. Every option is applied inside the plan's single kernel: no pass of
 * its own. Errors: QDQ_ERR_SHAPE for a rule above broken, QDQ_ERR_PTR /
 * QDQ_ERR_ALIGN for a bad x2, norm_w or argmax pointer. The plan then also
 * owns 16 bytes of device memory for the argmax.
 * ------------------------------------------------------------------------- */
enum qdq_x_op { QDQ_X_PLAIN = 0, QDQ_X_RMSNORM = 1, QDQ_X_SWIGLU = 2, QDQ_X_MUL = 3 };
enum qdq_y_op { QDQ_Y_STORE = 0, QDQ_Y_ADD = 1, QDQ_Y_SILU = 2 };
typedef struct qdq_gemv_opts {
    int32_t x_op;
    int32_t y_op;
    const float *x2;
    const float *norm_w;
    float eps;
    int32_t reserved;
    int64_t *argmax;
} qdq_gemv_opts;
int qdq_plan_create_ex(const qdq_gemv_desc *descs, const qdq_gemv_opts *opts, const int *level, int n,
                       int batch, qdq_plan **plan_out);
int qdq_plan_run(qdq_plan *plan, qdq_stream_t stream);
/* The same run with host I/O: copies x_host (every distinct x buffer of the
 * plan, concatenated in order of first use, each [batch][cols]) to the plan's x
 * buffers, runs, and copies every GEMV's y (concatenated in descriptor order)
 * into y_host. Host buffers should be pinned. Byte counts are returned through
 * h2d_bytes / d2h_bytes when non-NULL. */
int qdq_plan_run_io(qdq_plan *plan, const float *x_host, float *y_host, qdq_stream_t stream,
                    int64_t *h2d_bytes, int64_t *d2h_bytes);
int qdq_plan_reset(qdq_plan *plan, qdq_stream_t stream);
void qdq_plan_destroy(qdq_plan *plan);
/* Number of kernel launches one qdq_plan_run makes (1). */
int qdq_plan_launches(const qdq_plan *plan);

/* ---------------------------------------------------------------------------
 * qdq_gemv_levels_noalloc: the same computation as a plan built from (descs,
 * level, n, batch) and run once, for callers that cannot allocate device
 * memory (a host framework that owns the whole memory budget, a serving loop
 * that must not call the allocator, a process whose allocations all go through
 * another component). It calls no cudaMalloc or other allocating routine: the
 * level counters live in a 512-byte array in the library's module memory,
 * which every GPU that loads the library keeps until exit. No counterpart on
 * the pages: this is a deployment variant of the plan launch.
 * Limits: at most 128 levels (QDQ_ERR_LIMIT), 192 GEMVs, batch <= 8.
 * The array is shared by every call; each call clears the counters it uses on
 * `stream` first. Calls whose kernels overlap on the GPU race on the array, so
 * serialise them (one stream, or events). The first call on a device looks up
 * the array's device address with that device current; make that first call
 * before any stream capture.
 * ------------------------------------------------------------------------- */
int qdq_gemv_levels_noalloc(const qdq_gemv_desc *descs, const int *level, int n, int batch,
                            qdq_stream_t stream);

/* ---------------------------------------------------------------------------
 * qdq_rope_attention: the attention block of one decode position
 * ("S21 The Capstone: picoLM, in Python", section 4, model_forward, and section
 * 3 for the RoPE layout; "PETIT", How the pieces match: RoPE base, per head).
 *   1. RoPE in the interleaved layout: within each head, the pair
 *      (v[2i], v[2i+1]) of q and of k turns by pos * rope_base^(-2i/head_dim).
 *   2. The cache is fp16: the turned k and the v of this position are rounded
 *      to fp16 (to nearest even) and stored at row pos of k_cache / v_cache.
 *   3. For each query head h, with KV head g = h / (n_heads / n_kv_heads):
 *      out_h = sum_{t <= pos} p_t v_t, p = softmax_t(k_t . q_h / sqrt(head_dim)),
 *      every k_t, v_t in its fp16 value. Online softmax in fp32 (no score array).
 * q: [n_heads * head_dim]; k, v: [n_kv_heads * head_dim]; out: [n_heads *
 * head_dim], fp32 device buffers. k_cache, v_cache: [max_seq][n_kv_heads *
 * head_dim] fp16 bit patterns, device, owned by the caller; rows < pos must hold
 * earlier positions. head_dim even and <= 256, n_heads a multiple of n_kv_heads,
 * 0 <= pos < max_seq (else QDQ_ERR_SHAPE). One launch of n_heads CTAs.
 * ------------------------------------------------------------------------- */
int qdq_rope_attention(const float *q, const float *k, const float *v, uint16_t *k_cache,
                       uint16_t *v_cache, float *out, int n_heads, int n_kv_heads, int head_dim,
                       int pos, int max_seq, float rope_base, qdq_stream_t stream);

/* ---------------------------------------------------------------------------
 * A one-token forward pass of a Llama-architecture model over block-quantised
 * weights ("S21 The Capstone: picoLM, in Python", section 4, model_forward(m,
 * token, pos)): h = the token's embedding row (decoded); per layer
 *   h += Wo attention(rope(Wq n), rope(Wk n), Wv n),  n = rmsnorm(h, attn_norm)
 *   h += Wdown (silu(Wgate n') * Wup n'),              n' = rmsnorm(h, ffn_norm)
 * then logits = Wout rmsnorm(h, output_norm) and their argmax.
 * The embedding's row length in bytes must be a multiple of 16 (QDQ_ERR_ALIGN).
 * Weights are out x in (rows x cols) blocks of any of the four types, device
 * memory owned by the caller, which must outlive the model. layer.w[] and
 * layer.type[] are in the order q, k, v, o, gate, up, down with shapes q, o:
 * dim x dim; k, v: kv x dim (kv = n_kv_heads * dim / n_heads); gate, up:
 * hidden x dim; down: dim x hidden. Norm weights are fp32 device vectors [dim].
 * The model allocates its activations, the fp16 key/value cache
 * ([n_layers][max_seq][kv] each) and one plan in create, and frees them in
 * destroy. A forward call runs 2 launches on `stream`: the embedding row's
 * decode, then one plan of every layer's levels (q/k/v with the attention norm;
 * attention; o with the residual; gate/up with the FFN norm, the gate stored
 * through silu when dim <= 4096; down reading gate * up, or silu(gate) * up
 * when wider, with the residual) and the head with its argmax. Positions must
 * be run in order 0, 1, ... (a position reads the cache rows before it).
 * qdq_llama_buffers returns the device addresses of the logits [vocab], argmax
 * (one int64), the residual stream h [dim] and the two caches.
 * ------------------------------------------------------------------------- */
typedef struct qdq_llama_config {
    int32_t dim, hidden, n_layers, n_heads, n_kv_heads, vocab, max_seq, reserved;
    float rope_base; /* 10000 in PETIT */
    float norm_eps;  /* rmsnorm epsilon */
} qdq_llama_config;
typedef struct qdq_llama_layer {
    const void *w[7];
    int32_t type[7];
    int32_t reserved;
    const float *attn_norm;
    const float *ffn_norm;
} qdq_llama_layer;
typedef struct qdq_llama qdq_llama;
int qdq_llama_create(const qdq_llama_config *cfg, const void *token_embd, int embd_type,
                     const qdq_llama_layer *layers, const float *output_norm, const void *output,
                     int output_type, qdq_llama **model_out);
int qdq_llama_forward(qdq_llama *model, int token, int pos, qdq_stream_t stream);
int qdq_llama_buffers(const qdq_llama *model, float **logits, int64_t **argmax, float **hidden,
                      uint16_t **k_cache, uint16_t **v_cache);
int qdq_llama_launches(const qdq_llama *model);
void qdq_llama_destroy(qdq_llama *model);

/* ---------------------------------------------------------------------------
 * Serving several sequences: a paged key/value cache, the append of new tokens
 * to it, attention of a chunk of new tokens over it, and sampling. No
 * counterpart on the pages: the same step as qdq_rope_attention and the head's
 * argmax ("S21 The Capstone: picoLM, in Python", section 4) for a batch of
 * sequences of any lengths, prompts and single tokens alike.
 *
 * The cache is two pools of pages owned by the caller, keys and values, each
 * [n_layers][n_pages][page_size][n_kv_heads][head_dim] of fp16 or bf16. Which
 * page holds which positions is the caller's to decide: position j of a
 * sequence lives in row j % page_size of page page_table[seq][j / page_size].
 * A handle keeps the geometry, the rotation's frequency table and the attention's
 * workspace (all device memory it needs, 1152 bytes x SMs x head_dim x 2 and a little:
 * 45 MB at 128 dims; the calls allocate nothing).
 *
 * A step's batch (all arrays int32 on the device, 4-byte aligned, read when the
 * kernels run, so a captured graph replays with their new contents):
 *   q_start[n_seqs + 1]  the new tokens of sequence s are rows q_start[s] ..
 *                        q_start[s+1] - 1 of q, k, v; starts at 0, never falls
 *                        and never exceeds n_tokens. Rows from q_start[n_seqs]
 *                        on belong to no sequence: their outputs are not written.
 *   kv_len[n_seqs]       positions of the sequence, the new tokens included: its
 *                        token i of n is at position kv_len - n + i.
 *   page_table[n_seqs][max_pages]  page numbers; a position whose entry is not in
 *                        [0, n_pages), or is past max_pages pages, is absent: it
 *                        is not written and not attended to.
 * n_seqs <= 1024, max_pages * page_size <= 2^30 (QDQ_ERR_LIMIT).
 * ------------------------------------------------------------------------- */
enum qdq_float_type { QDQ_F32 = 1, QDQ_F16 = 2, QDQ_BF16 = 3, QDQ_E4M3 = 4 };

typedef struct qdq_paged_config {
    int32_t type;             /* of the pools: QDQ_F16 or QDQ_BF16 */
    int32_t n_layers, n_pages;
    int32_t page_size;        /* 16, 32, 64, 128 or 256 positions */
    int32_t n_heads, n_kv_heads; /* n_heads a multiple of n_kv_heads, at most 32 times it */
    int32_t head_dim;         /* 64 or 128 */
    int32_t rope_dim;         /* leading dims of a head that turn: a multiple of 8 in 0..head_dim */
    int32_t rope_interleaved; /* 1: pairs (2i, 2i+1); 0: pairs (i, i + rope_dim/2) */
    float rope_base;          /* pair i turns by position * rope_base^(-2i/rope_dim) */
} qdq_paged_config;
typedef struct qdq_paged_batch {
    int32_t n_seqs, n_tokens, max_pages, reserved;
    const int32_t *q_start, *kv_len, *page_table;
} qdq_paged_batch;
typedef struct qdq_paged qdq_paged;
/* A cache of e4m3 values (type QDQ_E4M3) keeps each key and value in eight bits, with a
 * scale for each 16 positions (of one page) and head: a value is its e4m3 value times
 * 2^(b - 127), b the scale's byte, with b - 127 in -40 .. 40 (others count as the nearest of
 * those). Pools: [n_layers][n_pages][n_kv_heads][page_size][head_dim] (a page's heads one
 * after the other), scales [n_layers][n_pages][n_kv_heads][page_size / 16]. Queries are fp16;
 * append takes fp32, fp16 or bf16 rows, and attention gives any of them. */
/* The pools must outlive the handle, and so must the scales. Attention calls of one handle must not overlap on
 * the GPU (they share the workspace); use one handle per stream otherwise. If
 * qdq_get_device_status() reports QDQ_ERR_TIMEOUT after one, destroy the handle and
 * create another before the next. */
int qdq_paged_create(const qdq_paged_config *cfg, void *k_pages, void *v_pages, qdq_paged **out);
int qdq_paged_create_e4m3(const qdq_paged_config *cfg, void *k_pages, void *v_pages, uint8_t *k_scales,
                          uint8_t *v_scales, qdq_paged **out);
void qdq_paged_destroy(qdq_paged *cache);

/* qdq_paged_append: one pass over the new tokens' q, k and v rows.
 *   y = x / sqrt(mean(x^2) + eps) * w over each head (q_norm, k_norm: fp32
 *       [head_dim], or NULL for none),
 *   q and k turned at their token's position (angles reduced modulo a turn
 *   exactly, from frequencies within 2^-54 turn, so up to position 2^28 they are
 *   those of the formula to fp32's rounding), all arithmetic in fp32,
 *   q_out[n_tokens][n_heads * head_dim] = q in the pools' type; k and v rounded
 *   to the pools' type and stored in `layer` of the pools (one rounding each).
 * in_type: QDQ_F32 (a GEMV's output) or the pools' type. Row strides are in
 * elements; every row 16-byte aligned. A token at a negative position (kv_len
 * below its sequence's new tokens) gets a zero q_out row and is not stored.
 * Into a cache of e4m3 values: q_out is fp16 (values beyond its range become its largest).
 * A block of 16 positions and a head gets the least e in -40 .. 40 with |x| <= 448 * 2^e for
 * each finite new x; where the block begins with earlier positions, not less than its own e,
 * and if that grows, their values are rescaled (exact but for values that fall below e4m3's
 * normal range, 2^-6 * 2^e, which are rounded again). x * 2^-e is rounded once to e4m3;
 * infinities become 448 * 2^e of their sign, what is no number stays none. Rows of a block
 * behind the new ones are left as they are. No two sequences of a call may write to one page. */
int qdq_paged_append(qdq_paged *cache, int layer, const qdq_paged_batch *batch, int in_type, const void *q,
                     int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                     const float *q_norm, const float *k_norm, float eps, void *q_out, qdq_stream_t stream);

/* qdq_paged_attention: for token t at position p of its sequence and query head h
 * with kv head h / (n_heads / n_kv_heads),
 *   out[t][h] = sum_j a_j v_j,  a = softmax_j(scale * q . k_j),
 * over the sequence's positions j <= p, and j > p - window when window > 0.
 * scale: of either sign, or 0 (the mean of the values); scale * log2(e) has to be
 * finite in fp32, over a cache of e4m3 values times 2^40 too (QDQ_ERR_SHAPE).
 * q: [n_tokens][n_heads * head_dim] of the pools' type (append's q_out), out: of
 * the pools' type or QDQ_F32; row strides in elements, rows 16-byte aligned.
 * lse (NULL or fp32 [n_tokens][n_heads]): log sum_j exp(scale * q . k_j).
 * Scores, maxima, sums and the accumulator are fp32. The softmax weights meet v in
 * the pools' type, as its matrix product takes them. A sequence's new tokens are
 * taken in blocks of 2 t, t = 128 / (n_heads / n_kv_heads); a block of at most t (a
 * single token, a short last piece) and any block of an fp32 out have the weights
 * in two terms, which keep 16 bits of each or more; other blocks have them rounded
 * once, an error of the size of the 16-bit out's own rounding. (fp16's smallest
 * step: a weight may be off by 2^-32 of the row's largest besides.) A token with
 * nothing to attend to gets a zero row and lse = -inf. Keys and values of
 * positions outside a sequence's range are never used, whatever they hold; values
 * inside it are taken to be finite (a position that only later tokens of a chunk
 * attend to has weight zero for the earlier ones, and 0 x inf is no number).
 * Over a cache of e4m3 values the query meets the keys' e4m3 values exactly and their scales
 * in fp32; a weight, with its value's scale in it, meets the values in two fp16 terms, or in
 * one, rounded once, for a 16-bit out where a step has more than 16 rows (tokens x query
 * heads of a kv head) a sequence on average.
 * One launch; results do not depend on timing (no floating-point atomics). */
int qdq_paged_attention(qdq_paged *cache, int layer, const qdq_paged_batch *batch, const void *q, int64_t q_stride,
                        int out_type, void *out, int64_t out_stride, float scale, int window, float *lse,
                        qdq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Attention over a few pages of a long sequence, chosen for each token and kv head. No
 * counterpart on the pages. Caches of any type; a page's number in these calls is its place
 * in the sequence's page table (positions number * page_size on).
 *
 * qdq_paged_key_bounds: bounds of the keys of each page that holds a new token of the batch
 * (call it after the append), over the page's positions below kv_len, for every kv head:
 *   E the least in -100 .. 121 with |k| <= 127 * 2^E (121 where a key is infinite),
 *   bounds[0][d] = ceil(max k_d * 2^-E), bounds[1][d] = floor(min k_d * 2^-E),
 * bounds: int8 [n_layers][n_pages][n_kv_heads][2][head_dim], 16-byte aligned; scales: bytes
 * E + 127, [n_layers][n_pages][n_kv_heads]; both the caller's, by page of the pool. Keys that are
 * no number do not count. Pages without a new token keep their bounds.
 *
 * qdq_paged_select_pages: for each token at position p and each kv head, the numbers of
 * n_select of the pages that hold positions up to p (those with a page in the table), in
 * rising order, then -1: pages[n_tokens][n_kv_heads][n_select], int32. Fewer pages than
 * n_select: all of them. The first n_first and the last n_last of the sequence's pages up to
 * p's are taken always (n_first + n_last <= n_select), of the others those of the highest score,
 * the lowest number first among equals. The score of a page is the largest over the kv
 * head's query heads of
 *   2^s * sum_d qi_d * bounds[qi_d < 0][d]    (of bounds, the largest that qi . k can be),
 * qi = rint(q * 2^-Eq) with Eq for the head's q as E for the keys, s = Eq + E inside -100 .. 100:
 * an integer times a power of two, so the selection is exact. It ranks pages by how large scale *
 * q . k can be for a positive scale. q as for attention. max_pages <= 32768 (QDQ_ERR_LIMIT). Rows
 * of no sequence are not written; a token at a negative position gets -1 throughout.
 *
 * qdq_paged_attention_pages: as qdq_paged_attention without a window, over the positions up to
 * the token's own that lie in the listed pages: pages as above. An entry counts if it is not
 * negative and larger than the one before it. A token with nothing to attend to gets a zero row
 * and lse = -inf. The weights meet the values in two terms. An attention call of its handle: it uses
 * the workspace, and must not overlap with another.
 * ------------------------------------------------------------------------- */
int qdq_paged_key_bounds(qdq_paged *cache, int layer, const qdq_paged_batch *batch, int8_t *bounds, uint8_t *scales,
                         qdq_stream_t stream);
int qdq_paged_select_pages(qdq_paged *cache, int layer, const qdq_paged_batch *batch, const void *q, int64_t q_stride,
                           const int8_t *bounds, const uint8_t *scales, int n_select, int n_first, int n_last,
                           int32_t *pages, qdq_stream_t stream);
int qdq_paged_attention_pages(qdq_paged *cache, int layer, const qdq_paged_batch *batch, const void *q, int64_t q_stride,
                              const int32_t *pages, int n_select, int out_type, void *out, int64_t out_stride,
                              float scale, float *lse, qdq_stream_t stream);

/* ---------------------------------------------------------------------------
 * qdq_sample: the next token of each row of logits, from given random numbers.
 * logits: rows x vocab of `type` (QDQ_F32, QDQ_F16, QDQ_BF16), row stride in
 * elements. Per row (device arrays of `rows`, 4-byte aligned; NULL switches the
 * filter off, a NULL temperature is 1):
 *   weights w_i = exp((l_i - max l) * (1 / temperature)) in fp32, entries ordered
 *   by logit, the lowest index first among equals;
 *   top_k  keeps the first top_k entries (<= 0: all);
 *   top_p  of those, keeps an entry while the mass before it is < top_p times
 *          their mass (>= 1: all; the first is always kept);
 *   min_p  of those, keeps entries with w_i >= min_p (min_p above 1 counts as 1);
 *   tokens[row] = the first index, in index order, at which the running mass of
 *   the kept entries exceeds u[row] times their whole mass (u in [0, 1); at u = 1
 *   the last kept index).
 * temperature <= 0 takes the largest logit, the lowest index on ties. Masses are
 * summed in 64-bit fixed point (units of 2^-44 of the largest weight), so they do
 * not depend on any order. NaN logits count as -inf; a row with nothing above
 * -inf gives token -1 and log-probability -inf. logprobs (may be NULL): the log
 * of the chosen entry's share of the kept mass. vocab <= 2^18 (QDQ_ERR_LIMIT).
 * ------------------------------------------------------------------------- */
int qdq_sample(int type, const void *logits, int64_t stride, int rows, int vocab, const float *temperature,
               const int32_t *top_k, const float *top_p, const float *min_p, const float *u, int64_t *tokens,
               float *logprobs, qdq_stream_t stream);

/* ---------------------------------------------------------------------------
 * qdq_quantize: fp32 values -> PETIT q8_0 or q4_0 blocks, the exporter's step
 * ("PETIT", What makes it fast & small; How the pieces match: q8_0 = fp32 scale
 * + 32 int8, q4_0 = fp16 scale + 16 nibble bytes read as (q - 8) * d, low
 * nibbles = weights 0..15, values zero-padded to a multiple of 32).
 * The scale rule is not on the pages; this library's reading, per block of 32:
 *   q8_0: d = amax / 127, q = clamp(rint(x / d), -127, 127)   (q = 0 if d = 0)
 *   q4_0: d = fp16(amax / 7), q = clamp(rint(x / d) + 8, 0, 15) (q = 8 if d = 0)
 * with amax = max |x| over the block and every operation in binary32 (the
 * division correctly rounded, rint halving to even), so the codes are those of
 * any CPU that follows the same steps. A q4_0 block whose amax / 7 exceeds the
 * fp16 range (amax > 458528) gets d = inf, which the format cannot represent:
 * its weights decode to NaN. x: n fp32 (device); blocks: ceil(n/32)
 * blocks (device). Both 16-byte aligned. Asynchronous on `stream`.
 * ------------------------------------------------------------------------- */
int qdq_quantize(int type, const float *x, int64_t n, void *blocks, qdq_stream_t stream);

/* ---------------------------------------------------------------------------
 * GGUF container, read from memory (for instance a mapped file): header,
 * metadata, tensor index ("S21 The Capstone: picoLM, in Python", section 1:
 * a header, self-describing metadata, a tensor index of (name, shape, type,
 * offset), padding to general.alignment, then one blob; each tensor is a byte
 * range at a known offset). Host-only, no device work; every read is bounds
 * checked (QDQ_ERR_FORMAT for a bad magic or version, a truncated file, an
 * offset that is not a multiple of the alignment or runs past the end).
 * qdq_gguf_parse fills up to max_tensors entries (QDQ_ERR_LIMIT if the file has
 * more) with the tensors' names, dims (dims[0] innermost: the row length),
 * GGUF type code, the library type that decodes it (QDQ_Q4_0 for type 2,
 * QDQ_Q5_0 for 6, QDQ_Q5_1 for 7, QDQ_Q8_0_GGML for 8, QDQ_Q2_K for 10,
 * QDQ_Q3_K for 11, QDQ_Q4_K for 12, QDQ_Q5_K for 13, QDQ_Q6_K for 14, else 0),
 * absolute byte offset and size.
 * qdq_gguf_find_kv locates a metadata value: its GGUF value type and the byte
 * offset of the value (QDQ_ERR_NOT_FOUND if the key is absent).
 * ------------------------------------------------------------------------- */
typedef struct qdq_gguf_tensor {
    char name[96];
    int32_t n_dims;
    int32_t ggml_type;
    int32_t qdq_type;
    int32_t reserved;
    int64_t dims[4];
    int64_t offset;
    int64_t bytes;
} qdq_gguf_tensor;
int qdq_gguf_parse(const void *file, int64_t size, qdq_gguf_tensor *tensors, int max_tensors,
                   int *n_tensors, int64_t *data_offset, uint32_t *alignment);
int qdq_gguf_find_kv(const void *file, int64_t size, const char *key, uint32_t *value_type,
                     int64_t *value_offset);

/* ---------------------------------------------------------------------------
 * Device status: synchronises `stream`, returns the first device-side error
 * recorded since the last call (QDQ_OK if none) and clears it.
 * ------------------------------------------------------------------------- */
int qdq_get_device_status(qdq_stream_t stream);

/* Runs the library's bounded inter-CTA wait on a device flag that nothing sets,
 * with a limit of `timeout_ns` nanoseconds, so that a test can see a wait run
 * out without a hang: afterwards qdq_get_device_status() returns
 * QDQ_ERR_TIMEOUT. */
int qdq_selftest_wait_timeout(int64_t timeout_ns, qdq_stream_t stream);

/* Number of streaming multiprocessors the library sizes its grids by. */
int qdq_device_sm_count(void);

#ifdef __cplusplus
}
#endif
#endif /* QDQ_H */
