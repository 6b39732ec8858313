/*
 * libqgemv -- quantized-weight decode GEMV for NVIDIA GB300 (sm_103a), C ABI.
 *
 * The operation (vllm.cpp PR #1936 "raise Qwen3.5-4B Q4_K_M gfx1100 decode", the SGLang/vLLM study
 * section): for single-token decode, each activation row is quantized ONCE to q8_1-style int8 blocks,
 * then every output row streams its 4/6/8-bit super-blocks, dequantizes them in registers and reduces
 * the dot product:
 *
 *     y[i, n] = sum_k  w[n, k] * xhat[i, k]          i < m (1..16), n < N, k < K
 *
 * where w is the dequantized weight and xhat = d * q the dequantized activation.  The integer block dots
 * are exact; scales and the final reduction run in fp32.  The W8A16 entry (MetaInfer-cpp README, the
 * W8A16 section; zLLM article "Decode 只有一行", the W8/W8A16 direct-read section) multiplies int8
 * weights directly against 16-bit activations with fp32 accumulation, with no activation quantization.
 *
 * Block formats.  No page fixes a bit packing; these layouts are this library's own.  All multi-byte
 * fields are little-endian; fp16 is IEEE binary16; bf16 is the top half of an IEEE binary32.
 *
 *   q8_1 activation block (36 B per 32 values):
 *       [0..1]  d  fp16     scale; xhat = d * q
 *       [2..3]  s  fp16     binary16(float(d) * sum(q))   (informational; the GEMV never reads it)
 *       [4..35] qs int8[32] q[j] is value 32*b + j of the row
 *     A row of K values is K/32 consecutive blocks; row i starts at byte i * (K/32) * 36.
 *
 *   QGEMV_Q4_K super-block (144 B per 256 weights):
 *       [0..1]   d     fp16
 *       [2..3]   dmin  fp16
 *       [4..15]  a 96-bit little-endian bit string; field f (f = 0..15) is bits 6f..6f+5;
 *                fields 0..7 are sc[0..7], fields 8..15 are mn[0..7] (unsigned 6-bit)
 *       [16..143] qs[128]: byte 32g+t (g < 4, t < 32) holds code of element 64g+t in its low nibble and
 *                of element 64g+32+t in its high nibble
 *       w[e] = d * sc[e/32] * q[e] - dmin * mn[e/32]
 *
 *   QGEMV_Q6_K super-block (210 B per 256 weights):
 *       [0..127]   ql: byte 64h+t (h < 2, t < 64) holds the low 4 bits of element 128h+t (low nibble)
 *                  and of element 128h+64+t (high nibble)
 *       [128..191] qh: byte 32h+t (h < 2, t < 32) holds bits 4..5 of element 128h+32k+t in its bits
 *                  2k..2k+1 (k < 4)
 *       [192..207] sc int8[16]
 *       [208..209] d fp16
 *       w[e] = d * sc[e/16] * (q[e] - 32),  q[e] in 0..63
 *
 *   QGEMV_Q8_0 block (34 B per 32 weights):
 *       [0..1] d fp16, [2..33] qs int8[32];  w = d * q  (q may be -128..127)
 *
 *   QGEMV_Q5_K super-block (176 B per 256 weights; vllm.cpp PR #1936 decodes Q5_K in the same dp4a
 *   inner loops as Q4_K and Q6_K, the amd_mixed_dot section, and keeps its attention qkv tensors
 *   [2560 -> 8192] in Q5_K, the keep-quant section):
 *       [0..15]   d, dmin and the 96-bit sc/mn bit string, exactly as QGEMV_Q4_K
 *       [16..47]  qh[32]: bit j (j < 8) of byte t (t < 32) is bit 4 of element 32j+t
 *       [48..175] qs[128]: the low 4 bits of each element, packed as QGEMV_Q4_K's qs
 *       w[e] = d * sc[e/32] * q[e] - dmin * mn[e/32],  q[e] in 0..31
 *
 *   A weight matrix [N, K] is row-major: row n is K/256 (K-quants) or K/32 (Q8_0) consecutive blocks;
 *   rows are contiguous with no padding (row n starts at byte n * qgemv_weight_bytes(fmt, 1, K)).
 *
 * Common rules for every entry point:
 *   - All data pointers are caller-owned DEVICE memory.  The library never allocates, frees or keeps a
 *     pointer after the call returns.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls only enqueue work: they do
 *     not synchronize, and results are valid in stream order.
 *   - Argument errors are detected on the host before anything is enqueued; on any non-zero status
 *     nothing was launched and no output byte was written.
 *   - m (activation rows) is 1..16; larger m returns QGEMV_ERR_UNSUPPORTED (never a partial result).
 *     m = 1..8 run kernels built for that m.  m = 9..16 run one 16-row build (rows past m are staged
 *     as zeros and not stored), or, where K exceeds that build's activation staging, two launches of 8
 *     and m - 8 rows; each output row gets the same arithmetic either way.
 *   - K is at most qgemv_max_k (131072 at every m).  A launch stages the whole activation row in shared
 *     memory; rows longer than one pass of staging at the call's m (qgemv_chunk_k(fmt, m, K) < K) run as
 *     one launch per K-chunk: each launch reads only its chunk of every weight row (every weight byte is
 *     still read once), stages only its chunk of the activation, and every launch after the first adds
 *     its partial sums to y, in stream order (no atomics; the result does not depend on timing).  A
 *     row's summation order is then fixed by (fmt, K, m) rather than (fmt, K).
 *   - Outputs are fully overwritten (no accumulation into y).
 *   - Inputs must be finite; a NaN or Inf in x gives unspecified output (no trap, no fault).
 *   - Thread safety: calls may be made from several host threads on different streams.
 */
#ifndef QGEMV_H
#define QGEMV_H

#include <stddef.h>

#if defined(__GNUC__)
#define QGEMV_API __attribute__((visibility("default")))
#else
#define QGEMV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    QGEMV_Q4_K = 1,
    QGEMV_Q6_K = 2,
    QGEMV_Q8_0 = 3,
    QGEMV_W8A16 = 4, /* Q8_0 weights against bf16 activations (qgemv_multi only; see qgemv_w8a16) */
    QGEMV_Q5_K = 5,
    QGEMV_W8A16_CHANNEL = 6 /* per-channel INT8 weights against bf16 activations (qgemv_plan_info only) */
} qgemv_fmt;

/* Activation kinds for qgemv_multi. */
typedef enum {
    QGEMV_ACT_Q8_1 = 0, /* q8_1 blocks as written by qgemv_quantize_act                       */
    QGEMV_ACT_F32 = 1,  /* fp32 [m, K]: quantized inside the GEMV launch (same bits as the quantizer) */
    QGEMV_ACT_BF16 = 2, /* bf16 [m, K]: W8A16 (not quantized), or qgemv_quantize_act_typed input   */
    QGEMV_ACT_F16 = 3   /* IEEE binary16 [m, K]: qgemv_quantize_act_typed input                    */
} qgemv_act;

/*
 * Launch flags (the *_ex and qgemv_multi entry points).
 *
 * QGEMV_FLAG_PDL: launch with programmatic dependent launch (sm_90+ stream semantics).  The kernel may
 * start while the kernels before it in the stream are still running, and it starts streaming its first
 * weight tiles from that moment; it waits for those kernels before it reads the activation or writes any
 * output.  The caller guarantees that the weight buffers are not written by kernels still in flight when
 * the call is enqueued.  Under CUDA graphs this removes most of the gap between consecutive decode
 * kernels.
 *
 * QGEMV_FLAG_PDL_LATE_TRIGGER (the quantizer entry points only, with QGEMV_FLAG_PDL): the launch lets the
 * next kernel of the stream start only once its own wait for the kernels before it has ended, instead of
 * at once.  It is a scheduling hint and changes no result.  Measured: before a short GEMV (weights below
 * about 4 MB, the launches of the register-capped single-row build) the later start was faster, the
 * following short launches above all; before a long GEMV it was slower, because that GEMV's weights
 * start streaming later.
 */
#define QGEMV_FLAG_PDL 1u
#define QGEMV_FLAG_PDL_LATE_TRIGGER 2u

/* Up to this many matrices share one activation in one qgemv_multi launch. */
#define QGEMV_MAX_GROUP 8

/* One weight matrix of a qgemv_multi group: W in the group's format, y fp32 [m, N]. */
typedef struct {
    const void* W;
    float* y;
    int N;
} qgemv_mat;

typedef enum {
    QGEMV_OK = 0,
    QGEMV_ERR_INVALID_ARG = 1, /* null pointer, bad format, non-positive size, K not a block multiple */
    QGEMV_ERR_UNSUPPORTED = 2, /* valid but outside the library's limits (m > 16, K too large for m)  */
    QGEMV_ERR_MISALIGNED = 3,  /* a pointer violates its alignment rule                              */
    QGEMV_ERR_CUDA = 4,        /* the CUDA runtime reported an error (see qgemv_last_cuda_error)      */
    QGEMV_ERR_DEVICE = 5,      /* the current device is not a compute-capability 10.3 (GB300) part    */
    QGEMV_ERR_OVERLAP = 6      /* the output range overlaps an input range                            */
} qgemv_status;

/*
 * Activation quantizer: x fp32 [m, K] row-major  ->  xq, m * (K/32) q8_1 blocks (qgemv_act_bytes(m, K)).
 *
 * Per block of 32 values (vllm.cpp PR #1936, QuantizeQ8KK / warp-coop section: block amax, scale
 * amax/127, nearest integer, clamp to 127; SGLang/vLLM study section: q8_1 = 32 int8 + scale + sum):
 *     amax = max|x|;  d32 = amax / 127 (fp32 IEEE division);  d = binary16_rne(d32);
 *     q = clamp(roundf(x / d32), -127, 127)   (IEEE fp32 division, halfway cases away from zero;
 *                                              q = 0 everywhere when d32 == 0);
 *     s = binary16_rne(float(d) * sum(q))     (the fp32 product is exact).
 * Codes and both fp16 fields are bit-exact with that definition.
 *
 * x: 16-byte aligned, m*K floats.  xq: 16-byte aligned, qgemv_act_bytes(m, K) bytes, not overlapping x.
 * 1 <= m <= 16, K > 0, K % 32 == 0.
 */
QGEMV_API int qgemv_quantize_act(const float* x, int m, int K, void* xq, void* stream);

/*
 * Quantized GEMV: y[i, n] = sum_k w[n, k] * xhat[i, k]   (fp32 out, [m, N] row-major).
 *
 * W: 16-byte aligned, qgemv_weight_bytes(fmt, N, K) bytes in the `fmt` layout above.
 * xq: 16-byte aligned, m*(K/32) q8_1 blocks as written by qgemv_quantize_act (row i = activation row i).
 * y: 4-byte aligned, m*N floats, must not overlap W or xq.
 * 1 <= m <= 16, N >= 1, K % 256 == 0 for Q4_K/Q5_K/Q6_K, K % 32 == 0 for Q8_0, K <= qgemv_max_k(fmt, m).
 * Integer block dots are exact; per-block scaling and the reduction are fp32, so y matches the exact
 * value to fp32 rounding (relative L2 error well under 1e-5 on N(0,1) activations).
 * Each output row's result depends only on its own weight row and the activation: stacking two weight
 * matrices row-wise concatenates their outputs bit for bit.
 */
QGEMV_API int qgemv(int fmt, const void* W, const void* xq, float* y, int m, int N, int K, void* stream);

/*
 * W8A16: y[i, n] = sum_b d[n, b] * sum_{j<32} q[n, 32b+j] * x[i, 32b+j]   (fp32 accumulation)
 *
 * W: Q8_0 layout, 16-byte aligned.  x_bf16: bf16 [m, K] row-major, 16-byte aligned.  y: fp32 [m, N],
 * 4-byte aligned, not overlapping W or x.  1 <= m <= 16, K % 32 == 0, K <= qgemv_max_k_w8a16(m).
 */
QGEMV_API int qgemv_w8a16(const void* W, const void* x_bf16, float* y, int m, int N, int K, void* stream);

/*
 * The activation quantizer for 16-bit activation rows: x_kind QGEMV_ACT_BF16 or QGEMV_ACT_F16 (or
 * QGEMV_ACT_F32, the same as qgemv_quantize_act).  Every 16-bit value widens exactly to fp32, and the q8_1
 * definition above is then applied unchanged, so the blocks are bit-identical to qgemv_quantize_act on
 * the widened rows.  (vllm.cpp PR #1936 quantizes the engine's activations, which its engines keep in
 * 16-bit types, the SGLang/vLLM study section; the library's own addition.)
 * x: 16-byte aligned, m*K values of the given kind; other rules as qgemv_quantize_act.  flags: 0,
 * QGEMV_FLAG_PDL, or QGEMV_FLAG_PDL | QGEMV_FLAG_PDL_LATE_TRIGGER (any other bit: QGEMV_ERR_INVALID_ARG).
 */
QGEMV_API int qgemv_quantize_act_typed(int x_kind, const void* x, int m, int K, void* xq, unsigned flags,
                                       void* stream);

/*
 * Per-output-channel INT8 W8A16 (MetaInfer-cpp README, the Qwen3-14B TP4 W8A16 decode section: signed
 * INT8 weights, one fp32 scale per output channel, bf16 activations, fp32 accumulation):
 *     y[i, n] = scale[n] * sum_k Wq[n, k] * x[i, k]
 * The sum is accumulated in fp32 over the exact products and multiplied by scale[n] once.
 * Wq: int8 [N, K] row-major (any value -128..127; symmetric quantizers write -127..127), 16-byte aligned.
 * scale: fp32 [N], 4-byte aligned.  x_bf16: bf16 [m, K], 16-byte aligned.  y: fp32 [m, N], 4-byte aligned,
 * not overlapping the inputs.  1 <= m <= 16, K % 32 == 0, K <= qgemv_max_k_w8a16_channel(m).
 */
QGEMV_API int qgemv_w8a16_channel(const void* Wq, const float* scale, const void* x_bf16, float* y, int m, int N,
                                  int K, void* stream);
QGEMV_API int qgemv_w8a16_channel_ex(const void* Wq, const float* scale, const void* x_bf16, float* y, int m,
                                     int N, int K, unsigned flags, void* stream);
QGEMV_API int qgemv_max_k_w8a16_channel(int m);

/*
 * GEMV with a fused argmax (the lm_head of greedy decoding): y = W * xhat as qgemv computes it, but y is
 * not written; idx_out[i] receives the first n with the largest y[i, n], val_out[i] that y value (NaN
 * counts as larger than every number, as in torch.argmax: a row whose y holds NaN gives the first NaN's
 * n; y itself can only hold NaN when an input is not finite).  Each CTA
 * reduces its rows, and the last CTA to finish combines the CTAs' results, so one launch replaces the
 * GEMV and a separate argmax pass.  (MetaInfer-cpp README, the device-sampling section: an lm_head that
 * returns the argmax without writing the logits; vllm.cpp PR #1936, the split-argmax section: ties go to
 * the lower index, which makes the combine associative and the result independent of its order.)
 * fmt: QGEMV_Q4_K / QGEMV_Q5_K / QGEMV_Q6_K / QGEMV_Q8_0, q8_1 activations, m = 1 (other m return
 * QGEMV_ERR_UNSUPPORTED).
 * scratch: device memory of at least qgemv_argmax_scratch_bytes(m) bytes, 16-byte aligned, whose first
 * 4 bytes must be zero before the first call (e.g. cudaMemset once); each call leaves them zero again.
 * Calls that share one scratch buffer must be ordered (same stream, or synchronized): concurrent calls
 * on the same scratch race.  idx_out: int[m], val_out: float[m], 4-byte aligned, not overlapping the
 * inputs or the scratch.
 */
QGEMV_API size_t qgemv_argmax_scratch_bytes(int m);
QGEMV_API int qgemv_argmax(int fmt, const void* W, const void* xq, int m, int N, int K, void* scratch,
                           size_t scratch_bytes, int* idx_out, float* val_out, unsigned flags, void* stream);

/*
 * qgemv_argmax on a scratch the library owns, for callers that have no allocator at hand.  The pages have
 * no counterpart of this entry point; it adds no arithmetic of its own.
 * The scratch is a fixed array of QGEMV_ARGMAX_STATIC_SCRATCH_BYTES bytes in the library's static device
 * memory, one per device.  A call allocates nothing (no cudaMalloc, no allocating library call).
 * - Size limit: a call that would need more than QGEMV_ARGMAX_STATIC_SCRATCH_BYTES of scratch
 *   (qgemv_argmax_scratch_bytes(m) > the limit, i.e. m >= 2) returns QGEMV_ERR_UNSUPPORTED before touching
 *   the device; m outside 1..8 returns QGEMV_ERR_INVALID_ARG.
 * - Zero at start: the array's first 4 bytes (the CTAs' arrival counter) must be zero when a call starts.
 *   Static device memory is zero when the library's module is loaded on a device, and every call that runs
 *   to completion leaves the counter at zero again; the rest of the array needs no initial value.
 * - Setup: the first call on each device looks up the array's device address (cudaGetSymbolAddress) and
 *   does qgemv_argmax's own first-call setup.  That first call must happen before any stream capture.
 * - Races: every call on a device shares the one array.  Calls must be ordered (one stream, or
 *   synchronized); calls that overlap in time, on different streams or from different threads, race on
 *   the counter and the partial results, and their outputs are undefined.
 * Otherwise the arguments, validation and results are those of qgemv_argmax.
 */
#define QGEMV_ARGMAX_STATIC_SCRATCH_BYTES 16384
QGEMV_API int qgemv_argmax_noalloc(int fmt, const void* W, const void* xq, int m, int N, int K, int* idx_out,
                                   float* val_out, unsigned flags, void* stream);

/* As qgemv_quantize_act / qgemv / qgemv_w8a16, with launch flags (QGEMV_FLAG_PDL or 0; the quantizer also
 * takes QGEMV_FLAG_PDL_LATE_TRIGGER, which the GEMV entry points reject with QGEMV_ERR_INVALID_ARG). */
QGEMV_API int qgemv_quantize_act_ex(const float* x, int m, int K, void* xq, unsigned flags, void* stream);
QGEMV_API int qgemv_ex(int fmt, const void* W, const void* xq, float* y, int m, int N, int K, unsigned flags,
                       void* stream);
QGEMV_API int qgemv_w8a16_ex(const void* W, const void* x_bf16, float* y, int m, int N, int K, unsigned flags,
                             void* stream);

/*
 * Several matrices that read the same activation, in one launch: y_j = W_j xhat for j < count
 * (e.g. the q/k/v or gate/up projections of a layer, as vllm.cpp PR #1936's merged gate+up section does
 * by stacking rows; here the matrices stay separate buffers).  Every output equals what the
 * single-matrix call returns, bit for bit (each row's result depends only on its own weights and the
 * activation).
 *
 * fmt: QGEMV_Q4_K / QGEMV_Q5_K / QGEMV_Q6_K / QGEMV_Q8_0 with act_kind QGEMV_ACT_Q8_1 or QGEMV_ACT_F32, or
 *      QGEMV_W8A16 with act_kind QGEMV_ACT_BF16.
 * act: the shared activation (16-byte aligned): q8_1 blocks, fp32 [m, K] or bf16 [m, K].
 *      With QGEMV_ACT_F32 the launch quantizes the rows itself (the quantizer folded into the GEMV, so
 *      one fewer launch per input); the codes are bit-identical to qgemv_quantize_act's.
 * xq_out: QGEMV_ACT_F32 only; if not NULL the launch also writes the q8_1 blocks there (16-byte aligned,
 *      qgemv_act_bytes(m, K) bytes) for later calls on the same input.  Must be NULL otherwise.
 * 1 <= count <= QGEMV_MAX_GROUP; every W_j 16-byte aligned in `fmt`; every y_j 4-byte aligned; no output
 * overlaps another output or any input.  Same limits on m and K as qgemv.
 */
QGEMV_API int qgemv_multi(int fmt, int count, const qgemv_mat* mats, int act_kind, const void* act, void* xq_out,
                          int m, int K, unsigned flags, void* stream);

/* Sizes in bytes; 0 for an invalid (fmt, N, K) or (m, K). */
QGEMV_API size_t qgemv_weight_bytes(int fmt, int N, int K);
QGEMV_API size_t qgemv_act_bytes(int m, int K);

/* Largest K the library serves at a given m (131072; rows beyond one pass of activation staging run as
 * K-chunks); 0 for an invalid argument. */
QGEMV_API int qgemv_max_k(int fmt, int m);
QGEMV_API int qgemv_max_k_w8a16(int m);

/*
 * Values per K-chunk of a call at (fmt, m, K): K itself when the rows take one pass of activation staging,
 * else the chunk width (a multiple of 256; every chunk that wide but the last).  fmt may also be
 * QGEMV_W8A16 or QGEMV_W8A16_CHANNEL.  0 for an invalid argument or K beyond qgemv_max_k.  The fused
 * argmax needs one pass (qgemv_chunk_k(fmt, 1, K) == K).  No device needed.
 */
QGEMV_API int qgemv_chunk_k(int fmt, int m, int K);

/* Human-readable status name (static string; never NULL). */
QGEMV_API const char* qgemv_status_string(int status);

/* The cudaError_t value behind the most recent QGEMV_ERR_CUDA on the calling thread (0 if none). */
QGEMV_API int qgemv_last_cuda_error(void);

/*
 * Route counters: how many times each kernel variant was launched by this process (a witness of which
 * path ran).  Fills out[0 .. min(n, QGEMV_NUM_ROUTES)-1] and returns QGEMV_NUM_ROUTES.
 * Route ids: 0 quantizer, 1..8 Q4_K at m=1..8, 9..16 Q6_K, 17..24 Q8_0, 25..32 W8A16, 36..43 Q5_K,
 * 44..51 per-channel INT8 W8A16 (one count per GEMV launch at m <= 8); 53 launches of the 16-row build
 * (m = 9..16, any format); 52 launches with the fused argmax; 33 launches that quantized fp32
 * activations in-kernel, 34 launches over >= 2 matrices, 35 launches with programmatic dependent launch
 * (quantizer included), 54 launches that covered one K-chunk of long rows; 55 rotary positions, 56 and 57
 * attention (which kernel ran), 58 sampling, 59 and 60 writes into and reads of a packed cache, 61 attention by the packed cache's own
 * kernel (over an unpacked copy it counts as 56 or 57).
 */
#define QGEMV_ROUTE_FUSED 33
#define QGEMV_ROUTE_GROUPED 34
#define QGEMV_ROUTE_PDL 35
#define QGEMV_ROUTE_Q5_K_M1 36
#define QGEMV_ROUTE_W8A16_CHANNEL_M1 44
#define QGEMV_ROUTE_ARGMAX 52
#define QGEMV_ROUTE_M16 53 /* a launch of the 16-row build (m = 9..16), any format */
#define QGEMV_ROUTE_CHUNKED 54 /* a launch that covered one K-chunk of the rows (also counted by format) */
#define QGEMV_ROUTE_ROPE 55        /* qgemv_rope launches */
#define QGEMV_ROUTE_ATTN_ROWS 56   /* qgemv_attn launches of the 16-row kernel (decode, drafts) */
#define QGEMV_ROUTE_ATTN_TILES 57  /* qgemv_attn launches of the 128-row tensor-memory kernel (chunks, prompts) */
#define QGEMV_ROUTE_SAMPLE 58      /* qgemv_sample launches */
#define QGEMV_ROUTE_CACHE_WRITE 59 /* qgemv_cache_write launches */
#define QGEMV_ROUTE_CACHE_READ 60  /* qgemv_cache_read launches */
#define QGEMV_ROUTE_ATTN_PACKED 61 /* qgemv_attn launches of the packed cache's own kernel */
#define QGEMV_NUM_ROUTES 62
QGEMV_API int qgemv_route_counts(unsigned long long* out, int n);
QGEMV_API void qgemv_route_reset(void);

/*
 * Launch-plan introspection (no device needed): the plan the GEMV would use for (fmt, m, N, K) on a part
 * with `num_sms` SMs and `ctas_per_sm` resident CTAs.  fmt = QGEMV_W8A16 (4) asks for the W8A16 kernel,
 * QGEMV_W8A16_CHANNEL (6) for the per-channel INT8 kernel.  Fills
 * out[0..12] = {lanes per row team, rows per tile, tiles, ring stages, bytes per ring slot, dynamic shared
 * memory bytes, grid, bytes per weight row, work units per row, activation staging bytes, threads per
 * CTA, warps per row team, multi-warp reduction bytes, kernel build (m for the m-row kernel, 0 for the
 * single-row streaming build)} (out must hold 14 values).  For K beyond one pass of staging, the plan of
 * the call's first K-chunk launch.
 */
QGEMV_API int qgemv_plan_info(int fmt, int m, int N, int K, int num_sms, int ctas_per_sm, long long* out);

/*
 * The plan of one K-chunk launch covering Kc values of each of N rows (rows longer than one pass of
 * staging run as such launches; qgemv_chunk_k gives the chunk width, the last chunk may be narrower).
 * Fills out[0..14]: qgemv_plan_info's 14 values (row bytes are the chunk's), then the bytes from one row to
 * the next in a ring slot (each row's chunk arrives as its own copy).  Kc beyond one chunk launch's
 * staging returns QGEMV_ERR_UNSUPPORTED.  No device needed.
 */
QGEMV_API int qgemv_plan_info_chunk(int fmt, int m, int N, int Kc, int num_sms, int ctas_per_sm, long long* out);

/*
 * Tuning hook for sweeps: forces the resident CTAs per SM that the grid is sized for (1..4), log2 lanes
 * per row team (2..5), rows per tile, ring stages (2..8) and the single-row kernel build (1 = the
 * register-capped build for short launches, 2 = the streaming build) for every later GEMV launch in the
 * process; a value outside its range (e.g. 0 or -1) leaves that choice to the planner.  Not for
 * production use: forced plans are only checked for shared-memory fit.
 */
/* Tuning hook: row pairs (two rows per row team, for the builds that have them) 0 = planner decides,
 * 1 = whenever they fit, 2 = never.  Rows are bit-identical either way. */
QGEMV_API void qgemv_tune_pairs(int mode);

/* Tuning hook: qgemv_attn's kernel, 0 = planner decides, 1 = the 16-row kernel (over a packed cache its own kernel), 2 = the 128-row
 * kernel (heads of up to 128; over a packed cache with the copy before it).  It also decides what qgemv_attn_scratch_bytes and
 * qgemv_attn_scratch_bytes_ex say. */
QGEMV_API void qgemv_tune_attn(int kernel);

QGEMV_API void qgemv_tune_override(int ctas_per_sm, int lanes_log2, int rows_per_tile, int stages,
                                   int kernel_build);

/*
 * Failure injection for callers' error paths (host side only): the next `count` entry-point calls on
 * any thread return `status` without launching anything.  count = 0 disarms it.
 */
QGEMV_API void qgemv_debug_fail_next(int status, int count);

/*
 * Device-side error word.  Kernels never trap: a bounded on-chip wait that gives up (it cannot in a
 * correct run) sets a bit here and the kernel returns.  Reads (and with reset != 0 clears) the word for
 * the current device; this call synchronizes the device.  Returns a status.
 */
QGEMV_API int qgemv_device_error(unsigned int* out, int reset);

/*
 * Launch timeline (diagnostics).  A traced build of the library (libqgemv_trace.so, compiled with
 * QGEMV_TRACE) stamps %globaltimer at fixed points of every CTA of the first `launches` kernel launches
 * after qgemv_trace_begin, into a buffer in its static device memory; the normal build does no tracing
 * and these calls return QGEMV_ERR_UNSUPPORTED.  Launch numbers are assigned when a launch is enqueued
 * (under stream capture: when it is captured, so a replayed graph rewrites the same records).
 *   qgemv_trace_info:  the buffer's shape: launches x ctas records of `fields` unsigned 64-bit values.
 *   qgemv_trace_begin: zero the buffer and restart the numbering at 0 (synchronizes the device).
 *   qgemv_trace_read:  copy the first `bytes` of the buffer to host memory; *launches receives how many
 *                      launches have been numbered since qgemv_trace_begin (capped at the buffer's size).
 * Record of (launch, CTA): 0 kernel entry, 1 dependency released, 2 activation staged, 3 CTA done,
 * 4 producer issued its last tile, 5 producer's copies all landed, 6 SM id, 7 kind (1 GEMV, 2 quantizer),
 * 8..13 the first three tiles' (full-slot wait done, decode done) times of consumer warp 0; times in ns,
 * unused fields 0.  Timing only: a traced launch computes exactly what an untraced one does.
 */
QGEMV_API int qgemv_trace_info(int* launches, int* ctas, int* fields);
QGEMV_API int qgemv_trace_begin(void);
QGEMV_API int qgemv_trace_read(unsigned long long* host, size_t bytes, int* launches);

/*
 * ---------------------------------------------------------------------------------------------------
 * The operators between the GEMVs of a serving step: rotary positions with the write into a paged cache,
 * attention of new tokens over that cache, and sampling from the lm_head's logits.  They follow the common
 * rules above (caller-owned device memory, host-side checks before anything is enqueued, results in stream
 * order, QGEMV_FLAG_PDL) and serve any number of tokens, not only 1..16.  They serve inference: no gradients.
 * Strides go up to 2^40 elements; a tensor, cache or page table that spans more than 9e15 elements is refused as unsupported.
 */

/*
 * A paged key/value cache.  Token `o` of page `p`, key/value head `h`, is the `dim` consecutive 16-bit values at
 * element offset p * k_page + o * k_token + h * k_head of `k` (and likewise of `v`), so both [page, token, head,
 * dim] and [page, head, token, dim] orders, and caches inside a larger allocation, are described by strides.
 * kind: QGEMV_ACT_BF16 or QGEMV_ACT_F16.  k, v: 16-byte aligned; strides non-negative multiples of 8 elements.
 * num_pages, page_size, heads >= 1; dim a multiple of 8, 8..256.  Slot s of the cache is token s % page_size of page
 * s / page_size.
 */
typedef struct {
    void* k;
    void* v;
    long long k_page, k_token, k_head; /* strides, elements */
    long long v_page, v_token, v_head;
    int kind;
    int num_pages, page_size, heads, dim;
} qgemv_cache;

/*
 * Packed caches: `kind` QGEMV_CACHE_Q4 or QGEMV_CACHE_Q8.  A row (one token, one key/value head) is `dim` codes c of 4 or 8 bits, and for
 * every block of 32 of them a step d >= 0 and a base m in fp16; a value stands as d * c + m:
 *     [0 .. dim*bits/8)   codes: Q8 byte e is element e's; Q4 byte j is element 2j's in its low half, element 2j+1's in its high half
 *     then dim/32 fp16    d of the blocks in their order
 *     then dim/32 fp16    m of the blocks in their order
 * qgemv_cache_row_bytes bytes, which is that rounded up to a multiple of 16 (the rest is not used): 80 and 144 for heads of 128.
 * The strides of such a cache are in BYTES, positive multiples of 16 below 2^31 for tokens and heads and at most 2^39 for pages (a
 * stride over a dimension of one element is not looked at); dim is a multiple of 32, 32..256; everything else is as above.
 * A block of values x, each clamped to +-65504 first, is written as follows, with L = 15 or 255, every operation rounded to fp32:
 *     m = the largest fp16 <= min x;   d = the smallest fp16 >= (max x - m) / L;   r = 1 / d;
 *     c = min(L, rint((x - m) * r))   (ties to even; 0 where d = 0)
 * so a value is off by at most d/2 (1 + 2^-12).  A block with a NaN is written as m = NaN, d = 0.  (A block that reaches up to 65504 may
 * stand for more than that by 2^-10 of its range, which may be +inf where it is read back to fp16.)
 */
#define QGEMV_CACHE_Q4 4
#define QGEMV_CACHE_Q8 8
/* Bytes of a row of a packed cache, 0 for an invalid kind or dim. */
QGEMV_API size_t qgemv_cache_row_bytes(int kind, int dim);

/* Pairing of the rotated elements of a head. */
typedef enum {
    QGEMV_ROPE_HALF = 0,       /* element i with element i + rot_dim/2 */
    QGEMV_ROPE_INTERLEAVED = 1 /* element 2i with element 2i + 1       */
} qgemv_rope_layout;

/* Scaling of the rotary frequencies for contexts longer than the trained one (qgemv_rope_freqs). */
typedef enum {
    QGEMV_ROPE_SCALE_NONE = 0,
    QGEMV_ROPE_SCALE_LINEAR = 1, /* every frequency divided by `factor` */
    QGEMV_ROPE_SCALE_BASE = 2,   /* theta multiplied by factor^(rot_dim / (rot_dim - 2)): the slowest pair is slowed by
                                    `factor`, the fastest keeps its frequency                                           */
    QGEMV_ROPE_SCALE_PARTS = 3,  /* pairs that turn fewer than `low` times over `trained` positions are divided by
                                    `factor`, those that turn more than `high` times are kept, a ramp linear in the pair
                                    index lies between; *mscale = 0.1 ln(factor) + 1                                     */
    QGEMV_ROPE_SCALE_BANDS = 4   /* wavelengths above trained/low divided by `factor`, below trained/high kept, between
                                    them a ramp linear in trained/wavelength                                             */
} qgemv_rope_scaling;

/*
 * Rotary frequencies, host arithmetic in 64 bits: out[i], i < rot_dim/2, is the turn of pair i per position in units of
 * 2^-64 of a turn, round(f_i / (2 pi) * 2^64) with f_i = theta^(-2i/rot_dim), scaled as asked.  The caller copies the
 * rot_dim/2 values to the device once.  The angle of position p is then 2 pi * frac(p * out[i] / 2^64): the product
 * wraps in 64-bit integer arithmetic, so whole turns fall away exactly and a position of a million is as exact as
 * position 1.  *mscale (may be NULL) receives the factor of the rotated values that the scaling asks for (1 unless
 * QGEMV_ROPE_SCALE_PARTS).  out is HOST memory.
 * rot_dim even, 2..256; theta > 1; factor >= 1 except for NONE; trained >= 1 and 0 < low < high for PARTS and BANDS.
 */
QGEMV_API int qgemv_rope_freqs(int rot_dim, double theta, int scaling, double factor, double trained, double low,
                               double high, unsigned long long* out, float* mscale);

/*
 * Rotary positions of new tokens' queries and keys, with the write of keys and values into a paged cache:
 *     (a, b) -> (mscale (a cos t - b sin t), mscale (b cos t + a sin t)),  t = angle of the token's position and the pair
 * for the first rot_dim elements of every query and key head; the other elements, and the values, are copied.  The
 * arithmetic is fp32 and each result is rounded once to the type it is stored in.
 *
 * q [tokens, heads, dim], k and v [tokens, kv_heads, dim], of kind x_kind (QGEMV_ACT_F32: a GEMV's output, e.g. three
 * slices of one qkv row; QGEMV_ACT_BF16; QGEMV_ACT_F16), the last dimension contiguous, token and head strides in elements.
 * q_out [tokens, heads, dim] and k_out [tokens, kv_heads, dim]: QGEMV_ACT_BF16 / QGEMV_ACT_F16 / QGEMV_ACT_F32 by
 * out_kind.  cache (may be NULL): rotated keys and the values go to slot slots[t] of it (rounded once to the cache's kind, or packed
 * as above from the fp32 results); a
 * negative slot writes nothing (a padding token).  A slot beyond the cache writes nothing and sets
 * QGEMV_DEVERR_BAD_INDEX in the device error word.  Slots that are >= 0 must differ: two tokens with one slot leave
 * unspecified values there.
 * q with q_out, or k with k_out and / or a cache, may be left out (NULL, and heads or kv_heads 0); v goes with the cache.
 * q_out may be q itself and k_out k itself (same kind and strides); other overlaps of an output with an input, or of
 * outputs, are refused.  positions: int[tokens] (any 32-bit value; negative positions turn backwards).
 * freqs: device copy of qgemv_rope_freqs' output, 8-byte aligned.  rot_dim even, 2..dim; dim a multiple of 8, 8..256.
 * Pointers 16-byte aligned; strides multiples of 16 bytes (of 8 elements for fp32).  tokens = 0 is valid and does nothing (the
 * tensors' addresses may then be NULL, here and below).
 */
typedef struct {
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    void* k_out;
    long long q_token, q_head, k_token, k_head, v_token, v_head; /* strides, elements */
    long long q_out_token, q_out_head, k_out_token, k_out_head;
    const int* positions;
    const unsigned long long* freqs;
    const qgemv_cache* cache;
    const long long* slots;
    int x_kind, out_kind;
    int tokens, heads, kv_heads, dim, rot_dim;
    int layout; /* qgemv_rope_layout */
    float mscale;
} qgemv_rope_args;

QGEMV_API int qgemv_rope(const qgemv_rope_args* args, unsigned flags, void* stream);

/*
 * Writes new tokens' keys and values into a packed cache as they are (qgemv_rope does it with their rotary positions):
 * k, v [tokens, cache->heads, cache->dim] of kind x_kind (QGEMV_ACT_F32 / BF16 / F16), last dimension contiguous, 16-byte aligned,
 * strides multiples of 8 elements and 16 bytes.  Token t goes to slot slots[t]; a negative slot writes nothing, one beyond the cache writes
 * nothing and sets QGEMV_DEVERR_BAD_INDEX in the device error word.  Slots that are >= 0 must differ.  tokens = 0 does nothing.
 */
typedef struct {
    const void* k;
    const void* v;
    long long k_token, k_head, v_token, v_head; /* strides, elements */
    const qgemv_cache* cache;
    const long long* slots;
    int x_kind, tokens;
} qgemv_cache_write_args;

QGEMV_API int qgemv_cache_write(const qgemv_cache_write_args* args, unsigned flags, void* stream);

/*
 * Reads keys and values back from a packed cache.  Sequence b (b < seqs) has the rows out_start[b] .. out_start[b+1] - 1 of
 * k_out and v_out [tokens, cache->heads, cache->dim] (either may be NULL): row out_start[b] + j receives its context token first[b] + j
 * (first NULL: token j), which is token t % page_size of page pages[b * pages_stride + t / page_size], as in qgemv_attn.  The value
 * d * c + m is computed in fp32 with one rounding (d * c is exact) and rounded to out_kind (QGEMV_ACT_F32 / BF16 / F16).
 * Rows outside every sequence are left as they are.  A token before 0, at max_kv or beyond it, beyond the row of the page
 * table (pages_stride * page_size), or on a page outside the cache, is read as zeros and sets QGEMV_DEVERR_BAD_INDEX.  out_start ascends; values outside 0..tokens are held to it.
 * Outputs: last dimension contiguous, 16-byte aligned, strides multiples of 8 elements and 16 bytes, apart from each other and the inputs.
 * tokens = 0 or seqs = 0 does nothing.
 */
typedef struct {
    const qgemv_cache* cache;
    const int* pages;
    long long pages_stride;
    const int* out_start; /* [seqs + 1] */
    const int* first;     /* [seqs] or NULL */
    void* k_out;
    void* v_out;
    long long k_token, k_head, v_token, v_head; /* strides, elements */
    int out_kind, tokens, seqs;
    int max_kv; /* context tokens that may be read */
} qgemv_cache_read_args;

QGEMV_API int qgemv_cache_read(const qgemv_cache_read_args* args, unsigned flags, void* stream);

/*
 * Attention of new tokens over a paged cache.  Sequence b (b < seqs) has the new tokens q_start[b] .. q_start[b+1] - 1 of
 * q (n_b of them, 0 allowed) and a context of kv_len[b] tokens in the cache, the new ones included: context token t is
 * token t % page_size of page pages[b * pages_stride + t / page_size].  New token j sits at position
 * kv_len[b] - n_b + j.  With query head h reading key/value head h / (heads / cache->heads):
 *     s_t = scale * <q, k_t>,  out = sum_t softmax(s)_t v_t,  lse = ln sum_t exp(s_t)
 * over the context tokens t that the new token sees: all of them, or with causal != 0 those up to its own position, and
 * with window > 0 only the `window` tokens that end at its position.  A token that sees nothing (a context of length 0, or
 * a position below 0) gets out = 0 and lse = -inf.  A query with a NaN gives NaN, in its own row only.
 * Scores, softmax statistics and sums are fp32; the probabilities meet the values in the 16-bit type of q (each rounded
 * once, unnormalised, their sum taken before the rounding; with f16, those below 2^-29 of the row's largest, or 2^-21 in the 128-row
 * kernel, have fewer bits, and none below 2^-40 or 2^-32); out is rounded once.
 *
 * Over a packed cache (QGEMV_CACHE_Q4 / QGEMV_CACHE_Q8) k_t and v_t are the values d * c + m, and q and out are of either type.  Few rows a
 * sequence read the codes themselves.  q then counts in f16 times a power of two of its own row: 11 bits (bf16: all 8) for elements down to 2^-19 of
 * the row's largest, an error of 2^-30 of that below.  The probabilities p keep 11 bits, and so do their products p d with the values' steps;
 * with f16 results p d is rounded from about 20 bits of p, and codes count from the middle one, Z = 8 or 128, so that of v = (m + Z d) + d (c - Z) either part's
 * sum is off by 2^-11 of what it adds up.  The sums of codes lose at most 17 2^-13 of the largest p d of 16 keys beside that.  Probabilities below 2^-24 of the row's largest have fewer bits.  Many rows read a copy of the contexts in f16 (11 bits, held to +-65504), which the call makes in
 * the scratch, and the probabilities are rounded as f16's above.
 * kind (QGEMV_ACT_BF16 / QGEMV_ACT_F16): type of q and out, and the cache's unless that is packed.  q, out [tokens, heads, cache->dim], last
 * dimension contiguous, 16-byte aligned, strides multiples of 8 elements.  lse: fp32 [tokens, heads] or NULL.
 * max_q, max_kv (at most 2^30): bounds of n_b and kv_len[b] over the batch, for the choice of kernel and its launch; the
 * values on the device must keep to them: tokens beyond max_q are left unwritten, context beyond max_kv or beyond the
 * row of the page table (pages_stride * page_size) is not read.  A page number outside the cache reads as if its tokens
 * were masked and sets QGEMV_DEVERR_BAD_INDEX in the device error word.
 * What lies in the cache beyond kv_len, or before the window of a sequence's first new token, is never used, whatever its bits, and the
 * pages that lie there wholly are not looked up (their entries may be anything).  Keys and values that some token of the call sees must
 * be finite, as must the steps and bases of a packed cache there.
 * scratch: at least qgemv_attn_scratch_bytes(...) bytes (over a packed cache qgemv_attn_scratch_least(...); with
 * qgemv_attn_scratch_bytes_ex(...) many rows are faster, see there), 16-byte aligned, whose first QGEMV_ATTN_SCRATCH_HEAD bytes must be
 * zero before the first call (e.g. cudaMemset once); each call leaves them zero again, so calls of any sizes may share one
 * scratch that is large enough for each: that of the largest sizes is (see below).  Calls that share a scratch must be ordered.
 * The result does not depend on timing: parts of a long context are joined in a fixed order.
 * heads a multiple of cache->heads; 0 < scale <= 1e30.  tokens = 0 or seqs = 0 does nothing.
 */
typedef struct {
    const void* q;
    void* out;
    float* lse;
    long long q_token, q_head, out_token, out_head; /* strides, elements */
    const qgemv_cache* cache;
    const int* pages;
    long long pages_stride;
    const int* q_start; /* [seqs + 1] */
    const int* kv_len;  /* [seqs] */
    void* scratch;
    size_t scratch_bytes;
    int kind;
    int tokens, heads, seqs;
    int max_q, max_kv;
    float scale;
    int causal, window;
} qgemv_attn_args;

QGEMV_API int qgemv_attn(const qgemv_attn_args* args, unsigned flags, void* stream);
/* Scratch that serves every call of these sizes or smaller seqs, tokens, max_q and max_kv, with these heads and any window (0 for invalid
 * sizes).  It never falls as a size grows.  No device needed. */
#define QGEMV_ATTN_SCRATCH_HEAD 65536
QGEMV_API size_t qgemv_attn_scratch_bytes(int seqs, int tokens, int heads, int kv_heads, int dim, int max_q, int max_kv);
/* The same for a cache of the given kind.  Over a packed one, calls that are served better by the 128-row kernel (many new tokens) read a copy of
 * their contexts in f16, which is made in the scratch: seqs * (max_kv + 128) tokens of kv_heads * dim * 4 + 4 bytes and tokens * heads rows of
 * dim * 2 + 4 (the sequences' bounds, whatever their lengths, windows and shared pages).  Of that the size counts at most QGEMV_ATTN_COPY_MAX bytes; a
 * scratch that is larger by what a copy takes beyond that is used for it too.  One scratch serves the calls of all layers, one after another.
 * A call whose copy the given scratch has no room for is served by the packed cache's own kernel, which needs none: its results differ within
 * their stated bits, and it is slower for many rows (32 and 8 heads of 128, 2000 new tokens over 24000: 3.2 ms for 0.6 to 0.7). */
#define QGEMV_ATTN_COPY_MAX 4294967296ull
QGEMV_API size_t qgemv_attn_scratch_bytes_ex(int cache_kind, int seqs, int tokens, int heads, int kv_heads, int dim, int max_q, int max_kv);
/* The scratch with which no call of these sizes or smaller ones is refused; less than that of qgemv_attn_scratch_bytes_ex over a packed cache,
 * the same over a 16-bit one. */
QGEMV_API size_t qgemv_attn_scratch_least(int cache_kind, int seqs, int tokens, int heads, int kv_heads, int dim, int max_q, int max_kv);

/* Launch-plan introspection (no device needed), as qgemv_plan_info: fills out[0..3] for a qgemv_attn call of these sizes, with kind the type of q, whose
 * scratch has room for whatever it would use: {the kernel, as its QGEMV_ROUTE_ATTN_ number; key/value heads that a block takes side by
 * side; rows of a row tile; bytes of scratch that this needs}. */
QGEMV_API int qgemv_attn_plan_info(int cache_kind, int kind, int seqs, int tokens, int heads, int kv_heads, int dim, int max_q, int max_kv, int window,
                                   long long* out);

/*
 * Sampling: one token per row of logits [m, N] (kind QGEMV_ACT_F32 / BF16 / F16, rows `row_stride` elements apart), from
 * one given uniform number u[i] in [0, 1) per row.  With top = max_n x_n and T = temperature[i]:
 *     e_n = exp((x_n - top) * (1 / T)),  w_n = floor(2^42 e_n)
 * (fp32 up to e_n; the w_n are whole numbers, so their sums are exact and do not depend on any order).  Tokens are ranked by
 * x_n, ties by the lower index.  A token is kept if its rank is below top_k[i], the w before it in that order sum to less
 * than top_p[i] times the sum of those that top_k keeps (the products in fp64), and e_n >= min_p[i]; rank 0 is always kept.  With W the sum
 * of the kept w, the token is the first n, in index order, whose running sum of kept w exceeds floor(u[i] * W).
 * token_out[i]: that n; prob_out[i] (may be NULL): e_n * 2^42 / W.
 * temperature <= 0 is greedy (rank 0, prob 1).  top_k <= 0, top_p >= 1 and min_p <= 0 filter nothing; NULL for any of the
 * four means: temperature 1, no filter.
 * -inf logits are never taken; a row of nothing but -inf gives token -1 and prob 0.  A row with a NaN gives the first NaN's
 * index, else a row with +inf the first +inf's, with prob NaN: the caller's model has failed there.
 * logits: 16-byte aligned; row_stride >= N (any, but rows that all start 16-byte aligned are read faster).
 * 1 <= N <= 2^20; m >= 0 (0 does nothing).  token_out, prob_out must not overlap the inputs or each other.
 */
QGEMV_API int qgemv_sample(int kind, const void* logits, long long row_stride, int m, int N, const float* temperature,
                           const int* top_k, const float* top_p, const float* min_p, const float* u, int* token_out,
                           float* prob_out, unsigned flags, void* stream);

/* Bit of the device error word: an index in device memory (cache slot, page number) was outside its range and skipped. */
#define QGEMV_DEVERR_BAD_INDEX 4u

#ifdef __cplusplus
}
#endif

#endif /* QGEMV_H */
