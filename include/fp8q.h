/*
 * fp8q.h -- C ABI of the B200 (sm_100a) FP8 W8A8 linear layer library, libfp8q.so.
 *
 * The layer is the one Llama-3.x "FP8-Dynamic" and "FP8-Block" checkpoints use:
 *
 *   - Weights are E4M3 codes with one scale per output channel, taken from a
 *     minmax observer ("Llama-3.1-8B-Instruct-FP8-Dynamic" explainer, FP8 动态量化
 *     table, weights row; "Llama-3.1-70B-FP8-Dynamic" explainer, section 1.2), or
 *     one scale per 128 x 128 block ("Llama-3.2-3B-Instruct-FP8-Block" explainer,
 *     quantization_config table, block_structure [128, 128]).
 *   - Activations are quantized at run time, one dynamic scale per token (the
 *     FP8-Dynamic table's input_activations row; 70B explainer FAQ Q2), or one
 *     per group of 128 input features (FP8-Block table, input activations row).
 *   - E4M3 has 4 exponent and 3 mantissa bits and tops out at 448 ("Llama 3 精读实录",
 *     section 2.1).  Codes are the E4M3FN bit patterns (no infinities; 0x7F and
 *     0xFF are NaN and never produced for finite input).
 *   - lm_head stays in high precision: it is not passed to this library (same
 *     tables, ignore row).
 *
 * Arithmetic, identical on every path:
 *   amax  = max |x| over the unit (row, 128-group or 128x128 block), exact in fp32
 *   scale = amax / 448 as one IEEE fp32 division; 1.0 when amax == 0
 *   code  = E4M3(x / scale): IEEE fp32 quotient, then round to nearest even,
 *           saturating to +-448, sign kept (-0 is 0x80)
 *   Y[m,n] = bf16_rne( acc[m,n] * x_scale[m] * w_scale[n] ),
 *           acc = fp32 sum over k of E4M3(xq[m,k]) * E4M3(wq[n,k]) (channel mode)
 *   Y[m,n] = bf16_rne( sum_kb  x_scale[m,kb] * w_scale[n/128,kb] * acc_kb[m,n] )
 *           with acc_kb the fp32 sum over the 128-wide K slice kb (block mode)
 *
 * Conventions for every entry point:
 *   - All data pointers are DEVICE pointers owned by the caller.  The library
 *     never allocates, frees or synchronizes; work is enqueued on `stream`
 *     (a cudaStream_t passed as void*; NULL is the legacy default stream).
 *   - Matrices are row-major; ld* arguments are row strides in ELEMENTS.
 *   - Arguments are checked before anything is launched.  A bad argument
 *     returns an error status and launches nothing.  A launch failure returns
 *     FP8Q_ERR_CUDA.  Errors that happen later on the device surface at the
 *     caller's next synchronization; a kernel whose internal wait runs out
 *     (about 4 s, which only a broken machine reaches) sets a device-side
 *     error word that fp8q_device_error() reads.
 *   - The calls are thread-safe; they keep no state between calls other than
 *     the device error word and a cached device-attribute table.
 */
#ifndef FP8Q_H_
#define FP8Q_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FP8Q_API __attribute__((visibility("default")))
#else
#define FP8Q_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP8Q_OK = 0,
    FP8Q_ERR_INVALID_ARG = 1,     /* null pointer, negative size, bad mode, ...        */
    FP8Q_ERR_UNSUPPORTED = 2,     /* valid but outside what the kernels cover          */
    FP8Q_ERR_MISALIGNED = 3,      /* pointer or stride breaks a 16-byte requirement     */
    FP8Q_ERR_CUDA = 4,            /* a CUDA runtime/driver call failed                  */
    FP8Q_ERR_DEVICE_TIMEOUT = 5   /* a kernel gave up waiting (see fp8q_device_error)   */
} fp8q_status;

typedef enum {
    FP8Q_CHANNEL_TOKEN = 0,       /* W: one scale per output channel; X: one per token  */
    FP8Q_BLOCK128 = 1,            /* W: one per 128x128 block;  X: one per 128-group     */
    /* Option, OR'ed into the mode of fp8_quant_weight / fp8_quant_act: round
     * every scale to bf16 before the codes are computed (the FP8 checkpoints
     * store bf16 scales), so the codes are those a bf16-scale checkpoint holds.
     * A scale that rounds to zero becomes 1.  fp8_linear accepts and ignores it. */
    FP8Q_SCALE_BF16 = 0x10
} fp8q_mode;

/*
 * fp8_quant_weight -- quantize a bf16 weight W[N, K] (nn.Linear layout, out x in).
 *
 *   W_bf16   [N, ldw] bf16, read-only.  ldw >= K, (ldw * 2) % 16 == 0, 16-byte aligned.
 *   Wq       [N, ldwq] uint8 E4M3 codes, written.  ldwq >= K, ldwq % 16 == 0, 16-byte aligned.
 *   w_scale  fp32, written:  [N]                              (FP8Q_CHANNEL_TOKEN)
 *                            [ceil(N/128), K/128] row-major   (FP8Q_BLOCK128)
 *   Requirements: N >= 0, K > 0, K % 16 == 0; K % 128 == 0 in block mode.
 *   In block mode the last row-block may hold fewer than 128 rows; its amax
 *   covers the rows that exist.
 */
FP8Q_API fp8q_status fp8_quant_weight(const void* W_bf16, int64_t N, int64_t K, int64_t ldw, int mode,
                             uint8_t* Wq, int64_t ldwq, float* w_scale, void* stream);

/*
 * fp8_quant_act -- quantize bf16 activations X[M, K] (one row per token).
 *
 *   X_bf16   [M, ldx] bf16, read-only.  Same stride/alignment rules as W.
 *   Xq       [M, ldxq] uint8 codes, written.
 *   x_scale  fp32, written:  [M]                  (FP8Q_CHANNEL_TOKEN, per token)
 *                            [M, K/128] row-major (FP8Q_BLOCK128, per 128-group)
 *   Requirements: M >= 0 (M == 0 is a no-op), K > 0, K % 16 == 0;
 *   K % 128 == 0 in block mode.
 */
FP8Q_API fp8q_status fp8_quant_act(const void* X_bf16, int64_t M, int64_t K, int64_t ldx, int mode,
                          uint8_t* Xq, int64_t ldxq, float* x_scale, void* stream);

/*
 * fp8_quant_act_static -- quantize bf16 activations with one fixed scale.
 *
 * The static alternative to the dynamic per-token scheme: "Llama 3 精读实录"
 * section 2 calibrates each tensor offline from percentiles of a calibration
 * set (its 0.1% and 99.9% quantiles as the range, not min/max).  Every element
 * is coded as E4M3(fl32(x / scale)), saturating beyond the range.
 *   X_bf16, Xq  as fp8_quant_act.
 *   scale       > 0, finite: the calibrated scale (range / 448).
 *   x_scale     [M] fp32, written with `scale` when not NULL, so that
 *               fp8_linear in FP8Q_CHANNEL_TOKEN mode consumes Xq unchanged.
 *   Requirements: M >= 0 (M == 0 is a no-op), K > 0, K % 16 == 0.
 */
FP8Q_API fp8q_status fp8_quant_act_static(const void* X_bf16, int64_t M, int64_t K, int64_t ldx, float scale,
                                          uint8_t* Xq, int64_t ldxq, float* x_scale, void* stream);

/*
 * fp8_calibrate_static_scale -- the static scale fp8_quant_act_static takes,
 * from a calibration tensor: "Llama 3 精读实录" section 2 uses its 0.1% and
 * 99.9% quantiles as the range instead of min / max.  Offline, once per tensor.
 *   q(p)   = v[i] + (v[j] - v[i]) * (p (n-1) - i),  i = floor(p (n-1)),
 *            j = min(i + 1, n - 1), v the n = M*K values sorted ascending (double)
 *   amax   = max(|q(lo)|, |q(hi)|);   scale = fl32(fl32(amax) / 448), 1 when amax == 0
 * The order statistics are exact: the kernels count the 65536 bf16 bit patterns.
 *   X_bf16  [M, ldx] bf16, read-only, 16-byte aligned, ldx >= K, ldx % 8 == 0.
 *   lo, hi  quantile levels in [0, 1] (0.001 and 0.999 for the pages' range).
 *   hist    device workspace of 65536 uint32 counts (262144 bytes), 4-byte
 *           aligned, zero-filled before its first use; every completed call
 *           leaves it all zero.  Not shared by concurrent calls.
 *   scale   one fp32 in device memory, written.
 * Requirements: M >= 1, K >= 1, K % 8 == 0, M * K < 2^32 (FP8Q_ERR_UNSUPPORTED
 * above).  Values must be finite.
 */
FP8Q_API fp8q_status fp8_calibrate_static_scale(const void* X_bf16, int64_t M, int64_t K, int64_t ldx, double lo,
                                                double hi, uint32_t* hist, float* scale, void* stream);

/*
 * fp8_rmsnorm_quant_act -- RMSNorm of bf16 activations, then per-token E4M3
 * quantization of the result, in one pass (the normalised bf16 rows are not
 * written).  Llama 3 normalises with RMSNorm (eps 1e-5) before attention and
 * before the MLP and keeps it in BF16 ("Llama 3 精读实录", sections 1.3 and 5),
 * so this produces exactly the codes and scales that fp8_quant_act in
 * FP8Q_CHANNEL_TOKEN mode gives for the bf16 RMSNorm output.
 *
 *   X_bf16     [M, ldx] bf16 hidden states, read-only (rules as fp8_quant_act).
 *   gamma_bf16 [K] bf16 RMSNorm weight, 16-byte aligned.
 *   eps        >= 0, finite (1e-5 for Llama 3).
 *   Xq, x_scale as fp8_quant_act in FP8Q_CHANNEL_TOKEN mode ([M] scales).
 *   rstd       [M] fp32, written when not NULL: the row's 1 / sqrt(ms + eps).
 *   Per row:  ms   = the mean over the row of x^2, rounded once to fp32
 *             rstd = 1 / sqrt(fl32(ms + eps)), correctly rounded fp32
 *             y    = bf16(gamma * bf16(x * rstd))           (fp32 products)
 *             codes and scale of y as fp8_quant_act.
 *   The squares are exact in fp64 and summed in fp64, so ms is the exactly
 *   rounded mean except for a mean within a few fp64 roundings of an fp32
 *   rounding boundary (then it may be one fp32 step off, and rstd with it).
 *   Everything after rstd is exact, so rstd determines y and the codes.  Rows
 *   whose mean of squares overflows fp32 are outside the contract.
 *   Requirements: M >= 0 (M == 0 is a no-op), K > 0, K % 16 == 0, and
 *   K <= 65536 (FP8Q_ERR_UNSUPPORTED above).
 */
FP8Q_API fp8q_status fp8_rmsnorm_quant_act(const void* X_bf16, const void* gamma_bf16, int64_t M, int64_t K,
                                           int64_t ldx, float eps, uint8_t* Xq, int64_t ldxq, float* x_scale,
                                           float* rstd, void* stream);

/*
 * fp8_linear -- Y[M, N] = dequant(Xq) . dequant(Wq)^T in bf16, on tcgen05 tensor cores.
 *
 *   Xq        [M, K] uint8 codes, contiguous (row stride K), 16-byte aligned.
 *   x_scale   [M] or [M, K/128] fp32 (as written by fp8_quant_act in `mode`).
 *   Wq        [N, K] uint8 codes, contiguous, 16-byte aligned.
 *   w_scale   [N] or [ceil(N/128), K/128] fp32 (as written by fp8_quant_weight).
 *   Y_bf16    [M, ldy] bf16, written.  ldy >= N, (ldy * 2) % 16 == 0, 16-byte aligned.
 *   workspace device scratch of at least fp8_linear_workspace_size(M, N, K, mode)
 *             bytes, 16-byte aligned (may be NULL when that size is 0).  For
 *             M <= 64 it is required: a NULL or misaligned one is refused
 *             before anything touches the device.  For M > 64 it is optional:
 *             a nonzero size means the stream-K prefill schedule is switched
 *             on (environment FP8Q_PREFILL_STREAMK=1; off by default) for this
 *             shape (channel mode, few 256 x 256 tiles per CTA pair) and runs
 *             when the workspace is given; without it (NULL, or shorter) the
 *             data-parallel schedule runs, with the same result up to the
 *             order of the fp32 sums.  It holds
 *             the split-K arrival counters and fp32 partial sums of the small-M
 *             (decode) path.  It must be zero-filled before its first use; every
 *             completed call leaves it all zero again, so one zeroed buffer
 *             serves any sequence of calls (of any shape) on one stream.  After
 *             a call that failed on the device (fp8q_device_error nonzero), zero
 *             it again.  Two calls that run concurrently must not share one
 *             workspace.
 *   Requirements: M >= 0 (M == 0 is a no-op), N > 0, K > 0, K % 16 == 0,
 *   N % 16 == 0; K % 128 == 0 in block mode.  The mode must be the one both
 *   operands were quantized with.
 *   Dispatch: M <= 64 takes the decode kernel (weights streamed once, swap-AB,
 *   stream-K split over all SMs; the last warp to finish a weight tile's
 *   channels adds its partial sums in a fixed order, so results are
 *   deterministic; small block-scaled problems split each weight tile's K over
 *   the CTAs of one thread-block cluster instead, summed in distributed shared
 *   memory, and leave the workspace untouched); larger M takes the
 *   persistent warp-specialised prefill kernels, with 256 x 256 tiles per CTA
 *   pair, data-parallel or stream-K
 *   (parts of a tile summed in a fixed order by the last pair to finish it).
 */
FP8Q_API fp8q_status fp8_linear(const uint8_t* Xq, const float* x_scale, const uint8_t* Wq,
                       const float* w_scale, int64_t M, int64_t N, int64_t K, int mode,
                       void* Y_bf16, int64_t ldy, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * fp8_linear_swiglu -- the Llama MLP's gate and up projections and their
 * SwiGLU combination in one kernel ("Llama 3 精读实录" section 1.3: gate and up
 * computed separately, then silu(gate) * up):
 *   g = bf16(Xq . Wq_gate^T scaled),  u = bf16(Xq . Wq_up^T scaled)   (as fp8_linear)
 *   Y = bf16( bf16(silu(g)) * u ),   silu(v) = v / (1 + e^-v)
 * Only Y ([M, N], the down projection's input) is written.
 *   Xq, x_scale      as fp8_linear, FP8Q_CHANNEL_TOKEN scales ([M]).
 *   Wq_gate, Wq_up   [N, K] codes of the two weights (contiguous, 16-byte aligned);
 *   w_scale_gate/up  [N] fp32 per-channel scales.
 *   Y_bf16           [M, ldy] bf16, written (rules as fp8_linear).
 * Requirements as fp8_linear in channel mode.  Any M >= 1 runs the CTA-pair
 * prefill schedule (256 tokens x 128 channels per pair).  silu uses the fast
 * exponential; g and u match fp8_linear's outputs.  No workspace.
 */
FP8Q_API fp8q_status fp8_linear_swiglu(const uint8_t* Xq, const float* x_scale, const uint8_t* Wq_gate,
                                       const float* w_scale_gate, const uint8_t* Wq_up, const float* w_scale_up,
                                       int64_t M, int64_t N, int64_t K, void* Y_bf16, int64_t ldy, void* stream);

/*
 * fp8_linear_w8a16 -- weight-only FP8: the layer as GPUs without FP8 tensor
 * cores run these checkpoints ("Llama-3.1-70B-FP8-Dynamic" explainer, section
 * 三's GPU choice list and FAQ Q1: the FP8 weights are dequantized at compute
 * time).  The activations stay bf16:
 *   Y[m, n] = bf16( w_scale[n] * sum_k X[m, k] * E4M3(Wq[n, k]) ),
 * products and sums in fp32 (any order).
 *   X_bf16   [M, ldx] bf16 activations, 16-byte aligned, ldx >= K, ldx % 8 == 0.
 *   Wq       [N, K] uint8 codes, contiguous, 16-byte aligned (fp8_quant_weight,
 *            FP8Q_CHANNEL_TOKEN).
 *   w_scale  [N] fp32 per-channel scales.
 *   Y_bf16   [M, ldy] bf16, written; ldy >= N, 2-byte aligned.
 *   workspace  device scratch of fp8_linear_w8a16_workspace_size(M, N, K)
 *            bytes (NULL when that is 0), 16-byte aligned, with fp8_linear's
 *            contract: zero-filled before its first use, left all zero by
 *            every completed call; not shared by concurrent calls.
 * Requirements: 0 <= M <= 64 (M == 0 is a no-op; larger M returns
 * FP8Q_ERR_UNSUPPORTED: quantize the activations and call fp8_linear),
 * N > 0, K > 0, K % 16 == 0.
 * Dispatch: one token runs a CUDA-core kernel that streams the weights through
 * shared memory (no workspace); 2..64 tokens run the decode kernel's schedule
 * on the tensor cores with the weight tiles widened to bf16 in shared memory
 * (exactly: every E4M3 value is a bf16 value) and bf16 MMAs.
 */
FP8Q_API size_t fp8_linear_w8a16_workspace_size(int64_t M, int64_t N, int64_t K);
FP8Q_API fp8q_status fp8_linear_w8a16(const void* X_bf16, int64_t ldx, const uint8_t* Wq, const float* w_scale,
                                      int64_t M, int64_t N, int64_t K, void* Y_bf16, int64_t ldy,
                                      void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace fp8_linear needs for this problem on the current device
 * (0 for the prefill path).  Returns 0 for invalid arguments as well. */
FP8Q_API size_t fp8_linear_workspace_size(int64_t M, int64_t N, int64_t K, int mode);

/* Human-readable name of a status code (static string, never NULL). */
FP8Q_API const char* fp8q_status_string(int status);

/* Reads the device-side error word of the current device: 0 when no kernel
 * has given up waiting or met a bad index, otherwise a nonzero code naming the
 * wait site, or 0x201 (a slot past the cache), 0x202 (a page outside it) or 0x203
 * (a sequence's lengths), set by the KV cache's entry points.  It
 * synchronizes the device.  clear != 0 resets the word to 0 afterwards and,
 * when it was nonzero, also zeroes fp8_linear_noalloc's in-library scratch on
 * this device.  Returns -1 when a CUDA call fails. */
FP8Q_API int fp8q_device_error(int clear);

/*
 * fp8_linear_noalloc -- fp8_linear for M <= 64 without a caller-supplied workspace.
 *
 * The pages have no counterpart to this entry point; it exists for callers that
 * cannot allocate device memory at the moment they call: plugin or enqueue
 * interfaces that hand over inputs and outputs but no scratch, code that must
 * not pay cudaMalloc's implicit device synchronisation on its critical path,
 * and programs whose device-memory budget is fixed before they run.
 *
 * Same arguments, requirements and result as fp8_linear, minus the workspace.
 * The split-K scratch is instead a fixed array of 16 MiB (16777216 bytes)
 * compiled into the library: every GPU that loads libfp8q.so holds it until the
 * process exits.  This call allocates nothing (no cudaMalloc,
 * cudaFree or allocating library routine).
 *   - M > 64 returns FP8Q_ERR_UNSUPPORTED: call fp8_linear with a NULL workspace
 *     there, which needs no scratch and allocates nothing either.
 *   - A problem whose scratch would exceed the array (the size
 *     fp8_linear_workspace_size reports) returns FP8Q_ERR_UNSUPPORTED.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before any stream capture.  With CUDA's lazy module loading (the default)
 *     the array is reserved on a device when the library's device code is
 *     first loaded there: by that first call, or by any earlier call of this
 *     library on the device.  A caller whose memory budget is fixed should
 *     therefore make one call at setup time.
 *   - Every call on a device shares the one array, which keeps whatever the last
 *     call left in it: zero-filled when the library is loaded, and every
 *     completed call leaves it all zero again.  Calls whose kernels overlap on the GPU
 *     (different streams, or different host threads) race on the array and give
 *     wrong results; serialise them.
 *   - A call whose kernel gave up waiting (fp8q_device_error nonzero) can leave
 *     counters and partial sums in the array.  fp8q_device_error(1) then zeroes
 *     the current device's array as well as the error word (cudaMemset, which
 *     allocates nothing); call it before the next fp8_linear_noalloc.
 */
FP8Q_API fp8q_status fp8_linear_noalloc(const uint8_t* Xq, const float* x_scale, const uint8_t* Wq,
                                        const float* w_scale, int64_t M, int64_t N, int64_t K, int mode,
                                        void* Y_bf16, int64_t ldy, void* stream);

/* ------------------------------------------- rotary positions, 4-bit KV cache ---
 *
 * The attention block between fp8_linear's q/k/v projections and o_proj: queries
 * are rotated (fp8q_rope), keys and values are appended to a paged cache with
 * the keys' rotation applied on the way (fp8q_kv4_append), and attention reads
 * that cache (fp8q_kv4_attention).  Heads are bf16 tensors [T, heads, D] with
 * contiguous elements and any token and head strides (in elements), so the
 * parts of a fused q/k/v row are passed as they are.
 */

enum {
    FP8Q_ROPE_HALF = 0,           /* pairs (i, i + R/2), R = rot_dim                     */
    FP8Q_ROPE_INTERLEAVED = 1,    /* pairs (2i, 2i + 1)                                  */
    FP8Q_ROPE_INVERSE = 2         /* flag: rotate back (also the forward pass's gradient)*/
};

enum { FP8Q_ROPE_UNSCALED = 0, FP8Q_ROPE_LINEAR = 1, FP8Q_ROPE_LLAMA3 = 2, FP8Q_ROPE_YARN = 3 };

/* How rotary frequencies are stretched for long contexts.  factor >= 1.
 *   LINEAR   every frequency / factor.
 *   LLAMA3   with t = original_max_position * f / 2 pi turns over the original
 *            context: f / factor for t <= low, f for t >= high, linear in t
 *            between (Llama 3.1: factor 8, low 1, high 4, original 8192).
 *   YARN     linear in the pair index between the indices that make `high` and
 *            `low` turns (Peng et al. 2023: beta_fast 32, beta_slow 1); its
 *            attention factor is the caller's mscale. */
typedef struct {
    int type;                     /* FP8Q_ROPE_UNSCALED, _LINEAR, _LLAMA3 or _YARN       */
    double factor, low, high, original_max_position;
} fp8q_rope_scaling;

/*
 * fp8q_rope_frequencies -- the rot_dim / 2 rotary frequencies in radians per
 * position, theta^(-2i / rot_dim) stretched by `scaling` (NULL: unscaled).
 * Host only: `freq` is HOST memory; copy it to the device for the calls below.
 */
FP8Q_API fp8q_status fp8q_rope_frequencies(double* freq, int64_t rot_dim, double theta,
                                           const fp8q_rope_scaling* scaling);

/*
 * fp8q_rope -- rotate bf16 heads X[T, H, D] by their tokens' positions.
 *   y0 = x0 c - x1 s,  y1 = x1 c + x0 s,  c = mscale cos(a), s = mscale sin(a),
 *   a = positions[t] * freq[i];  FP8Q_ROPE_INVERSE negates s.
 * The angle is computed in fp64, the rotation in fp32, rounded once to bf16.
 *   X_bf16     [T, H, D], read-only; any strides >= 0, 2-byte aligned (16-byte
 *              aligned rows and rot_dim % 16 == 0 are the fast case).
 *   positions  [T] int64.      freq  [rot_dim / 2] fp64.
 *   rot_dim    even, 2 <= rot_dim <= D; elements from rot_dim on are copied.
 *   flags      FP8Q_ROPE_HALF or _INTERLEAVED, optionally | FP8Q_ROPE_INVERSE.
 *   mscale     > 0, finite (1 unless the context scaling asks for another).
 *   Y_bf16     [T, H, D], written; its rows must not overlap each other.  Y may
 *              be X with the same strides (in place), else must not overlap X.
 * T == 0 is a no-op.  T * H < 2^31.
 */
FP8Q_API fp8q_status fp8q_rope(const void* X_bf16, int64_t T, int64_t H, int64_t D, int64_t x_token_stride,
                               int64_t x_head_stride, const int64_t* positions, const double* freq, int64_t rot_dim,
                               int flags, float mscale, void* Y_bf16, int64_t y_token_stride, int64_t y_head_stride,
                               void* stream);

/*
 * A paged KV cache of E2M1 codes with an E4M3 scale for each 16 elements.
 * k_pages and v_pages are device memory [num_pages, kv_heads, page_size * 9 D / 16]
 * bytes (contiguous, 16-byte aligned); one (page, head) slab is page_size rows
 * of D/2 code bytes (element 2i in the low nibble of byte i), then page_size
 * rows of D/16 scale bytes.  A value is E2M1(code) * E4M3(scale) * k_scale (or
 * v_scale), one static fp32 per tensor: amax / 2688 of a calibration set uses
 * the formats' whole range (fp8_calibrate_static_scale's result / 6).
 *   page_size 16, 32, 64, 128 or 256;  D = head_dim 64 or 128.
 * Slot s is row s % page_size of page s / page_size.
 */
typedef struct {
    void* k_pages;
    void* v_pages;
    int64_t num_pages;
    int32_t page_size, kv_heads, head_dim;
    float k_scale, v_scale;
} fp8q_kv4_cache;

/* Bytes of one page of k_pages (or v_pages); 0 for sizes that are not supported. */
FP8Q_API size_t fp8q_kv4_page_bytes(int64_t page_size, int64_t kv_heads, int64_t head_dim);

/*
 * fp8q_kv4_append -- write T tokens' keys and values into the cache.
 * K is rotated by its positions in fp64 and rounded once to fp32 (with
 * positions and freq NULL it is taken as it is).  Then, for each 16 elements x,
 * each fp32 operation rounded once:
 *   code_s = E4M3(amax|x| / (6 g)),  s = E4M3(code_s) * g,  g = k_scale or v_scale
 *   code   = E2M1(x / s), 0 where s = 0   (both round to nearest even and saturate)
 *   K_bf16, V_bf16  [T, kv_heads, D], read-only, 16-byte aligned, strides % 8 == 0.
 *   slots           [T] int64.  A negative slot's token is skipped (padding); one
 *                   past the cache is skipped and sets the device error word.
 *                   Two tokens of a call must not share a slot.
 *   positions, freq, rot_dim, flags, mscale  as fp8q_rope, without
 *                   FP8Q_ROPE_INVERSE; rot_dim % 8 == 0 (else FP8Q_ERR_UNSUPPORTED).
 * T == 0 is a no-op.  Values must be finite.
 */
FP8Q_API fp8q_status fp8q_kv4_append(const fp8q_kv4_cache* cache, const void* K_bf16, int64_t k_token_stride,
                                     int64_t k_head_stride, const void* V_bf16, int64_t v_token_stride,
                                     int64_t v_head_stride, const int64_t* slots, int64_t T, const int64_t* positions,
                                     const double* freq, int64_t rot_dim, int flags, float mscale, void* stream);

/*
 * fp8q_kv4_read -- the cached keys and values of T slots as bf16 [T, kv_heads, D]
 * (zeros for a negative slot; one past the cache also sets the device error
 * word).  16-byte aligned, strides % 8 == 0, rows that do not overlap.
 */
FP8Q_API fp8q_status fp8q_kv4_read(const fp8q_kv4_cache* cache, const int64_t* slots, int64_t T, void* K_bf16,
                                   int64_t k_token_stride, int64_t k_head_stride, void* V_bf16,
                                   int64_t v_token_stride, int64_t v_head_stride, void* stream);

/*
 * fp8q_kv4_attention -- attention of new tokens over the cache (which already
 * holds them).  Sequence b has kv_len[b] tokens in the cache, in the pages
 * page_table[b, 0 .. ), and the query rows q_start[b] .. q_start[b + 1] - 1,
 * its last tokens: row i of n stands at position kv_len[b] - n + i.
 *   O[row, h] = sum_j softmax_j(sm_scale * Q[row, h] . k_j) v_j over the keys j < kv_len[b]
 *               that are visible: j <= position where causal, j > position - window
 *               where window > 0; head h reads cache head h / (Hq / kv_heads).
 *   A row that sees no key gets zeros (lse -inf).  Rows that belong to no
 *   sequence (behind q_start[B]) are left as they were.
 *   Q_bf16, O_bf16  [T, Hq, D], 16-byte aligned, strides % 8 == 0; O's rows must
 *                   not overlap each other or Q.  Q's values must be finite.
 *   page_table      [B, max_pages] int32, row stride table_stride >= max_pages;
 *                   max_pages * page_size < 2^31 - 65536.  Entries that no visible
 *                   key needs are not read; NULL where max_pages is 0.
 *   kv_len          [B] int32, 0 <= kv_len[b] <= max_pages * page_size.
 *   q_start         [B + 1] int32, ascending, q_start[B] <= T; NULL for one row
 *                   per sequence (row b is sequence b's; then max_q_len is 1).
 *   sm_scale        > 0, finite, as is its product with k_scale (1 / sqrt(D) for most models).
 *                   Scores sm_scale q.k are to stay below 2^27 in magnitude (they are fp32, which
 *                   holds no fractions there).  Weights are rounded to f16 with the row's
 *                   largest at 2^7 .. 2^15: one below 2^-21 of it keeps fewer than 11 bits.
 *   max_q_len       the largest number of rows of a sequence; longer ones set the
 *                   device error word.  Lengths stay on the device: a captured call
 *                   can be replayed with other lengths up to these bounds.  It chooses
 *                   the kernel for all sequences of the call: prompts and single tokens
 *                   are faster in two calls (each with its part of Q and O).
 *   lse             [T, Hq] fp32, written when not NULL: log sum_j exp(sm_scale q.k_j).
 *   workspace       fp8q_kv4_attention_workspace_size bytes, 16-byte aligned.  Its first
 *                   FP8Q_KV4_WORKSPACE_HEADER bytes are zero before its first use and left
 *                   zero by every completed call, of any sizes; what lies behind them is
 *                   scratch (so it is not to be shared with fp8_linear's workspace).  Not
 *                   shared by concurrent calls.
 *   After a call that failed on the device (fp8q_device_error nonzero), zero the
 *   workspace's header again.
 *   A bad length or page index on the device never leads out of the tensors: it
 *   sets the device error word, and the rows concerned are not to be used.
 */
#define FP8Q_KV4_WORKSPACE_HEADER 8192
FP8Q_API size_t fp8q_kv4_attention_workspace_size(const fp8q_kv4_cache* cache, int64_t B, int64_t T, int64_t Hq,
                                                  int64_t max_q_len);
FP8Q_API fp8q_status fp8q_kv4_attention(const fp8q_kv4_cache* cache, const void* Q_bf16, int64_t q_token_stride,
                                        int64_t q_head_stride, int64_t T, int64_t Hq, const int32_t* page_table,
                                        int64_t table_stride, int64_t max_pages, const int32_t* kv_len,
                                        const int32_t* q_start, int64_t B, int64_t max_q_len, float sm_scale,
                                        int causal, int64_t window, void* O_bf16, int64_t o_token_stride,
                                        int64_t o_head_stride, float* lse, void* workspace, size_t workspace_bytes,
                                        void* stream);

/* Library version: major * 10000 + minor * 100 + patch. */
FP8Q_API int fp8q_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_H_ */
