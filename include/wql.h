/*
 * wql.h -- C ABI of the GB300 (sm_103a) weight-quantized linear library (libwql.so).
 *
 * Two quantized linear layers as used by LLM serving engines:
 *   - AWQ-format W4A16: int4 weights packed 8 per uint32, one fp16 scale and one 4-bit zero
 *     point per group of 32/64/128 input channels, fp16 activations and output.
 *   - SmoothQuant W8A8: RMSNorm fused with per-token dynamic int8 quantisation, then an
 *     int8 x int8 -> int32 GEMM dequantised by per-token x per-channel scales.
 *
 * Sources (titles of the public write-ups the operations follow):
 *   [AWQ]  "LMDeploy ... INT4 quantisation" tutorial, section 2: AWQ quantises weights per group
 *          with an asymmetric zero point from each group's own min/max; group sizes 32/64/128.
 *   [TM]   same tutorial, section 5.1: the fp16 x int4 GEMM kernel of the serving engine.
 *   [AUQ]  "AUQ dual-process framework" article, section 3.3 (per-group scale and zero point)
 *          and section 5.4 (checkpoint tensors qweight, scales, zeros; dim 0 of qweight is the
 *          grouped input dimension, a multiple of 128 for group 128).
 *   [W8A8] "LMDeploy W8A8 quantisation guide": weight smoothing (smooth_ln_fcs, alpha 0.5),
 *          QRMSNorm / QLinear modules, per_token_quant_int8 (scale = absmax / 127),
 *          per_channel_quant (fp32 scale per output channel), matmul_kernel_dynamic_quant
 *          (int32 accumulator, c = c * rms_scale * linear_scale), and its fp8 variant.
 *   [FastLLM] "FastLLM architecture" article, section 5.2: KV cache int8 in groups of 128.
 *
 * Conventions for every entry point:
 *   - Matrices are row-major and dense (no strides).  K = input features, N = output
 *     features, M = tokens (rows of the activation), G = group size.
 *   - fp16 data is passed as uint16_t bit patterns (IEEE binary16).
 *   - Every pointer is DEVICE memory owned by the caller, 16-byte aligned.  The library never
 *     allocates, frees or keeps a pointer after the call returns.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls only enqueue work
 *     on that stream and return; outputs are valid once the stream reaches that point.
 *   - Arguments are validated before anything is enqueued.  On WQL_EINVAL / WQL_EUNSUPPORTED
 *     nothing is launched and outputs are untouched; wql_last_error() describes the problem.
 *     WQL_ECUDA reports a launch failure (cudaGetLastError after the launch).
 *   - Kernels that wait on on-chip barriers give up after a bounded time instead of hanging;
 *     they then record a device-side error that wql_device_status() returns as WQL_ETIMEOUT.
 *   - M = 0 is a valid empty call: it returns WQL_OK and launches nothing.
 *   - The library holds no per-call state; calls on different streams may run concurrently.
 *     It keeps per-device state for the life of the process (kernel attributes, the device
 *     error word's address, the scratch-free GEMM's array address).  cudaDeviceReset
 *     invalidates that state: no call may follow a reset of that device in the same process.
 *   - Weight prefetch (programmatic dependent launch): the W4A16 GEMMs and the decode path of the
 *     W8A8 GEMMs (int8 and fp8, up to 16 tokens) are launched so that they may start while the
 *     kernel enqueued just before them on the stream is still running, and they begin copying
 *     their WEIGHT operands (qweight / scales / qzeros, or qw) before that kernel has finished;
 *     only the activations and the outputs wait for it.  So the weight buffers must already
 *     hold their final contents when the preceding kernel on the stream starts finishing:
 *       * the library's own weight writers (wql_awq_pack, wql_per_channel_quant_i8/_fp8) make
 *         their writes visible device-wide before they exit, so pack-then-GEMM on one stream
 *         with nothing in between is safe;
 *       * a caller's kernel that writes weight buffers and is enqueued directly before one of
 *         these GEMMs must end each thread's writes with a device-scope fence (__threadfence()),
 *         or the two must be separated by something that is not a kernel launch (an event
 *         record/wait, a memcpy, a stream synchronisation).
 *     Writes to a GEMM's weights from other streams must be ordered by the caller as usual.
 */
#ifndef WQL_H_
#define WQL_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum wql_status {
  WQL_OK = 0,
  WQL_EINVAL = 1,        /* bad argument: shape, alignment, null pointer, group size */
  WQL_EUNSUPPORTED = 2,  /* valid request the library does not cover (e.g. K too large) */
  WQL_ECUDA = 3,         /* CUDA runtime/driver error at launch */
  WQL_ETIMEOUT = 4       /* a kernel's bounded on-chip wait expired (see wql_device_status) */
} wql_status;

/* Short constant description of a status code. */
const char* wql_status_string(int status);

/* Detail message of the last failing call on this host thread ("" if none). */
const char* wql_last_error(void);

/* ABI version: major * 10000 + minor * 100 + patch. */
int wql_version(void);

/* Synchronises `stream`, then reports and clears the device-side error word of the current
 * device: WQL_ETIMEOUT if a kernel abandoned a bounded wait since the last check, WQL_EINVAL if
 * none did but one met a page, slot or length out of range in device memory, WQL_ECUDA if the
 * synchronisation itself failed, WQL_OK otherwise. */
wql_status wql_device_status(void* stream);

/* Diagnostic of the failure path: launches one thread that waits on an on-chip barrier which
 * nothing completes.  Its bounded wait gives up after the same time limit as every kernel's
 * (about 2 s) and records the same device-side error, so the next wql_device_status() returns
 * WQL_ETIMEOUT (and clears it); the context stays usable.  Launches nothing else and touches no
 * caller memory.  Returns WQL_ECUDA if the launch fails. */
wql_status wql_diag_expire_wait(void* stream);

/* Phase trace of the W4A16 kernels, for a developer build compiled with -DWQL_PHASE_TRACE (a
 * library file of its own; the default build returns WQL_EUNSUPPORTED and does nothing).
 * Registers a device buffer buf of launches x ctas x 32 uint64 (caller-owned, zero-filled by the
 * caller): every later w4a16 launch whose output pointer y lies at ybase + l * ystride
 * (0 <= l < launches) writes, per CTA c < ctas, %globaltimer nanoseconds at its phase points into
 * buf[(l * ctas + c) * 32 + slot], and its SM id into slot 31.  Launches whose y lies elsewhere
 * are not recorded.  buf == NULL switches the trace off.  Stamps only: the kernels skip and
 * reorder nothing.  Call it between launches, not while one may be running. */
wql_status wql_trace_setup(uint64_t* buf, const void* ybase, uint64_t ystride, int launches, int ctas);

/* ----------------------------------------------------------------------------------------
 * awq_pack  [AWQ] section 2; [AUQ] sections 3.3 and 5.4.
 * Quantise fp32 weights w [K, N] to asymmetric int4, per group of G consecutive input
 * channels (k) and per output channel (n):
 *     s  = fp16((max_k w - min_k w) / 15)       (1.0 if that rounds to zero)
 *     z  = clamp(round(-min_k w / s), 0, 15)
 *     q  = clamp(round(w / s) + z, 0, 15)        round = half to even, fp32 arithmetic
 * so that w ~ (q - z) * s.  Outputs (all written in full):
 *     qweight [K, N/8] uint32: code of column n at bits 4*(n%8) of word n/8 of row k
 *     scales  [K/G, N] fp16
 *     qzeros  [K/G, N/8] uint32: zero points packed like qweight
 * Requires G in {32, 64, 128}, K % G == 0, N % 32 == 0, K >= 1.
 * ---------------------------------------------------------------------------------------- */
wql_status wql_awq_pack(const float* w, int K, int N, int group, uint32_t* qweight,
                        uint16_t* scales, uint32_t* qzeros, void* stream);

/* ----------------------------------------------------------------------------------------
 * w4a16_gemm  [AWQ] section 2, [TM] section 5.1.
 *     y[m, n] = sum_k x[m, k] * (q[k, n] - z[k/G, n]) * s[k/G, n]
 * x [M, K] fp16, packed weight as produced by wql_awq_pack, y [M, N] fp16 (written in full;
 * accumulation in fp32).  Decode-shaped calls (small M) stream the packed weight once with
 * tensor-core dot products; prefill-shaped calls use the tcgen05 tensor-core kernel.
 * Requires G in {32, 64, 128}, K % G == 0, N % 32 == 0, M >= 0.
 * ---------------------------------------------------------------------------------------- */
wql_status wql_w4a16_gemm(const uint16_t* x, const uint32_t* qweight, const uint16_t* scales,
                          const uint32_t* qzeros, int M, int K, int N, int group, uint16_t* y,
                          void* stream);

/* ----------------------------------------------------------------------------------------
 * w4a16_gemm_silu_mul  [FastLLM] section 2: the gate and up projections of an MLP as one GEMM,
 * with SiLU(gate) * up fused into its epilogue.  Reading: the packed weight (wql_awq_pack of a
 * [K, N] matrix) interleaves the projections by output channel -- channel 2j is gate j and
 * channel 2j + 1 is up j -- and
 *     y[m, j] = fp16(silu(g) * u),  g = fp16(gemm[m, 2j]),  u = fp16(gemm[m, 2j + 1]),
 *     silu(g) = g / (1 + exp(-g))   (fp32; IEEE division, expf)
 * i.e. exactly the unfused GEMM's fp16 outputs followed by the activation, without writing them.
 * x [M, K] fp16; y [M, N / 2] fp16.  Same kernels and requirements as wql_w4a16_gemm, and
 * N % 64 == 0.
 * ---------------------------------------------------------------------------------------- */
wql_status wql_w4a16_gemm_silu_mul(const uint16_t* x, const uint32_t* qweight, const uint16_t* scales,
                                   const uint32_t* qzeros, int M, int K, int N, int group, uint16_t* y,
                                   void* stream);

/* ----------------------------------------------------------------------------------------
 * w4a16_kernel_for: the kernel wql_w4a16_gemm runs for an M x K x N call with group size
 * `group` on the current device: 0 = the weight-streaming decode kernel, 1 = the tcgen05
 * tensor-core kernel.  Up to 16 tokens it is always 0 and from 33 on always 1; in between it
 * depends on N, K and the group size.  Host-only, never fails (the WQL_FORCE_KERNEL
 * benchmarking switch is not consulted).
 * ---------------------------------------------------------------------------------------- */
int wql_w4a16_kernel_for(int M, int K, int N, int group);

/* ----------------------------------------------------------------------------------------
 * qrmsnorm_quant_i8  [W8A8] QRMSNorm.forward + rms_norm_dynamic_quant / per_token_quant_int8.
 * Per row m of x [M, K] fp16, with gamma [K] fp16 (smoothing already folded in):
 *     ss   = sum_k x^2 in a fixed order: element k joins lane (k/8) % 256, lanes add in
 *            increasing k, then lanes fold pairwise (t, t+128), (t, t+64), ..., (t, t+1)
 *     r    = 1 / sqrt(ss / K + eps)
 *     y_k  = (x_k * r) * gamma_k            (fp32, one rounding per operation, kept in fp32)
 *     xs_m = max_k |y_k| / 127              (1.0 if the row is all zero)
 *     q_mk = clamp(round_half_even(y_k / xs_m), -128, 127)
 * Outputs q [M, K] int8 and xs [M] fp32, bit-exact with the definition above.
 * Requires K % 8 == 0, 8 <= K <= 16384.
 * ---------------------------------------------------------------------------------------- */
wql_status wql_qrmsnorm_quant_i8(const uint16_t* x, const uint16_t* gamma, float eps, int M,
                                 int K, int8_t* q, float* xs, void* stream);

/* ----------------------------------------------------------------------------------------
 * add_qrmsnorm_quant_i8  [W8A8] "inference kernels": rms_norm_dynamic_quant with its residual
 * fusion (add_rms_norm_quant_kernel).  The page names the fusion, not its arithmetic; reading:
 *     h[m, k] = fp16(float(x[m, k]) + float(residual[m, k]))   (one fp32 add, one rounding)
 * h is written to residual_out [M, K] fp16 (the new residual stream; residual_out may be the
 * residual buffer itself), and q [M, K] int8, xs [M] fp32 are QRMSNorm + per-token int8 of h,
 * exactly as wql_qrmsnorm_quant_i8 computes them for an input h.
 * Requires K % 8 == 0, 8 <= K <= 16384; every pointer 16-byte aligned (xs: 4-byte).
 * ---------------------------------------------------------------------------------------- */
wql_status wql_add_qrmsnorm_quant_i8(const uint16_t* x, const uint16_t* residual,
                                     const uint16_t* gamma, float eps, int M, int K,
                                     uint16_t* residual_out, int8_t* q, float* xs, void* stream);

/* ----------------------------------------------------------------------------------------
 * per_token_quant_i8 / per_token_quant_fp8  [W8A8] per_token_quant_int8, the quantiser
 * QLinear.forward applies when its input is a plain tensor rather than QRMSNorm's output.
 * Per row m of x [M, K] fp16, with x_k the fp16 value widened to fp32:
 *     xs_m = max_k |x_k| / Q_MAX    (Q_MAX = 127 for int8, 448 for e4m3; 1.0 if the row is zero)
 *     q_mk = clamp(round_half_even(x_k / xs_m), -128, 127)     (int8)
 *     q_mk = e4m3(x_k / xs_m)       (fp8: the e4m3 value nearest the fp32 quotient, ties to even)
 * Outputs q [M, K] (int8, or e4m3 bytes) and xs [M] fp32, bit-exact with the definition above;
 * (q, xs) feed wql_w8a8_gemm / wql_w8a8_gemm_fp8 as QRMSNorm's outputs do.
 * Requires K % 8 == 0, 8 <= K <= 16384 (WQL_EUNSUPPORTED above); x and q 16-byte aligned, xs
 * 4-byte aligned.
 * ---------------------------------------------------------------------------------------- */
wql_status wql_per_token_quant_i8(const uint16_t* x, int M, int K, int8_t* q, float* xs, void* stream);
wql_status wql_per_token_quant_fp8(const uint16_t* x, int M, int K, uint8_t* q, float* xs, void* stream);

/* ----------------------------------------------------------------------------------------
 * w8a8_gemm  [W8A8] QLinear.forward / matmul_kernel_dynamic_quant.
 *     acc[m, n] = sum_k q[m, k] * qw[n, k]                 (exact int32)
 *     y[m, n]   = fp16((float(acc[m, n]) * xs[m]) * ws[n])  (fp32, left to right)
 * q [M, K] int8 with per-token scales xs [M] fp32; qw [N, K] int8 (input dimension
 * contiguous, as a torch Linear weight) with per-channel scales ws [N] fp32.
 * y [M, N] fp16 is written in full; acc_out [M, N] int32 is written too when non-NULL.
 * The int32 result is exact for every input (|acc| < 2^31 holds for K <= 131072).
 * workspace: device scratch of at least wql_w8a8_workspace_bytes(M, K, N) bytes (M * K * 2 +
 * 16384 for M >= 17: an fp16 copy of q and the largest row L1 norms of q; 0 below), used only
 * during the call (may be NULL when that size is 0).
 * Requires K % 16 == 0, N % 32 == 0, M >= 0, K <= 131072.
 * ---------------------------------------------------------------------------------------- */
size_t wql_w8a8_workspace_bytes(int M, int K, int N);
wql_status wql_w8a8_gemm(const int8_t* q, const float* xs, const int8_t* qw, const float* ws,
                         int M, int K, int N, uint16_t* y, int32_t* acc_out, void* workspace,
                         size_t workspace_bytes, void* stream);

/* ----------------------------------------------------------------------------------------
 * w8a8_gemm_fused  [W8A8] "inference kernels": the _linear_add variant of
 * matmul_kernel_dynamic_quant with its optional bias and residual.  The page names the
 * fusion, not its arithmetic; reading:
 *     y[m, n] = fp16(((float(acc[m, n]) * xs[m]) * ws[n] + float(bias[n])) + float(residual[m, n]))
 * in fp32, left to right, one rounding to fp16.  bias [N] fp16 and residual [M, N] fp16 are
 * each optional (NULL leaves the term out); residual may be y itself (in place).  Everything
 * else, including acc_out and the workspace, is as for wql_w8a8_gemm.
 * ---------------------------------------------------------------------------------------- */
wql_status wql_w8a8_gemm_fused(const int8_t* q, const float* xs, const int8_t* qw, const float* ws,
                               const uint16_t* bias, const uint16_t* residual, int M, int K, int N,
                               uint16_t* y, int32_t* acc_out, void* workspace,
                               size_t workspace_bytes, void* stream);

/* ----------------------------------------------------------------------------------------
 * w8a8_gemm_noalloc -- the same operation as wql_w8a8_gemm (same kernels, same results) for
 * callers that cannot allocate device memory at call time: an engine that has already handed
 * its whole memory budget to its own pool, a plugin whose host framework owns every allocation,
 * or a latency-critical loop that must not pay for the allocator's synchronisation.  The source
 * pages have no counterpart to this entry point; it exists for such callers only.
 * Instead of a caller workspace it uses a scratch array built into the library:
 *   - 32 MiB + 64 KiB, so M * K * 2 + 16384 <= 33619968 (e.g. M = K = 4096); larger calls return
 *     WQL_EUNSUPPORTED with a message in wql_last_error() and launch nothing;
 *   - one array per GPU that loads the library, held until the process exits;
 *   - the first call on a device looks up the array's device address (cudaGetSymbolAddress,
 *     with that device current) and keeps it; make that first call before any stream capture.
 *     cudaDeviceReset invalidates the kept address: no call may follow a reset of that device
 *     in the same process;
 *   - every call on a device shares the one array.  Calls that may overlap on the GPU (other
 *     streams, other threads) race on it and must be serialised by the caller.  Nothing in it
 *     needs to start at zero: each call overwrites every byte it later reads.
 * The library allocates and frees nothing in this call.
 * ---------------------------------------------------------------------------------------- */
wql_status wql_w8a8_gemm_noalloc(const int8_t* q, const float* xs, const int8_t* qw,
                                 const float* ws, int M, int K, int N, uint16_t* y,
                                 int32_t* acc_out, void* stream);

/* ----------------------------------------------------------------------------------------
 * Offline preparation for W8A8 ([W8A8] "weight smoothing" and QLinear.from_float).
 *
 * wql_act_absmax: calibration statistic a_j = max_m |RMSNorm_gamma(x)[m, j]| over x [M, K]
 *   (same fp32 RMSNorm as wql_qrmsnorm_quant_i8, original gamma).  absmax [K] fp32 is
 *   overwritten.  Requires K % 8 == 0, 8 <= K <= 16384.
 * wql_smooth: smooth_ln_fcs with alpha = 0.5 for one norm feeding one linear w [K, N] fp32:
 *     w_j = max_n |w[j, n]|;  s_j = sqrt(a_j / w_j)  (1 where a_j or w_j is 0)
 *     gamma_out_j = fp16(gamma_j / s_j);  w_out[j, n] = w[j, n] * s_j
 *   Outputs s [K] fp32, gamma_out [K] fp16, w_out [K, N] fp32 (may alias w).
 * wql_per_channel_quant_i8: ws_n = max_k |w[k, n]| / 127 (1.0 for a zero column);
 *     qw[n, k] = clamp(round_half_even(w[k, n] / ws_n), -127, 127)
 *   w [K, N] fp32 -> qw [N, K] int8 (transposed), ws [N] fp32.
 * Requires K % 16 == 0, N % 32 == 0.
 * ---------------------------------------------------------------------------------------- */
wql_status wql_act_absmax(const uint16_t* x, const uint16_t* gamma, float eps, int M, int K,
                          float* absmax, void* stream);
wql_status wql_smooth(const float* absmax, const uint16_t* gamma, const float* w, int K, int N,
                      float* s, uint16_t* gamma_out, float* w_out, void* stream);
wql_status wql_per_channel_quant_i8(const float* w, int K, int N, int8_t* qw, float* ws,
                                    void* stream);

/* ========================================================================================
 * FP8 variant of W8A8 ([W8A8]: quant_dtype "fp8", the short name of float8_e4m3fn).
 * Codes are float8 e4m3 bytes (1 sign, 4 exponent bits with bias 7, 3 fraction bits, no
 * infinity, largest value 448), passed as uint8_t.  Q_MAX = 448 (torch.finfo of the type)
 * replaces 127, and the page casts instead of rounding to an integer.  Reading of the cast:
 * nearest e4m3 value, ties to even, magnitudes beyond 448 saturated to 448.
 * ======================================================================================== */

/* ----------------------------------------------------------------------------------------
 * qrmsnorm_quant_fp8: wql_qrmsnorm_quant_i8 with fp8 codes.  y is the same fp32 RMSNorm;
 *     xs[m]   = max_k |y[m, k]| / 448   (1.0 for an all-zero row)
 *     q[m, k] = e4m3(y[m, k] / xs[m])   (the quotient correctly rounded in fp32 first)
 * add_qrmsnorm_quant_fp8: the residual fusion, exactly as wql_add_qrmsnorm_quant_i8 (h =
 * fp16(x + residual) goes to residual_out, which may be residual itself) with fp8 codes.
 * Requires K % 8 == 0, 8 <= K <= 16384; every pointer 16-byte aligned (xs: 4-byte).
 * ---------------------------------------------------------------------------------------- */
wql_status wql_qrmsnorm_quant_fp8(const uint16_t* x, const uint16_t* gamma, float eps, int M, int K,
                                  uint8_t* q, float* xs, void* stream);
wql_status wql_add_qrmsnorm_quant_fp8(const uint16_t* x, const uint16_t* residual,
                                      const uint16_t* gamma, float eps, int M, int K,
                                      uint16_t* residual_out, uint8_t* q, float* xs, void* stream);

/* ----------------------------------------------------------------------------------------
 * per_channel_quant_fp8: ws_n = max_k |w[k, n]| / 448 (1.0 for a zero column);
 *     qw[n, k] = e4m3(w[k, n] / ws_n)
 *   w [K, N] fp32 -> qw [N, K] e4m3 (transposed), ws [N] fp32.  Requires K % 16 == 0, N % 32 == 0.
 * ---------------------------------------------------------------------------------------- */
wql_status wql_per_channel_quant_fp8(const float* w, int K, int N, uint8_t* qw, float* ws,
                                     void* stream);

/* ----------------------------------------------------------------------------------------
 * w8a8_gemm_fp8  [W8A8] matmul_kernel_dynamic_quant with fp8 inputs (fp32 accumulator) and
 * the optional terms of its _linear_add variant:
 *     acc[m, n] = sum_k e4m3(q[m, k]) * e4m3(qw[n, k])       (fp32 accumulation)
 *     y[m, n]   = fp16(((acc[m, n] * xs[m]) * ws[n] + float(bias[n])) + float(residual[m, n]))
 * q [M, K], qw [N, K] e4m3; xs [M], ws [N] fp32; bias [N] and residual [M, N] fp16, each
 * optional (NULL leaves the term out; residual may be y itself).  y [M, N] fp16 is written in
 * full, and acc_out [M, N] fp32 too when non-NULL.  The order of the fp32 additions is the
 * kernel's own (tensor-core sums, then a fixed-order split-K reduction), so acc differs from
 * the exact sum by at most K * 2^-23 * sum_k |product| -- an fp32 rounding per addition.
 * No workspace.  Requires K % 16 == 0, N % 32 == 0, M >= 0.
 * ---------------------------------------------------------------------------------------- */
wql_status wql_w8a8_gemm_fp8(const uint8_t* q, const float* xs, const uint8_t* qw, const float* ws,
                             const uint16_t* bias, const uint16_t* residual, int M, int K, int N,
                             uint16_t* y, float* acc_out, void* stream);

/* ========================================================================================
 * KV cache int8 in groups of 128 ([FastLLM] section 5.2: the K and V cache stored as int8 with
 * group size 128, dequantised when read).  The page fixes the width and the group size only.
 * Reading: a group is 128 consecutive channels of one row (one token's K or V vector),
 * symmetric like [W8A8]'s per-token int8:
 *     scales[r, g] = max_{k in group g} |kv[r, k]| / 127      (fp32; 1.0 for an all-zero group)
 *     q[r, k]      = clamp(round_half_even(kv[r, k] / scales[r, k / 128]), -128, 127)
 * and the cache entry read back is out[r, k] = fp16(float(q[r, k]) * scales[r, k / 128]).
 * kv and out are [rows, D] fp16, q is [rows, D] int8, scales [rows, D / 128] fp32, all row-major
 * and contiguous (rows may count tokens x layers; a row is any run of D channels).
 * Requires D % 128 == 0, rows >= 0 (0 is a no-op); pointers 16-byte aligned (scales: 4-byte).
 * ======================================================================================== */
wql_status wql_kv_quant_i8(const uint16_t* kv, int64_t rows, int D, int8_t* q, float* scales,
                           void* stream);
wql_status wql_kv_dequant_i8(const int8_t* q, const float* scales, int64_t rows, int D,
                             uint16_t* out, void* stream);

/* ========================================================================================
 * Paged KV cache in 4 bits, and attention ([FastLLM] section 5.2 names int4 next to int8 for the
 * cache and section 3 its pages; [AWQ] section 3 the paged attention.  The pages fix no format;
 * the readings below are this library's).
 *
 * The cache is uint8 [pages, H, page_size / 16, 16 (D + 8)], H the K/V heads: blocks of 16 tokens
 * of one head, each block
 *     K codes [16, D / 2]   (channel 2i in the low half of byte i, channel 2i + 1 in the high)
 *     V codes [16, D / 2]
 *     K params [16] {fp16 s, fp16 lo}, V params [16] {fp16 s, fp16 lo}
 * with value = code * s + lo.  Token slot n lies in page n / page_size, block (n % page_size) / 16,
 * row n % 16.  D is 64 or 128 (WQL_EUNSUPPORTED otherwise); page_size is any multiple of 16;
 * pages * page_size < 2^31 (the byte offsets may pass 2^32).
 *
 * Activations here are token-major with a stride: element (t, h, d) of q, k or v lies at
 * t * stride + h * D + d, so that views of a fused QKV projection's output are taken as they are.
 * Strides count elements, are multiples of 8 and at least heads * D.  Outputs are dense.
 *
 * Lengths, slots and page numbers are read on the device, so nothing is copied to the host and a
 * captured call follows their contents.  One that is out of range is left out (see each entry) and
 * recorded: the next wql_device_status() returns WQL_EINVAL once.
 * ======================================================================================== */

/* ----------------------------------------------------------------------------------------
 * kv_plan_pages: block tables and slot maps from request lengths.  Request i holds ctx_lens[i]
 * tokens in ceil(ctx_lens[i] / page_size) pages, listed in row i of block_table [B, table_width],
 * and adds new_lens[i] tokens (negative lengths count as 0).  In request order it is given the
 * pages it lacks from the end of the free list: with n = free_count[0] and `before` the pages that
 * the requests before it lack, its k-th new page is free_pages[n - 1 - before - k], written
 * behind the pages it holds.  Requests that exceed table_width pages, and those from the first one
 * on that the free list cannot serve (except any that lack no page), are refused: they get none.
 *     cu_new [B + 1]   exclusive sums of new_lens: the first new token of each request
 *     kv_lens [B]      ctx_lens + new_lens; 0 for a refused request
 *     slots [T]        slot of each new token, in the packed order of cu_new; -1 for tokens of
 *                      refused requests and behind the last token (T may exceed cu_new[B]; tokens
 *                      from T on get no slot), and where the page number is negative or so large
 *                      that the slot would pass 2^31 - 1
 *     free_count_out   [1]: pages left, which are free_pages[0 .. free_count_out - 1]
 * Only the entries of new pages are written in block_table.  free_capacity is free_pages' size, and
 * free_count is taken as at most that.  Repeating a call gives the same result.
 * Requires B <= 4096, sum(new_lens) < 2^31, table_width * page_size < 2^31; slots 16-byte, the
 * others 4-byte aligned; no output may overlap an input (block_table, read and written, aside).
 * ---------------------------------------------------------------------------------------- */
wql_status wql_kv_plan_pages(const int32_t* ctx_lens, const int32_t* new_lens, int B, int page_size,
                             const int32_t* free_pages, int free_capacity, const int32_t* free_count,
                             int32_t* block_table, int table_width, int T, int32_t* cu_new,
                             int32_t* kv_lens, int32_t* slots, int32_t* free_count_out, void* stream);

/* ----------------------------------------------------------------------------------------
 * kv_append_i4: quantise rows k, v [T, H, D] fp16 into the cache at slots [T].  Per row x [D]:
 *     lo = min x;  s = fp16((max x - lo) / 15)   (1.0 if that is zero)
 *     code = clamp(round_half_even((x - lo) / s), 0, 15)
 * Differences and quotients are the real ones, rounded once, so the cache is bit-exact with this
 * definition.  A row that holds an infinity or a NaN gets s = lo = NaN and reads back as NaN.
 * s may be rounded up, so that code * s + lo passes the row's maximum by up to 2^-11 of max x - lo
 * (15 * 2^-25 where s is below 2^-14): a finite row with values near 65504 can hold more than fp16 does
 * (0 .. 65504: 15 * 4368 = 65520), which kv_read_i4 rounds to infinity and attention_kv_i4, whose sums
 * are fp32, takes as it is.
 * Negative slots are passed over (padding); slots behind the last page are left out and recorded.
 * No slot may occur twice in a call: what such a slot then holds is unspecified.  T * H < 2^31
 * (WQL_EUNSUPPORTED above), here and in kv_read_i4.
 * kv_read_i4: k, v [T, H, D] fp16 (dense) = fp16(code * s + lo) of the rows at slots, one rounding;
 * zeros for negative slots and slots out of range.  A slot may occur any number of times.
 * ---------------------------------------------------------------------------------------- */
wql_status wql_kv_append_i4(const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                            int T, int H, int D, const int32_t* slots, uint8_t* cache, int64_t pages,
                            int page_size, void* stream);
wql_status wql_kv_read_i4(const uint8_t* cache, int64_t pages, int page_size, int H, int D,
                          const int32_t* slots, int T, uint16_t* k, uint16_t* v, void* stream);

/* ----------------------------------------------------------------------------------------
 * attention_kv_i4: attention of the last Lq tokens of each of B sequences over the cache.
 * Sequence b has kv_lens[b] tokens (the Lq queried ones among them) in the pages of row b of
 * block_table [B, table_width].  For row r < Lq and query head h, with k and v of K/V head
 * h / (Hq / Hkv):
 *     out[b, r, h] = sum_t softmax_t(scale * q[b, r, h] . k[t]) v[t],   t <= kv_lens[b] - Lq + r
 * and zeros where no t is visible (kv_lens[b] = 0, or fewer tokens than rows).  |scale| <= 2^64, here
 * and in attention_prompt: scores of any fp16 rows are then finite.  q is [B * Lq, Hq,
 * D] fp16 with q_stride, out [B, Lq, Hq, D] fp16, dense.  Lq = 1 is the decode step; more rows verify
 * drafted tokens or run a chunk of a prompt over its cached beginning.
 * Score and value sums are fp32.  From five rows (Lq * Hq / Hkv) on, a weight times its token's s is
 * rounded to fp16 for the product with code - 7.5, so that the rounding adds at most 2^-11 p |s| |code -
 * 7.5| of a token with the weight p (2^-32 of the row's largest p |s| where p |s| is below 2^-21 of
 * that); a constant row, as kv_append_i4 stores it, adds exactly p v.  With fewer rows what the
 * rounding leaves is added too.  The result does not depend on what lies behind a
 * sequence's last token.
 * A length beyond table_width * page_size is cut there and recorded; a page number out of range
 * among the pages in use is recorded, and the outputs of that sequence are then unspecified.
 * workspace: device scratch of at least wql_attention_kv_i4_workspace_bytes(B, Lq, Hq, Hkv, D)
 * bytes (the current device's), with no contents to keep; calls that may run at the same time
 * need one each.  out must overlap no input.  Calls and results are deterministic.
 * Requires B * Hkv * ceil(Lq * Hq / Hkv / 8) * (table_width * page_size / 32 + 5) < 2^31
 * (WQL_EUNSUPPORTED above).
 * ---------------------------------------------------------------------------------------- */
size_t wql_attention_kv_i4_workspace_bytes(int B, int Lq, int Hq, int Hkv, int D);
wql_status wql_attention_kv_i4(const uint16_t* q, int64_t q_stride, int B, int Lq, int Hq, int Hkv,
                               int D, const uint8_t* cache, int64_t pages, int page_size,
                               const int32_t* block_table, int table_width, const int32_t* kv_lens,
                               float scale, uint16_t* out, void* workspace, size_t workspace_bytes,
                               void* stream);

/* ----------------------------------------------------------------------------------------
 * attention_prompt: causal attention over B packed prompts.  Sequence b is rows cu_seqlens[b] ..
 * cu_seqlens[b + 1] - 1 of q [T, Hq, D], k and v [T, Hkv, D] (fp16, strided); for its row r and
 * query head h, with k and v of K/V head h / (Hq / Hkv):
 *     out[r, h] = sum_{j <= r} softmax_j(scale * q[r, h] . k[j]) v[j]
 * out [T, Hq, D] fp16, dense; rows of no sequence are left as they were.  cu_seqlens [B + 1]: a
 * sequence with a negative start, a negative length or an end beyond T is left out and recorded;
 * rows that two of the others then share are written by both, in no order.
 * Sums are fp32, weights fp16.  A row depends on nothing but the rows up to it of its sequence: an
 * infinity or a NaN elsewhere does not reach it; one in v that it does see makes that channel of
 * it infinite or NaN.  No workspace.  Requires Hq <= 65535; out must overlap no input.
 * ---------------------------------------------------------------------------------------- */
wql_status wql_attention_prompt(const uint16_t* q, int64_t q_stride, const uint16_t* k,
                                int64_t k_stride, const uint16_t* v, int64_t v_stride, int T, int Hq,
                                int Hkv, int D, const int32_t* cu_seqlens, int B, float scale,
                                uint16_t* out, void* stream);

/* ----------------------------------------------------------------------------------------
 * attention_chunks_kv_i4: attention of packed chunks of new tokens over the cache, as a step of continuous
 * batching (chunked prefill, whole prompts, single tokens, all in one call) has them after kv_plan_pages and
 * kv_append_i4.  Sequence b's chunk is rows cu_new[b] .. cu_new[b + 1] - 1 of q [T, Hq, D] (fp16, strided), the
 * last n of the kv_lens[b] tokens that the pages of row b of block_table [B, table_width] hold.  For its row r < n
 * and query head h, with k and v of K/V head h / (Hq / Hkv):
 *     out[cu_new[b] + r, h] = sum_t softmax_t(scale * q . k[t]) v[t],   t <= kv_lens[b] - n + r
 *     lse[cu_new[b] + r, h] = ln(sum_t exp(scale * q . k[t]))
 * and zeros with lse = minus infinity where no t is visible (kv_lens[b] = 0, as kv_plan_pages gives a refused
 * request, or fewer tokens than rows).  out [T, Hq, D] fp16 and lse [T, Hq] fp32 are dense; lse may be NULL.  Rows of
 * no sequence are left as they were.
 * k and v are code * s + lo rounded to fp16, as kv_read_i4 gives them, but never infinite: what rounds to infinity is
 * taken as 65504.  A row of K or V whose parameters are not finite makes the rows that see it NaN.  Sums are fp32, weights
 * fp16: a weight is off by 2^-11 of itself (2^-32 of the row's largest one where it is below 2^-21 of that).  Tensor cores cut a
 * product off at the last place of the sum that it is added to: of n tokens with about the same weight that a CTA adds up (a 152nd of
 * those of all K/V heads and tiles of rows), up to n 2^-24 of the output is lost.  A row
 * depends on nothing behind the last token that it sees.  |scale| <= 2^64.
 * A sequence with a negative start, a negative length or an end beyond T is left out and recorded; a length beyond
 * table_width * page_size is cut there and recorded; a page number out of range among the pages in use is recorded, and
 * the outputs of that sequence are then unspecified.  Rows that two sequences share are written by both, in no order.
 * workspace: device scratch of at least wql_attention_chunks_kv_i4_workspace_bytes(T, B, Hq, Hkv, D) bytes (the
 * current device's), with no contents to keep; calls that may run at the same time need one each.  out and lse must
 * overlap no input and not each other.  Results are deterministic.
 * Requires B <= 4096, Hq <= 65535, Hq / Hkv <= 128, T * Hq < 2^31 (WQL_EUNSUPPORTED above).
 * ---------------------------------------------------------------------------------------- */
size_t wql_attention_chunks_kv_i4_workspace_bytes(int T, int B, int Hq, int Hkv, int D);
wql_status wql_attention_chunks_kv_i4(const uint16_t* q, int64_t q_stride, int T, int Hq, int Hkv, int D,
                                      const uint8_t* cache, int64_t pages, int page_size,
                                      const int32_t* block_table, int table_width, const int32_t* cu_new,
                                      const int32_t* kv_lens, int B, float scale, uint16_t* out, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream);

/* ----------------------------------------------------------------------------------------
 * kv_weights_i4: the attention weight that every cached token gets from the rows of packed chunks, added to
 * running sums.  q, cu_new, kv_lens, block_table, scale as in attention_chunks_kv_i4, whose lse [T, Hq] it takes:
 *     weights[b, kvh, t] += sum_{r, h} exp(scale * q[cu_new[b] + r, h] . k[t] - lse[cu_new[b] + r, h])
 * over the rows r of sequence b that see t and the query heads h of kvh's group.  weights is fp32
 * [B, Hkv, table_width * page_size], dense; entries from kv_lens[b] on, and those of sequences without rows, are left
 * as they were.  Each sum is formed in fp32 and added once.  k is what attention_chunks_kv_i4 takes; a row of K whose
 * parameters are not finite makes the sums that it belongs to NaN, and so does a row r whose lse is NaN.
 * Sequences, lengths and pages out of range: as there; the sums of a sequence with a bad page are unspecified.
 * A sum, or an entry that one is added to, of less than 2^-126 in magnitude may count as zero.
 * A weight exp(t), t = scale * q . k - lse, is off by a factor of at most e^d with d = 2^-20 + 2^-22 |t| + (D + 8) 2^-23 |scale|
 * sum_c |q_c k_c| for the lse that it is given.  What that lse is off comes on top, as d does: an fp32 number by 2^-24 of
 * itself at least, attention_chunks_kv_i4's by up to 2^-22 of it and of the row's largest score, and by the scores' own error.  So from
 * scores of about 2^18 on weights say which tokens rather than how much, and from 2^26 on one that should be 1 may be
 * anything, infinity too: sums of such weights are not worth keeping.
 * workspace: device scratch of at least wql_kv_weights_i4_workspace_bytes() bytes (the current device's), with no contents
 * to keep; calls that may run at the same time need a workspace and weights each.  weights must overlap no input.  Results
 * are deterministic.
 * Requires B <= 4096, Hq <= 65535, Hq / Hkv <= 128, T * Hq < 2^31 (WQL_EUNSUPPORTED above).
 * ---------------------------------------------------------------------------------------- */
size_t wql_kv_weights_i4_workspace_bytes(void);
wql_status wql_kv_weights_i4(const uint16_t* q, int64_t q_stride, int T, int Hq, int Hkv, int D,
                             const uint8_t* cache, int64_t pages, int page_size, const int32_t* block_table,
                             int table_width, const int32_t* cu_new, const int32_t* kv_lens, int B, float scale,
                             const float* lse, float* weights, void* workspace, size_t workspace_bytes, void* stream);

/* ----------------------------------------------------------------------------------------
 * kv_evict_i4: leave the least attended tokens behind.  Of the n = kv_lens[b] tokens of sequence b each K/V head
 * keeps n' = min(n, budget): the last min(recent, budget) ones and, of the others, those with the greatest
 * weights[b, h, t] (of equal ones the first; a NaN counts as greater than any number).  They go, in their order, into
 * the pages of row b of new_table [B, new_width], which kv_plan_pages may have planned for n' tokens:
 *     kept [B, H, budget]     the kept tokens' numbers, ascending; -1 from n' on
 *     new_weights [B, H, new_width * page_size]   their weights; 0 from n' on
 *     new_lens [B]            n'
 * and rows 0 .. n' - 1 of the new pages are the kept rows' codes and parameters as they are.  Heads keep tokens of their
 * own choice, so a slot then holds different tokens' rows in different heads; nothing that reads the cache minds.
 * weights is fp32 [B, H, table_width * page_size], dense.  No page of new_table in use may be in use in block_table or
 * twice in new_table: what such a page then holds is unspecified.  Pages that sequences share may be read by all of them.
 * The old pages stay as they are.  A length beyond table_width * page_size is cut there and recorded; rows whose old or
 * new page number is out of range are not moved and recorded.  Nothing may overlap but the cache with itself; new_table,
 * new_weights or new_lens that are block_table, weights or kv_lens are refused.
 * Requires B <= 4096, 1 <= budget <= new_width * page_size, recent >= 0, B * H * max(8, ceil(budget / 16)) <
 * 2^31 (WQL_EUNSUPPORTED above).
 * ---------------------------------------------------------------------------------------- */
wql_status wql_kv_evict_i4(const float* weights, uint8_t* cache, int64_t pages, int page_size, int H, int D,
                           const int32_t* block_table, int table_width, const int32_t* kv_lens, int B,
                           const int32_t* new_table, int new_width, int budget, int recent, int32_t* kept,
                           float* new_weights, int32_t* new_lens, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WQL_H_ */
