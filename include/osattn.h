/*
 * osattn.h - C ABI of libosattn, a fused scaled-dot-product attention forward
 * pass for one NVIDIA GB300 (sm_103a), built on the one-pass online-softmax
 * normaliser, with its backward pass and the standalone row softmax.
 *
 * Sources (cited by page title and section):
 *   [Ch6]  "CUDA 算子工程：手写 FlashAttention v2 之路", chapter 6
 *          "Softmax 与 Online Softmax" (yangyitao.com): the online (m, l)
 *          recurrence (§6.3.1), the guarded combine (§6.4, §6.4.1), LSE
 *          (§6.5), the blocked attention loop (§6.6), the fused additive
 *          mask (§6.7.3).
 *   [XXQK] m.xxqk.cn/news/563265 (article on parallel softmax and
 *          FlashAttention): the attention problem statement (§1.1), the
 *          inner loop with scale and mask and the single final O / l (§4.1),
 *          the causal diagonal-block pitfall (§6.3).
 *
 * Entry points:
 *   forward        osattn_fwd, osattn_fwd_strided (any (b, h, row) strides),
 *                  osattn_fwd_splitkv / _noalloc (key axis split and merged),
 *                  osattn_fwd_offload (host-memory tensors, pipelined copies)
 *   backward       osattn_bwd, osattn_bwd_strided, osattn_bwd_offload
 *   row softmax    osattn_softmax_rows, osattn_softmax_rows_offload
 *   modified scores  osattn_fwd_mod, osattn_bwd_mod (tanh cap, distance slopes
 *                  or a learned bias by distance bucket; shared key/value
 *                  heads), with the masks of osattn_mask_plan (causal, window,
 *                  prefix, packed documents, key lengths)
 *   paged cache    osattn_cache_append (new keys and values into the pages,
 *                  16-bit or 8-bit with scales, rotated on the way),
 *                  osattn_tree_attn and osattn_tree_attn_e4m3 (one token or a
 *                  tree of drafted tokens of every sequence over its pages)
 *   positions      osattn_rotary (rotation of queries and keys, and of their
 *                  gradients)
 *   helpers        workspace sizes, status strings, the device status word,
 *                  the version, and test hooks for the bounded waits
 *
 * Every entry point is callable from C; no C++ or framework types cross it.
 */
#ifndef OSATTN_H
#define OSATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define OSATTN_VERSION 1

/* Element types of Q, K, V and O (LSE is always fp32). */
#define OSATTN_BF16 0 /* bfloat16; runs on the tcgen05 tensor-core kernel */
#define OSATTN_FP32 1 /* float32; runs on the SIMT kernel (full fp32 FMA) */
#define OSATTN_FP16 2 /* IEEE float16; runs on the tcgen05 tensor-core kernel */
/* Element type of the pages of a cache only. */
#define OSATTN_E4M3 3 /* 8-bit floating point (4 exponent, 3 fraction bits, no infinities), with scales */

/* Status codes. */
#define OSATTN_OK 0
#define OSATTN_ERR_INVALID_ARG 1 /* null pointer, size < 1, misalignment, non-finite scale */
#define OSATTN_ERR_UNSUPPORTED 2 /* d or dtype outside the supported set */
#define OSATTN_ERR_CUDA 3        /* a CUDA call failed (launch, attribute, tensor map) */
#define OSATTN_ERR_TIMEOUT 4     /* a device-side wait ran past its limit (reported by
                                    osattn_get_device_status only) */
#define OSATTN_ERR_SCRATCH_LIMIT 5 /* osattn_fwd_splitkv_noalloc: the problem's partials need
                                      more than OSATTN_NOALLOC_SCRATCH_BYTES */

/*
 * osattn_fwd - attention forward with online softmax.
 *
 * Computes, for every batch b < B, head h < H and query row i < Nq,
 *     s_j    = scale * <Q[b,h,i,:], K[b,h,j,:]>                  ([XXQK] §1.1)
 *     J      = { j < min(max(key_len[b], 0), Nkv) and (causal == 0 or j <= i) }
 *     O[b,h,i,:] = sum_{j in J} e^{s_j} V[b,h,j,:] / sum_{j in J} e^{s_j}
 *     LSE[b,h,i] = log sum_{j in J} e^{s_j}        (natural log, [Ch6] §6.5)
 * by streaming K/V tiles with the running row max m and adjusted sum l
 * ([Ch6] §6.3.1, §6.6), rescaling the accumulated O only when m changes and
 * dividing by l once at the end ([XXQK] §4.1).  A row with J empty (keys all
 * masked) gets O = 0 and LSE = -inf, never NaN.
 *
 * Arguments
 *   Q        device, [B, H, Nq, d] contiguous, element type `dtype` (read)
 *   K, V     device, [B, H, Nkv, d] contiguous, element type `dtype` (read)
 *   O        device, [B, H, Nq, d] contiguous, element type `dtype` (written)
 *   LSE      device, [B, H, Nq] contiguous fp32 (written)
 *   B, H, Nq, Nkv   >= 1
 *   d        head dimension: 64 or 128
 *   scale    finite multiplier of the logits (1/sqrt(d) for the usual SDPA)
 *   causal   0: no causal mask; non-zero: key j visible to query i iff j <= i
 *            (top-left aligned, the same index for queries and keys)
 *   key_len  device int32 [B] or NULL; keys j >= key_len[b] are masked
 *            (values are clamped to [0, Nkv]; NULL means Nkv for every b).
 *            Combined with `causal` by logical AND.
 *   dtype    OSATTN_BF16, OSATTN_FP16 (tensor cores, fp32 accumulation,
 *            P rounded to the input type before P.V) or OSATTN_FP32 (SIMT)
 *   stream   cudaStream_t to enqueue on (NULL: the legacy default stream)
 *
 * Layout and alignment: Q, K, V and O must be 16-byte aligned; LSE and
 * key_len 4-byte aligned.  The d axis is fastest, then the sequence axis,
 * then H, then B.  O and LSE must not overlap the inputs.
 *
 * Ownership: all buffers are owned by the caller and stay owned by it.  The
 * call allocates no device memory and keeps no per-call state; it may read
 * device properties and set kernel attributes once per device.
 *
 * Asynchrony and errors: the call validates its arguments on the host, then
 * enqueues the kernel on `stream` and returns.  Results are valid once the
 * stream has reached that point.  The return value covers host validation
 * (OSATTN_ERR_INVALID_ARG / OSATTN_ERR_UNSUPPORTED, nothing enqueued) and
 * launch failures (OSATTN_ERR_CUDA, read with cudaGetLastError, no
 * synchronisation).  Device-side timeouts are reported by
 * osattn_get_device_status.  Nothing is printed and nothing aborts.
 */
int osattn_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE,
               int B, int H, int Nq, int Nkv, int d, float scale, int causal,
               const int32_t* key_len, int dtype, void* stream);

/*
 * osattn_fwd_strided - osattn_fwd on tensors with arbitrary strides, e.g.
 * the [B, N, H, d] layout a fused QKV projection leaves behind, without a
 * transposing copy.  Same computation, masking, results and errors as
 * osattn_fwd.
 *
 *   q_strides, k_strides, v_strides, o_strides
 *            host int64[3] each, or NULL: element strides of the B, H and
 *            sequence axes of Q, K, V and O (the d axis always has stride 1).
 *            NULL means the contiguous [B, H, N, d] layout, so osattn_fwd is
 *            this call with four NULLs.  Each stride must be >= 1, a multiple
 *            of 16 bytes (8 elements for bf16/fp16, 4 for fp32) and below
 *            2^40 bytes; otherwise OSATTN_ERR_INVALID_ARG.  Strides are read
 *            during the call only.  Views may interleave (Q, K and V slices
 *            of one packed tensor); O must not alias any input, and distinct
 *            (b, h, i) of O must not share memory.
 *   LSE      always [B, H, Nq] contiguous fp32.
 */
int osattn_fwd_strided(const void* Q, const void* K, const void* V, void* O, float* LSE,
                       int B, int H, int Nq, int Nkv, int d, const int64_t* q_strides,
                       const int64_t* k_strides, const int64_t* v_strides,
                       const int64_t* o_strides, float scale, int causal,
                       const int32_t* key_len, int dtype, void* stream);

/*
 * osattn_fwd_offload - osattn_fwd for inputs and outputs that live in host
 * memory: copies Q, K, V in, runs the forward pass and copies O and LSE out,
 * pipelined over chunks of heads so that the copy of one chunk in, the
 * attention of the previous one and the copy out of the one before that
 * overlap (one host-to-device and one device-to-host stream of the
 * library's; the chunks' attention launches alternate between `stream` and
 * a compute stream of the library's, so that one chunk's launch starts on
 * the SMs the end of the previous one leaves idle).  Same result as
 * osattn_fwd on the copied data.
 *
 *   Q_host, K_host, V_host   host, contiguous [B, H, N, d] (read); pinned
 *                            (page-locked) memory for the copies to overlap
 *   O_host, LSE_host         host, contiguous [B, H, Nq, d] / [B, H, Nq] (written)
 *   Q, K, V, O, LSE          device buffers of the same shapes (overwritten;
 *                            used as staging, and hold the inputs and outputs
 *                            afterwards); alignment as for osattn_fwd
 *   B .. dtype               as for osattn_fwd (key_len is a device array)
 *   heads_per_chunk          heads per pipeline chunk, within one batch entry
 *                            (larger than H: one chunk per batch entry); 0
 *                            picks enough heads for one wave of CTAs per
 *                            chunk; negative -> OSATTN_ERR_INVALID_ARG
 *   stream                   the copies wait for work enqueued on `stream`
 *                            before the call, and `stream` completes only
 *                            after the last copy out: synchronize `stream`
 *                            (or wait on an event recorded on it) before
 *                            reading O_host and LSE_host
 *
 * Errors as for osattn_fwd (a null host pointer is OSATTN_ERR_INVALID_ARG).
 * Calls from several host threads are serialised while they enqueue.
 */
int osattn_fwd_offload(const void* Q_host, const void* K_host, const void* V_host, void* O_host,
                       float* LSE_host, void* Q, void* K, void* V, void* O, float* LSE, int B,
                       int H, int Nq, int Nkv, int d, float scale, int causal,
                       const int32_t* key_len, int dtype, int heads_per_chunk, void* stream);

/* Largest num_splits osattn_fwd_splitkv accepts. */
#define OSATTN_MAX_SPLITS 128

/*
 * osattn_splitkv_workspace_bytes - device workspace osattn_fwd_splitkv needs:
 * num_splits * B*H*Nq * (d + 1) fp32 values (a normalised partial O row and
 * its partial LSE per key range).  Returns 0 for sizes < 1.
 */
size_t osattn_splitkv_workspace_bytes(int B, int H, int Nq, int d, int num_splits);

/*
 * osattn_fwd_splitkv - the same result as osattn_fwd (same arguments,
 * layouts, masking and fully-masked-row rule), computed with the key axis
 * cut into num_splits ranges so that few (b, h) rows with long key sequences
 * still fill the GPU.
 *
 * Each CTA runs the online-softmax loop over one key range and writes a
 * partial O_s = O / l_s (fp32) and lse_s = m_s + ln l_s; a second kernel
 * folds the partials of every row with the guarded (m, l) combine of [Ch6]
 * §6.4.1 - the two-stage reduction [Ch6] §6.7.1 describes for a row split
 * across blocks - and writes O and LSE.  A key range with no visible
 * key contributes the (-inf, 0) identity.
 *
 *   dtype            OSATTN_BF16 or OSATTN_FP16 (OSATTN_FP32 -> OSATTN_ERR_UNSUPPORTED);
 *                    O is written in that type
 *   num_splits       1 .. OSATTN_MAX_SPLITS (else OSATTN_ERR_INVALID_ARG); ranges are
 *                    equal cuts of each 256-row query block's 128-key tiles, so
 *                    splits beyond the tile count receive empty ranges
 *   workspace        caller-owned device memory, 16-byte aligned, at least
 *                    osattn_splitkv_workspace_bytes(B, H, Nq, d, num_splits) bytes
 *                    (else OSATTN_ERR_INVALID_ARG); overwritten by the call and
 *                    free for other use once the stream passes it
 *
 * Both kernels are enqueued on `stream`; the call allocates nothing.
 * Errors as for osattn_fwd.
 */
int osattn_fwd_splitkv(const void* Q, const void* K, const void* V, void* O, float* LSE,
                       int B, int H, int Nq, int Nkv, int d, float scale, int causal,
                       const int32_t* key_len, int dtype, int num_splits, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Size of the scratch array built into the library for
 * osattn_fwd_splitkv_noalloc (32 MiB on every GPU that loads the library). */
#define OSATTN_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)

/*
 * osattn_fwd_splitkv_noalloc - osattn_fwd_splitkv without a caller-provided
 * workspace, for callers that cannot allocate device memory: an application
 * whose own memory manager owns the device budget and forbids other
 * allocations, or a latency-critical path that cannot pay for cudaMalloc's
 * implicit synchronisation.  (The pages have no counterpart; this is an
 * interface convenience, not part of the method.)
 *
 * Same arguments, results and errors as osattn_fwd_splitkv, minus the
 * workspace: the partial results go to a fixed array of
 * OSATTN_NOALLOC_SCRATCH_BYTES compiled into the library.  A problem with
 * osattn_splitkv_workspace_bytes(B, H, Nq, d, num_splits) greater than that
 * is rejected with OSATTN_ERR_SCRATCH_LIMIT before anything is enqueued;
 * use fewer splits, or osattn_fwd_splitkv with your own workspace.
 *
 * Arguments are checked first, with the statuses osattn_fwd_splitkv
 * returns; OSATTN_ERR_SCRATCH_LIMIT only follows for valid arguments.
 *
 * The call allocates nothing.  Its first call on a device looks up that
 * device's copy of the array (cudaGetSymbolAddress, with the device
 * current) and keeps the address; make that first call before any stream
 * capture.  The address belongs to the runtime's primary context: the entry
 * point assumes the caller uses that context and does not reset the device
 * (cudaDeviceReset) between calls.  Every call on a device shares the one
 * array and leaves its contents behind; a successful call writes every
 * partial it reads, so nothing in it has to start at zero.  After
 * osattn_get_device_status reports OSATTN_ERR_TIMEOUT, O and LSE of the
 * calls since the last status read may hold data left in the array by
 * earlier calls: discard them.  Calls whose kernels can overlap on the GPU
 * (for example on two streams without ordering between them) race on the
 * array and give undefined results: order them on one stream or with events.
 */
int osattn_fwd_splitkv_noalloc(const void* Q, const void* K, const void* V, void* O,
                               float* LSE, int B, int H, int Nq, int Nkv, int d, float scale,
                               int causal, const int32_t* key_len, int dtype, int num_splits,
                               void* stream);

/*
 * osattn_bwd_workspace_bytes - device workspace osattn_bwd needs: one fp32
 * per query row (B*H*Nq floats).  Returns 0 for sizes < 1.
 */
size_t osattn_bwd_workspace_bytes(int B, int H, int Nq);

/*
 * osattn_bwd - gradients of osattn_fwd for an upstream gradient dO.
 *
 * With P_ij = e^{s_ij - LSE_i} on the visible keys J_i (s, J and LSE exactly
 * as in osattn_fwd; the forward pass keeps LSE per row so that the backward
 * pass can rebuild P, [Ch6] §6.5, recomputing the scores, [XXQK] §5.2):
 *     D_i   = <dO_i, O_i>
 *     dS_ij = P_ij (<dO_i, V_j> - D_i)
 *     dQ_i  = scale * sum_j dS_ij K_j
 *     dK_j  = scale * sum_i dS_ij Q_i
 *     dV_j  = sum_i P_ij dO_i
 * (the chain rule on the forward definition).  Rows with J empty contribute
 * nothing; keys no row sees get dK = dV = 0.
 *
 *   Q, K, V   device, as for osattn_fwd (contiguous [B, H, N, d]) (read)
 *   O, LSE    device, the outputs of osattn_fwd for these Q, K, V, scale,
 *             causal and key_len (read)
 *   dO        device, [B, H, Nq, d] contiguous, element type `dtype` (read)
 *   dQ        device, [B, H, Nq, d] contiguous, element type `dtype` (written)
 *   dK, dV    device, [B, H, Nkv, d] contiguous, element type `dtype` (written)
 *   B .. key_len   as for osattn_fwd
 *   dtype     OSATTN_BF16, OSATTN_FP16 (tensor cores: P and dS rounded to the
 *             input type for the products, fp32 accumulation) or OSATTN_FP32
 *             (SIMT FMAs and expf throughout, for the fp32 forward)
 *   workspace caller-owned device memory, 16-byte aligned, at least
 *             osattn_bwd_workspace_bytes(B, H, Nq) bytes (else
 *             OSATTN_ERR_INVALID_ARG); overwritten, free once the stream
 *             passes the call
 *
 * dO, dQ, dK, dV must be 16-byte aligned and must not overlap each other or
 * the inputs.  Three kernels are enqueued on `stream` (D, then dK/dV, then
 * dQ); each output element is written by one CTA (one thread for fp32), so
 * the results do not depend on scheduling.  The call allocates nothing.  Errors as for
 * osattn_fwd.
 */
int osattn_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
               const float* LSE, void* dQ, void* dK, void* dV, int B, int H, int Nq, int Nkv,
               int d, float scale, int causal, const int32_t* key_len, int dtype,
               void* workspace, size_t workspace_bytes, void* stream);

/*
 * osattn_bwd_offload - osattn_bwd for tensors that live in host memory:
 * copies Q, K, V, O, dO and LSE in, computes the gradients and copies dQ,
 * dK and dV out, pipelined over chunks of heads as osattn_fwd_offload
 * (when Nq is not a multiple of 4 every chunk's kernels run on `stream`:
 * the chunks then share the start of the workspace).  Same results as
 * osattn_bwd on the copied data.
 *
 *   *_host     host, contiguous (Q, O, dO, dQ [B, H, Nq, d]; K, V, dK, dV
 *              [B, H, Nkv, d]; LSE [B, H, Nq] fp32); inputs read, dQ_host,
 *              dK_host, dV_host written; pinned memory for the copies to
 *              overlap the compute
 *   Q .. dV    device buffers of the same shapes (overwritten staging)
 *   B .. dtype, workspace, workspace_bytes   as for osattn_bwd
 *   heads_per_chunk   as for osattn_fwd_offload (0: two waves of dK/dV
 *              CTAs per chunk)
 *   stream     as for osattn_fwd_offload
 *
 * Errors as for osattn_bwd (a null host pointer is OSATTN_ERR_INVALID_ARG).
 */
int osattn_bwd_offload(const void* Q_host, const void* K_host, const void* V_host,
                       const void* O_host, const void* dO_host, const float* LSE_host,
                       void* dQ_host, void* dK_host, void* dV_host, void* Q, void* K, void* V,
                       void* O, void* dO, float* LSE, void* dQ, void* dK, void* dV, int B, int H,
                       int Nq, int Nkv, int d, float scale, int causal, const int32_t* key_len,
                       int dtype, void* workspace, size_t workspace_bytes, int heads_per_chunk,
                       void* stream);

/*
 * osattn_bwd_strided - osattn_bwd on tensors with arbitrary strides (e.g.
 * the [B, N, H, d] layout), without transposing copies.  Same computation,
 * results and errors as osattn_bwd.
 *
 *   q_strides .. dv_strides
 *            host int64[3] each, or NULL: element strides of the B, H and
 *            sequence axes of Q, K, V, O, dO, dQ, dK and dV (the d axis
 *            always has stride 1; NULL means the contiguous [B, H, N, d]
 *            layout, so osattn_bwd is this call with eight NULLs).  Each
 *            stride must be >= 1, a multiple of 16 bytes (8 elements) and
 *            below 2^40 bytes; otherwise OSATTN_ERR_INVALID_ARG.  Read during
 *            the call only.  Distinct rows of dQ, dK and dV must not share
 *            memory, and the outputs must not overlap the inputs.
 *   LSE      always [B, H, Nq] contiguous fp32.
 */
int osattn_bwd_strided(const void* Q, const void* K, const void* V, const void* O,
                       const void* dO, const float* LSE, void* dQ, void* dK, void* dV, int B,
                       int H, int Nq, int Nkv, int d, const int64_t* q_strides,
                       const int64_t* k_strides, const int64_t* v_strides,
                       const int64_t* o_strides, const int64_t* do_strides,
                       const int64_t* dq_strides, const int64_t* dk_strides,
                       const int64_t* dv_strides, float scale, int causal,
                       const int32_t* key_len, int dtype, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * osattn_softmax_rows - row softmax of a [rows, N] matrix with the online
 * (m, l) normaliser of [Ch6] §6.4: per row,
 *     y_i = e^{x_i - m} / l,  m = max_i x_i,  l = sum_i e^{x_i - m},
 *     LSE = m + ln l                                          ([Ch6] §6.5)
 * with per-thread states merged by the guarded combine of [Ch6] §6.4.1.
 * Rows of up to 32768 elements are held in registers: read once and written
 * once; longer rows are read twice.  -inf entries act as the additive mask
 * of [Ch6] §6.7.3; a row of only -inf gives y = 0 and LSE = -inf (no NaN).
 *
 *   in, out  device, [rows, N] contiguous, element type `dtype` (bf16, fp16
 *            or fp32);
 *            element-aligned; in == out (in place) is allowed
 *   lse      device fp32 [rows], or NULL to skip it
 *   rows, N  >= 1
 *   stream   cudaStream_t (NULL: legacy default stream)
 * Errors: OSATTN_ERR_INVALID_ARG (null/size/alignment), OSATTN_ERR_UNSUPPORTED
 * (dtype), OSATTN_ERR_CUDA (launch).  Asynchronous like osattn_fwd.
 */
int osattn_softmax_rows(const void* in, void* out, float* lse, int64_t rows, int N, int dtype,
                        void* stream);

/*
 * osattn_softmax_rows_offload - osattn_softmax_rows for a matrix in host
 * memory: copies it in, normalises and copies y (and LSE) out, pipelined
 * over chunks of rows as osattn_fwd_offload does over heads.  Same result as
 * osattn_softmax_rows on the copied data.
 *
 *   in_host    host, [rows, N] row-major, element type `dtype` (read); pinned
 *              memory for the copies to overlap
 *   out_host   host, [rows, N] (written)
 *   lse_host   host fp32 [rows] (written) or NULL; NULL exactly when `lse` is
 *   in, out, lse   device buffers of the same shapes (overwritten staging)
 *   rows_per_chunk   rows per pipeline chunk; 0 picks 16 chunks; negative ->
 *              OSATTN_ERR_INVALID_ARG
 *   stream     as for osattn_fwd_offload
 *
 * Errors as for osattn_softmax_rows (null host pointers, or lse_host and lse
 * not both given or both NULL: OSATTN_ERR_INVALID_ARG; rows above 2^31 - 1:
 * OSATTN_ERR_INVALID_ARG).
 */
int osattn_softmax_rows_offload(const void* in_host, void* out_host, float* lse_host, void* in,
                                void* out, float* lse, int64_t rows, int N, int dtype,
                                int64_t rows_per_chunk, void* stream);

/* Static, human-readable text for a status code (never NULL). */
const char* osattn_status_string(int status);

/*
 * osattn_get_device_status - synchronises `stream`, then returns and clears
 * the device status word of the current device: OSATTN_OK, or
 * OSATTN_ERR_TIMEOUT if a kernel's bounded wait on an mbarrier ran past its
 * limit since the last call (that kernel returned early; its outputs are
 * undefined).  Returns OSATTN_ERR_CUDA if the synchronisation itself fails.
 * Every device-side wait in libosattn is bounded; none traps.
 */
int osattn_get_device_status(void* stream);

/* OSATTN_VERSION of the built library. */
int osattn_version(void);

/*
 * Test hooks (no counterpart on the pages; they exist so the failure path can
 * be exercised without faulting a GPU).
 *
 * osattn_set_wait_limit_ns - sets the time limit (nanoseconds, >= 1000) that
 *   every device-side wait of later launches on any device uses; returns the
 *   previous limit.  Default 4e9 (4 s).  Values below 1000 are clamped.
 * osattn_test_wait_timeout - enqueues a one-warp kernel that waits on an
 *   mbarrier nobody arrives on, with the current limit; the wait gives up,
 *   records OSATTN_ERR_TIMEOUT in the status word and the kernel returns.
 *   Returns OSATTN_OK or OSATTN_ERR_CUDA (launch failure).
 */
uint64_t osattn_set_wait_limit_ns(uint64_t ns);
int osattn_test_wait_timeout(void* stream);

/* Site code of the first wait that gave up, as read by the most recent
 * osattn_get_device_status call that returned OSATTN_ERR_TIMEOUT (0 if none).
 * Codes identify the waiting role (producer, MMA issuer, softmax, epilogue). */
int osattn_last_timeout_site(void);

/*
 * osattn_step_trace_read - profiling hook (no counterpart in the method).
 * A library built with OSATTN_STEP_TRACE=1 (a separate profiling build,
 * never the product) records SM clock stamps at the phases of every K/V
 * step of the first 8 CTAs of each bf16/fp16 forward launch: long long
 * [8 CTAs][7 roles][128 steps][4 stamps]; role 0/1 = softmax of query tile
 * 0/1, its first warp (S seen, S in registers, alpha published, P
 * published); role 2 = MMA warp (K/V seen, P of tile 0 seen, P of tile 1
 * seen, step issued); role 3/4 = P published by each of the four softmax
 * warps of tile 0/1; role 5/6 = correction of tile 0/1, its first warp
 * (alpha seen, O rescaled, arrived, and 1 if the warp rescaled O - a flag,
 * not a clock).  Then long long [4096 CTAs][6] for the first 4096 CTAs of
 * the last launch: global-timer nanoseconds at start, end of setup, first S
 * seen, epilogue start (tile 0) and end, and the SM it ran on.
 * Copies them to `host` (bytes >= *needed) after the stream has
 * synchronised.  *needed (if not NULL) gets the size.  Returns OSATTN_OK,
 * OSATTN_ERR_INVALID_ARG (buffer too small) or, in a product build,
 * OSATTN_ERR_UNSUPPORTED.
 */
int osattn_step_trace_read(void* host, size_t bytes, size_t* needed);

/* ------------------------------------------------------- modified scores */

/*
 * osattn_mask_plan - the keys that each query row sees, as one interval a
 * row, for osattn_fwd_mod and osattn_bwd_mod.  A plan depends on the masks
 * only, so one plan serves every layer and both passes of a step.
 *
 * Query row i of batch entry b stands at position p = i + q_offset among the
 * keys.  Key j < Nkv is visible to it iff all of these hold:
 *   j < min(max(key_len[b], 0), Nkv)            (key_len not NULL)
 *   j <= p, or j < prefix_len[b]                (causal; prefix_len may be NULL)
 *   |j - p| < window                            (window > 0)
 *   j and p lie in one document                 (doc_ids not NULL)
 * A document is a run of equal, non-negative ids in doc_ids[b][0 .. Nkv): the
 * same id again after another one is another document, and positions with a
 * negative id, or outside [0, Nkv), see nothing.
 *
 *   plan       device, 16-byte aligned, osattn_mask_plan_bytes(B, Nq) bytes
 *              (written).  Its content is private to the library.
 *   B, Nq, Nkv >= 1; Nq, Nkv <= 2^30;  |q_offset| <= 2^30
 *   window     0: none
 *   key_len, prefix_len   device int32 [B] or NULL; prefix_len needs causal
 *   doc_ids    device int32 [B, Nkv] contiguous, or NULL
 * Enqueued on `stream`; errors as for osattn_fwd.
 */
size_t osattn_mask_plan_bytes(int B, int Nq);
int osattn_mask_plan(void* plan, size_t plan_bytes, int B, int Nq, int Nkv, int q_offset,
                     int causal, int window, const int32_t* key_len, const int32_t* prefix_len,
                     const int32_t* doc_ids, void* stream);

/*
 * What happens to a scaled score before the softmax.  For query row i, with
 * p = i + q_offset, and key j:
 *   y = scale * <Q[b,h,i,:], K[b,h/(H/Hkv),j,:]>
 *   y = softcap * tanh(y / softcap)                         (softcap > 0)
 *   y = y - slopes[h] * |j - p|                             (slopes), or
 *   y = y + rel_table[rel_map[clamp(j - p, -R, R) + R]][h]  (rel_table), R = rel_range
 * slopes and rel_table exclude each other (OSATTN_ERR_INVALID_ARG); softcap
 * with rel_table is OSATTN_ERR_UNSUPPORTED.  Capped scores are computed to
 * 2^-20 softcap, and to 2^-22 relative where all scores around them (those of
 * 32 rows and a tile of keys) are below 0.4 softcap (osattn_tree_attn: with
 * softcap above 64).  Slopes are applied in fp32, those up to 1 in magnitude
 * with an error of up to 5e-5 of the slope in a logit.
 */
typedef struct osattn_score {
  float softcap;          /* 0: no cap; else 0.001 .. 10000 (others: OSATTN_ERR_INVALID_ARG) */
  const float* slopes;    /* device fp32 [H] or NULL */
  const void* rel_table;  /* device [rel_num, H] contiguous, element type `dtype`, or NULL */
  const int32_t* rel_map; /* device int32 [2 R + 1]: bucket of each distance -R .. R; an entry
                             outside [0, rel_num) adds nothing and has no gradient */
  int rel_num;            /* >= 1 */
  int rel_range;          /* R: 1 .. 1024 (more: OSATTN_ERR_UNSUPPORTED) */
  int q_offset;           /* position of query row 0, the one the plan was made with */
} osattn_score;

/*
 * osattn_fwd_mod - attention forward with modified scores:
 *     O[b,h,i,:] = sum_j e^{y_j} V[b,h/(H/Hkv),j,:] / sum_j e^{y_j},  LSE = log sum_j e^{y_j}
 * over the keys j that the plan lets row i see.  A row that sees none gets
 * O = 0 and LSE = -inf.
 *
 *   Q, O    device [B, H, Nq, d], K, V  device [B, Hkv, Nkv, d], with element
 *           strides as for osattn_fwd_strided (NULL: contiguous); Hkv divides
 *           H, and query heads h with the same h / (H / Hkv) share a key head
 *   LSE     device fp32 [B, H, Nq] contiguous (written)
 *   scale   finite;  score  NULL: y is the scaled score
 *   plan    from osattn_mask_plan for the same B, Nq, Nkv and q_offset, or
 *           NULL: every row sees every key
 *   dtype   OSATTN_BF16 or OSATTN_FP16 (fp32: OSATTN_ERR_UNSUPPORTED);
 *           products accumulate in fp32, P is rounded to dtype before P V
 *   d       64 or 128
 * K and V may hold anything (NaN included) at keys before the first and
 * behind the last key that a block of 256 query rows (rows 256 n ..) sees;
 * within that range a non-finite V row reaches all rows of the block.
 * The sums of P V before the division by the row's sum are finite for V up to
 * 2^56 in magnitude.
 * Alignment, ownership, asynchrony and errors as for osattn_fwd_strided.
 */
int osattn_fwd_mod(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
                   int Hkv, int Nq, int Nkv, int d, const int64_t* q_strides,
                   const int64_t* k_strides, const int64_t* v_strides, const int64_t* o_strides,
                   float scale, const osattn_score* score, const void* plan, int dtype,
                   void* stream);

/*
 * osattn_bwd_mod - gradients of osattn_fwd_mod from its O and LSE and the
 * upstream gradient dO: dQ, dK, dV (dK and dV summed over the query heads
 * that share a key head) and, with a rel_table, its gradient
 *     dRel[k][h] = sum over b and the visible pairs of bucket k of dy.
 * slopes get no gradient.  Rows that see no key, and keys that no row sees,
 * get zeros, whatever Q, dO, K and V hold there (K and V under the rule of
 * osattn_fwd_mod; a non-finite Q or dO row that sees a key reaches dK and dV
 * of the whole 128-key tile).  dQ takes D = rowsum(dO O) with O as given, in 16
 * bits; without a cap dK and dRel take it corrected by the row's sum of dy, which
 * is 0 for the O and LSE of all keys that the row sees (an LSE over more keys
 * than the call's would make them wrong).  No atomics: the same call gives the
 * same bits.
 *
 *   dRel       device [rel_num, H], element type `dtype` (written), exactly
 *              when score->rel_table is given, else NULL
 *   workspace  device, 16-byte aligned, osattn_bwd_mod_workspace_bytes(B, H,
 *              Nq, Nkv, rel_range or 0 without a rel_table) bytes
 * The other arguments as for osattn_fwd_mod; errors likewise.
 */
size_t osattn_bwd_mod_workspace_bytes(int B, int H, int Nq, int Nkv, int rel_range);
int osattn_bwd_mod(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                   const float* LSE, void* dQ, void* dK, void* dV, void* dRel, int B, int H,
                   int Hkv, int Nq, int Nkv, int d, const int64_t* q_strides,
                   const int64_t* k_strides, const int64_t* v_strides, const int64_t* o_strides,
                   const int64_t* do_strides, const int64_t* dq_strides,
                   const int64_t* dk_strides, const int64_t* dv_strides, float scale,
                   const osattn_score* score, const void* plan, int dtype, void* workspace,
                   size_t workspace_bytes, void* stream);

/* ----------------------------------------------------------- paged cache */

/*
 * osattn_tree_attn - T drafted tokens of every sequence attend to the
 * sequence's paged cache and to the drafts on their own line; T = 1 is the
 * ordinary decode step.
 *
 * Sequence b has ctx_len[b] cached keys; the drafts' own keys and values
 * follow them in the same pages, at positions ctx_len[b] .. + T - 1 (the
 * caller has written them).  The key at position x is row x mod page_size of
 * page page_table[b][x / page_size].  Bit u of tree_mask[b][t] says that
 * draft t sees draft u (for a tree: its ancestors and itself; bits from T on
 * say nothing); tree_mask NULL is the chain u <= t.  A draft whose mask is 0
 * is padding: it sees nothing and gets O = 0, LSE = -inf.  Otherwise it sees
 * the whole context besides.
 *
 * Positions, for the window and the slopes: a cached key stands at its index,
 * draft t at ctx_len[b] + (bits of its mask) - 1 (padding too, for a draft that
 * sees it).  With y the scaled score, capped as in osattn_score, and dist =
 * |position of the query less that of the key|:
 *   y = y - slopes[h] * dist;  key visible only if dist < window (window > 0)
 * O and LSE as for osattn_fwd_mod, head h reading key head h / (H / Hkv).
 *
 *   Q, O       device [B, H, T, d] with element strides as for
 *              osattn_fwd_strided (NULL: contiguous)
 *   K_pages, V_pages   device [num_pages, Hkv, page_size, d], strides of the
 *              page, head and row axes likewise
 *   page_table device int32 [B, max_pages]; only the entries of pages that
 *              hold a visible key are used.  Such an entry outside
 *              [0, num_pages) reads as zeros, and osattn_get_device_status
 *              then returns OSATTN_ERR_INVALID_ARG
 *   ctx_len    device int32 [B], 0 .. max_pages * page_size - T (values
 *              outside are clamped, with the same status)
 *   tree_mask  device int64 [B, T] or NULL
 *   LSE        device fp32 [B, H, T] contiguous
 *   T          1 .. 64, H / Hkv <= 128, d 64 or 128, bf16 or fp16 (else
 *              OSATTN_ERR_UNSUPPORTED); max_pages * page_size in T .. 2^30
 *   page_size  a divisor of 128 from 8 on, or a multiple of 128 (else
 *              OSATTN_ERR_UNSUPPORTED)
 *   workspace  device, 16-byte aligned, osattn_tree_workspace_bytes(...)
 *              bytes; holds nothing between calls
 * Pages may hold anything (NaN included) at positions that no draft sees.
 * No atomics on results: the same call gives the same bits.  Alignment,
 * ownership, asynchrony and errors as for osattn_fwd_strided.
 */
size_t osattn_tree_workspace_bytes(int B, int H, int Hkv, int T, int d);
int osattn_tree_attn(const void* Q, const void* K_pages, const void* V_pages,
                     const int32_t* page_table, const int32_t* ctx_len, const int64_t* tree_mask,
                     void* O, float* LSE, int B, int H, int Hkv, int T, int d, int num_pages,
                     int page_size, int max_pages, const int64_t* q_strides,
                     const int64_t* k_strides, const int64_t* v_strides, const int64_t* o_strides,
                     float scale, float softcap, const float* slopes, int window, int dtype,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * osattn_tree_attn_e4m3 - osattn_tree_attn over pages of e4m3 values, one fp32
 * scale for each block of scale_block tokens of a page and key head.  A step of few
 * query rows a key head takes half the time of 16-bit pages over long contexts;
 * trees of 17 rows and more take up to a third longer than there, for half the
 * memory.  The key at
 * row r of a page is K_scale[page][head][r / scale_block] times the values of
 * K_pages there, and likewise V.  Everything else is as for osattn_tree_attn:
 * masks, positions, window, cap, slopes, shared heads, pages that do not exist.
 *
 *   K_pages, V_pages   device [num_pages, Hkv, page_size, d] of bytes, strides
 *              of the page, head and row axes in elements, multiples of 16
 *   K_scale, V_scale   device fp32 [num_pages, Hkv, page_size / scale_block]
 *              contiguous, finite where a draft sees a key, and V_scale not
 *              negative (below 2^-100 it counts as that; above 2^112 the sums
 *              of weights lose bits)
 *   scale_block   a divisor of page_size
 *   dtype      of Q and O: OSATTN_BF16 or OSATTN_FP16
 *   workspace  osattn_tree_e4m3_workspace_bytes(...) bytes
 * Pages and scales may hold anything (NaN included) at positions that no draft
 * sees.  Of the weights of V, probabilities times V_scale, those below 2^-34 of the
 * greatest of a CTA's part of a row (2^-26 with more than 16 query rows T H / Hkv
 * and blocks of 8 tokens or more) may count in LSE and not in O: with N keys there
 * O is off by at most N times that of max |V|.  Those below 2^-136 count in neither.
 */
size_t osattn_tree_e4m3_workspace_bytes(int B, int H, int Hkv, int T, int d);
int osattn_tree_attn_e4m3(const void* Q, const void* K_pages, const void* V_pages,
                          const float* K_scale, const float* V_scale, const int32_t* page_table,
                          const int32_t* ctx_len, const int64_t* tree_mask, void* O, float* LSE,
                          int B, int H, int Hkv, int T, int d, int num_pages, int page_size,
                          int max_pages, int scale_block, const int64_t* q_strides,
                          const int64_t* k_strides, const int64_t* v_strides,
                          const int64_t* o_strides, float scale, float softcap,
                          const float* slopes, int window, int dtype, void* workspace,
                          size_t workspace_bytes, void* stream);

/* ------------------------------------------------------- rotary positions */

/* How rows turn with their position p: pair i of a row's first `rot` elements,
 * (a, b), becomes
 *     amplitude (a cos t - b sin t),  amplitude (a sin t + b cos t),  t = p freqs[i];
 * the elements from `rot` on stay.  t is exact to p freqs[i] 2^-52 and 2^-24
 * besides, for any 32-bit p. */
typedef struct osattn_rotation {
  const double* freqs; /* device fp64 [rot / 2]: radians a position */
  int rot;             /* even, 2 .. d */
  int interleaved;     /* 0: pairs (i, rot / 2 + i); else (2 i, 2 i + 1) */
  float amplitude;     /* finite; 1 for a plain rotation */
} osattn_rotation;

/*
 * osattn_rotary - rotates the rows of Q and K by their positions; with
 * `inverse` by the negative angles, which is the gradient: dQ = rotary of dQ_out,
 * amplitude included.
 *
 *   Q, Q_out   device [B, H, N, d] with (b, h, row) element strides (NULL:
 *              contiguous); those of Q may be 0, those of Q_out at least 1 where
 *              the axis is longer than 1; Q_out may be Q with the same strides
 *              (with others it is refused)
 *   K, K_out   device [B, Hkv, N, d] likewise; Hkv = 0: none
 *   positions  device int32 [N], or [B, N] with batch_positions, or NULL: row n
 *              stands at offset + n
 *   d          2 .. 512;  dtype  OSATTN_BF16, OSATTN_FP16 or OSATTN_FP32
 * Rotated in fp32 and rounded once.  Elements, strides and rot / 2 that allow it
 * (multiples of 16 bytes) are taken 16 bytes at a time, others 8, 4 or 2.
 * Ownership, asynchrony and errors as for osattn_fwd_strided.
 */
int osattn_rotary(const void* Q, const void* K, void* Q_out, void* K_out, int B, int H, int Hkv,
                  int N, int d, const int64_t* q_strides, const int64_t* k_strides,
                  const int64_t* qo_strides, const int64_t* ko_strides,
                  const osattn_rotation* rotation, const int32_t* positions, int batch_positions,
                  int offset, int inverse, int dtype, void* stream);

/*
 * osattn_cache_append - writes the keys and values of T new tokens of every
 * sequence into its pages, at places ctx_len[b] .. ctx_len[b] + n - 1 with
 * n = new_len[b] (clamped to 0 .. T; NULL: T); rows t >= n are padding and write
 * nothing.  With a rotation K is rotated on the way, and Q into Q_out.
 *
 *   K, V       device [B, Hkv, T, d], element type `dtype`, strides as for
 *              osattn_fwd_strided
 *   Q, Q_out   device [B, H, T, d] likewise, or both NULL; needs a rotation; all
 *              T rows are written.  Q_out may be Q with the same strides (with others
 *              it is refused)
 *   positions  device int32 [B, T] for the rotation (a tree's drafts stand at
 *              their depths), or NULL: ctx_len[b] + t
 *   K_pages, V_pages, page_table   as for osattn_tree_attn, cache_dtype being
 *              `dtype`, or as for osattn_tree_attn_e4m3 with OSATTN_E4M3
 *   K_scale, V_scale, scale_block   as there (cache_dtype OSATTN_E4M3), written
 *   d          64 or 128;  dtype  OSATTN_BF16 or OSATTN_FP16
 *
 * e4m3: a block's scale is the least power of two s with every finite magnitude
 * of its new rows at most 448 s (2^-100 for zeros), and values are rounded once,
 * from fp32; infinities become 448 s, NaN stays.  A block whose first rows are
 * older (places before ctx_len[b]) keeps its scale unless the new rows need a
 * greater one; then its older rows are brought to that, rounded once (to zeros
 * from a scale of 0, with their signs from a negative one).  A scale there that is
 * NaN, infinite, or negative and greater in magnitude than the new rows' leaves
 * the older rows as NaN.  The scale of a block without older rows is not read.
 *
 * Nothing else in the pages is written.  A sequence whose n rows do not fit the
 * table, or a negative ctx_len, or a page outside [0, num_pages), leaves its
 * rows out, and osattn_get_device_status then returns OSATTN_ERR_INVALID_ARG.
 * A page written here belongs to one sequence.  Ownership, asynchrony and
 * errors as for osattn_fwd_strided.
 */
int osattn_cache_append(const void* K, const void* V, const void* Q, void* K_pages, void* V_pages,
                        float* K_scale, float* V_scale, void* Q_out, const int32_t* page_table,
                        const int32_t* ctx_len, const int32_t* new_len, const int32_t* positions,
                        int B, int H, int Hkv, int T, int d, int num_pages, int page_size,
                        int max_pages, int scale_block, const int64_t* k_strides,
                        const int64_t* v_strides, const int64_t* q_strides,
                        const int64_t* kp_strides, const int64_t* vp_strides,
                        const int64_t* qo_strides, const osattn_rotation* rotation, int dtype,
                        int cache_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* OSATTN_H */
