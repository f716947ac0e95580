/*
 * kda.h -- C ABI of the B200 (sm_100a) Kimi Delta Attention (KDA) recurrence library.
 *
 * KDA is a gated delta-rule linear attention with a per-channel forget gate.  Per
 * batch element b and head h it carries a state S in R^{dk x dv} and, for each token t,
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(exp g_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t
 *
 * i.e. decay every row i of the state by exp(g_t[i]), let the decayed memory predict v_t
 * from k_t, write only the residual (scaled by beta_t) back along k_t, then read the
 * updated state with q_t.  Sources:
 *   - "Day 21" course page (ai.air7.fun/decks/k3-course-30/day-21): interview item D19
 *     (fixed-size d x d state, delta-rule residual update, per-channel decay gate),
 *     quiz Q8 (state built from k^T v products, O(1) memory), quiz Q9 (predict with the
 *     old memory, overwrite with the residual v - S k only);
 *   - Kimi K3 skill card (skillsmp.com), quick facts: the log-decay is a lower-bounded
 *     scaled sigmoid with g_min = -5, which keeps the diagonal tiles of the chunked form
 *     dense enough for tensor-core products;
 *   - podcast show-notes (scripod.com), section 2.1: chunk-recurrent form (RetNet) and
 *     gated delta rule (Gated DeltaNet), which this library's prefill follows.
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller (except in
 *     kda_forward_chunked_host, which takes HOST buffers and a caller-owned device
 *     workspace).  The library never allocates, frees or retains caller memory.  It owns one
 *     small static device status word per device (see kda_get_device_status) and the fixed
 *     scratch array of kda_forward_chunked_host_noalloc (KDA_NOALLOC_SCRATCH_BYTES per device).
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy default
 *     stream).  A return of KDA_OK means the work was validated and enqueued.
 *   - Tensors are contiguous, row-major, with the layouts stated per function.
 *   - `dtype` applies to q, k, v, g, beta and o.  The state is always fp32.
 *   - g is the per-channel LOG-decay itself (g <= 0; the gate nonlinearity is the
 *     caller's).  There is no query scaling and no q/k normalisation inside the library.
 *   - Supported sizes: dk, dv in {64, 128}; B, H >= 1; T >= 0 (T == 0 copies S0 to S_T).
 *     Every pointer must be 16-byte aligned.
 *   - Errors: argument checks happen before anything is enqueued and return a negative
 *     kda_status; a failed launch returns KDA_ERR_CUDA.  A device-side wait that runs
 *     out (it never hangs) sets the device status word to KDA_ERR_TIMEOUT, which
 *     kda_get_device_status reports.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* == cudaStream_t's pointee; keeps this header free of CUDA includes */

/* Exported symbols (the library is built with hidden visibility by default). */
#if defined(__GNUC__)
#define KDA_API __attribute__((visibility("default")))
#else
#define KDA_API
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = -1, /* null pointer, non-positive size, aliasing that is not allowed */
    KDA_ERR_UNSUPPORTED = -2, /* dtype or head size the library has no kernel for */
    KDA_ERR_MISALIGNED = -3,  /* a pointer is not 16-byte aligned */
    KDA_ERR_CUDA = -4,        /* a CUDA runtime/driver call failed (launch, attribute, ...) */
    KDA_ERR_TIMEOUT = -5      /* a device-side bounded wait gave up (reported by the status word) */
} kda_status;

typedef enum { KDA_DTYPE_BF16 = 0, KDA_DTYPE_FP32 = 1 } kda_dtype;

/* Prefill kernel selection for kda_forward_chunked_impl. */
typedef enum {
    KDA_IMPL_AUTO = 0,    /* bf16 inputs: the tcgen05 kernel (every supported head size); fp32
                             inputs: the SIMT kernel (the only fp32 kernel: bf16 tensor-core
                             operands cannot meet an fp32 accuracy bar) */
    KDA_IMPL_TCGEN05 = 1, /* chunkwise tensor-core kernel: bf16, dk and dv each 64 or 128.  It
                             always computes 128 x 128 states; a head size of 64 is embedded in
                             them with zero channels (exact), so it costs what 128 does */
    KDA_IMPL_SIMT = 2     /* token-serial fp32 CUDA-core kernel: every supported dtype and size */
} kda_impl;

/*
 * kda_forward_chunked -- prefill: run the recurrence over T tokens for every (b, h).
 *
 * Computes o_t for t = 1..T and the final state S_T, starting from S0 (the chunkwise
 * parallel form with 64-token chunks; exact up to rounding, see the header comment).
 *
 *   q, k, g : [B, T, H, dk]   dtype     (g = log-decay, per channel)
 *   v       : [B, T, H, dv]   dtype
 *   beta    : [B, T, H]       dtype     (write strength, one scalar per token and head)
 *   S0      : [B, H, dk, dv]  fp32, or NULL for a zero initial state
 *   o       : [B, T, H, dv]   dtype     output (bf16 outputs are rounded to nearest even)
 *   S_T     : [B, H, dk, dv]  fp32, or NULL when the final state is not wanted.
 *             S_T may alias S0 exactly (in-place state carry); any other overlap
 *             between outputs and inputs is not allowed.
 *   dtype   : kda_dtype.
 *
 * Kernel: KDA_IMPL_AUTO (see kda_impl): bf16 runs the chunkwise tensor-core kernel, fp32 the
 * fp32 kernel.
 *
 * Returns KDA_OK, or a negative kda_status (nothing is enqueued on error).
 */
KDA_API int kda_forward_chunked(const void* q, const void* k, const void* v, const void* g,
                        const void* beta, const float* S0, void* o, float* S_T, int B, int T,
                        int H, int dk, int dv, int dtype, struct CUstream_st* stream);

/*
 * kda_forward_chunked_impl -- kda_forward_chunked with an explicit kernel choice
 * (kda_impl).  Same arguments, layouts and semantics; returns KDA_ERR_UNSUPPORTED when
 * the requested kernel does not cover the dtype/shape.
 */
KDA_API int kda_forward_chunked_impl(const void* q, const void* k, const void* v, const void* g,
                             const void* beta, const float* S0, void* o, float* S_T, int B,
                             int T, int H, int dk, int dv, int dtype, int impl,
                             struct CUstream_st* stream);

/*
 * kda_forward_chunked_states -- kda_forward_chunked that also writes the state after every
 * `interval` tokens: the boundaries from which a prefix cache resumes the recurrence
 * (podcast show-notes (scripod.com), outline item 5.3.1 "KDA-Aware Prefix Cache Management";
 * the channel post on the K3 report (t.iss.one), online-inference paragraph: prefixes are
 * reused at 512-token boundaries).
 *
 *   S_mid    : [B, H, n_mid, dk, dv] fp32 output, n_mid = T / interval (integer division):
 *              S_mid[b][h][n] is the state after the first (n+1)*interval tokens of (b, h),
 *              the same values a kda_forward_chunked over those tokens returns as S_T.
 *              Must not overlap any other argument.  May be NULL only when n_mid == 0.
 *   interval : a positive multiple of 64 (the prefill's chunk length).
 *   impl     : kda_impl, as for kda_forward_chunked_impl.
 *
 * Every other argument, layout and rule as kda_forward_chunked; o and S_T are the values it
 * would produce.  Returns KDA_ERR_INVALID_ARG for interval <= 0, KDA_ERR_UNSUPPORTED for an
 * interval that is not a multiple of 64.
 */
KDA_API int kda_forward_chunked_states(const void* q, const void* k, const void* v, const void* g,
                               const void* beta, const float* S0, void* o, float* S_T,
                               float* S_mid, int interval, int B, int T, int H, int dk, int dv,
                               int dtype, int impl, struct CUstream_st* stream);

/*
 * kda_forward_chunked_host -- kda_forward_chunked on HOST buffers: the library copies the
 * inputs in, runs the prefill and copies o (and S_T) out.  The work is cut into segments of
 * one batch entry and at most 2048 tokens (a multiple of the 64-token chunk); the state passes
 * from one segment of a sequence to the next in device memory, so o and S_T are bitwise those
 * of kda_forward_chunked on the same values.  Copy-in of the next segment, the kernel of the
 * current one and copy-out of the previous one overlap (two internal streams, created and
 * destroyed by the call, ordered by events with `stream`).
 *
 *   q, k, v, g, beta, S0, o, S_T : layouts, dtypes and NULL rules of kda_forward_chunked, in
 *              HOST memory owned by the caller.  Page-locked memory makes the copies
 *              asynchronous; with pageable memory they are staged and the call blocks the host
 *              thread.  S_T may be S0 itself; no other output may overlap an input.  Inputs
 *              must stay unchanged, and outputs unread, until the work on `stream` completes.
 *   workspace       : DEVICE memory owned by the caller, 16-byte aligned, of at least
 *                     kda_forward_chunked_host_workspace(T, H, dk, dv, dtype) bytes; it must
 *                     not be used by anything else until the work on `stream` completes.
 *   workspace_bytes : its size.
 *   impl            : kda_impl, as for kda_forward_chunked_impl.
 *
 * Asynchronous on `stream`: everything the call enqueues comes after the work already on
 * `stream`, and work enqueued on `stream` afterwards comes after all of it (after the last
 * copy-out).  Returns KDA_OK; KDA_ERR_INVALID_ARG for a missing or too small workspace or a
 * bad size or overlap; KDA_ERR_MISALIGNED for an unaligned workspace; KDA_ERR_UNSUPPORTED as
 * kda_forward_chunked_impl (these checks happen before anything is enqueued); KDA_ERR_CUDA if
 * a stream, event, copy or launch fails part-way (work already enqueued still completes, and
 * `stream` still waits for it).
 */
KDA_API int kda_forward_chunked_host(const void* q, const void* k, const void* v, const void* g,
                             const void* beta, const float* S0, void* o, float* S_T, int B,
                             int T, int H, int dk, int dv, int dtype, void* workspace,
                             size_t workspace_bytes, int impl, struct CUstream_st* stream);

/*
 * kda_forward_chunked_host_workspace -- bytes of device workspace kda_forward_chunked_host
 * needs for sequences of T tokens with H heads (independent of B): two segments' inputs and
 * outputs plus two states.  Returns 0 for an unsupported dtype or head size, H <= 0 or T < 0.
 */
KDA_API size_t kda_forward_chunked_host_workspace(int T, int H, int dk, int dv, int dtype);

/*
 * KDA_NOALLOC_SCRATCH_BYTES -- size of the fixed device scratch array that
 * kda_forward_chunked_host_noalloc stages its work through (32 MiB).  The library reserves it
 * in the device memory of every GPU it is loaded on, when it is loaded, and holds it until the
 * process exits.
 */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)

/*
 * kda_forward_chunked_host_noalloc -- kda_forward_chunked_host for callers that cannot allocate
 * device memory.  (The pages describe no such entry point: it is an interface matter of this
 * library, with no counterpart in the method.)
 *
 * Who needs it: a caller that holds only host arrays and reaches the library through a plain C
 * foreign-function interface, with no CUDA allocator of its own to create the device workspace
 * kda_forward_chunked_host asks for; or an engine whose device memory is all owned by a pool that
 * forbids allocations outside it (and in which a cudaMalloc would also synchronise the device in
 * the middle of its work).  This call allocates nothing, on the device or the host: it calls no
 * cudaMalloc, cudaFree, stream or event creation, or any other allocating routine.  Instead it
 * stages the work through one fixed scratch array of KDA_NOALLOC_SCRATCH_BYTES that the library
 * reserves when it is loaded.
 *
 *   q, k, v, g, beta, S0, o, S_T : HOST buffers, with the layouts, dtypes, NULL rules and overlap
 *              rules of kda_forward_chunked_host (S_T may be S0 itself).  Page-locked memory makes
 *              the copies asynchronous.  With pageable memory the copies are staged by the driver
 *              and the call blocks the host thread.  Inputs must stay unchanged, and outputs unread,
 *              until the work on `stream` completes.
 *   impl     : kda_impl, as for kda_forward_chunked_impl.
 *
 * Every step runs in order on `stream`: the inputs of one segment are copied in, the prefill runs
 * on them, and o (and S_T after a sequence's last segment) is copied out.  A segment is one batch
 * entry and the largest multiple of 64 tokens whose q, k, g, v, beta and o fit the scratch
 * together with one fp32 state [H, dk, dv]: 192 tokens for H = 96 and bf16 d = 128.
 * The state carried between the segments of a sequence stays in fp32 device memory, so o and S_T
 * are bitwise those of kda_forward_chunked_host and kda_forward_chunked on the same values.  There
 * is no overlap of copies with kernels: this entry point trades speed for needing no memory.
 *
 * Maximum size: the state of one batch entry plus 64 tokens of inputs and outputs (T tokens when
 * T < 64) must fit the scratch: 256-byte-rounded H*dk*dv*4 + 3*n*dk*e + 2*n*dv*e + n*e bytes, with
 * n = H * min(T, 64) and e = 2 (bf16) or 4 (fp32).  So H <= 227 at bf16 d = 128 and H <= 146 at
 * fp32 d = 128.  Larger problems return KDA_ERR_UNSUPPORTED before anything is enqueued.
 *
 * Shared scratch: the array is one per device, shared by every call on that device, and it keeps
 * the last call's contents.  Nothing in it needs to start at zero: a sequence without S0 starts
 * from the zero state inside the kernel, and every byte a segment reads is first written by that
 * same segment's copy-in.  Calls whose work overlaps on the GPU (on different streams, or on one
 * stream from different host threads without ordering) race on the scratch and give undefined
 * results: run them in order, on one stream.
 *
 * First call on a device: it looks up the device address of the scratch (cudaGetSymbolAddress,
 * with that device current) and keeps it for later calls.  Make that first call before any
 * stream capture on the device.
 *
 * Returns KDA_OK; KDA_ERR_INVALID_ARG or KDA_ERR_UNSUPPORTED (also: the problem does not fit the
 * scratch, as above) before anything is enqueued, as kda_forward_chunked_host; KDA_ERR_CUDA if the
 * scratch's address cannot be looked up, or if a copy or launch fails part-way (work already
 * enqueued on `stream` still runs).
 */
KDA_API int kda_forward_chunked_host_noalloc(const void* q, const void* k, const void* v, const void* g,
                                             const void* beta, const float* S0, void* o, float* S_T, int B,
                                             int T, int H, int dk, int dv, int dtype, int impl,
                                             struct CUstream_st* stream);

/*
 * kda_decode_step -- one token for every (b, h), state updated in place.
 *
 * Same recurrence with T = 1 (the memory-bound state read-modify-write of decoding):
 *   S <- Diag(exp g) S;  u = beta (v - S^T k);  S <- S + k u^T;  o = S^T q.
 *
 *   q, k, g : [B, H, dk]      dtype
 *   v       : [B, H, dv]      dtype
 *   beta    : [B, H]          dtype
 *   S       : [B, H, dk, dv]  fp32, read and written in place (must not be NULL)
 *   o       : [B, H, dv]      dtype output
 *
 * Returns KDA_OK or a negative kda_status (nothing is enqueued on error).
 */
KDA_API int kda_decode_step(const void* q, const void* k, const void* v, const void* g,
                    const void* beta, float* S, void* o, int B, int H, int dk, int dv,
                    int dtype, struct CUstream_st* stream);

/*
 * kda_forward_chunked_fused -- kda_forward_chunked with the gate and normalisation prologue fused
 * into the kernels' load stage, so no separate elementwise pass over q, k, g and beta is needed:
 *
 *   g    = -5 * sigmoid(z_g)           per channel (the bounded scaled-sigmoid log-decay with
 *                                      lower bound -5: Kimi K3 skill card (skillsmp.com), quick facts)
 *   beta = sigmoid(z_beta)             per token and head
 *   q, k = q_raw / |q_raw|, k_raw / |k_raw|   (L2 over the head dimension; a zero row stays zero)
 *
 * then exactly the recurrence of kda_forward_chunked.  Layouts, dtypes, sizes and rules as for
 * kda_forward_chunked_impl with (q_raw, k_raw, v, z_g, z_beta) in the places of (q, k, v, g, beta).
 * The tensor-core kernel forms sigmoid and the inverse norms with the hardware's approximate
 * exponential, reciprocal and reciprocal square root (fp32, relative error ~1e-6); the fp32
 * kernel with expf and rsqrtf.
 */
KDA_API int kda_forward_chunked_fused(const void* q_raw, const void* k_raw, const void* v, const void* z_g,
                                      const void* z_beta, const float* S0, void* o, float* S_T, int B, int T,
                                      int H, int dk, int dv, int dtype, int impl, struct CUstream_st* stream);

/*
 * kda_forward_varlen -- prefill over packed sequences of different lengths (continuous batching).
 *
 * N sequences stored back to back along the token axis (the layout a paged serving engine
 * batches prefills in; podcast show-notes (scripod.com), outline item 5.3.1, and the channel
 * post on the K3 report (t.iss.one), online-inference paragraph: one paged pool for the KDA
 * states):
 *
 *   q, k, g    : [T_total, H, dk]   dtype
 *   v          : [T_total, H, dv]   dtype
 *   beta       : [T_total, H]       dtype
 *   cu_seqlens : [N + 1] int32 DEVICE array: sequence n is tokens cu_seqlens[n] .. cu_seqlens[n+1]-1,
 *                with 0 <= cu_seqlens[0] <= cu_seqlens[1] <= ... <= cu_seqlens[N] <= T_total (so no two
 *                sequences share a token; gaps between them are allowed).  The kernels check the whole
 *                array: if it breaks any of these rules, EVERY sequence is processed as empty (S_T = S0,
 *                no o row written) and the device status word is set to KDA_ERR_INVALID_ARG.  o rows of
 *                tokens outside every range are not written.
 *   S0, S_T    : [N, H, dk, dv] fp32, S0 may be NULL (zeros), S_T may be NULL or alias S0
 *   o          : [T_total, H, dv]   dtype
 *   impl       : kda_impl.
 *
 * Every sequence gives exactly what kda_forward_chunked gives for it alone.  Returns KDA_OK
 * or a negative kda_status (nothing enqueued on error).
 */
KDA_API int kda_forward_varlen(const void* q, const void* k, const void* v, const void* g, const void* beta,
                               const int* cu_seqlens, const float* S0, void* o, float* S_T, int N,
                               int T_total, int H, int dk, int dv, int dtype, int impl,
                               struct CUstream_st* stream);

/*
 * kda_decode_step_paged -- kda_decode_step with the states in a pool indexed per sequence.
 *
 *   S_pool : [n_slots, H, dk, dv] fp32, read and written in place
 *   slots  : [B] int32 DEVICE array: sequence b uses S_pool[slots[b]]; slots[b] < 0 skips sequence
 *            b (nothing read or written, o[b] untouched).  Active slots must be distinct.  A slot
 *            >= n_slots is skipped and sets the device status word to KDA_ERR_INVALID_ARG.
 *   q, k, g, v, beta, o : as kda_decode_step (per sequence b).
 *
 * Returns KDA_OK or a negative kda_status (nothing enqueued on error).
 */
KDA_API int kda_decode_step_paged(const void* q, const void* k, const void* v, const void* g, const void* beta,
                                  float* S_pool, int n_slots, const int* slots, void* o, int B, int H,
                                  int dk, int dv, int dtype, struct CUstream_st* stream);

/*
 * kda_state_compose -- apply a segment's state map: S_out = M S_in + N for `count` heads (fp32).
 *
 * Over a segment of tokens the recurrence is affine in its initial state: S_end = M S_start + N,
 * with M = prod_t (I - beta_t k_t k_t^T) Diag(exp g_t) and N the final state from a zero start.
 * Splitting a long sequence over devices then only needs this fixed-size pair exchanged
 * (KDA context parallelism: channel post on the K3 report (t.iss.one), infrastructure
 * paragraph).  A segment's pair comes from two kda_forward_chunked calls: N with S0 = NULL,
 * M as S_T with v = 0 (dv = dk) and S0 = the identity.
 *
 *   M      : [count, dk, dk] fp32
 *   S_in   : [count, dk, dv] fp32
 *   N      : [count, dk, dv] fp32, or NULL for zero
 *   S_out  : [count, dk, dv] fp32 output; may be S_in or N itself (in place), must not
 *            overlap M or partially overlap S_in / N
 *
 * dk, dv in {64, 128}.  Returns KDA_OK or a negative kda_status (nothing enqueued on error).
 */
KDA_API int kda_state_compose(const float* M, const float* S_in, const float* N, float* S_out, int count,
                              int dk, int dv, struct CUstream_st* stream);

/*
 * kda_output_correct -- correct the outputs of a segment that was run from a zero state, once the
 * state it really starts from is known: o_out[b,t,h,:] = o_in[b,t,h,:] + S_in[b,h]^T C[b,t,h,:].
 *
 * Over a segment S_t = Phi_t S_in + S_t^0 (Phi_t = prod_{u<=t} (I - beta_u k_u k_u^T) Diag(exp g_u),
 * S_t^0 the state from a zero start), so o_t = o_t^0 + S_in^T (Phi_t^T q_t).  The correction operand
 * C_t = Phi_t^T q_t is the output of kda_forward_chunked on the same q, k, g, beta with v = 0 (dv = dk)
 * and S0 = the identity; its S_T is the segment's map M (see kda_state_compose).  This is the one
 * exchange step of KDA context parallelism (channel post on the K3 report (t.iss.one),
 * infrastructure paragraph): a rank runs its segment before its incoming state is known, then
 * applies this correction.
 *
 *   C      : [B, T, H, dk]  dtype
 *   S_in   : [B, H, dk, dv] fp32
 *   o_in   : [B, T, H, dv]  dtype (the zero-start outputs)
 *   o_out  : [B, T, H, dv]  dtype output (bf16 rounded to nearest even); may be o_in itself
 *
 * bf16 with dk = dv = 128 runs on the tensor core (S_in rounded to bf16 as the product's operand,
 * fp32 accumulation); other shapes and fp32 on CUDA cores in fp32.  T == 0 does nothing.  Returns
 * KDA_OK or a negative kda_status (nothing enqueued on error).
 */
KDA_API int kda_output_correct(const void* C, const float* S_in, const void* o_in, void* o_out, int B, int T, int H,
                               int dk, int dv, int dtype, struct CUstream_st* stream);

/*
 * ---------------------------------------------------------------------------------------------
 * The short causal convolution, the selective scan and the state pools: what a serving engine runs
 * beside the KDA recurrence.  Conventions as above, with one difference: the activations may be
 * slices of wider rows.  Each `ld*` argument is the distance in elements from one token's row to the
 * next (the row itself is contiguous), so that the q, k, v or x, B, C parts of one projection are
 * passed without a copy; batch entry b starts at row b*T.  Rows of vector-loaded tensors (x, y, Bm,
 * Cm) start on 16-byte boundaries: their ld is a multiple of 16 bytes.  dt, A, D and dt_bias need
 * their element's alignment only.  Inputs and outputs are compared by the whole range from their
 * first to their last byte: an output may not lie between the rows of an input.
 */

/* Activation of the short convolution. */
typedef enum { KDA_ACT_NONE = 0, KDA_ACT_SILU = 1 } kda_activation;

/*
 * kda_short_conv -- the depthwise causal convolution of width W before the recurrence (each of its
 * inputs q, k, v, or x, B, C of the selective scan, is such a convolution of its projection):
 *
 *   y[b,t,c] = act( bias[c] + sum_{w < W} weight[c,w] u[b, t-(W-1)+w, c] )
 *
 * where u is the sequence x[b] preceded by its last W-1 inputs, `state`.  fp32 arithmetic.
 *
 *   x         : [B, T, C]     dtype, row stride ldx >= C
 *   weight    : [C, W]        dtype (a depthwise kernel as frameworks keep it)
 *   bias      : [C]           dtype, or NULL for none
 *   state     : [B, W-1, C]   dtype, the inputs before token 0 (oldest first), or NULL for zeros
 *   y         : [B, T, C]     dtype output, row stride ldy >= C
 *   state_out : [B, W-1, C]   dtype output, the last W-1 inputs (of `state` too when T < W-1), or NULL.
 *               May be `state` itself; no other overlap between outputs and inputs.
 *   W         : 2, 3 or 4.  C: a positive multiple of 8.
 *
 * The KDA prefill takes contiguous q, k and v.  Where they are slices of one projection, a call for each
 * slice (x with the projection's row stride, the slice's rows of weight and bias, a state of its own)
 * leaves them contiguous without a copy.
 *
 * T == 0 copies state to state_out.  Returns KDA_OK; KDA_ERR_UNSUPPORTED for another W, a C that is
 * not a multiple of 8, another dtype or activation; KDA_ERR_INVALID_ARG for a B or T above 2e9 too.
 */
KDA_API int kda_short_conv(const void* x, const void* weight, const void* bias, const void* state, void* y,
                           void* state_out, int B, int T, int C, int W, long long ldx, long long ldy,
                           int activation, int dtype, struct CUstream_st* stream);

/*
 * kda_short_conv_varlen -- kda_short_conv over N sequences packed along the token axis.
 *
 *   x, y             : [T_total, C]; cu_seqlens : [N + 1] int32 DEVICE array, rules of kda_forward_varlen
 *                      (checked by the kernel: offsets that break them leave every sequence empty and
 *                      set the status word).  y rows outside every sequence are not written.
 *   state, state_out : [N, W-1, C]
 */
KDA_API int kda_short_conv_varlen(const void* x, const void* weight, const void* bias, const int* cu_seqlens,
                                  const void* state, void* y, void* state_out, int N, int T_total, int C, int W,
                                  long long ldx, long long ldy, int activation, int dtype,
                                  struct CUstream_st* stream);

/*
 * kda_short_conv_step -- one token for every sequence; `state` [B, W-1, C] is shifted in place.
 *   x, y : [B, C], row strides ldx, ldy.
 */
KDA_API int kda_short_conv_step(const void* x, const void* weight, const void* bias, void* state, void* y, int B,
                                int C, int W, long long ldx, long long ldy, int activation, int dtype,
                                struct CUstream_st* stream);

/*
 * kda_short_conv_step_paged -- kda_short_conv_step with the states in a pool [n_slots, W-1, C]:
 * sequence b uses slots[b]; rules of kda_decode_step_paged (negative: skipped, y[b] untouched; a slot
 * >= n_slots is skipped and sets the status word; active slots are distinct).
 */
KDA_API int kda_short_conv_step_paged(const void* x, const void* weight, const void* bias, void* state_pool,
                                      int n_slots, const int* slots, void* y, int B, int C, int W, long long ldx,
                                      long long ldy, int activation, int dtype, struct CUstream_st* stream);

/*
 * kda_ssm_forward -- prefill of the selective state space scan with one decay per head:
 *
 *   s_t = softplus(dt_t + dt_bias)                      (per token and head)
 *   S_t = exp(s_t A) S_{t-1} + B_t (s_t x_t)^T          (S in R^{N x P}, fp32)
 *   y_t = S_t^T C_t + D x_t
 *
 * i.e. the recurrence of kda_forward_chunked with a scalar decay and no delta rule: B, C, x stand in
 * the places of k, q, v.  The H heads share G pairs (B, C): head h uses pair h / (H / G).
 *
 *   x       : [B, T, H, P]  dtype, token stride ldx >= H*P
 *   dt      : [B, T, H]     dtype, token stride lddt >= H
 *   A       : [H]           fp32 (A <= 0: a decay)
 *   Bm, Cm  : [B, T, G, N]  dtype, token strides ldb, ldc >= G*N
 *   D       : [H]           fp32, or NULL for no skip term
 *   dt_bias : [H]           fp32, or NULL for zero
 *   S0      : [B, H, N, P]  fp32, or NULL for zero
 *   y       : [B, T, H, P]  dtype output, contiguous
 *   S_T     : [B, H, N, P]  fp32 output, or NULL; may be S0 itself; no other overlap
 *   N, P    : 64 or 128.  G divides H.
 *   impl    : kda_impl.  KDA_IMPL_AUTO runs the chunked tensor-core kernel for bf16 and the
 *             token-serial fp32 kernel for fp32; KDA_IMPL_TCGEN05 refuses fp32.  KDA_IMPL_SIMT takes
 *             bf16 too, at many times the time.
 *   workspace, workspace_bytes : DEVICE memory of at least kda_ssm_workspace(...) bytes, 16-byte
 *             aligned (NULL when that is 0), not used by anything else until the work is done.
 *
 * Precision.  The token-serial kernel and the single-token steps compute in fp32 throughout; a token's
 * decay is one fp32 number, off by up to 2^-25 of the state where it is near 1.  The tensor-core kernel
 * holds S in fp32, reads it and the decayed scores C.B as bf16 operands for y (2^-8 of a term of y at most,
 * beside the rounding of y itself), and adds to S terms that are off by 3 * 2^-16 of themselves at most.
 * The tensor core's sums are rounded towards zero, 16 times for a chunk of 128 tokens: S loses up to
 * 16 * 2^-23 of itself for each chunk that it remembers (about 8e-7: 6e-6 of a state that remembers a
 * thousand tokens, 4e-4 after 65536 tokens without any decay).
 *
 * The tensor-core kernel forms whole 128-token blocks: a non-finite value in one token's x, B or dt
 * may reach the outputs of other tokens of its block, earlier ones too.  A NaN in A[h] makes head h's
 * outputs and state NaN; A[h] = -infinity forgets everything before each token.  T == 0 copies S0 to S_T.
 */
KDA_API int kda_ssm_forward(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                            const float* D, const float* dt_bias, const float* S0, void* y, float* S_T, int B,
                            int T, int H, int G, int N, int P, long long ldx, long long lddt, long long ldb,
                            long long ldc, int dtype, int impl, void* workspace, size_t workspace_bytes,
                            struct CUstream_st* stream);

/*
 * kda_ssm_forward_varlen -- kda_ssm_forward over n_seq sequences packed along the token axis.
 *
 *   x, dt, Bm, Cm, y : [T_total, ...]; cu_seqlens : [n_seq + 1] int32 DEVICE array, rules of
 *                      kda_forward_varlen.  y rows outside every sequence are not written.
 *   S0, S_T          : [n_seq, H, N, P]
 *
 * The tensor-core kernel cuts sequences into segments that run side by side where heads and sequences are
 * few, by the mean length T_total / n_seq (the offsets are not read on the host): one long sequence packed
 * with many short ones is not cut, and is faster in a call of its own.
 */
KDA_API int kda_ssm_forward_varlen(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                                   const int* cu_seqlens, const float* D, const float* dt_bias, const float* S0,
                                   void* y, float* S_T, int n_seq, int T_total, int H, int G, int N, int P,
                                   long long ldx, long long lddt, long long ldb, long long ldc, int dtype, int impl,
                                   void* workspace, size_t workspace_bytes, struct CUstream_st* stream);

/*
 * kda_ssm_workspace -- bytes of device workspace kda_ssm_forward (n_seq = B, T_total = B*T) or
 * kda_ssm_forward_varlen needs.  0 where none is needed (and for sizes the calls refuse).
 */
KDA_API size_t kda_ssm_workspace(int n_seq, int T_total, int H, int N, int P, int dtype, int impl);

/*
 * kda_ssm_decode_step -- one token for every (b, h), S [B, H, N, P] updated in place.
 *   x, y : [B, H, P] (x with row stride ldx, y contiguous); dt : [B, H]; Bm, Cm : [B, G, N].
 */
KDA_API int kda_ssm_decode_step(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                                const float* D, const float* dt_bias, float* S, void* y, int B, int H, int G, int N,
                                int P, long long ldx, long long lddt, long long ldb, long long ldc, int dtype,
                                struct CUstream_st* stream);

/*
 * kda_ssm_decode_step_paged -- kda_ssm_decode_step with the states in a pool [n_slots, H, N, P]:
 * sequence b uses slots[b]; rules of kda_decode_step_paged.
 */
KDA_API int kda_ssm_decode_step_paged(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                                      const float* D, const float* dt_bias, float* S_pool, int n_slots,
                                      const int* slots, void* y, int B, int H, int G, int N, int P, long long ldx,
                                      long long lddt, long long ldb, long long ldc, int dtype,
                                      struct CUstream_st* stream);

/*
 * kda_pool -- one state pool as the pool operators see it: n_slots slots of `pieces` runs of
 * piece_bytes each.  A pool [n_slots, H, dk, dv] is one piece a slot; the boundary states of one batch
 * entry, S_mid[b] of kda_forward_chunked_states ([H, n_mid, dk, dv], slot = boundary), are H pieces.
 * All byte counts and the base are multiples of 16.  Pools are told apart by the whole range from their
 * first to their last byte: layers that interleave in memory ([n_slots, layers, ...]) go into a call as one
 * pool whose slots hold them all.
 */
typedef struct {
    void* base;
    long long slot_stride;  /* bytes from one slot to the next */
    long long pieces;       /* runs of contiguous bytes in a slot */
    long long piece_stride; /* bytes from one run of a slot to the next */
    long long piece_bytes;  /* bytes of one run */
} kda_pool;

/*
 * kda_pool_copy -- copy slots, in every pool at once: slot dst_idx[i] of dst[p] becomes slot
 * src_idx[i] of src[p], for i < n and p < n_pools (all layers of a model in one call).  One source may
 * feed many destinations (forking a sequence).
 *
 *   dst, src         : HOST arrays of n_pools pools; dst[p] and src[p] have the same pieces and
 *                      piece_bytes, and are the same pool or do not overlap
 *   n_dst, n_src     : slots of every dst and every src pool
 *   src_idx, dst_idx : [n] int32 DEVICE arrays, n at most 2^20; a pair with a negative index is skipped
 *
 * A pair is not copied, and the status word is set to KDA_ERR_INVALID_ARG, when an index is past its
 * pool, when another pair has the same destination, or when (dst[p] being src[p]) its destination is
 * the source of another pair: the result never depends on the order of the copies.  A pair of a slot
 * with itself does nothing.  Finding such pairs costs one reading of the list for each 512 pairs of it (for
 * each pair up to 1024 pairs): 3 ms for 65536 pairs in 16 pools, which is long only beside small slots.
 */
KDA_API int kda_pool_copy(const kda_pool* dst, const kda_pool* src, int n_pools, int n_dst, int n_src,
                          const int* src_idx, const int* dst_idx, int n, struct CUstream_st* stream);

/*
 * kda_pool_clear -- set slots to zero bytes in every pool: the state a new sequence starts from.
 *   idx : [n] int32 DEVICE array, n at most 2^20; negative entries are skipped, entries >= n_slots are skipped and set
 *         the status word.
 */
KDA_API int kda_pool_clear(const kda_pool* pools, int n_pools, int n_slots, const int* idx, int n,
                           struct CUstream_st* stream);

/*
 * kda_pool_compact -- drop the sequences that ended and move the live ones' states to the front.
 *
 * Sequence b is live if slots[b] >= 0 and done[b] == 0.  With L live sequences, the live slots >= L, in
 * ascending order, move into the slots < L that are not live, in ascending order, in every pool; the
 * other slots keep their contents.
 *
 *   slots     : [B] int32 DEVICE array, the table of kda_decode_step_paged; B at most 2^20
 *   done      : [B] bytes (0 or not) in DEVICE memory, or NULL for none ended
 *   slots_out : [B] int32 DEVICE output: the new table, -1 for sequences that are not live.  May be
 *               slots itself.
 *   workspace : DEVICE int32 array of n_slots + 1 entries (16-byte aligned) that nothing else uses until
 *               the work is done; entry 0 receives the number of slots moved.
 *   n_slots   : at most 65536 (KDA_ERR_UNSUPPORTED above)
 *
 * Two live sequences on one slot, or a live slot >= n_slots, set the status word to
 * KDA_ERR_INVALID_ARG; then nothing moves and slots_out is slots.
 */
KDA_API int kda_pool_compact(const kda_pool* pools, int n_pools, int n_slots, const int* slots,
                             const unsigned char* done, int* slots_out, int B, int* workspace,
                             struct CUstream_st* stream);

/*
 * kda_get_device_status -- synchronise `stream`, then return and clear the status word
 * of the current device: KDA_OK, KDA_ERR_TIMEOUT (a kernel's bounded wait gave up; its
 * outputs are then undefined), KDA_ERR_INVALID_ARG (a kernel found an out-of-range device
 * index: a sequence offset or a state slot), or KDA_ERR_CUDA if the synchronisation itself
 * failed.
 *
 * The word belongs to the DEVICE, not to a call or a stream: every kernel of the library on that
 * device, on any stream, sets the same word (the first error wins), and a read clears it.  Only
 * `stream` is synchronised, so with work on several streams a kernel still running on another one
 * may set the word after the read, and the error read may come from another stream's call.  When
 * several streams are in use, synchronise the device (cudaDeviceSynchronize) before calling this
 * to attribute an error to the work enqueued before that point.
 */
KDA_API int kda_get_device_status(struct CUstream_st* stream);

/* kda_status_string -- static, human-readable name of a kda_status value. */
KDA_API const char* kda_status_string(int status);

/* kda_version -- library version as major*10000 + minor*100 + patch. */
KDA_API int kda_version(void);

/*
 * kda_debug_set_wait_fault -- TEST HOOK for the device-side timeout path (not for production).
 *
 * The tensor-core prefill coordinates its two warp groups with mbarrier waits, each bounded
 * in wall time (2 s by default); a wait that runs out sets the status word to
 * KDA_ERR_TIMEOUT, lets every warp of the CTA leave its loop, drains the outstanding
 * tensor-core and TMA work, frees the tensor memory and returns.  Nothing traps, faults or
 * hangs, and the CUDA context stays usable.
 *
 *   mode 1: subsequent tcgen05 prefill launches skip the first hand-off from the operand
 *           warps to the recurrence warps, so a wait is guaranteed to run out; every wait
 *           is limited to timeout_ns (1 ms .. 10 s).  Outputs of such launches are undefined.
 *           Tensor-core calls of the selective scan skip their first hand-off too (where a prompt is
 *           cut into segments, that of the launch over the segments' states).
 *   mode 0: normal operation (the timeout_ns argument is ignored; 2 s limit).
 *
 * Process-wide setting, read at launch.  Returns KDA_OK or KDA_ERR_INVALID_ARG.
 */
KDA_API int kda_debug_set_wait_fault(int mode, unsigned long long timeout_ns);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
