/*
 * gdn2.h -- C ABI of the MI355X (gfx950) Gated DeltaNet-2 recurrence library.
 *
 * The operation is the GDN-2 state update of the page "Why NVIDIA Gated
 * DeltaNet-2 separates erase and write gates" (axbrief.com), section
 * "Gated Delta Rule-2: channel-wise separation of erase and write", its
 * recurrence equation:
 *
 *     S_t = (I - k_t (b_t . k_t)^T) Diag(alpha_t) S_{t-1} + k_t (w_t . v_t)^T
 *     o_t = S_t^T q_t                       (read-out after the update)
 *
 * S is dk x dv (rows are key channels), alpha_t = exp(log_alpha_t) is a decay
 * per key channel, b_t in [0,1]^dk is the erase gate (key side) and
 * w_t in [0,1]^dv the write gate (value side).  There is no query scale.
 *
 * The calls: a chunk-parallel forward over whole sequences (the same page,
 * section "Gated Delta Rule-2", gives the chunk size of 64 used by the fused
 * training kernels), the same forward from gate logits (activations formed in
 * the kernels), the same forward over packed sequences of different
 * lengths, its backward pass (vector-Jacobian product; the same section: the
 * gates enter the gradient inner products, so the backward is derived with
 * them), a single-token recurrent decode step (the page's opening section:
 * decoding keeps a constant-size state), and the mixer's fused elementwise
 * passes on either side of the recurrence.  Beside them stand the calls of a
 * state space block (its scan, convolution and norm) and of an attention block
 * (attention, rotary positions and norm), described with them below.
 *
 * Conventions for every call:
 *   - Tensor pointers are DEVICE pointers (HIP global memory) of the current
 *     device, contiguous and row-major in the layouts stated below, and
 *     16-byte aligned.
 *   - `stream` is a hipStream_t (NULL = the legacy default stream).  Work is
 *     enqueued asynchronously; the caller keeps every buffer alive until the
 *     stream has passed the call.
 *   - The library never allocates, frees or synchronises and keeps no reference
 *     after returning.  Its only global state is the per-device address of the
 *     fixed array gdn2_chunk_bwd_noalloc works in, looked up once under a lock;
 *     every other call is reentrant.
 *   - All validation happens before anything is enqueued.  On any error the
 *     call returns a non-zero status and writes nothing.  A launch rejected by
 *     the HIP runtime returns GDN2_ERR_HIP.  Faults inside a kernel surface at
 *     the caller's next synchronisation, as for any HIP kernel.
 *   - Inputs are not range-checked on the device: log_alpha must be finite and
 *     <= 0; b and w are expected in [0,1] (values outside are used as given).
 */
#ifndef GDN2_H
#define GDN2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Chunk length of the chunk-parallel forward (tokens per chunk). */
#define GDN2_CHUNK 64

/* Element type of q, k, v, b, w (`dtype`) and of o (`o_dtype`).  Arithmetic
 * inside is fp32 either way; log_alpha and the state are always float32. */
typedef enum gdn2_dtype {
    GDN2_DTYPE_F32 = 0,
    GDN2_DTYPE_BF16 = 1
} gdn2_dtype_t;

typedef enum gdn2_status {
    GDN2_OK = 0,
    GDN2_ERR_NULL = 1,        /* a required pointer is NULL */
    GDN2_ERR_SHAPE = 2,       /* a size is < 1 or too large for 32-bit indexing of a row */
    GDN2_ERR_UNSUPPORTED = 3, /* (dk, dv, dtype) is not built into this library */
    GDN2_ERR_MISALIGNED = 4,  /* a tensor pointer is not 16-byte aligned */
    GDN2_ERR_ALIAS = 5,       /* an output overlaps an input it must not overlap */
    GDN2_ERR_WORKSPACE = 6,   /* the workspace is NULL or smaller than required */
    GDN2_ERR_HIP = 7          /* the HIP runtime rejected a query or a launch */
} gdn2_status_t;

/*
 * gdn2_chunk_fwd -- forward over B sequences of T tokens and H heads.
 *
 *   q, k, b       [B, T, H, dk]  dtype        query, key, erase gate
 *   v, w          [B, T, H, dv]  dtype        value, write gate
 *   log_alpha     [B, T, H, dk]  float32      log of the per-channel decay
 *   initial_state [B, H, dk, dv] float32      S_0, or NULL for zeros
 *   o             [B, T, H, dv]  o_dtype      out: o_t = S_t^T q_t
 *   final_state   [B, H, dk, dv] float32      out: S_T, or NULL to skip;
 *                                             may be the same pointer as
 *                                             initial_state (updated in place)
 *
 * T may be any value >= 1 (a last partial chunk is handled exactly).
 * Built combinations: dtype BF16 with (dk, dv) = (64, 64) or (128, 128);
 * dtype F32 with (64, 64).  o_dtype is F32, or equal to dtype: with bf16
 * inputs an F32 output keeps the fp32 accumulation all the way out, a BF16
 * output rounds it once on the store.  Others return GDN2_ERR_UNSUPPORTED.
 * o must not overlap any input; final_state must not overlap any input other
 * than an identical initial_state.  H * dk and H * dv (the elements between
 * consecutive tokens of one tensor) must be below 2^22, else GDN2_ERR_SHAPE.
 * workspace / workspace_bytes select the implementation.  With a workspace of
 * at least gdn2_chunk_fwd_split_workspace_bytes(...) bytes (device memory owned by
 * the caller, 256-byte aligned, overlapping no argument; its contents on entry
 * do not matter and on return are unspecified) the forward runs as two kernels
 * per batch of chunks: one forms every chunk's state-independent quantities in
 * parallel, the other carries the state through the chunks.  With
 * workspace = NULL and workspace_bytes = 0 it runs as one fused kernel (same
 * results within the parity bar, no workspace).  A workspace passed where the
 * two-kernel form does not exist, or a shorter one, returns GDN2_ERR_WORKSPACE.
 * gdn2_chunk_fwd_workspace_bytes says which form is faster for a shape.
 */
gdn2_status_t gdn2_chunk_fwd(const void* q, const void* k, const void* v,
                             const float* log_alpha, const void* b, const void* w,
                             const float* initial_state, void* o, float* final_state,
                             int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv,
                             gdn2_dtype_t dtype, gdn2_dtype_t o_dtype, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * gdn2_chunk_fwd_logits -- gdn2_chunk_fwd with the gate activations done in
 * the kernels: it takes the projections' outputs instead of the activated
 * decay and gates.  The erase and write gates are sigmoids of projections of
 * the token (page "Why NVIDIA Gated DeltaNet-2 separates erase and write
 * gates", axbrief.com, section "Gated Delta Rule-2"); the decay takes the
 * same form (alpha = sigmoid(a), so log alpha = log sigmoid(a)).  Forming the
 * activation inside the recurrence kernel so that no full-sequence activation
 * tensor is stored is the "gate-in-kernel" fusion of page "CARVE:
 * Content-Aware Recurrent with Value Efficiency for Chunk-Parallel Linear
 * Attention" (gist.science), section 2.3 "Key-Axis Decay and Fusion".
 *
 *   a_logit       [B, T, H, dk]  dtype        decay logits: alpha = sigmoid(a)
 *   b_logit       [B, T, H, dk]  dtype        erase-gate logits: b = sigmoid(.)
 *   w_logit       [B, T, H, dv]  dtype        write-gate logits: w = sigmoid(.)
 *
 * Every other argument, the workspace rule (gdn2_chunk_fwd_workspace_bytes
 * applies unchanged) and every error are as for gdn2_chunk_fwd.  dtype must be
 * BF16 (dk = dv = 64 or 128), else GDN2_ERR_UNSUPPORTED.  The activations are
 * formed in fp32 from the bf16 logits; a logit below about -88 gives a decay
 * or gate of exactly 0.
 */
gdn2_status_t gdn2_chunk_fwd_logits(const void* q, const void* k, const void* v,
                                    const void* a_logit, const void* b_logit, const void* w_logit,
                                    const float* initial_state, void* o, float* final_state,
                                    int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv,
                                    gdn2_dtype_t dtype, gdn2_dtype_t o_dtype, void* workspace,
                                    size_t workspace_bytes, void* stream);

/*
 * gdn2_chunk_fwd_split_workspace_bytes -- bytes of device workspace that the
 * two-kernel form of gdn2_chunk_fwd needs for these sizes on the current device:
 * the chunk records of one batch of about a thousand (sequence, head, chunk)
 * triples, 68,608 bytes each at dk = dv = 128 (44,032 at 64), plus one fp32
 * state [B, H, dk, dv].  When the (sequence, head) chains (one workgroup of
 * the state pass each) fill at most half of the device's compute units and the
 * sequences hold at least 32 chunks, the form instead cuts every sequence into
 * segments walked in
 * parallel and joined through their state transitions: it then needs every
 * chunk's record plus, per (sequence, head), a [dk][2 dv] fp32 transition for
 * every segment but the last and a [dk][dv] fp32 start state for every
 * segment.  The
 * two-kernel form exists for BF16 inputs with dk = dv = 64 or 128; for every
 * other combination (and for sizes out of range) this returns 0.
 */
size_t gdn2_chunk_fwd_split_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv,
                                            gdn2_dtype_t dtype);

/*
 * gdn2_chunk_fwd_workspace_bytes -- the workspace to pass to gdn2_chunk_fwd for
 * its faster form on the current device: the two-kernel form's size (as above)
 * when the fused kernel's chains, one per (sequence, head, 64 value columns),
 * are fewer than the device's compute units, else 0 (run with workspace = NULL,
 * workspace_bytes = 0: the fused kernel).
 */
size_t gdn2_chunk_fwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv,
                                      gdn2_dtype_t dtype);

/*
 * gdn2_chunk_fwd_varlen -- the same forward over N sequences of different
 * lengths packed along one token axis (prefill of a serving batch).
 *
 *   q, k, b       [total_T, H, dk]  dtype
 *   v, w          [total_T, H, dv]  dtype
 *   log_alpha     [total_T, H, dk]  float32
 *   cu_seqlens    [N + 1]           int64, DEVICE memory, 8-byte aligned:
 *                                   sequence n holds tokens
 *                                   [cu_seqlens[n], cu_seqlens[n + 1])
 *   initial_state [N, H, dk, dv]    float32, or NULL for zeros
 *   o             [total_T, H, dv]  o_dtype
 *   final_state   [N, H, dk, dv]    float32 or NULL; may equal initial_state
 *
 * The offsets are expected to be non-decreasing with cu_seqlens[0] = 0 and
 * cu_seqlens[N] = total_T (they are in device memory and are not read on the
 * host).  Each sequence's range is clamped into [0, total_T] on the device, so
 * any offsets keep every access inside the tensors; tokens outside every
 * sequence are left unwritten in o.  A sequence of length 0 passes its initial
 * state (or zeros) through to final_state.  The final states are laid out as
 * gdn2_decode_step's state, so decoding continues from them directly.
 * N >= 1, total_T >= 0; everything else as for gdn2_chunk_fwd (supported
 * shapes and dtypes, alignment, aliasing; cu_seqlens must not overlap o or
 * final_state).
 */
gdn2_status_t gdn2_chunk_fwd_varlen(const void* q, const void* k, const void* v,
                                    const float* log_alpha, const void* b, const void* w,
                                    const float* initial_state, void* o, float* final_state,
                                    const int64_t* cu_seqlens, int64_t N, int64_t total_T,
                                    int64_t H, int64_t dk, int64_t dv, gdn2_dtype_t dtype,
                                    gdn2_dtype_t o_dtype, void* stream);

/*
 * gdn2_decode_step -- one recurrent step for N independent sequences.
 *
 *   q, k, b       [N, H, dk]     dtype
 *   v, w          [N, H, dv]     dtype
 *   log_alpha     [N, H, dk]     float32
 *   state         [N, H, dk, dv] float32      read and updated in place
 *   o             [N, H, dv]     o_dtype      out: o = S_new^T q
 *
 * Built combinations: dtype BF16 or F32 with (dk, dv) = (64, 64) or (128, 128);
 * o_dtype is F32 or equal to dtype.
 * o must not overlap any input or the state.
 */
gdn2_status_t gdn2_decode_step(const void* q, const void* k, const void* v,
                               const float* log_alpha, const void* b, const void* w,
                               float* state, void* o, int64_t N, int64_t H, int64_t dk,
                               int64_t dv, gdn2_dtype_t dtype, gdn2_dtype_t o_dtype,
                               void* stream);

/*
 * gdn2_chunk_bwd_workspace_bytes -- bytes of device workspace gdn2_chunk_bwd
 * needs for these sizes (NC = ceil(T / 64)): 4 * (2 B H NC dk dv +
 * 2 B T H dv + B H NC R), each of the five parts rounded up to 256 bytes, where
 * R = 2*64*64 + 5*64*dk + 64*dv + dk rounded up to a multiple of 64 (one record
 * of chunk-local quantities per chunk).  Returns 0 if the sizes overflow or dk
 * or dv exceeds 2^20.
 */
size_t gdn2_chunk_bwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv);

/*
 * gdn2_chunk_bwd -- backward pass of gdn2_chunk_fwd: the gradients of
 * L = sum(d_o * o) + sum(d_final_state * S_T) with respect to every input.
 *
 *   q, k, v, log_alpha, b, w, initial_state   as for gdn2_chunk_fwd (dtype)
 *   d_o            [B, T, H, dv]  float32     upstream gradient of o
 *   d_final_state  [B, H, dk, dv] float32     upstream gradient of S_T, or NULL
 *                                             for zeros
 *   dq, dk, db     [B, T, H, dk]  float32     out
 *   dv, dw         [B, T, H, dv]  float32     out
 *   dlog_alpha     [B, T, H, dk]  float32     out
 *   d_initial_state [B, H, dk, dv] float32    out: gradient of S_0, or NULL to
 *                                             skip (zeros S_0 when
 *                                             initial_state is NULL)
 *   workspace      device memory of at least
 *                  gdn2_chunk_bwd_workspace_bytes(B, T, H, dk, dv) bytes,
 *                  16-byte aligned, owned by the caller; its contents on entry
 *                  do not matter and on return are unspecified
 *
 * The call re-runs the forward to recover the state entering every chunk, so
 * it needs neither o nor any saved state.  Built combinations and the limits
 * on sizes are those of gdn2_chunk_fwd (B, T >= 1).  No output may overlap
 * another output, an input or the workspace, and the workspace may not
 * overlap an input (GDN2_ERR_ALIAS); a missing or short workspace returns
 * GDN2_ERR_WORKSPACE.
 */
gdn2_status_t gdn2_chunk_bwd(const void* q, const void* k, const void* v,
                             const float* log_alpha, const void* b, const void* w,
                             const float* initial_state, const float* d_o,
                             const float* d_final_state, float* dq, float* dk, float* dv,
                             float* dlog_alpha, float* db, float* dw, float* d_initial_state,
                             void* workspace, size_t workspace_bytes, int64_t B, int64_t T,
                             int64_t H, int64_t dk_dim, int64_t dv_dim, gdn2_dtype_t dtype,
                             void* stream);

/* Bytes of the device array that gdn2_chunk_bwd_noalloc uses as its workspace (64 MiB). */
#define GDN2_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * gdn2_chunk_bwd_noalloc -- gdn2_chunk_bwd for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving or training loops,
 * harnesses that forbid hipMalloc): the same gradients, computed by the same
 * kernels, with the workspace taken from a fixed array of GDN2_SCRATCH_BYTES
 * inside the library instead of from the caller.  Nothing is allocated or freed.
 *
 *   arguments       as for gdn2_chunk_bwd, without workspace / workspace_bytes
 *
 * Calls whose gdn2_chunk_bwd_workspace_bytes(B, T, H, dk, dv) exceeds
 * GDN2_SCRATCH_BYTES return GDN2_ERR_WORKSPACE (for example B = 1, H = 16,
 * dk = dv = 128 fits up to T = 576).  Each GPU the library runs on holds its own
 * array from the first call on that device until the process ends; the first
 * call on a device looks up the array's address (GDN2_ERR_HIP if that fails).
 * Every call on one GPU uses that GPU's one array, which keeps the last call's
 * contents: calls that may run at the same time on one GPU (different streams,
 * different host threads without ordering) race and must not overlap.  No part
 * of the array needs clearing: every call writes each slot before reading it.
 */
gdn2_status_t gdn2_chunk_bwd_noalloc(const void* q, const void* k, const void* v,
                                     const float* log_alpha, const void* b, const void* w,
                                     const float* initial_state, const float* d_o,
                                     const float* d_final_state, float* dq, float* dk, float* dv,
                                     float* dlog_alpha, float* db, float* dw,
                                     float* d_initial_state, int64_t B, int64_t T, int64_t H,
                                     int64_t dk_dim, int64_t dv_dim, gdn2_dtype_t dtype,
                                     void* stream);

/*
 * gdn2_mixer_prep -- the elementwise steps between the layer's projections and
 * the recurrence, in one pass (page "Why NVIDIA Gated DeltaNet-2 separates
 * erase and write gates", the section on the layer's architecture: query and
 * key through a short causal convolution, SiLU and L2 normalisation, value
 * through the convolution and SiLU; section "Gated Delta Rule-2": erase and
 * write gates are sigmoids of projections):
 *
 *   q = xq' / sqrt(|xq'|^2 + eps),  xq' = SiLU(conv(xq))   (norm over dk)
 *   k likewise from xk;  v = SiLU(conv(xv))
 *   b = sigmoid(xb),  w = sigmoid(xw),  log_alpha = log sigmoid(xa)
 *
 *   xq, xk, xb, xa  [B, T, H, dk]  dtype   projection outputs (pre-activation)
 *   xv, xw          [B, T, H, dv]  dtype
 *   conv_q, conv_k  [H * dk, 4]    float32 depthwise causal taps: tap j of a
 *   conv_v          [H * dv, 4]    float32 channel multiplies its input at token
 *                                          t - 3 + j; tokens before 0 are zero
 *   q, k, b         [B, T, H, dk]  dtype   out
 *   v, w            [B, T, H, dv]  dtype   out
 *   log_alpha       [B, T, H, dk]  float32 out (<= 0)
 *
 * The sigmoid form of the decay is this library's reading: the pages give the
 * decay no activation.  Built: dtype BF16 or F32 with dk = dv = 64 or 128.  No
 * output may overlap an input or another output.  eps >= 0.
 * With b, w and log_alpha all NULL only q, k and v are formed (xb, xw and xa
 * are then not read and may be NULL): the gates are left to
 * gdn2_chunk_fwd_logits, which activates them inside the recurrence kernels.
 * Some but not all of b, w, log_alpha NULL returns GDN2_ERR_NULL.
 */
gdn2_status_t gdn2_mixer_prep(const void* xq, const void* xk, const void* xv, const void* xb,
                              const void* xw, const void* xa, const float* conv_q,
                              const float* conv_k, const float* conv_v, void* q, void* k,
                              void* v, void* b, void* w, float* log_alpha, int64_t B, int64_t T,
                              int64_t H, int64_t dk, int64_t dv, float eps, gdn2_dtype_t dtype,
                              void* stream);

/*
 * gdn2_mixer_out -- the layer output from the recurrence output, in one pass
 * (same page and section: RMS normalisation and a SiLU output gate):
 *
 *   y = o / sqrt(mean(o^2) + eps) * gamma * SiLU(z)      (mean over dv)
 *
 *   o      [B, T, H, dv]  o_dtype  recurrence output (F32, or equal to dtype)
 *   z      [B, T, H, dv]  dtype    output-gate projection
 *   gamma  [dv]           float32  norm weight, shared by the heads
 *   y      [B, T, H, dv]  dtype    out; must not overlap o, z or gamma
 *
 * Built: dtype BF16 or F32 with dv = 64 or 128.  eps >= 0.
 */
gdn2_status_t gdn2_mixer_out(const void* o, const void* z, const float* gamma, void* y, int64_t B,
                             int64_t T, int64_t H, int64_t dv, float eps, gdn2_dtype_t dtype,
                             gdn2_dtype_t o_dtype, void* stream);

/*
 * The state space block.  Hybrid stacks put selective state space layers beside
 * the layers above (page "GDN-2-3B", orcarouter.ai: a listed stack of 52 layers
 * holds 23 of them).  Such a layer is a layer norm, projections (the caller's),
 * a short causal convolution with SiLU, the scan, and gdn2_mixer_out on the
 * scan's output.  These calls follow the conventions at the top; beyond them:
 *   - x, b, c and dt may have a token stride of their own, so that they can be
 *     parts of one wider tensor; a token's own elements are contiguous, and so
 *     is every output.
 *   - Each is built for dtype BF16 and F32, and its outputs have that dtype; A,
 *     D, biases, taps, norm weights, statistics and scan states are float32.
 */

/*
 * gdn2_ssm_fwd -- the selective state space scan over B sequences of T tokens.
 * Per sequence and head, with a state S of dk rows and dv columns:
 *
 *   dt_t = softplus(raw_t + dt_bias)          (raw_t + dt_bias if softplus = 0)
 *   S_t  = exp(dt_t A) S_{t-1} + dt_t b_t x_t^T,   y_t = S_t^T c_t + D x_t
 *
 *   x             [B, T, H, dv]  dtype    x_stride elements between tokens
 *   dt            [B, T, H]      dtype    raw time steps, dt_stride
 *   b, c          [B, T, G, dk]  dtype    shared by the H / G heads of a group:
 *                                         head h takes group h / (H / G);
 *                                         b_stride, c_stride
 *   A             [H]            float32  expected < 0; a decay below 2^-149 is 0
 *   D, dt_bias    [H]            float32  each NULL for zeros
 *   initial_state [B, H, dk, dv] float32  or NULL for zeros
 *   y             [B, T, H, dv]  dtype    out
 *   final_state   [B, H, dk, dv] float32  out, or NULL to skip; may be the same
 *                                         pointer as initial_state
 *
 * Token t of sequence n starts at element (n T + t) * stride of its tensor.
 * Built for dk and dv of 64 or 128 each.  The strides are at least a token's
 * elements and below 2^22; x_stride, b_stride and c_stride are whole 16-byte
 * units; H is a multiple of G, and H * dv is below 2^22; B * H is below 2^23, T
 * at most 2^31 - 1025 (GDN2_ERR_SHAPE, or GDN2_ERR_MISALIGNED).  dt needs the
 * alignment of its elements only.  A NaN or an infinity reaches no earlier token:
 * in x its column of y and of the state from its token on, in c its token's y, in
 * b and dt the y and states of their heads from their token on.
 * With workspace = NULL and workspace_bytes = 0 every sequence is walked whole.
 * With a workspace of gdn2_ssm_fwd_workspace_bytes bytes (256-byte aligned,
 * overlapping no argument) sequences are cut into segments that are walked in
 * parallel.  A shorter workspace, or one where that call says 0, returns
 * GDN2_ERR_WORKSPACE.
 */
gdn2_status_t gdn2_ssm_fwd(const void* x, const void* dt, const void* b, const void* c,
                           const float* A, const float* D, const float* dt_bias,
                           const float* initial_state, void* y, float* final_state, int64_t B,
                           int64_t T, int64_t H, int64_t G, int64_t dk, int64_t dv,
                           int64_t x_stride, int64_t dt_stride, int64_t b_stride, int64_t c_stride,
                           gdn2_dtype_t dtype, int softplus, void* workspace,
                           size_t workspace_bytes, void* stream);

/* The workspace with which gdn2_ssm_fwd is fastest for these sizes on the
 * current device: 0 where the (sequence, head) chains fill it by themselves. */
size_t gdn2_ssm_fwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv,
                                    gdn2_dtype_t dtype);

/*
 * gdn2_ssm_fwd_varlen -- the scan over N sequences packed along one token axis:
 * tensors as above with [total_T, ...] for [B, T, ...] and states [N, H, dk, dv];
 * cu_seqlens as for gdn2_chunk_fwd_varlen (int64 [N + 1] in device memory, each
 * range clamped into [0, total_T]; tokens of no sequence are left as they were
 * in y; an empty sequence hands its initial state on).  The workspace works as
 * for gdn2_ssm_fwd: without one every sequence is walked whole, with one of
 * gdn2_ssm_fwd_varlen_workspace_bytes bytes the long ones are cut.
 */
gdn2_status_t gdn2_ssm_fwd_varlen(const void* x, const void* dt, const void* b, const void* c,
                                  const float* A, const float* D, const float* dt_bias,
                                  const float* initial_state, void* y, float* final_state,
                                  const int64_t* cu_seqlens, int64_t N, int64_t total_T, int64_t H,
                                  int64_t G, int64_t dk, int64_t dv, int64_t x_stride,
                                  int64_t dt_stride, int64_t b_stride, int64_t c_stride,
                                  gdn2_dtype_t dtype, int softplus, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* The workspace with which gdn2_ssm_fwd_varlen is fastest for these sizes on the
 * current device (0 where no sequence of total_T tokens would be cut). */
size_t gdn2_ssm_fwd_varlen_workspace_bytes(int64_t N, int64_t total_T, int64_t H, int64_t dk,
                                           int64_t dv, gdn2_dtype_t dtype);

/* gdn2_ssm_step -- one token for each of N sequences: x [N, H, dv], dt [N, H],
 * b, c [N, G, dk], y [N, H, dv]; state [N, H, dk, dv] is updated in place.
 * Strides below 2^31: the last tokens of N prompts lie a prompt apart. */
gdn2_status_t gdn2_ssm_step(const void* x, const void* dt, const void* b, const void* c,
                            const float* A, const float* D, const float* dt_bias, float* state,
                            void* y, int64_t N, int64_t H, int64_t G, int64_t dk, int64_t dv,
                            int64_t x_stride, int64_t dt_stride, int64_t b_stride, int64_t c_stride,
                            gdn2_dtype_t dtype, int softplus, void* stream);

/*
 * gdn2_short_conv -- a causal depthwise convolution of four taps, with bias and
 * SiLU, that keeps its last inputs: gdn2_mixer_prep's convolution for channels
 * of any split and for sequences that go on.
 *
 *   y[t, i] = SiLU(bias[i] + sum_j taps[i, j] x[t - 3 + j, i]),  j = 0 .. 3
 *
 *   x             [B, T, C]  dtype    x_stride elements between tokens
 *   taps          [C, 4]     float32  (three taps: a first tap of zero)
 *   bias          [C]        float32  or NULL for zeros
 *   initial_state [B, 3, C]  dtype    the three inputs before the first token,
 *                                     oldest first; NULL for zeros
 *   y             [B, T, C]  dtype    out
 *   final_state   [B, 3, C]  dtype    out: the last three inputs, those of
 *                                     initial_state among them where T < 3; NULL
 *                                     to skip; may be the same pointer as
 *                                     initial_state
 *
 * C is a multiple of 8 below 2^22, x_stride at least C and below 2^22, and
 * B (ceil(T / 16) + 1) C / 4 is below 2^32 - 1024 (packed: (ceil(total_T / 16) + N)
 * C / 4), else GDN2_ERR_SHAPE.  x and its tokens need the alignment of their
 * elements only.
 */
gdn2_status_t gdn2_short_conv(const void* x, const float* taps, const float* bias,
                              const void* initial_state, void* y, void* final_state, int64_t B,
                              int64_t T, int64_t C, int64_t x_stride, gdn2_dtype_t dtype,
                              void* stream);

/* gdn2_short_conv_varlen -- the same over N packed sequences: x, y [total_T, C],
 * states [N, 3, C], cu_seqlens as for gdn2_ssm_fwd_varlen (offsets that decrease
 * leave the tokens between them unspecified). */
gdn2_status_t gdn2_short_conv_varlen(const void* x, const float* taps, const float* bias,
                                     const void* initial_state, void* y, void* final_state,
                                     const int64_t* cu_seqlens, int64_t N, int64_t total_T,
                                     int64_t C, int64_t x_stride, gdn2_dtype_t dtype, void* stream);

/* gdn2_short_conv_step -- one token for each of N sequences: x, y [N, C]; state
 * [N, 3, C] is updated in place.  x_stride below 2^31. */
gdn2_status_t gdn2_short_conv_step(const void* x, const float* taps, const float* bias, void* state,
                                   void* y, int64_t N, int64_t C, int64_t x_stride,
                                   gdn2_dtype_t dtype, void* stream);

/*
 * gdn2_layer_norm -- y = (x - mean) rstd gamma + beta over rows of `width`, with
 * rstd = 1 / sqrt(mean((x - mean)^2) + eps).
 *
 *   x, y        [rows, width]  dtype    y must not overlap an input
 *   gamma       [width]        float32
 *   beta        [width]        float32  or NULL for zeros
 *   mean, rstd  [rows]         float32  out, for the backward pass; both NULL to
 *                                       skip
 *
 * width may be any value from 1 to 16384, rows any from 0 on.  eps >= 0.
 */
gdn2_status_t gdn2_layer_norm(const void* x, const float* gamma, const float* beta, void* y,
                              float* mean, float* rstd, int64_t rows, int64_t width, float eps,
                              gdn2_dtype_t dtype, void* stream);

/* Bytes of device workspace that gdn2_layer_norm_bwd needs: partial sums of
 * dgamma and dbeta.  0 for few rows, and if the sizes are out of range. */
size_t gdn2_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t width);

/*
 * gdn2_layer_norm_bwd -- gradients of sum(dy * y) for gdn2_layer_norm.
 *
 *   dy, x       [rows, width]  dtype
 *   gamma       [width]        float32
 *   mean, rstd  [rows]         float32  as the forward pass gave them
 *   dx          [rows, width]  dtype    out; may not overlap an input
 *   dgamma      [width]        float32  out
 *   dbeta       [width]        float32  out, or NULL to skip
 *   workspace   16-byte aligned, overlapping no argument
 *
 * The sums over rows are formed in a fixed order: equal calls give equal bits.
 * With rows = 0 dgamma and dbeta are zeros.
 */
gdn2_status_t gdn2_layer_norm_bwd(const void* dy, const void* x, const float* gamma,
                                  const float* mean, const float* rstd, void* dx, float* dgamma,
                                  float* dbeta, void* workspace, size_t workspace_bytes,
                                  int64_t rows, int64_t width, gdn2_dtype_t dtype, void* stream);

/*
 * The attention block.  Hybrid stacks put attention over a sliding window
 * between the layers above (page "Why NVIDIA Gated DeltaNet-2 separates erase
 * and write gates", axbrief.com: a hybrid cell alternates the recurrence with
 * attention over a window of 2K tokens).  Such a layer is a norm with the
 * residual's addition, projections (the caller's), rotary positions and
 * attention.  These calls follow the conventions at the top; as in the state
 * space block, q, k and v may have a token stride of their own.
 */

/*
 * gdn2_attn_fwd -- causal attention of T queries over S keys in each of B
 * sequences.  Query t stands at position S - T + t of the S keys and sees the
 * keys at its own position and before it, with a window > 0 the last `window` of
 * them; head h of H reads key head h / (H / G) of G.
 *
 *   s_j = scale q . k_j,  o = sum_j e^(s_j - lse) v_j,  lse = log sum_j e^(s_j)
 *
 *   q     [B, T, H, d]  dtype    q_stride elements between tokens
 *   k, v  [B, S, G, d]  dtype    k_stride, v_stride
 *   o     [B, T, H, d]  dtype    out
 *   lse   [B, T, H]     float32  out, for the backward pass; or NULL to skip
 *
 * Built for d = 64 and 128, BF16 and F32.  T and S may be any sizes from 0 on, T
 * greater than S too: a query that sees no key (or none with a score above
 * minus infinity) has o = 0 and lse = -infinity.
 * A NaN or an infinity in k or v reaches no query that does not see it.
 * Finite values below 2^127 in size give a finite o where the scores are finite.  (A
 * query that sees values above 2^73 may take those below 2^-60 in its other channels
 * for zero.)
 * scale > 0.  H is a multiple of G; strides are at least a token's elements,
 * below 2^22 and whole 16-byte units; H * d is below 2^22, T and S at most
 * 2^31 - 1025, B * T below 2^29, and B * G * ceil(T / 128) * (H / G) and
 * B * G * ceil(S / 128) below 2^23 (GDN2_ERR_SHAPE, or GDN2_ERR_MISALIGNED).
 * With workspace = NULL and workspace_bytes = 0 a block of queries walks all its
 * keys.  With a workspace of gdn2_attn_fwd_workspace_bytes bytes (16-byte
 * aligned, overlapping no argument) the keys of few queries are taken in parts.
 * A shorter workspace, or one where that call says 0, returns
 * GDN2_ERR_WORKSPACE.
 */
gdn2_status_t gdn2_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B,
                            int64_t T, int64_t S, int64_t H, int64_t G, int64_t d, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, int64_t window, float scale,
                            gdn2_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream);

/* The workspace with which gdn2_attn_fwd is fastest for these sizes on the current
 * device: 0 where the blocks of queries fill it by themselves. */
size_t gdn2_attn_fwd_workspace_bytes(int64_t B, int64_t T, int64_t S, int64_t H, int64_t G, int64_t d,
                                     int64_t window, gdn2_dtype_t dtype);

/*
 * gdn2_attn_fwd_varlen -- the same over N sequences packed along the token axis:
 * sequence n has the queries [cu_seqlens[n], cu_seqlens[n + 1]) and the keys
 * [cu_seqlens_k[n], cu_seqlens_k[n + 1]) (both int64 [N + 1] in device memory; the
 * same pointer where the sequences stand alone).  q, o [total_T, H, d], k, v
 * [total_S, G, d], lse [total_T, H].  Each range is clamped into the tensor;
 * tokens of no sequence are left as they were in o and lse.  Offsets that
 * decrease or overlap leave results unspecified.  The conditions on sizes hold
 * with total_T / 128 + N for B * ceil(T / 128), and likewise for the keys.
 */
gdn2_status_t gdn2_attn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                                   const int64_t* cu_seqlens, const int64_t* cu_seqlens_k, int64_t N,
                                   int64_t total_T, int64_t total_S, int64_t H, int64_t G, int64_t d,
                                   int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t window,
                                   float scale, gdn2_dtype_t dtype, void* workspace,
                                   size_t workspace_bytes, void* stream);

size_t gdn2_attn_fwd_varlen_workspace_bytes(int64_t N, int64_t total_T, int64_t total_S, int64_t H,
                                            int64_t G, int64_t d, int64_t window, gdn2_dtype_t dtype);

/*
 * gdn2_attn_bwd -- gradients of sum(d_o * o) for gdn2_attn_fwd, from its o and lse.
 *
 *   d_o, o      [B, T, H, d]  dtype    q, k, v, lse and all sizes as above
 *   dq          [B, T, H, d]  dtype    out
 *   dk, dv      [B, S, G, d]  dtype    out, summed over the heads that share them
 *   workspace   16-byte aligned, overlapping no argument
 *
 * Sums are formed in a fixed order: equal calls give equal bits.  A NaN or an
 * infinity of one token reaches the gradients only of tokens that it sees or that
 * see it.
 */
gdn2_status_t gdn2_attn_bwd(const void* d_o, const void* q, const void* k, const void* v, const void* o,
                            const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t T,
                            int64_t S, int64_t H, int64_t G, int64_t d, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, int64_t window, float scale,
                            gdn2_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream);

/* gdn2_attn_bwd_varlen -- the same for gdn2_attn_fwd_varlen; gradients of tokens of no
 * sequence are left as they were. */
gdn2_status_t gdn2_attn_bwd_varlen(const void* d_o, const void* q, const void* k, const void* v,
                                   const void* o, const float* lse, void* dq, void* dk, void* dv,
                                   const int64_t* cu_seqlens, const int64_t* cu_seqlens_k, int64_t N,
                                   int64_t total_T, int64_t total_S, int64_t H, int64_t G, int64_t d,
                                   int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t window,
                                   float scale, gdn2_dtype_t dtype, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* Bytes of device workspace that they need for these sizes on the current device (0: none). */
size_t gdn2_attn_bwd_workspace_bytes(int64_t B, int64_t T, int64_t S, int64_t H, int64_t G, int64_t d,
                                     int64_t window, gdn2_dtype_t dtype);
size_t gdn2_attn_bwd_varlen_workspace_bytes(int64_t N, int64_t total_T, int64_t total_S, int64_t H,
                                            int64_t G, int64_t d, int64_t window, gdn2_dtype_t dtype);

/*
 * gdn2_attn_step -- attention of one token for each of N sequences over a cache of
 * its last C tokens, which the step's key and value join: the token at position p
 * lies in slot p mod C.
 *
 *   q                 [N, H, d]     dtype  q_stride elements between sequences
 *   k, v              [N, G, d]     dtype  the token's own; k_stride, v_stride
 *   k_cache, v_cache  [N, C, G, d]  dtype  slot p mod C is written
 *   positions         [N]           int64  p of each sequence's token, in device
 *                                          memory
 *   o                 [N, H, d]     dtype  out
 *
 * The token sees the last min(p + 1, C) tokens, itself among them, with a
 * window > 0 at most `window` of them.  A position below 0 is no token: its output is zero and its
 * cache is left as it was.  Slots behind a sequence's last token are not read.
 * Finite values below 2^127 over the number of tokens seen give a finite o.
 * Strides below 2^31, N * G * ceil(H / G / 32) below 2^23; otherwise as for
 * gdn2_attn_fwd.  With a workspace of gdn2_attn_step_workspace_bytes bytes (16-byte
 * aligned) a sequence's tokens are taken in parts; NULL and 0: whole.
 */
gdn2_status_t gdn2_attn_step(const void* q, const void* k, const void* v, void* k_cache, void* v_cache,
                             const int64_t* positions, void* o, int64_t N, int64_t H, int64_t G,
                             int64_t d, int64_t C, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                             int64_t window, float scale, gdn2_dtype_t dtype, void* workspace,
                             size_t workspace_bytes, void* stream);

/* The workspace with which gdn2_attn_step is fastest on the current device (0: none). */
size_t gdn2_attn_step_workspace_bytes(int64_t N, int64_t H, int64_t G, int64_t d, int64_t C,
                                      int64_t window, gdn2_dtype_t dtype);

/*
 * gdn2_rotary -- rotary positions on the first `rot` channels of the heads of q and k:
 *
 *   (a, b) -> scale (a cos t - b sin t, a sin t + b cos t),  t = position freq[i]
 *
 * for the pairs i of rot / 2: channels i and i + rot / 2, or with interleaved != 0
 * channels 2 i and 2 i + 1.  The other channels are copied.  inverse != 0 turns by
 * -t, which is the gradient of the call without it (scale is the same).
 *
 *   q, q_out   [tokens, H, d]  dtype    strides in elements between tokens
 *   k, k_out   [tokens, G, d]  dtype    G = 0: q alone
 *   freq       [rot / 2]       float32  radians a position
 *   positions  [tokens]        int64    or NULL: token n is at n mod T
 *
 * Angles are formed and reduced in 64 bits: off by 2^-51 of themselves, which stays
 * below fp32's own 2^-24 of a turn for angles up to 2^29 radians.  q_out may be q and
 * k_out k, with the same strides (in place; the channels from rot on are then not
 * touched); outputs may be parts of one wider tensor, but share no byte with
 * anything else.  rot is even, from 2 to d; d from 2 to 512; (H + G) d below 2^22;
 * strides at least a token's elements and below 2^31; tensors need the alignment
 * of their elements only.  scale > 0.  A launch has less than 2^32 threads: up to
 * 2^25 - 8 tokens are always taken, up to 2^27 - 8 where (H + G) d <= 192, and where
 * more would not fit they are refused (GDN2_ERR_SHAPE).
 */
gdn2_status_t gdn2_rotary(const void* q, const void* k, const float* freq, const int64_t* positions,
                          void* q_out, void* k_out, int64_t tokens, int64_t T, int64_t H, int64_t G,
                          int64_t d, int64_t rot, int64_t q_stride, int64_t k_stride,
                          int64_t q_out_stride, int64_t k_out_stride, int interleaved, int inverse,
                          float scale, gdn2_dtype_t dtype, void* stream);

/*
 * gdn2_rms_norm -- root-mean-square norm of a residual sum:
 *
 *   h = x + residual,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd gamma
 *
 *   x, y      [rows, width]  dtype           y must not overlap an input
 *   residual  [rows, width]  residual_dtype  (dtype or F32) or NULL: h = x
 *   gamma     [width]        float32
 *   h         [rows, width]  residual_dtype  out, with a residual; may be the same
 *                                            pointer as residual
 *   rstd      [rows]         float32         out, for the backward pass; NULL to skip
 *
 * y and rstd are formed from the sum before it is rounded to h, the sum of squares in
 * fp32: sizes below 2^63 / sqrt(width) are in its range.  width may be any value from
 * 1 to 16384, rows any from 0 on.  eps >= 0.
 */
gdn2_status_t gdn2_rms_norm(const void* x, const void* residual, const float* gamma, void* y, void* h,
                            float* rstd, int64_t rows, int64_t width, float eps, gdn2_dtype_t dtype,
                            gdn2_dtype_t residual_dtype, void* stream);

/* gdn2_rms_norm_fp8 -- the same with y in 8 bits (e4m3, [rows, width] bytes) and a scale for
 * each row (float32 [rows]): scale = max|y| / 448, or 1 for a row of zeros, and the byte is
 * the value nearest to y (448 / max|y|), y and both products rounded to fp32: where y / scale
 * is within 2^-22 of itself of the middle of two values it may be either.  (max|y| counts as
 * 2^-110 if it is less and not zero.) */
gdn2_status_t gdn2_rms_norm_fp8(const void* x, const void* residual, const float* gamma, void* y,
                                float* scales, void* h, float* rstd, int64_t rows, int64_t width,
                                float eps, gdn2_dtype_t dtype, gdn2_dtype_t residual_dtype, void* stream);

/* Bytes of device workspace that gdn2_rms_norm_bwd needs: partial sums of dgamma.  0 for
 * few rows, and if the sizes are out of range. */
size_t gdn2_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t width);

/*
 * gdn2_rms_norm_bwd -- gradients of sum(dy * y) + sum(dh * h) for gdn2_rms_norm:
 *
 *   dx = dh + rstd (v - u mean(u v)),  u = h rstd,  v = dy gamma   (of x and of the residual)
 *   dgamma = sum over rows of dy u
 *
 *   dy          [rows, width]  dtype
 *   h, dh, dx   [rows, width]  residual_dtype  dh may be NULL for zeros; dx may be dh
 *                                              (h = x without a residual)
 *   rstd        [rows]         float32         as the forward pass gave it
 *   gamma, dgamma  [width]     float32
 *   workspace   16-byte aligned, overlapping no argument
 *
 * The sums over rows are formed in a fixed order: equal calls give equal bits.
 * With rows = 0 dgamma is zeros.
 */
gdn2_status_t gdn2_rms_norm_bwd(const void* dy, const void* h, const float* gamma, const float* rstd,
                                const void* dh, void* dx, float* dgamma, void* workspace,
                                size_t workspace_bytes, int64_t rows, int64_t width, gdn2_dtype_t dtype,
                                gdn2_dtype_t residual_dtype, void* stream);

/* 1 if gdn2_chunk_fwd and gdn2_chunk_fwd_varlen (which = 0), gdn2_decode_step
 * (which = 1), gdn2_chunk_bwd (which = 2), gdn2_mixer_prep and gdn2_mixer_out
 * (which = 3), gdn2_ssm_fwd, gdn2_ssm_fwd_varlen and gdn2_ssm_step (which = 5) or the
 * gdn2_attn calls (which = 6, with dk = dv = d) support (dk, dv, dtype), else 0. */
int gdn2_supported(int which, int64_t dk, int64_t dv, gdn2_dtype_t dtype);

/* Static, NUL-terminated description of a status code. */
const char* gdn2_status_string(gdn2_status_t status);

/* Static version string of the library. */
const char* gdn2_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN2_H */
