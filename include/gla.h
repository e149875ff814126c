/*
 * gla.h - C ABI of the B200 (sm_100a) chunkwise Gated Linear Attention library.
 *
 * Operators
 * ---------
 * GLA (key-gated linear recurrence over a matrix memory, one head):
 *     S_t = diag(exp g_t) . S_{t-1} + k_t^T v_t ,      o_t = q_t . S_t
 *   q_t, k_t, g_t in R^dk, v_t in R^dv, S_t in R^{dk x dv}.
 *   Described in words by "Gated Linear Attention for Efficient Long Sequences" (panels "Core
 *   move" and "Step-by-step memory update") and by "MS-GLA: Multi-Scale Gated Linear
 *   Attention ...", section 2.1 (data-dependent forget gate that scales rows of the memory;
 *   chunkwise training with sequential inter-chunk and parallel intra-chunk work).
 * GSA (Gated Slot Attention, m memory slots):
 *     o1 = GLA_v(q, k, phi, g)  (pass 1: gate on the slot axis, which is the value axis)
 *     p  = softmax over the m slots of o1
 *     o  = GLA(p, phi, v, g)    (pass 2: keys phi, the same slot gates, now on the key axis)
 *   "Gated Slot Attention for Efficient Linear-Time Sequence Modeling", abstract (two-layer
 *   GLA linked via softmax) and "Approach" (two-pass linear attention, per-slot forget gates).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layout      Per-token tensors are contiguous [B, H, T, D] (D fastest).  States and their
 *             gradients (h0, hT, dhT, dh0, S) are contiguous float32 [B, H, rows, cols]:
 *             GLA [B,H,dk,dv]; GSA pass 1 [B,H,dk,m]; GSA pass 2 [B,H,m,dv].
 * dtype       GLA_DTYPE_BF16: q, k, v, g, phi, o, p and all per-token gradients are bf16;
 *             arithmetic accumulates in fp32.  GLA_DTYPE_F32: all of them are fp32 and no
 *             reduced-precision (bf16 or TF32) arithmetic is used anywhere.
 * Gate        g is the log of the decay (alpha = exp g).  It must be finite and <= 0;
 *             g = 0 means "keep", very negative g means "forget".  No scale is applied to q.
 * chunk       Chunk length of the chunkwise algorithm: 16, 32 or 64.  It changes rounding
 *             only, never the mathematical result.
 * Tails       T need not be a multiple of chunk.  T == 0 is allowed: per-token pointers may
 *             then be NULL, hT is set to h0 (or zeros) and dh0 to dhT (or zeros).
 * Optional    A NULL optional input means zeros (h0, dhT).  A NULL optional output is not
 *             written (hT, dh0, p_save).
 * Ownership   The caller owns every buffer, including the workspace; nothing is allocated,
 *             freed or retained by the library between calls.  Device pointers must be
 *             16-byte aligned.  Buffers of one call must not overlap, except where stated.
 * Streams     All work is enqueued on `stream` (a cudaStream_t passed as void*; NULL is the
 *             legacy default stream).  Calls return once the work is enqueued.
 * Workspace   `*_workspace()` returns the bytes the matching call needs for those sizes (0 is
 *             possible).  Pass at least that many bytes, 256-byte aligned.  The workspace
 *             contents on entry do not matter; on exit they are unspecified.
 * Errors      Invalid arguments are rejected before anything is enqueued:
 *               GLA_ERR_INVALID_ARG   NULL required pointer, negative or zero size where a
 *                                     positive one is required, misaligned pointer
 *               GLA_ERR_UNSUPPORTED   dtype, chunk or a dimension outside the supported set
 *               GLA_ERR_WORKSPACE     workspace NULL or smaller than *_workspace() returned
 *             A failed kernel launch returns GLA_ERR_CUDA.  Kernels never trap: every wait on
 *             an mbarrier is bounded, and a wait that runs out records GLA_ERR_TIMEOUT in a
 *             device-side latch that gla_device_error() reads.
 * Supported   1 <= dk, dv, m <= 512; dk, dv, m multiples of 8; B*H <= 2^31-1.
 */
#ifndef GLA_B200_H
#define GLA_B200_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GLA_OK = 0,
  GLA_ERR_INVALID_ARG = 1,
  GLA_ERR_UNSUPPORTED = 2,
  GLA_ERR_WORKSPACE = 3,
  GLA_ERR_CUDA = 4,
  GLA_ERR_TIMEOUT = 5
} gla_status;

typedef enum { GLA_DTYPE_F32 = 0, GLA_DTYPE_BF16 = 1 } gla_dtype;

/* Human-readable name of a status code (static string, never NULL). */
const char* gla_status_string(int status);

/* Library ABI version: major * 10000 + minor * 100 + patch. */
int gla_version(void);

/* ---------------------------------------------------------------------------------------
 * gla_chunk_fwd - chunkwise GLA forward.
 *   in : q, k, g [B,H,T,dk]; v [B,H,T,dv]; h0 [B,H,dk,dv] fp32 (optional, NULL = zeros)
 *   out: o [B,H,T,dv]; hT = S_T [B,H,dk,dv] fp32 (optional)
 * Chunkwise form ("MS-GLA", section 2.1): the state is carried chunk to chunk; inside a chunk
 * the output is the inter-chunk term (q * exp(b)) S_in plus the gated causal intra-chunk term.
 * ------------------------------------------------------------------------------------- */
size_t gla_chunk_fwd_workspace(int B, int H, int T, int dk, int dv, int chunk, int dtype);
int gla_chunk_fwd(const void* q, const void* k, const void* v, const void* g, const float* h0,
                  void* o, float* hT, int B, int H, int T, int dk, int dv, int chunk, int dtype,
                  void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------------------
 * gla_chunk_bwd - gradients of L(o, hT) for the same inputs as gla_chunk_fwd.
 *   in : q, k, g, v, h0 (optional) as in gla_chunk_fwd; dO [B,H,T,dv];
 *        dhT [B,H,dk,dv] fp32 (optional, NULL = zeros)
 *   out: dq, dk, dg [B,H,T,dk]; dv [B,H,T,dv]; dh0 [B,H,dk,dv] fp32 (optional)
 * The reverse-mode recurrence is derived from the forward recurrence; dg is the reverse
 * cumulative sum over t of q*dq - k*dk plus, for every t, sum_j dhT[i,j] hT[i,j].
 * It is the gradient of the same chunkwise form ("MS-GLA", section 2.1: chunkwise parallel
 * training of the gated recurrence, sequential across chunks and parallel inside a chunk),
 * evaluated chunk by chunk in reverse with the state gradient kept on chip ("Gated Linear
 * Attention for Efficient Long Sequences", "Why chunking and SRAM locality matter": only
 * inputs and gradients cross HBM, no per-step state is written).
 * ------------------------------------------------------------------------------------- */
size_t gla_chunk_bwd_workspace(int B, int H, int T, int dk, int dv, int chunk, int dtype);
int gla_chunk_bwd(const void* q, const void* k, const void* v, const void* g, const float* h0,
                  const void* dO, const float* dhT, void* dq, void* dk, void* dv, void* dg,
                  float* dh0, int B, int H, int T, int dk_dim, int dv_dim, int chunk, int dtype,
                  void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------------------
 * gla_chunk_fwd_logit / gla_chunk_bwd_logit - gla_chunk_fwd / gla_chunk_bwd with the gate given
 * as raw logits: x [B,H,T,dk] in place of g, with g = logsigmoid(x) / tau formed inside the
 * kernels' gate runs ("MS-GLA", section 2.1: a data-dependent forget gate; "Gated Slot
 * Attention ...", "Approach": sigmoid forget gates, alpha = sigmoid(x)^(1/tau)).  The log-gates
 * equal, value for value, what gla_gate_logsigmoid stores for x (so these calls return exactly
 * what gla_gate_logsigmoid followed by gla_chunk_fwd / gla_chunk_bwd returns), without that
 * pass's trip through memory.  The backward writes dx = dg * sigmoid(-x) / tau into `dx` in
 * place of dg.  tau > 0 and finite (else GLA_ERR_INVALID_ARG).  Everything else, including the
 * errors, as for gla_chunk_fwd / gla_chunk_bwd; the workspace is what the *_logit_workspace()
 * query returns (the shapes the generic kernels serve need room for g behind their own).
 * ------------------------------------------------------------------------------------- */
size_t gla_chunk_fwd_logit_workspace(int B, int H, int T, int dk, int dv, int chunk, int dtype);
int gla_chunk_fwd_logit(const void* q, const void* k, const void* v, const void* x, float tau,
                        const float* h0, void* o, float* hT, int B, int H, int T, int dk, int dv,
                        int chunk, int dtype, void* workspace, size_t workspace_bytes, void* stream);
size_t gla_chunk_bwd_logit_workspace(int B, int H, int T, int dk, int dv, int chunk, int dtype);
int gla_chunk_bwd_logit(const void* q, const void* k, const void* v, const void* x, float tau,
                        const float* h0, const void* dO, const float* dhT, void* dq, void* dk,
                        void* dv, void* dx, float* dh0, int B, int H, int T, int dk_dim,
                        int dv_dim, int chunk, int dtype, void* workspace, size_t workspace_bytes,
                        void* stream);

/* ---------------------------------------------------------------------------------------
 * gla_recurrent_step - one token of recurrent inference, in place on the state.
 *   in : q, k, g [B,H,dk]; v [B,H,dv]; S [B,H,dk,dv] fp32 (read, then overwritten)
 *   out: o [B,H,dv];  S <- diag(exp g) S + k^T v ; o = q S
 * "MS-GLA", section 1 (O(1) inference memory per token).  No workspace.  S may not alias
 * any other argument.
 * ------------------------------------------------------------------------------------- */
int gla_recurrent_step(const void* q, const void* k, const void* v, const void* g, float* S,
                       void* o, int B, int H, int dk, int dv, int dtype, void* stream);

/* ---------------------------------------------------------------------------------------
 * gsa_fwd - Gated Slot Attention forward.
 *   in : q, k [B,H,T,dk]; v [B,H,T,dv]; phi, g [B,H,T,m] (g: per-slot log forget gate);
 *        h0_1 [B,H,dk,m], h0_2 [B,H,m,dv] fp32 (optional)
 *   out: o [B,H,T,dv]; p_save [B,H,T,m] (optional: the slot softmax p, in dtype);
 *        hT1 [B,H,dk,m], hT2 [B,H,m,dv] fp32 (optional)
 * "Gated Slot Attention ...", abstract (a two-layer GLA linked via softmax) and "Approach"
 * (two-pass linear attention with a softmax in between; a data-dependent forget gate per
 * slot; reuses GLA's chunkwise training form): pass 1 writes k into the m slots weighted by
 * phi under the slot gates and reads them with q; the softmax over the slots gives p; pass 2
 * reads the values written under the same gates with p.
 * ------------------------------------------------------------------------------------- */
size_t gsa_fwd_workspace(int B, int H, int T, int dk, int dv, int m, int chunk, int dtype);
int gsa_fwd(const void* q, const void* k, const void* v, const void* phi, const void* g,
            const float* h0_1, const float* h0_2, void* o, void* p_save, float* hT1, float* hT2,
            int B, int H, int T, int dk, int dv, int m, int chunk, int dtype, void* workspace,
            size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------------------
 * gsa_bwd - gradients of L(o, hT1, hT2) for the inputs of gsa_fwd.
 *   in : as gsa_fwd, plus dO [B,H,T,dv]; dhT1 [B,H,dk,m], dhT2 [B,H,m,dv] fp32 (optional)
 *   out: dq, dk [B,H,T,dk]; dv [B,H,T,dv]; dphi, dg [B,H,T,m];
 *        dh0_1 [B,H,dk,m], dh0_2 [B,H,m,dv] fp32 (optional)
 * Pass 2 is differentiated first, then the softmax Jacobian do1 = p * (dp - <p, dp>), then
 * pass 1; dphi and dg sum the contributions of both passes.  The reverse mode of the two-pass
 * form of "Gated Slot Attention ...", "Approach" (two GLA passes sharing the per-slot forget
 * gates, joined by a softmax over the slots); each pass's gradient is that of a chunkwise GLA
 * ("MS-GLA", section 2.1).
 * ------------------------------------------------------------------------------------- */
size_t gsa_bwd_workspace(int B, int H, int T, int dk, int dv, int m, int chunk, int dtype);
int gsa_bwd(const void* q, const void* k, const void* v, const void* phi, const void* g,
            const float* h0_1, const float* h0_2, const void* dO, const float* dhT1,
            const float* dhT2, void* dq, void* dk, void* dv, void* dphi, void* dg, float* dh0_1,
            float* dh0_2, int B, int H, int T, int dk_dim, int dv_dim, int m, int chunk,
            int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------------------
 * gsa_recurrent_step - one token of GSA recurrent inference, in place on both states.
 *   in : q, k [B,H,dk]; v [B,H,dv]; phi, g [B,H,m];
 *        S1 [B,H,dk,m], S2 [B,H,m,dv] fp32 (read, then overwritten)
 *   out: o [B,H,dv]
 *   S1 <- S1 diag(exp g) + k^T phi ; p = softmax(q S1) ; S2 <- diag(exp g) S2 + phi^T v ;
 *   o = p S2.  "Gated Slot Attention ...", abstract (efficient recurrent inference with a
 *   small state).  No workspace.
 * ------------------------------------------------------------------------------------- */
int gsa_recurrent_step(const void* q, const void* k, const void* v, const void* phi,
                       const void* g, float* S1, float* S2, void* o, int B, int H, int dk,
                       int dv, int m, int dtype, void* stream);

/* ---------------------------------------------------------------------------------------
 * gla_chunk_bwd_noalloc - gla_chunk_bwd without a workspace argument, for callers that cannot
 * provide one.  (A library entry point only; the source pages have no counterpart of it.)
 *
 * Who needs it: callers that have no means to obtain device memory for a workspace, such as a
 * plain C host without a device allocator, a runtime that has carved up device memory in advance
 * and hands it out only for tensors, or code that must not call cudaMalloc because that call may
 * synchronise the device while its work is in flight.
 * What it uses instead: a fixed 128 MiB scratch array compiled into the library, reserved on
 * every device that loads this part of the library and held until the process exits.  The first
 * call on a device looks up that array's device address (cudaGetSymbolAddress); make the first
 * call on each device before any stream capture.  All calls share the array: calls that overlap
 * on the GPU (different streams or host threads) race on it.  Nothing in it needs to start at zero.
 * Arguments, layouts and outputs are those of gla_chunk_bwd.  Supported: bf16, chunk 64,
 * d_k = 128, d_v in {128, 256}, T >= 1 (else GLA_ERR_UNSUPPORTED / GLA_ERR_INVALID_ARG), and
 * scratch within the 128 MiB (else GLA_ERR_WORKSPACE): the bytes gla_chunk_bwd_workspace()
 * reports for the same sizes, (66 + d_v/2 + d_v/64)*B*H*ceil(T/64)*d_k*4 + nseg*B*H*d_k*4 +
 * 16640*B*H*ceil(T/64) (seven parts, each rounded up to 256 bytes), plus 2*nseg*B*H*d_k*d_v*4 +
 * nseg*B*H*d_k*4 when few heads leave SMs idle and the sequence is split into nseg segments.
 * It allocates nothing.
 * ------------------------------------------------------------------------------------- */
int gla_chunk_bwd_noalloc(const void* q, const void* k, const void* v, const void* g, const float* h0,
                          const void* dO, const float* dhT, void* dq, void* dk, void* dv, void* dg,
                          float* dh0, int B, int H, int T, int dk_dim, int dv_dim, int chunk, int dtype,
                          void* stream);

/* ---------------------------------------------------------------------------------------
 * gla_gate_logsigmoid - raw-logit gate entry: g = logsigmoid(x) / tau, element by element.
 * The operators take the log-gate g (alpha = exp g <= 1); models build it from a logit x as
 * log(sigmoid(x)) / tau ("MS-GLA ...", section 2.1: data-dependent forget gate; "Gated Slot
 * Attention ...", "Approach": sigmoid forget gates, alpha = sigmoid(x)^(1/tau)).
 *   x, g   n values of `dtype` (any layout; g may alias x).  tau > 0 and finite.
 * n == 0 enqueues nothing.  Errors: GLA_ERR_INVALID_ARG (NULL or misaligned pointer with
 * n > 0, tau not positive), GLA_ERR_UNSUPPORTED (dtype).  No workspace.
 * ------------------------------------------------------------------------------------- */
int gla_gate_logsigmoid(const void* x, void* g, size_t n, float tau, int dtype, void* stream);

/* gla_gate_logsigmoid_bwd - its backward: dx = dg * sigmoid(-x) / tau (dx may alias dg). */
int gla_gate_logsigmoid_bwd(const void* x, const void* dg, void* dx, size_t n, float tau, int dtype,
                            void* stream);

/* ---------------------------------------------------------------------------------------
 * MS-GLA temporal pooling and causal hold ("MS-GLA: Multi-Scale Gated Linear Attention ...",
 * sections 3.1 and 3.3), the reshaping around a GLA branch that runs at scale s.
 *   gla_msgla_pool       x [B,H,T,D] -> y [B,H,P,D], P = ceil(T/s): y_p is the mean of tokens
 *                        p*s .. min(T,(p+1)*s)-1 (a short last block averages only its tokens).
 *   gla_msgla_pool_bwd   dy [B,H,P,D] -> dx [B,H,T,D]: dx_t = dy_{t/s} / (tokens in block t/s).
 *   gla_msgla_hold       y [B,H,P,D] -> out [B,H,T,D]: out_t = y_{(t+1)/s - 1}, zeros while
 *                        (t+1)/s = 0 (a block is visible from its last token on).
 *   gla_msgla_hold_bwd   dout [B,H,T,D] -> dy [B,H,P,D]: the transpose (sum over the tokens that
 *                        read block p).
 * Arguments are (in, out, B, H, T, D, s, dtype, stream) for all four; in and out must not
 * overlap.  D in 8..512, a multiple of 8; s >= 1; T == 0 enqueues nothing.  Errors as for the
 * operators.  No workspace.
 * ------------------------------------------------------------------------------------- */
int gla_msgla_pool(const void* x, void* y, int B, int H, int T, int D, int s, int dtype, void* stream);
int gla_msgla_pool_bwd(const void* dy, void* dx, int B, int H, int T, int D, int s, int dtype, void* stream);
int gla_msgla_hold(const void* y, void* out, int B, int H, int T, int D, int s, int dtype, void* stream);
int gla_msgla_hold_bwd(const void* dout, void* dy, int B, int H, int T, int D, int s, int dtype,
                       void* stream);

/* ---------------------------------------------------------------------------------------
 * gla_scan_* - the elementwise gated linear recurrence: a state of one value per channel instead
 * of a matrix, scanned over the sequence.
 *     h_t = a_t h_{t-1} + b_t ,   o_t = h_t ,   a_t = exp g_t
 *     b_t = x_t                 (GLA_SCAN_ADD)
 *     b_t = (1 - a_t) x_t       (GLA_SCAN_COMPLEMENT: the input gate is what the forget gate leaves;
 *                                1 - a is formed without cancellation for g near 0)
 * The gate is the log of the decay as for gla_chunk_fwd ("MS-GLA", section 2.1: a data-dependent
 * forget gate), g <= 0; here g = -inf is allowed too and restarts the channel at that token (packed
 * sequences), provided the state before it is finite.
 *   gla_scan_fwd   in : g, x [B,H,T,D]; h0 [B,H,D] fp32 (optional)
 *                  out: o [B,H,T,D]; hT [B,H,D] fp32 (optional);
 *                       hc [B,H,ceil(T/64),D] fp32 (optional): the state before tokens 0, 64, 128, ...
 *   gla_scan_bwd   in : g, x, h0 as above; hc as gla_scan_fwd wrote it (optional: when it is NULL the
 *                       states are recomputed from g, x and h0 into the workspace, else h0 is not read);
 *                       dO [B,H,T,D]; dhT [B,H,D] fp32 (optional)
 *                  out: dg, dx [B,H,T,D]; dh0 [B,H,D] fp32 (optional)
 *                  with d_t = dO_t + a_{t+1} d_{t+1} (the last token's also takes dhT):
 *                  dx = d, dg = a h_{t-1} d  or, for the complement, dx = (1 - a) d,
 *                  dg = a (h_{t-1} - x) d;  dh0 = a_1 d_1.
 *   gla_scan_step  one token: g, x [B,H,D], S [B,H,D] fp32 (read, then overwritten), o [B,H,D].
 * A model without heads passes its [B,T,C] tensors as H = 1, D = C.  D >= 1 and B*H*ceil(D/16) <=
 * 2^27 (else GLA_ERR_UNSUPPORTED); T == 0 as for gla_chunk_fwd.  Pointers of these and the following
 * operators need the alignment of their element type only; 16-byte aligned ones with rows of a
 * multiple of 16 bytes run the vector form.  Results do not depend on the number of SMs or on the
 * order in which blocks run; a tensor off its alignment may give other last bits than an aligned copy.
 * At fp32 a and 1 - a are off by a few 2^-24 of themselves for every g (an a below 2^-126 is zero); at bf16
 * a by 2^-22 + |g| 2^-24 and 1 - a by 2^-20.7.
 * ------------------------------------------------------------------------------------- */
typedef enum { GLA_SCAN_ADD = 0, GLA_SCAN_COMPLEMENT = 1 } gla_scan_input;

int gla_scan_fwd(const void* g, const void* x, const float* h0, void* o, float* hT, float* hc, int B, int H,
                 int T, int D, int input, int dtype, void* stream);
size_t gla_scan_bwd_workspace(int B, int H, int T, int D, int have_hc);
int gla_scan_bwd(const void* g, const void* x, const float* h0, const float* hc, const void* dO,
                 const float* dhT, void* dg, void* dx, float* dh0, int B, int H, int T, int D, int input,
                 int dtype, void* workspace, size_t workspace_bytes, void* stream);
int gla_scan_step(const void* g, const void* x, float* S, void* o, int B, int H, int D, int input, int dtype,
                  void* stream);

/* ---------------------------------------------------------------------------------------
 * gla_group_norm_* - the norm and output gate behind a recurrence: every head's D outputs of a
 * token are one group, normalised on their own, scaled, gated, and left channels last for the output
 * projection (statistics over the tokens would let a causal model see the future).
 *     n = (x - mean) / sqrt(var + eps)          GLA_NORM_GROUP (var is the biased variance)
 *     n = x / sqrt(mean(x^2) + eps)             GLA_NORM_RMS
 *     u = n * w + b ;   y = u * act(z)  or, without z,  y = act(u)
 *   act: GLA_ACT_NONE (identity), GLA_ACT_SILU, GLA_ACT_SIGMOID
 *   gla_group_norm_fwd  in : x in `layout` (GLA_LAYOUT_BHTD [B,H,T,D], what the operators above write,
 *                            or GLA_LAYOUT_BTHD [B,T,H,D]); z [B,T,H,D] (optional);
 *                            w, b [weight_rows, D] fp32 (optional: ones, zeros)
 *                       out: y [B,T,H,D]
 *   gla_group_norm_bwd  in : x, z, w, b, dy [B,T,H,D]
 *                       out: dx in `layout`; dz [B,T,H,D] (optional; needs z);
 *                            dw, db [weight_rows, D] fp32 (optional), summed in a fixed order
 * weight_rows: H (a weight for each channel) or 1 (one row shared by the heads).  1 <= D <= 8192,
 * H <= 65535 and B*T <= 2^31-1 (else GLA_ERR_UNSUPPORTED); eps > 0 and finite.  T == 0: dw and db are zeroed, nothing else is
 * written.  Statistics and sums are fp32.  Workspace of the backward: per-block partial sums of dw
 * and db (0 bytes when neither is asked for).
 * ------------------------------------------------------------------------------------- */
typedef enum { GLA_NORM_GROUP = 0, GLA_NORM_RMS = 1 } gla_norm_kind;
typedef enum { GLA_ACT_NONE = 0, GLA_ACT_SILU = 1, GLA_ACT_SIGMOID = 2 } gla_activation;
typedef enum { GLA_LAYOUT_BHTD = 0, GLA_LAYOUT_BTHD = 1 } gla_layout;

int gla_group_norm_fwd(const void* x, const void* z, const float* w, const float* b, void* y, int B, int H,
                       int T, int D, int weight_rows, int kind, int act, float eps, int layout, int dtype,
                       void* stream);
size_t gla_group_norm_bwd_workspace(int B, int H, int T, int D, int weight_rows, int need_dw, int need_db);
int gla_group_norm_bwd(const void* x, const void* z, const float* w, const float* b, const void* dy, void* dx,
                       void* dz, float* dw, float* db, int B, int H, int T, int D, int weight_rows, int kind,
                       int act, float eps, int layout, int dtype, void* workspace, size_t workspace_bytes,
                       void* stream);

/* ---------------------------------------------------------------------------------------
 * gla_rotary - rotary positions of q and, in the same launch, k.
 *     (u_i, v_i) <- scale * (u_i cos A_i - v_i sin A_i,  v_i cos A_i + u_i sin A_i),  A_i = p * freq_i
 * for the R/2 pairs of the first R channels of every head: (u_i, v_i) are channels (i, i + R/2), or
 * (2i, 2i + 1) when `interleaved`.  Channels R .. D-1 are copied as they are.
 *   in : q [B,Hq,T,D], k [B,Hk,T,D] (NULL with Hk = 0) in `in_layout`; freq [R/2] float64, radians a
 *        position; pos int64: NULL with pos_rows = 0 (p = pos0 + t), [T] with pos_rows = 1 or [B,T]
 *        with pos_rows = B (p = pos0 + pos)
 *   out: qo, ko in `out_layout`; with equal layouts qo = q and ko = k (in place) are allowed
 * The angle is formed and reduced to a turn in 64 bits, and rounded to 32 bits of a turn: it is off by
 * |p freq| 2^-52 + |p| 2^-62 + 2^-30 radians at most, so far positions keep fp32 accuracy relative to |u| + |v|;
 * freq has to be finite.  The rotation is fp32 and rounded once.
 * inverse != 0 rotates by -A with the same scale, which is the transpose: the backward of a call is
 * the call with inverse set and the layouts exchanged.  1 <= D <= 8192, R even, 2 <= R <= D; scale
 * finite; B*T and B*T*ceil(D/2) at most 2^31 - 512 (else GLA_ERR_UNSUPPORTED).  T == 0 enqueues nothing.
 * ------------------------------------------------------------------------------------- */
int gla_rotary(const void* q, const void* k, void* qo, void* ko, const double* freq, const long long* pos,
               long long pos0, int pos_rows, int B, int Hq, int Hk, int T, int D, int R, float scale,
               int interleaved, int inverse, int in_layout, int out_layout, int dtype, void* stream);

/* ---------------------------------------------------------------------------------------
 * gla_device_error - read (and optionally clear) the device-side error latch.
 * Synchronises `stream`, then stores GLA_OK or the first error a kernel recorded since the
 * last reset (GLA_ERR_TIMEOUT: a bounded wait ran out) in *code.  Returns GLA_ERR_CUDA if
 * the copy fails, GLA_ERR_INVALID_ARG if code is NULL, else GLA_OK.
 * ------------------------------------------------------------------------------------- */
int gla_device_error(void* stream, int reset, int* code);

#ifdef __cplusplus
}
#endif

#endif /* GLA_B200_H */
