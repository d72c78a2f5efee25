/*
 * gbla.h — C ABI of the GB300 (sm_103a) Gated Bidirectional Linear Attention
 * (GBLA) layer library, libgbla.so.
 *
 * What the layer computes ("Gated Bidirectional Linear Attention for
 * Generative Retrieval", section "Core method"), per sequence and head h:
 *   Eq. 4  x~ = Conv1d(x);  q = x~ W_Q^h,  k = x~ W_K^h,  v = x~ W_V^h
 *   Eq. 5  g_j = gate(x~_j . w_g^h)  (sigmoid with bias, or softmax over the
 *          sequence, see gbla_gate)
 *   Eq. 6  q~ = phi(q), k~_j = g_j phi(k_j), phi = elu + 1;
 *          S = sum_j k~_j v_j^T (d_h x d_h),  z = sum_j k~_j,
 *          o_i = q~_i^T S / q~_i^T z        (global, non-causal: bidirectional)
 *   Eq. 7  y = RmsNorm(o) (.) gamma (.) SiLU(x~ W_R^h)
 *   "Multi-head" paragraph: each head owns its W_Q^h, W_K^h, W_V^h, w_g^h, W_R^h.
 * The heads' outputs are concatenated: y is [tokens, H*d_h].  No output
 * projection, residual or FFN is part of this library.
 *
 * Conventions shared by every call
 * --------------------------------
 * - Every tensor pointer is a DEVICE pointer owned by the caller.  The library
 *   allocates no device memory: scratch comes from the caller's workspace
 *   `ws` of `ws_bytes` bytes, sized by gbla_workspace_size().  The workspace
 *   need not be zeroed and must be 256-byte aligned.
 * - All calls are asynchronous on the caller's CUDA stream (`stream` is a
 *   cudaStream_t passed as void*; NULL = the legacy default stream).  Calls
 *   that share a workspace must be stream-ordered.  The library keeps no state
 *   between calls; results are deterministic (bitwise reproducible for the same
 *   shape and inputs): no floating-point atomics are used.
 * - Row-major layouts.  Token-major tensors have one row per token: in the
 *   dense and padded forms there are B*L rows (sequence b owns rows b*L ..
 *   b*L+L-1); in the varlen form there are T = L rows and sequence b owns
 *   rows cu_seqlens[b] .. cu_seqlens[b+1]-1.
 * - Weights use the x W convention: W_* is [d, H*d_h] and column block
 *   h*d_h .. h*d_h+d_h-1 belongs to head h; w_g is [d, H].
 * - dtypes: tensors named "(io)" have the shape's io_dtype (fp32 or bf16);
 *   gate values g, logits, den, state and every PARAMETER GRADIENT are fp32.
 *   Accumulation is fp32 everywhere.
 * - Padding and varlen: rows that belong to no sequence (a padded row, i.e.
 *   position >= seq_lens[b]) get zero outputs and zero input gradients.  The
 *   conv window and the state sums never cross a sequence boundary.
 * - Errors: argument errors are detected on the host before anything is
 *   launched and returned as a status.  A launch failure returns
 *   GBLA_ERR_CUDA (gbla_last_error() gives the CUDA text).  Bad sequence data
 *   that only the device can see (cu_seqlens not starting at 0, decreasing,
 *   or not ending at T; seq_lens outside [0, L]) sets an error word in the
 *   workspace, every kernel then skips its work, and gbla_check_device_status()
 *   reports GBLA_ERR_DEVICE_CHECK.  No kernel traps, and none waits on another
 *   CTA but those of glr_forward and glr_backward, whose tiles wait for the
 *   states of tiles handed out before them (a bounded wait, as below).
 *   The tensor-core kernels wait on their own copies and MMAs through
 *   mbarriers; every such wait is bounded, and one that gives up (a device
 *   that stopped making progress) sets a timeout bit in the error word instead
 *   of hanging: gbla_check_device_status() then reports GBLA_ERR_DEVICE_TIMEOUT.
 */
#ifndef GBLA_H
#define GBLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GBLA_OK = 0,
  GBLA_ERR_INVALID_ARG = -1,  /* null/misaligned pointer, bad dimension      */
  GBLA_ERR_UNSUPPORTED = -2,  /* a valid shape this build has no kernel for  */
  GBLA_ERR_WORKSPACE = -3,    /* ws NULL, misaligned, or ws_bytes too small  */
  GBLA_ERR_CUDA = -4,         /* a CUDA runtime call or launch failed        */
  GBLA_ERR_DEVICE_CHECK = -5, /* bad sequence data detected on the device   */
  GBLA_ERR_DEVICE_TIMEOUT = -6 /* a kernel's bounded wait gave up            */
} gbla_status;

typedef enum { GBLA_F32 = 0, GBLA_BF16 = 1 } gbla_dtype;

/* Key gate of Eq. 5.  SIGMOID: g = sigmoid(x~ . w_g + b_g) per token and head.
 * SOFTMAX: the pages' g = softmax_j(x~_j . w_g) over the valid tokens of each
 * sequence; its normaliser (and any b_g) cancels between the numerator and
 * denominator of Eq. 5, so the kernels use exp(s_j - m) with a per-sequence
 * running max m and db_g is 0. */
typedef enum { GBLA_GATE_SIGMOID = 0, GBLA_GATE_SOFTMAX = 1 } gbla_gate;

typedef enum {
  GBLA_OP_FORWARD = 0,        /* gbla_forward                                */
  GBLA_OP_BACKWARD = 1,       /* gbla_backward                               */
  GBLA_OP_CORE_FORWARD = 2,   /* bla_core_forward                            */
  GBLA_OP_CORE_BACKWARD = 3,  /* bla_core_backward                           */
  GBLA_OP_DECAY_FORWARD = 4,  /* bla_decay_core_forward                      */
  GBLA_OP_SA_FORWARD = 5,     /* sa_core_forward                             */
  GBLA_OP_GLR_FORWARD = 6,    /* glr_forward                                 */
  GBLA_OP_GLR_BACKWARD = 7    /* glr_backward                                */
} gbla_op;

typedef struct {
  int B;       /* batch (dense/padded forms); must be 1 with cu_seqlens       */
  int L;       /* tokens per sequence slot; with cu_seqlens: T, total rows    */
  int d;       /* model width (channels of x)                                 */
  int H;       /* heads                                                       */
  int d_h;     /* head width: bf16 {32, 64, 128}; fp32 1..128                 */
  const int32_t* cu_seqlens; /* device [num_seqs+1] or NULL (varlen form)     */
  int num_seqs;              /* sequences in the varlen form                  */
  const int32_t* seq_lens;   /* device [B] or NULL (padded form: valid rows)  */
  int io_dtype;              /* gbla_dtype                                    */
  int gate;                  /* gbla_gate                                     */
  float rms_eps;             /* RmsNorm epsilon (Eq. 7); e.g. 1e-6            */
} gbla_shape;

/* Bytes of workspace `ws` that call `op` needs for this shape (0 on a shape
 * error; check gbla_validate_shape). */
size_t gbla_workspace_size(const gbla_shape* shape, int op);

/* Bytes of the activation buffer that gbla_forward fills for gbla_backward
 * (x~, the q|k|v|r projections, the gate, the state).  Caller-owned. */
size_t gbla_saved_size(const gbla_shape* shape);

/* Host-side validation of a shape alone; GBLA_OK or the reason. */
gbla_status gbla_validate_shape(const gbla_shape* shape);

/*
 * Layer forward, Eq. 4-7.
 *   x       (io) [rows, d]
 *   conv_w  (io) [d, 4]   depthwise causal taps; tap t multiplies x[l-3+t]
 *   conv_b  (io) [d] or NULL (no bias)
 *   W_q, W_k, W_v, W_r (io) [d, H*d_h]
 *   w_g     (io) [d, H];  b_g (io) [H] or NULL (zero bias)
 *   rms_w   (io) [d_h] or NULL (ones): RmsNorm scale gamma, shared by heads
 *   y       (io) [rows, H*d_h]  output
 *   saved   NULL (inference) or gbla_saved_size() bytes, 256-byte aligned:
 *           filled for gbla_backward
 * bf16 requires every pointer 16-byte aligned and d % 64 == 0.
 */
gbla_status gbla_forward(const gbla_shape* shape, const void* x,
                         const void* conv_w, const void* conv_b,
                         const void* W_q, const void* W_k, const void* W_v,
                         const void* W_r, const void* w_g, const void* b_g,
                         const void* rms_w, void* y, void* saved, void* ws,
                         size_t ws_bytes, void* stream);

/*
 * Layer backward for the scalar <dy, y>: the same inputs as gbla_forward, the
 * `saved` buffer that a training forward of the same inputs filled, and dy
 * (io) [rows, H*d_h].  Outputs (any parameter gradient may be NULL to skip
 * writing it; dx is required):
 *   dx (io) [rows, d];  dconv_w fp32 [d, 4];  dconv_b fp32 [d];
 *   dW_q, dW_k, dW_v, dW_r fp32 [d, H*d_h];  dw_g fp32 [d, H];  db_g fp32 [H];
 *   drms_w fp32 [d_h].
 * Gradients overwrite (they are not accumulated into).
 */
gbla_status gbla_backward(const gbla_shape* shape, const void* x,
                          const void* conv_w, const void* conv_b,
                          const void* W_q, const void* W_k, const void* W_v,
                          const void* W_r, const void* w_g, const void* b_g,
                          const void* rms_w, const void* saved, const void* dy,
                          void* dx, float* dconv_w, float* dconv_b,
                          float* dW_q, float* dW_k, float* dW_v, float* dW_r,
                          float* dw_g, float* db_g, float* drms_w, void* ws,
                          size_t ws_bytes, void* stream);

/*
 * The gated BLA core alone, Eq. 5/6, from raw projections:
 *   q, k, v (io) [rows, H*d_h]  (phi is applied inside)
 *   g       fp32 [rows, H]      gate VALUES g_j >= 0 (not logits)
 *   o       (io) [rows, H*d_h]  o_i = phi(q_i)^T S / phi(q_i)^T z
 *   den     fp32 [rows, H] or NULL: phi(q_i)^T z
 *   state   fp32 [n_seq, H, d_h, d_h+1] or NULL: [S | z] (z = column d_h);
 *           n_seq = B, or num_seqs in the varlen form
 * The shape's d, gate and rms_eps are ignored.
 */
gbla_status bla_core_forward(const gbla_shape* shape, const void* q,
                             const void* k, const void* v, const float* g,
                             void* o, float* den, float* state, void* ws,
                             size_t ws_bytes, void* stream);

/*
 * Backward of bla_core_forward for the scalar <d_o, o>.
 *   d_o (io) [rows, H*d_h];  dq, dk, dv (io) [rows, H*d_h];  dg fp32 [rows, H]
 *   (the gradient with respect to the gate values g).
 * The state is recomputed from q, k, v, g.
 */
gbla_status bla_core_backward(const gbla_shape* shape, const void* q,
                              const void* k, const void* v, const float* g,
                              const void* d_o, void* dq, void* dk, void* dv,
                              float* dg, void* ws, size_t ws_bytes,
                              void* stream);

/*
 * The gated core under LION's decay masks ("Linear Attention for Efficient
 * Bidirectional Sequence Modeling": mask construction and the Lion-d /
 * Lion-s models), with this layer's phi = elu + 1 and key gate (Eq. 5):
 *   M^F_ij = prod_{t=j+1..i} lam_t (j <= i),  M^B_ij = prod_{t=i+1..j} lam_t (j >= i),
 *   M = M^F + M^B - I,
 *   o_i = sum_j M_ij g_j (phi(q_i).phi(k_j)) v_j / sum_j M_ij g_j (phi(q_i).phi(k_j)).
 * Lion-d passes one constant decay for every token (M_ij = lam^|i-j|), Lion-s
 * a decay per token (e.g. sigmoid(W x_t + b)); lam = 1 everywhere is
 * bla_core_forward.  Computed in the bidirectional chunkwise form: 128-row
 * chunks, their local states, a forward and a backward scan over the chunk
 * states, then each chunk's decayed attention plus the two scanned states.
 *   q, k, v (bf16) [rows, H*d_h] (phi is applied inside); g fp32 [rows, H]
 *   gate values >= 0; lam fp32 [rows, H] decays in [0, 1] (lam_t of a
 *   sequence's first token enters no product); o (bf16) [rows, H*d_h];
 *   den fp32 [rows, H] or NULL.
 *   bf16 I/O and d_h = 64 only (GBLA_ERR_UNSUPPORTED otherwise).  Workspace:
 *   gbla_workspace_size(shape, GBLA_OP_DECAY_FORWARD).  The shape's d, gate and
 *   rms_eps are ignored.
 */
gbla_status bla_decay_core_forward(const gbla_shape* shape, const void* q,
                                   const void* k, const void* v, const float* g,
                                   const float* lam, void* o, float* den,
                                   void* ws, size_t ws_bytes, void* stream);

/*
 * The attention of the SA blocks of the hybrid [SA, LA, LA] encoder: the
 * bidirectional softmax attention of Eq. 1 ("Gated Bidirectional Linear
 * Attention for Generative Retrieval", Core method 1; the hybrid encoder
 * interleaves one such block with two GBLA blocks):
 *   o_i = sum_j exp(q_i . k_j / sqrt(d_h)) v_j / sum_j exp(q_i . k_j / sqrt(d_h))
 * over every key j of query i's sequence, per head (no mask: both
 * directions).  Quadratic in the sequence length: the baseline the pages
 * compare GBLA with (Table 5, single-layer latency).
 *   q, k, v, o (bf16) [rows, H*d_h], head h at columns h*d_h .. h*d_h+d_h-1.
 *   Rows of a padded slot past its sequence get o = 0.
 *   bf16 I/O and d_h = 64 only (GBLA_ERR_UNSUPPORTED otherwise).  Workspace:
 *   gbla_workspace_size(shape, GBLA_OP_SA_FORWARD).  The shape's d, gate and
 *   rms_eps are ignored.
 */
gbla_status sa_core_forward(const gbla_shape* shape, const void* q,
                            const void* k, const void* v, void* o, void* ws,
                            size_t ws_bytes, void* stream);

/*
 * Gated linear recurrence: a state per channel that decays by an amount read
 * from the token, the token-by-token counterpart of the layer's global sums
 * (the same operator serves one token at a time: L = 1 with h0 and hT).  Per
 * sequence and channel, over the tokens t in order (reverse = 0) or from the
 * last to the first (reverse = 1; a bidirectional encoder runs both):
 *   s_t = c softplus(lam) sigmoid(r_t),  a_t = exp(-s_t),
 *   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,   y_t = h_t,
 * with h = h0 (or 0) before the sequence's first token.
 *   x, r, i (io) [rows, d] with row stride ld elements (ld >= d; ld = d when
 *           contiguous, ld = 3 d when x | r | i are columns of one
 *           projection): values and the logits of the two gates.  r = -inf
 *           gives a_t = 1 and leaves the state as it is for finite x and i.
 *   lam     fp32 [d]; c > 0 (e.g. 8)
 *   h0      fp32 [n_seq, d] or NULL (zeros); n_seq = B, or num_seqs (varlen)
 *   y       (io) [rows, d]
 *   hT      fp32 [n_seq, d] or NULL: the state after the sequence's last token
 *           in the recurrence's order (h0, or 0, where the sequence is
 *           empty).  hT may be h0: the state is then updated in place.
 *   saved   NULL (inference) or glr_saved_size() bytes, 256-byte aligned,
 *           filled for glr_backward
 * States, sums and gates are fp32; y is rounded once.  d and ld are free
 * (any d >= 1); the pointers are aligned to their element; tensors do not
 * overlap (but hT = h0).  The shape's H, d_h, gate and rms_eps are ignored
 * (gbla_validate_shape does not apply); rows <= 2^30, d <= 2^20.  Workspace:
 * gbla_workspace_size(shape, GBLA_OP_GLR_FORWARD).
 */
gbla_status glr_forward(const gbla_shape* shape, const void* x, const void* r,
                        const void* i, int64_t ld, const float* lam, float c,
                        int reverse, const float* h0, void* y, float* hT,
                        void* saved, void* ws, size_t ws_bytes, void* stream);

/* Bytes of the buffer that glr_forward fills for glr_backward (0 on a shape
 * error).  Caller-owned. */
size_t glr_saved_size(const gbla_shape* shape);

/*
 * Backward of glr_forward for the scalar <dy, y> + <dhT, hT>: the forward's
 * inputs (h0 as it was then: not one that the call updated in place), its
 * `saved` (of the same shape and direction), dy (io) [rows, d] and dhT fp32
 * [n_seq, d] or NULL (zeros).  Outputs:
 *   dx, dr, di (io) [rows, d] with row stride ldd (ldd >= d; e.g. the columns
 *   of one gradient matrix); dlam fp32 [d] or NULL; dh0 fp32 [n_seq, d] or
 *   NULL (an empty sequence's is its dhT).  Gradients overwrite.
 * Workspace: gbla_workspace_size(shape, GBLA_OP_GLR_BACKWARD).
 */
gbla_status glr_backward(const gbla_shape* shape, const void* x, const void* r,
                         const void* i, int64_t ld, const float* lam, float c,
                         int reverse, const float* h0, const void* saved,
                         const void* dy, const float* dhT, void* dx, void* dr,
                         void* di, int64_t ldd, float* dlam, float* dh0,
                         void* ws, size_t ws_bytes, void* stream);

/*
 * AdamW over many tensors at once: the update of the parameters whose
 * gradients gbla_backward and glr_backward return.  With t the step's number
 * (from 1), g the gradient times the clip factor, in fp32 whatever the types:
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2,
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps).
 * A tensor's m and v are fp32 (m_scale = v_scale = NULL), or 8-bit: m and
 * sqrt(v) as e4m3 values times an fp32 scale per block of
 * GBLA_ADAMW_BLOCK consecutive values (the block's largest magnitude / 448;
 * scale 0 and values 0 below 2^-100).  They are rounded up or down with the
 * odds of the remainder, by a hash of (seed, t, the value's place), because v
 * moves by a thousandth of itself a step and rounding to nearest would hold it
 * still; a sqrt(v) above 0 does not become 0.  The same call with the same
 * seed gives the same bits.  Zero-filled states (and scales) are the start.
 */
#define GBLA_ADAMW_BLOCK 256
typedef struct {
  void* param;        /* [n], param_dtype                                     */
  float* master;      /* [n] or NULL: the fp32 values that a bf16 param is
                         rounded from; without it bf16 values are updated     */
  const void* grad;   /* [n], grad_dtype                                      */
  void* m;            /* [n] fp32 or e4m3                                     */
  void* v;            /* [n] fp32, or e4m3 sqrt(v)                            */
  float* m_scale;     /* [ceil(n / GBLA_ADAMW_BLOCK)] or NULL: fp32 states    */
  float* v_scale;     /* as m_scale                                           */
  int64_t n;          /* values, >= 0                                         */
  int param_dtype;    /* gbla_dtype                                           */
  int grad_dtype;     /* gbla_dtype                                           */
  double weight_decay;
} gbla_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps; /* lr >= 0, 0 <= beta <= 0.9999999, eps >= 1e-30      */
  double max_norm;    /* > 0, with `norm`: gradients are scaled by
                         min(1, max_norm / (norm + 1e-6)); 0: no clipping     */
  uint32_t seed;      /* of the 8-bit states' rounding                        */
} gbla_adamw_config;

/* Bytes of workspace that gbla_grad_norm and gbla_adamw_step need for these
 * tensors (a host array; 0 on an argument error).  Both leave its error word
 * at 0: gbla_check_device_status() reports GBLA_OK. */
size_t gbla_adamw_workspace_size(const gbla_adamw_tensor* tensors, int n_tensors);

/* The global 2-norm of the tensors' gradients into norm (fp32, device; one
 * value).  Squares are summed in two fp32 words a thread (in fp64 where their
 * sum passes the fp32 range) and in fp64 beyond, in a fixed order; a single
 * square over the fp32 range counts as not finite, one under it as 0.  Only grad,
 * grad_dtype and n are read. */
gbla_status gbla_grad_norm(const gbla_adamw_tensor* tensors, int n_tensors,
                           float* norm, void* ws, size_t ws_bytes, void* stream);

/* One AdamW step.
 *   tensors  host array of n_tensors >= 0 entries (read during the call), whose
 *            tensors do not overlap; pointers aligned to their element (16-byte
 *            aligned ones are read in wider pieces)
 *   step     int64, device: the steps taken so far; the call adds 1, so that a
 *            captured and replayed call counts on
 *   norm     NULL, or the device value of gbla_grad_norm: clips by max_norm; and
 *            where it is not finite the call leaves everything, the step count
 *            included, as it was
 */
gbla_status gbla_adamw_step(const gbla_adamw_tensor* tensors, int n_tensors,
                            const gbla_adamw_config* config, int64_t* step,
                            const float* norm, void* ws, size_t ws_bytes,
                            void* stream);

/*
 * Token embedding: rows of a table by ids, k of them a token (items named by
 * several hashes into one shared table; their rows stand side by side):
 *   y[t, j d .. (j + 1) d - 1] = scale table[ids[t, j]].
 *   shape   B, L, d (the width of a table row), io_dtype and the sequence
 *           form; a token of a padded slot past its sequence has a row of
 *           zeros and its ids count for nothing; cu_seqlens is not read
 *   ids     [rows, k] int32 (wide_ids = 0) or int64 (1); an id below 0 is no
 *           token: zeros.  An id >= vocab sets the error word
 *           (GBLA_ERR_DEVICE_CHECK), and so does a seq_lens value outside
 *           [0, L]: they count as no token and as an empty sequence
 *   table   (io) [vocab, d];  y (io) [rows, k d], rounded once
 * d, k and vocab are free: rows k <= 2^30, vocab <= 2^30, k <= 2^20, d <= 2^20,
 * vocab d <= 2^38, rows k d <= 2^40.  Pointers are aligned to their element (rows
 * of a multiple of 16 bytes in 16-byte aligned tensors are read in wider pieces).
 * The shape's H, d_h, gate and rms_eps are ignored.  Workspace: embed_workspace_size(.., 0).
 */
gbla_status embed_forward(const gbla_shape* shape, const void* ids,
                          int wide_ids, int k, const void* table,
                          int64_t vocab, float scale, void* y, void* ws,
                          size_t ws_bytes, void* stream);

/*
 * The table's gradient for the scalar <dy, y>: dtable fp32 [vocab, d],
 *   dtable[v] = scale sum of dy[t, j d ..] over the (t, j) with ids[t, j] = v,
 * all of it written (rows without a token: 0).  dy (io) [rows, k d].  The sums
 * run over the tokens in their order, in pieces of fixed size: the same bits
 * again for the same call.  Workspace: embed_workspace_size(.., 1).
 */
gbla_status embed_backward(const gbla_shape* shape, const void* ids,
                           int wide_ids, int k, const void* dy, int64_t vocab,
                           float scale, float* dtable, void* ws,
                           size_t ws_bytes, void* stream);

/* Bytes of workspace of embed_forward (backward = 0) or embed_backward (1; it
 * serves the forward too); 0 on an argument error. */
size_t embed_workspace_size(const gbla_shape* shape, int64_t vocab, int k,
                            int backward);

/*
 * Layer norm of each token, with the residual stream's addition before it:
 *   s = x + res,  m = mean(s),  r = 1 / sqrt(mean((s - m)^2) + eps),
 *   y = (s - m) r w + b.
 *   shape   B, L, d, io_dtype and the sequence form; tokens of padded slots past
 *           their sequence get zeros in every output (a seq_lens value outside
 *           [0, L] sets the error word and counts as 0); cu_seqlens is not read
 *   x       (io) [rows, d], row stride ldx, d .. 2^40
 *   res     (io) [rows, d] or NULL (s = x)
 *   w, b    (io) [d] or NULL (ones, zeros)
 *   sum     (io) [rows, d]: s, rounded once, which is what is normed; NULL without
 *           res, and where s is not wanted.  It may be res, or x with ldx = d
 *   y       (io) [rows, d]
 *   stats   fp32 [rows, 2] (m, r) for the backward, 8-byte aligned, or NULL
 * rows <= 2^30, d <= 2^20; pointers aligned to their element; tensors do not
 * overlap (but sum as above).  The shape's H, d_h, gate and rms_eps are ignored.
 * Workspace: layer_norm_workspace_size(shape, 0).
 */
gbla_status layer_norm_forward(const gbla_shape* shape, const void* x,
                               int64_t ldx, const void* res, const void* w,
                               const void* b, float eps, void* sum, void* y,
                               float* stats, void* ws, size_t ws_bytes,
                               void* stream);

/*
 * Backward for <dy, y> + <ds, s>: x, ldx are what was normed (sum, where there
 * was a res), stats the forward's; with z = (s - m) r and g = dy w
 *   dx = r (g - mean(g) - z mean(g z)) + ds   (the gradient of x and of res),
 *   dw = sum over the tokens of dy z,  db = sum over the tokens of dy.
 *   dy (io) [rows, d];  ds (io) [rows, d] or NULL;  dx (io) [rows, d], may be ds;
 *   dw, db fp32 [d] or NULL.  Gradients overwrite; fixed order of sums.
 * Workspace: layer_norm_workspace_size(shape, 1).
 */
gbla_status layer_norm_backward(const gbla_shape* shape, const void* x,
                                int64_t ldx, const void* w, const float* stats,
                                const void* dy, const void* ds, void* dx,
                                float* dw, float* db, void* ws, size_t ws_bytes,
                                void* stream);

/* Bytes of workspace of layer_norm_forward (backward = 0) or
 * layer_norm_backward (1; it serves the forward too); 0 on a shape error. */
size_t layer_norm_workspace_size(const gbla_shape* shape, int backward);

/*
 * A step of beam search.  Of each of B groups' K beams x V tokens, the n_out of
 * highest
 *   score(b, t) = scores[b] + logits[b, t] - log sum_t' exp(logits[b, t']),
 * in falling order, ties to the lowest beam and then the lowest token.
 */
typedef struct {
  int B, K, V;       /* groups; beams of each, 1 .. 1024; tokens                  */
  int n_out;         /* beams that go on, 1 .. 1024 (K = 1 starts a search)       */
  int io_dtype;      /* gbla_dtype of the logits                                  */
  int eos;           /* the token that ends a beam, or -1                         */
  int over_allowed;  /* 1: the logarithm's sum runs over the allowed tokens alone */
} gbla_beam;

/*
 *   logits   (io) [B K, V], row stride ld, V .. 2^40, aligned to the element
 *   scores   fp32 [B, K]; a beam of -inf or NaN has no candidates (the beams but
 *            the first of a search that starts with K copies)
 *   allowed  uint32 [B K, ceil(V / 32)] or NULL: bit t % 32 of word t / 32 lets
 *            token t be a candidate (valid continuations of an item's code)
 *   done     uint8 [B, K] or NULL (needs eos >= 0): an ended beam's only candidate
 *            is (b, eos) with scores[b], whatever its logits and mask are
 *   new_scores fp32, tokens, parents int32 [B, n_out]: parents in 0 .. K - 1;
 *            new_done uint8 [B, n_out] or NULL: done[parent], or token = eos.
 *            Where there are fewer candidates than n_out the last are (-inf, token
 *            -1, parent 0, not done).
 * Logits of -inf and rows with a NaN or +inf among those summed have no candidates.
 * A token that has all of its beam's sum (the only one that may follow) has the
 * logarithm 0: the beam keeps its score exactly.
 * Exponentials are summed, and scores compared, in two fp32 words: which of two
 * candidates is first is decided to 2^-26 (to 2^-30 on the mean), and a score is
 * rounded once.
 * V <= 2^30, K V <= 2^32, B K V / 1024 <= 2^31.  Outputs do not overlap inputs.  Workspace:
 * beam_workspace_size().
 */
gbla_status beam_select(const gbla_beam* beam, const void* logits, int64_t ld,
                        const float* scores, const uint32_t* allowed,
                        const uint8_t* done, float* new_scores, int32_t* tokens,
                        int32_t* parents, uint8_t* new_done, void* ws,
                        size_t ws_bytes, void* stream);

/* Bytes of workspace of beam_select and beam_reorder; 0 on an argument error. */
size_t beam_workspace_size(const gbla_beam* beam);

/* What a beam keeps: rows of row_bytes bytes, [B K] in src, [B n_out] in dst. */
typedef struct {
  void* dst;         /* may be src, with n_out = K: moved in place               */
  const void* src;
  int64_t row_bytes; /* 0 .. 2^30; B n_out row_bytes <= 2^39                     */
} gbla_beam_state;

/*
 * The beams' states (of a recurrence: its h) follow their parents, any number of
 * tensors: dst[b n_out + i] = src[b K + parents[b, i]].  A parent outside
 * 0 .. K - 1 sets the error word (GBLA_ERR_DEVICE_CHECK) and leaves its row of dst as
 * it was.  states: host array, read during the call; tensors do not overlap (but
 * dst = src).  beam: checked as a whole, as beam_select does; B, K and n_out are what counts.
 */
gbla_status beam_reorder(const gbla_beam* beam, const gbla_beam_state* states,
                         int n_states, const int32_t* parents, void* ws,
                         size_t ws_bytes, void* stream);

/*
 * bla_core_forward without a caller workspace (the pages have no counterpart:
 * this is a deployment convenience).  Some callers cannot call cudaMalloc or
 * hand the library a scratch buffer: a plugin running inside a host framework
 * that owns all device memory through its own pool and passes only its
 * tensors, or a latency-bound serving loop where an allocation would
 * synchronise the device and stall the other streams.  This entry point
 * allocates nothing: the split-L partial states, combine counters, error word
 * and combined state live in one file-scope device array of 64 MiB
 * (GBLA_NOALLOC_SCRATCH_BYTES) that every GPU which loads the library holds
 * until the process exits.
 *   Arguments, layouts and results are those of bla_core_forward.
 *   GBLA_ERR_WORKSPACE: the shape needs more than 64 MiB of scratch
 *   (gbla_workspace_size(shape, GBLA_OP_CORE_FORWARD) > 64 MiB); nothing runs.
 *   The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress, with that device current); make that first call
 *   before any stream capture.
 *   Every call on a device shares the one array: calls whose kernels overlap
 *   on the GPU (two streams, or two host threads) race and corrupt each
 *   other's results.  Order them on one stream.  The counters and the error
 *   word are cleared at the start of every call; the error word of the last
 *   call is read by bla_core_noalloc_check_device_status (below).
 */
#define GBLA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
gbla_status bla_core_forward_noalloc(const gbla_shape* shape, const void* q,
                                     const void* k, const void* v,
                                     const float* g, void* o, float* den,
                                     float* state, void* stream);

/* Synchronises `stream` and reads the device error word of the workspace that
 * the last call on it used: GBLA_OK, GBLA_ERR_DEVICE_CHECK (bad cu_seqlens /
 * seq_lens; reported first), GBLA_ERR_DEVICE_TIMEOUT (a bounded wait gave up),
 * or GBLA_ERR_CUDA if the stream itself failed. */
gbla_status gbla_check_device_status(const void* ws, void* stream);

/* gbla_check_device_status for bla_core_forward_noalloc: synchronises
 * `stream` and reads the error word of the library's fixed scratch array on
 * the current device (the last no-allocation call's).  It allocates nothing. */
gbla_status bla_core_noalloc_check_device_status(void* stream);

/* Diagnostic of the timeout path (no counterpart on the pages).  Clears the
 * error word at the start of `ws` (any workspace of at least 16 bytes,
 * 256-byte aligned) and launches one CTA that waits, with the kernels' own
 * bounded mbarrier wait cut to `polls` polls (1 .. 2^20), on a barrier that
 * nothing arrives at.  The wait gives up, sets the timeout bit, and the kernel
 * returns; nothing faults or hangs.  gbla_check_device_status(ws, stream)
 * then reports GBLA_ERR_DEVICE_TIMEOUT.  Asynchronous on `stream`. */
gbla_status gbla_diag_bounded_wait(void* ws, size_t ws_bytes, unsigned polls, void* stream);

/* Static text for a status code. */
const char* gbla_status_string(int status);

/* Text of the last CUDA error seen by this thread (empty if none). */
const char* gbla_last_error(void);

/* Library version, major*10000 + minor*100 + patch. */
int gbla_version(void);

/* Per-launch timing for benchmarks and profiling (no counterpart on the
 * pages).  While enabled, every kernel or memset that a gbla_* / bla_core_*
 * call of the CALLING THREAD launches is bracketed by two CUDA events recorded
 * on that call's stream.  gbla_profiling_read() synchronises on the last
 * event, writes up to `cap` entries (static name strings, milliseconds) and
 * returns the number of launches recorded since the previous read, then
 * clears the record.  Either output array may be NULL.  A name is the step
 * followed by the kernel variant that ran, e.g. "bwd_q[tc]" (5th-generation
 * tensor cores, tcgen05), "bwd_q[mma]" (mma.sync), "bwd_q[f32]" (fp32 I/O),
 * "conv[bulk]" (bulk-copy staged) or "conv[plain]". */
void gbla_profiling_enable(int on);
int gbla_profiling_read(const char** names, float* ms, int cap);

/* Kernel selection of the CALLING THREAD's later calls (no counterpart on the
 * pages).  GBLA_POLICY_AUTO (the default) picks, per step, the kernel that is
 * fastest for the shape: e.g. the state reduction runs on the 5th-generation
 * tensor cores only when every SM gets at least 20 of its 256-row tiles, and
 * on mma.sync otherwise.  GBLA_POLICY_TC takes the tcgen05 kernel wherever it
 * applies (d_h and gate permitting), whatever the size: for tests that check
 * those kernels on small shapes.  GBLA_POLICY_MMA takes the mma.sync kernel
 * of every step that has one beside its tcgen05 kernel: for tests of the
 * mma.sync kernels at the shapes AUTO runs on tcgen05.  Results agree within
 * the tolerances either way.  GBLA_ERR_INVALID_ARG for another value. */
typedef enum { GBLA_POLICY_AUTO = 0, GBLA_POLICY_TC = 1, GBLA_POLICY_MMA = 2 } gbla_policy;
gbla_status gbla_set_kernel_policy(int policy);

#ifdef __cplusplus
}
#endif

#endif /* GBLA_H */
