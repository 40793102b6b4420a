/*
 * muon_gb300.h -- C ABI of the GB300 (sm_103a) Muon optimizer step.
 *
 * The Muon step, as the pages describe it:
 *   [MCS] "Muon Custom Sizing 实战：modded-nanogpt 将注意力与 MLP 参数合并进同一
 *         reduce_scatter 调用，把 124M GPT 训练压进 150 秒", section 2.3 (batched
 *         NS of the QKVO view, coefficients (a,b,c) = (3.4445, -4.7750, 2.0315),
 *         five rounds) and section 四 (momentum lerp, Nesterov blend, decoupled
 *         decay lr*wd, write-back with alpha = -lr * max(1, hdim/dim)^0.5);
 *   [PG]  "parameter-golf train_gpt.py 源码精读：Muon 优化器、Int8 量化与 DDP 数据
 *         加载全解", part 1, section 核心思想 (the Newton-Schulz function:
 *         X /= ||X||; repeat A = X X^T, B = bA + cA^2, X = aX + BX) and section
 *         分布式细节 (rescale of the result by max(1, m/n)^0.5).
 *
 * Conventions shared by every entry point:
 *   - Matrices are row-major and contiguous, stacked as [batch, rows, cols].
 *     A stack of same-shape weights is one call; the [MCS] QKVO weight stored
 *     as (hdim, 4*dim) is passed as batch 4 of (hdim, dim): the same bytes.
 *   - Every data pointer is device memory owned by the caller, 16-byte
 *     aligned.  Parameters and momentum buffers are updated in place;
 *     gradients are only read.  No call allocates device memory; the one
 *     device memory the library itself holds is the fixed 64 MiB scratch of
 *     muon_step_noalloc(), a static array that every GPU which loads the
 *     library keeps until the process exits.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  All
 *     work is enqueued on it asynchronously; no entry point synchronises
 *     except muon_workspace_status().
 *   - The workspace is caller-owned device memory of at least the size that
 *     muon_workspace_bytes()/muon_grouped_workspace_bytes() return, 256-byte
 *     aligned, and zero-filled before its first use (it carries a sticky
 *     device error word).  Calls that share a workspace must not overlap on
 *     the GPU.
 *   - Failure (no counterpart on the pages): every device-side wait is
 *     bounded (2 s).  A wait that gives up sets the workspace's error word;
 *     from then on the waits of the other kernels still running end within
 *     microseconds, and every kernel of every later call on that workspace
 *     returns at entry, so those calls change nothing (parameters, momentum
 *     and outputs keep their values) until muon_workspace_status() clears
 *     the word.  The call during which the wait gave up may have written part
 *     of its results.
 *   - Argument errors are reported before anything is enqueued.  A CUDA error
 *     while enqueuing gives MUON_ERR_CUDA.  No C++ exception crosses the ABI.
 *   - NS runs in bf16 on the tensor cores (fp32 accumulation and epilogues)
 *     for min(rows, cols) >= 64; smaller matrices run the same iteration in
 *     fp32 on the CUDA cores (bf16 is too coarse for, e.g., a 1x12 gate).
 *   - When rows > cols the iteration runs on the transpose (A is the
 *     min(rows,cols)^2 Gram matrix); the result comes back in the input's
 *     orientation.  The norm is Frobenius, divided as ||X||_F + eps.
 */
#ifndef MUON_GB300_H
#define MUON_GB300_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum muon_status {
  MUON_OK = 0,
  MUON_ERR_INVALID_ARG = 1,  /* bad pointer, size, alignment, dtype or scalar     */
  MUON_ERR_UNSUPPORTED = 2,  /* no sm_103a device current, or shape out of range  */
  MUON_ERR_CUDA = 3,         /* a CUDA runtime/driver call failed                 */
  MUON_ERR_TIMEOUT = 4,      /* a bounded device-side wait gave up (see status)   */
  MUON_ERR_WORKSPACE = 5     /* workspace NULL, misaligned or too small           */
} muon_status;

typedef enum muon_dtype {
  MUON_F32 = 0,
  MUON_BF16 = 1
} muon_dtype;

/* One stack of same-shape 2-D weights for muon_step_grouped(). */
typedef struct muon_group {
  float* params;        /* [batch, rows, cols] fp32, updated in place            */
  const void* grads;    /* [batch, rows, cols] in g_dtype, read only             */
  float* momentum_buf;  /* [batch, rows, cols] fp32, updated in place            */
  int g_dtype;          /* muon_dtype of grads                                   */
  int batch;            /* 0..65535; 0 skips the group                           */
  int rows, cols;       /* >= 1 each, <= 65536 each                              */
  float lr_scale;       /* <= 0: max(1, rows/cols)^0.5 ([PG] 分布式细节)          */
} muon_group;

/* Kinds of kernel the library launches (trace records, launch counts). */
typedef enum muon_kernel_kind {
  MUON_K_PROLOGUE = 0,   /* momentum, Nesterov blend, bf16 cast, norm partials  */
  MUON_K_SMALL_NS = 1,   /* whole step in fp32 for min(rows,cols) < 64          */
  MUON_K_GRAM = 2,       /* A = s^2 X X^T, upper 256 x 256 tiles only           */
  MUON_K_POLY = 3,       /* B' = a I + b A + c A A, upper 256 x 256 tiles only  */
  MUON_K_UPDATE = 4,     /* X <- s B' X  (= s (a X + B X))                      */
  MUON_K_APPLY = 5,      /* p <- (1 - lr wd) p - lr scale O (or O as bf16)      */
  MUON_K_ADAM = 6,       /* DistAdam update of non-matrix parameters            */
  MUON_K_FUSED_NS = 7,   /* all NS rounds, one CTA pair per matrix, 64<=m<=256,
                            n<=512 (see muon_set_fused_ns)                      */
  MUON_K_ROUNDS = 8,     /* all Gram/Poly/Update stages of every round in one
                            persistent launch (see muon_set_persistent_rounds)  */
  MUON_K_NORM_ROPE = 9,      /* norm and rotation of the query and key heads    */
  MUON_K_NORM_ROPE_BWD = 10, /* its gradients                                   */
  MUON_K_ATTENTION = 11,     /* attention, forward                              */
  MUON_K_ATTENTION_DQ = 12,  /* attention, gradient of the queries              */
  MUON_K_ATTENTION_DKV = 13, /* attention, gradients of the keys and values     */
  MUON_K_LINEAR = 14,        /* products with a weight matrix                   */
  MUON_K_LINEAR_FINISH = 15, /* sums of a split product, its epilogue           */
  MUON_K_LINEAR_DZ = 16,     /* dz = dout act'(z), and the bias' gradient       */
  MUON_K_LINEAR_TOKEN = 17,  /* the product for up to 4 tokens                  */
  MUON_K_RMS_NORM = 18,      /* residual's addition and RMS norm                */
  MUON_K_RMS_NORM_BWD = 19,  /* its gradients                                   */
  MUON_K_RMS_NORM_WEIGHT = 20, /* the weight's gradient: sum of the blocks' parts */
  MUON_K_EMBEDDING = 21,     /* rows of a token table                           */
  MUON_K_EMBEDDING_SORT = 22, /* tokens sorted by id, the table's gradient cleared */
  MUON_K_EMBEDDING_SUM = 23, /* sums of the runs of equal ids                   */
  MUON_K_EMBEDDING_JOIN = 24, /* ... of those that several warps share          */
  MUON_K_GRAD_SQUARES = 25,  /* sum of squares of the gradients                 */
  MUON_K_CLIP = 26           /* their norm, and the clipped gradients           */
} muon_kernel_kind;

/* Workspace bytes for one muon_step()/muon_ns5() call on [batch, rows, cols].
 * Returns 0 if the sizes are invalid. */
size_t muon_workspace_bytes(int batch, int rows, int cols);

/* Workspace bytes for one muon_step_grouped() call; 0 if a group is invalid. */
size_t muon_grouped_workspace_bytes(const muon_group* groups, int n_groups);

/*
 * The Newton-Schulz function ([PG] 核心思想) on every matrix of a stack:
 *   X = G / (||G||_F + eps)  (on G^T if rows > cols),
 *   `steps` times: A = X X^T;  B = b A + c A A;  X = a X + B X,
 *   out = X (transposed back), written as bf16 [batch, rows, cols].
 * G: [batch, rows, cols] fp32 or bf16 (g_dtype).  steps in 1..16; batch in
 * 0..65535, rows and cols in 1..65536 (the same limits hold for every call).
 */
muon_status muon_ns5(const void* G, int g_dtype, void* out_bf16,
                     int batch, int rows, int cols, int steps,
                     float a, float b, float c, float eps,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * One Muon step on a stack of same-shape weights ([MCS] 四, [PG] 核心思想/分布式细节):
 *   buf <- buf + (1 - momentum) (g - buf)
 *   u   <- g + momentum (buf - g)  if nesterov, else buf
 *   O   <- NS(u) as in muon_ns5 (bf16, as the last Newton-Schulz update writes it)
 *   p   <- (1 - lr weight_decay) p - lr s O,   s = lr_scale > 0 ? lr_scale
 *                                                 : max(1, rows/cols)^0.5
 * momentum in [0, 1]; steps in 1..16; eps >= 0; all scalars finite.
 */
muon_status muon_step(float* params, const void* grads, int g_dtype, float* momentum_buf,
                      int batch, int rows, int cols,
                      float momentum, int nesterov, float lr, float weight_decay,
                      float lr_scale, int steps, float a, float b, float c, float eps,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * muon_step without a workspace, for callers that cannot call cudaMalloc: code
 * running under an allocator that has already reserved the whole GPU, plug-ins
 * allowed to touch only the memory they are handed, or training loops that
 * forbid any allocation after start-up.  The pages have no counterpart: this is
 * an interface addition, not part of the method.
 * Arguments and results are those of muon_step, minus the workspace.  Scratch is
 * a 64 MiB array built into the library (held by every GPU that loads it until
 * the process exits); a call whose muon_workspace_bytes(batch, rows, cols)
 * exceeds 64 MiB returns MUON_ERR_WORKSPACE.  The first call on a device looks
 * up the array's device address, so make it before any stream capture.  All
 * calls on a device share the array: calls that overlap on the GPU race.
 * Each call clears the array's sticky error word on `stream` after its
 * argument checks and before its first kernel, so the word reports the latest
 * call on the device: read it with muon_noalloc_status().
 */
muon_status muon_step_noalloc(float* params, const void* grads, int g_dtype, float* momentum_buf,
                              int batch, int rows, int cols,
                              float momentum, int nesterov, float lr, float weight_decay,
                              float lr_scale, int steps, float a, float b, float c, float eps,
                              void* stream);

/*
 * muon_workspace_status() for the built-in scratch of muon_step_noalloc() on
 * the current device (no counterpart on the pages): synchronises `stream`,
 * then returns MUON_OK, or MUON_ERR_TIMEOUT if a bounded device-side wait
 * gave up during the latest muon_step_noalloc() call on this device (or
 * during a muon_selftest_wait_timeout() on the scratch since).  clear != 0
 * resets the word afterwards.
 */
muon_status muon_noalloc_status(void* stream, int clear);

/*
 * muon_step on every group of a model at once (the pages stack the weights of
 * each parameter group, [MCS] 四 第一遍/第二遍).  Groups share the scalars; the
 * NS rounds of all tensor-core groups run as one grouped launch per stage.
 * n_groups >= 0; groups may be NULL only when n_groups == 0.  The arrays of
 * different groups must not overlap.
 */
muon_status muon_step_grouped(const muon_group* groups, int n_groups,
                              float momentum, int nesterov, float lr, float weight_decay,
                              int steps, float a, float b, float c, float eps,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * Synchronises `stream`, then reads the workspace's sticky device error word:
 * MUON_OK, or MUON_ERR_TIMEOUT if a bounded wait inside a kernel gave up since
 * the word was last cleared.  clear != 0 resets the word to zero afterwards.
 */
muon_status muon_workspace_status(const void* workspace, size_t workspace_bytes,
                                  void* stream, int clear);

/*
 * Self-test of the device-side timeout path (no counterpart on the pages).
 * Enqueues one kernel whose bounded wait, the same code every GEMM role waits
 * with, is on a barrier that nothing completes; after `limit_us` (1..100000)
 * it gives up and records the timeout in the workspace's status word, as a
 * stalled GEMM would.  muon_workspace_status() then reports MUON_ERR_TIMEOUT.
 * workspace = NULL targets the built-in scratch of muon_step_noalloc() on the
 * current device instead (workspace_bytes is then ignored), read back with
 * muon_noalloc_status().  Nothing faults, hangs or is left pending on the GPU.
 */
muon_status muon_selftest_wait_timeout(void* workspace, size_t workspace_bytes, int limit_us,
                                       void* stream);

/*
 * The Adam half of the optimizer: the DistAdam update that trains the
 * parameters Muon does not take (embeddings, output head, {0,1}-D scalars).
 * Defined by the DistAdam step() printed in "将 Adam 梯度同步（Reduce-Scatter）
 * 移入反向 Hook：modded-nanogpt 分布式优化器每步提速约 0.7 秒的工程实践",
 * section 改动二, with lr_eff = lr * lr_scale and t = `step`:
 *   if weight_decay != 0:  p *= 1 - lr_eff * weight_decay * wd_scale
 *   m = beta1 m + (1 - beta1) g;   v = beta2 v + (1 - beta2) g^2
 *   p -= lr_eff * sqrt(1 - beta2^t) / (1 - beta1^t) * m / (sqrt(v) + eps)
 * ([MCS] section 四 gives lr 0.008, betas (0.8, 0.95), eps 1e-8 for it.)
 * On one GPU the reduce-scatter / all-gather of that page has no work: each
 * tensor is updated whole, as one flat array of `numel` elements.
 */
typedef struct muon_adam_tensor {
  float* param;         /* [numel] fp32, updated in place                        */
  const void* grad;     /* [numel] in g_dtype, read only                         */
  float* exp_avg;       /* [numel] fp32 first moment m, updated in place         */
  float* exp_avg_sq;    /* [numel] fp32 second moment v, updated in place        */
  long long numel;      /* >= 0; 0 skips the tensor (its pointers may be NULL)   */
  int g_dtype;          /* muon_dtype of grad                                    */
  float lr_scale;       /* per-parameter lr multiplier (1 = none), finite, >= 0  */
  float wd_scale;       /* per-parameter weight-decay multiplier (1 = none)      */
} muon_adam_tensor;

/*
 * One Adam step over n_tensors >= 0 tensors (tensors may be NULL only when
 * n_tensors == 0), all at step count `step` >= 1 (the value after the
 * increment).  0 <= beta1, beta2 < 1; eps >= 0; lr and weight_decay finite.
 * Pointers 16-byte aligned; the arrays of different tensors must not overlap.
 * Up to 64 tensors go in one kernel launch; more take one launch per 64.
 * Needs no workspace and has no waits.
 */
muon_status muon_adam_step(const muon_adam_tensor* tensors, int n_tensors, int step, float lr,
                           float beta1, float beta2, float eps, float weight_decay,
                           void* stream);

/*
 * The attention path of a GPT block, the block whose c_q, c_k, c_v and proj
 * weights muon_step trains: the norm and rotation of the query and key heads,
 * and the attention itself, each with its gradients.  The pages name the model
 * ([MCS] section 2.1) and print none of this; it is an addition.
 *
 * Heads are passed as strided views, so that the columns of a fused q, k, v
 * projection's output (and of its gradient) are used in place: element d of
 * head h of token t lies at data[t token_stride + h head_stride + d].  Strides
 * are in elements.  data and both strides are 16-byte aligned (a stride whose
 * dimension has one entry is ignored) and strides are positive: a broadcast view
 * (stride 0) is refused, its gradient would be a sum that no call here takes.
 * Rows of different (t, h) do not overlap in an output.  An output shares no
 * bytes with an input or another output (refused as an invalid argument; views
 * that interleave have to have one token stride), but for muon_qk_norm_rope and
 * its gradients, whose output may be the very view of its own input or gradient.
 * head_dim is a multiple of 8.
 */
typedef struct muon_heads {
  void* data;
  long long token_stride;
  long long head_stride;
} muon_heads;

/*
 * For every token t and head x of q (q_heads of them) and of k (k_heads):
 *   n = x (mean_d x_d^2 + eps)^-1/2 w     (norm != 0; w = 1 where the weight is
 *                                          NULL; n = x where norm == 0)
 *   y_a = n_a c_i - n_b s_i,  y_b = n_b c_i + n_a s_i   for the pairs
 *         i < rot_dim / 2: (a, b) = (i, i + rot_dim / 2), or (2i, 2i + 1) when
 *         interleaved != 0; elements from rot_dim on pass unrotated,
 * with c_i, s_i row positions[t] (t itself where positions is NULL) of the
 * tables cos, sin ([table_len, rot_dim / 2] fp32, contiguous).  Scalings for
 * long contexts are a matter of the tables.  A position outside the tables
 * makes the token's outputs NaN.  All in fp32, rounded once to the outputs' type.
 */
typedef struct muon_norm_rope {
  int dtype;               /* muon_dtype of every muon_heads of the call          */
  int tokens;              /* >= 0; tokens (q_heads + k_heads) < 2^31 - 2^16      */
  int q_heads, k_heads;    /* 0..65535, not both 0 (the views of none are unused) */
  int head_dim;            /* multiple of 8, 8..256                               */
  int rot_dim;             /* multiple of 8, 0..head_dim                          */
  int norm, interleaved;   /* 0 or 1                                              */
  float eps;               /* finite, >= 0                                        */
  int table_len;           /* rows of cos and sin, >= 1 if rot_dim > 0            */
  const float* cos;        /* 16-byte aligned; unused if rot_dim == 0             */
  const float* sin;
  const int* positions;    /* [tokens] or NULL                                    */
  const float* q_weight;   /* [head_dim] or NULL; NULL if norm == 0; 16-byte      */
  const float* k_weight;   /*   aligned                                           */
} muon_norm_rope;

muon_status muon_qk_norm_rope(const muon_norm_rope* spec, muon_heads q, muon_heads k,
                              muon_heads q_out, muon_heads k_out, void* stream);

/*
 * Gradients of muon_qk_norm_rope: dq, dk (the inputs') from dq_out, dk_out (the
 * outputs'), and the weights' in fp32 where the weight is given (dq_weight and
 * dk_weight are then required: [head_dim], overwritten).  Sums over tokens and
 * heads are taken in a fixed order: repeated calls give equal bits.
 */
size_t muon_norm_rope_workspace_bytes(int head_dim);
muon_status muon_qk_norm_rope_backward(const muon_norm_rope* spec, muon_heads dq_out,
                                       muon_heads dk_out, muon_heads q, muon_heads k,
                                       muon_heads dq, muon_heads dk, float* dq_weight,
                                       float* dk_weight, void* workspace,
                                       size_t workspace_bytes, void* stream);

/*
 * Causal attention over sequences packed along the tokens.  Sequence s holds the
 * tokens cu_seqlens[s] <= t < cu_seqlens[s + 1] (n_seqs + 1 ascending int32 on the
 * device, from 0 to at most `tokens`; empty sequences are allowed; NULL with
 * n_seqs = 0: one sequence of all tokens).  Query head h reads key/value head
 * h / (q_heads / kv_heads).  For token i of a sequence that starts at a:
 *   s_ij = scale q_i . k_j,  a <= j <= i;   lse_i = log sum_j exp(s_ij)
 *   out_i = sum_j exp(s_ij - lse_i) v_j
 * Tokens past the last sequence get out = 0 and lse = -inf, and no gradient.
 * A token of a sequence whose visible scores are all -inf gets NaN in both.
 * A token's results depend on its own sequence's tokens up to it alone: Inf or
 * NaN elsewhere does not reach them.  Offsets that do not ascend give undefined
 * results (no access leaves the tensors).
 * bf16 heads; products in bf16 with fp32 sums, softmax in fp32; the weights
 * exp(s_ij - m) are rounded to bf16 for their product with v.
 */
typedef struct muon_attention_spec {
  int tokens;              /* >= 0; tokens q_heads < 2^31 - 2^16                  */
  int q_heads, kv_heads;   /* 1..65535; q_heads a multiple of kv_heads            */
  int head_dim;            /* multiple of 8, 8..128                               */
  int n_seqs;              /* >= 0                                                */
  const int* cu_seqlens;   /* [n_seqs + 1] device memory, or NULL                 */
  float scale;             /* finite, > 0                                         */
} muon_attention_spec;

/* Workspace bytes of muon_attention and muon_attention_backward; 0 if invalid. */
size_t muon_attention_workspace_bytes(int tokens, int q_heads, int kv_heads, int head_dim);

/* out: bf16 heads (q_heads of them); lse: [q_heads, tokens] fp32, natural log. */
muon_status muon_attention(const muon_attention_spec* spec, muon_heads q, muon_heads k,
                           muon_heads v, muon_heads out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * Gradients of muon_attention's out with respect to q, k and v, from its out and
 * lse for the same q, k, v and offsets (of any other out the results are not
 * defined: delta is corrected by what out was rounded by).  With
 * delta_i = dout_i . out_i and ds_ij = p_ij (dout_i . v_j - delta_i):
 *   dq_i = scale sum_j ds_ij k_j;  dk_j = scale sum_i ds_ij q_i;  dv_j = sum_i p_ij dout_i
 * (dk and dv summed over the query heads that share the key/value head, in fp32).
 * Fixed summation order, no atomics: repeated calls give equal bits.
 */
muon_status muon_attention_backward(const muon_attention_spec* spec, muon_heads dout,
                                    muon_heads q, muon_heads k, muon_heads v, muon_heads out,
                                    const float* lse, muon_heads dq, muon_heads dk,
                                    muon_heads dv, void* workspace, size_t workspace_bytes,
                                    void* stream);

/*
 * Products with a weight matrix, the operators between the attention path and the
 * weights that muon_step trains (c_q, c_k, c_v, proj and the MLP's matrices).  The
 * pages name the layers ([PG] CastedLinear, the relu^2 MLP) and print none of this;
 * it is an addition.
 *
 * A matrix is passed as a strided view: element j of row i lies at
 * data[i row_stride + j].  data and row_stride are 16-byte aligned (the stride of a
 * single row is ignored), row_stride is at least the width: columns of a wider
 * tensor are used in place, and a width that is no multiple of 8 needs padded rows.
 * Padding is neither read into a result nor written.  An output shares no bytes
 * with an input or another output, but where the text allows it (refused as an
 * invalid argument; views that interleave have to have one stride).
 */
typedef struct muon_matrix {
  void* data;
  long long row_stride;
} muon_matrix;

typedef enum muon_activation {
  MUON_ACT_NONE = 0,
  MUON_ACT_RELU2 = 1,    /* max(z, 0)^2                                             */
  MUON_ACT_GELU = 2      /* z / (1 + exp(-2 u)), u = (2/pi)^1/2 (z + 0.044715 z^3):
                            GELU's tanh form                                        */
} muon_activation;

/*
 * z = x W^T + b,  out = act(z) + r:  x [tokens, in_features], W [out_features,
 * in_features], b [out_features] or NULL, r [tokens, out_features] or data NULL, all
 * bf16.  Products in bf16 with fp32 sums; bias, activation and residual in fp32 on
 * the sum; one rounding to bf16.  preact (or data NULL) receives z, rounded, for the
 * gradients.  out may be the very view of the residual.
 */
typedef struct muon_linear_spec {
  int tokens;                        /* 0..2^31 - 65537                             */
  int in_features, out_features;     /* 1..2^20                                     */
  int activation;                    /* muon_activation                             */
  const void* bias;                  /* bf16, 16-byte aligned, or NULL              */
} muon_linear_spec;

/* Workspace bytes of muon_linear and muon_linear_backward; 0 if invalid. */
size_t muon_linear_workspace_bytes(int tokens, int in_features, int out_features);

muon_status muon_linear(const muon_linear_spec* spec, muon_matrix x, muon_matrix weight,
                        muon_matrix residual, muon_matrix preact, muon_matrix out,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of muon_linear: with dz = dout act'(z) (dout itself without activation),
 *   dx = dz W,   dweight = dz^T x,   dbias = sum over tokens of dz
 * in bf16 from fp32 sums.  With an activation, preact is the z that muon_linear
 * left, and dz [tokens, out_features] is a buffer that the call fills with dz rounded
 * to bf16 for the products (dbias sums the unrounded); without, both are unused.
 * dbias: [out_features] or NULL; spec->bias is not read.  The residual's gradient is
 * dout.  Fixed summation order: repeated calls give equal bits.
 */
muon_status muon_linear_backward(const muon_linear_spec* spec, muon_matrix dout, muon_matrix x,
                                 muon_matrix weight, muon_matrix preact, muon_matrix dz,
                                 muon_matrix dx, muon_matrix dweight, void* dbias,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * The residual's addition and the RMS norm of the sum, the input of a block's halves.
 * ([PG] has the norm before each half; the pages print no code of it.)  Per token:
 *   h = x + residual  (x where residual's data is NULL),
 *   y = h (mean h^2 + eps)^-1/2 w   (w = 1 where weight is NULL),
 * with x, residual, out (y) and sum (h) [tokens, dim] in one type.  h stays in fp32 for
 * the norm and is rounded to be stored; y is rounded once.  Finite rows of any magnitude
 * are right: one whose squares leave fp32's range is scaled by a power of two first (with a
 * residual, its y is that of h as stored).  sum is given where residual is.  out and sum
 * may each be the very view of x or of residual (not of each other).
 */
typedef struct muon_rms_norm_spec {
  int dtype;               /* muon_dtype of every muon_matrix of the call           */
  int tokens;              /* 0..2^31 - 65537                                       */
  int dim;                 /* multiple of 8, 8..16384                               */
  float eps;               /* finite, >= 0                                          */
  const float* weight;     /* [dim], 16-byte aligned, or NULL                       */
} muon_rms_norm_spec;

muon_status muon_rms_norm(const muon_rms_norm_spec* spec, muon_matrix x, muon_matrix residual,
                          muon_matrix out, muon_matrix sum, void* stream);

/*
 * The same with y in 8 bits: y = scale q, q in e4m3 (out: bytes, rows 8-byte aligned),
 * one scale a row (group = 0; scales [tokens]) or for each 128 columns (group = 128;
 * scales [tokens, ceil(dim / 128)]).  A scale is the least power of two (from 2^-126 on)
 * that brings the group's largest |y| to 448 or less, 1 where that is 0: e4m3's is the only
 * rounding.  Where a y of the group is not finite its scale and all its q are NaN.
 */
muon_status muon_rms_norm_fp8(const muon_rms_norm_spec* spec, int group, muon_matrix x,
                              muon_matrix residual, muon_matrix out, float* scales,
                              muon_matrix sum, void* stream);

/*
 * Gradients of muon_rms_norm from dout (y's) and h as stored (sum; x without a
 * residual).  With r = (mean h^2 + eps)^-1/2, n = h r, G = dout w:
 *   dx = r (G - n mean(G n)) + dresidual,   dweight = sum over tokens of dout n
 * dresidual: h's gradient from where else it went, or data NULL; dx is the gradient of x
 * and of residual alike, and infinite where 1 / r is below 2^-126.  dx may be the very
 * view of dout, sum or dresidual.  dweight ([dim] fp32, overwritten) is given where the
 * weight is.  Fixed summation order: repeated calls give equal bits.
 */
size_t muon_rms_norm_workspace_bytes(int dim);
muon_status muon_rms_norm_backward(const muon_rms_norm_spec* spec, muon_matrix dout,
                                   muon_matrix sum, muon_matrix dresidual, muon_matrix dx,
                                   float* dweight, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * The token embedding, the table that muon_adam_step trains:
 *   out[t] = scale table[ids[t]]
 * for table [rows, dim] and out [tokens, dim], each fp32 or bf16.  A token whose id is
 * outside the table gets NaN.
 */
typedef struct muon_embedding_spec {
  int tokens;              /* 0..2^31 - 65537                                       */
  int rows;                /* 1..2^30                                               */
  int dim;                 /* multiple of 8, 8..65536                               */
  int id_bytes;            /* 4 (int32) or 8 (int64)                                */
  const void* ids;         /* [tokens] device memory, aligned to id_bytes           */
  float scale;             /* finite                                                */
} muon_embedding_spec;

muon_status muon_embedding(const muon_embedding_spec* spec, int table_dtype, muon_matrix table,
                           int out_dtype, muon_matrix out, void* stream);

/*
 * The table's gradient: dtable[v] = scale times the sum of dout[t] over the tokens with
 * ids[t] = v, in fp32 and rounded once; rows that no token names are 0.  Tokens whose id
 * is outside the table enter no sum.  dout and dtable are fp32 or bf16 each.  Fixed
 * summation order (tokens sorted by id), no atomics: repeated calls give equal bits.
 */
size_t muon_embedding_workspace_bytes(int tokens, int dim);
muon_status muon_embedding_backward(const muon_embedding_spec* spec, int dout_dtype,
                                    muon_matrix dout, int dtable_dtype, muon_matrix dtable,
                                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * The norm of all gradients of a model together, and the gradients clipped by it, in
 * front of muon_step_grouped and muon_adam_step:
 *   norm = (sum over all tensors and elements of g^2)^1/2
 *   out  = g min(1, max_norm / (norm + eps))
 * norm: one float on the device.  out may be the gradient itself (in one type), or a
 * tensor of either type.  With max_norm = INFINITY the factor is 1 whatever the norm, and
 * where every out is the gradient itself or NULL only the norm is computed.  At factor 1 a
 * gradient whose out it is itself is not written.  The arrays of different tensors must not
 * overlap.  With a finite max_norm a norm that is NaN or infinite makes the factor NaN or
 * 0, as the formula has it.  Squares are summed in fp32: magnitudes from 2^58 on may make
 * the norm infinite, those below 2^-75 add nothing.
 * Fixed summation order: repeated calls give equal bits.
 */
typedef struct muon_grad_tensor {
  const void* grad;        /* [numel] in g_dtype, 16-byte aligned                   */
  void* out;               /* [numel] in out_dtype, 16-byte aligned                 */
  long long numel;         /* >= 0; 0 skips the tensor (its pointers may be NULL)   */
  int g_dtype, out_dtype;  /* muon_dtype                                            */
} muon_grad_tensor;

size_t muon_clip_workspace_bytes(int n_tensors);
muon_status muon_clip_grad_norm(const muon_grad_tensor* tensors, int n_tensors, float max_norm,
                                float eps, float* norm, void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * Path selection (no counterpart on the pages).  With enable = 1 (the default)
 * every matrix with 64 <= min(rows, cols) <= 256 and max(rows, cols) <= 512
 * runs all its NS rounds in one kernel, one CTA pair per matrix, with X, A and
 * B' held on chip between rounds; enable = 0 sends it through the staged
 * tensor-core path (three GEMM launches per round, with A and B' in the
 * workspace).  The grouped prologue and apply are the same on both paths.
 * A call that also holds matrices outside that range (which need the staged
 * launches) runs all of them staged, since the fused kernel would run before
 * the staged chain rather than beside it.
 * Both compute the same step and need the same workspace size.  Process-wide;
 * affects calls made afterwards.  Returns the previous setting, or -1 (nothing
 * changed) if enable is not 0 or 1.
 */
int muon_set_fused_ns(int enable);

/*
 * Launch structure of the tensor-core NS rounds (no counterpart on the pages).
 * mode = 0: one grouped launch per stage and round (Gram, Poly, Update; 15
 * launches for five rounds), each waiting for the one before.
 * mode = 1: one persistent launch covers every stage of every round; a tile
 * starts as soon as the tiles of the stages before it of the same matrix are
 * stored (per-matrix completion counters in the workspace), so one matrix's
 * next stage overlaps other matrices' current one.
 * mode = 2 (the default): 1 for groups whose rounds are short (estimated
 * tensor-core time of a round under 400 us), where the stage boundaries weigh
 * most; 0 otherwise.  Same results and workspace size in every mode.
 * The persistent launch needs all of its clusters (one per two SMs that fit
 * at once) resident together, since tiles wait for tiles of other clusters:
 * kernels on other streams that hold SMs delay it, and if they hold them for
 * more than its 2 s wait limit the step reports MUON_ERR_TIMEOUT.  Mode 0 has
 * no such requirement.
 * Process-wide; affects calls made afterwards.  Returns the previous mode, or
 * -1 (nothing changed) if mode is not 0, 1 or 2.
 */
int muon_set_persistent_rounds(int mode);

/*
 * Where the parameter write runs (no counterpart on the pages).  enable = 1
 * (the default): when every tensor-core matrix of a muon_step or
 * muon_step_grouped call goes through one staged NS chain (one persistent
 * rounds launch, or one launch per stage and round; see above), every weight's
 * cols is a multiple of 8, and rows and cols of every rows > cols weight are
 * multiples of 8, the write is launched right behind the last update (the
 * rounds kernel, or the last round's update launch) and runs beside it: its
 * blocks take the matrices in the order that update ends them (waiting,
 * bounded, on per-matrix completion counters), and the last round stores O of
 * a rows > cols matrix already transposed.  enable = 0: the write runs after
 * the NS.  Same results and workspace size either way; muon_ns5 always uses
 * the second form.
 * Process-wide; affects calls made afterwards.  Returns the previous setting.
 */
int muon_set_streamed_apply(int enable);

/* Static English text for a status code. */
const char* muon_status_string(muon_status status);

/* Kernels this library has launched in this process (all devices, all calls). */
unsigned long long muon_kernel_launch_count(void);

/*
 * Optional kernel timing trace (off by default; host-side bookkeeping only).
 * muon_trace_begin(n): from now on, record a CUDA event before and after each
 * kernel the library launches, on that launch's stream, for up to n launches.
 * muon_trace_end(out, max, &count): synchronise on the recorded events, fill
 * up to `max` records (in launch order), set `count`, and stop tracing.
 * flops/bytes are the launch's algorithmic work: for GEMM stages the dense
 * flops of the tiles the stage is defined on (2 m^2 n for the Gram and for the
 * update, 2 m^3 for the polynomial, each counted once for symmetric outputs
 * as m(m+1)/2 entries), for the prologue the bytes it must move.
 */
typedef struct muon_trace_record {
  int kind;        /* muon_kernel_kind                          */
  int round;       /* NS round (0-based), -1 if not an NS stage */
  float ms;        /* event-to-event time on the launch stream  */
  double flops;    /* algorithmic flops of the launch           */
  double bytes;    /* algorithmic HBM bytes of the launch       */
} muon_trace_record;

muon_status muon_trace_begin(int max_launches);
muon_status muon_trace_end(muon_trace_record* out, int max_records, int* count);

#ifdef __cplusplus
}
#endif

#endif /* MUON_GB300_H */
