/*
 * flce_train.h -- C ABI of the training-step operators around the head, in libflce.so next to
 * flce.h's entry points: the norm of queries and keys per head with the position rotation in the
 * same pass (the write-ups' model: QK-norm, RoPE, grouped-query attention), the AdamW step over
 * many tensors at once (the write-ups' optimizer for the head, the embeddings and the norms) and
 * the global gradient norm with its clip factor.
 *
 * Conventions are flce.h's: device pointers owned by the caller, caller-owned workspace, nothing
 * allocated, `stream` a cudaStream_t (NULL = legacy default stream), asynchronous, argument errors
 * returned as a negative flce_status before anything is launched, results bitwise reproducible
 * from call to call on one device, no kernel traps.  Every call may be captured into a CUDA graph.
 * The device is the current one: every pointer must belong to it.
 */
#ifndef FLCE_TRAIN_H_
#define FLCE_TRAIN_H_

#include "flce.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ query / key norm + rotation
 * For every token and head, x one row of D elements of q (with gamma_q) or k (with gamma_k):
 *   rstd = 1 / sqrt(mean_j x_j^2 + eps),   n = x rstd gamma
 *   y = n with the pairs of its first `rot` elements rotated by angle_i = position * inv_freq[i],
 *       i < rot / 2:  (y_a, y_b) = (n_a cos - n_b sin, n_a sin + n_b cos)
 *   pairs: interleaved = 0: a = i, b = i + rot/2;  interleaved = 1: a = 2i, b = 2i + 1.
 *   Elements rot .. D-1 are normed only.  rot = 0: no rotation.
 * Norm and rotation run in fp32 and the result is rounded once.  The angle is formed in 64 bits and
 * reduced by whole turns before the sine and cosine are taken in fp32 (with what fp32 loses of the
 * reduced angle made up for): its error is about |position * inv_freq| 2^-52, so positions may be
 * far (or negative).
 */
typedef struct {
  int64_t B, T;          /* sequences, tokens of each; B * T < 2^31; 0 allowed */
  int64_t Hq, Hk;        /* query and key heads, each 0 .. 4096 (grouped-query attention: Hk < Hq) */
  int64_t D;             /* head size: a multiple of 16, at most 512 */
  int64_t rot;           /* rotated elements: a multiple of 16, 0 .. D */
  float eps;             /* >= 0 */
  int32_t interleaved;   /* pairing, see above */
  int32_t dtype;         /* FLCE_DTYPE_* of q, k, the outputs and their gradients */
  int32_t gamma_dtype;   /* FLCE_DTYPE_* of gamma_q and gamma_k */
} flce_qk_shape;

/* A [B, T, H, D] array: element (b, t, h, j) is ptr[b*batch + t*token + h*head + j] (strides in
 * elements).  ptr must be 16-byte aligned and each stride of a dimension larger than 1 a multiple
 * of 16 bytes.  ptr may be NULL only when the array has no element.  Arrays that are written must
 * not overlap themselves. */
typedef struct {
  void* ptr;
  int64_t batch, token, head;
} flce_qk_view;

/*
 * Forward.  gamma_q / gamma_k [D], 16-byte aligned, NULL = all ones.  inv_freq [rot/2] fp32
 * (NULL when rot = 0).  positions: int64, token t of sequence b at
 * positions[b*positions_batch + t] (positions_batch = 0: the same for every sequence), 8-byte
 * aligned; NULL: position t.  q_out / k_out may be the same views as q / k (in place); other
 * overlaps between inputs and outputs, or of one output with the other, are not allowed.
 */
int flce_qk_norm_rope_forward(const flce_qk_shape* shape, const flce_qk_view* q,
                              const flce_qk_view* k, const void* gamma_q, const void* gamma_k,
                              const float* inv_freq, const int64_t* positions,
                              int64_t positions_batch, const flce_qk_view* q_out,
                              const flce_qk_view* k_out, void* stream);

/*
 * Backward, from the gradients dq_out / dk_out of the forward's outputs and its inputs q, k (the
 * statistics are formed again from the rows, which are read anyway).  With d the gradient rotated
 * back, xh = x rstd and g = d gamma:
 *   dx = rstd (g - xh mean_j(g xh)),    dgamma = sum over tokens and heads of d xh
 * dq / dk are written (they may be the same views as dq_out / dk_out); dgamma_q / dgamma_k [D] fp32
 * are written, or added to with accumulate_dgamma = 1, and may be NULL (not wanted); they must not
 * overlap each other (FLCE_ERR_ARG): one gamma for queries and keys takes two gradients, whose sum is
 * its own.  dgamma is summed in a fixed order: per block of the launch in `workspace`, then over the blocks.
 * workspace: flce_qk_norm_rope_workspace_bytes(shape) bytes, 256-byte aligned; contents on entry
 * ignored.  Without rows, dgamma is zero.
 */
size_t flce_qk_norm_rope_workspace_bytes(const flce_qk_shape* shape);
int flce_qk_norm_rope_backward(const flce_qk_shape* shape, const flce_qk_view* dq_out,
                               const flce_qk_view* dk_out, const flce_qk_view* q,
                               const flce_qk_view* k, const void* gamma_q, const void* gamma_k,
                               const float* inv_freq, const int64_t* positions,
                               int64_t positions_batch, const flce_qk_view* dq,
                               const flce_qk_view* dk, float* dgamma_q, float* dgamma_k,
                               int accumulate_dgamma, void* workspace, size_t workspace_bytes,
                               void* stream);

/* ------------------------------------------------------------------------------------- AdamW
 * One step over `count` tensors, in one launch for every 384 of them.  With t = *step + 1 and
 * s = *grad_scale (1 when NULL), for every element, in fp32:
 *   g = s * grad,  m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
 *   w = w (1 - lr weight_decay) - lr/(1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
 * w is the fp32 master copy where there is one (param then receives w rounded), else the param.
 *
 * States in 8 bits (FLCE_STATE_E4M3): m and r = sqrt(v) are e4m3 codes with an fp32 scale for
 * every FLCE_STATE_BLOCK consecutive elements of the tensor (the last block may be shorter):
 *   scale = amax * (1/448 rounded to fp32), rounded: at most one unit of the last place from
 *     the rounded amax / 448; 0 where it is below 2^-126 (the block then holds zeros);
 *   code = e4m3(x / scale), nearest even;  an r > 0 gets at least the smallest code, so that a
 *     denominator does not vanish next to a first moment that does not (the next step's v, the
 *     square of code * scale, is 0 only where that is below 2^-75).
 * The step itself uses m and v before they are rounded.
 */
enum { FLCE_STATE_F32 = 0, FLCE_STATE_E4M3 = 1 };
#define FLCE_STATE_BLOCK 256
#define FLCE_ADAMW_MAX_GROUPS 16

typedef struct {
  void* param;       /* [n], param_dtype */
  void* m;           /* [n] fp32 or e4m3 codes */
  void* v;           /* [n] fp32 v, or the e4m3 codes of r = sqrt(v) */
  float* m_scale;    /* [ceil(n / FLCE_STATE_BLOCK)]; 8-bit states only */
  float* r_scale;    /* the same for r */
  float* master;     /* [n] fp32, or NULL; needs a bf16 param */
  int64_t n;         /* elements, >= 0 */
  int32_t param_dtype, grad_dtype;   /* FLCE_DTYPE_* */
  int32_t state;                     /* FLCE_STATE_* */
  int32_t group;                     /* index into groups */
} flce_adamw_tensor;

typedef struct {
  double lr;              /* used when lr_device is NULL */
  const float* lr_device; /* learning rate on the device, so that a captured step can change it */
  double beta1, beta2;    /* in [0, 1) */
  double eps;             /* >= 2^-60: a v below 2^-126 counts as 0 in the denominator */
  double weight_decay;
} flce_adamw_group;

/*
 *   tensors, grads [count]: host arrays, read before the call returns.  grads[i] is a device
 *     pointer to n elements of grad_dtype; NULL leaves tensor i as it is.
 *   No two tensors may overlap, nor a gradient another tensor's arrays (a step writes its tensors in
 *     any order).  Pointers need their element's alignment only; the fast path takes fp32 arrays at
 *     32 and bf16 arrays and codes at 16 bytes.
 *   groups [n_groups], 1 <= n_groups <= FLCE_ADAMW_MAX_GROUPS: host array.
 *   step: device int64, the steps done so far; the call adds 1.  8-byte aligned.
 *   skip_nonfinite = 1: a grad_scale that is not finite (flce_grad_norm of gradients with an
 *     infinity or a NaN) leaves every tensor and *step as they are.
 *   scratch: four 32-bit words on the device, 16-byte aligned, zeroed before the first step; every
 *     call leaves them zero, but for word 1: it takes FLCE_DEV_TIMEOUT if a wait inside the kernel
 *     ran out (every wait is bounded).  Steps that share scratch or step must not overlap on the
 *     GPU.
 */
int flce_adamw_step(const flce_adamw_tensor* tensors, const void* const* grads, int64_t count,
                    const flce_adamw_group* groups, int n_groups, const float* grad_scale,
                    int64_t* step, int skip_nonfinite, void* scratch, void* stream);

/* -------------------------------------------------------------------------- gradient norm
 * norm[0] = sqrt(sum over all tensors of g^2) and, where factor is not NULL, the factor that clips
 * it: factor[0] = min(1, max_norm / (norm + 1e-6)), or NaN when norm is not finite.  Squares are
 * summed in fp32 by each thread, 64 of them (a gradient beyond 1.8e19 gives an infinite norm, the
 * square of one below 2.6e-23 counts as 0), and in 64 bits over threads, in a fixed order.
 *   grads, sizes, dtypes [count]: host arrays; grads[i] may be NULL (no gradient).
 *   workspace: flce_grad_norm_workspace_bytes(count) bytes, 256-byte aligned, contents on entry
 *   ignored.
 */
size_t flce_grad_norm_workspace_bytes(int64_t count);
int flce_grad_norm(const void* const* grads, const int64_t* sizes, const int32_t* dtypes,
                   int64_t count, float max_norm, float* norm, float* factor, void* workspace,
                   size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FLCE_TRAIN_H_ */
