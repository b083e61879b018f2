/*
 * libtaco -- the update of a training step for AMD Instinct MI355X (gfx950):
 * Adam with decoupled weight decay over many tensors at once, with its states in
 * fp32 or in 8 bits, and the global norm of their gradients.  Part of libtaco.so
 * beside the operators of taco_linear.h, whose block format holds the 8-bit
 * states and whose conventions hold here too.
 *
 * Tensors.  A call takes an array of descriptors in HOST memory, which is read
 * before the call returns; the pointers in it are DEVICE pointers, owned by the
 * caller.  A tensor is `count` consecutive elements, 0 <= count <= 2^34; one of no
 * elements is passed over, whatever its pointers.  Parameters, gradients, fp32
 * states and copies need no more than their element's alignment; codes are
 * 16-byte and scale bytes 4-byte aligned.  At most 2^20 tensors.
 *
 * Calls enqueue work on `stream` and return.  Arguments are checked on the host
 * before any launch: TACO_ERR_NULL, TACO_ERR_SHAPE (also for a number out of its
 * range), TACO_ERR_FLAGS (an unknown type), TACO_ERR_ALIGN, TACO_ERR_WORKSPACE,
 * TACO_ERR_ALIAS (anything written overlaps anything else that the call reads or
 * writes), and TACO_ERR_HIP for a failed launch.
 *
 * Results are deterministic: no atomics, every sum in one order for given counts.
 */
#ifndef TACO_OPTIM_H
#define TACO_OPTIM_H

#include "taco.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TACO_TYPE_FP32 0
#define TACO_TYPE_BF16 1

/*
 * A parameter tensor with its gradient and states.
 *   m, m_scale  the first moment: fp32 [count] and NULL, or uint8 codes and scale
 *               bytes of one row of `count` columns in the block format of
 *               taco_linear.h (of any length: count rounded up to 128 codes, one
 *               scale byte for each 128, rounded up to 4)
 *   v, v_scale  the same of the second moment: fp32 v, or codes of its root sqrt(v).
 *               Both states are in 8 bits, or neither.
 *   copy        bf16 [count]: receives the new parameters, for a product that takes
 *               them so; may be NULL, and is for bf16 parameters
 * A state before the first step is zeros (codes 0, scale bytes 127).
 */
typedef struct {
  void* param;
  const void* grad;
  void* m;
  void* v;
  uint8_t* m_scale;
  uint8_t* v_scale;
  void* copy;
  int64_t count;
  int32_t param_type;               /* TACO_TYPE_* */
  int32_t grad_type;
} taco_adamw_tensor_t;

/*
 *   step         of this update, from 1 on
 *   seed         of the stochastic roundings
 *   lr_device    fp32, step_device int64, one element each: read on the device in
 *                place of lr and step, so that a captured graph can be replayed
 *                with others (a step below 1 counts as 1); may be NULL
 *   grad_scale   fp32, one element on the device: a factor of every gradient; may be
 *                NULL.  Where it is not finite, the update is left out: nothing is
 *                written.
 * lr and weight_decay finite, betas in [0, 1), eps finite and >= 0.
 */
typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;
  uint64_t seed;
  const float* lr_device;
  const int64_t* step_device;
  const float* grad_scale;
} taco_adamw_options_t;

/*
 * One step for every tensor, in place, in fp32 for each element:
 *   g = grad * grad_scale
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   param = param (1 - lr weight_decay)
 *           - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * The update takes m and v before their rounding to 8 bits.
 *
 * Roundings.  Each product and sum of m and v, and sqrt(v), is rounded once to
 * nearest; fp32 states and parameters, and the bf16 copy, to nearest too.  A 3-bit
 * mantissa cannot follow moments that move by a thousandth a step, nor a bf16
 * parameter its updates, so these are rounded stochastically: a magnitude between
 * two neighbours of the format, a fraction f of their distance above the lower one,
 * becomes the upper one where f + (u + 1/2) / 2^16 >= 1, for 16 random bits u.
 * So the stored values follow the exact ones in the mean.  A root above 0 is never
 * stored as 0, but as the smallest code of its block at least: an element whose m
 * is stored would otherwise be divided by eps alone.
 *
 * The bits are Philox4x32 with seven rounds (Salmon et al., "Parallel random
 * numbers: as easy as 1, 2, 3", 2011), key seed (low word, high word), counter
 * (element / 8, call, tensor's place in the array, low word of step): with e =
 * element % 8, call e / 4, word e % 4 holds m's 16 bits and above them sqrt(v)'s;
 * call 2, word e / 2 holds those of a bf16 parameter, below for even e.
 *
 * A block of 8-bit states that comes to hold a NaN or an infinity is NaN throughout
 * from then on, as everywhere in the block format.
 */
taco_status_t taco_adamw_step(const taco_adamw_tensor_t* tensors, int64_t count,
                              const taco_adamw_options_t* options, taco_stream_t stream);

typedef struct {
  const void* data;
  int64_t count;
  int32_t type;                     /* TACO_TYPE_* */
} taco_norm_tensor_t;

/*
 * The global norm of many tensors, and the factor that clips it:
 *   out[0] = norm = sqrt(sum over all elements of x^2)
 *   out[1] = max_norm / norm where norm > max_norm, otherwise 1; NaN where norm is
 *            not finite (taco_adamw_step leaves such an update out)
 *   max_norm   > 0, or infinity: no clipping
 *   out        out: fp32 [2], 4-byte aligned
 *   workspace  partial sums, 256-byte aligned; needs no zero-fill
 * Squares and sums are fp64: no overflow, and one rounding to fp32 at the end.
 */
size_t taco_gradient_norm_workspace_bytes(int64_t count);
taco_status_t taco_gradient_norm(const taco_norm_tensor_t* tensors, int64_t count, double max_norm,
                                 float* out, void* workspace, size_t workspace_bytes,
                                 taco_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TACO_OPTIM_H */
