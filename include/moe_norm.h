/*
 * moe_norm.h - C ABI of the norms around a block (sm_100a): the RMS norm after a block, its
 * gate and residual scale, the residual add and the RMS norm before the next block in one
 * call, and their gradients. Conventions and status codes are those of moe.h.
 *
 * Per token t (report §2.1: the layer's blocks sit on a residual stream):
 *   n1 = w_post * block_t * rstd(block_t)          (w_post NULL: n1 = block_t)
 *   r  = residual_t + scale * gate * n1            rounded to dtype: residual_out_t
 *   n2 = w_pre * r * rstd(r)                       of the rounded r: normed_t
 * with rstd(v) = 1 / sqrt(mean(v^2) + eps). Everything is fp32 and rounded once on its way
 * out. Since n2 reads the r that is stored, one call gives the bits of two.
 *
 * Parts are left out by NULL pointers, which have to agree with one another:
 *   block NULL   r = residual: no w_post, gate, residual_out or rstd_block
 *   w_pre NULL   no norm before the next block: no normed or rstd_res
 * Limits: H % 16 == 0, H <= 16384, T < 2^24 (MOE_ERR_UNSUPPORTED otherwise). T = 0 is valid
 * (the [T, H] and [T] pointers may then be anything): the backward writes zeros to the sums
 * over tokens that it is given, and nothing else is written.
 */
#ifndef MOE_B200_NORM_H_
#define MOE_B200_NORM_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* gate: none (1), one fp32 per token [T], or one fp32 per channel [H]. */
typedef enum { MOE_GATE_NONE = 0, MOE_GATE_TOKEN = 1, MOE_GATE_CHANNEL = 2 } moe_gate_t;

typedef struct {
  int32_t T, H;
  int32_t dtype;     /* moe_dtype_t: residual, block, residual_out, normed and gradients  */
  int32_t gate;      /* moe_gate_t                                                        */
  float eps;         /* > 0                                                               */
  float scale;       /* residual scale on the gated block output; finite                  */
} moe_norm_t;

/*   residual      device [T, H] dtype
 *   block         device [T, H] dtype or NULL
 *   w_post        device [H] fp32 or NULL
 *   gate          device fp32 [T] or [H] by n->gate, NULL for none
 *   w_pre         device [H] fp32 or NULL
 *   residual_out  device [T, H] dtype (may be `residual` itself)
 *   normed        device [T, H] dtype
 *   rstd_block    device [T] fp32 or NULL: kept for the backward (with w_post only)
 *   rstd_res      device [T] fp32 or NULL: kept for the backward */
int moe_block_norm(const moe_norm_t* n, const void* residual, const void* block,
                   const float* w_post, const float* gate, const float* w_pre,
                   void* residual_out, void* normed, float* rstd_block, float* rstd_res,
                   void* stream);

/* Gradients of moe_block_norm for d_residual_out and d_normed, the gradients that come back
 * on the residual stream and on the next block's input:
 *   g       = d_residual_out + through the norm before the next block, from d_normed
 *   d_residual = g;  d_gate = scale * sum g n1;  dn1 = scale * gate * g
 *   d_block = through the norm after the block, from dn1;  d_w_post = sum_t dn1 * block rstd
 *   d_w_pre = sum_t d_normed * residual_out rstd
 * The rounding of r is passed through as the identity. Inputs as above, and
 *   residual_out          device [T, H] dtype: the forward's (with block NULL: `residual`)
 *   rstd_block, rstd_res  device [T] fp32 from the forward
 *   d_residual_out        device [T, H] dtype or NULL: zero
 *   d_normed              device [T, H] dtype (with w_pre)
 * Outputs: d_residual [T, H] dtype, d_block [T, H] dtype, d_w_post [H], d_w_pre [H] and d_gate
 * ([T] or [H]) fp32, written, each for the parts the forward had and NULL otherwise. The sums
 * over tokens go in a fixed order: bit-reproducible.
 *   ws  device, >= moe_block_norm_workspace_size bytes, zeroed before first use (status word, read
 *       with moe_read_device_status; partial sums); calls that run at once need one each */
int moe_block_norm_workspace_size(const moe_norm_t* n, size_t* bytes);
int moe_block_norm_backward(const moe_norm_t* n, const void* d_residual_out, const void* d_normed,
                            const void* residual_out, const void* block, const float* w_post,
                            const float* gate, const float* w_pre, const float* rstd_block,
                            const float* rstd_res, void* d_residual, void* d_block,
                            float* d_w_post, float* d_gate, float* d_w_pre, void* ws,
                            size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif
