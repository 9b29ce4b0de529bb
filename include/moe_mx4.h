/*
 * moe_mx4.h - C ABI of the layer's experts in microscaled 4-bit floating point (sm_100a):
 * quantisation, the ragged grouped product on two 4-bit operands and the grouped SwiGLU FFN
 * made of it. Conventions, status codes and limits are those of moe.h: buffers are the
 * caller's, calls are asynchronous on `stream`, arguments are checked on the host before
 * anything is launched, nothing allocates or synchronises, every call can be captured.
 *
 * Formats. A row of K elements is split into blocks that share a scale. An element is an
 * e2m1 number: 0, 0.5, 1, 1.5, 2, 3, 4, 6 or the negative of one. With |x| the largest
 * magnitude of a block and e2m1() rounding to nearest, ties to even, at most 6:
 *   MOE_MX4_MXFP4  blocks of 32, scale byte e8m0: b = max(floor(log2 |x|) - 2, -127) + 127,
 *                  element e2m1(x * 2^(127 - b)), value element * 2^(b - 127). A block that
 *                  holds an infinity or a NaN gets b = 255, and all its values are NaN.
 *   MOE_MX4_NVFP4  blocks of 16, scale byte e4m3: s = e4m3(|x| / (6 t)) (at most 448), element
 *                  e2m1(x / (s t)), value element * s * t, with t the tensor's fp32 factor
 *                  (1 when no factor is given; positive, from 2^-100 to 2^100). A block with
 *                  s = 0 is all zeros. A block with an infinity or a NaN gets the e4m3 NaN,
 *                  and all its values are NaN.
 * The fp32 operations round to nearest: 6 t, |x| / (6 t), s t and x / (s t), one each.
 *
 * Rows and groups. A 4-bit matrix has `rows` rows of K elements in `groups` groups, group g
 * the rows [o_g, o_{g+1}):
 *   ragged   o = `offsets`, device int32 [groups + 1], ascending from 0, o_groups <= rows.
 *            Rows from o_groups on belong to no group: no call writes them, and what they hold
 *            has no effect. (The products report offsets that are not so as
 *            MOE_ERR_DEVICE_CHECK and keep to the buffers; their outputs are then undefined,
 *            and not written where the offsets are out of order.)
 *   uniform  `offsets` NULL: o_g = g * group_rows, groups * group_rows == rows.
 *
 * Layout. codes: [rows, K / 2] bytes, the even element of a pair in the low half. scales: the
 * tensor cores read the scales of 128 rows x 4 blocks as one 512-byte piece, so row l of a
 * group (counted within the group) keeps the scale of block b at
 *   ((o_g / 128 + g + l / 128) * (K / (4 B)) + b / 4) * 512 + (l % 32) * 16
 *   + (l % 128) / 32 * 4 + b % 4                         (B elements per block, / rounds down)
 * A group's pieces start at o_g / 128 + g, which leaves every group room for its last,
 * partly filled 128 rows whatever the offsets are; moe_mx4_scale_bytes gives the buffer's
 * size. Scale bytes of rows that a group does not have are never used.
 *
 * Limits: K >= 128 and a multiple of 128, 1 <= groups <= 1024, 0 <= rows < 2^31 - 1025,
 * rows * K < 2^46. Other sizes give MOE_ERR_UNSUPPORTED (negative ones and a group_rows that
 * does not match MOE_ERR_INVALID_ARG). rows = 0 checks the arguments and launches nothing.
 */
#ifndef MOE_B200_MX4_H_
#define MOE_B200_MX4_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_MX4_MXFP4 = 0, MOE_MX4_NVFP4 = 1 } moe_mx4_format_t;

/* One 4-bit matrix. */
typedef struct {
  int32_t format;            /* moe_mx4_format_t                                          */
  int32_t rows;              /* rows of the codes buffer                                  */
  int32_t K;                 /* elements per row                                          */
  int32_t groups;
  int32_t group_rows;        /* uniform groups: rows per group; ragged groups: 0          */
  int32_t factor_per_group;  /* NVFP4: `factor` holds one fp32 per group (1) or one (0)   */
  const int32_t* offsets;    /* device [groups + 1], or NULL: uniform groups              */
  const float* factor;       /* device fp32, positive: t above; NULL: 1. NULL for MXFP4   */
  void* codes;               /* device                                                    */
  void* scales;              /* device                                                    */
} moe_mx4_t;

/* Bytes of the scales buffer of a matrix (its pointers are not looked at). */
int moe_mx4_scale_bytes(const moe_mx4_t* m, size_t* bytes);

/* Quantises the rows of x into m.
 *   x       device, `dtype` elements (moe_dtype_t), row r at x + r * ld; ld >= K, and the
 *           rows 16-byte aligned
 *   row_of  NULL: row r of m is row r of x (tokens == rows, picks ignored). Else device
 *           int32 [tokens, picks]: row t of x goes to the rows row_of[t, 0 .. picks) of m
 *           that are not negative (moe_permute's row_of: the rows of the token's FFN picks,
 *           each token read and rounded once). Entries >= o_groups are skipped. At most 32
 *           picks, and no factor_per_group.
 *   status  device int32 or NULL: MOE_ERR_DEVICE_CHECK for an entry >= o_groups */
int moe_mx4_quantize(const moe_mx4_t* m, const void* x, int32_t dtype, int64_t ld,
                     const int32_t* row_of, int32_t tokens, int32_t picks, int32_t* status,
                     void* stream);

/* The values of m: out device, `dtype` elements, row r at out + r * ld (as for x above),
 * rounded once to bf16. Rows that belong to no group are not written. */
int moe_mx4_dequantize(const moe_mx4_t* m, void* out, int32_t dtype, int64_t ld, void* stream);

/* Scale bytes of a checkpoint, row-major device [rows, K / B], into m's scales (m's codes are
 * not looked at: a checkpoint's packed codes are used as they are). */
int moe_mx4_pack_scales(const moe_mx4_t* m, const void* row_major, void* stream);

/* y[r, n] = sum_k A[r, k] W[g, n, k] for the rows r of group g: the product of ragged rows
 * with each group's own weight, in 4 bits on both sides, accumulated in fp32.
 *   a       [rows, K] in ragged (or uniform) groups, one factor at most
 *   w       uniform groups: group_rows = N rows of K elements per group; same groups, K and
 *           format as a; one factor per group, or one
 *   out     device [a.rows, N] `dtype` elements; rows that belong to no group are not written
 *   ws      device, >= moe_mx4_gemm_workspace_size bytes, zeroed before first use (a status
 *           word: moe_read_device_status). Calls that run at once need one each. */
int moe_mx4_gemm_workspace_size(size_t* bytes);
int moe_mx4_grouped_gemm(const moe_mx4_t* a, const moe_mx4_t* w, void* out, int32_t dtype,
                         void* ws, size_t ws_bytes, void* stream);

/* Grouped SwiGLU FFN on 4-bit experts (report §2.4: intermediate I per expert):
 *   h = q(silu(A Wg^T) * (A Wu^T)),  y = h Wd^T
 * with q() the rounding of h to a's format (h_factor: its t, device fp32 [1] or NULL; NULL
 * for MXFP4) by the operations above. silu and the product are fp32, good to a few units in the
 * last place, and the sums A Wg^T, A Wu^T go in the tensor cores' order: an h that lies that
 * near the middle of two 4-bit numbers, or its block's |h| / (6 t) that of two scales, may go
 * either way. h never exists in more than 4 bits.
 *   a          [rows, H], ragged or uniform groups
 *   w_gate_up  uniform groups of 2I rows of H elements: rows [0, I) gate, [I, 2I) up
 *   w_down     uniform groups of H rows of I elements
 *   out        store (perm_token NULL): device [a.rows, H] `dtype`, out[r] = y[r].
 *              fused combine: device fp32 [*, H] (dtype MOE_FP32), out[perm_token[r]] +=
 *              scale * row_gate[r] * y[r] by fp32 atomic adds (moe_permute's perm_token and
 *              row_gate, which go together, [a.rows] each; the summation order, hence the last
 *              bits, vary run to run)
 *   ws         device, >= moe_mx4_ffn_workspace_size bytes, zeroed before first use (status
 *              word, h). Calls that run at once need one each.
 * I is a multiple of 128. */
int moe_mx4_ffn_workspace_size(const moe_mx4_t* a, const moe_mx4_t* w_gate_up, size_t* bytes);
int moe_mx4_grouped_ffn(const moe_mx4_t* a, const moe_mx4_t* w_gate_up, const moe_mx4_t* w_down,
                        const float* h_factor, const int32_t* perm_token, const float* row_gate,
                        float scale, void* out, int32_t dtype, void* ws, size_t ws_bytes,
                        void* stream);

#ifdef __cplusplus
}
#endif
#endif
