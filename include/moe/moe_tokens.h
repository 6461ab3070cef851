/*
 * moe_tokens.h — C ABI of the gfx950 token movement around an expert layer:
 * tokens sorted by expert, gathered into the token groups that the grouped
 * casts and products take, and their answers summed back with the router's
 * weights, with the gradients of both moves.
 *
 * A router gives each of T tokens k expert ids and k weights. Slot i = t*k + j
 * is token t's j-th choice; R = T*k. A slot whose id lies outside
 * [0, num_experts) belongs to an expert held elsewhere and is "dropped".
 *
 * The plan (moe_sort_tokens), integers only and the same on every run:
 *   group_end_offsets[e]  number of slots with an id in [0, e]: the cumulative
 *                         ends (rows) that every M-groups entry point takes.
 *   order[r]              sorted row r < group_end_offsets[E-1]: its slot. Rows
 *                         are sorted by expert, slots of one expert ascending.
 *                         The rows past the last end hold the dropped slots,
 *                         ascending, each as ~slot (a negative number).
 *   position[i]           slot i's row; ~row for a dropped slot.
 *
 * The moves (rows in bf16, f16 or f32; sums in binary32, in the order of j,
 * rounded once to the rows' type):
 *   gather            out[position[i]] = x[t];  rows of dropped slots are zero
 *   gather_backward   dx[t] = sum_j dgathered[position[t*k+j]]
 *   combine           out[t] = sum_j w[t,j] * y[position[t*k+j]]
 *   combine_backward  dy[position[i]] = w[i] * dout[t], zero for dropped slots;
 *                     dweights[i] = <dout[t], y[position[i]]>, 0 for dropped
 * A dropped slot adds nothing to a sum, whatever its row holds (infinities and
 * NaN included). A token whose slots are all dropped gets a row of zeros.
 *
 * Positions outside [-R, R) are taken as dropped and nothing is written for
 * them, so no call reads or writes outside its buffers.
 *
 * Sizes: R + 4096 < 2^31; 1 <= topk <= 64; 1 <= num_experts <= 4096; row widths
 * cols <= 2^24; row strides (elements) in [cols, 2^26]. Rows need only their
 * type's alignment.
 * Ownership: the caller owns every buffer, the workspace too; nothing is
 * allocated or kept. Calls are thread-safe. Errors: the MX_REARRANGE_* status
 * codes of mx_rearrange.h, nothing enqueued.
 */
#ifndef MOE_TOKENS_H
#define MOE_TOKENS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct ihipStream_t;
typedef struct ihipStream_t *hipStream_t;

/* Element types of the moved rows. */
enum { MOE_BF16 = 0, MOE_F16 = 1, MOE_F32 = 2 };

/* The size helper below is a static inline function of this header, not a library symbol. */

/*
 * Bytes of the workspace of moe_sort_tokens: one count for each expert (and one
 * for the dropped slots) and run of 1024 slots, and one total for each; 0 for up to
 * 16384 slots and 2048 experts, which one workgroup sorts alone, and for no slots.
 * -1 for invalid sizes.
 */
static inline int64_t moe_sort_tokens_workspace_bytes(int64_t tokens, int32_t topk, int32_t num_experts) {
  if (tokens < 0 || topk < 1 || topk > 64 || num_experts < 1 || num_experts > 4096 ||
      tokens > ((int64_t)0x7fffffff - 4096) / topk)
    return -1;
  if (tokens == 0 || (tokens * topk <= 16384 && num_experts <= 2048)) return 0;
  return 4 * ((int64_t)num_experts + 1) * ((tokens * topk + 1023) / 1024 + 1);
}

/*
 * expert_ids         device, tokens x topk ids of id_bytes bytes each (4: int32,
 *                    8: int64), token t's at element t*row_stride; NULL allowed
 *                    when tokens == 0.
 * row_stride         topk <= row_stride <= 2^26 elements.
 * group_end_offsets  device int32[num_experts]; order, position: device
 *                    int32[tokens*topk], NULL allowed when tokens == 0.
 * workspace          device, 4-byte aligned, moe_sort_tokens_workspace_bytes
 *                    bytes; NULL allowed when that is 0.
 * One kernel on `stream` where the workspace is 0 bytes, two up to 64 runs, else three.
 */
int moe_sort_tokens(const void *expert_ids, int32_t id_bytes, int64_t tokens, int32_t topk, int64_t row_stride,
                    int32_t num_experts, int32_t *group_end_offsets, int32_t *order, int32_t *position,
                    void *workspace, hipStream_t stream);

/*
 * x          device, tokens x cols of `type`, row t at x + t*row_stride elements.
 * position   device int32[tokens*topk].
 * out        device, (tokens*topk) x cols, row stride out_stride elements.
 * One kernel on `stream`; every row of a valid plan is written.
 */
int moe_gather_tokens(const void *x, int32_t type, int64_t tokens, int32_t topk, int64_t cols, int64_t row_stride,
                      const int32_t *position, void *out, int64_t out_stride, hipStream_t stream);

/*
 * y          device, (tokens*topk) x cols of `type`, row stride row_stride.
 * weights    device float[tokens*topk], or NULL: every weight 1 (the gradient of
 *            moe_gather_tokens).
 * out        device, tokens x cols, row stride out_stride.
 */
int moe_combine_tokens(const void *y, int32_t type, int64_t tokens, int32_t topk, int64_t cols, int64_t row_stride,
                       const int32_t *position, const float *weights, void *out, int64_t out_stride,
                       hipStream_t stream);

/*
 * dout       device, tokens x cols, row stride dout_stride; y as above.
 * weights    device float[tokens*topk]
 * dy         device, (tokens*topk) x cols, row stride dy_stride; must not overlap y.
 * dweights   device float[tokens*topk].
 */
int moe_combine_tokens_backward(const void *dout, int32_t type, int64_t tokens, int32_t topk, int64_t cols,
                                int64_t dout_stride, const void *y, int64_t row_stride, const int32_t *position,
                                const float *weights, void *dy, int64_t dy_stride, float *dweights,
                                hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TOKENS_H */
