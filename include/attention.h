/*
 * attention -- softmax(scale * Q K^T) V on AMD Instinct MI355X (gfx950), in
 * fp16 and bf16, beside the products of gemm_f16_nt.h in the same library.
 *
 * Heads: a tensor has `heads` query heads and `kv_heads` key/value heads,
 * heads a multiple of kv_heads; query head h reads kv head
 * h / (heads / kv_heads).  head_dim is a multiple of 8 up to 128 (64, 96 and
 * 128 run at full speed, others as the next of these).
 *
 * Scores, softmax statistics, sums and the output accumulate in fp32; the
 * softmax weights are rounded to the operands' type before the product with
 * V (where no more than 32 rows meet the keys the rest of that rounding goes
 * as a second operand), and O is rounded once, to nearest even.  q . k may be
 * as large as fp32 holds.  O is finite for finite V: in fp16 always, in bf16
 * where a row's weights, the largest taken as 1, add up to 256 or less, or V
 * stays that much below the type's largest value.  A value of V that is not
 * finite, at a key that a row reads, makes that element of the row's O an
 * infinity or NaN.  A row that no key is left for
 * gets O = +0 and lse = -inf.  lse, where asked for, is the natural
 * logarithm of sum_j exp(scale * q . k_j), fp32.  A negative scale is taken
 * as it is; for scale 0 every score is 0, whatever Q and K hold.
 *
 * The calls compute results, not gradients.
 *
 * Keys that a mask or a length leaves out have no part in the results of
 * the rows they are left out for, whatever they hold (infinities and NaN
 * included).
 *
 * Strides are in elements.  Elements of a head are contiguous, Q, K, V and O
 * and all their strides are on 16-byte boundaries (multiples of 8 elements),
 * strides are >= 0 (0 repeats an input), and a row of keys or values is less
 * than 2^23 elements from the next.  A call has at most 2^22 units of work,
 * kv_heads times (total_q * group / 128 + sequences) for attn_prompt and
 * kv_heads times (batch * group / 128 + batch * ceil(group / 32) *
 * (slot_rows / 2048 + 1)) for attn_shared_prefix, with group = heads /
 * kv_heads; more is UNSUPPORTED.  O and lse must not overlap an input or
 * each other, where a tensor counts as all memory from its first to its last
 * element; and O's rows and heads must not overlap each other.
 *
 * Calls are asynchronous and stream-ordered: they validate, enqueue and
 * return; validation comes before any HIP call, and an invalid call launches
 * nothing.  Lengths and offsets that live in device memory are read by the
 * kernels and clamped to the tensors' sizes, so that no value in them leads
 * to an access out of bounds.  The library keeps nothing between calls; the
 * same inputs give the same bits.  Status codes are those of gemm_f16_nt.h.
 *
 * Workspace: some calls split the keys among workgroups and join the parts
 * in a second launch.  They need attn_*_workspace(...) bytes of device
 * memory (16-byte aligned, not overlapping the other arguments; contents are
 * scratch, nothing needs clearing).  The size follows from the descriptor's
 * sizes and `causal` alone, not from lengths in device memory.  Calls that may overlap in
 * time need a workspace each.
 */
#ifndef ATTENTION_H
#define ATTENTION_H

#include <stdint.h>

#include "gemm_f16_nt.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_F16 0
#define ATTN_BF16 1

/* Attention of whole prompts, packed without padding.  Sequence b of `batch`
 * has queries cu_q[b] .. cu_q[b+1] - 1, rows of Q, O and lse, and keys
 * cu_k[b] .. cu_k[b+1] - 1, rows of K and V (int32, device memory, batch + 1
 * values each, not decreasing).  With `causal`, query i of n reads keys
 * j <= i + (keys - n): the last query reads every key, so a chunk of a prompt
 * runs against all keys so far, and a single new token against its cache.
 * Rows of O and lse that belong to no sequence are left as they were.  Each
 * workgroup looks through the sequences, 64 at a time, for its own. */
typedef struct attn_prompt_desc {
    int32_t dtype;  /* ATTN_F16 or ATTN_BF16 */
    int32_t causal; /* 0 or 1 */
    int32_t heads, kv_heads, head_dim;
    int32_t batch;             /* sequences */
    int64_t total_q, total_k;  /* rows of Q (O, lse) and of K (V) */
    const void* Q;             /* row r, head h at Q + r*q_row + h*q_head */
    const void* K;
    const void* V;
    void* O;
    float* lse;                /* total_q x heads, contiguous; or NULL */
    const int32_t* cu_q;
    const int32_t* cu_k;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;
    float scale;
} attn_prompt_desc;

int attn_prompt(const attn_prompt_desc* d, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace attn_prompt needs for d on the current device (0: none),
 * or a negative status. */
int64_t attn_prompt_workspace(const attn_prompt_desc* d);

/* The status attn_prompt would return before launching anything; no HIP
 * call.  The workspace is not looked at. */
int attn_prompt_check(const attn_prompt_desc* d);

/* One new token for each sequence of a batch that shares a prefix: row b of
 * Q attends to all `prefix` keys of Kp and Vp and to the first lens[b] rows
 * of its own slot of Ks and Vs (int32, device memory; the token's own key
 * among them, if it is to be read).  The prefix is read once for all rows of
 * the batch.  lens[b] above `slot_rows` counts as slot_rows; where lens[b] is
 * negative the slot is not in use, and row b of O and lse is left as it
 * was. */
typedef struct attn_shared_prefix_desc {
    int32_t dtype;
    int32_t heads, kv_heads, head_dim;
    int64_t batch;      /* rows of Q, O and lse, slots of Ks and Vs */
    int64_t prefix;     /* rows of Kp and Vp */
    int64_t slot_rows;  /* rows of a slot */
    const void* Q;      /* batch x heads x head_dim */
    const void* Kp;     /* prefix x kv_heads x head_dim */
    const void* Vp;
    const void* Ks;     /* batch x slot_rows x kv_heads x head_dim */
    const void* Vs;
    void* O;
    float* lse;         /* batch x heads, contiguous; or NULL */
    const int32_t* lens;
    int64_t q_row, q_head, kp_row, kp_head, vp_row, vp_head;
    int64_t ks_slot, ks_row, ks_head, vs_slot, vs_row, vs_head, o_row, o_head;
    float scale;
} attn_shared_prefix_desc;

int attn_shared_prefix(const attn_shared_prefix_desc* d, void* workspace, int64_t workspace_bytes, void* stream);
int64_t attn_shared_prefix_workspace(const attn_shared_prefix_desc* d);
int attn_shared_prefix_check(const attn_shared_prefix_desc* d);

#ifdef __cplusplus
}
#endif

#endif /* ATTENTION_H */
