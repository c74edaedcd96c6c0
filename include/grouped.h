/*
 * grouped -- products of many matrices in one call on AMD Instinct MI355X
 * (gfx950), in fp16 and bf16, beside the products of gemm_f16_nt.h in the same
 * library: the three products of layers whose rows are divided among matrices
 * (experts), and a projection shared by all rows with the low-rank adapters of
 * many requests beside it.
 *
 * Rows of a tensor are divided by a table of offsets in device memory: group e
 * (a matrix, or a request) has the rows cu[e] .. cu[e + 1] - 1 (int32, groups +
 * 1 values, not decreasing).  Groups may be empty.  The kernels read the table
 * and clamp it to the tensors' sizes, so that no value in it leads to an
 * access out of bounds; no call synchronises.  Rows before the first and
 * behind the last group are left as they were in what a call writes, and have
 * no part in any result.
 *
 * Sums accumulate in fp32 and are rounded once, to nearest even.  An output
 * depends on its own row and matrix alone: values elsewhere, infinities and
 * NaN included, have no part in it.
 *
 * Strides are in elements.  Elements of a row are contiguous; N, K and rank
 * are multiples of 8 and all rows start on 16-byte boundaries (strides are
 * multiples of 8, addresses of 16); others are UNSUPPORTED, as are widths and
 * row pitches of 2^22 elements or more, 2^22 groups, requests or adapters or
 * more, more than 2^31 - 1024 rows, and calls of more than 2^22 output tiles
 * (counted as 128 x 128 elements, for the low-rank projections 64 x 128).  Row
 * pitches are at least as long as a row; matrices that are read may repeat
 * (stride_b 0).  What a call writes must not overlap anything that it reads.
 *
 * Calls are asynchronous and stream-ordered: they validate, enqueue and
 * return; validation comes before any HIP call, and an invalid call launches
 * nothing.  The library keeps nothing between calls; the same inputs give the
 * same bits.  Status codes are those of gemm_f16_nt.h.
 *
 * Workspace: calls with few tiles and a long contraction divide it among
 * workgroups and join the parts in a second launch; adapter_nt keeps the
 * low-rank projections.  They need ..._workspace(...) bytes of device memory
 * (16-byte aligned, not overlapping the other arguments; contents are scratch,
 * nothing needs clearing).  The size follows from the descriptor's sizes and
 * strides alone, not from the tables in device memory.  Calls that may overlap
 * in time need a workspace each.
 */
#ifndef GROUPED_H
#define GROUPED_H

#include <stdint.h>

#include "gemm_f16_nt.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GROUPED_F16 0
#define GROUPED_BF16 1

#define GROUPED_NT 0
#define GROUPED_NN 1
#define GROUPED_TN 2

/* Rows r of group e and the group's matrix B_e (N x K):
 *
 *   grouped_nt   D[r] = B_e A[r]                            reads A, B, writes D
 *   grouped_nn   A[r] = B_e^T D[r]                          reads D, B, writes A
 *   grouped_tn   B_e = sum over the rows of D[r] A[r]^T     reads D, A, writes B
 *
 * With A and D taken as gradients where they are written or read as such, the
 * second and third are the gradients of the first.  grouped_tn writes every
 * matrix: zeros for a group without rows. */
typedef struct grouped_desc {
    int32_t dtype;   /* GROUPED_F16 or GROUPED_BF16, of A, B and D */
    int32_t b_fp32;  /* 1: grouped_tn writes B in fp32 (ldb and stride_b count its elements); otherwise 0 */
    int64_t groups;
    int64_t rows;    /* of A and D */
    int64_t N, K;
    void* A;         /* rows x K, row r at A + r*lda */
    void* B;         /* groups x N x K, row n of matrix e at B + e*stride_b + n*ldb */
    void* D;         /* rows x N, row r at D + r*ldd */
    int64_t lda, ldb, stride_b, ldd;
    const int32_t* cu;
} grouped_desc;

int grouped_nt(const grouped_desc* d, void* workspace, int64_t workspace_bytes, void* stream);
int grouped_nn(const grouped_desc* d, void* workspace, int64_t workspace_bytes, void* stream);
int grouped_tn(const grouped_desc* d, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace a call needs on the current device (0: none), or a
 * negative status. */
int64_t grouped_nt_workspace(const grouped_desc* d);
int64_t grouped_nn_workspace(const grouped_desc* d);
int64_t grouped_tn_workspace(const grouped_desc* d);

/* The status a call would return before launching anything; no HIP call. */
int grouped_nt_check(const grouped_desc* d);
int grouped_nn_check(const grouped_desc* d);
int grouped_tn_check(const grouped_desc* d);

/* Host evaluation of what a call (`product`: GROUPED_NT, ...) runs on a device
 * with `cus` compute units, no HIP call: tiles of tile[0] rows and tile[1]
 * columns, and *parts parts of the contraction (0: the device divides a last
 * round of large tiles where that is a small one).  All are 0 for a call that
 * writes nothing.  Returns 0 or a negative status. */
int gemm_f16_nt_grouped_plan(const grouped_desc* d, int product, int cus, int tile[2], int64_t* parts);

/* One projection for all rows, and beside it the adapter that a row's request
 * asks for:
 *
 *   D[r] = B A[r] + scale_a * up_a (down_a A[r]),   a = ids[request of r]
 *
 * ids[b] outside 0 .. adapters - 1 (-1, say) means that request b has no
 * adapter: its rows are B A[r].  Any number of requests may share an adapter,
 * and a request is any number of rows: a prompt, or one token.
 *
 * scale_a * (down_a A[r]) is summed in fp32 and, as an operand of the second
 * product, held in two terms of the operands' type, which are off by at most
 * 2^-16 of it in bf16, by 2^-20 of it or 2^-25 in fp16 (calls with few rows for
 * a request keep it in fp32).  In fp16 it has to lie in that type's range;
 * everything else is one sum in fp32, rounded once. */
typedef struct adapter_desc {
    int32_t dtype;
    int32_t rank;          /* at most 128; smaller adapters are padded with zeros */
    int64_t adapters;
    int64_t requests;
    int64_t rows;          /* of A and D */
    int64_t N, K;
    const void* A;         /* rows x K */
    const void* B;         /* N x K, shared */
    void* D;               /* rows x N */
    const void* down;      /* adapters x rank x K */
    const void* up;        /* adapters x N x rank */
    const float* scales;   /* one for each adapter; or NULL: 1 */
    const int32_t* cu;     /* requests + 1 offsets of rows */
    const int32_t* ids;    /* the adapter of each request */
    int64_t lda, ldb, ldd, ld_down, stride_down, ld_up, stride_up;
} adapter_desc;

int adapter_nt(const adapter_desc* d, void* workspace, int64_t workspace_bytes, void* stream);
int64_t adapter_nt_workspace(const adapter_desc* d);
int adapter_nt_check(const adapter_desc* d);

/* The ways of a call: */
#define ADAPTER_ONE_LAUNCH 1   /* the projections as columns of the shared product's tiles */
#define ADAPTER_DOTS 2         /* the projections beside the shared product, then a dot product for each output */
#define ADAPTER_SUMS 3         /* the same, then tiles that begin with the shared product's sums */
#define ADAPTER_TILES 4        /* the projections, then tiles with the adapters as more of the contraction */
#define ADAPTER_EACH 5         /* the same in large tiles of one request each */

/* Host evaluation as above: the way, the shared product's tiles and parts, and
 * the projections' (0 without adapters or in one launch). */
int gemm_f16_nt_adapter_plan(const adapter_desc* d, int cus, int* way, int tile[2], int64_t* parts, int low_tile[2], int64_t* low_parts);

#ifdef __cplusplus
}
#endif

#endif /* GROUPED_H */
