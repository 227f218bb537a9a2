/*
 * packed_attn.h - C ABI of causal attention over packed sequences with
 * grouped heads, forward and backward (libpacked_attn.so).
 *
 * What is computed.  Sequences of different lengths n_0, n_1, ... lie one
 * behind another in the rows of q [T, Hq, D], k and v [T, Hkv, D]; the
 * sequence s owns rows c_s .. c_s + n_s - 1 with c_s = n_0 + ... + n_(s-1).
 * Hq is a multiple of Hkv and query head h reads K/V head h / (Hq / Hkv).
 * For a row i and the rows j <= i of its own sequence
 *     S_ij = scale <q_i, k_j>,  lse_i = log sum_j exp S_ij,
 *     P = exp(S - lse),  o_i = sum_j P_ij v_j
 * and, in the backward pass, the gradients dq, dk, dv of sum(o * dO):
 *     delta_i = <dO_i, o_i>,  dS_ij = P_ij (<dO_i, v_j> - delta_i),
 *     dv_j = sum_i P_ij dO_i,  dk_j = scale sum_i dS_ij q_i,
 *     dq_i = scale sum_j dS_ij k_j,
 * the sums of dk and dv running over every query head of the group.  No row
 * is empty (j = i is always there).  Rows behind the last sequence
 * (sum of the lengths <= row < T) are not read into any result and the
 * output rows there are left as they were.  Nothing crosses from one
 * sequence into another, not even from rows that hold infinities or NaN.
 * Within one sequence a value that is not finite may reach rows of its own
 * 128-row tile that come before it (0 * inf in the masked half of a tile).
 * Scores of -inf weigh nothing; a row that has no others has lse = -inf and
 * no o (NaN).
 *
 * Tensors.  bf16 or fp16 (one type a call), D in {32, 64, 128}; a tensor is
 * its first element, the distance of two rows and of two heads in elements
 * (pa_tensor), so a slice of a fused q/k/v projection is taken as it is; the
 * D elements of a (row, head) are contiguous.  Addresses are 16-byte
 * aligned and strides positive multiples of 8 elements (a stride whose
 * extent is 1 is not looked at).  lse: float32 [Hq][lse_stride], natural
 * logarithm.  Score products, softmax and gradient sums are float32; P and
 * dS are rounded to the tensors' type before their second product, outputs
 * once at the end.  Every sum has a fixed order: the same call on the same
 * device gives the same bits.  fp16: P and dS = P (dP - delta) are scaled by
 * powers of two for their products (dS by the largest norms of the rows of dO
 * and v that it is made of) and the sums scaled back, so dO may be of any size
 * whose gradients fp16 holds.
 *
 * Every call is asynchronous on `stream` (a cudaStream_t, or NULL for the
 * legacy default stream), runs on the current device, and returns an
 * sa_status of sparse_attn.h; argument errors are returned before any
 * device work.  Calls from several host threads are safe; calls whose GPU
 * work overlaps must not share a workspace.
 */
#ifndef PACKED_ATTN_H
#define PACKED_ATTN_H

#include <stddef.h>
#include <stdint.h>

#include "sparse_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pa_layout pa_layout;

enum pa_dtype { PA_BF16 = 0, PA_FP16 = 1 };

typedef struct pa_tensor {
  void* data;
  int64_t row_stride;  /* elements from a row to the next */
  int64_t head_stride; /* elements from a head to the next */
} pa_tensor;

/*
 * packed_attn_layout - the tile tables of one packing.  lengths: host array
 * of n_seqs sequence lengths, each >= 0 (n_seqs 0 and empty sequences are
 * allowed).  Free with packed_attn_layout_free once no call or captured
 * graph uses it any more.
 * Errors: SA_ERR_INVALID_ARG (a null pointer, a negative length or count, or
 * more than 2^31 - 1024 rows in all).
 */
int packed_attn_layout(const int32_t* lengths, int n_seqs, pa_layout** out);
void packed_attn_layout_free(pa_layout* layout);
/* Rows of all sequences together (-1 for a null layout). */
int64_t packed_attn_layout_rows(const pa_layout* layout);
/* Copies the tables to the current device, which the first call on a device
 * does by itself: it allocates, and waits for the copy and for what is queued
 * on the legacy default stream (packed_attn_layout_free waits for the device).
 * A call that is captured into a CUDA graph needs it done before (it refuses
 * with SA_ERR_INVALID_ARG otherwise). */
int packed_attn_layout_upload(const pa_layout* layout, void* stream);

/*
 * packed_attn_fwd - o and lse of `rows` rows (>= packed_attn_layout_rows).
 * Errors: SA_ERR_INVALID_ARG (null pointer, head counts below 1 or Hq not a
 * multiple of Hkv, more than 65535 heads, rows below the layout's, unknown
 * type, misaligned address or stride, an output whose rows would overlap or
 * that begins where an input does, scale not finite and positive, lse_stride
 * below rows), SA_ERR_UNSUPPORTED (D), SA_ERR_CUDA.  Outputs must not overlap
 * inputs or one another in any other way either, which is not looked for.
 */
int packed_attn_fwd(const pa_tensor* q, const pa_tensor* k, const pa_tensor* v, const pa_tensor* o, float* lse,
                    int64_t lse_stride, int64_t rows, int Hq, int Hkv, int D, int dtype, float scale,
                    const pa_layout* layout, void* stream);

/* Bytes of device workspace packed_attn_bwd needs; 0 for a shape it refuses. */
size_t packed_attn_bwd_workspace_size(int Hq, int Hkv, int D, const pa_layout* layout);

/*
 * packed_attn_bwd - dq, dk, dv from q, k, v, the forward's o and lse, and dO.
 * workspace: packed_attn_bwd_workspace_size() bytes, 256-byte aligned,
 * contents on entry irrelevant, on exit unspecified.
 * Errors: those of packed_attn_fwd, SA_ERR_WORKSPACE.
 */
int packed_attn_bwd(const pa_tensor* q, const pa_tensor* k, const pa_tensor* v, const pa_tensor* o, const float* lse,
                    int64_t lse_stride, const pa_tensor* dO, const pa_tensor* dq, const pa_tensor* dk,
                    const pa_tensor* dv, int64_t rows, int Hq, int Hkv, int D, int dtype, float scale,
                    const pa_layout* layout, void* workspace, size_t ws_bytes, void* stream);

/* Waits for the stream and returns (and clears) the device status word of
 * this library: SA_OK, or SA_ERR_TIMEOUT if a bounded wait in a kernel ran
 * out. */
int packed_attn_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PACKED_ATTN_H */
