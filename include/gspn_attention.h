/*
 * gspn_attention.h -- C ABI of libgspn's attention operators: what a layer
 * that looks at every earlier token needs next to gspn_sequence.h's layers
 * that carry a state.
 *
 *   head_rotary   each head's queries and keys normalised and rotated by their
 *                 positions, which may have several axes (time, height, width)
 *   attention     softmax attention with grouped heads: whole prompts, prompts
 *                 that continue a cache entry, single tokens, gradients
 *
 * Status codes, storage types, streams, ownership and errors are gspn.h's;
 * rows, sequences, slots, empty calls and aliasing are gspn_sequence.h's, but
 * for what stands here:
 *  - Row tensors are [rows][heads][d], heads and d contiguous, with a row
 *    stride `ld` in elements (heads * d <= ld <= 2^26); heads at most 4096.
 *  - Sequences number at most 2^23 (2^16 with slots); seq.resume is NULL:
 *    `held` says how many rows an entry holds.
 *  - Sums, softmax statistics and norms are fp32.  The kernels for GSPN_BF16
 *    round the softmax's numerators, and in the backward the scores'
 *    gradients, to bf16 as factors of matrix products that add up in fp32 (a
 *    step's numerators keep 16 bits); those for GSPN_F32 round nothing below
 *    fp32.
 */
#ifndef GSPN_ATTENTION_H_
#define GSPN_ATTENTION_H_

#include "gspn_sequence.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GSPN_ATTENTION_MAX_HEAD 128
#define GSPN_ROTARY_MAX_HEAD 256
#define GSPN_ROTARY_MAX_AXES 4

/*
 * Per row and head x of queries (and of keys):
 *   y = weight ? x / sqrt(mean(x^2) + eps) * weight : x
 *   (y_a, y_b) of pair j -> (y_a cos t - y_b sin t, y_a sin t + y_b cos t),
 *     t = positions[row][axis of j] * freqs[j]
 * pairs <= d / 2; pair j is elements (j, pairs + j), or (2 j, 2 j + 1) with
 * `interleaved`; elements behind the pairs are not rotated.  The first
 * section[0] pairs turn by axis 0, the next section[1] by axis 1, and so on
 * (axes 1 to 4; the sections add up to `pairs`).  Angles are formed in 64
 * bits and reduced to a turn before they are rounded.
 *   q, q_out     [rows][heads][d];  k, k_out [rows][kv_heads][d] (kv_heads 0: none)
 *   q_weight, k_weight [d] fp32 or NULL: no norm
 *   positions    int32 [rows][axes], row stride ldpos >= axes
 *   freqs        64-bit [pairs], radians a position
 * d <= 256 (else GSPN_ERR_UNSUPPORTED).  A norm's sum of squares is fp32: heads
 * past 1e19 lose theirs to Inf.
 * gspn_head_rotary_bwd: for gq, gk writes dq, dk and, where the weight is given
 *   and the gradient wanted, dq_weight, dk_weight [d] fp32.  q and k are read
 *   where they are normalised.  workspace:
 *   gspn_head_rotary_bwd_workspace_bytes(rows, d) bytes, 4-byte aligned, needed
 *   with dq_weight or dk_weight.
 */
typedef struct {
    int64_t rows, heads, kv_heads, d, pairs, axes, interleaved;
    int64_t section[GSPN_ROTARY_MAX_AXES];
    double eps;
    const void* q;
    int64_t ldq;
    const void* k;
    int64_t ldk;
    const float* q_weight;
    const float* k_weight;
    const int32_t* positions;
    int64_t ldpos;
    const double* freqs;
    void* q_out;
    int64_t ldqo;
    void* k_out;
    int64_t ldko;
    /* backward */
    const void* gq;
    int64_t ldgq;
    const void* gk;
    int64_t ldgk;
    void* dq;
    int64_t lddq;
    void* dk;
    int64_t lddk;
    float* dq_weight;
    float* dk_weight;
    void* workspace;
    int64_t workspace_bytes;
} gspn_rotary_args;

gspn_status gspn_head_rotary_fwd(const gspn_rotary_args* args, int dtype, void* stream);
int64_t gspn_head_rotary_bwd_workspace_bytes(int64_t rows, int64_t d);
gspn_status gspn_head_rotary_bwd(const gspn_rotary_args* args, int dtype, void* stream);

/*
 * Attention within each sequence; query head h reads key head
 * h / (heads / kv_heads):
 *   p_ij = exp(scale <q_i, k_j>) / sum over the keys j that row i sees
 *   out_i = sum_j p_ij v_j;   lse_i = log sum_j exp(scale <q_i, k_j>)
 * Of a sequence with n_q rows and n_k keys, row i sees every key, or with
 * `causal` those with j <= i + n_k - n_q: the last row sees all of them.  A row
 * that sees no key has out = 0 and lse = -Inf.  Keys that a row does not see
 * count for nothing, whatever they hold, if they lie in another sequence,
 * outside all of them or behind an entry's rows; of the row's own sequence,
 * a later key's v must be finite (a product with weight 0), in the backward
 * also its k, and q and gout of the rows that do not see a key.
 *   q, out  [rows][heads][d];  k, v [kv_rows][kv_heads][d]; d 1 to 128 (else
 *           GSPN_ERR_UNSUPPORTED); kv_heads divides heads
 *   lse     [heads][rows] fp32 or NULL (the backward needs it)
 *   scale   finite, also times log2 e in fp32: |scale| < 2.35e38
 * Keys' sequences: kv_cu is a device array of nseq + 1 offsets into the
 *   kv_rows rows; NULL: as the queries' (kv_rows == rows with seq.cu; without,
 *   equal lengths kv_rows / nseq).  A sequence may have no key.
 * Cache (k_pool and v_pool, both or neither): [nslots][capacity][kv_heads][d] in
 *   the storage type, contiguous.  held (device int32 [nseq]; NULL: none): the
 *   rows that each sequence's entry holds.  The call writes the sequence's new
 *   rows k, v behind them and attends to held + n_q keys; held itself is left
 *   as it is.  kv_cu must be NULL and kv_rows == rows.  Slots as in
 *   gspn_sequence.h: a padding sequence attends to its new rows alone and keeps
 *   nothing.  held < 0 or held + n_q > capacity is an error that only the
 *   device sees, like a bad slot: NaN rows, the pool untouched.
 * gspn_attention_step: one row per sequence (rows == nseq; seq.cu, kv_cu and
 *   lse NULL) over the cache, which it requires, with `held`.  Padding rows are
 *   left as they are.  workspace: gspn_attention_step_workspace_bytes() bytes,
 *   16-byte aligned.
 * gspn_attention_bwd: for dL/dout = gout, without a cache, from the forward's
 *   out and lse: dq [rows][heads][d], dk, dv [kv_rows][kv_heads][d].  workspace:
 *   gspn_attention_bwd_workspace_bytes() bytes, 16-byte aligned.  Rows outside
 *   every sequence have zero gradients.  No sum goes through atomics: repeated
 *   calls give the same bits.
 */
typedef struct {
    gspn_sequences seq;
    int64_t kv_rows;
    const int32_t* kv_cu;
    int64_t heads, kv_heads, d, causal;
    double scale;
    const void* q;
    int64_t ldq;
    const void* k;
    int64_t ldk;
    const void* v;
    int64_t ldv;
    void* out;
    int64_t ldo;
    float* lse;
    void* k_pool;
    void* v_pool;
    int64_t capacity;
    const int32_t* held;
    /* backward */
    const void* gout;
    int64_t ldgo;
    void* dq;
    int64_t lddq;
    void* dk;
    int64_t lddk;
    void* dv;
    int64_t lddv;
    void* workspace;
    int64_t workspace_bytes;
} gspn_attn_args;

gspn_status gspn_attention_fwd(const gspn_attn_args* args, int dtype, void* stream);
int64_t gspn_attention_step_workspace_bytes(int64_t nseq, int64_t heads, int64_t kv_heads, int64_t d, int64_t capacity);
gspn_status gspn_attention_step(const gspn_attn_args* args, int dtype, void* stream);
int64_t gspn_attention_bwd_workspace_bytes(int64_t rows, int64_t nseq, int64_t heads, int64_t kv_rows,
                                           int64_t kv_heads, int64_t d);
gspn_status gspn_attention_bwd(const gspn_attn_args* args, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GSPN_ATTENTION_H_ */
