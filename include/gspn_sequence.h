/*
 * gspn_sequence.h -- C ABI of libgspn's sequence operators: linear recurrences
 * over token rows next to gspn.h's recurrences over image lines.
 *
 *   causal_conv      the short depthwise causal convolution before a scan
 *   selective_scan   the selective state space scan: a diagonal linear
 *                    recurrence whose decay and input depend on the token
 *   block_join       a block's output normalised, gated, scaled and added to
 *                    the residual stream, and the norm before the next block
 *
 * Status codes, storage types, streams, ownership and errors are gspn.h's:
 * host-side validation first, then asynchronous launches on `stream`; no
 * allocation, no synchronisation, no global state; no C++ exception crosses.
 *
 * Conventions shared by every call here
 * -------------------------------------
 *  - Rows.  A tensor [rows][c] has unit column stride and a row stride `ld`
 *    in elements (c <= ld <= 2^26), so that the halves or slices of a projection's
 *    rows are taken as they are.  Alignment: the element size.  Row strides
 *    and offsets may pass 32 bits; rows <= 2^30, c <= 2^19.
 *  - Storage type: x, dt, z, B, C, h, gate and their gradients and outputs
 *    are GSPN_F32 or GSPN_BF16, one type per call.  Parameters (weights,
 *    biases, scales, A, D, dt_bias), their gradients and the scan's states
 *    are fp32 whatever the storage type.  Arithmetic is fp32; a result is
 *    rounded once, at its store.
 *  - Sequences.  `rows` rows hold nseq sequences, one after another.
 *    cu == NULL: equal lengths rows / nseq (nseq must divide rows).
 *    Otherwise cu is a device array of nseq + 1 offsets, not decreasing,
 *    0 <= cu[i] <= rows: sequence i is rows [cu[i], cu[i+1]); it may be
 *    empty.  Rows outside every sequence are not read, and not written but
 *    by the backward calls, which give them zero gradients (with nseq == 0:
 *    to every row, and to the parameters; no workspace or checkpoints then).
 *    Offsets that break these rules give unspecified results inside the
 *    caller's buffers (they are clamped to [0, rows]).
 *    At most 2^23 sequences (rows + nseq <= 2^30), 2^16 with slots.
 *  - Slots.  A call that carries state works on a pool of nslots entries.
 *    slots == NULL: sequence i uses entry i (nslots >= nseq).  Otherwise
 *    slots is a device array of nseq indices.  A negative index is a padding
 *    sequence: a step leaves its output row as it was; a prompt runs from
 *    zeros and keeps nothing.  An index >= nslots, and every repeat of an
 *    index that an earlier sequence of the call already names, is an error
 *    that only the device sees: that sequence's output rows are NaN and no
 *    entry of the pool is touched for it.
 *    resume (prompts; device bytes [nseq]): nonzero continues from the
 *    entry, zero starts from zeros; NULL: every sequence starts from zeros.
 *  - Empty calls (no rows and no sequence, a forward without a sequence, or
 *    no channel) return GSPN_OK and queue nothing; the scan's backward of rows
 *    without a channel gives them zero dB and dC.
 *  - Aliasing: an output, a state pool, a workspace may overlap nothing else
 *    (inputs may overlap inputs).  Row tensors of the same row stride in
 *    bytes may be column slices of one matrix; of different strides they are
 *    compared by the bytes from their first to their last element.
 *  - Sums over rows (gradients of parameters) are formed in fixed order:
 *    repeated calls give the same bits.
 */
#ifndef GSPN_SEQUENCE_H_
#define GSPN_SEQUENCE_H_

#include "gspn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GSPN_CONV_MIN_WIDTH 2
#define GSPN_CONV_MAX_WIDTH 4
#define GSPN_SCAN_MAX_STATE 16
#define GSPN_JOIN_MAX_CHANNELS 16384
/* Rows between two kept states of a scan (gspn_selective_scan_fwd). */
#define GSPN_SCAN_CHECKPOINT_ROWS 8

/* The sequences of one call (see "Sequences" and "Slots" above). */
typedef struct {
    int64_t rows, nseq;
    const int32_t* cu;
    const int32_t* slots;
    const uint8_t* resume;
    int64_t nslots;
} gspn_sequences;

/*
 * The short causal convolution, channel by channel, within each sequence:
 *   p_t[c] = bias[c] + sum_{j < width} weight[c][j] x_{t - width + 1 + j}[c]
 *   y_t    = silu ? p_t * sigmoid(p_t) : p_t
 * A row before the sequence's first is the pool entry's (resumed) or zero.
 *   weight [c][width] fp32, width 2 to 4 (else GSPN_ERR_UNSUPPORTED);
 *   bias   [c] fp32 or NULL;
 *   state  pool [nslots][width - 1][c] in the storage type, contiguous,
 *          oldest row first, or NULL: receives the last width - 1 rows of
 *          (entry or zeros, x); an empty sequence keeps its entry if it
 *          resumes and clears it otherwise.
 * gspn_causal_conv_step: one row per sequence (rows == nseq), each continuing
 *   its pool entry (state required, cu and resume must be NULL).
 * gspn_causal_conv_bwd: for dL/dy = gy, without a state: dx [rows][c],
 *   dweight [c][width], dbias [c] (NULL: not wanted), written; the pre-
 *   activation is recomputed.  workspace: gspn_causal_conv_bwd_workspace_bytes
 *   bytes, 4-byte aligned.
 */
typedef struct {
    gspn_sequences seq;
    int64_t c, width, silu;
    const void* x;
    int64_t ldx;
    const float* weight;
    const float* bias;
    void* y;
    int64_t ldy;
    void* state;
    /* backward */
    const void* gy;
    int64_t ldgy;
    void* dx;
    int64_t lddx;
    float* dweight;
    float* dbias;
    void* workspace;
    int64_t workspace_bytes;
} gspn_conv_args;

gspn_status gspn_causal_conv_fwd(const gspn_conv_args* args, int dtype, void* stream);
gspn_status gspn_causal_conv_step(const gspn_conv_args* args, int dtype, void* stream);
int64_t gspn_causal_conv_bwd_workspace_bytes(int64_t rows, int64_t nseq, int64_t c, int64_t width);
gspn_status gspn_causal_conv_bwd(const gspn_conv_args* args, int dtype, void* stream);

/*
 * The selective scan, per channel c and state n, within each sequence
 * (group g = c / (channels / groups)):
 *   d_t = softplus ? log(1 + exp(dt_t + dt_bias)) : dt_t + dt_bias
 *   h_t[n] = exp(d_t A[c][n]) h_{t-1}[n] + d_t x_t B_t[g][n]
 *   y_t = sum_n C_t[g][n] h_t[n] + D[c] x_t;   out_t = y_t silu(z_t)
 * from h = 0 or the resumed pool entry.  dt = -Inf
 * skips a row whose x and B are finite (softplus), whatever A <= 0: A log2 e
 * below the range of fp32, -Inf too, is taken as the range's lower end.
 *   x, dt, z, out  [rows][channels]; z NULL: no gate; D, dt_bias NULL: 0
 *   B, C           [rows][groups][n], row strides ldb, ldc (groups and n
 *                  contiguous); groups divides channels; groups times the
 *                  64-channel blocks of a group at most 65535 (else
 *                  GSPN_ERR_UNSUPPORTED)
 *   A              [channels][n], n 1 to 16 (else GSPN_ERR_UNSUPPORTED)
 *   state          pool [nslots][channels][n] fp32 or NULL: receives h after
 *                  the last row (an empty sequence as in the convolution)
 *   checkpoints    NULL, or gspn_selective_scan_checkpoint_bytes() bytes: the
 *                  fp32 states before every 8th row of each sequence, for
 *                  the backward
 *   workspace      gspn_selective_scan_workspace_bytes() bytes, 4-byte aligned
 * gspn_selective_scan_step: one row per sequence (rows == nseq; cu and resume
 *   NULL; no workspace), each continuing its pool entry.
 * gspn_selective_scan_bwd: for dL/dout = gy and sequences from h = 0 (state
 *   NULL), from the checkpoints of the forward on the same inputs (required):
 *   dx, ddt, dz (z given) [rows][channels], dB, dC [rows][groups][n]
 *   contiguous; dA [channels][n], dD (D given), ddt_bias (dt_bias given)
 *   [channels] fp32.  workspace: gspn_selective_scan_bwd_workspace_bytes().
 */
typedef struct {
    gspn_sequences seq;
    int64_t channels, groups, n, softplus;
    const void* x;
    int64_t ldx;
    const void* dt;
    int64_t lddt;
    const void* z;
    int64_t ldz;
    const void* B;
    int64_t ldb;
    const void* C;
    int64_t ldc;
    const float* A;
    const float* D;
    const float* dt_bias;
    void* out;
    int64_t ldo;
    float* state;
    float* checkpoints;
    void* workspace;
    int64_t workspace_bytes;
    /* backward */
    const void* gy;
    int64_t ldgy;
    void* dx;
    int64_t lddx;
    void* ddt;
    int64_t ldddt;
    void* dz;
    int64_t lddz;
    void* dB;
    void* dC;
    float* dA;
    float* dD;
    float* ddt_bias;
} gspn_selscan_args;

int64_t gspn_selective_scan_workspace_bytes(int64_t rows, int64_t nseq, int64_t channels, int64_t groups, int64_t n,
                                            int ragged);
int64_t gspn_selective_scan_checkpoint_bytes(int64_t rows, int64_t nseq, int64_t channels, int64_t n, int ragged);
int64_t gspn_selective_scan_bwd_workspace_bytes(int64_t rows, int64_t nseq, int64_t channels, int64_t groups,
                                                int64_t n, int ragged);
gspn_status gspn_selective_scan_fwd(const gspn_selscan_args* args, int dtype, void* stream);
gspn_status gspn_selective_scan_step(const gspn_selscan_args* args, int dtype, void* stream);
gspn_status gspn_selective_scan_bwd(const gspn_selscan_args* args, int dtype, void* stream);

/*
 * The join of a block's output h to the residual stream, row by row:
 *   q = post ? h / rms(h) * post : h        rms(v) = sqrt(mean(v^2) + eps)
 *   e = gate ? q * silu(gate) : q
 *   joined = residual + scale * e           (residual, scale: where given)
 *   normed = joined / rms(joined) * pre     (pre given; of joined as stored)
 * h, gate, normed [rows][c] in the storage type; post, scale, pre [c] fp32 or
 * NULL; residual and joined in residual_dtype (the storage type, or GSPN_F32
 * for a wide residual stream; without a residual, the storage type).  A norm's
 * sum of squares is fp32: rows past 1e19 lose theirs to Inf.
 * c <= 16384.  gspn_block_join_bwd: from joined (read where pre is given),
 * gjoined (NULL: zero) and gnormed (where pre is given) writes dh, dgate,
 * dresidual (where the input is given and the gradient wanted), dpost,
 * dscale, dpre (each wanted only where its parameter is given).  workspace:
 * gspn_block_join_bwd_workspace_bytes() bytes, 4-byte aligned.
 */
typedef struct {
    int64_t rows, c;
    int64_t residual_dtype;
    double eps;
    const void* h;
    int64_t ldh;
    const void* gate;
    int64_t ldgate;
    const void* residual;
    int64_t ldres;
    const float* post;
    const float* scale;
    const float* pre;
    void* joined;
    int64_t ldjoined;
    void* normed;
    int64_t ldnormed;
    /* backward */
    const void* gjoined;
    int64_t ldgjoined;
    const void* gnormed;
    int64_t ldgnormed;
    void* dh;
    int64_t lddh;
    void* dgate;
    int64_t lddgate;
    void* dresidual;
    int64_t lddres;
    float* dpost;
    float* dscale;
    float* dpre;
    void* workspace;
    int64_t workspace_bytes;
} gspn_join_args;

gspn_status gspn_block_join_fwd(const gspn_join_args* args, int dtype, void* stream);
int64_t gspn_block_join_bwd_workspace_bytes(int64_t rows, int64_t c);
gspn_status gspn_block_join_bwd(const gspn_join_args* args, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GSPN_SEQUENCE_H_ */
