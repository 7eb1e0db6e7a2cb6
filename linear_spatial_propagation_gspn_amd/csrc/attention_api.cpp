// attention_api.cpp -- the C ABI of the attention operators (declared in
// include/gspn_attention.h): host-side validation of every argument, then
// kernel launches on the caller's stream.
#include "../../include/gspn_attention.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "attention.hpp"
#include "buffers.hpp"

namespace {

using namespace gspn::api;

constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxGrid = (int64_t{1} << 24) - 1;  // of workgroups of 256: 2^32 lanes

enum Which { kFwd, kStep, kBwd };

gspn_status check_rotary(const gspn_rotary_args* a, int dtype, bool bwd, bool* empty) {
    if (!a) return GSPN_ERR_NULL_POINTER;
    if (!valid_dtype(dtype)) return GSPN_ERR_BAD_DTYPE;
    if (a->rows < 0 || a->rows > kMaxRows || a->heads < 1 || a->kv_heads < 0 || a->d < 1) return GSPN_ERR_BAD_SHAPE;
    if (!(a->eps >= 0.0) || !std::isfinite(a->eps)) return GSPN_ERR_BAD_SHAPE;
    if (a->d > GSPN_ROTARY_MAX_HEAD || a->axes > GSPN_ROTARY_MAX_AXES || a->heads > kMaxHeads ||
        a->kv_heads > kMaxHeads)
        return GSPN_ERR_UNSUPPORTED;
    if (a->axes < 1 || a->pairs < 0 || a->pairs > a->d / 2) return GSPN_ERR_BAD_SHAPE;
    int64_t sum = 0;
    for (int i = 0; i < a->axes; ++i) {
        if (a->section[i] < 0 || a->section[i] > a->pairs) return GSPN_ERR_BAD_SHAPE;
        sum += a->section[i];
    }
    if (sum != a->pairs) return GSPN_ERR_BAD_SHAPE;
    *empty = a->rows == 0 && !(bwd && (a->dq_weight || a->dk_weight));
    if (*empty) return GSPN_OK;
    const int64_t es = elem_size(dtype), n = a->rows, cq = a->heads * a->d, ck = a->kv_heads * a->d;
    const bool keys = a->kv_heads > 0;
    Buffers b;
    b.flat(a->q_weight, a->d * 4, 4, false, true);
    b.flat(a->k_weight, a->d * 4, 4, false, true);
    b.rows(a->positions, n, a->ldpos, a->axes, 4, false);
    b.flat(a->freqs, a->pairs * 8, 8, false);
    if (!bwd || a->q_weight) b.rows(a->q, n, a->ldq, cq, es, false);
    if (keys && (!bwd || a->k_weight)) b.rows(a->k, n, a->ldk, ck, es, false);
    if (!bwd) {
        b.rows(a->q_out, n, a->ldqo, cq, es, true);
        if (keys) b.rows(a->k_out, n, a->ldko, ck, es, true);
        return b.done();
    }
    b.rows(a->gq, n, a->ldgq, cq, es, false);
    b.rows(a->dq, n, a->lddq, cq, es, true);
    if (keys) {
        b.rows(a->gk, n, a->ldgk, ck, es, false);
        b.rows(a->dk, n, a->lddk, ck, es, true);
    }
    if ((a->dq_weight && !a->q_weight) || (a->dk_weight && !(a->k_weight && keys))) return GSPN_ERR_NULL_POINTER;
    b.flat(a->dq_weight, a->d * 4, 4, true, true);
    b.flat(a->dk_weight, a->d * 4, 4, true, true);
    if (a->dq_weight || a->dk_weight) {
        const int64_t need = gspn_head_rotary_bwd_workspace_bytes(n, a->d);
        if (a->workspace_bytes < need) return GSPN_ERR_WORKSPACE;
        b.flat(a->workspace, need, 4, true);
    }
    return b.done();
}

bool attn_sizes_ok(int64_t rows, int64_t nseq, int64_t heads, int64_t kv_heads, int64_t d) {
    return rows >= 0 && nseq >= 0 && rows <= kMaxRows && nseq <= kMaxRows - rows && kv_heads >= 1 && heads >= 1 &&
           heads <= kMaxHeads && heads % kv_heads == 0 && d >= 1 && d <= GSPN_ATTENTION_MAX_HEAD;
}

gspn_status check_attn(const gspn_attn_args* a, int dtype, Which which, bool* empty) {
    if (!a) return GSPN_ERR_NULL_POINTER;
    if (!valid_dtype(dtype)) return GSPN_ERR_BAD_DTYPE;
    if (a->heads < 1 || a->kv_heads < 1 || a->heads % a->kv_heads != 0 || a->d < 1) return GSPN_ERR_BAD_SHAPE;
    if (!std::isfinite(gspn::scale_log2(a->scale))) return GSPN_ERR_BAD_SHAPE;
    if (a->d > GSPN_ATTENTION_MAX_HEAD || a->heads > kMaxHeads) return GSPN_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype), rows = a->seq.rows, nseq = a->seq.nseq, kv = a->kv_rows;
    const bool pool = a->k_pool || a->v_pool || which == kStep;
    if (which == kBwd && pool) return GSPN_ERR_UNSUPPORTED;
    Buffers b;
    gspn_status s = check_seq(a->seq, pool, which == kStep, empty, &b);
    if (s != GSPN_OK) return s;
    if (a->seq.resume) return GSPN_ERR_BAD_SHAPE;
    if (kv < 0 || kv > kMaxRows || kv + nseq > kMaxRows) return GSPN_ERR_BAD_SHAPE;
    const bool none = *empty;  // a backward has rows to clear, also where there is no sequence
    *empty = which == kBwd ? rows == 0 && kv == 0 : none || rows == 0;
    if (*empty) return GSPN_OK;
    if (!none) {
        if (a->kv_cu ? pool : (a->seq.cu || pool) ? kv != rows : kv % nseq != 0) return GSPN_ERR_BAD_SHAPE;
        b.flat(a->kv_cu, (nseq + 1) * 4, 4, false, true);
        const int64_t ids = gspn::chunk_ids(true, rows, nseq, gspn::kAttnShift) * a->heads;
        const int64_t kv_ids = gspn::chunk_ids(true, kv, nseq, gspn::kKeyShift) * a->kv_heads;
        const int64_t copies = pool ? gspn::chunk_ids(true, rows, nseq, gspn::kAppendShift) : 0;
        if (ids + copies > kMaxGrid || kv_ids > kMaxGrid) return GSPN_ERR_UNSUPPORTED;
    }
    const int64_t cq = a->heads * a->d, ck = a->kv_heads * a->d;
    b.rows(a->q, rows, a->ldq, cq, es, false);
    b.rows(a->k, kv, a->ldk, ck, es, false);
    b.rows(a->v, kv, a->ldv, ck, es, false);
    b.rows(a->out, rows, a->ldo, cq, es, which != kBwd);
    b.flat(a->lse, a->heads * rows * 4, 4, which != kBwd, which != kBwd);
    if (which == kStep && a->lse) return GSPN_ERR_BAD_SHAPE;
    if (which == kBwd) {
        b.rows(a->gout, rows, a->ldgo, cq, es, false);
        b.rows(a->dq, rows, a->lddq, cq, es, true);
        b.rows(a->dk, kv, a->lddk, ck, es, true);
        b.rows(a->dv, kv, a->lddv, ck, es, true);
        const int64_t need =
            none ? 0 : gspn_attention_bwd_workspace_bytes(rows, nseq, a->heads, kv, a->kv_heads, a->d);
        if (a->workspace_bytes < need) return GSPN_ERR_WORKSPACE;
        b.flat(a->workspace, need, 16, true);
    }
    if (pool) {
        if (!a->k_pool || !a->v_pool || (which == kStep && !a->held)) return GSPN_ERR_NULL_POINTER;
        if (a->capacity < 1 || a->capacity > kMaxRows) return GSPN_ERR_BAD_SHAPE;
        if (a->seq.nslots > (int64_t{1} << 46) / (a->capacity * ck)) return GSPN_ERR_UNSUPPORTED;
        const int64_t bytes = a->seq.nslots * a->capacity * ck * es;
        b.flat(a->k_pool, bytes, es, true);
        b.flat(a->v_pool, bytes, es, true);
        b.flat(a->held, nseq * 4, 4, false, true);
    } else if (a->held) {
        return GSPN_ERR_BAD_SHAPE;
    }
    if (which == kStep) {
        const int64_t need = gspn_attention_step_workspace_bytes(nseq, a->heads, a->kv_heads, a->d, a->capacity);
        if (a->workspace_bytes < need) return GSPN_ERR_WORKSPACE;
        b.flat(a->workspace, need, 16, true);
    }
    return b.done();
}

}  // namespace

extern "C" {

gspn_status gspn_head_rotary_fwd(const gspn_rotary_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_rotary(args, dtype, false, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_rotary_fwd(*args, dtype, as_stream(stream)));
}

int64_t gspn_head_rotary_bwd_workspace_bytes(int64_t rows, int64_t d) {
    if (rows < 0 || rows > kMaxRows || d < 1 || d > GSPN_ROTARY_MAX_HEAD) return -1;
    return gspn::rotary_bwd_parts(rows) * 2 * d * 4;
}

gspn_status gspn_head_rotary_bwd(const gspn_rotary_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_rotary(args, dtype, true, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_rotary_bwd(*args, dtype, as_stream(stream)));
}

gspn_status gspn_attention_fwd(const gspn_attn_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_attn(args, dtype, kFwd, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_attn_fwd(*args, dtype, as_stream(stream)));
}

int64_t gspn_attention_step_workspace_bytes(int64_t nseq, int64_t heads, int64_t kv_heads, int64_t d,
                                            int64_t capacity) {
    if (!attn_sizes_ok(0, nseq, heads, kv_heads, d) || capacity < 1 || capacity > kMaxRows) return -1;
    const int64_t n = gspn::attn_splits(nseq, heads, kv_heads, capacity);
    return n == 1 ? 0 : nseq * heads * n * (d + 2) * 4;
}

gspn_status gspn_attention_step(const gspn_attn_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_attn(args, dtype, kStep, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_attn_step(*args, dtype, as_stream(stream)));
}

int64_t gspn_attention_bwd_workspace_bytes(int64_t rows, int64_t nseq, int64_t heads, int64_t kv_rows,
                                           int64_t kv_heads, int64_t d) {
    if (nseq < 1 || !attn_sizes_ok(rows, nseq, heads, kv_heads, d) || !attn_sizes_ok(kv_rows, nseq, heads, kv_heads, d)) return -1;
    const int64_t parts = gspn::attn_bwd_parts(rows, nseq, heads, kv_rows, kv_heads);
    return (rows * heads + 3) / 4 * 16 + (parts > 1 ? parts * 2 * kv_rows * kv_heads * d * 4 : 0);
}

gspn_status gspn_attention_bwd(const gspn_attn_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_attn(args, dtype, kBwd, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_attn_bwd(*args, dtype, as_stream(stream)));
}

}  // extern "C"
