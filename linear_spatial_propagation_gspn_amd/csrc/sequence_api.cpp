// sequence_api.cpp -- the C ABI of the sequence operators (declared in
// include/gspn_sequence.h): host-side validation of every argument, then
// kernel launches on the caller's stream.
#include "../../include/gspn_sequence.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "launch.hpp"
#include "sequence.hpp"

namespace {

constexpr int64_t kMaxRows = int64_t{1} << 30;  // row numbers and a tile behind them stay within 32 bits
constexpr int64_t kMaxSeqs = int64_t{1} << 23;
constexpr int64_t kMaxSlotSeqs = int64_t{1} << 16;  // each looks through the slots before it
constexpr int64_t kMaxChannels = int64_t{1} << 19;
constexpr int64_t kMaxStride = int64_t{1} << 26;

bool valid_dtype(int64_t dt) { return dt == GSPN_F32 || dt == GSPN_BF16; }
int64_t elem_size(int64_t dt) { return dt == GSPN_F32 ? 4 : 2; }
hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }
gspn_status from_hip(hipError_t e) { return e == hipSuccess ? GSPN_OK : GSPN_ERR_HIP; }

// The tensors of one call: each must be given (or may be absent), aligned,
// and an output may overlap nothing else.
class Buffers {
  public:
    // [rows][c] elements of es bytes, rows ld apart.
    void rows(const void* p, int64_t n, int64_t ld, int64_t c, int64_t es, bool out, bool optional = false) {
        if (ld < c) fail(GSPN_ERR_BAD_SHAPE);
        if (ld > kMaxStride) fail(GSPN_ERR_UNSUPPORTED);
        add(p, n < 1 || c < 1 ? 0 : ((n - 1) * ld + c) * es, es, out, optional, ld * es, c * es);
    }
    void flat(const void* p, int64_t bytes, int64_t align, bool out, bool optional = false) {
        add(p, bytes, align, out, optional);
    }
    gspn_status done() const {
        if (st_ != GSPN_OK) return st_;
        for (int i = 0; i < count_; ++i) {
            if (!b_[i].out) continue;
            for (int j = 0; j < count_; ++j) {
                if (i == j || (b_[j].out && j < i)) continue;
                if (overlap(b_[i], b_[j])) return GSPN_ERR_ALIASING;
            }
        }
        return GSPN_OK;
    }

  private:
    struct One {
        const void* p;
        int64_t bytes;
        int64_t pitch, width;  // bytes from row to row and of a row; 0: one run
        bool out;
    };
    static constexpr int kMax = 32;
    One b_[kMax] = {};
    int count_ = 0;
    gspn_status st_ = GSPN_OK;

    // Whether two tensors share a byte.  Row tensors of one pitch may lie in
    // one another's gaps, as column slices of one matrix do.
    static bool overlap(const One& a, const One& b) {
        const int64_t a0 = reinterpret_cast<int64_t>(a.p), b0 = reinterpret_cast<int64_t>(b.p);
        if (a0 >= b0 + b.bytes || b0 >= a0 + a.bytes) return false;
        if (a.pitch == 0 || a.pitch != b.pitch) return true;
        const int64_t d = ((b0 - a0) % a.pitch + a.pitch) % a.pitch;  // b's columns after a's
        return d < a.width || d + b.width > a.pitch;
    }

    void fail(gspn_status s) {
        if (st_ == GSPN_OK) st_ = s;
    }
    void add(const void* p, int64_t bytes, int64_t align, bool out, bool optional, int64_t pitch = 0,
             int64_t width = 0) {
        if (bytes == 0) return;  // nothing of it is touched
        if (!p) {
            if (!optional) fail(GSPN_ERR_NULL_POINTER);
            return;
        }
        if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(align) != 0) fail(GSPN_ERR_MISALIGNED);
        if (count_ < kMax) b_[count_++] = {p, bytes, pitch, width, out};
    }
};

// Sequences of a call.  step: one row each.  empty: no sequence.
gspn_status check_seq(const gspn_sequences& s, bool pool, bool step, bool* empty, Buffers* b) {
    if (s.rows < 0 || s.rows > kMaxRows || s.nseq < 0 || s.nseq > kMaxRows || s.nslots < 0 || s.nslots > kMaxRows)
        return GSPN_ERR_BAD_SHAPE;
    if (s.nseq > kMaxSeqs || (s.slots && s.nseq > kMaxSlotSeqs)) return GSPN_ERR_UNSUPPORTED;
    if (s.rows + s.nseq > kMaxRows) return GSPN_ERR_BAD_SHAPE;  // chunk ids
    *empty = s.nseq == 0;
    if (s.nseq == 0) return s.rows == 0 || s.cu ? GSPN_OK : GSPN_ERR_BAD_SHAPE;
    if (step && (s.rows != s.nseq || s.cu || s.resume)) return GSPN_ERR_BAD_SHAPE;
    if (!s.cu && s.rows % s.nseq != 0) return GSPN_ERR_BAD_SHAPE;
    if (!pool && (s.slots || s.resume)) return GSPN_ERR_BAD_SHAPE;
    if (pool && !s.slots && s.nslots < s.nseq) return GSPN_ERR_BAD_SHAPE;
    if (pool && s.nslots < 1) return GSPN_ERR_BAD_SHAPE;
    b->flat(s.cu, (s.nseq + 1) * 4, 4, false, true);
    b->flat(s.slots, s.nseq * 4, 4, false, true);
    b->flat(s.resume, s.nseq, 1, false, true);
    return GSPN_OK;
}

gspn_status check_conv(const gspn_conv_args* a, int dtype, int which, bool* empty) {
    if (!a) return GSPN_ERR_NULL_POINTER;
    if (!valid_dtype(dtype)) return GSPN_ERR_BAD_DTYPE;
    if (a->c < 0 || a->c > kMaxChannels) return GSPN_ERR_BAD_SHAPE;
    if (a->width < GSPN_CONV_MIN_WIDTH || a->width > GSPN_CONV_MAX_WIDTH) return GSPN_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype), rows = a->seq.rows;
    const bool pool = a->state != nullptr;
    if (which == 2 && pool) return GSPN_ERR_UNSUPPORTED;
    Buffers b;
    const gspn_status s = check_seq(a->seq, pool || which == 1, which == 1, empty, &b);
    if (s != GSPN_OK) return s;
    // a backward has rows outside the sequences to clear, also where there is no sequence
    const bool none = *empty;
    *empty = (none && (which != 2 || rows == 0)) || a->c == 0;
    if (*empty) return GSPN_OK;
    if (which == 1 && !a->state) return GSPN_ERR_NULL_POINTER;
    b.rows(a->x, rows, a->ldx, a->c, es, false);
    b.flat(a->weight, a->c * a->width * 4, 4, false);
    b.flat(a->bias, a->c * 4, 4, false, true);
    if (which == 2) {
        b.rows(a->gy, rows, a->ldgy, a->c, es, false);
        b.rows(a->dx, rows, a->lddx, a->c, es, true);
        b.flat(a->dweight, a->c * a->width * 4, 4, true);
        b.flat(a->dbias, a->c * 4, 4, true, true);
        const int64_t need = none ? 0 : gspn_causal_conv_bwd_workspace_bytes(rows, a->seq.nseq, a->c, a->width);
        if (a->workspace_bytes < need) return GSPN_ERR_WORKSPACE;
        b.flat(a->workspace, need, 4, true);
    } else {
        b.rows(a->y, rows, a->ldy, a->c, es, true);
        b.flat(a->state, a->seq.nslots * (a->width - 1) * a->c * es, es, true, true);
    }
    return b.done();
}

bool scan_sizes_ok(int64_t rows, int64_t nseq, int64_t channels, int64_t groups, int64_t n) {
    return rows >= 0 && nseq >= 0 && rows + nseq <= kMaxRows && rows <= kMaxRows && channels >= 0 &&
           channels <= kMaxChannels && groups >= 1 && channels % groups == 0 && n >= 1 && n <= GSPN_SCAN_MAX_STATE;
}

gspn_status check_scan(const gspn_selscan_args* a, int dtype, int which, bool* empty) {
    if (!a) return GSPN_ERR_NULL_POINTER;
    if (!valid_dtype(dtype)) return GSPN_ERR_BAD_DTYPE;
    if (a->channels < 0 || a->channels > kMaxChannels || a->groups < 1 || a->channels % a->groups != 0 || a->n < 1)
        return GSPN_ERR_BAD_SHAPE;
    if (a->n > GSPN_SCAN_MAX_STATE) return GSPN_ERR_UNSUPPORTED;
    // one grid row per channel block of a group
    if (a->groups * ((a->channels / a->groups + 63) / 64) > 65535) return GSPN_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype), rows = a->seq.rows, nseq = a->seq.nseq;
    const bool pool = a->state != nullptr;
    if (which == 2 && pool) return GSPN_ERR_UNSUPPORTED;
    Buffers b;
    const gspn_status s = check_seq(a->seq, pool || which == 1, which == 1, empty, &b);
    if (s != GSPN_OK) return s;
    // as in the convolution; without a channel dB and dC are sums over none
    const bool none = *empty || a->channels == 0;
    *empty = none && (which != 2 || rows == 0);
    if (*empty) return GSPN_OK;
    if (which == 1 && !a->state) return GSPN_ERR_NULL_POINTER;
    const int64_t c = a->channels, gn = a->groups * a->n;
    const int ragged = a->seq.cu != nullptr;
    b.rows(a->x, rows, a->ldx, c, es, false);
    b.rows(a->dt, rows, a->lddt, c, es, false);
    if (a->z) b.rows(a->z, rows, a->ldz, c, es, false);
    b.rows(a->B, rows, a->ldb, gn, es, false);
    b.rows(a->C, rows, a->ldc, gn, es, false);
    b.flat(a->A, c * a->n * 4, 4, false);
    b.flat(a->D, c * 4, 4, false, true);
    b.flat(a->dt_bias, c * 4, 4, false, true);
    const int64_t kept = none ? 0 : gspn_selective_scan_checkpoint_bytes(rows, nseq, c, a->n, ragged);
    if (which == 2) {
        b.rows(a->gy, rows, a->ldgy, c, es, false);
        b.flat(a->checkpoints, kept, 4, false);
        b.rows(a->dx, rows, a->lddx, c, es, true);
        b.rows(a->ddt, rows, a->ldddt, c, es, true);
        if (a->z) b.rows(a->dz, rows, a->lddz, c, es, true);
        b.flat(a->dB, rows * gn * es, es, true);
        b.flat(a->dC, rows * gn * es, es, true);
        b.flat(a->dA, c * a->n * 4, 4, true);
        b.flat(a->dD, c * 4, 4, true, true);
        b.flat(a->ddt_bias, c * 4, 4, true, true);
        const int64_t need =
            none ? 0 : gspn_selective_scan_bwd_workspace_bytes(rows, nseq, c, a->groups, a->n, ragged);
        if (a->workspace_bytes < need) return GSPN_ERR_WORKSPACE;
        b.flat(a->workspace, need, 4, true);
    } else {
        b.rows(a->out, rows, a->ldo, c, es, true);
        b.flat(a->state, a->seq.nslots * c * a->n * 4, 4, true, true);
        if (which == 0) {
            b.flat(a->checkpoints, kept, 4, true, true);
            const int64_t need = gspn_selective_scan_workspace_bytes(rows, nseq, c, a->groups, a->n, ragged);
            if (a->workspace_bytes < need) return GSPN_ERR_WORKSPACE;
            b.flat(a->workspace, need, 4, true);
        }
    }
    return b.done();
}

gspn_status check_join(const gspn_join_args* a, int dtype, bool bwd, bool* empty) {
    if (!a) return GSPN_ERR_NULL_POINTER;
    if (!valid_dtype(dtype) || !valid_dtype(a->residual_dtype)) return GSPN_ERR_BAD_DTYPE;
    if (a->residual_dtype != dtype && a->residual_dtype != GSPN_F32) return GSPN_ERR_BAD_DTYPE;
    if (a->rows < 0 || a->rows > kMaxRows || a->c < 0) return GSPN_ERR_BAD_SHAPE;
    if (!(a->eps >= 0.0) || !std::isfinite(a->eps)) return GSPN_ERR_BAD_SHAPE;
    if (a->c > GSPN_JOIN_MAX_CHANNELS) return GSPN_ERR_UNSUPPORTED;
    *empty = a->c == 0 || (a->rows == 0 && !bwd);
    if (*empty) return GSPN_OK;
    const int64_t es = elem_size(dtype), rs = elem_size(a->residual_dtype), n = a->rows, c = a->c;
    Buffers b;
    b.rows(a->h, n, a->ldh, c, es, false);
    if (a->gate) b.rows(a->gate, n, a->ldgate, c, es, false);
    b.flat(a->post, c * 4, 4, false, true);
    b.flat(a->scale, c * 4, 4, false, true);
    b.flat(a->pre, c * 4, 4, false, true);
    if (!bwd) {
        if (a->residual) b.rows(a->residual, n, a->ldres, c, rs, false);
        b.rows(a->joined, n, a->ldjoined, c, rs, true);
        if (a->pre) b.rows(a->normed, n, a->ldnormed, c, es, true);
        return b.done();
    }
    if (a->gjoined) b.rows(a->gjoined, n, a->ldgjoined, c, rs, false);
    if (a->pre) {
        b.rows(a->joined, n, a->ldjoined, c, rs, false);
        b.rows(a->gnormed, n, a->ldgnormed, c, es, false);
    }
    if ((a->dgate && !a->gate) || (a->dpost && !a->post) || (a->dscale && !a->scale) || (a->dpre && !a->pre))
        return GSPN_ERR_NULL_POINTER;
    if (a->dh) b.rows(a->dh, n, a->lddh, c, es, true);
    if (a->dgate) b.rows(a->dgate, n, a->lddgate, c, es, true);
    if (a->dresidual) b.rows(a->dresidual, n, a->lddres, c, rs, true);
    b.flat(a->dpost, c * 4, 4, true, true);
    b.flat(a->dscale, c * 4, 4, true, true);
    b.flat(a->dpre, c * 4, 4, true, true);
    if (a->dpost || a->dscale || a->dpre) {
        const int64_t need = gspn_block_join_bwd_workspace_bytes(n, c);
        if (a->workspace_bytes < need) return GSPN_ERR_WORKSPACE;
        b.flat(a->workspace, need, 4, true);
    }
    return b.done();
}

}  // namespace

extern "C" {

gspn_status gspn_causal_conv_fwd(const gspn_conv_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_conv(args, dtype, 0, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_conv_fwd(*args, dtype, as_stream(stream)));
}

gspn_status gspn_causal_conv_step(const gspn_conv_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_conv(args, dtype, 1, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_conv_step(*args, dtype, as_stream(stream)));
}

int64_t gspn_causal_conv_bwd_workspace_bytes(int64_t rows, int64_t nseq, int64_t c, int64_t width) {
    if (rows < 0 || nseq < 1 || rows + nseq > kMaxRows || c < 1 || c > kMaxChannels || width < GSPN_CONV_MIN_WIDTH ||
        width > GSPN_CONV_MAX_WIDTH)
        return -1;
    return gspn::conv_bwd_parts(rows, nseq, c) * (width + 1) * c * 4;
}

gspn_status gspn_causal_conv_bwd(const gspn_conv_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_conv(args, dtype, 2, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_conv_bwd(*args, dtype, as_stream(stream)));
}

int64_t gspn_selective_scan_workspace_bytes(int64_t rows, int64_t nseq, int64_t channels, int64_t groups, int64_t n,
                                            int ragged) {
    if (!scan_sizes_ok(rows, nseq, channels, groups, n) || nseq < 1) return -1;
    if (channels == 0) return 0;
    const int shift = gspn::selscan_shift(rows, nseq, channels, groups, n, ragged != 0);
    if (shift == gspn::kWholeQuad || (int64_t{1} << shift) >= (ragged ? rows : rows / nseq)) return 0;
    return gspn::chunk_ids(ragged != 0, rows, nseq, shift) * (n + 1) * channels * 4;
}

int64_t gspn_selective_scan_checkpoint_bytes(int64_t rows, int64_t nseq, int64_t channels, int64_t n, int ragged) {
    if (!scan_sizes_ok(rows, nseq, channels, 1, n) || nseq < 1) return -1;
    return gspn::chunk_ids(ragged != 0, rows, nseq, gspn::kCheckShift) * n * channels * 4;
}

gspn_status gspn_selective_scan_fwd(const gspn_selscan_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_scan(args, dtype, 0, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_selscan_fwd(*args, dtype, as_stream(stream)));
}

gspn_status gspn_selective_scan_step(const gspn_selscan_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_scan(args, dtype, 1, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_selscan_step(*args, dtype, as_stream(stream)));
}

int64_t gspn_selective_scan_bwd_workspace_bytes(int64_t rows, int64_t nseq, int64_t channels, int64_t groups,
                                                int64_t n, int ragged) {
    if (!scan_sizes_ok(rows, nseq, channels, groups, n) || nseq < 1) return -1;
    if (channels == 0) return 0;
    const int shift = gspn::selscan_bwd_shift(rows, nseq, channels, groups, n, ragged != 0);
    const int64_t ids = gspn::chunk_ids(ragged != 0, rows, nseq, shift);
    const int64_t floats = gspn::selscan_bwd_blocks(channels, groups, n) * rows * 2 * groups * n +
                           ids * (n + 2) * channels + ids * (n + 1) * channels;
    return floats * 4;
}

gspn_status gspn_selective_scan_bwd(const gspn_selscan_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_scan(args, dtype, 2, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_selscan_bwd(*args, dtype, as_stream(stream)));
}

gspn_status gspn_block_join_fwd(const gspn_join_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_join(args, dtype, false, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_join_fwd(*args, dtype, as_stream(stream)));
}

int64_t gspn_block_join_bwd_workspace_bytes(int64_t rows, int64_t c) {
    if (rows < 0 || rows > kMaxRows || c < 0 || c > GSPN_JOIN_MAX_CHANNELS) return -1;
    return gspn::join_bwd_parts(rows, c) * 3 * c * 4;
}

gspn_status gspn_block_join_bwd(const gspn_join_args* args, int dtype, void* stream) {
    bool empty = false;
    const gspn_status s = check_join(args, dtype, true, &empty);
    if (s != GSPN_OK || empty) return s;
    return from_hip(gspn::launch_join_bwd(*args, dtype, as_stream(stream)));
}

}  // extern "C"
