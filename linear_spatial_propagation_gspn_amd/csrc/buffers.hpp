// buffers.hpp -- what the host-side checks of the sequence and attention
// operators share: limits, storage types, a call's tensors and their overlap,
// a call's sequences (internal to libgspn).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gspn_sequence.h"

namespace gspn {
namespace api {

constexpr int64_t kMaxRows = int64_t{1} << 30;  // row numbers and a tile behind them stay within 32 bits
constexpr int64_t kMaxSeqs = int64_t{1} << 23;
constexpr int64_t kMaxSlotSeqs = int64_t{1} << 16;  // each looks through the slots before it
constexpr int64_t kMaxChannels = int64_t{1} << 19;
constexpr int64_t kMaxStride = int64_t{1} << 26;

inline bool valid_dtype(int64_t dt) { return dt == GSPN_F32 || dt == GSPN_BF16; }
inline int64_t elem_size(int64_t dt) { return dt == GSPN_F32 ? 4 : 2; }
inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }
inline gspn_status from_hip(hipError_t e) { return e == hipSuccess ? GSPN_OK : GSPN_ERR_HIP; }

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
inline gspn_status check_seq(const gspn_sequences& s, bool pool, bool step, bool* empty, Buffers* b) {
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

}  // namespace api
}  // namespace gspn
