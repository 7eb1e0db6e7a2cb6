// sequence.hpp -- what the sequence operators' kernels share: how a launch
// finds its sequence and chunk, how a sequence finds its pool entry, vector
// loads and stores, the reduction of partial sums (internal to libgspn).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gspn_sequence.h"
#include "check.hpp"
#include "device.hpp"
#include "launch.hpp"

namespace gspn {

// The sequences of a launch.  len: the equal length (cu null).
struct SeqK {
    const int32_t* cu;
    const int32_t* slots;
    const uint8_t* resume;
    int32_t rows, nseq, len, nslots;
};

// Chunks of 1 << shift rows, counted within each sequence.  The ids of
// sequence i's chunks start at chunk_base(i): for equal lengths the count a
// sequence has times i; for packed offsets cu[i] / rows-per-chunk + i, which
// leaves every sequence room for its chunks (and one id for an empty one)
// without a pass over the lengths.
GSPN_HD int64_t chunks_each(int64_t len, int shift) {
    const int64_t k = (len + (int64_t{1} << shift) - 1) >> shift;
    return k < 1 ? 1 : k;
}

GSPN_HD int64_t chunk_ids(bool ragged, int64_t rows, int64_t nseq, int shift) {
    return ragged ? (rows >> shift) + nseq : nseq * chunks_each(rows / nseq, shift);
}

__device__ __forceinline__ int clamp_row(const SeqK& s, int v) { return v < 0 ? 0 : v > s.rows ? s.rows : v; }

// A sequence's rows (i the same for the whole wave, so the rows are put into
// scalar registers).
__device__ __forceinline__ int seq_begin(const SeqK& s, int i) {
    return s.cu ? __builtin_amdgcn_readfirstlane(clamp_row(s, s.cu[i])) : i * s.len;
}

__device__ __forceinline__ int seq_end(const SeqK& s, int i, int begin) {
    if (!s.cu) return begin + s.len;
    const int e = __builtin_amdgcn_readfirstlane(clamp_row(s, s.cu[i + 1]));
    return e < begin ? begin : e;
}

__device__ __forceinline__ int64_t chunk_base(const SeqK& s, int i, int begin, int shift) {
    return s.cu ? static_cast<int64_t>(begin >> shift) + i : i * chunks_each(s.len, shift);
}

// Chunk id -> its sequence and place.  Uniform over a wave; every lane of the
// wave must call it.
struct Chunk {
    int seq;       // sequence, -1: no such chunk
    int k;         // chunk number within the sequence
    int count;     // chunks the sequence has (1 for an empty one)
    int begin, end;  // the sequence's rows
    int r0, r1;    // the chunk's rows
};

__device__ __forceinline__ Chunk find_chunk(const SeqK& s, int64_t id, int shift) {
    Chunk c;
    int i;
    if (!s.cu) {
        const int64_t each = chunks_each(s.len, shift);
        i = static_cast<int>(id / each);
    } else {
        // largest i whose first id is <= id: 64 probes a step, one a lane
        const int lane = __lane_id();
        int lo = 0, span = s.nseq;
        while (span > 1) {
            const int step = (span + 63) / 64;
            const int at = lo + lane * step;
            const bool in = lane * step < span &&
                            static_cast<int64_t>(clamp_row(s, s.cu[at]) >> shift) + at <= id;
            const int hit = __popcll(__ballot(in));
            const int b = hit > 0 ? hit - 1 : 0;
            lo += b * step;
            span = span - b * step < step ? span - b * step : step;
        }
        i = __builtin_amdgcn_readfirstlane(lo);
    }
    c.seq = -1;
    c.begin = c.end = c.r0 = c.r1 = c.k = c.count = 0;
    if (i >= s.nseq) return c;
    c.begin = seq_begin(s, i);
    c.end = seq_end(s, i, c.begin);
    const int64_t k = id - chunk_base(s, i, c.begin, shift);
    const int64_t n = chunks_each(c.end - c.begin, shift);
    if (k < 0 || k >= n) return c;
    c.seq = i;
    c.k = static_cast<int>(k);
    c.count = static_cast<int>(n);
    c.r0 = c.begin + (c.k << shift);
    const int64_t r1 = static_cast<int64_t>(c.r0) + (int64_t{1} << shift);
    c.r1 = r1 < c.end ? static_cast<int>(r1) : c.end;
    return c;
}

// Sequence i's pool entry: >= 0, kNoSlot (padding) or kBadSlot (out of range,
// or a repeat of an earlier sequence's entry).  Uniform over a wave; every
// lane of the wave must call it.
constexpr int kNoSlot = -1;
constexpr int kBadSlot = -2;

__device__ __forceinline__ int slot_of(const SeqK& s, int i) {
    if (!s.slots) return i;
    const int v = __builtin_amdgcn_readfirstlane(s.slots[i]);
    if (v < 0) return kNoSlot;
    if (v >= s.nslots) return kBadSlot;
    const int lane = __lane_id();
    for (int j0 = 0; j0 < i; j0 += 256) {
        bool same = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = j0 + j * 64 + lane;
            same = same || (at < i && s.slots[at] == v);
        }
        if (__any(same)) return kBadSlot;
    }
    return v;
}

// V consecutive elements of the storage type, widened to fp32, in 16-byte
// accesses (or one shorter access) that the pointer is aligned to.
constexpr int pack_align(int bytes) { return (bytes & -bytes) < 16 ? bytes & -bytes : 16; }
template <typename T, int V>
struct alignas(pack_align(sizeof(T) * V)) Pack {
    T e[V];
};

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> ld_pack(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}

template <typename T, int V>
__device__ __forceinline__ void widen(const Pack<T, V>& v, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = Store<T>::ld(&v.e[i]);
}

template <typename T, int V>
__device__ __forceinline__ void st_pack(T* p, const float (&f)[V]) {
    Pack<T, V> v;
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        __builtin_memcpy(&v, w, sizeof v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) Store<T>::st(&v.e[i], f[i]);
    }
    *reinterpret_cast<Pack<T, V>*>(p) = v;
}

// The logistic function of a gate whose result goes to storage type T.  For
// fp32 the compensated form, which stops at v = -87; a gate multiplies by v,
// so the tail beyond it counts (v = -3e38 gave silu(v) = -5) and is continued
// as e^{v + 87}.  For bf16 the exponent's argument is rounded once
// (relative error at most |v| 2^-24 + 3 ulp, under a hundredth of the half
// step 2^-8 of a bf16 result), and a result below 2^-126 is 0 (at v = -87.4: an
// error of 1.1e-36 in silu at most).
template <typename T>
__device__ __forceinline__ float gate_sigmoid(float v) {
    if constexpr (sizeof(T) == 4)
        return sigmoid(v) * __builtin_amdgcn_exp2f(
                                __builtin_fminf(__builtin_fmaf(v, 1.44269504088896340736f, 125.514468f), 0.0f));
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504088896340736f));
}

// d silu(v) / dv, given sg = sigmoid(v).
__device__ __forceinline__ float silu_grad(float v, float sg) {
    return sg * __builtin_fmaf(v, 1.0f - sg, 1.0f);
}

// Cross-lane sums without a trip through LDS: DPP within rows of 16 lanes,
// swaps between halves and rows of the wave.
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), kCtrl, 0xf, 0xf, true));
}

// Lanes 0-31 receive a's sum with its upper half, lanes 32-63 b's; likewise
// between the even and odd rows of 16 lanes.
__device__ __forceinline__ float swap_add32(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ float swap_add16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The sum over the wave, the same bits in every lane (each step adds the same
// two partial sums in all the lanes that share them).
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0xB1>(v);   // lanes 1 0 3 2 of each quad
    v += dpp<0x4E>(v);   // lanes 2 3 0 1
    v += dpp<0x128>(v);  // rows of 16 rotated by 8
    v += dpp<0x124>(v);  // by 4
    v = swap_add16(v, v);
    return swap_add32(v, v);
}

// Partial sums [parts][cols] (rows `ld` floats apart) summed over the parts in
// a fixed order.  The columns are consecutive planes of `c` (column = plane *
// c + channel); plane p's channel ch goes to the output that holds the plane.
struct ReduceOut {
    float* out;        // null: dropped
    int32_t planes;
    int64_t sc, sp;    // out[channel * sc + plane * sp]
};
struct ReduceK {
    const float* part;
    int64_t parts, ld, c, cols;
    ReduceOut o[3];
};

// Zeros in the rows before the first and behind the last packed sequence (all:
// in every row), of up to five tensors (p null: none; es: bytes of an element).
// It rides on the reduction's launch; seq.cu null and not all: nothing to do.
struct OutsideK {
    SeqK seq;
    int32_t es;
    int32_t all;
    struct {
        void* p;
        int64_t ld, c;
    } t[5];
};
hipError_t launch_reduce_parts(const ReduceK& k, const OutsideK& o, hipStream_t stream);

// Host side ---------------------------------------------------------------

inline SeqK make_seq(const gspn_sequences& s) {
    SeqK k;
    k.cu = s.cu;
    k.slots = s.slots;
    k.resume = s.resume;
    k.rows = static_cast<int32_t>(s.rows);
    k.nseq = static_cast<int32_t>(s.nseq);
    k.len = s.cu || s.nseq == 0 ? 0 : static_cast<int32_t>(s.rows / s.nseq);
    k.nslots = static_cast<int32_t>(s.nslots);
    return k;
}

inline bool aligned_rows(const void* p, int64_t ld, int es, int bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * es % bytes == 0;
}

hipError_t launch_conv_fwd(const gspn_conv_args& a, int dtype, hipStream_t stream);
hipError_t launch_conv_step(const gspn_conv_args& a, int dtype, hipStream_t stream);
// (no sequence: zero gradients)
hipError_t launch_conv_bwd(const gspn_conv_args& a, int dtype, hipStream_t stream);
int64_t conv_bwd_parts(int64_t rows, int64_t nseq, int64_t c);

// How a scan is cut.  shift: rows per chunk as a power of two; a forward or
// backward of one chunk per sequence needs no carries.
int selscan_shift(int64_t rows, int64_t nseq, int64_t channels, int64_t groups, int64_t n, bool ragged);
int selscan_bwd_shift(int64_t rows, int64_t nseq, int64_t channels, int64_t groups, int64_t n, bool ragged);
int64_t selscan_bwd_blocks(int64_t channels, int64_t groups, int64_t n);  // channel blocks of the backward
constexpr int kCheckShift = 3;  // GSPN_SCAN_CHECKPOINT_ROWS
constexpr int kMinChunkShift = 4;
constexpr int kWholeQuad = 63;  // of selscan_shift: no chunks

hipError_t launch_selscan_fwd(const gspn_selscan_args& a, int dtype, hipStream_t stream);
hipError_t launch_selscan_step(const gspn_selscan_args& a, int dtype, hipStream_t stream);
// (no sequence, or no channel: zero gradients)
hipError_t launch_selscan_bwd(const gspn_selscan_args& a, int dtype, hipStream_t stream);

hipError_t launch_join_fwd(const gspn_join_args& a, int dtype, hipStream_t stream);
hipError_t launch_join_bwd(const gspn_join_args& a, int dtype, hipStream_t stream);
int64_t join_bwd_parts(int64_t rows, int64_t c);

#ifdef GSPN_CHECK_LAUNCHES
namespace check {
// Host replay of row-strided accesses: every row's first and last element of
// [rows][c] (elements of es bytes, rows ld apart) must lie in one buffer.
// A row's ends bound its accesses: kernels guard columns beyond c, and take a
// vector where it lies wholly within the row, either because c is whole vectors
// or, in the block join, because a row's last vector starts at c - V (c >= V)
// and its store goes column by column.
inline void replay_rows(const char* kn, const char* what, const void* p, int64_t rows, int64_t ld, int64_t c,
                        int64_t es) {
    if (!p || rows < 1 || c < 1) return;
    const Region r = region_of(p, kn, what);
    int64_t bad = 0;
    for (int64_t i = 0; i < rows; ++i)
        if (!in_region(r, p, i * ld * es, c * es)) ++bad;
    if (bad) violation(kn, what, "%lld rows outside", static_cast<long long>(bad));
    count_accesses(rows * c);
}
}  // namespace check
#define GSPN_REPLAY_ROWS(...) ::gspn::check::replay_rows(__VA_ARGS__)
#define GSPN_REPLAYED(...) ::gspn::check::replayed(__VA_ARGS__)
#else
#define GSPN_REPLAY_ROWS(...) ((void)0)
#define GSPN_REPLAYED(...) ((void)0)
#endif

}  // namespace gspn
