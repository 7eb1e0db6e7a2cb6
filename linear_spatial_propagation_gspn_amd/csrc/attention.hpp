// attention.hpp -- what the attention kernels share: parameters, tiles of rows
// in LDS, matrix products of them (internal to libgspn).
//
// Every product here is v_mfma 32x32 with fp32 sums.  Lane l of a wave holds
// row l % 32 of the first factor and column l % 32 of the second; h = l / 32
// picks which of the summed indices the lane holds, and any order of those
// will do if both factors use the same.  A result has column l % 32 in lane l
// and rows 8 (r / 4) + 4 h + r % 4 in its registers r < 16.  So scores are
// formed with their queries (or, for the keys' gradients, their keys) as
// columns: a lane then holds one softmax row, and its registers are the second
// factor of the next product as they stand, without a trip through LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <type_traits>

#include "../../include/gspn_attention.h"
#include "sequence.hpp"

namespace gspn {

// Queries of a workgroup: four waves of 32.
constexpr int kAttnShift = 7;
constexpr int kAttnRows = 1 << kAttnShift;
constexpr int kAttnThreads = 256;
constexpr int kKeyShift = 6;     // keys of a workgroup of their gradients
constexpr int kKeyRows = 1 << kKeyShift;
constexpr int kAppendShift = 3;  // 8 rows a workgroup go into their entries

struct AttnK {
    SeqK seq, kv;
    int32_t heads, kv_heads, group, d, causal;
    int32_t flip;      // scale < 0: queries (keys) enter the scores negated
    float scale;       // as given
    float scale_log2;  // |scale| log2 e, at least 2^-149
    const void* q;
    const void* k;
    const void* v;
    void* out;
    float* lse;
    void* k_pool;
    void* v_pool;
    int64_t capacity;
    const int32_t* held;
    const void* gout;
    void* dq;
    void* dk;
    void* dv;
    float* delta;  // [heads][rows]: <gout, out> of each row
    float* part;   // of the step's splits
    int64_t ldq, ldk, ldv, ldo, ldgo, lddq, lddk, lddv;
    int32_t splits;
    int32_t walks;  // workgroups before those that copy new rows into their entries
};

template <typename T>
constexpr bool kIsBf16 = std::is_same_v<T, bf16_t>;

// Rows of a tile: 16 KB of them at the widest.
template <typename T>
constexpr int kTileRows = kIsBf16<T> ? 64 : 32;


// Blocks of 32 columns that heads of up to D elements take as columns of a result.
template <int D>
constexpr int kBlocks = (D + 31) / 32;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t Quad __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) float lds_float;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) Quad lds_quad;

// The byte address of LDS memory within the workgroup's.
__device__ __forceinline__ uint32_t lds_at(const void* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_char*)p));
}

// 16 bytes at any element's address, zeros behind the `left` elements that the
// head still has.
template <typename T>
__device__ __forceinline__ Quad ld16(const T* p, int left) {
    constexpr int kE = 16 / sizeof(T);
    Quad v = {0, 0, 0, 0};
    if (left >= kE) {
        __builtin_memcpy(&v, p, 16);
    } else if (left > 0) {
        T e[kE];
#pragma unroll
        for (int i = 0; i < kE; ++i) e[i] = i < left ? p[i] : T(0);
        __builtin_memcpy(&v, e, 16);
    }
    return v;
}

// Four consecutive elements of a head, those behind its end left out.
template <typename T>
__device__ __forceinline__ void st4(T* p, int left, float a, float b, float c, float d) {
    Pack<T, 4> v;
    const float f[4] = {a, b, c, d};
    st_pack<T, 4>(&v.e[0], f);
    if (left >= 4) {
        __builtin_memcpy(p, &v, sizeof v);
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < left) p[i] = v.e[i];
    }
}

// a b + c over the 32 bytes a row that two fragments hold between their halves.
template <typename T>
__device__ __forceinline__ f32x16 mma(Quad a, Quad b, f32x16 c) {
    if constexpr (kIsBf16<T>) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
        return c;
    }
}

// The alignment of arrays of tiles.
constexpr int kTileAlign = 256;

// A tile of rows of D elements in LDS, by its byte address there.  LDS gives 256
// bytes a cycle, in banks: its 16-byte chunks are swizzled so that 16 rows'
// chunks of one column (row fragments) and four rows' four of them (transposed
// ones) lie apart.  Chunk c of a row lies at c ^ flip(row), which moves it within
// an aligned span of chunks; flip is linear in the row's bits, so an address is the
// lane's own, exclusive-or a constant, plus a constant: one instruction a read and
// one register a tile.
template <typename T, int D>
struct Tile {
    static constexpr int kRow = 32 * kBlocks<D> * static_cast<int>(sizeof(T));  // bytes
    static constexpr int kChunks = kRow / 16;
    static constexpr int kSteps = D * static_cast<int>(sizeof(T)) / 32;  // products over a whole row
    static constexpr int kE = 16 / static_cast<int>(sizeof(T));
    static constexpr int kSpan = kRow % 256 == 0 ? 16 : kRow % 256 == 128 ? 8 : 4;
    // What a tile's address must be a multiple of: at() changes the address' bits below.
    static constexpr int kAlign = kSpan * 16;
    static_assert(kRow % kAlign == 0 && kAlign <= kTileAlign);

    // Whether step i of a product over a row holds any of the head's d elements.
    // (Only fp32 products take long enough for the question: 2003 rows over 539
    // keys, 6 heads of 40, 77 us in the three kernels of a training step, 72 so.)
    static __device__ __forceinline__ bool holds(int i, int d) { return kIsBf16<T> || 2 * i * kE < d; }

    static __device__ __forceinline__ constexpr int flip(int row) {
        return kSpan == 16  ? (row & 3) << 2 | ((row >> 2) & 3)
               : kSpan == 8 ? (row & 2) << 1 | ((row >> 2) & 3)
                            : (row >> 2) & 3;
    }
    static __device__ __forceinline__ int swizzle(int row, int chunk) { return chunk ^ flip(row); }
    // Chunk c (of the constant part) from a lane's address on.
    static __device__ __forceinline__ uint32_t at(uint32_t x, int c) {
        return (x ^ ((c & (kSpan - 1)) * 16)) + c / kSpan * kSpan * 16;
    }

    // A lane's address for rows().
    static __device__ __forceinline__ uint32_t rows_at(uint32_t tile) {
        const int lane = threadIdx.x & 63, row = lane & 31;
        return tile + row * kRow + (flip(row) ^ (lane >> 5)) * 16;
    }
    // Rows row0 + l % 32 (row0 a multiple of 32) as a first factor, summed over
    // columns: step s.
    static __device__ __forceinline__ Quad rows(uint32_t x, int row0, int s) {
        return *(const lds_quad*)(at(x, 2 * s) + row0 * kRow);
    }

    // A lane's address for columns().
    static __device__ __forceinline__ uint32_t columns_at(uint32_t tile) {
        const int lane = threadIdx.x & 63;
        if constexpr (kIsBf16<T>) {
            // a group of 16 lanes reads four rows of 16 elements and gets them by columns
            const int row = 4 * (lane >> 5) + ((lane & 15) >> 2);
            const int chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
            return tile + row * kRow + (flip(row) ^ chunk) * 16 + 8 * (lane & 1);
        } else {
            const int row = 4 * (lane >> 5);
            return tile + row * kRow + (flip(row) ^ ((lane & 31) >> 2)) * 16 + 4 * (lane & 3);
        }
    }
    // Columns 32 b .. of rows row0 + 16 i .. + 15, transposed: a first factor whose
    // rows are the tile's columns, summed over the tile's rows in the order in
    // which a result's registers 8 i .. hold them.
    static __device__ __forceinline__ Quad column(uint32_t x, int row0, int b, int i) {
        s16x4 v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            v[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4*)(at(x, (4 * b) ^ flip(8 * j)) + (row0 + 16 * i + 8 * j) * kRow));
        Quad a;
        __builtin_memcpy(&a, v, 16);
        return a;
    }
    // c + (columns 32 b .. of rows row0 .. row0 + 31, transposed) p.
    static __device__ __forceinline__ f32x16 columns(uint32_t x, int row0, int b, const Quad (&p)[2], f32x16 c) {
#pragma unroll
        for (int i = 0; i < 2; ++i) c = mma<T>(column(x, row0, b, i), p[i], c);
        return c;
    }
    static __device__ __forceinline__ f32x16 columns(uint32_t x, int row0, int b, const float (&p)[16], f32x16 c) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float a = *(const lds_float*)(at(x, (8 * b) ^ flip(8 * (r / 4) + r % 4)) + (row0 + 8 * (r / 4) + r % 4) * kRow);
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(a, p[r], c, 0, 0, 0);
        }
        return c;
    }
};

// A result's registers as a second factor of Tile::columns.  For bf16 tiles they are
// rounded to bf16, since a product of fp32 factors takes 16 times as long.
template <typename T>
struct Factor;
template <>
struct Factor<bf16_t> {
    Quad p[2];
    __device__ __forceinline__ explicit Factor(const f32x16& f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i / 4][i % 4] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
    // What its rounding took from f: the two together hold f to 2^-16.
    __device__ __forceinline__ Factor left_of(const f32x16& f) const {
        f32x16 r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[2 * i] = f[2 * i] - __uint_as_float(p[i / 4][i % 4] << 16);
            r[2 * i + 1] = f[2 * i + 1] - __uint_as_float(p[i / 4][i % 4] & 0xffff0000u);
        }
        return Factor(r);
    }
};
template <>
struct Factor<float> {
    float p[16];
    __device__ __forceinline__ explicit Factor(const f32x16& f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = f[i];
    }
};

// A sequence's rows of keys or values: those that its cache entry holds, then
// the new ones.
template <typename T>
struct Rows {
    const T* fresh;
    const T* entry;
    int64_t ld, ld_held;
    int32_t held;
    __device__ __forceinline__ const T* at(int row) const {
        return row < held ? entry + row * ld_held : fresh + (row - held) * ld;
    }
};

// A pointer that is the same for the wave, in scalar registers.
template <typename T>
__device__ __forceinline__ const T* same(const T* p) {
    const uint64_t x = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32));
    return reinterpret_cast<const T*>(static_cast<uint64_t>(hi) << 32 | lo);
}

// ROWS rows on their way from memory to a tile, over kThreads threads.
// kDirect: straight to LDS, 1 KB a wave and instruction, which the wave only
// waits for before the barrier that hands the tile over (when it was chosen, a
// prompt of 16384 rows, 32 heads of 128: 2.9 ms through registers, 2.2 so).  It takes rows of whole, aligned
// 16-byte chunks; the swizzle is in the chunk that a lane asks for, and chunks
// behind the head's end keep the zeros that clear() left.
template <typename T, int D, int ROWS, int kThreads, bool kDirect>
struct Stage {
    using Tl = Tile<T, D>;
    static constexpr int kN = ROWS * Tl::kChunks / kThreads;
    static_assert(ROWS * Tl::kChunks % kThreads == 0);
    Quad v[kDirect ? 1 : kN];

    // Rows row0 .., those behind `last` as the last again.
    __device__ __forceinline__ void fetch(int tid, const T* base, int64_t ld, int row0, int last, int d, char* tile) {
        if constexpr (kDirect) {
            fetch_run(tid, base + row0 * ld, ld, last - row0, d, tile);
        } else {
            fetch(tid, Rows<T>{base, nullptr, ld, 0, 0}, row0, last, d, tile);
        }
    }
    __device__ __forceinline__ void fetch(int tid, const Rows<T>& rows, int row0, int last, int d, char* tile) {
        if constexpr (kDirect) {
            if (rows.held <= row0 || rows.held > last || rows.held >= row0 + ROWS) {
                fetch_run(tid, same(rows.at(row0)), rows.held <= row0 ? rows.ld : rows.ld_held, last - row0, d, tile);
                return;
            }
            const uint32_t to = lds_at(tile) + __builtin_amdgcn_readfirstlane(tid >> 6) * 1024;
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int at = i * kThreads + tid;
                const int r = at / Tl::kChunks;
                const int c = Tl::swizzle(r, at % Tl::kChunks);
                const T* const from = rows.at(row0 + r < last ? row0 + r : last) + c * Tl::kE;
                if (c * Tl::kE < d)
                    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to + i * kThreads * 16),
                                 "v"(from)
                                 : "memory", "m0");
            }
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int at = i * kThreads + tid;
                const int row = row0 + at / Tl::kChunks, c = at % Tl::kChunks * Tl::kE;
                v[i] = ld16(rows.at(row < last ? row : last) + c, d - c);
            }
        }
    }
    // Straight to LDS, rows `from` .. of one pitch; `from` is the same for the wave, as the tile's address is.
    __device__ __forceinline__ void fetch_run(int tid, const T* from, int64_t ld, int last, int d, char* tile) {
        const uint32_t pitch = static_cast<uint32_t>(ld) * sizeof(T);
        const uint32_t to = lds_at(tile) + __builtin_amdgcn_readfirstlane(tid >> 6) * 1024;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int at = i * kThreads + tid;
            const int r = at / Tl::kChunks;
            const int c = Tl::swizzle(r, at % Tl::kChunks);
            const uint32_t off = static_cast<uint32_t>(r < last ? r : last) * pitch + c * 16;
            if (c * Tl::kE < d)
                asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to + i * kThreads * 16), "v"(off),
                             "s"(from)
                             : "memory", "m0");
        }
    }
    __device__ __forceinline__ void commit(int tid, char* tile) const {
        if constexpr (kDirect) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int at = i * kThreads + tid;
                const int r = at / Tl::kChunks, c = at % Tl::kChunks;
                *reinterpret_cast<Quad*>(tile + r * Tl::kRow + Tl::swizzle(r, c) * 16) = v[i];
            }
        }
    }
};

// Zeros in `bytes` of tiles, where some of their chunks will not be fetched.
template <bool kDirect>
__device__ __forceinline__ void clear_tiles(int tid, int threads, char* tiles, int bytes, bool whole) {
    if (kDirect && !whole) {
        for (int i = tid * 16; i < bytes; i += threads * 16) *reinterpret_cast<Quad*>(tiles + i) = Quad{0, 0, 0, 0};
        __syncthreads();
    }
}

// A wave's row fragments straight from memory: row `row` (this lane's) of D
// elements, zeros where the row is not wanted.
template <typename T, int D>
__device__ __forceinline__ void ld_rows(const T* row, bool wanted, int d, bool flip, Quad (&f)[Tile<T, D>::kSteps]) {
    const int h = (threadIdx.x & 63) >> 5;
    constexpr int kE = Tile<T, D>::kE;
    constexpr uint32_t kSign = kIsBf16<T> ? 0x80008000u : 0x80000000u;
#pragma unroll
    for (int s = 0; s < Tile<T, D>::kSteps; ++s) {
        const int c = (2 * s + h) * kE;
        f[s] = ld16(row + c, wanted ? d - c : 0);
        if (flip) f[s] ^= Quad{kSign, kSign, kSign, kSign};
    }
}

// The larger, and the sum, of a lane's value and the one 32 lanes away.
__device__ __forceinline__ float both_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float both_sum(float v) { return swap_add32(v, v); }

// The row of a result that its register r holds in this lane.
__device__ __forceinline__ int result_row(int r) { return 8 * (r / 4) + 4 * ((threadIdx.x & 63) >> 5) + r % 4; }

// One row of the result (transposed: this lane's column, blocks of 32 rows),
// times f.
template <typename T, int D>
__device__ __forceinline__ void st_result(T* row, const f32x16 (&o)[kBlocks<D>], float f, int d) {
#pragma unroll
    for (int b = 0; b < kBlocks<D>; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int c = 32 * b + result_row(4 * g);
            st4(row + c, d - c, o[b][4 * g] * f, o[b][4 * g + 1] * f, o[b][4 * g + 2] * f, o[b][4 * g + 3] * f);
        }
}

// The softmax of the rows that a wave's lanes hold, over tiles: the running
// maximum of the scores (unscaled), the sum of this lane's half of the
// numerators and their products with the values.  The maximum that the
// numerators are taken from follows the true one only once it is 2^8 behind (a
// published idea), so that the products are rarely scaled anew; no numerator
// exceeds 2^8.
template <int D>
struct Softmax {
    float m = -INFINITY, l = 0.0f;
    f32x16 o[kBlocks<D>];

    __device__ __forceinline__ Softmax() {
#pragma unroll
        for (int b = 0; b < kBlocks<D>; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[b][r] = 0.0f;
    }
    // The maximum goes on over scores s, -Inf where hidden.
    template <int N>
    __device__ __forceinline__ void meet(const f32x16 (&s)[N], float scale_log2) {
        meet(most(s), scale_log2);
    }
    template <int N>
    static __device__ __forceinline__ float most(const f32x16 (&s)[N]) {
        float t = s[0][0];
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) t = __builtin_fmaxf(t, s[n][r]);
        return t;
    }
    __device__ __forceinline__ void meet(float t, float scale_log2) {
        t = both_max(t);
        if (__any((t - m) * scale_log2 > 8.0f || t != t)) {
            const float top = __builtin_fmaxf(m, t);
            const float a = top == m ? 1.0f : __builtin_amdgcn_exp2f((m - top) * scale_log2);
            m = top;
            l *= a;
#pragma unroll
            for (int b = 0; b < kBlocks<D>; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[b][r] *= a;
        }
    }
    // Scores into numerators.
    template <int N>
    __device__ __forceinline__ void weigh(f32x16 (&s)[N], float scale_log2) {
        const float base = m == -INFINITY ? 0.0f : m * scale_log2;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[n][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][r], scale_log2, -base));
    }
    // Numerators into their sum.
    template <int N>
    __device__ __forceinline__ void add(const f32x16 (&s)[N]) {
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) sum[r % 4] += s[n][r];
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
};

// Where a sequence's keys lie, and how many there are.  state: 0 as they are,
// kNoSlot (padding), kBadSlot (an error).
template <typename T>
struct Keys {
    Rows<T> k, v;
    int32_t count, state;
};

template <typename T>
__device__ __forceinline__ Keys<T> find_keys(const AttnK& a, int seq, int begin, int rows, int kv_head) {
    Keys<T> w = {};
    w.k.ld = a.ldk;
    w.v.ld = a.ldv;
    w.count = rows;
    int first = begin;
    if (a.k_pool) {
        const int slot = slot_of(a.seq, seq);
        if (slot < 0) w.state = slot;
        if (slot >= 0) {
            const int held = a.held ? __builtin_amdgcn_readfirstlane(a.held[seq]) : 0;
            if (held < 0 || held > a.capacity - rows) {
                w.state = kBadSlot;
            } else {
                const int64_t at = (slot * a.capacity * a.kv_heads + kv_head) * a.d;
                w.k.entry = static_cast<const T*>(a.k_pool) + at;
                w.v.entry = static_cast<const T*>(a.v_pool) + at;
                w.k.ld_held = w.v.ld_held = static_cast<int64_t>(a.kv_heads) * a.d;
                w.k.held = w.v.held = held;
                w.count = held + rows;
            }
        }
    } else {
        first = seq_begin(a.kv, seq);
        w.count = seq_end(a.kv, seq, first) - first;
    }
    w.k.fresh = static_cast<const T*>(a.k) + first * a.ldk + static_cast<int64_t>(kv_head) * a.d;
    w.v.fresh = static_cast<const T*>(a.v) + first * a.ldv + static_cast<int64_t>(kv_head) * a.d;
    return w;
}

// A workgroup's queries and head.
struct AttnItem {
    Chunk c;
    int head;
};

// The chunks' ids are counted backwards within a sequence where the last see
// most, so that the longest walks start first.
__device__ __forceinline__ AttnItem find_item(const SeqK& s, int heads, bool backwards, int shift, uint32_t id) {
    AttnItem w;
    w.head = static_cast<int>(id % heads);
    uint32_t chunk = id / heads;
    if (!s.cu) {  // equal sequences take turns
        const uint32_t each = static_cast<uint32_t>(chunks_each(s.len, shift));
        chunk = chunk % s.nseq * each + chunk / s.nseq;
    }
    w.c = find_chunk(s, chunk, shift);
    if (backwards && w.c.seq >= 0) {
        w.c.k = w.c.count - 1 - w.c.k;
        w.c.r0 = w.c.begin + (w.c.k << shift);
        const int64_t r1 = static_cast<int64_t>(w.c.r0) + (int64_t{1} << shift);
        w.c.r1 = r1 < w.c.end ? static_cast<int>(r1) : w.c.end;
    }
    return w;
}


// Host side ---------------------------------------------------------------

AttnK make_attn(const gspn_attn_args& a);
// |scale| log2 e, which a call needs to be finite.
inline float scale_log2(double scale) { return static_cast<float>(std::fabs(scale) * 1.4426950408889634); }
int attn_splits(int64_t nseq, int64_t heads, int64_t kv_heads, int64_t capacity);
constexpr int kAttnMaxSplits = 64;
int attn_bwd_parts(int64_t rows, int64_t nseq, int64_t heads, int64_t kv_rows, int64_t kv_heads);
constexpr int kAttnMaxParts = 16;

hipError_t launch_attn_fwd(const gspn_attn_args& a, int dtype, hipStream_t stream);
hipError_t launch_attn_step(const gspn_attn_args& a, int dtype, hipStream_t stream);
// (no sequence: zero gradients)
hipError_t launch_attn_bwd(const gspn_attn_args& a, int dtype, hipStream_t stream);

hipError_t launch_rotary_fwd(const gspn_rotary_args& a, int dtype, hipStream_t stream);
hipError_t launch_rotary_bwd(const gspn_rotary_args& a, int dtype, hipStream_t stream);
int64_t rotary_bwd_parts(int64_t rows);

// Calls f with the storage type, the width of the tiles that heads of d
// elements take, and whether their rows go straight to LDS.  Widths are whole
// blocks of 32 columns, but for bf16 heads of 65 to 80 elements, whose scores
// take five steps of 16, not six (four maps of 3136 tokens, 16 heads of 72, a
// training step: 1180 us at 96, 1130 so).  fp32 leaves such steps out anyway.
template <typename F>
void attn_dispatch(int dtype, int64_t d, bool direct, F&& f) {
    auto width = [&](auto t, auto straight) {
        constexpr int kOver64 = kIsBf16<decltype(t)> ? 80 : 96;
        if (d <= 64)
            f(t, std::integral_constant<int, 64>{}, straight);
        else if (d <= kOver64)
            f(t, std::integral_constant<int, kOver64>{}, straight);
        else if (d <= 96)
            f(t, std::integral_constant<int, 96>{}, straight);
        else
            f(t, std::integral_constant<int, 128>{}, straight);
    };
    auto way = [&](auto t) {
        if (direct)
            width(t, std::true_type{});
        else
            width(t, std::false_type{});
    };
    if (dtype == GSPN_F32)
        way(float{});
    else
        way(bf16_t{});
}

// Whether rows are whole 16-byte chunks, and a tile's within 2^31 bytes.
inline bool attn_direct(const void* p, int64_t ld, int64_t d, int64_t es) {
    return d * es % 16 == 0 && ld * es <= (int64_t{1} << 25) && aligned_rows(p, ld, static_cast<int>(es), 16);
}

}  // namespace gspn
