// selscan.hpp -- what the selective scan's forward and backward share: the
// launch parameters, the softplus, the wave-uniform loads of B_t and C_t.
#pragma once

#include "sequence.hpp"

namespace gspn {

constexpr float kLog2E = 1.44269504088896340736f;

struct SelK {
    SeqK seq;
    int32_t channels, groups, n, per;  // per: channels a group
    int32_t softplus, shift, blocks;   // blocks: 64-channel blocks a group
    const void* x;
    const void* dt;
    const void* z;
    const void* B;
    const void* C;
    void* out;
    int64_t ldx, lddt, ldz, ldb, ldc, ldo;
    const float* A;
    const float* D;
    const float* bias;
    float* state;   // pool
    float* check;   // kept states [id][n][channels], or null
    float* carry;   // [chunk][n][channels]: last states, then first states
    float* sums;    // [chunk][channels]: sum of d
    // backward
    const void* gy;
    void* dx;
    void* ddt;
    void* dz;
    int64_t ldgy, lddx, ldddt, lddz;
    float* part;    // [chunk][n + 2][channels]: sums for dA, dD, ddt_bias
    float* partbc;  // [channel block][row][2][groups][n]: sums for dB, dC
};

// log(1 + e^v).  With e = e^{-|v|} it is max(v, 0) + log(1 + e); the sum 1 + e
// drops the low bits of a small e, which are added back to first order (the
// whole error of u = 1 + e is e - (u - 1), and log(1 + e) changes by it over u,
// with u between 1 and 2 wherever it matters).
// slope: its derivative 1 / (1 + e^{-v}), from the same e.
__device__ __forceinline__ float softplus_f(float v, float* slope = nullptr) {
    const float e = __builtin_amdgcn_exp2f(-__builtin_fabsf(v) * kLog2E);
    const float u = 1.0f + e;
    const float l = __builtin_amdgcn_logf(u) * 0.693147180559945309417f + (e - (u - 1.0f));
    if (slope) *slope = (v > 0.0f ? 1.0f : e) * __builtin_amdgcn_rcpf(u);
    return (v > 0.0f ? v : 0.0f) + l;
}

// A in units of log2, so that a row's decay is 2^(d A2).  Where that falls
// below the range of fp32 the range's lower end stands for it: it forgets as
// fast, and a step of zero, a skipped row's or one past a chunk's end, leaves a
// state as it is instead of making 0 x Inf of it.
__device__ __forceinline__ float decay_rate(float A) {
    const float v = A * kLog2E, least = -3.402823466e38f;
    return v < least ? least : v;
}

// A wave's B_t and C_t: N values each, the same for every lane.
//  kScalar: N values at a 4-byte aligned address, loaded as dwords by scalar
//    loads (N == NP, even for 16-bit types).
//  otherwise lane i < NP holds B_t[i], lane NP + i C_t[i], and each value is
//    broadcast by a lane read (any N, any alignment).
template <typename T, int NP>
struct Words {
    static constexpr int kCount = NP * static_cast<int>(sizeof(T)) / 4 > 0 ? NP * static_cast<int>(sizeof(T)) / 4 : 1;
    uint32_t w[kCount];
};

typedef const __attribute__((address_space(4))) uint32_t* const_words;

template <typename T, int NP>
__device__ __forceinline__ Words<T, NP> ld_words(const T* p) {
    Words<T, NP> r;
    const const_words q = (const_words)(reinterpret_cast<uintptr_t>(p));
#pragma unroll
    for (int i = 0; i < Words<T, NP>::kCount; ++i) r.w[i] = q[i];
    return r;
}

template <typename T, int NP>
__device__ __forceinline__ float word_value(const Words<T, NP>& r, int i) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[i]);
    const uint32_t w = r.w[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
}

// The n (<= NP) values of a channel's row of A or of a pool entry.  kWhole: n is
// NP and the rows are 16-byte aligned (NP a multiple of 4): one cache line a
// lane in four accesses instead of 16.
template <int NP, bool kWhole>
__device__ __forceinline__ void ld_states(const float* p, int n, float (&v)[NP]) {
    if constexpr (kWhole && NP % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NP; i += 4) {
            const Pack<float, 4> q = ld_pack<float, 4>(p + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i + j] = q.e[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) v[i] = i < n ? p[i] : 0.0f;
    }
}

// A chunk's sum of d, for its whole decay.  Steps that add up to Inf are taken as
// the most that fp32 holds, so that A = 0 still leaves a state as it is.  (A step
// that is Inf or NaN itself has made a NaN of the chunk's own state, or a zero of
// its decay, either way.)
__device__ __forceinline__ float step_sum(float sum) {
    const float most = 3.402823466e38f;
    return __builtin_fmaxf(__builtin_fminf(sum, most), -most);
}

// A state (or gradient) h taken over a chunk whose decay is 2^(2 half), plus
// the chunk's own.  In two halves up to 2^254, where every normal h overflows,
// and a third factor beyond, for a subnormal one, up to 2^381, where that does
// too: a decay past the range of fp32 (A > 0) leaves zero at zero and gives a
// small h what the rows one by one give it.
__device__ __forceinline__ float carry_over(float half, float h, float own) {
    const float e = __builtin_amdgcn_exp2f(half < 127.0f ? half : 127.0f);
    const float over = __builtin_fmaf(2.0f, half, -254.0f);
    const float f = __builtin_amdgcn_exp2f(__builtin_fminf(__builtin_fmaxf(over, 0.0f), 127.0f));
    return __builtin_fmaf(h * e * f, e, own);
}

__device__ __forceinline__ float lane_value(float v, int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

// A uniform pointer to `row` of a tensor, kept in scalar registers: without
// this the compiler carries a 64-bit vector address for every tensor and row of
// a tile over the loop, and spills.
template <typename T>
__device__ __forceinline__ __attribute__((address_space(1))) T* row_at(const void* p, int64_t row, int64_t ld) {
    uintptr_t a = reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(row * ld) * sizeof(T);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
    a = (static_cast<uintptr_t>(hi) << 32) | lo;
    asm volatile("" : "+s"(a));
    return (__attribute__((address_space(1))) T*)a;
}

// A uniform pointer that steps over the rows of a tensor, in scalar registers.
struct RowWalk {
    uintptr_t a;
    __device__ __forceinline__ RowWalk(const void* p, int64_t row, int64_t ld, int es) {
        a = reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(row * ld * es);
        const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
        const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
        a = (static_cast<uintptr_t>(hi) << 32) | lo;
    }
    template <typename T>
    __device__ __forceinline__ __attribute__((address_space(1))) T* at() const {
        return (__attribute__((address_space(1))) T*)a;
    }
    __device__ __forceinline__ void step(int64_t bytes) {
        a += static_cast<uintptr_t>(bytes);
        asm volatile("" : "+s"(a));
    }
};

__device__ __forceinline__ void st_at(__attribute__((address_space(1))) float* p, float v) { *p = v; }
__device__ __forceinline__ void st_at(__attribute__((address_space(1))) bf16_t* p, float v) { *p = f32_to_bf16(v); }

// Lane J of each quad to all four (SPLIT 4), or the lane's own value.
template <int SPLIT, int J>
__device__ __forceinline__ float quad_of(float v) {
    if constexpr (SPLIT == 1) return v;
    return dpp<J * 0x55>(v);
}

template <int SPLIT>
__device__ __forceinline__ float quad_sum(float v) {
    if constexpr (SPLIT == 1) return v;
    v += dpp<0xB1>(v);  // lanes 1 0 3 2
    v += dpp<0x4E>(v);  // lanes 2 3 0 1
    return v;
}

// Four values summed over each quad; lane J of the quad receives the sum of
// v[J].  Each step keeps half of the values and hands over the other half.
__device__ __forceinline__ float quad_gather(const float (&v)[4], int sub) {
    const bool odd = (sub & 1) != 0, high = (sub & 2) != 0;
    const float a = (odd ? v[1] : v[0]) + dpp<0xB1>(odd ? v[0] : v[1]);
    const float b = (odd ? v[3] : v[2]) + dpp<0xB1>(odd ? v[2] : v[3]);
    return (high ? b : a) + dpp<0x4E>(high ? a : b);
}

// Sequences of up to this many chunks need no launch to join them: a chunk
// walks over those before it (or behind it, in the backward) by itself, at
// about one row's work each.  Longer walks cost more than the launch: 16
// prompts in 2048 rows of 4096 channels took 84 us, and 92 at 16 chunks; their
// backward 219 and 242.
constexpr int kDirectChunks = 4;

inline bool needs_join(const gspn_selscan_args& a, int shift) {
    return (a.seq.cu ? (a.seq.rows >> shift) + 1 : chunks_each(a.seq.rows / a.seq.nseq, shift)) > kDirectChunks;
}

// A grid of `blocks` workgroups for each sequence, the sequence's own side by
// side: they spread over the XCDs, whatever its neighbours' lengths.  (With the
// sequences side by side instead, all of one sequence's went to one XCD wherever
// their number was a multiple of eight: a prompt of 8192 rows behind 63 single
// tokens, 4096 channels, took 478 us against 250.)
inline dim3 sequence_grid(int64_t blocks, int64_t nseq) {
    const int64_t y = nseq < 65535 ? nseq : 65535;
    return dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(y), static_cast<unsigned>((nseq + y - 1) / y));
}

// The sequence of a workgroup of such a grid; nseq or more: none.
__device__ __forceinline__ int64_t sequence_of_grid() {
    return static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y;
}

inline SelK selscan_params(const gspn_selscan_args& a) {
    SelK k{};
    k.seq = make_seq(a.seq);
    k.channels = static_cast<int32_t>(a.channels);
    k.groups = static_cast<int32_t>(a.groups);
    k.n = static_cast<int32_t>(a.n);
    k.per = static_cast<int32_t>(a.channels / a.groups);
    k.softplus = a.softplus != 0;
    k.blocks = (k.per + 63) / 64;
    k.x = a.x;
    k.dt = a.dt;
    k.z = a.z;
    k.B = a.B;
    k.C = a.C;
    k.out = a.out;
    k.ldx = a.ldx;
    k.lddt = a.lddt;
    k.ldz = a.ldz;
    k.ldb = a.ldb;
    k.ldc = a.ldc;
    k.ldo = a.ldo;
    k.A = a.A;
    k.D = a.D;
    k.bias = a.dt_bias;
    k.state = a.state;
    k.check = a.checkpoints;
    k.gy = a.gy;
    k.dx = a.dx;
    k.ddt = a.ddt;
    k.dz = a.dz;
    k.ldgy = a.ldgy;
    k.lddx = a.lddx;
    k.ldddt = a.ldddt;
    k.lddz = a.lddz;
    return k;
}

#ifdef GSPN_CHECK_LAUNCHES
inline void replay_selscan(const char* kn, const gspn_selscan_args& a, const SelK& k, int64_t ids, int es) {
    GSPN_REPLAY_ROWS(kn, "x", a.x, a.seq.rows, a.ldx, a.channels, es);
    GSPN_REPLAY_ROWS(kn, "dt", a.dt, a.seq.rows, a.lddt, a.channels, es);
    GSPN_REPLAY_ROWS(kn, "z", a.z, a.seq.rows, a.ldz, a.channels, es);
    GSPN_REPLAY_ROWS(kn, "B", a.B, a.seq.rows, a.ldb, a.groups * a.n, es);
    GSPN_REPLAY_ROWS(kn, "C", a.C, a.seq.rows, a.ldc, a.groups * a.n, es);
    GSPN_REPLAY_ROWS(kn, "out", a.out, a.seq.rows, a.ldo, a.channels, es);
    GSPN_REPLAY_ROWS(kn, "A", a.A, a.channels, a.n, a.n, 4);
    GSPN_REPLAY_ROWS(kn, "state", a.state, a.seq.nslots, a.channels * a.n, a.channels * a.n, 4);
    if (k.carry) {
        GSPN_REPLAY_ROWS(kn, "carry", k.carry, ids * a.n, a.channels, a.channels, 4);
        GSPN_REPLAY_ROWS(kn, "sums", k.sums, ids, a.channels, a.channels, 4);
    }
    if (a.checkpoints) {
        const int64_t kept = chunk_ids(a.seq.cu != nullptr, a.seq.rows, a.seq.nseq, kCheckShift);
        GSPN_REPLAY_ROWS(kn, "checkpoints", a.checkpoints, kept * a.n, a.channels, a.channels, 4);
    }
}
#endif

}  // namespace gspn
