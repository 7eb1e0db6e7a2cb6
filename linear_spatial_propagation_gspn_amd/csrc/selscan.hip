// selscan.hip -- the selective scan over token rows: forward (prompts and
// training, keeping states for the backward) and single tokens.
//
// Per channel c and state n the recurrence is h = exp(d A) h + d x B.  It
// costs five vector instructions an element and state, one of them an
// exponential, against 2 bytes an element for each of x, dt, z and out: with
// 16 states the kernels are bound by the vector ALU, not by memory.
//
// One lane holds one channel with all its states.  B_t and C_t are the same
// for a whole wave and come through scalar loads into scalar registers, where
// each is an operand that costs no vector instruction (even bf16's widening
// is a scalar shift).  The rows are cut into chunks so that a few sequences
// fill the GPU: chunk sums first (the chunk run from zero, its last state and
// sum of d), a join over the chunks (the decay of a whole chunk is
// exp(A sum d)), then every chunk again from its true first state.  Where a
// sequence is one chunk, only the last pass runs.
#include "selscan.hpp"

namespace gspn {
namespace {

constexpr int kSelRows = 4;  // rows whose loads are in flight together

// One wave: one chunk of one sequence, 64 channels of one group.
// kOut false: the chunk from zero; its last state and sum of d to carry/sums.
// kOut true: the chunk from its first state (carry, or the pool entry for a
// sequence of one chunk), out, kept states, and the pool's new entry.
template <typename T, int NP, bool kScalar, bool kOut>
__global__ __launch_bounds__(64) void selscan_kernel(const SelK p) {
    const Chunk ck = find_chunk(p.seq, blockIdx.x, p.shift);
    if (ck.seq < 0) return;
    if (!kOut && ck.k + 1 == ck.count) return;  // nothing follows
    const int g = blockIdx.y / p.blocks;
    const int local = (blockIdx.y - g * p.blocks) * 64 + static_cast<int>(threadIdx.x);
    const bool live = local < p.per;
    const int c = g * p.per + (live ? local : p.per - 1);

    int slot = kNoSlot;
    if (kOut && p.state) slot = slot_of(p.seq, ck.seq);

    float A2[NP], h[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        A2[i] = i < p.n ? p.A[static_cast<int64_t>(c) * p.n + i] * kLog2E : 0.0f;
        h[i] = 0.0f;
    }
    const int64_t id = chunk_base(p.seq, ck.seq, ck.begin, p.shift) + ck.k;
    const int64_t plane = static_cast<int64_t>(p.channels);
    if (kOut) {
        if (ck.count > 1) {
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (i < p.n) h[i] = p.carry[(id * p.n + i) * plane + c];
        } else if (slot >= 0 && p.seq.resume && p.seq.resume[ck.seq] != 0) {
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (i < p.n) h[i] = p.state[(static_cast<int64_t>(slot) * plane + c) * p.n + i];
        }
    }
    const float bias = p.bias ? p.bias[c] : 0.0f;
    const float skip = p.D ? p.D[c] : 0.0f;
    const bool gated = p.z != nullptr;
    const T* const x = static_cast<const T*>(p.x);
    const T* const dt = static_cast<const T*>(p.dt);
    const T* const z = static_cast<const T*>(p.z);
    const T* const B = static_cast<const T*>(p.B) + static_cast<int64_t>(g) * p.n;
    const T* const C = static_cast<const T*>(p.C) + static_cast<int64_t>(g) * p.n;
    T* const out = static_cast<T*>(p.out);
    const int lane = threadIdx.x;
    const bool mine = lane < 2 * NP && (lane & (NP - 1)) < p.n;
    const T* const bc = (lane < NP ? B : C) + (lane & (NP - 1));
    const int64_t ldbc = lane < NP ? p.ldb : p.ldc;

    float sum = 0.0f;
    float nx[kSelRows], nd[kSelRows], nz[kSelRows], nb[kSelRows];
    auto load = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kSelRows; ++i) {
            const int64_t t = t0 + i < ck.r1 ? t0 + i : ck.r1 - 1;
            nx[i] = Store<T>::ld(x + t * p.ldx + c);
            nd[i] = Store<T>::ld(dt + t * p.lddt + c);
            nz[i] = kOut && gated ? Store<T>::ld(z + t * p.ldz + c) : 0.0f;
            if constexpr (!kScalar) nb[i] = mine ? Store<T>::ld(bc + t * ldbc) : 0.0f;
        }
    };
    if (ck.r0 < ck.r1) load(ck.r0);
    for (int t0 = ck.r0; t0 < ck.r1; t0 += kSelRows) {
        if (kOut && p.check && ((t0 - ck.begin) & ((1 << kCheckShift) - 1)) == 0) {
            const int64_t kid = chunk_base(p.seq, ck.seq, ck.begin, kCheckShift) + ((t0 - ck.begin) >> kCheckShift);
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (i < p.n && live) p.check[(kid * p.n + i) * plane + c] = h[i];
        }
        float xv[kSelRows], dv[kSelRows], zv[kSelRows], bv[kSelRows];
#pragma unroll
        for (int i = 0; i < kSelRows; ++i) {
            xv[i] = nx[i];
            dv[i] = nd[i];
            zv[i] = nz[i];
            if constexpr (!kScalar) bv[i] = nb[i];
        }
        if (t0 + kSelRows < ck.r1) load(t0 + kSelRows);
#pragma unroll
        for (int i = 0; i < kSelRows; ++i) {
            const int t = t0 + i;
            if (t >= ck.r1) break;
            Words<T, NP> bw, cw;
            if constexpr (kScalar) {
                bw = ld_words<T, NP>(B + t * p.ldb);
                if (kOut) cw = ld_words<T, NP>(C + t * p.ldc);
            }
            float d = dv[i] + bias;
            if (p.softplus) d = softplus_f(d);
            const float u = d * xv[i];
            sum += d;
            float y = 0.0f;
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                const float b = kScalar ? word_value<T, NP>(bw, n) : lane_value(bv[i], n);
                const float a = __builtin_amdgcn_exp2f(d * A2[n]);
                h[n] = __builtin_fmaf(a, h[n], u * b);
                if (kOut) {
                    const float cc = kScalar ? word_value<T, NP>(cw, n) : lane_value(bv[i], NP + n);
                    y = __builtin_fmaf(cc, h[n], y);
                }
            }
            if (kOut) {
                y = __builtin_fmaf(skip, xv[i], y);
                if (gated) y *= zv[i] * gate_sigmoid<T>(zv[i]);
                if (slot == kBadSlot) y = __builtin_nanf("");
                if (live && p.out) Store<T>::st(out + t * p.ldo + c, y);
            }
        }
    }
    if (!live) return;
    if (!kOut) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (i < p.n) p.carry[(id * p.n + i) * plane + c] = h[i];
        p.sums[id * plane + c] = sum;
    } else if (slot >= 0 && ck.k + 1 == ck.count) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (i < p.n) p.state[(static_cast<int64_t>(slot) * plane + c) * p.n + i] = h[i];
    }
}

// The join over a sequence's chunks: carry[k] := the state before chunk k.
// A lane per (state, channel); the chunks' values are loaded eight at a time
// ahead of the serial products.
__global__ __launch_bounds__(256) void selscan_join_kernel(const SelK p) {
    const int s = blockIdx.x;
    const int begin = seq_begin(p.seq, s);
    const int end = seq_end(p.seq, s, begin);
    const int count = static_cast<int>(chunks_each(end - begin, p.shift));
    if (count < 2) return;
    const int slot = p.state ? slot_of(p.seq, s) : kNoSlot;
    const int64_t e = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x;  // n * channels + c
    if (e >= static_cast<int64_t>(p.channels) * p.n) return;
    const int i = static_cast<int>(e / p.channels);
    const int c = static_cast<int>(e - static_cast<int64_t>(i) * p.channels);
    const float A2 = p.A[static_cast<int64_t>(c) * p.n + i] * kLog2E;
    float h = 0.0f;
    if (slot >= 0 && p.seq.resume && p.seq.resume[s] != 0)
        h = p.state[(static_cast<int64_t>(slot) * p.channels + c) * p.n + i];
    const int64_t base = chunk_base(p.seq, s, begin, p.shift);
    const int64_t step = static_cast<int64_t>(p.channels) * p.n;
    float* const q = p.carry + base * step + e;
    const float* const sd = p.sums + base * p.channels + c;
    constexpr int U = 8;
    for (int k0 = 0; k0 < count; k0 += U) {
        float last[U], d[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const bool in = k0 + j + 1 < count;  // the last chunk left nothing
            last[j] = in ? q[(k0 + j) * step] : 0.0f;
            d[j] = in ? sd[static_cast<int64_t>(k0 + j) * p.channels] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (k0 + j < count) {
                q[(k0 + j) * step] = h;
                h = __builtin_fmaf(__builtin_amdgcn_exp2f(d[j] * A2), h, last[j]);
            }
        }
    }
}

// One token per sequence.  SPLIT lanes share a channel, each with NP / SPLIT
// neighbouring states, so that the pool is read and written in whole cache
// lines; y is summed over the SPLIT lanes.  Bound by the pool's bytes.
template <typename T, int NP, int SPLIT, bool kVec>
__global__ __launch_bounds__(256) void selscan_step_kernel(const SelK p) {
    constexpr int SPL = NP / SPLIT;
    const int s = blockIdx.x;
    const int slot = slot_of(p.seq, s);
    if (slot == kNoSlot) return;
    const int sub = threadIdx.x % SPLIT;
    const int c = static_cast<int>(blockIdx.y * (256 / SPLIT) + threadIdx.x / SPLIT);
    const bool live = c < p.channels;
    const int cc = live ? c : p.channels - 1;
    const int g = cc / p.per;
    T* const out = static_cast<T*>(p.out) + s * p.ldo + cc;
    if (slot == kBadSlot) {
        if (live && sub == 0) Store<T>::st(out, __builtin_nanf(""));
        return;
    }
    const int n0 = sub * SPL;
    float* const pool = p.state + (static_cast<int64_t>(slot) * p.channels + cc) * p.n + n0;
    const float* const Ar = p.A + static_cast<int64_t>(cc) * p.n + n0;
    const T* const B = static_cast<const T*>(p.B) + s * p.ldb + static_cast<int64_t>(g) * p.n + n0;
    const T* const C = static_cast<const T*>(p.C) + s * p.ldc + static_cast<int64_t>(g) * p.n + n0;
    float h[SPL], A2[SPL], b[SPL], cv[SPL];
    if constexpr (kVec) {
        widen(ld_pack<float, SPL>(pool), h);
        widen(ld_pack<float, SPL>(Ar), A2);
#pragma unroll
        for (int i = 0; i < SPL; ++i) {
            b[i] = Store<T>::ld(B + i);
            cv[i] = Store<T>::ld(C + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < SPL; ++i) {
            const bool in = n0 + i < p.n;
            h[i] = in ? pool[i] : 0.0f;
            A2[i] = in ? Ar[i] : 0.0f;
            b[i] = in ? Store<T>::ld(B + i) : 0.0f;
            cv[i] = in ? Store<T>::ld(C + i) : 0.0f;
        }
    }
    const float xv = Store<T>::ld(static_cast<const T*>(p.x) + s * p.ldx + cc);
    float d = Store<T>::ld(static_cast<const T*>(p.dt) + s * p.lddt + cc) + (p.bias ? p.bias[cc] : 0.0f);
    if (p.softplus) d = softplus_f(d);
    const float u = d * xv;
    float y = 0.0f;
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * (A2[i] * kLog2E)), h[i], u * b[i]);
        y = __builtin_fmaf(cv[i], h[i], y);
    }
#pragma unroll
    for (int m = 1; m < SPLIT; m *= 2) y += __shfl_xor(y, m);
    if (!live) return;
    if constexpr (kVec) {
        st_pack<float, SPL>(pool, h);
    } else {
#pragma unroll
        for (int i = 0; i < SPL; ++i)
            if (n0 + i < p.n) pool[i] = h[i];
    }
    if (sub == 0) {
        if (p.D) y = __builtin_fmaf(p.D[cc], xv, y);
        if (p.z) {
            const float zv = Store<T>::ld(static_cast<const T*>(p.z) + s * p.ldz + cc);
            y *= zv * gate_sigmoid<T>(zv);
        }
        Store<T>::st(out, y);
    }
}

template <typename T, int NP>
void run_selscan(bool out, bool scalar, const SelK& k, dim3 grid, hipStream_t stream) {
    if (out) {
        if (scalar) hipLaunchKernelGGL((selscan_kernel<T, NP, true, true>), grid, dim3(64), 0, stream, k);
        else hipLaunchKernelGGL((selscan_kernel<T, NP, false, true>), grid, dim3(64), 0, stream, k);
    } else {
        if (scalar) hipLaunchKernelGGL((selscan_kernel<T, NP, true, false>), grid, dim3(64), 0, stream, k);
        else hipLaunchKernelGGL((selscan_kernel<T, NP, false, false>), grid, dim3(64), 0, stream, k);
    }
}

template <typename T>
void run_selscan_n(bool out, const SelK& k, dim3 grid, hipStream_t stream) {
    const int es = sizeof(T);
    auto scalar = [&](int np) {
        return k.n == np && np * es % 4 == 0 && aligned_rows(k.B, k.ldb, es, 4) && aligned_rows(k.C, k.ldc, es, 4);
    };
    if (k.n <= 1) run_selscan<T, 1>(out, sizeof(T) == 4 && scalar(1), k, grid, stream);
    else if (k.n <= 4) run_selscan<T, 4>(out, scalar(4), k, grid, stream);
    else if (k.n <= 8) run_selscan<T, 8>(out, scalar(8), k, grid, stream);
    else run_selscan<T, 16>(out, scalar(16), k, grid, stream);
}

template <typename T>
void run_step(const SelK& k, bool vec, hipStream_t stream) {
    const int split = k.n <= 1 ? 1 : 4;
    const dim3 grid(static_cast<unsigned>(k.seq.nseq), static_cast<unsigned>((k.channels * split + 255) / 256));
    if (k.n <= 1) hipLaunchKernelGGL((selscan_step_kernel<T, 1, 1, false>), grid, dim3(256), 0, stream, k);
    else if (k.n <= 4) hipLaunchKernelGGL((selscan_step_kernel<T, 4, 4, false>), grid, dim3(256), 0, stream, k);
    else if (k.n == 8 && vec) hipLaunchKernelGGL((selscan_step_kernel<T, 8, 4, true>), grid, dim3(256), 0, stream, k);
    else if (k.n <= 8) hipLaunchKernelGGL((selscan_step_kernel<T, 8, 4, false>), grid, dim3(256), 0, stream, k);
    else if (k.n == 16 && vec) hipLaunchKernelGGL((selscan_step_kernel<T, 16, 4, true>), grid, dim3(256), 0, stream, k);
    else hipLaunchKernelGGL((selscan_step_kernel<T, 16, 4, false>), grid, dim3(256), 0, stream, k);
}

}  // namespace

// Rows per chunk.  Cutting a sequence costs a second pass over all but its
// last chunk, so equal sequences stay whole where they fill the GPU by
// themselves (a wave and a half a SIMD); otherwise the chunks are as long as
// four waves a SIMD allow, 16 rows at least.
int selscan_shift(int64_t rows, int64_t nseq, int64_t channels, int64_t groups, bool ragged) {
    const int64_t waves = groups * ((channels / groups + 63) / 64);
    int64_t longest = rows;
    if (!ragged && nseq > 0) longest = rows / nseq;
    int whole = kCheckShift;
    while ((int64_t{1} << whole) < longest) ++whole;
    if (!ragged && nseq * waves >= 1536) return whole;
    int shift = whole;
    while (shift > kCheckShift && (rows >> shift) * waves < 4096) --shift;
    return shift;
}

hipError_t launch_selscan_fwd(const gspn_selscan_args& a, int dtype, hipStream_t stream) {
    SelK k = selscan_params(a);
    const bool ragged = a.seq.cu != nullptr;
    k.shift = selscan_shift(a.seq.rows, a.seq.nseq, a.channels, a.groups, ragged);
    const int64_t ids = chunk_ids(ragged, a.seq.rows, a.seq.nseq, k.shift);
    const bool cut = (int64_t{1} << k.shift) < (ragged ? a.seq.rows : a.seq.rows / a.seq.nseq);
    if (cut) {
        k.carry = static_cast<float*>(a.workspace);
        k.sums = k.carry + ids * a.n * a.channels;
    }
    const dim3 grid(static_cast<unsigned>(ids), static_cast<unsigned>(k.groups * k.blocks));
    const int es = dtype == kF32 ? 4 : 2;
    (void)es;
    if (cut) {
#ifdef GSPN_CHECK_LAUNCHES
        replay_selscan("selscan_kernel", a, k, ids, es);
#endif
        GSPN_REPLAYED("selscan_kernel", 64, 0);
        if (dtype == kF32) run_selscan_n<float>(false, k, grid, stream);
        else run_selscan_n<bf16_t>(false, k, grid, stream);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const dim3 jg(static_cast<unsigned>(a.seq.nseq), static_cast<unsigned>((a.channels * a.n + 255) / 256));
        GSPN_REPLAYED("selscan_join_kernel", 256, 0);
        hipLaunchKernelGGL(selscan_join_kernel, jg, dim3(256), 0, stream, k);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
#ifdef GSPN_CHECK_LAUNCHES
    replay_selscan("selscan_kernel", a, k, ids, es);
#endif
    GSPN_REPLAYED("selscan_kernel", 64, 0);
    if (dtype == kF32) run_selscan_n<float>(true, k, grid, stream);
    else run_selscan_n<bf16_t>(true, k, grid, stream);
    return hipGetLastError();
}

hipError_t launch_selscan_step(const gspn_selscan_args& a, int dtype, hipStream_t stream) {
    const SelK k = selscan_params(a);
    const int spl = a.n == 16 ? 16 : 8;  // bytes of a lane's states
    const bool vec = aligned_rows(a.state, a.n, 4, spl) && aligned_rows(a.A, a.n, 4, spl);
#ifdef GSPN_CHECK_LAUNCHES
    replay_selscan("selscan_step_kernel", a, k, 0, dtype == kF32 ? 4 : 2);
#endif
    GSPN_REPLAYED("selscan_step_kernel", 256, 0);
    if (dtype == kF32) run_step<float>(k, vec, stream);
    else run_step<bf16_t>(k, vec, stream);
    return hipGetLastError();
}

}  // namespace gspn
