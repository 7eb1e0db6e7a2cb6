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
//
// Measured (bf16, 16 states, gated): one sequence of 65536 rows and 2048
// channels 385 + 70 + 533 us by its kernels, 840 in a row of calls.  The states'
// 5 and 4 instructions alone are 24 + 20 cycles a wave (an exponential counts
// 8), 600 us at 2.4 GHz; the rest is what is per row (step size, gate, loads)
// and the join; x, dt, z, out twice over would be 260 us of memory traffic.
#include "selscan.hpp"

#include <type_traits>

namespace gspn {
namespace {

// One wave: one chunk of one sequence, 64 channels of one group.
// kOut false: the chunk from zero; its last state and sum of d to carry/sums.
// kOut true: the chunk from its first state (carry, or the pool entry for a
// sequence of one chunk), out, kept states, and the pool's new entry.
template <typename T, int NP, bool kScalar, bool kOut>
__global__ __launch_bounds__(64) void selscan_kernel(const SelK p) {
    const Chunk ck = find_chunk(p.seq, blockIdx.x, p.shift);
    if (ck.seq < 0) return;
    if (!kOut && ck.k + 1 == ck.count) return;  // nothing follows
    const int N = kScalar ? NP : p.n;
    const int g = blockIdx.y / p.blocks;
    const int local = (blockIdx.y - g * p.blocks) * 64 + static_cast<int>(threadIdx.x);
    const bool live = local < p.per;
    const int c = g * p.per + (live ? local : p.per - 1);

    // Only the first chunk starts from the pool entry.  The chunk sums take
    // it in (what they leave for the next chunk includes it) and keep a copy
    // in the last chunk's place, which nothing else uses: the second pass
    // overwrites the entry while its first chunk starts.
    int slot = kNoSlot;
    if (p.state && (kOut || ck.k == 0)) slot = slot_of(p.seq, ck.seq);

    float A2[NP], h[NP];
    ld_states<NP, kScalar>(p.A + static_cast<int64_t>(c) * N, N, A2);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        A2[i] = decay_rate(A2[i]);
        h[i] = 0.0f;
    }
    const int64_t plane = static_cast<int64_t>(p.channels);
    const int64_t id = chunk_base(p.seq, ck.seq, ck.begin, p.shift) + ck.k;
    float* const carry = p.carry + id * N * plane;  // null for whole sequences, and then unused
    if (ck.k == 0 && (!kOut || ck.count == 1)) {
        if (slot >= 0 && p.seq.resume && p.seq.resume[ck.seq] != 0)
            ld_states<NP, kScalar>(p.state + (static_cast<int64_t>(slot) * plane + c) * N, N, h);
        if (!kOut && live) {
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (i < N) carry[((ck.count - 1) * static_cast<int64_t>(N) + i) * plane + c] = h[i];
        }
    } else if (kOut && ck.k == 0) {
        const int64_t from = ck.count > kDirectChunks ? 0 : ck.count - 1;  // the join has put it in its place
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (i < N) h[i] = carry[(from * N + i) * plane + c];
    } else if (kOut && ck.count > kDirectChunks) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (i < N) h[i] = carry[i * plane + c];
    } else if (kOut) {
        for (int k = -ck.k; k < 0; ++k) {
            const float d = 0.5f * p.sums[(id + k) * plane + c];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const float last = i < N ? carry[(k * static_cast<int64_t>(N) + i) * plane + c] : 0.0f;
                h[i] = carry_over(d * A2[i], h[i], last);
            }
        }
    }
    const float bias = p.bias ? p.bias[c] : 0.0f;
    const float skip = p.D ? p.D[c] : 0.0f;
    const bool gated = kOut && p.z != nullptr;
    // Row pointers are uniform (scalar registers) and step row by row; the
    // lane's column is a 32-bit offset.  Past the chunk they stay on its last
    // row.
    const unsigned col = static_cast<unsigned>(c);
    const int64_t first = ck.r0;
    const T* xr = static_cast<const T*>(p.x) + first * p.ldx;
    const T* dr = static_cast<const T*>(p.dt) + first * p.lddt;
    const T* zr = gated ? static_cast<const T*>(p.z) + first * p.ldz : nullptr;
    const T* Br = static_cast<const T*>(p.B) + first * p.ldb + static_cast<int64_t>(g) * N;
    const T* Cr = static_cast<const T*>(p.C) + first * p.ldc + static_cast<int64_t>(g) * N;
    T* outr = kOut ? static_cast<T*>(p.out) + first * p.ldo : nullptr;
    const int lane = threadIdx.x;
    const bool mine = lane < 2 * NP && (lane & (NP - 1)) < N;
    // lanes without a value read the last one: a load that only some lanes make
    // is waited for at once (16 x 1024 rows of 2304 channels with one state: 196 us)
    const unsigned bcol = static_cast<unsigned>((lane & (NP - 1)) < N ? lane & (NP - 1) : N - 1);

    constexpr int kSelRows = NP == 1 ? 8 : 4;  // rows whose loads are in flight together
    float sum = 0.0f;
    T nx[kSelRows], nd[kSelRows], nz[kSelRows], nb[kSelRows];
    int loaded = ck.r0;  // the row that the pointers are on
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < kSelRows; ++i) {
            nx[i] = xr[col];
            nd[i] = dr[col];
            if (gated) nz[i] = zr[col];
            if constexpr (!kScalar) nb[i] = (lane < NP ? Br : Cr)[bcol];
            if (++loaded < ck.r1) {
                xr += p.ldx;
                dr += p.lddt;
                if (gated) zr += p.ldz;
                if constexpr (!kScalar) {
                    Br += p.ldb;
                    Cr += p.ldc;
                }
            }
        }
    };
    Words<T, NP> bw, cw, bw1, cw1;
    int words = ck.r0;
    if (ck.r0 < ck.r1) {
        load();
        if constexpr (kScalar) {
            bw1 = ld_words<T, NP>(Br);
            if (kOut) cw1 = ld_words<T, NP>(Cr);
        }
    }
    for (int t0 = ck.r0; t0 < ck.r1; t0 += kSelRows) {
        if (kOut && p.check && ((t0 - ck.begin) & ((1 << kCheckShift) - 1)) == 0) {
            const int64_t kid = chunk_base(p.seq, ck.seq, ck.begin, kCheckShift) + ((t0 - ck.begin) >> kCheckShift);
            float* const q = p.check + kid * N * plane;
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (i < N && live) q[i * plane + col] = h[i];
        }
        // what is per row and channel, four rows at once; a row past the
        // chunk gets a step of zero, which leaves the state as it is
        float xv[kSelRows], d[kSelRows], f[kSelRows], bv[kSelRows];
#pragma unroll
        for (int i = 0; i < kSelRows; ++i) {
            xv[i] = Store<T>::ld(&nx[i]);
            d[i] = Store<T>::ld(&nd[i]) + bias;
            f[i] = 1.0f;
            if constexpr (!kScalar) bv[i] = mine ? Store<T>::ld(&nb[i]) : 0.0f;
        }
        if (p.softplus) {
#pragma unroll
            for (int i = 0; i < kSelRows; ++i) d[i] = softplus_f(d[i]);
        }
        if (gated) {
#pragma unroll
            for (int i = 0; i < kSelRows; ++i) {
                const float zv = Store<T>::ld(&nz[i]);
                f[i] = zv * gate_sigmoid<T>(zv);
            }
        }
        if (t0 + kSelRows > ck.r1) {
#pragma unroll
            for (int i = 0; i < kSelRows; ++i) {
                if (t0 + i >= ck.r1) d[i] = xv[i] = 0.0f;
            }
        } else if (t0 + kSelRows < ck.r1) {
            load();
        }
#pragma unroll
        for (int i = 0; i < kSelRows; ++i) {
            if constexpr (kScalar) {
                bw = bw1;
                cw = cw1;
                if (++words < ck.r1) {  // the next row's words come while this one is computed
                    Br += p.ldb;
                    Cr += p.ldc;
                }
                bw1 = ld_words<T, NP>(Br);
                if (kOut) cw1 = ld_words<T, NP>(Cr);
            }
            const float u = d[i] * xv[i];
            float y = kOut ? skip * xv[i] : 0.0f;
            sum += d[i];
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                const float b = kScalar ? word_value<T, NP>(bw, n) : lane_value(bv[i], n);
                const float a = __builtin_amdgcn_exp2f(d[i] * A2[n]);
                h[n] = __builtin_fmaf(a, h[n], u * b);
                if (kOut) {
                    const float cc = kScalar ? word_value<T, NP>(cw, n) : lane_value(bv[i], NP + n);
                    y = __builtin_fmaf(cc, h[n], y);
                }
            }
            if (kOut && t0 + i < ck.r1) {
                y *= f[i];
                if (slot == kBadSlot) y = __builtin_nanf("");
                if (live) Store<T>::st(outr + col, y);
                outr += p.ldo;
            }
        }
    }
    if (!live) return;
    if (!kOut) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (i < N) p.carry[(id * N + i) * plane + c] = h[i];
        p.sums[id * plane + c] = step_sum(sum);
    } else if (slot >= 0 && ck.k + 1 == ck.count) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float* const q = p.state + (static_cast<int64_t>(slot) * plane + c) * N + i;
            if constexpr (kScalar && NP % 4 == 0) {
                const float four[4] = {h[i & ~3], h[(i & ~3) + 1], h[(i & ~3) + 2], h[(i & ~3) + 3]};
                if (i % 4 == 0) st_pack<float, 4>(q, four);
            } else if (i < N) {
                *q = h[i];
            }
        }
    }
}

// Whole sequences, four lanes a channel: a block takes 64 channels of one
// sequence from its first row to its last, with no chunks to join.  Four lanes
// share a channel (NP / 4 states each), so a sequence offers four times the
// waves of the kernel above and a row a quarter of its instructions; each of
// the four computes a quarter of the rows' step sizes and gates and hands them
// to the others as DPP operands.  B and C are staged through LDS, 16 rows at a
// time, and the next 16 rows' loads are in flight meanwhile.
// A wave of 16 channels (16 states) takes 284 cycles a row alone on its SIMD and
// 194 among others: it takes batches that fill the GPU with whole sequences,
// and short ones, where it is one launch.  Alone, a short one is bound by latency:
// 1 to 16 rows of 1152 channels, fp32, take 5.9 us, 57 11.7, 113 19.3 and 160 23.2,
// which is 4 us of launch, slot and first loads and 120 ns a row.
template <typename T, int NP, bool kGate>
__global__ __launch_bounds__(256) void selscan_quad_kernel(const SelK p) {
    constexpr int SPL = NP / 4;
    constexpr int kRows = 16;
    constexpr int R = kRows / 4;  // rows a lane has to itself
    constexpr int kBC = (kRows * 2 * NP + 255) / 256;
    __shared__ __attribute__((aligned(16))) float bc[2][kRows][2 * NP];
    if (sequence_of_grid() >= p.seq.nseq) return;
    const int s = static_cast<int>(sequence_of_grid());
    const int begin = seq_begin(p.seq, s);
    const int end = seq_end(p.seq, s, begin);
    const int g = blockIdx.x / p.blocks;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int sub = lane & 3;
    const int local = (blockIdx.x - g * p.blocks) * 64 + (tid >> 2);
    const bool live = local < p.per;
    const int c = g * p.per + (live ? local : p.per - 1);
    const int n0 = sub * SPL;
    const int slot = p.state ? slot_of(p.seq, s) : kNoSlot;

    // The first loads all at once: states beyond n read the last one, and become
    // zero once every load is under way.
    float A2[SPL], h[SPL];
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        A2[i] = p.A[static_cast<int64_t>(c) * p.n + (n0 + i < p.n ? n0 + i : p.n - 1)];
        h[i] = 0.0f;
    }
    float* const pool = p.state + (static_cast<int64_t>(slot >= 0 ? slot : 0) * p.channels + c) * p.n + n0;
    if (slot >= 0 && p.seq.resume && p.seq.resume[s] != 0) {
#pragma unroll
        for (int i = 0; i < SPL; ++i)
            if (n0 + i < p.n) h[i] = pool[i];
    }
    const float bias = p.bias ? p.bias[c] : 0.0f;
    const float skip = p.D ? p.D[c] : 0.0f;
    const T* const B = static_cast<const T*>(p.B) + static_cast<int64_t>(g) * p.n;
    const T* const C = static_cast<const T*>(p.C) + static_cast<int64_t>(g) * p.n;
    const int64_t check0 = chunk_base(p.seq, s, begin, kCheckShift);
    auto place = [&](int64_t ld) { return static_cast<unsigned>(sub * static_cast<int>(ld) + c); };
    const unsigned ox = place(p.ldx), od = place(p.lddt), oz = kGate ? place(p.ldz) : 0, oo = place(p.ldo);

    // four rows of bytes each; the walks are on the next rows to load, or store
    constexpr int es = sizeof(T);
    RowWalk wx(p.x, begin, p.ldx, es), wd(p.dt, begin, p.lddt, es), wz(p.z, kGate ? begin : 0, p.ldz, es);
    RowWalk wo(p.out, begin, p.ldo, es), wb(B, begin, p.ldb, es), wc(C, begin, p.ldc, es);
    const int64_t fx = p.ldx * 4 * es, fd = p.lddt * 4 * es, fz = p.ldz * 4 * es, fo = p.ldo * 4 * es;
    // a lane's values of B and C within 16 rows
    unsigned obc[kBC];
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
        const int v = tid + i * 256;
        const int64_t ld = (v / NP) % 2 == 0 ? p.ldb : p.ldc;
        obc[i] = static_cast<unsigned>(v / (2 * NP) * static_cast<int>(ld) + v % NP);
    }

    T nx[R], nd[R], nz[R], nbc[kBC];
    auto load = [&](int base) {
        const int left = end - base - sub;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            nx[i] = nd[i] = nz[i] = T{};
            if (i * 4 < left) {
                nx[i] = wx.at<const T>()[ox];
                nd[i] = wd.at<const T>()[od];
                if constexpr (kGate) nz[i] = wz.at<const T>()[oz];
            }
            wx.step(fx);
            wd.step(fd);
            if constexpr (kGate) wz.step(fz);
        }
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            const int v = tid + i * 256;
            nbc[i] = T{};
            if (v < kRows * 2 * NP && v % NP < p.n && base + v / (2 * NP) < end) {
                if ((v / NP) % 2 == 0) nbc[i] = wb.at<const T>()[obc[i]];
                else nbc[i] = wc.at<const T>()[obc[i]];
            }
        }
        wb.step(p.ldb * kRows * es);
        wc.step(p.ldc * kRows * es);
    };
    if (begin < end) load(begin);
#pragma unroll
    for (int i = 0; i < SPL; ++i) A2[i] = n0 + i < p.n ? decay_rate(A2[i]) : 0.0f;
    int buf = 0;
    for (int base = begin; base < end; base += kRows, buf ^= 1) {
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            const int v = tid + i * 256;
            if (v < kRows * 2 * NP) (&bc[buf][0][0])[v] = Store<T>::ld(&nbc[i]);
        }
        float xv[R], dv[R], uv[R], f[R], yv[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            xv[i] = Store<T>::ld(&nx[i]);
            dv[i] = Store<T>::ld(&nd[i]) + bias;
            f[i] = 1.0f;
            yv[i] = 0.0f;
        }
        if (p.softplus) {
#pragma unroll
            for (int i = 0; i < R; ++i) dv[i] = softplus_f(dv[i]);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if constexpr (kGate) {
                const float zv = Store<T>::ld(&nz[i]);
                f[i] = zv * gate_sigmoid<T>(zv);
            }
            // a row behind the sequence: a step of zero leaves the state as it is
            if (i * 4 >= end - base - sub) dv[i] = xv[i] = 0.0f;
            uv[i] = dv[i] * xv[i];
        }
        __syncthreads();
        if (base + kRows < end) load(base + kRows);

        // Four rows at a time: their B and C come from LDS while the four
        // before are computed, and their decays and inputs are ready before the
        // serial products, so that a wave alone on its SIMD does not wait.
        float b[2][4][SPL], cv[2][4][SPL];
        auto fetch = [&](int i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                widen(ld_pack<float, SPL>(&bc[buf][i * 4 + j][n0]), b[i & 1][j]);
                widen(ld_pack<float, SPL>(&bc[buf][i * 4 + j][NP + n0]), cv[i & 1][j]);
            }
        };
        fetch(0);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (i + 1 < R) fetch(i + 1);
            float a[4][SPL], w[4][SPL], y[4];
            auto ready = [&](auto jc) {
                constexpr int J = decltype(jc)::value;
                const float d = quad_of<4, J>(dv[i]);
                const float u = quad_of<4, J>(uv[i]);
#pragma unroll
                for (int k = 0; k < SPL; ++k) {
                    a[J][k] = __builtin_amdgcn_exp2f(d * A2[k]);
                    w[J][k] = u * b[i & 1][J][k];
                }
            };
            ready(std::integral_constant<int, 0>{});
            ready(std::integral_constant<int, 1>{});
            ready(std::integral_constant<int, 2>{});
            ready(std::integral_constant<int, 3>{});
            __builtin_amdgcn_sched_barrier(0);
            if (p.check && ((i * 4) & ((1 << kCheckShift) - 1)) == 0 && base + i * 4 < end) {
                auto q = row_at<float>(p.check, (check0 + ((base - begin + i * 4) >> kCheckShift)) * p.n, p.channels);
#pragma unroll
                for (int k = 0; k < SPL; ++k)
                    if (live && n0 + k < p.n) st_at(q + static_cast<unsigned>((n0 + k) * p.channels + c), h[k]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[j] = 0.0f;
#pragma unroll
                for (int k = 0; k < SPL; ++k) h[k] = __builtin_fmaf(a[j][k], h[k], w[j][k]);
#pragma unroll
                for (int k = 0; k < SPL; ++k) y[j] = __builtin_fmaf(cv[i & 1][j][k], h[k], y[j]);
            }
            yv[i] = quad_gather(y, sub);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float y = __builtin_fmaf(skip, xv[i], yv[i]) * f[i];
            if (slot == kBadSlot) y = __builtin_nanf("");
            if (live && i * 4 < end - base - sub) st_at(wo.at<T>() + oo, y);
            wo.step(fo);
        }
    }
    if (slot < 0 || !live) return;
#pragma unroll
    for (int i = 0; i < SPL; ++i)
        if (n0 + i < p.n) pool[i] = h[i];
}

// The join over the chunks of a long sequence: carry[k] := the state before
// chunk k.  A lane takes one state of one channel; 16 chunks' values are loaded
// ahead of their serial products.  Bound by the latency of those loads where the
// sequences are few (65536 rows of 2048 channels: 32 turns in 67 us), by the
// carries' bytes where they are many.  At 8 ahead that scan took 854 us in all,
// at 16 840, at 32 835; 16 ragged prompts of 4096 channels, 24 us slower then,
// 261, 263 and 275.
// Four channels a lane, in wider loads, left too few lanes: 852 against 877 us
// for that scan.
__global__ __launch_bounds__(256) void selscan_join_kernel(const SelK p) {
    if (sequence_of_grid() >= p.seq.nseq) return;
    const int s = static_cast<int>(sequence_of_grid());
    const int begin = seq_begin(p.seq, s);
    const int end = seq_end(p.seq, s, begin);
    const int count = static_cast<int>(chunks_each(end - begin, p.shift));
    if (count <= kDirectChunks) return;
    const int e = static_cast<int>(blockIdx.x * 256 + threadIdx.x);  // n * channels + c
    if (e >= p.channels * p.n) return;
    const int i = e / p.channels;
    const int c = e - i * p.channels;
    const int64_t base = chunk_base(p.seq, s, begin, p.shift);
    const int64_t step = static_cast<int64_t>(p.channels) * p.n;
    float* const q = p.carry + base * step + e;
    const float* const sd = p.sums + base * p.channels + c;
    const float A2 = 0.5f * decay_rate(p.A[static_cast<int64_t>(c) * p.n + i]);
    float h = q[(count - 1) * step];  // the state before the sequence
    constexpr int U = 16;
    for (int k0 = 0; k0 < count; k0 += U) {
        float last[U], d[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            // from the last chunk on the values are of no use: what follows is not stored
            const int64_t k = k0 + j < count ? k0 + j : count - 1;
            last[j] = q[k * step];
            d[j] = sd[k * p.channels];
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (k0 + j < count) {
                q[(k0 + j) * step] = h;
                // the first chunk's last state includes the one it began with
                h = carry_over(d[j] * A2, k0 + j > 0 ? h : 0.0f, last[j]);
            }
        }
    }
}

// One token per sequence.  SPLIT lanes share a channel, each with NP / SPLIT
// neighbouring states, so that the pool is read and written in whole cache
// lines; y is summed over the SPLIT lanes.  Bound by the pool's bytes behind a
// latency: 64 sequences of 4096 channels with 16 states 10 us, 3.6 TB/s of 36 MB.
// Three loads follow one another there: the slot, the slots before it, and the
// entry, whose address is the slot's; then an exponential and the store.
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
        // states beyond n read the last one: loads that every lane makes, none waited for by itself
#pragma unroll
        for (int i = 0; i < SPL; ++i) {
            const int at = (n0 + i < p.n ? n0 + i : p.n - 1) - n0;
            h[i] = pool[at];
            A2[i] = Ar[at];
            b[i] = Store<T>::ld(B + at);
            cv[i] = Store<T>::ld(C + at);
        }
    }
    const T xr = static_cast<const T*>(p.x)[s * p.ldx + cc];
    const T dr = static_cast<const T*>(p.dt)[s * p.lddt + cc];
    T zr{};
    if (p.z) zr = static_cast<const T*>(p.z)[s * p.ldz + cc];
    const float bias = p.bias ? p.bias[cc] : 0.0f;
    const float skip = p.D ? p.D[cc] : 0.0f;
    if constexpr (!kVec) {
#pragma unroll
        for (int i = 0; i < SPL; ++i)
            if (n0 + i >= p.n) h[i] = A2[i] = b[i] = cv[i] = 0.0f;
    }
    const float xv = Store<T>::ld(&xr);
    float d = Store<T>::ld(&dr) + bias;
    if (p.softplus) d = softplus_f(d);
    const float u = d * xv;
    float y = 0.0f;
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * decay_rate(A2[i])), h[i], u * b[i]);
        y = __builtin_fmaf(cv[i], h[i], y);
    }
    y = quad_sum<SPLIT>(y);
    if (!live) return;
    if constexpr (kVec) {
        st_pack<float, SPL>(pool, h);
    } else {
#pragma unroll
        for (int i = 0; i < SPL; ++i)
            if (n0 + i < p.n) pool[i] = h[i];
    }
    if (sub == 0) {
        if (p.D) y = __builtin_fmaf(skip, xv, y);
        if (p.z) {
            const float zv = Store<T>::ld(&zr);
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
        return k.n == np && np * es % 4 == 0 && aligned_rows(k.B, k.ldb, es, 4) && aligned_rows(k.C, k.ldc, es, 4) &&
               (np < 4 || (aligned_rows(k.A, k.n, 4, 16) && aligned_rows(k.state, k.n, 4, 16)));
    };
    if (k.n <= 1) run_selscan<T, 1>(out, sizeof(T) == 4 && scalar(1), k, grid, stream);
    else if (k.n <= 4) run_selscan<T, 4>(out, scalar(4), k, grid, stream);
    else if (k.n <= 8) run_selscan<T, 8>(out, scalar(8), k, grid, stream);
    else run_selscan<T, 16>(out, scalar(16), k, grid, stream);
}

template <typename T, int NP>
void run_quad(const SelK& k, dim3 grid, hipStream_t stream) {
    if (k.z) hipLaunchKernelGGL((selscan_quad_kernel<T, NP, true>), grid, dim3(256), 0, stream, k);
    else hipLaunchKernelGGL((selscan_quad_kernel<T, NP, false>), grid, dim3(256), 0, stream, k);
}

template <typename T>
void run_quad_n(const SelK& k, hipStream_t stream) {
    const dim3 grid = sequence_grid(static_cast<int64_t>(k.groups) * k.blocks, k.seq.nseq);
    if (k.n <= 4) run_quad<T, 4>(k, grid, stream);
    else if (k.n <= 8) run_quad<T, 8>(k, grid, stream);
    else run_quad<T, 16>(k, grid, stream);
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

// How the forward is cut: kWholeQuad, or rows per chunk (a power of two; one
// chunk that holds the longest sequence: whole sequences, one lane a channel).
//
// The three ways by their measured cycles at 16 states, taken for any number of
// them: whole sequences with four lanes a channel take longest x (194 R + 90)
// where R counts their waves over the SIMDs, one lane a channel longest x (600 R
// + 300), chunks 980 for each wave and row spread over the SIMDs and some 48000
// for three launches.  Packed sequences are taken as one, the longest they can
// hold.  Measured with pools, four lanes against chunks (us; 16 states): 57 fp32
// rows of 1152 channels 12.2 and 20.4, 113 rows 20.0 and 22.0, 160 24.1 and 22.7,
// 512 66 and 27; bf16, 8 x 1024 rows of 2304 185 and 144, 16 x 1024 of 4096 368 and
// 426, 32 x 1024 of 2304 425 and 471; one lane, 64 x 64 of 4096 73 (four 85, chunks
// 117).  Near a crossing it errs: 4 x 1024 of 4096 runs whole at 144 where chunks
// take 126.  With fewer states chunks gain more than the costs say: that batch with
// four states runs whole at 103 against 72 (8 x 512 of 2304 is cut, 53 against 63),
// and 16 x 1024 of 4096 with one state whole at 370 against 239 (8 and 16 maps of
// 196 rows of 768 are cut, 18 against 48 and 23 against 55).
//
// Chunks of L rows, 16 at least, are as long as their cost is least: the passes'
// uneven end, which grows with L (some 2 (220 + 50 n) L cycles), against the
// join's walk, 312 cycles a chunk of the longest sequence (packed ones are taken
// to hold up to twice the mean, or a quarter of the rows), and the carries' bytes.  Measured at 16, 32, 64,
// 128 and 256 rows (us): 8 x 1024 rows of 2304 channels 142, 139 (and 79, 75, 84
// with 4 states), 16 ragged prompts in 8192 rows of 4096 278 at 16, 240 at 32,
// 261 at 64; 32 x 1024 of 2304 493 at 32, 466, 499 at 128; one of 65536 and 2048
// channels 876 at 64, 830, 849 at 256; four of 3136 rows with one state (768
// channels, fp32) 61, 53, 57.
int selscan_shift(int64_t rows, int64_t nseq, int64_t channels, int64_t groups, int64_t n, bool ragged) {
    const int64_t waves = groups * ((channels / groups + 63) / 64);
    const int64_t longest = ragged || nseq < 1 ? rows : rows / nseq;
    auto per_simd = [](int64_t w) { return (w + 1023) / 1024; };
    const int64_t chunks = rows * waves * 980 / 1024 + 48000;
    const int64_t lanes1 = longest * (600 * per_simd(nseq * waves) + 300);
    const int64_t lanes4 = longest * (194 * per_simd(nseq * waves * 4) + 90);
    if (n > 1 && lanes4 <= lanes1 && lanes4 <= chunks) return kWholeQuad;
    int whole = kMinChunkShift;
    while ((int64_t{1} << whole) < longest) ++whole;
    if (lanes1 <= chunks) return whole;
    int64_t walk = longest;
    if (ragged) {
        const int64_t likely = 2 * rows / nseq > rows / 4 ? 2 * rows / nseq : rows / 4;
        if (walk > likely) walk = likely;
    }
    const int64_t per_chunk = 312 * walk + rows * waves * n * 36 / 100;
    int best = kMinChunkShift;
    int64_t least = 0;
    for (int shift = kMinChunkShift; shift <= whole; ++shift) {
        const int64_t cost = ((440 + 100 * n) << shift) + (per_chunk >> shift);
        if (shift == kMinChunkShift || cost < least) {
            least = cost;
            best = shift;
        }
    }
    return best;
}

hipError_t launch_selscan_fwd(const gspn_selscan_args& a, int dtype, hipStream_t stream) {
    SelK k = selscan_params(a);
    const bool ragged = a.seq.cu != nullptr;
    k.shift = selscan_shift(a.seq.rows, a.seq.nseq, a.channels, a.groups, a.n, ragged);
    if (k.shift == kWholeQuad) {
#ifdef GSPN_CHECK_LAUNCHES
        replay_selscan("selscan_quad_kernel", a, k, 0, dtype == kF32 ? 4 : 2);
#endif
        GSPN_REPLAYED("selscan_quad_kernel", 256, 2 * 16 * 32 * 4);
        if (dtype == kF32) run_quad_n<float>(k, stream);
        else run_quad_n<bf16_t>(k, stream);
        return hipGetLastError();
    }
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
        if (needs_join(a, k.shift)) {
            const dim3 jg = sequence_grid((a.channels * a.n + 255) / 256, a.seq.nseq);
            GSPN_REPLAYED("selscan_join_kernel", 256, 0);
            hipLaunchKernelGGL(selscan_join_kernel, jg, dim3(256), 0, stream, k);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
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
