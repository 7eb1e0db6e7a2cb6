// selscan_bwd.hip -- gradients of the selective scan.
//
// With gy' = gy silu(z) and g = dL/dh: g_t = C_t gy'_t + a_{t+1} g_{t+1}, run
// against the row order, and
//   dC_t[n] = sum_c gy' h_t       dB_t[n] = sum_c g_t d x
//   dx = d sum_n g B + D gy'      dd = sum_n g (A a h_{t-1} + x B)
//   dA = sum_t g d a h_{t-1}      ddt = dd softplus'(dt + bias)
// The states come back from the forward's checkpoints, one every 8 rows: a
// wave reruns 8 rows forward, keeping the decays and states in registers, and
// walks back over them.  Four lanes share a channel (SPL states each), which
// keeps those 8 rows within 64 registers.  Each of the four takes a quarter
// of the rows for what is per row and channel (softplus, gate, the outputs);
// the row's values reach the others as DPP operands.
//
// dB and dC are sums over channels: inside a wave by lane swaps (four values
// a swap pair, so that each half, then quarter, of the wave carries another
// value), over a block's four waves in LDS, over blocks by a second pass in a
// fixed order.  The sums over rows (dA, dD, ddt_bias) stay in registers per
// chunk and are joined the same way.
//
// Bound by the vector ALU (busy in 87% of the cycles, by its counter, at two
// waves a SIMD): 8 x 1024 rows of 2304 channels, 16 states, bf16, gated, take
// 300 us here, 79 + 11 for the chunks' own gradients and their join, 16 for the
// sums; the bytes alone would be 58.
#include "selscan.hpp"

#include <type_traits>

namespace gspn {
namespace {

constexpr float kLn2 = 0.693147180559945309417f;
constexpr int kTile = 1 << kCheckShift;  // rows rerun together

// Four values summed over the wave's channels (lanes equal modulo SPLIT): the
// 16-lane row r of the wave receives the sum of v[r == 1 ? 2 : r == 2 ? 1 : r],
// the same bits in the lanes that share it.
template <int SPLIT>
__device__ __forceinline__ float channel_sum(const float (&v)[4]) {
    float s = swap_add16(swap_add32(v[0], v[1]), swap_add32(v[2], v[3]));
    s += dpp<0x128>(s);  // row rotate by 8
    s += dpp<0x124>(s);  // by 4
    if constexpr (SPLIT == 1) {
        s += dpp<0x122>(s);
        s += dpp<0x121>(s);
    }
    return s;
}

// The chunk's own part of dL/dh before its first row, and its sum of d: what
// the join over chunks needs.  One lane a channel, as in the forward.
template <typename T, int NP, bool kScalar>
__global__ __launch_bounds__(64) void selscan_bwd_local_kernel(const SelK p) {
    const Chunk ck = find_chunk(p.seq, blockIdx.x, p.shift);
    if (ck.seq < 0 || ck.k == 0) return;  // nothing before it
    const int N = kScalar ? NP : p.n;
    const int g = blockIdx.y / p.blocks;
    const int local = (blockIdx.y - g * p.blocks) * 64 + static_cast<int>(threadIdx.x);
    const bool live = local < p.per;
    const int c = g * p.per + (live ? local : p.per - 1);
    float A2[NP], ag[NP];
    ld_states<NP, kScalar>(p.A + static_cast<int64_t>(c) * N, N, A2);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        A2[i] = decay_rate(A2[i]);
        ag[i] = 0.0f;
    }
    const float bias = p.bias ? p.bias[c] : 0.0f;
    const unsigned col = static_cast<unsigned>(c);
    const int64_t last = ck.r1 - 1;
    const T* dr = static_cast<const T*>(p.dt) + last * p.lddt;
    const T* gr = static_cast<const T*>(p.gy) + last * p.ldgy;
    const T* zr = p.z ? static_cast<const T*>(p.z) + last * p.ldz : nullptr;
    const T* Cr = static_cast<const T*>(p.C) + last * p.ldc + static_cast<int64_t>(g) * N;
    const int lane = threadIdx.x;
    float sum = 0.0f;
    constexpr int U = NP == 1 ? 8 : 4;
    T nd[U], ng[U], nz[U], nc[U];
    const int bcol = lane < N ? lane : N - 1;
    int loaded = ck.r1 - 1;  // the row that the pointers are on
    auto load = [&]() {      // the next U rows against the row order; past the chunk, its first row again
#pragma unroll
        for (int i = 0; i < U; ++i) {
            nd[i] = dr[col];
            ng[i] = gr[col];
            if (zr) nz[i] = zr[col];
            if constexpr (!kScalar) nc[i] = Cr[bcol];
            if (loaded-- > ck.r0) {
                dr -= p.lddt;
                gr -= p.ldgy;
                if (zr) zr -= p.ldz;
                if constexpr (!kScalar) Cr -= p.ldc;
            }
        }
    };
    Words<T, NP> cw, cw1;
    int words = ck.r1 - 1;
    load();
    if constexpr (kScalar) cw1 = ld_words<T, NP>(Cr);
    for (int t0 = ck.r1 - 1; t0 >= ck.r0; t0 -= U) {
        float d[U], gp[U], cv[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            d[i] = Store<T>::ld(&nd[i]) + bias;
            gp[i] = Store<T>::ld(&ng[i]);
            if constexpr (!kScalar) cv[i] = lane < N ? Store<T>::ld(&nc[i]) : 0.0f;
        }
        if (p.softplus) {
#pragma unroll
            for (int i = 0; i < U; ++i) d[i] = softplus_f(d[i]);
        }
        if (p.z) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float zv = Store<T>::ld(&nz[i]);
                gp[i] *= zv * gate_sigmoid<T>(zv);
            }
        }
        if (t0 - U + 1 < ck.r0) {  // rows before the chunk: no decay, no gradient
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (t0 - i < ck.r0) d[i] = gp[i] = 0.0f;
            }
        } else if (t0 - U >= ck.r0) {
            load();
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if constexpr (kScalar) {
                cw = cw1;
                if (words-- > ck.r0) Cr -= p.ldc;
                cw1 = ld_words<T, NP>(Cr);
            }
            sum += d[i];
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                const float cc = kScalar ? word_value<T, NP>(cw, n) : lane_value(cv[i], n);
                ag[n] = __builtin_amdgcn_exp2f(d[i] * A2[n]) * __builtin_fmaf(cc, gp[i], ag[n]);
            }
        }
    }
    if (!live) return;
    const int64_t id = chunk_base(p.seq, ck.seq, ck.begin, p.shift) + ck.k;
#pragma unroll
    for (int i = 0; i < NP; ++i)
        if (i < N) p.carry[(id * N + i) * p.channels + c] = ag[i];
    p.sums[id * p.channels + c] = step_sum(sum);
}

// The join of long sequences, against the row order: carry[k] := dL/dh after
// chunk k's last row.
__global__ __launch_bounds__(256) void selscan_bwd_join_kernel(const SelK p) {
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
    float g = 0.0f;
    constexpr int U = 16;
    for (int k0 = count - 1; k0 >= 0; k0 -= U) {
        float own[U], d[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            // from the first chunk on the values are of no use: what follows is not stored
            const int64_t k = k0 - j > 0 ? k0 - j : 0;
            own[j] = q[k * step];
            d[j] = sd[k * p.channels];
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (k0 - j >= 0) {
                q[(k0 - j) * step] = g;
                g = carry_over(d[j] * A2, g, own[j]);
            }
        }
    }
}

template <int NP>
struct Split {
    static constexpr int kLanes = NP >= 4 ? 4 : 1;      // lanes sharing a channel
    static constexpr int kStates = NP / kLanes;         // states a lane
    static constexpr int kRows = kTile / kLanes;        // rows of a tile a lane has to itself
    static constexpr int kWaveCh = 64 / kLanes;         // channels a wave
    static constexpr int kBlockCh = 4 * kWaveCh;        // channels a block
};

template <typename T, int NP, bool kGate>
__global__ __launch_bounds__(256, 2) void selscan_bwd_kernel(const SelK p) {
    typedef Split<NP> S;
    constexpr int SPLIT = S::kLanes, SPL = S::kStates, R = S::kRows;
    __shared__ __attribute__((aligned(16))) float bc[2][kTile][2 * NP];
    __shared__ float red[2][4][kTile][2 * NP];
    const Chunk ck = find_chunk(p.seq, blockIdx.x, p.shift);
    const int g = blockIdx.y / p.blocks;
    const int cb = blockIdx.y - g * p.blocks;
    const int tid = threadIdx.x;
    const int wave = tid >> 6;
    const int lane = tid & 63;
    const int sub = lane % SPLIT;
    const int local = cb * S::kBlockCh + wave * S::kWaveCh + lane / SPLIT;
    const bool live = local < p.per;
    const int c = g * p.per + (live ? local : p.per - 1);
    const int n0 = sub * SPL;
    float dA[SPL], dD = 0.0f, db = 0.0f;
#pragma unroll
    for (int s = 0; s < SPL; ++s) dA[s] = 0.0f;

    if (ck.seq >= 0 && ck.r1 > ck.r0) {
        // states beyond n read the last one, and become zero once the loads are under way
        auto state = [&](int s) { return n0 + s < p.n ? n0 + s : p.n - 1; };
        float A2[SPL], ag[SPL];
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
            A2[s] = p.A[static_cast<int64_t>(c) * p.n + state(s)];
            ag[s] = 0.0f;
        }
        const int64_t id = chunk_base(p.seq, ck.seq, ck.begin, p.shift) + ck.k;
        // dL/dh after the chunk: the join's, or the chunks behind it here
        if (ck.count > kDirectChunks) {
#pragma unroll
            for (int s = 0; s < SPL; ++s) ag[s] = p.carry[(id * p.n + state(s)) * p.channels + c];
#pragma unroll
            for (int s = 0; s < SPL; ++s) {
                A2[s] = n0 + s < p.n ? decay_rate(A2[s]) : 0.0f;
                ag[s] = n0 + s < p.n ? ag[s] : 0.0f;
            }
        } else {
            constexpr int U = kDirectChunks - 1;
            float d[U], own[U][SPL];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                d[j] = 0.0f;
#pragma unroll
                for (int s = 0; s < SPL; ++s) own[j][s] = 0.0f;
                if (ck.k + 1 + j < ck.count) {
                    d[j] = p.sums[(id + 1 + j) * p.channels + c];
#pragma unroll
                    for (int s = 0; s < SPL; ++s)
                        own[j][s] = p.carry[((id + 1 + j) * p.n + state(s)) * p.channels + c];
                }
            }
#pragma unroll
            for (int s = 0; s < SPL; ++s) A2[s] = n0 + s < p.n ? decay_rate(A2[s]) : 0.0f;
#pragma unroll
            for (int j = U - 1; j >= 0; --j)  // behind the last: nothing yet, and nothing added
#pragma unroll
                for (int s = 0; s < SPL; ++s)
                    ag[s] = carry_over(0.5f * d[j] * A2[s], ag[s], n0 + s < p.n ? own[j][s] : 0.0f);
        }
        const float bias = p.bias ? p.bias[c] : 0.0f;
        const float skip = p.D ? p.D[c] : 0.0f;
        const T* const B = static_cast<const T*>(p.B) + static_cast<int64_t>(g) * p.n;
        const T* const C = static_cast<const T*>(p.C) + static_cast<int64_t>(g) * p.n;
        const int64_t check0 =
            chunk_base(p.seq, ck.seq, ck.begin, kCheckShift) + ((ck.r0 - ck.begin) >> kCheckShift);
        // A lane's place in a group of SPLIT rows, from the group's uniform
        // first row: four row strides fit 32 bits.
        auto place = [&](int64_t ld) { return static_cast<unsigned>(sub * static_cast<int>(ld) + c); };
        const unsigned ox = place(p.ldx), od = place(p.lddt), og = place(p.ldgy), oz = kGate ? place(p.ldz) : 0;
        const unsigned qx = place(p.lddx), qd = place(p.ldddt), qz = kGate ? place(p.lddz) : 0;

        constexpr int kBC = (kTile * 2 * NP + 255) / 256;  // values of B and C a lane stages
        const int tiles = (ck.r1 - ck.r0 + kTile - 1) / kTile;
        // The walks are on the first rows of the tile to load, or to store,
        // against the row order; within a tile they step by SPLIT rows.
        constexpr int es = sizeof(T);
        const int64_t top = ck.r0 + (tiles - 1) * kTile;
        RowWalk wx(p.x, top, p.ldx, es), wd(p.dt, top, p.lddt, es), wg(p.gy, top, p.ldgy, es);
        RowWalk wz(p.z, kGate ? top : 0, p.ldz, es), wb(B, top, p.ldb, es), wc(C, top, p.ldc, es);
        RowWalk vx(p.dx, top, p.lddx, es), vd(p.ddt, top, p.ldddt, es), vz(p.dz, kGate ? top : 0, p.lddz, es);
        // after a tile's R groups: back to its first row and a tile up
        auto next = [&](RowWalk& w, int64_t ld, int i) { w.step(ld * es * (i + 1 < R ? SPLIT : SPLIT - 2 * kTile)); };
        unsigned obc[kBC];
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            const int v = tid + i * 256;
            const int64_t ld = (v / NP) % 2 == 0 ? p.ldb : p.ldc;
            obc[i] = static_cast<unsigned>(v / (2 * NP) * static_cast<int>(ld) + v % NP);
        }
        T nx[R], nd[R], ng[R], nz[R], nbc[kBC];
        float nh[SPL];
        auto load = [&](int tile) {
            const int base = ck.r0 + tile * kTile;
            const int left = ck.r1 - base - sub;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                nx[i] = nd[i] = ng[i] = nz[i] = T{};
                if (i * SPLIT < left) {
                    nx[i] = wx.at<const T>()[ox];
                    nd[i] = wd.at<const T>()[od];
                    ng[i] = wg.at<const T>()[og];
                    if constexpr (kGate) nz[i] = wz.at<const T>()[oz];
                }
                next(wx, p.ldx, i);
                next(wd, p.lddt, i);
                next(wg, p.ldgy, i);
                if constexpr (kGate) next(wz, p.ldz, i);
            }
#pragma unroll
            for (int i = 0; i < kBC; ++i) {
                const int v = tid + i * 256;
                nbc[i] = T{};
                if (v < kTile * 2 * NP && v % NP < p.n && base + v / (2 * NP) < ck.r1) {
                    if ((v / NP) % 2 == 0) nbc[i] = wb.at<const T>()[obc[i]];
                    else nbc[i] = wc.at<const T>()[obc[i]];
                }
            }
            wb.step(-p.ldb * kTile * es);
            wc.step(-p.ldc * kTile * es);
            const auto q = row_at<const float>(p.check, (check0 + tile) * p.n, p.channels);
#pragma unroll
            for (int s = 0; s < SPL; ++s) nh[s] = q[static_cast<unsigned>(state(s) * p.channels + c)];
        };
        // the block's sums of dB and dC of a finished tile
        auto flush = [&](int tile, int buf) {
#pragma unroll
            for (int i = 0; i < kBC; ++i) {
                const int v = tid + i * 256;
                const int row = v / (2 * NP);
                const int n = v % NP;
                const int r = ck.r0 + tile * kTile + row;
                if (v < kTile * 2 * NP && n < p.n && r < ck.r1) {
                    const int m = v % (2 * NP);
                    const float s = (red[buf][0][row][m] + red[buf][1][row][m]) +
                                    (red[buf][2][row][m] + red[buf][3][row][m]);
                    const int64_t o = ((static_cast<int64_t>(cb) * p.seq.rows + r) * 2 + (v / NP) % 2) * p.groups + g;
                    p.partbc[o * p.n + n] = s;
                }
            }
        };

        load(tiles - 1);
        int buf = 0;
        for (int tile = tiles - 1; tile >= 0; --tile, buf ^= 1) {
            const int base = ck.r0 + tile * kTile;
#pragma unroll
            for (int i = 0; i < kBC; ++i) {
                const int v = tid + i * 256;
                if (v < kTile * 2 * NP) (&bc[buf][0][0])[v] = Store<T>::ld(&nbc[i]);
            }
            float xv[R], dv[R], uv[R], gp[R], sg[R], gz[R], yv[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const bool in = live && base + i * SPLIT + sub < ck.r1;
                const float v = Store<T>::ld(&nd[i]) + bias;
                sg[i] = 1.0f;
                dv[i] = p.softplus ? softplus_f(v, &sg[i]) : v;
                dv[i] = in ? dv[i] : 0.0f;
                xv[i] = in ? Store<T>::ld(&nx[i]) : 0.0f;
                gp[i] = in ? Store<T>::ld(&ng[i]) : 0.0f;
                gz[i] = yv[i] = 0.0f;
                if constexpr (kGate) {
                    const float zv = Store<T>::ld(&nz[i]);
                    const float s = gate_sigmoid<T>(zv);
                    gz[i] = gp[i] * silu_grad(zv, s);
                    gp[i] *= zv * s;
                    gp[i] = in ? gp[i] : 0.0f;
                }
                uv[i] = dv[i] * xv[i];
            }
            __syncthreads();
            if (tile + 1 < tiles) flush(tile + 1, buf ^ 1);
            float a[kTile][SPL], hs[kTile + 1][SPL];  // decays; states before each row, and the last
#pragma unroll
            for (int s = 0; s < SPL; ++s) hs[0][s] = n0 + s < p.n ? nh[s] : 0.0f;
            float sy[4], sb4[4], sa4[4];  // of four rows, until their sums over the quad
            auto forward = [&](auto jc, int i) {
                constexpr int J = decltype(jc)::value;
                const int t = i * SPLIT + J;
                float b[SPL];
                widen(ld_pack<float, SPL>(&bc[buf][t][n0]), b);
                const float d = quad_of<SPLIT, J>(dv[i]);
                const float u = quad_of<SPLIT, J>(uv[i]);
#pragma unroll
                for (int s = 0; s < SPL; ++s) {
                    a[t][s] = __builtin_amdgcn_exp2f(d * A2[s]);
                    hs[t + 1][s] = __builtin_fmaf(a[t][s], hs[t][s], u * b[s]);
                }
                if constexpr (kGate) {
                    float cv[SPL], y = 0.0f;
                    widen(ld_pack<float, SPL>(&bc[buf][t][NP + n0]), cv);
#pragma unroll
                    for (int s = 0; s < SPL; ++s) y = __builtin_fmaf(cv[s], hs[t + 1][s], y);
                    if constexpr (SPLIT == 1) yv[i] = y;
                    else sy[J] = y;
                }
            };
#pragma unroll
            for (int i = 0; i < R; ++i) {
                forward(std::integral_constant<int, 0>{}, i);
                if constexpr (SPLIT == 4) {
                    forward(std::integral_constant<int, 1>{}, i);
                    forward(std::integral_constant<int, 2>{}, i);
                    forward(std::integral_constant<int, 3>{}, i);
                    if constexpr (kGate) yv[i] = quad_gather(sy, sub);
                }
            }

            // the next tile's loads, in flight over the way back alone: over the way
            // forward too they held 14 registers more (325 against 311 us)
            __builtin_amdgcn_sched_barrier(0);
            if (tile > 0) load(tile - 1);
            float gb[R], ga[R], vB[4], vC[4];
            auto back = [&](auto jc, int i) {
                constexpr int J = decltype(jc)::value;
                const int t = i * SPLIT + J;
                float b[SPL], cv[SPL];
                widen(ld_pack<float, SPL>(&bc[buf][t][n0]), b);
                widen(ld_pack<float, SPL>(&bc[buf][t][NP + n0]), cv);
                const float d = quad_of<SPLIT, J>(dv[i]);
                const float u = quad_of<SPLIT, J>(uv[i]);
                const float y = quad_of<SPLIT, J>(gp[i]);
                float sb = 0.0f, sa = 0.0f;
#pragma unroll
                for (int s = 0; s < SPL; ++s) {
                    const float gt = __builtin_fmaf(cv[s], y, ag[s]);
                    const int m = ((kTile - 1 - t) * SPL + s) % 4;
                    vC[m] = y * hs[t + 1][s];
                    vB[m] = gt * u;
                    sb = __builtin_fmaf(gt, b[s], sb);
                    ag[s] = a[t][s] * gt;
                    const float gq = ag[s] * hs[t][s];  // g a h_{t-1}
                    sa = __builtin_fmaf(gq, A2[s], sa);
                    dA[s] = __builtin_fmaf(gq, d, dA[s]);
                }
                if constexpr (SPLIT == 1) {
                    gb[i] = sb;
                    ga[i] = sa;
                } else {
                    sb4[J] = sb;
                    sa4[J] = sa;
                }
                if (((kTile - 1 - t) * SPL + SPL) % 4 == 0) {
                    // row r of the wave holds value m(r): row t + 4 / SPL - 1 - m / SPL, state m % SPL
                    const float rb = channel_sum<SPLIT>(vB);
                    const float rc = channel_sum<SPLIT>(vC);
                    const int r = lane >> 4;
                    const int m = r == 1 ? 2 : r == 2 ? 1 : r;
                    // every lane of a row holds the same bits for its state, and writes
                    // them: a branch for one quad alone cost five instructions a row
                    float* const o = &red[buf][wave][t + 4 / SPL - 1 - m / SPL][n0 + m % SPL];
                    o[0] = rb;
                    o[NP] = rc;
                }
            };
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                if constexpr (SPLIT == 4) {
                    back(std::integral_constant<int, 3>{}, i);
                    back(std::integral_constant<int, 2>{}, i);
                    back(std::integral_constant<int, 1>{}, i);
                }
                back(std::integral_constant<int, 0>{}, i);
                if constexpr (SPLIT == 4) {
                    gb[i] = quad_gather(sb4, sub);
                    ga[i] = quad_gather(sa4, sub);
                }
            }

#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (live && i * SPLIT < ck.r1 - base - sub) {
                    const float ddt = __builtin_fmaf(xv[i], gb[i], ga[i] * kLn2) * sg[i];
                    st_at(vx.at<T>() + qx, __builtin_fmaf(skip, gp[i], dv[i] * gb[i]));
                    st_at(vd.at<T>() + qd, ddt);
                    dD = __builtin_fmaf(gp[i], xv[i], dD);
                    db += ddt;
                    if constexpr (kGate) st_at(vz.at<T>() + qz, gz[i] * __builtin_fmaf(skip, xv[i], yv[i]));
                }
                next(vx, p.lddx, i);
                next(vd, p.ldddt, i);
                if constexpr (kGate) next(vz, p.lddz, i);
            }
        }
        __syncthreads();
        flush(0, buf ^ 1);
    }

    float* const part = p.part + static_cast<int64_t>(blockIdx.x) * (p.n + 2) * p.channels + c;
    dD = quad_sum<SPLIT>(dD);
    db = quad_sum<SPLIT>(db);
    if (!live) return;
#pragma unroll
    for (int s = 0; s < SPL; ++s)
        if (n0 + s < p.n) part[static_cast<int64_t>(n0 + s) * p.channels] = dA[s];
    if (sub == 0) {
        part[static_cast<int64_t>(p.n) * p.channels] = dD;
        part[static_cast<int64_t>(p.n + 1) * p.channels] = db;
    }
}

// dB and dC from the channel blocks' sums [block][row][2][groups * n], in the
// blocks' order; rows outside the sequences have no sums and are not written here.
// Bound by the sums' bytes: 38 MB in 8.6 us for 8192 rows of 2304 channels.
template <typename T>
__global__ __launch_bounds__(256) void selscan_bc_kernel(const SelK p, T* __restrict__ dB, T* __restrict__ dC) {
    const int64_t gn = static_cast<int64_t>(p.groups) * p.n;
    const int64_t per = static_cast<int64_t>(p.seq.rows) * 2 * gn;
    const int lo = seq_begin(p.seq, 0);
    const int hi = seq_end(p.seq, p.seq.nseq - 1, seq_begin(p.seq, p.seq.nseq - 1));
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < per;
         e += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = e / (2 * gn);
        const int64_t m = e - row * 2 * gn;
        if (row < lo || row >= hi) continue;
        float s = 0.0f;
        int b = 0;
        for (; b + 8 <= p.blocks; b += 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = p.partbc[(b + j) * per + e];
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[j];
        }
        for (; b < p.blocks; ++b) s += p.partbc[b * per + e];
        if (m < gn) Store<T>::st(dB + row * gn + m, s);
        else Store<T>::st(dC + row * gn + (m - gn), s);
    }
}

template <typename T, int NP>
void run_bwd(const SelK& k, dim3 grid, hipStream_t stream) {
    if (k.z) hipLaunchKernelGGL((selscan_bwd_kernel<T, NP, true>), grid, dim3(256), 0, stream, k);
    else hipLaunchKernelGGL((selscan_bwd_kernel<T, NP, false>), grid, dim3(256), 0, stream, k);
}

template <typename T>
void run_bwd_n(const SelK& k, dim3 grid, hipStream_t stream) {
    if (k.n <= 1) run_bwd<T, 1>(k, grid, stream);
    else if (k.n <= 4) run_bwd<T, 4>(k, grid, stream);
    else if (k.n <= 8) run_bwd<T, 8>(k, grid, stream);
    else run_bwd<T, 16>(k, grid, stream);
}

template <typename T, int NP>
void run_local(bool scalar, const SelK& k, dim3 grid, hipStream_t stream) {
    if (scalar) hipLaunchKernelGGL((selscan_bwd_local_kernel<T, NP, true>), grid, dim3(64), 0, stream, k);
    else hipLaunchKernelGGL((selscan_bwd_local_kernel<T, NP, false>), grid, dim3(64), 0, stream, k);
}

template <typename T>
void run_local_n(const SelK& k, dim3 grid, hipStream_t stream) {
    const int es = sizeof(T);
    auto scalar = [&](int np) {
        return k.n == np && np * es % 4 == 0 && aligned_rows(k.C, k.ldc, es, 4) &&
               (np < 4 || aligned_rows(k.A, k.n, 4, 16));
    };
    if (k.n <= 1) run_local<T, 1>(sizeof(T) == 4 && scalar(1), k, grid, stream);
    else if (k.n <= 4) run_local<T, 4>(scalar(4), k, grid, stream);
    else if (k.n <= 8) run_local<T, 8>(scalar(8), k, grid, stream);
    else run_local<T, 16>(scalar(16), k, grid, stream);
}

int64_t block_channels(int64_t n) { return n <= 1 ? Split<1>::kBlockCh : Split<4>::kBlockCh; }

}  // namespace

int64_t selscan_bwd_blocks(int64_t channels, int64_t groups, int64_t n) {
    const int64_t bch = block_channels(n);
    return (channels / groups + bch - 1) / bch;
}

// Rows per chunk of the backward.  A cut costs the pass that finds the chunks'
// own gradients, a quarter of the main pass; whole sequences leave SIMDs idle
// where their waves are no multiple of the two a SIMD holds.  By their measured
// times: whole sequences take 485 ns a row for every 2048 waves and 325 for a
// last turn of one wave a SIMD, chunks 0.29 ns for each wave and row.  Measured
// (bf16, 16 states, whole against cut): 8 x 1024 rows of 2304 channels 483 and
// 369 us, 16 x 1024 of 2048 497 and 625, 16 x 1024 of 2304 743 and 687, 32 x
// 1024 of 2304 1175 and 1318, 2 x 2048 of 4096 665 and 339; with 4 states, whose
// times are in the same proportion, 263 and 181, 275 and 295, 346 and 330.  With
// one state, whose waves take 64 channels, whole from two waves a SIMD.  Packed
// sequences are always cut.
//
// Chunks are as long as 16 waves a SIMD allow (four with one state): 8 x 1024
// rows of 2304 channels took 448 us at 4 waves, 374 at 8, 369 at 16 (with 4
// states 243, 197, 181); four of 3136 rows with one state (768 channels, fp32)
// 94 at 4, 103 at 8.
int selscan_bwd_shift(int64_t rows, int64_t nseq, int64_t channels, int64_t groups, int64_t n, bool ragged) {
    const int64_t waves = 4 * groups * selscan_bwd_blocks(channels, groups, n);
    int64_t longest = rows;
    if (!ragged && nseq > 0) longest = rows / nseq;
    int whole = kMinChunkShift;
    while ((int64_t{1} << whole) < longest) ++whole;
    if (!ragged) {
        const int64_t all = nseq * waves, rest = all % 2048;
        const int64_t turns = all / 2048 * 485 + (rest == 0 ? 0 : rest <= 1024 ? 325 : 485);
        if (n > 1 ? longest * turns <= rows * waves * 29 / 100 + 15000 : all >= 2048) return whole;
    }
    int shift = whole;
    while (shift > kMinChunkShift && (rows >> shift) * waves < (n > 1 ? 16384 : 4096)) --shift;
    return shift;
}

namespace {

// The sums over `parts` chunks that lie in `part`, and zeros in the rows
// outside the sequences (none: in every row).
hipError_t finish_selscan_bwd(const gspn_selscan_args& a, const float* part, int64_t parts, bool none, int es,
                              hipStream_t stream) {
    ReduceK r{};
    r.part = part;
    r.parts = parts;
    r.c = a.channels;
    r.ld = r.cols = (a.n + 2) * a.channels;
    r.o[0] = {a.dA, static_cast<int32_t>(a.n), a.n, 1};
    r.o[1] = {a.dD, 1, 1, 0};
    r.o[2] = {a.ddt_bias, 1, 1, 0};
    OutsideK o{};
    o.seq = make_seq(a.seq);
    o.es = es;
    o.all = none;
    o.t[0] = {a.dx, a.lddx, a.channels};
    o.t[1] = {a.ddt, a.ldddt, a.channels};
    o.t[2] = {a.z ? a.dz : nullptr, a.lddz, a.channels};
    o.t[3] = {a.dB, a.groups * a.n, a.groups * a.n};
    o.t[4] = {a.dC, a.groups * a.n, a.groups * a.n};
    return launch_reduce_parts(r, o, stream);
}

}  // namespace

hipError_t launch_selscan_bwd(const gspn_selscan_args& a, int dtype, hipStream_t stream) {
    if (a.seq.nseq == 0 || a.channels == 0)
        return finish_selscan_bwd(a, nullptr, 0, true, dtype == kF32 ? 4 : 2, stream);
    SelK k = selscan_params(a);
    const bool ragged = a.seq.cu != nullptr;
    k.shift = selscan_bwd_shift(a.seq.rows, a.seq.nseq, a.channels, a.groups, a.n, ragged);
    const int64_t ids = chunk_ids(ragged, a.seq.rows, a.seq.nseq, k.shift);
    const bool cut = (int64_t{1} << k.shift) < (ragged ? a.seq.rows : a.seq.rows / a.seq.nseq);
    const int64_t bcb = selscan_bwd_blocks(a.channels, a.groups, a.n);
    // workspace: [dB/dC sums][dA, dD, ddt_bias sums][carries][sums of d]
    k.partbc = static_cast<float*>(a.workspace);
    k.part = k.partbc + bcb * a.seq.rows * 2 * a.groups * a.n;
    k.carry = k.part + ids * (a.n + 2) * a.channels;
    k.sums = k.carry + ids * a.n * a.channels;
    const int es = dtype == kF32 ? 4 : 2;
    (void)es;
    hipError_t e;
    if (cut) {
        const dim3 lg(static_cast<unsigned>(ids), static_cast<unsigned>(k.groups * k.blocks));
#ifdef GSPN_CHECK_LAUNCHES
        replay_selscan("selscan_bwd_local_kernel", a, k, ids, es);
#endif
        GSPN_REPLAYED("selscan_bwd_local_kernel", 64, 0);
        if (dtype == kF32) run_local_n<float>(k, lg, stream);
        else run_local_n<bf16_t>(k, lg, stream);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (needs_join(a, k.shift)) {
            const dim3 jg = sequence_grid((a.channels * a.n + 255) / 256, a.seq.nseq);
            GSPN_REPLAYED("selscan_bwd_join_kernel", 256, 0);
            hipLaunchKernelGGL(selscan_bwd_join_kernel, jg, dim3(256), 0, stream, k);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }
    k.blocks = static_cast<int32_t>(bcb);
    const dim3 grid(static_cast<unsigned>(ids), static_cast<unsigned>(k.groups * bcb));
#ifdef GSPN_CHECK_LAUNCHES
    if (!cut) k.carry = nullptr;
    replay_selscan("selscan_bwd_kernel", a, k, ids, es);
    GSPN_REPLAY_ROWS("selscan_bwd_kernel", "gy", a.gy, a.seq.rows, a.ldgy, a.channels, es);
    GSPN_REPLAY_ROWS("selscan_bwd_kernel", "dx", a.dx, a.seq.rows, a.lddx, a.channels, es);
    GSPN_REPLAY_ROWS("selscan_bwd_kernel", "ddt", a.ddt, a.seq.rows, a.ldddt, a.channels, es);
    GSPN_REPLAY_ROWS("selscan_bwd_kernel", "dz", a.dz, a.seq.rows, a.lddz, a.channels, es);
    GSPN_REPLAY_ROWS("selscan_bwd_kernel", "row sums", k.part, ids * (a.n + 2), a.channels, a.channels, 4);
    GSPN_REPLAY_ROWS("selscan_bwd_kernel", "channel sums", k.partbc, bcb * a.seq.rows, 2 * a.groups * a.n,
                     2 * a.groups * a.n, 4);
#endif
    GSPN_REPLAYED("selscan_bwd_kernel", 256, 2 * kTile * 32 * 4 * 5);
    if (dtype == kF32) run_bwd_n<float>(k, grid, stream);
    else run_bwd_n<bf16_t>(k, grid, stream);
    if ((e = hipGetLastError()) != hipSuccess) return e;

    const int64_t values = a.seq.rows * 2 * a.groups * a.n;
    if (values > 0) {
        const int64_t most = int64_t{1} << 20;  // workgroups; beyond, each takes several runs of values
        const dim3 bg(static_cast<unsigned>((values + 255) / 256 < most ? (values + 255) / 256 : most));
        GSPN_REPLAY_ROWS("selscan_bc_kernel", "dB", a.dB, a.seq.rows, a.groups * a.n, a.groups * a.n, es);
        GSPN_REPLAY_ROWS("selscan_bc_kernel", "dC", a.dC, a.seq.rows, a.groups * a.n, a.groups * a.n, es);
        GSPN_REPLAYED("selscan_bc_kernel", 256, 0);
        if (dtype == kF32)
            hipLaunchKernelGGL(selscan_bc_kernel<float>, bg, dim3(256), 0, stream, k, static_cast<float*>(a.dB),
                               static_cast<float*>(a.dC));
        else
            hipLaunchKernelGGL(selscan_bc_kernel<bf16_t>, bg, dim3(256), 0, stream, k, static_cast<bf16_t*>(a.dB),
                               static_cast<bf16_t*>(a.dC));
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return finish_selscan_bwd(a, k.part, ids, false, es, stream);
}

}  // namespace gspn
