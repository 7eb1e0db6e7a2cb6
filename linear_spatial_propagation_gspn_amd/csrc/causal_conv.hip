// causal_conv.hip -- the short depthwise causal convolution over token rows:
// prompts (with a state to continue and to leave behind), single tokens, and
// the gradients.
//
// Each output reads width <= 4 rows of its own channel, so the work is a few
// fma an element and the kernels are bound by the bytes of x and y.  A lane
// takes two channels (one where sizes or alignment forbid) and walks down a
// run of rows with the last width - 1 rows in registers, so every row is read
// once but for the halo at the run's start.  Two channels a lane, so that many
// waves with few registers each keep the loads in flight: with eight (16
// bytes of bf16) 8192 rows of 2304 channels took 19.8 us forward and 42
// backward, with four 16.9 and 29.0, with two 16.3 and 27.4 (5.2 TB/s of x and
// y would be 14.5 and 21.7).
#include "sequence.hpp"

namespace gspn {
namespace {

struct ConvK {
    SeqK seq;
    int32_t c;
    int32_t silu;
    const void* x;
    const void* gy;
    void* y;
    void* dx;
    int64_t ldx, ldy, ldgy, lddx;
    const float* w;
    const float* bias;
    void* state;
    float* part;  // backward: [chunk][width + 1][c] partial sums of dweight and dbias
    int32_t shift;
};

constexpr int kConvThreads = 64;
constexpr int kConvRows = 8;  // rows whose loads are in flight together

// Weights [c][K] and the bias of a lane's V channels.
template <int K, int V>
__device__ __forceinline__ void conv_weights(const ConvK& p, int c0, float (&w)[K][V], float (&b)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][v] = p.w[static_cast<int64_t>(c0 + v) * K + j];
        b[v] = p.bias ? p.bias[c0 + v] : 0.0f;
    }
}

template <int K, int V>
__device__ __forceinline__ void conv_pre(const float (&hist)[K - 1][V], const float (&x)[V], const float (&w)[K][V],
                                         const float (&b)[V], float (&pre)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float s = b[v];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) s = __builtin_fmaf(w[j][v], hist[j][v], s);
        pre[v] = __builtin_fmaf(w[K - 1][v], x[v], s);
    }
}

template <int K, int V>
__device__ __forceinline__ void conv_shift(float (&hist)[K - 1][V], const float (&x)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j + 1 < K - 1; ++j) hist[j][v] = hist[j + 1][v];
        hist[K - 2][v] = x[v];
    }
}

// One block: one chunk of rows of one sequence, 64 lanes of V channels.  The
// lanes of a sequence's first chunk also bring the pool entry up to date:
// they alone have read it, so no other block's read can follow their write,
// and what they write is rows of x, which every block only reads.
template <typename T, int K, int V>
__global__ __launch_bounds__(kConvThreads) void conv_fwd_kernel(const ConvK p) {
    const Chunk ck = find_chunk(p.seq, blockIdx.x, p.shift);
    if (ck.seq < 0) return;
    int slot = kNoSlot;
    bool resumed = false;
    if (p.state) {
        slot = slot_of(p.seq, ck.seq);
        resumed = slot >= 0 && p.seq.resume && p.seq.resume[ck.seq] != 0;
    }
    const int c0 = (blockIdx.y * kConvThreads + static_cast<int>(threadIdx.x)) * V;
    if (c0 >= p.c) return;
    const T* __restrict__ x = static_cast<const T*>(p.x) + c0;
    T* __restrict__ y = static_cast<T*>(p.y) + c0;
    T* const pool = static_cast<T*>(p.state) + (slot >= 0 ? static_cast<int64_t>(slot) * (K - 1) * p.c + c0 : 0);

    // Nothing loaded is converted before everything that a run starts with is
    // under way: each conversion between the loads would wait for one of them.
    Pack<T, V> before[K - 1], raw[kConvRows];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int t = ck.r0 - (K - 1) + j;
        before[j] = Pack<T, V>{};
        if (t >= ck.begin) {
            before[j] = ld_pack<T, V>(x + t * p.ldx);
        } else if (resumed) {
            before[j] = ld_pack<T, V>(pool + static_cast<int64_t>(t - ck.begin + K - 1) * p.c);
        }
    }
    auto load = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kConvRows; ++i) {
            const int t = t0 + i < ck.r1 ? t0 + i : ck.r1 - 1;
            raw[i] = ld_pack<T, V>(x + t * p.ldx);
        }
    };
    float w[K][V], b[V];
    conv_weights<K, V>(p, c0, w, b);
    if (ck.r0 < ck.r1) load(ck.r0);
    if (ck.k == 0 && slot >= 0) {
        const int n = ck.end - ck.begin;
        Pack<T, V> tail[K - 1];  // all read before the first is written: short sequences shift the entry
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int t = n - (K - 1) + j;  // row of the sequence, negative: of the entry
            tail[j] = Pack<T, V>{};
            if (t >= 0) {
                tail[j] = ld_pack<T, V>(x + (ck.begin + static_cast<int64_t>(t)) * p.ldx);
            } else if (resumed) {
                tail[j] = ld_pack<T, V>(pool + static_cast<int64_t>(t + K - 1) * p.c);
            }
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) *reinterpret_cast<Pack<T, V>*>(pool + static_cast<int64_t>(j) * p.c) = tail[j];
    }
    float hist[K - 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) widen(before[j], hist[j]);
    for (int t0 = ck.r0; t0 < ck.r1; t0 += kConvRows) {
        if (t0 > ck.r0) load(t0);
#pragma unroll
        for (int i = 0; i < kConvRows; ++i) {
            if (t0 + i < ck.r1) {
                float xv[V], pre[V];
                widen(raw[i], xv);
                conv_pre<K, V>(hist, xv, w, b, pre);
                conv_shift<K, V>(hist, xv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (p.silu) pre[v] *= gate_sigmoid<T>(pre[v]);
                    if (slot == kBadSlot) pre[v] = __builtin_nanf("");
                }
                st_pack<T, V>(y + (t0 + i) * p.ldy, pre);
            }
        }
    }
}

// One token per sequence: the entry's rows and x in, one row out, the entry
// shifted by one row.  Bound by latency: 64 sequences of 4096 channels (4 MB)
// take 3.7 us.
template <typename T, int K, int V>
__global__ __launch_bounds__(kConvThreads) void conv_step_kernel(const ConvK p) {
    const int s = blockIdx.x;
    const int slot = slot_of(p.seq, s);
    if (slot == kNoSlot) return;
    const int c0 = (blockIdx.y * kConvThreads + static_cast<int>(threadIdx.x)) * V;
    if (c0 >= p.c) return;
    T* const yr = static_cast<T*>(p.y) + s * p.ldy + c0;
    if (slot == kBadSlot) {
        float nan[V];
#pragma unroll
        for (int v = 0; v < V; ++v) nan[v] = __builtin_nanf("");
        st_pack<T, V>(yr, nan);
        return;
    }
    T* const pool = static_cast<T*>(p.state) + static_cast<int64_t>(slot) * (K - 1) * p.c + c0;
    float hist[K - 1][V], xv[V], pre[V], w[K][V], b[V];
    widen(ld_pack<T, V>(static_cast<const T*>(p.x) + s * p.ldx + c0), xv);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) widen(ld_pack<T, V>(pool + static_cast<int64_t>(j) * p.c), hist[j]);
    conv_weights<K, V>(p, c0, w, b);
    conv_pre<K, V>(hist, xv, w, b, pre);
    conv_shift<K, V>(hist, xv);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) st_pack<T, V>(pool + static_cast<int64_t>(j) * p.c, hist[j]);
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (p.silu) pre[v] *= gate_sigmoid<T>(pre[v]);
    st_pack<T, V>(yr, pre);
}

// Gradients.  With e_t = gy_t silu'(p_t): dx_t = sum_j w[j] e_{t + K-1-j}, so
// a run of rows walks K - 1 rows past its end (within the sequence) and emits
// dx K - 1 rows behind; dweight and dbias take e of the run's own rows.  Each
// chunk leaves its sums in `part`, joined in a fixed order afterwards.
template <typename T, int K, int V>
__global__ __launch_bounds__(kConvThreads) void conv_bwd_kernel(const ConvK p) {
    const Chunk ck = find_chunk(p.seq, blockIdx.x, p.shift);
    const int c0 = (blockIdx.y * kConvThreads + static_cast<int>(threadIdx.x)) * V;
    if (c0 >= p.c) return;
    float dw[K + 1][V];
#pragma unroll
    for (int j = 0; j <= K; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[j][v] = 0.0f;

    if (ck.seq >= 0 && ck.r1 > ck.r0) {
        const T* __restrict__ x = static_cast<const T*>(p.x) + c0;
        const T* __restrict__ gy = static_cast<const T*>(p.gy) + c0;
        T* __restrict__ dx = static_cast<T*>(p.dx) + c0;
        float w[K][V], b[V];
        conv_weights<K, V>(p, c0, w, b);
        float hist[K - 1][V], e[K][V];  // rows before t; e[i] = e_{t - (K-1) + i}
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) e[j][v] = 0.0f;
        constexpr int R = kConvRows / 2;
        const int stop = ck.r1 + K - 1;
        Pack<T, V> before[K - 1], rx[R], rg[R];  // converted once the run's first loads are all under way
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int t = ck.r0 - (K - 1) + j;
            before[j] = Pack<T, V>{};
            if (t >= ck.begin) before[j] = ld_pack<T, V>(x + t * p.ldx);
        }
        auto load = [&](int t0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int t = t0 + i < ck.end ? t0 + i : ck.end - 1;
                rx[i] = ld_pack<T, V>(x + t * p.ldx);
                rg[i] = ld_pack<T, V>(gy + t * p.ldgy);
            }
        };
        load(ck.r0);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) widen(before[j], hist[j]);
        for (int t0 = ck.r0; t0 < stop; t0 += R) {
            if (t0 > ck.r0) load(t0);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int t = t0 + i;
                if (t < stop) {
                    float xv[V], gv[V], pre[V];
                    widen(rx[i], xv);
                    widen(rg[i], gv);
                    conv_pre<K, V>(hist, xv, w, b, pre);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
#pragma unroll
                        for (int j = 0; j + 1 < K; ++j) e[j][v] = e[j + 1][v];
                        float d = gv[v];
                        if (p.silu) d *= silu_grad(pre[v], gate_sigmoid<T>(pre[v]));
                        e[K - 1][v] = t < ck.end ? d : 0.0f;
                        if (t < ck.r1) {
#pragma unroll
                            for (int j = 0; j < K - 1; ++j)
                                dw[j][v] = __builtin_fmaf(e[K - 1][v], hist[j][v], dw[j][v]);
                            dw[K - 1][v] = __builtin_fmaf(e[K - 1][v], xv[v], dw[K - 1][v]);
                            dw[K][v] += e[K - 1][v];
                        }
                    }
                    conv_shift<K, V>(hist, xv);
                    if (t - (K - 1) >= ck.r0) {
                        float d[V];
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            d[v] = 0.0f;
#pragma unroll
                            for (int j = 0; j < K; ++j) d[v] = __builtin_fmaf(w[j][v], e[K - 1 - j][v], d[v]);
                        }
                        st_pack<T, V>(dx + (t - (K - 1)) * p.lddx, d);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j <= K; ++j)
        st_pack<float, V>(p.part + (static_cast<int64_t>(blockIdx.x) * (K + 1) + j) * p.c + c0, dw[j]);
}

// Zeros in the rows outside the sequences, one wave a row.  Where the sequences
// cover every row, as they mostly do, it costs next to nothing, against a pass
// over all the gradients to clear them beforehand.
__device__ __forceinline__ void zero_outside(const OutsideK& k, int64_t wave, int64_t waves, int lane) {
    int lo = 0, hi = 0;
    if (!k.all) {
        lo = seq_begin(k.seq, 0);
        const int last = k.seq.nseq - 1;
        hi = seq_end(k.seq, last, seq_begin(k.seq, last));
    }
    const int64_t outside = lo + static_cast<int64_t>(k.seq.rows > hi ? k.seq.rows - hi : 0);
    for (int64_t i = wave; i < outside; i += waves) {
        const int64_t row = i < lo ? i : hi + (i - lo);
#pragma unroll
        for (int j = 0; j < 5; ++j) {
            if (!k.t[j].p) continue;
            if (k.es == 4) {
                float* const q = static_cast<float*>(k.t[j].p) + row * k.t[j].ld;
                for (int64_t e = lane; e < k.t[j].c; e += 64) q[e] = 0.0f;
            } else {
                bf16_t* const q = static_cast<bf16_t*>(k.t[j].p) + row * k.t[j].ld;
                for (int64_t e = lane; e < k.t[j].c; e += 64) q[e] = 0;
            }
        }
    }
}

// A column of partial sums per lane, 64 columns and 16 runs of parts a block:
// each run adds its parts in order, then the runs are added in order: 256 parts
// of 11520 columns in 4.2 us (2.8 TB/s), about the time a small launch takes.
// The blocks behind those clear the rows outside the sequences.
constexpr int kReduceRuns = 16;
constexpr int kOutsideBlocks = 64;

__global__ __launch_bounds__(64 * kReduceRuns) void reduce_parts_kernel(const ReduceK k, const OutsideK o) {
    __shared__ float sums[kReduceRuns][64];
    const int lane = threadIdx.x & 63;
    const int run = threadIdx.x >> 6;
    const int64_t mine = (k.cols + 63) / 64;
    if (blockIdx.x >= mine) {
        zero_outside(o, (blockIdx.x - mine) * kReduceRuns + run, kOutsideBlocks * kReduceRuns, lane);
        return;
    }
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + lane;
    const int64_t each = (k.parts + kReduceRuns - 1) / kReduceRuns;
    const int64_t p0 = run * each;
    const int64_t p1 = p0 + each < k.parts ? p0 + each : k.parts;
    float s = 0.0f;
    if (col < k.cols) {
        const float* __restrict__ q = k.part + col;
        int64_t i = p0;
        for (; i + 8 <= p1; i += 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = q[(i + j) * k.ld];
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[j];
        }
        for (; i < p1; ++i) s += q[i * k.ld];
    }
    sums[run][lane] = s;
    __syncthreads();
    if (run != 0 || col >= k.cols) return;
#pragma unroll
    for (int r = 1; r < kReduceRuns; ++r) s += sums[r][lane];
    int64_t plane = col / k.c;
    const int64_t ch = col - plane * k.c;
#pragma unroll
    for (int o = 0; o < 3; ++o) {
        if (plane >= 0 && plane < k.o[o].planes && k.o[o].out)
            k.o[o].out[ch * k.o[o].sc + plane * k.o[o].sp] = s;
        plane -= k.o[o].planes;
    }
}

// Rows per chunk: the longest of 64, 32, 16 that still gives four waves a SIMD
// (of 128 channels), 8 where 16 give less than two.  A longer run re-reads fewer
// halo rows and leaves fewer partial sums: backward, with the reduction, 8192
// rows of 2304 channels took 33 us at 32 and at 16 rows, 928 fp32 rows of 5343
// (2.4 waves a SIMD at 16) 23 at 16 and 29 at 8, 512 rows of 2304 11.6 at 8, 11.8
// at 16 and 15.4 at 32.
int conv_shift_for(int64_t rows, int64_t c) {
    int shift = 6;
    while (shift > 3 && ((rows >> shift) + 1) * ((c + 127) / 128) < (shift > 4 ? 4096 : 2048)) --shift;
    return shift;
}

template <typename T, int K, int V>
void run_conv(int which, const ConvK& k, dim3 grid, hipStream_t stream) {
    if (which == 0) {
        hipLaunchKernelGGL((conv_fwd_kernel<T, K, V>), grid, dim3(kConvThreads), 0, stream, k);
    } else if (which == 1) {
        hipLaunchKernelGGL((conv_step_kernel<T, K, V>), grid, dim3(kConvThreads), 0, stream, k);
    } else {
        hipLaunchKernelGGL((conv_bwd_kernel<T, K, V>), grid, dim3(kConvThreads), 0, stream, k);
    }
}

template <typename T, int V>
void run_conv_width(int which, int64_t width, const ConvK& k, dim3 grid, hipStream_t stream) {
    if (width == 2) run_conv<T, 2, V>(which, k, grid, stream);
    else if (width == 3) run_conv<T, 3, V>(which, k, grid, stream);
    else run_conv<T, 4, V>(which, k, grid, stream);
}

ConvK conv_params(const gspn_conv_args& a) {
    ConvK k{};
    k.seq = make_seq(a.seq);
    k.c = static_cast<int32_t>(a.c);
    k.silu = a.silu != 0;
    k.x = a.x;
    k.gy = a.gy;
    k.y = a.y;
    k.dx = a.dx;
    k.ldx = a.ldx;
    k.ldy = a.ldy;
    k.ldgy = a.ldgy;
    k.lddx = a.lddx;
    k.w = a.weight;
    k.bias = a.bias;
    k.state = a.state;
    k.part = static_cast<float*>(a.workspace);
    return k;
}

hipError_t launch_conv(int which, const gspn_conv_args& a, int dtype, hipStream_t stream) {
    ConvK k = conv_params(a);
    const int es = dtype == kF32 ? 4 : 2;
    const int v = 2, vb = v * es;
    bool vec = a.c % v == 0 && aligned_rows(a.x, a.ldx, es, vb);
    if (which == 2) {
        vec = vec && aligned_rows(a.gy, a.ldgy, es, vb) && aligned_rows(a.dx, a.lddx, es, vb) &&
              aligned_rows(a.workspace, a.c, 4, 8);
    } else {
        vec = vec && aligned_rows(a.y, a.ldy, es, vb) && (!a.state || aligned_rows(a.state, a.c, es, vb));
    }
    const int lanev = vec ? v : 1;
    k.shift = conv_shift_for(a.seq.rows, a.c);
    const int64_t ids = which == 1 ? a.seq.nseq : chunk_ids(a.seq.cu != nullptr, a.seq.rows, a.seq.nseq, k.shift);
    const dim3 grid(static_cast<unsigned>(ids), static_cast<unsigned>((a.c + kConvThreads * lanev - 1) /
                                                                      (kConvThreads * lanev)));
    const char* kn = which == 0 ? "conv_fwd_kernel" : which == 1 ? "conv_step_kernel" : "conv_bwd_kernel";
    (void)kn;
    GSPN_REPLAY_ROWS(kn, "x", a.x, a.seq.rows, a.ldx, a.c, es);
    if (which == 2) {
        GSPN_REPLAY_ROWS(kn, "gy", a.gy, a.seq.rows, a.ldgy, a.c, es);
        GSPN_REPLAY_ROWS(kn, "dx", a.dx, a.seq.rows, a.lddx, a.c, es);
        GSPN_REPLAY_ROWS(kn, "partial sums", a.workspace, ids * (a.width + 1), a.c, a.c, 4);
    } else {
        GSPN_REPLAY_ROWS(kn, "y", a.y, a.seq.rows, a.ldy, a.c, es);
        GSPN_REPLAY_ROWS(kn, "state", a.state, a.seq.nslots * (a.width - 1), a.c, a.c, es);
    }
    GSPN_REPLAY_ROWS(kn, "weight", a.weight, a.c, a.width, a.width, 4);
    GSPN_REPLAYED(kn, kConvThreads, 0);
    if (dtype == kF32) {
        if (vec) run_conv_width<float, 2>(which, a.width, k, grid, stream);
        else run_conv_width<float, 1>(which, a.width, k, grid, stream);
    } else {
        if (vec) run_conv_width<bf16_t, 2>(which, a.width, k, grid, stream);
        else run_conv_width<bf16_t, 1>(which, a.width, k, grid, stream);
    }
    return hipGetLastError();
}

}  // namespace

int64_t conv_bwd_parts(int64_t rows, int64_t nseq, int64_t c) {
    // the larger of the two ways to count, so that the workspace does not depend on the offsets
    const int64_t a = chunk_ids(true, rows, nseq, conv_shift_for(rows, c));
    const int64_t b = chunk_ids(false, rows, nseq, conv_shift_for(rows, c));
    return a > b ? a : b;
}

hipError_t launch_conv_fwd(const gspn_conv_args& a, int dtype, hipStream_t stream) {
    return launch_conv(0, a, dtype, stream);
}

hipError_t launch_conv_step(const gspn_conv_args& a, int dtype, hipStream_t stream) {
    return launch_conv(1, a, dtype, stream);
}

hipError_t launch_conv_bwd(const gspn_conv_args& a, int dtype, hipStream_t stream) {
    const bool none = a.seq.nseq == 0;  // every row is outside, and the sums are over no parts
    const hipError_t e = none ? hipSuccess : launch_conv(2, a, dtype, stream);
    if (e != hipSuccess) return e;
    OutsideK o{};
    o.seq = make_seq(a.seq);
    o.all = none;
    o.es = dtype == kF32 ? 4 : 2;
    o.t[0] = {a.dx, a.lddx, a.c};
    ReduceK r{};
    r.part = static_cast<const float*>(a.workspace);
    if (!none) r.parts = chunk_ids(a.seq.cu != nullptr, a.seq.rows, a.seq.nseq, conv_shift_for(a.seq.rows, a.c));
    r.ld = (a.width + 1) * a.c;
    r.c = a.c;
    r.cols = r.ld;
    r.o[0] = {a.dweight, static_cast<int32_t>(a.width), a.width, 1};
    r.o[1] = {a.dbias, 1, 1, 0};
    r.o[2] = {nullptr, 0, 0, 0};
    return launch_reduce_parts(r, o, stream);
}

hipError_t launch_reduce_parts(const ReduceK& k, const OutsideK& o, hipStream_t stream) {
    const bool outside = o.seq.cu || o.all;
    const dim3 grid(static_cast<unsigned>((k.cols + 63) / 64 + (outside ? kOutsideBlocks : 0)));
    for (const auto& t : o.t) {
        (void)t;
        if (outside) GSPN_REPLAY_ROWS("reduce_parts_kernel", "gradient", t.p, o.seq.rows, t.ld, t.c, o.es);
    }
    GSPN_REPLAY_ROWS("reduce_parts_kernel", "partial sums", k.part, k.parts, k.ld, k.cols, 4);
    GSPN_REPLAYED("reduce_parts_kernel", 64 * kReduceRuns, 64 * kReduceRuns * 4);
    hipLaunchKernelGGL(reduce_parts_kernel, grid, dim3(64 * kReduceRuns), 0, stream, k, o);
    return hipGetLastError();
}

}  // namespace gspn
