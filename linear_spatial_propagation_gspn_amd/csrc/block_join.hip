// block_join.hip -- a block's output joined to the residual stream, with the
// norms around it: optional norm, gate, scale and residual, and the norm that
// the next block reads.
//
// Row by row; every tensor is read once and written once, so the kernels are
// bound by those bytes: 16384 rows of 2304 channels (bf16, gate, fp32 residual,
// all parts) take 108 us forward and 175 + 6 backward, 4.9 and 4.7 TB/s against
// the 5.2 of a large copy.  A row lives in the registers of the lanes that share
// it, eight channels each: a wave for up to 512 channels, a workgroup of as
// many waves as the row fills above.  The backward keeps the columns' sums for
// the parameters' gradients in registers over all the rows a workgroup walks and
// leaves one partial row each, joined in a fixed order.
#include "sequence.hpp"

#include <type_traits>

namespace gspn {
namespace {

constexpr int64_t kWaveRow = 512;  // channels up to which a wave takes a row

struct JoinK {
    int32_t rows, c;
    float eps;
    const void* h;
    const void* gate;
    const void* res;
    const float* post;
    const float* scale;
    const float* pre;
    void* joined;
    void* normed;
    const void* gjoined;
    const void* gnormed;
    void* dh;
    void* dgate;
    void* dres;
    float* part;  // [workgroup][3][c]: sums for dpost, dscale, dpre
    int64_t ldh, ldg, ldr, ldj, ldn, ldgj, ldgn, lddh, lddg, lddr;
};

// V columns of a row from `col` < c on.  kAny: the row starts at any element
// (the memory takes 16 bytes at any address) and may end within them (c >= V):
// its last lane loads the row's last V columns instead, and shifts them once
// they are used, zeros behind the end.  16384 bf16 rows of 2305 channels, fp32
// residual, took 133 us forward and 214 backward (2312: 106 and 163), 262 and
// 243 column by column; with a last lane that loads its columns one by one,
// where the whole wave then waits, 146 and 301.
template <bool kAny, int V, typename T>
__device__ __forceinline__ Pack<T, V> ld_cols(const T* p, int col, int c) {
    if constexpr (!kAny) return ld_pack<T, V>(p + col);
    Pack<T, V> r;
    __builtin_memcpy(&r, p + (col + V <= c ? col : c - V), sizeof r);
    return r;
}

// Those columns, widened.
template <bool kAny, int V, typename T>
__device__ __forceinline__ void widen_cols(const Pack<T, V>& r, int col, int c, float (&f)[V]) {
    widen(r, f);
    if constexpr (kAny && V > 1) {
        const int s = col + V - c;
        if (s > 0) {
#pragma unroll
            for (int k = 1; k < V; k *= 2) {
                if (s & k) {
#pragma unroll
                    for (int v = 0; v < V; ++v) f[v] = v + k < V ? f[v + k] : 0.0f;
                }
            }
        }
    }
}

template <bool kAny, int V, typename T>
__device__ __forceinline__ void st_cols(T* p, int col, int c, const float (&f)[V]) {
    if constexpr (!kAny) {
        st_pack<T, V>(p + col, f);
    } else {
        Pack<T, V> r;
        st_pack<T, V>(&r.e[0], f);
        if (col + V <= c) {
            __builtin_memcpy(p + col, &r, sizeof r);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (col + v < c) p[col + v] = r.e[v];
        }
    }
}

// How a row lies on the lanes.  kWave: one wave a row, four rows a block;
// otherwise the whole block, as many waves as the row fills, up to MAXT lanes.
template <bool kWave, int MAXT>
struct Row {
    static __device__ __forceinline__ int lanes() { return kWave ? 64 : static_cast<int>(blockDim.x); }
    static __device__ __forceinline__ int lane() {
        return kWave ? static_cast<int>(threadIdx.x & 63) : static_cast<int>(threadIdx.x);
    }
    static __device__ __forceinline__ int per_block() { return kWave ? 4 : 1; }
    static __device__ __forceinline__ int of_block() { return kWave ? static_cast<int>(threadIdx.x >> 6) : 0; }

    // The sums of K values over the lanes of a row, the same bits in each.
    // lds: two buffers taken in turn, so that one barrier a sum is enough.
    template <int K>
    static __device__ __forceinline__ void sums(float (&v)[K], float (*lds)[MAXT / 64][3], int* turn) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
        if constexpr (!kWave) {
            float (*const buf)[3] = lds[*turn];
            *turn ^= 1;
            if ((threadIdx.x & 63) == 0) {
#pragma unroll
                for (int k = 0; k < K; ++k) buf[threadIdx.x >> 6][k] = v[k];
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] = 0.0f;
            for (int w = 0; w < static_cast<int>(blockDim.x >> 6); ++w)
#pragma unroll
                for (int k = 0; k < K; ++k) v[k] += buf[w][k];
        }
    }
};

// 1 / rms of a row from its sum of squares (hardware root, 1 ulp).
__device__ __forceinline__ float rnorm(float ss, float c, float eps) {
    return __builtin_amdgcn_rsqf(__builtin_fmaf(ss, 1.0f / c, eps));
}

template <typename T, typename RT, int V, int NV, bool kWave, int MAXT, bool kAny>
__global__ __launch_bounds__(kWave ? 256 : MAXT) void join_fwd_kernel(const JoinK p) {
    typedef Row<kWave, MAXT> L;
    __shared__ float lds[2][MAXT / 64][3];
    int turn = 0;
    const int TPR = L::lanes();
    const int lane = L::lane();
    const float cf = static_cast<float>(p.c);
    // one row, unless there are more than a grid holds
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * L::per_block() + L::of_block(); row < p.rows;
         row += static_cast<int64_t>(gridDim.x) * L::per_block()) {
        float e[NV][V], o[NV][V];
        Pack<T, V> h[NV], g[NV];
        Pack<RT, V> r[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
            h[i] = Pack<T, V>{};
            if (col < p.c) {
                h[i] = ld_cols<kAny, V>(static_cast<const T*>(p.h) + row * p.ldh, col, p.c);
                if (p.gate) g[i] = ld_cols<kAny, V>(static_cast<const T*>(p.gate) + row * p.ldg, col, p.c);
                if (p.res) r[i] = ld_cols<kAny, V>(static_cast<const RT*>(p.res) + row * p.ldr, col, p.c);
            }
        }
        float ss[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
            widen_cols<kAny>(h[i], col, p.c, e[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) ss[0] = __builtin_fmaf(e[i][v], e[i][v], ss[0]);
        }
        float r1 = 1.0f;
        if (p.post) {
            L::template sums<1>(ss, lds, &turn);
            r1 = rnorm(ss[0], cf, p.eps);
        }
        ss[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
            if (col < p.c) {
                float w[V];
                if (p.post) {
                    widen_cols<kAny>(ld_cols<kAny, V>(p.post, col, p.c), col, p.c, w);
#pragma unroll
                    for (int v = 0; v < V; ++v) e[i][v] *= r1 * w[v];
                }
                if (p.gate) {
                    widen_cols<kAny>(g[i], col, p.c, w);
#pragma unroll
                    for (int v = 0; v < V; ++v) e[i][v] *= w[v] * gate_sigmoid<float>(w[v]);
                }
                if (p.scale) {
                    widen_cols<kAny>(ld_cols<kAny, V>(p.scale, col, p.c), col, p.c, w);
#pragma unroll
                    for (int v = 0; v < V; ++v) e[i][v] *= w[v];
                }
                if (p.res) {
                    widen_cols<kAny>(r[i], col, p.c, w);
#pragma unroll
                    for (int v = 0; v < V; ++v) e[i][v] += w[v];
                }
                st_cols<kAny, V>(static_cast<RT*>(p.joined) + row * p.ldj, col, p.c, e[i]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                RT s;  // the norm is that of the rows as they are stored
                Store<RT>::st(&s, e[i][v]);
                o[i][v] = Store<RT>::ld(&s);
                if (col < p.c) ss[0] = __builtin_fmaf(o[i][v], o[i][v], ss[0]);
            }
        }
        if (!p.pre) continue;
        L::template sums<1>(ss, lds, &turn);
        const float r2 = rnorm(ss[0], cf, p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
            if (col < p.c) {
                float w[V];
                widen_cols<kAny>(ld_cols<kAny, V>(p.pre, col, p.c), col, p.c, w);
#pragma unroll
                for (int v = 0; v < V; ++v) w[v] *= o[i][v] * r2;
                st_cols<kAny, V>(static_cast<T*>(p.normed) + row * p.ldn, col, p.c, w);
            }
        }
    }
}

// With o = joined, gw = gnormed pre: do = gjoined + r2 (gw - o r2^2 mean(gw o));
// then back through the residual, scale, gate and the first norm.
// kAhead, for up to eight channels a lane: the row stays in registers and the
// next row's loads are in flight while it is computed (its two sums over the
// row leave no other work between).  Otherwise each phase reads the row again,
// from the caches: held, 16 channels a lane spilled and took three times the
// time that the memory needs.
template <typename T, typename RT, int V, int NV, bool kWave, int MAXT, bool kAhead, bool kAny>
__global__ __launch_bounds__(kWave ? 256 : MAXT) void join_bwd_kernel(const JoinK p) {
    typedef Row<kWave, MAXT> L;
    __shared__ float lds[2][MAXT / 64][3];
    int turn = 0;
    const int TPR = L::lanes();
    const int lane = L::lane();
    const int worker = static_cast<int>(blockIdx.x) * L::per_block() + L::of_block();
    const int workers = static_cast<int>(gridDim.x) * L::per_block();
    const float cf = static_cast<float>(p.c);
    const float inv = 1.0f / cf;
    float sp[NV][V], sc[NV][V], sn[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) sp[i][v] = sc[i][v] = sn[i][v] = 0.0f;

    // The parameters of a lane's columns, held over the rows where there is
    // room: loaded at each row's turn they were three waits a row.
    constexpr bool kHold = kAhead;
    float wpost[NV][V], wscale[NV][V], wpre[NV][V];
    auto param = [&](const float* q, int i, float (&w)[V]) {
        const int col = (i * TPR + lane) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] = 1.0f;
        if (q && col < p.c) widen_cols<kAny>(ld_cols<kAny, V>(q, col, p.c), col, p.c, w);
    };
    if (kHold) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            param(p.post, i, wpost[i]);
            param(p.scale, i, wscale[i]);
            param(p.pre, i, wpre[i]);
        }
    }
    Pack<T, V> hp[NV], gp[NV], np[NV], hq[NV], gq[NV], nq[NV];
    Pack<RT, V> op[NV], jp[NV], oq[NV], jq[NV];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
            if (col < p.c) {
                hq[i] = ld_cols<kAny, V>(static_cast<const T*>(p.h) + row * p.ldh, col, p.c);
                if (p.gate) gq[i] = ld_cols<kAny, V>(static_cast<const T*>(p.gate) + row * p.ldg, col, p.c);
                if (p.gjoined) jq[i] = ld_cols<kAny, V>(static_cast<const RT*>(p.gjoined) + row * p.ldgj, col, p.c);
                if (p.pre) {
                    oq[i] = ld_cols<kAny, V>(static_cast<const RT*>(p.joined) + row * p.ldj, col, p.c);
                    nq[i] = ld_cols<kAny, V>(static_cast<const T*>(p.gnormed) + row * p.ldgn, col, p.c);
                }
            }
        }
    };
    if (kAhead && worker < p.rows) load(worker);
    for (int64_t row = worker; row < p.rows; row += workers) {
        if (kAhead) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                hp[i] = hq[i];
                gp[i] = gq[i];
                np[i] = nq[i];
                op[i] = oq[i];
                jp[i] = jq[i];
            }
            if (row + workers < p.rows) load(row + workers);
        }
        auto get = [&](const auto& held, const void* q, int64_t ld, int i, float (&f)[V]) {
            typedef std::remove_const_t<std::remove_reference_t<decltype(held.e[0])>> E;
            const int col = (i * TPR + lane) * V;
            if constexpr (kAhead) widen_cols<kAny>(held, col, p.c, f);
            else widen_cols<kAny>(ld_cols<kAny, V>(static_cast<const E*>(q) + row * ld, col, p.c), col, p.c, f);
        };
        float go[NV][V];
        float sum[3] = {0.0f, 0.0f, 0.0f};  // of h^2, o^2 and gw o
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
#pragma unroll
            for (int v = 0; v < V; ++v) go[i][v] = 0.0f;
            if (col < p.c) {
                float h[V];
                get(hp[i], p.h, p.ldh, i, h);
                if (p.gjoined) get(jp[i], p.gjoined, p.ldgj, i, go[i]);
#pragma unroll
                for (int v = 0; v < V; ++v) sum[0] = __builtin_fmaf(h[v], h[v], sum[0]);
                if (p.pre) {
                    float o[V], n[V];
                    get(op[i], p.joined, p.ldj, i, o);
                    get(np[i], p.gnormed, p.ldgn, i, n);
                    if (!kHold) param(p.pre, i, wpre[i]);
                    const float (&w)[V] = wpre[i];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        sum[1] = __builtin_fmaf(o[v], o[v], sum[1]);
                        sum[2] = __builtin_fmaf(n[v] * w[v], o[v], sum[2]);
                    }
                }
            }
        }
        if (p.pre || p.post) L::template sums<3>(sum, lds, &turn);
        const float r1 = p.post ? rnorm(sum[0], cf, p.eps) : 1.0f;
        if (p.pre) {
            const float r2 = rnorm(sum[1], cf, p.eps);
            const float k = r2 * r2 * sum[2] * inv;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int col = (i * TPR + lane) * V;
                if (col < p.c) {
                    float o[V], n[V];
                    get(op[i], p.joined, p.ldj, i, o);
                    get(np[i], p.gnormed, p.ldgn, i, n);
                    if (!kHold) param(p.pre, i, wpre[i]);
                    const float (&w)[V] = wpre[i];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        go[i][v] = __builtin_fmaf(r2, __builtin_fmaf(-o[v], k, n[v] * w[v]), go[i][v]);
                        sn[i][v] = __builtin_fmaf(n[v], o[v] * r2, sn[i][v]);
                    }
                }
            }
        }
        float dot[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
            if (col < p.c) {
                if (p.dres) st_cols<kAny, V>(static_cast<RT*>(p.dres) + row * p.lddr, col, p.c, go[i]);
                float h[V], q[V], a[V], gv[V], dg[V];
                get(hp[i], p.h, p.ldh, i, h);
                if (!kHold) {
                    param(p.post, i, wpost[i]);
                    param(p.scale, i, wscale[i]);
                }
                const float (&w)[V] = wpost[i];
                const float (&s)[V] = wscale[i];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    a[v] = 1.0f;
                    q[v] = h[v] * (r1 * w[v]);
                }
                if (p.gate) {
                    get(gp[i], p.gate, p.ldg, i, gv);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float sg = gate_sigmoid<float>(gv[v]);
                        a[v] = gv[v] * sg;
                        dg[v] = silu_grad(gv[v], sg);
                    }
                }
                if (p.scale) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        sc[i][v] = __builtin_fmaf(go[i][v], q[v] * a[v], sc[i][v]);
                        go[i][v] *= s[v];
                    }
                }
                if (p.gate && p.dgate) {
#pragma unroll
                    for (int v = 0; v < V; ++v) dg[v] *= go[i][v] * q[v];
                    st_cols<kAny, V>(static_cast<T*>(p.dgate) + row * p.lddg, col, p.c, dg);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    go[i][v] *= a[v];  // dL/dq
                    if (p.post) {
                        sp[i][v] = __builtin_fmaf(go[i][v], h[v] * r1, sp[i][v]);
                        go[i][v] *= w[v];
                        dot[0] = __builtin_fmaf(go[i][v], h[v], dot[0]);
                    }
                }
            }
        }
        if (!p.dh) continue;
        float k = 0.0f;
        if (p.post) {
            L::template sums<1>(dot, lds, &turn);
            k = r1 * r1 * dot[0] * inv;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
            if (col < p.c) {
                float h[V];
                get(hp[i], p.h, p.ldh, i, h);
#pragma unroll
                for (int v = 0; v < V; ++v)  // without the norm h has no part in it, whatever it holds
                    if (p.post) go[i][v] = r1 * __builtin_fmaf(-h[v], k, go[i][v]);
                st_cols<kAny, V>(static_cast<T*>(p.dh) + row * p.lddh, col, p.c, go[i]);
            }
        }
    }
    if (!p.part) return;
    if constexpr (kWave) {  // the block's four waves leave one partial row
        __shared__ float all[4][3][kWaveRow];
        float (*const mine)[kWaveRow] = all[L::of_block()];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int col = (i * TPR + lane) * V + v;
                mine[0][col] = sp[i][v];
                mine[1][col] = sc[i][v];
                mine[2][col] = sn[i][v];
            }
        }
        __syncthreads();
        float* const part = p.part + static_cast<int64_t>(blockIdx.x) * 3 * p.c;
        for (int e = threadIdx.x; e < 3 * static_cast<int>(kWaveRow); e += 256) {
            const int plane = e / static_cast<int>(kWaveRow), col = e % static_cast<int>(kWaveRow);
            if (col < p.c)
                part[plane * p.c + col] =
                    (all[0][plane][col] + all[1][plane][col]) + (all[2][plane][col] + all[3][plane][col]);
        }
    } else {
        float* const part = p.part + static_cast<int64_t>(worker) * 3 * p.c;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
            if (col < p.c) {
                st_cols<kAny, V>(part, col, p.c, sp[i]);
                st_cols<kAny, V>(part + p.c, col, p.c, sc[i]);
                st_cols<kAny, V>(part + 2 * static_cast<int64_t>(p.c), col, p.c, sn[i]);
            }
        }
    }
}

JoinK join_params(const gspn_join_args& a) {
    JoinK k{};
    k.rows = static_cast<int32_t>(a.rows);
    k.c = static_cast<int32_t>(a.c);
    k.eps = static_cast<float>(a.eps);
    k.h = a.h;
    k.gate = a.gate;
    k.res = a.residual;
    k.post = a.post;
    k.scale = a.scale;
    k.pre = a.pre;
    k.joined = a.joined;
    k.normed = a.normed;
    k.gjoined = a.gjoined;
    k.gnormed = a.gnormed;
    k.dh = a.dh;
    k.dgate = a.dgate;
    k.dres = a.dresidual;
    k.ldh = a.ldh;
    k.ldg = a.ldgate;
    k.ldr = a.ldres;
    k.ldj = a.ldjoined;
    k.ldn = a.ldnormed;
    k.ldgj = a.ldgjoined;
    k.ldgn = a.ldgnormed;
    k.lddh = a.lddh;
    k.lddg = a.lddgate;
    k.lddr = a.lddres;
    return k;
}

// Lanes of a row of c channels, V at a time.
int lanes_for(int64_t c, int v) { return static_cast<int>((c + 64 * v - 1) / (64 * v) * 64); }

// NV values of V channels a lane: as many lanes as the row fills, or all.
template <typename T, typename RT, int V, int NV, bool kWave, int MAXT, bool kAny>
void run_join_fwd(const JoinK& k, int64_t workers, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(kWave ? (workers + 3) / 4 : workers));
    const dim3 block(kWave ? 256 : lanes_for(k.c, V * NV));
    hipLaunchKernelGGL((join_fwd_kernel<T, RT, V, NV, kWave, MAXT, kAny>), grid, block, 0, stream, k);
}

template <typename T, typename RT, int V, int NV, bool kWave, int MAXT, bool kAhead, bool kAny>
void run_join_bwd(const JoinK& k, int64_t workers, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(kWave ? (workers + 3) / 4 : workers));
    const dim3 block(kWave ? 256 : lanes_for(k.c, V * NV));
    hipLaunchKernelGGL((join_bwd_kernel<T, RT, V, NV, kWave, MAXT, kAhead, kAny>), grid, block, 0, stream, k);
}

template <typename T, typename RT, bool kAny>
void run_join_c(bool bwd, const JoinK& k, int64_t workers, hipStream_t stream) {
    if (kAny && k.c < 8) {  // no whole vector to load a row's end from
        if (!bwd) run_join_fwd<T, RT, 1, 1, true, 64, kAny>(k, workers, stream);
        else run_join_bwd<T, RT, 1, 1, true, 64, true, kAny>(k, workers, stream);
    } else if (!bwd) {
        if (k.c <= kWaveRow) run_join_fwd<T, RT, 8, 1, true, 64, kAny>(k, workers, stream);
        // Four columns at a time where they lie anywhere (us against eight): 11107 fp32 rows of 1418 59 and 70, 8192 of
        // 4093 126 and 135, 8192 bf16 rows of 4095 with an fp32 residual 101 and 113, 16384 of 2305 135 and 136; but with
        // a bf16 residual 137 and 123, and 20000 fp32 rows of 515 43 and 42.
        else if (k.c <= 4096) run_join_fwd<T, RT, kAny ? 4 : 8, kAny ? 2 : 1, false, 512, kAny>(k, workers, stream);
        else if (k.c <= 8192) run_join_fwd<T, RT, 8, 1, false, 1024, kAny>(k, workers, stream);
        else run_join_fwd<T, RT, 8, 2, false, 1024, kAny>(k, workers, stream);
    } else {
        if (k.c <= kWaveRow) run_join_bwd<T, RT, 4, 2, true, 64, true, kAny>(k, workers, stream);
        else if (k.c <= 4096) run_join_bwd<T, RT, 4, 1, false, 1024, true, kAny>(k, workers, stream);
        else if (k.c <= 8192) run_join_bwd<T, RT, 8, 1, false, 1024, false, kAny>(k, workers, stream);
        else run_join_bwd<T, RT, 8, 2, false, 1024, false, kAny>(k, workers, stream);
    }
}

template <typename T, typename RT>
void run_join(bool bwd, bool vec, const JoinK& k, int64_t workers, hipStream_t stream) {
    if (vec) run_join_c<T, RT, false>(bwd, k, workers, stream);
    else run_join_c<T, RT, true>(bwd, k, workers, stream);
}

hipError_t launch_join(bool bwd, const gspn_join_args& a, const JoinK& k, int64_t workers, int dtype,
                       hipStream_t stream) {
    const int es = dtype == kF32 ? 4 : 2;
    const int rs = a.residual_dtype == kF32 ? 4 : 2;
    bool vec = a.c % 8 == 0;
    const char* kn = bwd ? "join_bwd_kernel" : "join_fwd_kernel";
    (void)kn;
    auto rows = [&](const char* what, const void* p, int64_t ld, int s) {
        (void)what;
        if (!p) return;
        vec = vec && aligned_rows(p, ld, s, 16);
        GSPN_REPLAY_ROWS(kn, what, p, a.rows, ld, a.c, s);
    };
    rows("h", a.h, a.ldh, es);
    rows("gate", a.gate, a.ldgate, es);
    rows("joined", a.joined, a.ldjoined, rs);
    if (bwd) {
        rows("gjoined", a.gjoined, a.ldgjoined, rs);
        rows("gnormed", a.gnormed, a.ldgnormed, es);
        rows("dh", a.dh, a.lddh, es);
        rows("dgate", a.dgate, a.lddgate, es);
        rows("dresidual", a.dresidual, a.lddres, rs);
        if (k.part) {
            vec = vec && aligned_rows(k.part, a.c, 4, 16);
            GSPN_REPLAY_ROWS(kn, "partial sums", k.part, join_bwd_parts(a.rows, a.c) * 3, a.c, a.c, 4);
        }
    } else {
        rows("residual", a.residual, a.ldres, rs);
        rows("normed", a.normed, a.ldnormed, es);
    }
    for (const float* w : {a.post, a.scale, a.pre}) {
        if (!w) continue;
        vec = vec && aligned_rows(w, 0, 4, 16);
        GSPN_REPLAY_ROWS(kn, "parameter", w, 1, a.c, a.c, 4);
    }
    GSPN_REPLAYED(kn, a.c > kWaveRow ? 1024 : 256, a.c > kWaveRow ? 2 * 16 * 3 * 4 : 4 * 3 * kWaveRow * 4 + 24);
    if (dtype == kF32) run_join<float, float>(bwd, vec, k, workers, stream);
    else if (a.residual_dtype == kF32) run_join<bf16_t, float>(bwd, vec, k, workers, stream);
    else run_join<bf16_t, bf16_t>(bwd, vec, k, workers, stream);
    return hipGetLastError();
}

}  // namespace

// Workers (rows in flight) of the backward: a row each up to a workgroup a CU,
// then up to four rows each, up to what is resident at once (some 20 waves a CU,
// of 256 channels); their partial rows stay a small part of the traffic.  64 rows
// of 8192 channels take 18 us at a row each and 31 at four, 1024 rows of 2304
// 22 and 19.5.  A multiple of the rows a workgroup takes.
int64_t join_bwd_workers(int64_t rows, int64_t c) {
    const int64_t waves = c <= kWaveRow ? 1 : (c + 255) / 256;
    int64_t a_cu = 20 / waves;
    if (a_cu < 1) a_cu = 1;
    const int64_t first = c <= kWaveRow ? 1024 : 256;
    int64_t w = (rows + 3) / 4;
    if (w < first) w = rows < first ? rows : first;
    if (w > 256 * a_cu) w = 256 * a_cu;
    if (w < 1) w = 1;
    return c <= kWaveRow ? (w + 3) / 4 * 4 : w;
}

// Partial rows, one a workgroup.
int64_t join_bwd_parts(int64_t rows, int64_t c) {
    return join_bwd_workers(rows, c) / (c <= kWaveRow ? 4 : 1);
}

hipError_t launch_join_fwd(const gspn_join_args& a, int dtype, hipStream_t stream) {
    const int64_t most = int64_t{1} << 21;  // rows of a grid; beyond, a workgroup takes several
    return launch_join(false, a, join_params(a), a.rows < most ? a.rows : most, dtype, stream);
}

hipError_t launch_join_bwd(const gspn_join_args& a, int dtype, hipStream_t stream) {
    JoinK k = join_params(a);
    const bool sums = a.dpost || a.dscale || a.dpre;
    if (sums) k.part = static_cast<float*>(a.workspace);
    const int64_t workers = join_bwd_workers(a.rows, a.c);
    const hipError_t e = launch_join(true, a, k, workers, dtype, stream);
    if (e != hipSuccess || !sums) return e;
    ReduceK r{};
    r.part = k.part;
    r.parts = join_bwd_parts(a.rows, a.c);
    r.c = a.c;
    r.ld = r.cols = 3 * a.c;
    r.o[0] = {a.dpost, 1, 1, 0};
    r.o[1] = {a.dscale, 1, 1, 0};
    r.o[2] = {a.dpre, 1, 1, 0};
    return launch_reduce_parts(r, OutsideK{}, stream);
}

}  // namespace gspn
