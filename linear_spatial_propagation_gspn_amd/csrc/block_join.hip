// block_join.hip -- a block's output joined to the residual stream, with the
// norms around it: optional norm, gate, scale and residual, and the norm that
// the next block reads.
//
// Row by row; every tensor is read once and written once, so the kernels are
// bound by those bytes.  A row lives in the registers of the lanes that share
// it: a wave for up to 1024 channels, 256 lanes for up to 4096, 1024 lanes
// above.  The backward keeps the columns' sums for the parameters' gradients
// in registers over all the rows a workgroup walks and leaves one partial row
// each, joined in a fixed order.
#include "sequence.hpp"

namespace gspn {
namespace {

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
    float* part;  // [worker][3][c]: sums for dpost, dscale, dpre
    int64_t ldh, ldg, ldr, ldj, ldn, ldgj, ldgn, lddh, lddg, lddr;
};

// The sums of two values over the TPR lanes of a row, the same bits in each.
template <int TPR>
__device__ __forceinline__ void row_sums(float& a, float& b, float (*lds)[2]) {
#pragma unroll
    for (int m = 32; m; m >>= 1) {
        a += __shfl_xor(a, m);
        b += __shfl_xor(b, m);
    }
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        __syncthreads();  // the last sums have been read
        if ((threadIdx.x & 63) == 0) {
            lds[threadIdx.x >> 6][0] = a;
            lds[threadIdx.x >> 6][1] = b;
        }
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            a += lds[w][0];
            b += lds[w][1];
        }
    }
}

// 1 / rms of a row from its sum of squares (hardware root, 1 ulp).
__device__ __forceinline__ float rnorm(float ss, float c, float eps) {
    return __builtin_amdgcn_rsqf(__builtin_fmaf(ss, 1.0f / c, eps));
}

template <int TPR>
constexpr int threads_for() {
    return TPR > 256 ? TPR : 256;
}

template <typename T, typename RT, int V, int NV, int TPR>
__global__ __launch_bounds__(threads_for<TPR>()) void join_fwd_kernel(const JoinK p) {
    __shared__ float lds[TPR / 64][2];
    constexpr int WPB = threads_for<TPR>() / TPR;
    const int lane = threadIdx.x % TPR;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * WPB + threadIdx.x / TPR;
    if (row >= p.rows) return;  // a whole wave, or the whole block
    const float cf = static_cast<float>(p.c);
    float e[NV][V], o[NV][V];
    Pack<T, V> g[NV];
    Pack<RT, V> r[NV];
    float ss = 0.0f, unused = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + lane) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) e[i][v] = 0.0f;
        if (col < p.c) {
            widen(ld_pack<T, V>(static_cast<const T*>(p.h) + row * p.ldh + col), e[i]);
            if (p.gate) g[i] = ld_pack<T, V>(static_cast<const T*>(p.gate) + row * p.ldg + col);
            if (p.res) r[i] = ld_pack<RT, V>(static_cast<const RT*>(p.res) + row * p.ldr + col);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) ss = __builtin_fmaf(e[i][v], e[i][v], ss);
    }
    float r1 = 1.0f;
    if (p.post) {
        row_sums<TPR>(ss, unused, lds);
        r1 = rnorm(ss, cf, p.eps);
    }
    ss = unused = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + lane) * V;
        if (col < p.c) {
            float w[V];
            if (p.post) {
                widen(ld_pack<float, V>(p.post + col), w);
#pragma unroll
                for (int v = 0; v < V; ++v) e[i][v] *= r1 * w[v];
            }
            if (p.gate) {
                widen(g[i], w);
#pragma unroll
                for (int v = 0; v < V; ++v) e[i][v] *= w[v] * gate_sigmoid<float>(w[v]);
            }
            if (p.scale) {
                widen(ld_pack<float, V>(p.scale + col), w);
#pragma unroll
                for (int v = 0; v < V; ++v) e[i][v] *= w[v];
            }
            if (p.res) {
                widen(r[i], w);
#pragma unroll
                for (int v = 0; v < V; ++v) e[i][v] += w[v];
            }
            st_pack<RT, V>(static_cast<RT*>(p.joined) + row * p.ldj + col, e[i]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            RT s;  // the norm is that of the rows as they are stored
            Store<RT>::st(&s, e[i][v]);
            o[i][v] = Store<RT>::ld(&s);
            if (col < p.c) ss = __builtin_fmaf(o[i][v], o[i][v], ss);
        }
    }
    if (!p.pre) return;
    row_sums<TPR>(ss, unused, lds);
    const float r2 = rnorm(ss, cf, p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + lane) * V;
        if (col < p.c) {
            float w[V];
            widen(ld_pack<float, V>(p.pre + col), w);
#pragma unroll
            for (int v = 0; v < V; ++v) w[v] *= o[i][v] * r2;
            st_pack<T, V>(static_cast<T*>(p.normed) + row * p.ldn + col, w);
        }
    }
}

// With o = joined, gw = gnormed pre: do = gjoined + r2 (gw - o r2^2 mean(gw o));
// then back through the residual, scale, gate and the first norm.
template <typename T, typename RT, int V, int NV, int TPR>
__global__ __launch_bounds__(threads_for<TPR>()) void join_bwd_kernel(const JoinK p) {
    __shared__ float lds[TPR / 64][2];
    constexpr int WPB = threads_for<TPR>() / TPR;
    const int lane = threadIdx.x % TPR;
    const int worker = static_cast<int>(blockIdx.x) * WPB + static_cast<int>(threadIdx.x) / TPR;
    const int workers = static_cast<int>(gridDim.x) * WPB;
    const float cf = static_cast<float>(p.c);
    const float inv = 1.0f / cf;
    float sp[NV][V], sc[NV][V], sn[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) sp[i][v] = sc[i][v] = sn[i][v] = 0.0f;

    for (int64_t row = worker; row < p.rows; row += workers) {
        Pack<T, V> hp[NV], gp[NV], np[NV];
        Pack<RT, V> op[NV], jp[NV];
        float go[NV][V];
        float ss = 0.0f, so = 0.0f, dot = 0.0f, unused = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
            if (col < p.c) {
                hp[i] = ld_pack<T, V>(static_cast<const T*>(p.h) + row * p.ldh + col);
                if (p.gate) gp[i] = ld_pack<T, V>(static_cast<const T*>(p.gate) + row * p.ldg + col);
                if (p.gjoined) jp[i] = ld_pack<RT, V>(static_cast<const RT*>(p.gjoined) + row * p.ldgj + col);
                if (p.pre) {
                    op[i] = ld_pack<RT, V>(static_cast<const RT*>(p.joined) + row * p.ldj + col);
                    np[i] = ld_pack<T, V>(static_cast<const T*>(p.gnormed) + row * p.ldgn + col);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
#pragma unroll
            for (int v = 0; v < V; ++v) go[i][v] = 0.0f;
            if (col < p.c) {
                float h[V];
                widen(hp[i], h);
                if (p.gjoined) widen(jp[i], go[i]);
#pragma unroll
                for (int v = 0; v < V; ++v) ss = __builtin_fmaf(h[v], h[v], ss);
                if (p.pre) {
                    float o[V], n[V], w[V];
                    widen(op[i], o);
                    widen(np[i], n);
                    widen(ld_pack<float, V>(p.pre + col), w);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        so = __builtin_fmaf(o[v], o[v], so);
                        dot = __builtin_fmaf(n[v] * w[v], o[v], dot);
                    }
                }
            }
        }
        float r1 = 1.0f;
        if (p.pre) {
            row_sums<TPR>(so, dot, lds);
            const float r2 = rnorm(so, cf, p.eps);
            const float k = r2 * r2 * dot * inv;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int col = (i * TPR + lane) * V;
                if (col < p.c) {
                    float o[V], n[V], w[V];
                    widen(op[i], o);
                    widen(np[i], n);
                    widen(ld_pack<float, V>(p.pre + col), w);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        go[i][v] = __builtin_fmaf(r2, __builtin_fmaf(-o[v], k, n[v] * w[v]), go[i][v]);
                        sn[i][v] = __builtin_fmaf(n[v], o[v] * r2, sn[i][v]);
                    }
                }
            }
        }
        if (p.post) {
            row_sums<TPR>(ss, unused, lds);
            r1 = rnorm(ss, cf, p.eps);
        }
        dot = unused = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
            if (col < p.c) {
                if (p.dres) st_pack<RT, V>(static_cast<RT*>(p.dres) + row * p.lddr + col, go[i]);
                float h[V], q[V], w[V], a[V], gv[V], dg[V];
                widen(hp[i], h);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    w[v] = 1.0f;
                    a[v] = 1.0f;
                }
                if (p.post) widen(ld_pack<float, V>(p.post + col), w);
#pragma unroll
                for (int v = 0; v < V; ++v) q[v] = h[v] * (r1 * w[v]);
                if (p.gate) {
                    widen(gp[i], gv);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float sg = gate_sigmoid<float>(gv[v]);
                        a[v] = gv[v] * sg;
                        dg[v] = silu_grad(gv[v], sg);
                    }
                }
                if (p.scale) {
                    float s[V];
                    widen(ld_pack<float, V>(p.scale + col), s);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        sc[i][v] = __builtin_fmaf(go[i][v], q[v] * a[v], sc[i][v]);
                        go[i][v] *= s[v];
                    }
                }
                if (p.gate && p.dgate) {
#pragma unroll
                    for (int v = 0; v < V; ++v) dg[v] *= go[i][v] * q[v];
                    st_pack<T, V>(static_cast<T*>(p.dgate) + row * p.lddg + col, dg);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    go[i][v] *= a[v];  // dL/dq
                    if (p.post) {
                        sp[i][v] = __builtin_fmaf(go[i][v], h[v] * r1, sp[i][v]);
                        go[i][v] *= w[v];
                        dot = __builtin_fmaf(go[i][v], h[v], dot);
                    }
                }
            }
        }
        if (!p.dh) continue;
        float k = 0.0f;
        if (p.post) {
            row_sums<TPR>(dot, unused, lds);
            k = r1 * r1 * dot * inv;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + lane) * V;
            if (col < p.c) {
                float h[V];
                widen(hp[i], h);
#pragma unroll
                for (int v = 0; v < V; ++v) go[i][v] = r1 * __builtin_fmaf(-h[v], k, go[i][v]);
                st_pack<T, V>(static_cast<T*>(p.dh) + row * p.lddh + col, go[i]);
            }
        }
    }
    if (!p.part) return;
    float* const part = p.part + static_cast<int64_t>(worker) * 3 * p.c;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + lane) * V;
        if (col < p.c) {
            st_pack<float, V>(part + col, sp[i]);
            st_pack<float, V>(part + p.c + col, sc[i]);
            st_pack<float, V>(part + 2 * static_cast<int64_t>(p.c) + col, sn[i]);
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

// Lanes a row takes (see the top of the file).
int lanes_for(int64_t c) { return c <= 1024 ? 64 : c <= 4096 ? 256 : 1024; }

template <typename T, typename RT, int V, int NV, int TPR>
void run_join(bool bwd, const JoinK& k, int64_t workers, hipStream_t stream) {
    constexpr int th = threads_for<TPR>();
    constexpr int wpb = th / TPR;
    const dim3 grid(static_cast<unsigned>((workers + wpb - 1) / wpb));
    if (bwd) hipLaunchKernelGGL((join_bwd_kernel<T, RT, V, NV, TPR>), grid, dim3(th), 0, stream, k);
    else hipLaunchKernelGGL((join_fwd_kernel<T, RT, V, NV, TPR>), grid, dim3(th), 0, stream, k);
}

template <typename T, typename RT>
void run_join_c(bool bwd, bool vec, const JoinK& k, int64_t workers, hipStream_t stream) {
    if (vec) {
        if (k.c <= 512) run_join<T, RT, 8, 1, 64>(bwd, k, workers, stream);
        else if (k.c <= 1024) run_join<T, RT, 8, 2, 64>(bwd, k, workers, stream);
        else if (k.c <= 2048) run_join<T, RT, 8, 1, 256>(bwd, k, workers, stream);
        else if (k.c <= 4096) run_join<T, RT, 8, 2, 256>(bwd, k, workers, stream);
        else if (k.c <= 8192) run_join<T, RT, 8, 1, 1024>(bwd, k, workers, stream);
        else run_join<T, RT, 8, 2, 1024>(bwd, k, workers, stream);
    } else {
        if (k.c <= 256) run_join<T, RT, 1, 4, 64>(bwd, k, workers, stream);
        else if (k.c <= 1024) run_join<T, RT, 1, 16, 64>(bwd, k, workers, stream);
        else if (k.c <= 4096) run_join<T, RT, 1, 16, 256>(bwd, k, workers, stream);
        else run_join<T, RT, 1, 16, 1024>(bwd, k, workers, stream);
    }
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
            GSPN_REPLAY_ROWS(kn, "partial sums", k.part, workers * 3, a.c, a.c, 4);
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
    GSPN_REPLAYED(kn, a.c > 4096 ? 1024 : 256, lanes_for(a.c) / 64 * 8);
    if (dtype == kF32) run_join_c<float, float>(bwd, vec, k, workers, stream);
    else if (a.residual_dtype == kF32) run_join_c<bf16_t, float>(bwd, vec, k, workers, stream);
    else run_join_c<bf16_t, bf16_t>(bwd, vec, k, workers, stream);
    return hipGetLastError();
}

}  // namespace

// Workers (rows in flight) of the backward: enough to fill the GPU, few
// enough that their partial rows stay a small part of the traffic; a multiple
// of the rows a workgroup takes.
int64_t join_bwd_parts(int64_t rows, int64_t c) {
    const int64_t cap = c <= 1024 ? 4096 : c <= 4096 ? 1024 : 512;
    int64_t w = (rows + 3) / 4;
    if (w > cap) w = cap;
    if (c <= 1024) w = (w + 3) / 4 * 4;
    return w < 1 ? 1 : w;
}

hipError_t launch_join_fwd(const gspn_join_args& a, int dtype, hipStream_t stream) {
    return launch_join(false, a, join_params(a), a.rows, dtype, stream);
}

hipError_t launch_join_bwd(const gspn_join_args& a, int dtype, hipStream_t stream) {
    JoinK k = join_params(a);
    const bool sums = a.dpost || a.dscale || a.dpre;
    if (sums) k.part = static_cast<float*>(a.workspace);
    const int64_t workers = join_bwd_parts(a.rows, a.c);
    const hipError_t e = launch_join(true, a, k, workers, dtype, stream);
    if (e != hipSuccess || !sums) return e;
    ReduceK r{};
    r.part = k.part;
    r.parts = workers;
    r.c = a.c;
    r.ld = r.cols = 3 * a.c;
    r.o[0] = {a.dpost, 1, 1, 0};
    r.o[1] = {a.dscale, 1, 1, 0};
    r.o[2] = {a.dpre, 1, 1, 0};
    return launch_reduce_parts(r, stream);
}

}  // namespace gspn
