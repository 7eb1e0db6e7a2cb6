// head_rotary.hip -- each head's queries and keys normalised and rotated by
// their positions in one pass, and the gradients.
//
// Bound by the bytes of q and k.  A head lies on the lanes of a group, V pairs
// (2 V elements) a lane: for pairs of halves V elements at j and V at pairs + j,
// for neighbours 2 V in a row; elements behind the pairs are dealt out the same
// way and turn by nothing.  A lane keeps its pairs' sines and cosines for all the
// heads of a row.
#include "attention.hpp"

namespace gspn {
namespace {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryWaves = kRotaryThreads / 64;
constexpr int64_t kRotaryBlocks = 1 << 16;

struct RotaryK {
    int32_t rows, heads, kv_heads, d, pairs, axes, interleaved;
    int32_t upto[GSPN_ROTARY_MAX_AXES];  // the end of each axis' pairs
    int32_t slices;                      // waves that share a row's heads
    float eps;
    const void* q;
    const void* k;
    const float* qw;
    const float* kw;
    const int32_t* pos;
    const double* freqs;
    void* q_out;  // the backward's dq, dk
    void* k_out;
    const void* gq;
    const void* gk;
    float* part;  // [workgroup][2][d]
    int64_t ldq, ldk, ldpos, ldqo, ldko, ldgq, ldgk;
};


// sin and cos of 2 pi t for a 64-bit t: reduced to an eighth of a turn either
// way, then the first terms of their series (the next are below 2^-28).
__device__ __forceinline__ void sincos_turn(double t, float* s, float* c) {
    t -= __builtin_rint(t);
    const double quarter = __builtin_rint(4.0 * t);
    const float x = static_cast<float>(t - 0.25 * quarter) * 6.28318530717958647692f;
    const float y = x * x;
    float a = __builtin_fmaf(y, 2.75573192e-6f, -1.98412698e-4f);  // 1/9!, -1/7!
    a = __builtin_fmaf(a, y, 8.33333333e-3f);                      // 1/5!
    a = __builtin_fmaf(a, y, -1.66666667e-1f);                     // -1/3!
    a = __builtin_fmaf(a * y, x, x);
    float b = __builtin_fmaf(y, -2.75573192e-7f, 2.48015873e-5f);  // -1/10!, 1/8!
    b = __builtin_fmaf(b, y, -1.38888889e-3f);                     // -1/6!
    b = __builtin_fmaf(b, y, 4.16666667e-2f);                      // 1/4!
    b = __builtin_fmaf(b, y, -0.5f);
    b = __builtin_fmaf(b, y, 1.0f);
    const int n = static_cast<int>(quarter) & 3;
    const float u = n & 1 ? b : a, v = n & 1 ? a : b;
    *s = n & 2 ? -u : u;
    *c = (n == 1 || n == 2) ? -v : v;
}

// V elements from p on, `left` of them in range (the others 0).
template <typename T, int V>
__device__ __forceinline__ void ld_some(const T* p, int left, float (&f)[V]) {
    if (left >= V) {
        Pack<T, V> v;
        __builtin_memcpy(&v, p, sizeof v);
        widen<T, V>(v, f);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = i < left ? Store<T>::ld(p + i) : 0.0f;
    }
}

template <typename T, int V>
__device__ __forceinline__ void st_some(T* p, int left, const float (&f)[V]) {
    if (left >= V) {
        Pack<T, V> v;
        st_pack<T, V>(&v.e[0], f);
        __builtin_memcpy(p, &v, sizeof v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < left) Store<T>::st(p + i, f[i]);
    }
}

// A lane's place in a head: its pairs (a[i], b[i]) begin at these elements, of
// which na, nb are in range.
struct Place {
    int a, b, na, nb;
    bool turns;
};

template <int V>
__device__ __forceinline__ Place place_of(const RotaryK& k, int unit) {
    const int turning = (k.pairs + V - 1) / V;
    Place p;
    p.turns = unit < turning;
    if (p.turns) {
        const int j = unit * V;
        p.na = k.pairs - j < V ? k.pairs - j : V;
        p.nb = p.na;
        p.a = k.interleaved ? 2 * j : j;
        p.b = k.interleaved ? 2 * j + V : k.pairs + j;
    } else {
        p.a = 2 * k.pairs + (unit - turning) * 2 * V;
        p.b = p.a + V;
        p.na = k.d - p.a;
        p.nb = k.d - p.b;
        p.na = p.na < 0 ? 0 : p.na < V ? p.na : V;
        p.nb = p.nb < 0 ? 0 : p.nb < V ? p.nb : V;
    }
    return p;
}

// The 2 V elements of a place as pairs.  Interleaved pairs are 2 V in a row.
template <typename T, int V>
__device__ __forceinline__ void ld_pairs(const RotaryK& k, const Place& p, const T* head, float (&a)[V], float (&b)[V]) {
    if (p.turns && k.interleaved) {
        float f[2 * V];
        ld_some<T, 2 * V>(head + p.a, 2 * p.na, f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            a[i] = f[2 * i];
            b[i] = f[2 * i + 1];
        }
    } else {
        ld_some<T, V>(head + p.a, p.na, a);
        ld_some<T, V>(head + p.b, p.nb, b);
    }
}

template <typename T, int V>
__device__ __forceinline__ void st_pairs(const RotaryK& k, const Place& p, T* head, const float (&a)[V],
                                         const float (&b)[V]) {
    if (p.turns && k.interleaved) {
        float f[2 * V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f[2 * i] = a[i];
            f[2 * i + 1] = b[i];
        }
        st_some<T, 2 * V>(head + p.a, 2 * p.na, f);
    } else {
        st_some<T, V>(head + p.a, p.na, a);
        st_some<T, V>(head + p.b, p.nb, b);
    }
}

// The sum over the G lanes of a group, in each of them.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
    if constexpr (G >= 2) v += dpp<0xB1>(v);
    if constexpr (G >= 4) v += dpp<0x4E>(v);
    if constexpr (G >= 8) v += dpp<0x141>(v);   // rows of 16 mirrored by halves: quads swapped
    if constexpr (G >= 16) v += dpp<0x128>(v);  // rotated by 8
    if constexpr (G >= 32) v = swap_add16(v, v);
    if constexpr (G >= 64) v = swap_add32(v, v);
    return v;
}

template <int V>
__device__ __forceinline__ void turns_of(const RotaryK& k, const Place& p, int unit, int64_t row, float (&s)[V],
                                         float (&c)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s[i] = 0.0f;
        c[i] = 1.0f;
        const int j = unit * V + i;
        if (p.turns && i < p.na) {
            int axis = 0;
#pragma unroll
            for (int x = 0; x < GSPN_ROTARY_MAX_AXES - 1; ++x) axis += x + 1 < k.axes && j >= k.upto[x];
            const double t = static_cast<double>(k.pos[row * k.ldpos + axis]) * k.freqs[j];
            sincos_turn(t * 0.15915494309189533577, &s[i], &c[i]);
        }
    }
}

template <typename T, int V, int G>
__global__ __launch_bounds__(kRotaryThreads) void rotary_fwd_kernel(const RotaryK k) {
    const int lane = threadIdx.x & 63, unit = lane % G;
    const Place p = place_of<V>(k, unit);
    const int total = k.heads + k.kv_heads;
    const int64_t waves = static_cast<int64_t>(gridDim.x) * kRotaryWaves;
    for (int64_t id = static_cast<int64_t>(blockIdx.x) * kRotaryWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
         id < static_cast<int64_t>(k.rows) * k.slices; id += waves) {
    const int64_t row = id / k.slices;
    const int slice = static_cast<int>(id - row * k.slices);
    float s[V], c[V];
    turns_of<V>(k, p, unit, row, s, c);
    for (int h = slice * (64 / G) + lane / G; h < total; h += k.slices * (64 / G)) {
        const bool key = h >= k.heads;
        const int hh = key ? h - k.heads : h;
        const T* const x = static_cast<const T*>(key ? k.k : k.q) + row * (key ? k.ldk : k.ldq) + hh * k.d;
        T* const y = static_cast<T*>(key ? k.k_out : k.q_out) + row * (key ? k.ldko : k.ldqo) + hh * k.d;
        const float* const w = key ? k.kw : k.qw;
        float a[V], b[V];
        ld_pairs<T, V>(k, p, x, a, b);
        if (w) {
            float u[V], v[V], sum = 0.0f;
            ld_pairs<float, V>(k, p, w, u, v);
#pragma unroll
            for (int i = 0; i < V; ++i) sum = __builtin_fmaf(a[i], a[i], __builtin_fmaf(b[i], b[i], sum));
            const float r = 1.0f / __builtin_sqrtf(group_sum<G>(sum) / static_cast<float>(k.d) + k.eps);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                a[i] *= r * u[i];
                b[i] *= r * v[i];
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float t = a[i];
            if (p.turns) {
                a[i] = t * c[i] - b[i] * s[i];
                b[i] = t * s[i] + b[i] * c[i];
            }
        }
        st_pairs<T, V>(k, p, y, a, b);
    }
    }
}

// g turned back is the gradient of the normalised head; with n = x r,
// r = 1 / rms(x): dweight = sum g n, dx = r (g w - n mean(g w n)).
template <typename T, int V, int G>
__global__ __launch_bounds__(kRotaryThreads) void rotary_bwd_kernel(const RotaryK k) {
    __shared__ float sums[kRotaryWaves][64][4 * V];
    const int lane = threadIdx.x & 63, unit = lane % G, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place p = place_of<V>(k, unit);
    const int total = k.heads + k.kv_heads;
    float wa[2][V], wb[2][V];  // gradients of the weights
#pragma unroll
    for (int i = 0; i < V; ++i) wa[0][i] = wb[0][i] = wa[1][i] = wb[1][i] = 0.0f;
    const int64_t waves = static_cast<int64_t>(gridDim.x) * kRotaryWaves;
    for (int64_t id = static_cast<int64_t>(blockIdx.x) * kRotaryWaves + wave; id < static_cast<int64_t>(k.rows) * k.slices;
         id += waves) {
        const int64_t row = id / k.slices;
        const int slice = static_cast<int>(id - row * k.slices);
        float s[V], c[V];
        turns_of<V>(k, p, unit, row, s, c);
        for (int h = slice * (64 / G) + lane / G; h < total; h += k.slices * (64 / G)) {
            const bool key = h >= k.heads;
            const int hh = key ? h - k.heads : h;
            const T* const g = static_cast<const T*>(key ? k.gk : k.gq) + row * (key ? k.ldgk : k.ldgq) + hh * k.d;
            T* const dx = static_cast<T*>(key ? k.k_out : k.q_out) + row * (key ? k.ldko : k.ldqo) + hh * k.d;
            const float* const w = key ? k.kw : k.qw;
            float ga[V], gb[V];
            ld_pairs<T, V>(k, p, g, ga, gb);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float t = ga[i];
                if (p.turns) {
                    ga[i] = t * c[i] + gb[i] * s[i];
                    gb[i] = gb[i] * c[i] - t * s[i];
                }
            }
            if (w) {
                const T* const x = static_cast<const T*>(key ? k.k : k.q) + row * (key ? k.ldk : k.ldq) + hh * k.d;
                float a[V], b[V], u[V], v[V], sum = 0.0f, dot = 0.0f;
                ld_pairs<T, V>(k, p, x, a, b);
                ld_pairs<float, V>(k, p, w, u, v);
#pragma unroll
                for (int i = 0; i < V; ++i) sum = __builtin_fmaf(a[i], a[i], __builtin_fmaf(b[i], b[i], sum));
                const float r = 1.0f / __builtin_sqrtf(group_sum<G>(sum) / static_cast<float>(k.d) + k.eps);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    a[i] *= r;
                    b[i] *= r;
                    wa[0][i] += key ? 0.0f : ga[i] * a[i];
                    wb[0][i] += key ? 0.0f : gb[i] * b[i];
                    wa[1][i] += key ? ga[i] * a[i] : 0.0f;
                    wb[1][i] += key ? gb[i] * b[i] : 0.0f;
                    ga[i] *= u[i];
                    gb[i] *= v[i];
                    dot = __builtin_fmaf(ga[i], a[i], __builtin_fmaf(gb[i], b[i], dot));
                }
                dot = group_sum<G>(dot) / static_cast<float>(k.d);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    ga[i] = r * (ga[i] - a[i] * dot);
                    gb[i] = r * (gb[i] - b[i] * dot);
                }
            }
            st_pairs<T, V>(k, p, dx, ga, gb);
        }
    }
    if (!k.part) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        sums[wave][lane][i] = wa[0][i];
        sums[wave][lane][V + i] = wb[0][i];
        sums[wave][lane][2 * V + i] = wa[1][i];
        sums[wave][lane][3 * V + i] = wb[1][i];
    }
    __syncthreads();
    // one lane a unit and value, over the groups and waves in order
    for (int at = threadIdx.x; at < G * 4 * V; at += kRotaryThreads) {
        const int u = at / (4 * V), i = at % (4 * V);
        float t = 0.0f;
        for (int w = 0; w < kRotaryWaves; ++w)
            for (int g = 0; g < 64 / G; ++g) t += sums[w][g * G + u][i];
        const Place z = place_of<V>(k, u);
        const int e = i % V;
        const bool second = i / V % 2;
        if (e >= (second ? z.nb : z.na)) continue;
        const int col = z.turns && k.interleaved ? z.a + 2 * e + second : (second ? z.b : z.a) + e;
        k.part[(static_cast<int64_t>(blockIdx.x) * 2 + i / (2 * V)) * k.d + col] = t;
    }
}


RotaryK make_rotary(const gspn_rotary_args& a) {
    RotaryK k = {};
    k.rows = static_cast<int32_t>(a.rows);
    k.heads = static_cast<int32_t>(a.heads);
    k.kv_heads = static_cast<int32_t>(a.kv_heads);
    k.d = static_cast<int32_t>(a.d);
    k.pairs = static_cast<int32_t>(a.pairs);
    k.axes = static_cast<int32_t>(a.axes);
    k.interleaved = a.interleaved != 0;
    int32_t at = 0;
    for (int i = 0; i < k.axes; ++i) k.upto[i] = at += static_cast<int32_t>(a.section[i]);
    k.eps = static_cast<float>(a.eps);
    k.q = a.q;
    k.k = a.k;
    k.qw = a.q_weight;
    k.kw = a.k_weight;
    k.pos = a.positions;
    k.freqs = a.freqs;
    k.ldq = a.ldq;
    k.ldk = a.ldk;
    k.ldpos = a.ldpos;
    return k;
}

// Waves that share a row's heads, so that few rows still fill the SIMDs.
int slices_for(int64_t rows, int64_t heads, int group) {
    const int64_t most = (heads + 64 / group - 1) / (64 / group);
    const int64_t want = rows < 1 ? 1 : (2048 + rows - 1) / rows;
    return static_cast<int>(want < most ? want : most);
}

// Calls f with the storage type, the pairs a lane takes (16 bytes of them) and
// the lanes of a head.
template <typename F>
void rotary_dispatch(int dtype, const RotaryK& k, F&& f) {
    const auto lanes = [&](auto t, auto v) {
        constexpr int V = decltype(v)::value;
        const int units = (k.pairs + V - 1) / V + (k.d - 2 * k.pairs + 2 * V - 1) / (2 * V);
        if (units <= 8)
            f(t, v, std::integral_constant<int, 8>{});
        else if (units <= 16)
            f(t, v, std::integral_constant<int, 16>{});
        else if (units <= 32)
            f(t, v, std::integral_constant<int, 32>{});
        else
            f(t, v, std::integral_constant<int, 64>{});
    };
    if (dtype == GSPN_F32)
        lanes(float{}, std::integral_constant<int, 4>{});
    else
        lanes(bf16_t{}, std::integral_constant<int, 8>{});
}

void replay(const char* kn, const gspn_rotary_args& a, bool bwd, int64_t es) {
    (void)kn;
    (void)a;
    (void)es;
    (void)bwd;
    const int64_t cq = a.heads * a.d, ck = a.kv_heads * a.d;
    (void)cq;
    (void)ck;
    if (!bwd || a.q_weight) GSPN_REPLAY_ROWS(kn, "q", a.q, a.rows, a.ldq, cq, es);
    if (!bwd || a.k_weight) GSPN_REPLAY_ROWS(kn, "k", a.k, a.rows, a.ldk, ck, es);
    GSPN_REPLAY_ROWS(kn, "positions", a.positions, a.rows, a.ldpos, a.axes, 4);
    GSPN_REPLAY_ROWS(kn, "freqs", a.freqs, 1, a.pairs, a.pairs, 8);
    GSPN_REPLAY_ROWS(kn, "q_weight", a.q_weight, 1, a.d, a.d, 4);
    GSPN_REPLAY_ROWS(kn, "k_weight", a.k_weight, 1, a.d, a.d, 4);
}

}  // namespace

// Workgroups that walk the rows of a backward: four a CU, each with a wave for
// at least one row.
int64_t rotary_bwd_parts(int64_t rows) {
    const int64_t n = (rows + kRotaryWaves - 1) / kRotaryWaves;
    return n < 1 ? 1 : n < 1024 ? n : 1024;
}

hipError_t launch_rotary_fwd(const gspn_rotary_args& a, int dtype, hipStream_t stream) {
    RotaryK k = make_rotary(a);
    k.q_out = a.q_out;
    k.k_out = a.k_out;
    k.ldqo = a.ldqo;
    k.ldko = a.ldko;
    const int64_t es = dtype == GSPN_F32 ? 4 : 2;
    replay("rotary_fwd_kernel", a, false, es);
    GSPN_REPLAY_ROWS("rotary_fwd_kernel", "q_out", a.q_out, a.rows, a.ldqo, a.heads * a.d, es);
    GSPN_REPLAY_ROWS("rotary_fwd_kernel", "k_out", a.k_out, a.rows, a.ldko, a.kv_heads * a.d, es);
    rotary_dispatch(dtype, k, [&](auto t, auto v, auto g) {
        using T = decltype(t);
        constexpr int V = decltype(v)::value, G = decltype(g)::value;
        k.slices = slices_for(a.rows, a.heads + a.kv_heads, G);
        const int64_t blocks = (a.rows * k.slices + kRotaryWaves - 1) / kRotaryWaves;
        const dim3 grid(static_cast<unsigned>(blocks < kRotaryBlocks ? blocks : kRotaryBlocks));
        GSPN_REPLAYED("rotary_fwd_kernel", kRotaryThreads, 0);
        hipLaunchKernelGGL((rotary_fwd_kernel<T, V, G>), grid, dim3(kRotaryThreads), 0, stream, k);
    });
    return hipGetLastError();
}

hipError_t launch_rotary_bwd(const gspn_rotary_args& a, int dtype, hipStream_t stream) {
    RotaryK k = make_rotary(a);
    k.q_out = a.dq;
    k.k_out = a.dk;
    k.ldqo = a.lddq;
    k.ldko = a.lddk;
    k.gq = a.gq;
    k.gk = a.gk;
    k.ldgq = a.ldgq;
    k.ldgk = a.ldgk;
    const bool sums = a.dq_weight || a.dk_weight;
    k.part = sums ? static_cast<float*>(a.workspace) : nullptr;
    const int64_t es = dtype == GSPN_F32 ? 4 : 2, parts = rotary_bwd_parts(a.rows);
    if (a.rows > 0) {
        replay("rotary_bwd_kernel", a, true, es);
        GSPN_REPLAY_ROWS("rotary_bwd_kernel", "gq", a.gq, a.rows, a.ldgq, a.heads * a.d, es);
        GSPN_REPLAY_ROWS("rotary_bwd_kernel", "dq", a.dq, a.rows, a.lddq, a.heads * a.d, es);
        GSPN_REPLAY_ROWS("rotary_bwd_kernel", "gk", a.gk, a.rows, a.ldgk, a.kv_heads * a.d, es);
        GSPN_REPLAY_ROWS("rotary_bwd_kernel", "dk", a.dk, a.rows, a.lddk, a.kv_heads * a.d, es);
        if (sums) GSPN_REPLAY_ROWS("rotary_bwd_kernel", "partial sums", a.workspace, parts, 2 * a.d, 2 * a.d, 4);
        rotary_dispatch(dtype, k, [&](auto t, auto v, auto g) {
            using T = decltype(t);
            constexpr int V = decltype(v)::value, G = decltype(g)::value;
            k.slices = slices_for(a.rows, a.heads + a.kv_heads, G);
            GSPN_REPLAYED("rotary_bwd_kernel", kRotaryThreads, kRotaryThreads * 4 * V * 4);
            hipLaunchKernelGGL((rotary_bwd_kernel<T, V, G>), dim3(static_cast<unsigned>(parts)), dim3(kRotaryThreads), 0,
                               stream, k);
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!sums) return hipSuccess;
    ReduceK r = {};
    r.part = k.part;
    r.parts = a.rows > 0 ? parts : 0;
    r.ld = r.cols = 2 * a.d;
    r.c = a.d;
    r.o[0] = {a.dq_weight, 1, 1, 0};
    r.o[1] = {a.dk_weight, 1, 1, 0};
    return launch_reduce_parts(r, OutsideK{}, stream);
}

}  // namespace gspn
