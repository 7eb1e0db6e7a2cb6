// head_rotary.hip -- each head's queries and keys normalised and rotated by
// their positions in one pass, and the gradients.
//
// Bound by the bytes of q and k.  A head lies on the lanes of a group, V pairs
// (2 V elements) a lane: for pairs of halves V elements at j and V at pairs + j,
// for neighbours 2 V in a row; elements behind the pairs are dealt out the same
// way and turn by nothing.  A lane keeps its pairs' sines and cosines for all the
// heads of a row.  16384 rows of 40 heads of 128 bf16 elements: 71 us, 4700 GB/s, 91%
// of what a copy reaches; 12544 rows of 32 heads of 72, interleaved: 26 us forward,
// 4400 GB/s, 41 backward, 4250.
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
// way, an angle that is rounded once (in 64 bits up to here: a product in fp32 would
// leave 1.26 2^-24 of it, not 2^-25), then the first terms of their series (the next are
// below 2^-28).
__device__ __forceinline__ void sincos_turn(double t, float* s, float* c) {
    t -= __builtin_rint(t);
    const double quarter = __builtin_rint(4.0 * t);
    const float x = static_cast<float>((t - 0.25 * quarter) * 6.28318530717958647692);
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

// A lane's place in a head: V pairs (a[i], b[i]), their elements from these on, or
// 2 V elements in a row behind the pairs (as a, then b, or as neighbours where
// pairs are).  Where units do not come out even (kEven: they do), the last of
// either kind ends where its kind does and so begins within the one before: its
// first `skip` values are that one's too, count for nothing in sums, and are
// stored twice, the same bits; where there are not V of a kind, `left` are in range.
struct Place {
    int a, b, skip, left;
    bool turns, idle;
};

template <int V, bool kInter, bool kEven>
__device__ __forceinline__ Place place_of(const RotaryK& k, int unit) {
    const int turning = (k.pairs + V - 1) / V;
    Place p;
    p.turns = unit < turning;
    const int all = p.turns ? k.pairs : k.d - 2 * k.pairs;  // of its kind: pairs, or elements
    const int each = p.turns ? V : 2 * V;
    const int first = (p.turns ? unit : unit - turning) * each;
    p.idle = first >= all;
    int at = first;
    p.skip = 0;
    p.left = each;
    if (!kEven && !p.idle && first + each > all) {
        if (all >= each) {
            at = all - each;
            p.skip = first - at;
        } else {
            p.left = all;
        }
    }
    if (p.turns) {
        p.a = kInter ? 2 * at : at;
        p.b = kInter ? 2 * at + V : k.pairs + at;
    } else {
        p.a = 2 * k.pairs + at;
        p.b = p.a + V;
    }
    return p;
}

// Which of a place's values are its own, in range and not another unit's too.
template <int V, bool kInter, bool kEven>
__device__ __forceinline__ bool own_a(const Place& p, int i) {
    const int j = p.turns || !kInter ? i : 2 * i;
    return kEven || (j >= p.skip && j < p.left);
}
template <int V, bool kInter, bool kEven>
__device__ __forceinline__ bool own_b(const Place& p, int i) {
    const int j = p.turns ? i : kInter ? 2 * i + 1 : V + i;
    return kEven || (j >= p.skip && j < p.left);
}

// The values of a place on their way; 0 where it is idle or out of range.
template <typename T, int V>
struct Raw {
    Pack<T, V> a, b;
};

template <typename T, int V, bool kInter, bool kEven>
__device__ __forceinline__ Raw<T, V> ld_raw(const Place& p, const T* head) {
    Raw<T, V> r = {};
    if (p.idle) return r;
    if (kEven || p.left >= (p.turns ? V : 2 * V)) {
        __builtin_memcpy(&r.a, head + p.a, sizeof r.a);
        __builtin_memcpy(&r.b, head + p.b, sizeof r.b);
    } else {
        // interleaved pairs are 2 V elements in a row, as elements behind the pairs are
        const bool row = !p.turns || kInter;
        const int n = p.turns && kInter ? 2 * p.left : p.left;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i < n) r.a.e[i] = head[p.a + i];
            if ((row ? V + i : i) < n) r.b.e[i] = head[p.b + i];
        }
    }
    return r;
}

template <typename T, int V, bool kInter>
__device__ __forceinline__ void pairs_of(const Raw<T, V>& r, float (&a)[V], float (&b)[V]) {
    widen<T, V>(r.a, a);
    widen<T, V>(r.b, b);
    if constexpr (kInter) {
        float f[2 * V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f[i] = a[i];
            f[V + i] = b[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            a[i] = f[2 * i];
            b[i] = f[2 * i + 1];
        }
    }
}

template <typename T, int V, bool kInter, bool kEven>
__device__ __forceinline__ void st_pairs(const Place& p, T* head, float (&a)[V], float (&b)[V]) {
    if constexpr (kInter) {
        float f[2 * V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f[2 * i] = a[i];
            f[2 * i + 1] = b[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            a[i] = f[i];
            b[i] = f[V + i];
        }
    }
    if (p.idle) return;
    if (kEven || p.left >= (p.turns ? V : 2 * V)) {
        Pack<T, V> v;
        st_pack<T, V>(&v.e[0], a);
        __builtin_memcpy(head + p.a, &v, sizeof v);
        st_pack<T, V>(&v.e[0], b);
        __builtin_memcpy(head + p.b, &v, sizeof v);
    } else {
        const bool row = !p.turns || kInter;
        const int n = p.turns && kInter ? 2 * p.left : p.left;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i < n) Store<T>::st(head + p.a + i, a[i]);
            if ((row ? V + i : i) < n) Store<T>::st(head + p.b + i, b[i]);
        }
    }
}

// A weight's values at a place, for queries or keys; loaded anew only where a
// group of lanes goes from the ones to the others.
template <int V>
struct Weight {
    float u[V], v[V];
    int of = -1;
    template <bool kInter, bool kEven>
    __device__ __forceinline__ void load(const Place& p, const float* w, bool key) {
        if (of == key) return;
        of = key;
        pairs_of<float, V, kInter>(ld_raw<float, V, kInter, kEven>(p, w), u, v);
    }
};

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

// Sines and cosines of a row's pairs: a pair a lane, then to where they are
// wanted through the wave's own LDS (each lane forming its V of them was half of
// the whole forward's time).
constexpr int kMaxPairs = GSPN_ROTARY_MAX_HEAD / 2;

template <int V, bool kInter>
__device__ __forceinline__ void turns_of(const RotaryK& k, const Place& p, int64_t row, float (*table)[kMaxPairs],
                                         float (&s)[V], float (&c)[V]) {
    const int lane = threadIdx.x & 63;
    for (int j = lane; j < k.pairs; j += 64) {
        int axis = 0;
#pragma unroll
        for (int x = 0; x < GSPN_ROTARY_MAX_AXES - 1; ++x) axis += x + 1 < k.axes && j >= k.upto[x];
        const double t = static_cast<double>(k.pos[row * k.ldpos + axis]) * k.freqs[j];
        sincos_turn(t * 0.15915494309189533577, &table[0][j], &table[1][j]);
    }
    __builtin_amdgcn_wave_barrier();
    const int at = kInter ? p.a / 2 : p.a;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const bool in = p.turns && i < p.left;
        s[i] = in ? table[0][at + i] : 0.0f;
        c[i] = in ? table[1][at + i] : 1.0f;
    }
    __builtin_amdgcn_wave_barrier();
}

// The heads of a row that a group of lanes takes, queries first.
struct HeadAt {
    bool key;
    int head;
    int64_t in;  // elements into its tensor's row
};

__device__ __forceinline__ HeadAt head_at(const RotaryK& k, int h) {
    HeadAt w;
    w.key = h >= k.heads;
    w.head = w.key ? h - k.heads : h;
    w.in = static_cast<int64_t>(w.head) * k.d;
    return w;
}

template <typename T, int V, int G, bool kInter, bool kEven>
__global__ __launch_bounds__(kRotaryThreads) void rotary_fwd_kernel(const RotaryK k) {
    __shared__ float table[kRotaryWaves][2][kMaxPairs];
    const int lane = threadIdx.x & 63, unit = lane % G, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place p = place_of<V, kInter, kEven>(k, unit);
    const int total = k.heads + k.kv_heads, step = k.slices * (64 / G);
    Weight<V> wt;
    const int64_t waves = static_cast<int64_t>(gridDim.x) * kRotaryWaves;
    for (int64_t id = static_cast<int64_t>(blockIdx.x) * kRotaryWaves + wave; id < static_cast<int64_t>(k.rows) * k.slices;
         id += waves) {
        const int64_t row = id / k.slices;
        int h = static_cast<int>(id - row * k.slices) * (64 / G) + lane / G;
        const auto load = [&](int at) {
            const HeadAt w = head_at(k, at);
            return ld_raw<T, V, kInter, kEven>(p, static_cast<const T*>(w.key ? k.k : k.q) + row * (w.key ? k.ldk : k.ldq) + w.in);
        };
        // two heads are on their way while one is worked on
        Raw<T, V> x, next;
        if (h < total) x = load(h);
        if (h + step < total) next = load(h + step);
        float s[V], c[V];
        turns_of<V, kInter>(k, p, row, table[wave], s, c);
        for (; h < total; h += step) {
            const HeadAt w = head_at(k, h);
            float a[V], b[V];
            pairs_of<T, V, kInter>(x, a, b);
            x = next;
            if (h + 2 * step < total) next = load(h + 2 * step);
            const float* const weight = w.key ? k.kw : k.qw;
            if (weight) {
                float sum = 0.0f;
                wt.template load<kInter, kEven>(p, weight, w.key);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    sum = __builtin_fmaf(own_a<V, kInter, kEven>(p, i) ? a[i] : 0.0f, a[i], sum);
                    sum = __builtin_fmaf(own_b<V, kInter, kEven>(p, i) ? b[i] : 0.0f, b[i], sum);
                }
                const float r = 1.0f / __builtin_sqrtf(group_sum<G>(sum) / static_cast<float>(k.d) + k.eps);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    a[i] *= r * wt.u[i];
                    b[i] *= r * wt.v[i];
                }
            }
            if (p.turns) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float t = a[i];
                    a[i] = t * c[i] - b[i] * s[i];
                    b[i] = t * s[i] + b[i] * c[i];
                }
            }
            st_pairs<T, V, kInter, kEven>(p, static_cast<T*>(w.key ? k.k_out : k.q_out) + row * (w.key ? k.ldko : k.ldqo) + w.in, a, b);
        }
    }
}

// g turned back is the gradient of the normalised head; with n = x r,
// r = 1 / rms(x): dweight = sum g n, dx = r (g w - n mean(g w n)).
template <typename T, int V, int G, bool kInter, bool kEven>
__global__ __launch_bounds__(kRotaryThreads) void rotary_bwd_kernel(const RotaryK k) {
    __shared__ float lds[kRotaryWaves][64 * 4 * V];
    static_assert(64 * 4 * V >= 2 * kMaxPairs);
    const int lane = threadIdx.x & 63, unit = lane % G, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float(*const table)[kMaxPairs] = reinterpret_cast<float(*)[kMaxPairs]>(lds[wave]);
    const Place p = place_of<V, kInter, kEven>(k, unit);
    const int total = k.heads + k.kv_heads, step = k.slices * (64 / G);
    float wa[2][V], wb[2][V];  // gradients of the weights
#pragma unroll
    for (int i = 0; i < V; ++i) wa[0][i] = wb[0][i] = wa[1][i] = wb[1][i] = 0.0f;
    Weight<V> wt;
    const int64_t waves = static_cast<int64_t>(gridDim.x) * kRotaryWaves;
    for (int64_t id = static_cast<int64_t>(blockIdx.x) * kRotaryWaves + wave; id < static_cast<int64_t>(k.rows) * k.slices;
         id += waves) {
        const int64_t row = id / k.slices;
        int h = static_cast<int>(id - row * k.slices) * (64 / G) + lane / G;
        struct Both {
            Raw<T, V> g, x;
        };
        const auto load = [&](int at) {
            const HeadAt w = head_at(k, at);
            Both r;
            r.g = ld_raw<T, V, kInter, kEven>(p, static_cast<const T*>(w.key ? k.gk : k.gq) + row * (w.key ? k.ldgk : k.ldgq) + w.in);
            if (w.key ? k.kw : k.qw)
                r.x = ld_raw<T, V, kInter, kEven>(p, static_cast<const T*>(w.key ? k.k : k.q) + row * (w.key ? k.ldk : k.ldq) + w.in);
            return r;
        };
        Both now, next;
        if (h < total) now = load(h);
        if (h + step < total) next = load(h + step);
        float s[V], c[V];
        turns_of<V, kInter>(k, p, row, table, s, c);
        for (; h < total; h += step) {
            const HeadAt w = head_at(k, h);
            const float* const weight = w.key ? k.kw : k.qw;
            float ga[V], gb[V], a[V], b[V];
            pairs_of<T, V, kInter>(now.g, ga, gb);
            if (weight) pairs_of<T, V, kInter>(now.x, a, b);
            now = next;
            if (h + 2 * step < total) next = load(h + 2 * step);
            if (p.turns) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float t = ga[i];
                    ga[i] = t * c[i] + gb[i] * s[i];
                    gb[i] = gb[i] * c[i] - t * s[i];
                }
            }
            if (weight) {
                float sum = 0.0f, dot = 0.0f;
                wt.template load<kInter, kEven>(p, weight, w.key);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    sum = __builtin_fmaf(own_a<V, kInter, kEven>(p, i) ? a[i] : 0.0f, a[i], sum);
                    sum = __builtin_fmaf(own_b<V, kInter, kEven>(p, i) ? b[i] : 0.0f, b[i], sum);
                }
                const float r = 1.0f / __builtin_sqrtf(group_sum<G>(sum) / static_cast<float>(k.d) + k.eps);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    a[i] *= r;
                    b[i] *= r;
                    const float x = ga[i] * a[i], y = gb[i] * b[i];
                    wa[0][i] += w.key ? 0.0f : x;
                    wb[0][i] += w.key ? 0.0f : y;
                    wa[1][i] += w.key ? x : 0.0f;
                    wb[1][i] += w.key ? y : 0.0f;
                    ga[i] *= wt.u[i];
                    gb[i] *= wt.v[i];
                    dot = __builtin_fmaf(own_a<V, kInter, kEven>(p, i) ? ga[i] : 0.0f, a[i], dot);
                    dot = __builtin_fmaf(own_b<V, kInter, kEven>(p, i) ? gb[i] : 0.0f, b[i], dot);
                }
                dot = group_sum<G>(dot) / static_cast<float>(k.d);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    ga[i] = r * (ga[i] - a[i] * dot);
                    gb[i] = r * (gb[i] - b[i] * dot);
                }
            }
            st_pairs<T, V, kInter, kEven>(p, static_cast<T*>(w.key ? k.k_out : k.q_out) + row * (w.key ? k.ldko : k.ldqo) + w.in, ga,
                           gb);
        }
    }
    if (!k.part) return;
    __syncthreads();
    float(*const sums)[4 * V] = reinterpret_cast<float(*)[4 * V]>(lds[wave]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        sums[lane][i] = wa[0][i];
        sums[lane][V + i] = wb[0][i];
        sums[lane][2 * V + i] = wa[1][i];
        sums[lane][3 * V + i] = wb[1][i];
    }
    __syncthreads();
    // one lane a unit and value, over the groups and waves in order
    for (int at = threadIdx.x; at < G * 4 * V; at += kRotaryThreads) {
        const int u = at / (4 * V), i = at % (4 * V), e = i % V;
        const bool second = i / V % 2;
        const Place z = place_of<V, kInter, kEven>(k, u);
        if (z.idle || !(second ? own_b<V, kInter, kEven>(z, e) : own_a<V, kInter, kEven>(z, e))) continue;
        float t = 0.0f;
        for (int w = 0; w < kRotaryWaves; ++w)
            for (int g = 0; g < 64 / G; ++g) t += reinterpret_cast<float(*)[4 * V]>(lds[w])[g * G + u][i];
        const int col = kInter ? z.a + 2 * e + second : (second ? z.b : z.a) + e;
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

// Waves that share a row's heads, so that few rows still fill the SIMDs: two a
// SIMD; more would only form a row's sines more often.  A backward's waves leave sums
// of the weights' gradients too: it has no more than those two (2000 rows, 32 + 8 heads
// of 128 bf16 elements: 19.7 us with one slice, 25.6 with two; 500 rows 17.6 with a
// workgroup for every four rows, 12.1 with four slices, 64 rows 15.6 and 8.9).
int64_t most_slices(int64_t rows, bool bwd) {
    const int64_t n = rows < 1 ? 1 : bwd ? 2048 / rows : (2048 + rows - 1) / rows;
    return n < 1 ? 1 : n;
}

int slices_for(int64_t rows, int64_t heads, int group, bool bwd) {
    const int64_t most = (heads + 64 / group - 1) / (64 / group), want = most_slices(rows, bwd);
    return static_cast<int>(want < most ? want : most);
}

// Calls f with the storage type, the pairs a lane takes, the lanes of a head, and
// the two flags.  A lane takes 16 bytes of pairs, or where they come out even 12 or
// 8, whichever leaves fewest lanes idle (32 heads of 72, forward: 8 bytes on nine
// lanes of 16 33 us, 12 on six of 8 25; of 64: 16 on four of 8 28, 8 on eight 23).
template <typename F>
void rotary_dispatch(int dtype, const RotaryK& k, F&& f) {
    const int rest = k.d - 2 * k.pairs;
    const auto lanes_of = [&](int v) {
        const int units = (k.pairs + v - 1) / v + (rest + 2 * v - 1) / (2 * v);
        return units <= 8 ? 8 : units <= 16 ? 16 : units <= 32 ? 32 : 64;
    };
    const auto flags = [&](auto t, auto v, auto g, auto even) {
        if (k.interleaved)
            f(t, v, g, std::true_type{}, even);
        else
            f(t, v, g, std::false_type{}, even);
    };
    const auto lanes = [&](auto t, auto v, auto even) {
        constexpr int V = decltype(v)::value;
        const int g = lanes_of(V);
        if (g == 8)
            flags(t, v, std::integral_constant<int, 8>{}, even);
        else if (g == 16)
            flags(t, v, std::integral_constant<int, 16>{}, even);
        else if (decltype(even)::value || g == 32)
            flags(t, v, std::integral_constant<int, 32>{}, even);
        else if constexpr (!decltype(even)::value)
            flags(t, v, std::integral_constant<int, 64>{}, even);
    };
    const auto even = [&](int v) { return k.pairs % v == 0 && rest % (2 * v) == 0; };
    if (dtype == GSPN_F32) {
        if (even(4))
            lanes(float{}, std::integral_constant<int, 4>{}, std::true_type{});
        else
            lanes(float{}, std::integral_constant<int, 4>{}, std::false_type{});
        return;
    }
    int best = 0;
    for (const int v : {8, 6, 4})
        if (even(v) && (best == 0 || lanes_of(v) * v < lanes_of(best) * best)) best = v;
    if (best == 8)
        lanes(bf16_t{}, std::integral_constant<int, 8>{}, std::true_type{});
    else if (best == 6)
        lanes(bf16_t{}, std::integral_constant<int, 6>{}, std::true_type{});
    else if (best == 4)
        lanes(bf16_t{}, std::integral_constant<int, 4>{}, std::true_type{});
    else
        lanes(bf16_t{}, std::integral_constant<int, 8>{}, std::false_type{});
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

// Workgroups that walk the rows of a backward: four a CU at most, each wave with at
// least one row's slice of heads.
int64_t rotary_bwd_groups(int64_t rows, int64_t slices) {
    const int64_t n = (rows * slices + kRotaryWaves - 1) / kRotaryWaves;
    return n < 1 ? 1 : n < 1024 ? n : 1024;
}

// Their partial sums, whatever the heads.
int64_t rotary_bwd_parts(int64_t rows) { return rotary_bwd_groups(rows, most_slices(rows, true)); }

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
    rotary_dispatch(dtype, k, [&](auto t, auto v, auto g, auto inter, auto even) {
        using T = decltype(t);
        constexpr int V = decltype(v)::value, G = decltype(g)::value;
        constexpr bool kInter = decltype(inter)::value, kEven = decltype(even)::value;
        k.slices = slices_for(a.rows, a.heads + a.kv_heads, G, false);
        const int64_t blocks = (a.rows * k.slices + kRotaryWaves - 1) / kRotaryWaves;
        const dim3 grid(static_cast<unsigned>(blocks < kRotaryBlocks ? blocks : kRotaryBlocks));
        GSPN_REPLAYED("rotary_fwd_kernel", kRotaryThreads, 0);
        hipLaunchKernelGGL((rotary_fwd_kernel<T, V, G, kInter, kEven>), grid, dim3(kRotaryThreads), 0, stream, k);
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
    const int64_t es = dtype == GSPN_F32 ? 4 : 2;
    int64_t parts = 0;
    if (a.rows > 0) {
        replay("rotary_bwd_kernel", a, true, es);
        GSPN_REPLAY_ROWS("rotary_bwd_kernel", "gq", a.gq, a.rows, a.ldgq, a.heads * a.d, es);
        GSPN_REPLAY_ROWS("rotary_bwd_kernel", "dq", a.dq, a.rows, a.lddq, a.heads * a.d, es);
        GSPN_REPLAY_ROWS("rotary_bwd_kernel", "gk", a.gk, a.rows, a.ldgk, a.kv_heads * a.d, es);
        GSPN_REPLAY_ROWS("rotary_bwd_kernel", "dk", a.dk, a.rows, a.lddk, a.kv_heads * a.d, es);
        rotary_dispatch(dtype, k, [&](auto t, auto v, auto g, auto inter, auto even) {
            using T = decltype(t);
            constexpr int V = decltype(v)::value, G = decltype(g)::value;
            constexpr bool kInter = decltype(inter)::value, kEven = decltype(even)::value;
            k.slices = slices_for(a.rows, a.heads + a.kv_heads, G, true);
            parts = rotary_bwd_groups(a.rows, k.slices);
            if (sums) GSPN_REPLAY_ROWS("rotary_bwd_kernel", "partial sums", a.workspace, parts, 2 * a.d, 2 * a.d, 4);
            GSPN_REPLAYED("rotary_bwd_kernel", kRotaryThreads, kRotaryThreads * 4 * V * 4);
            hipLaunchKernelGGL((rotary_bwd_kernel<T, V, G, kInter, kEven>), dim3(static_cast<unsigned>(parts)), dim3(kRotaryThreads), 0,
                               stream, k);
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!sums) return hipSuccess;
    ReduceK r = {};
    r.part = k.part;
    r.parts = parts;
    r.ld = r.cols = 2 * a.d;
    r.c = a.d;
    r.o[0] = {a.dq_weight, 1, 1, 0};
    r.o[1] = {a.dk_weight, 1, 1, 0};
    return launch_reduce_parts(r, OutsideK{}, stream);
}

}  // namespace gspn
