// attention_bwd.hip -- gradients of attention.hip's attention.
//
// With p the softmax (formed again from the scores and lse), D_i = <gout_i,
// out_i> and ds_ij = p_ij (<gout_i, v_j> - D_i):
//   dq_i = scale sum_j ds_ij k_j;  dk_j = scale sum_i ds_ij q_i;  dv_j = sum_i p_ij gout_i
// Two kernels, one with the queries at rest (dq, and D for the other), one with
// the keys (dk, dv, over all the heads that share them): the scores are formed
// twice, seven products instead of five, and nothing is added through memory.
//
// D from a bf16 out carries its rounding, as large against ds as one over the
// root of the keys: rows that see one tile of keys or less get theirs from the
// weights, sum_j p_ij <gout_i, v_j>.  A row that sees one key has p = 1 whatever
// the score: its ds is 0, not the rounding that is left of the difference.
#include "attention.hpp"

#include <array>
#include <initializer_list>

namespace gspn {
namespace {

// lse in powers of two; +Inf where there is none, so that every weight is 0.
__device__ __forceinline__ float log2_sum(float lse) {
    return lse == -INFINITY ? INFINITY : lse * 1.44269504088896340736f;
}

template <typename T, int D, bool kDirect>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_dq_kernel(const AttnK a) {
    using Tl = Tile<T, D>;
    constexpr int BN = kTileRows<T>;
    __shared__ __attribute__((aligned(16))) char lds[2][2][BN * Tl::kRow];
    const AttnItem w = find_item(a.seq, a.heads, a.causal != 0, kAttnShift);
    if (w.c.seq < 0 || w.c.r0 >= w.c.r1) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int rows = w.c.end - w.c.begin;
    const Keys keys = find_keys<T>(a, w.c.seq, w.c.begin, rows, w.head / a.group);
    const int off = keys.count - rows;

    const int wave0 = w.c.r0 - w.c.begin + __builtin_amdgcn_readfirstlane(tid >> 6) * 32;
    const int row = wave0 + (lane & 31);
    const bool mine = row < rows;
    const int64_t at = static_cast<int64_t>(w.c.begin) + (mine ? row : 0);
    const int64_t col = static_cast<int64_t>(w.head) * a.d;

    Quad q[Tl::kSteps], g[Tl::kSteps];
    ld_rows<T, D>(static_cast<const T*>(a.q) + at * a.ldq + col, mine, a.d, a.flip, q);
    ld_rows<T, D>(static_cast<const T*>(a.gout) + at * a.ldgo + col, mine, a.d, false, g);
    float delta = 0.0f;
    {
        Quad o[Tl::kSteps];
        ld_rows<T, D>(static_cast<const T*>(a.out) + at * a.ldo + col, mine, a.d, false, o);
#pragma unroll
        for (int i = 0; i < Tl::kSteps; ++i) {
            float x[Tl::kE], y[Tl::kE];
            widen<T, Tl::kE>(__builtin_bit_cast(Pack<T, Tl::kE>, o[i]), x);
            widen<T, Tl::kE>(__builtin_bit_cast(Pack<T, Tl::kE>, g[i]), y);
#pragma unroll
            for (int j = 0; j < Tl::kE; ++j) delta = __builtin_fmaf(x[j], y[j], delta);
        }
        delta = both_sum(delta);
    }
    const int64_t stat = static_cast<int64_t>(w.head) * a.seq.rows + at;
    const float lse2 = log2_sum(a.lse[stat]);

    const auto seen = [&](int r) {
        const int n = a.causal ? r + off + 1 : keys.count;
        return n < 0 ? 0 : n < keys.count ? n : keys.count;
    };
    const int tiles = (seen(w.c.r1 - 1 - w.c.begin) + BN - 1) / BN;
    const int wave_last = wave0 + 31 < rows ? wave0 + 31 : rows - 1;
    const int wave_keys = wave0 < rows ? seen(wave_last) : 0;
    const int wave_all = wave0 < rows ? seen(wave0) : 0;
    const int my_keys = mine ? seen(row) : 0;

    f32x16 dq[D / 32];
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) dq[b][r] = 0.0f;
    Stage<T, D, BN, kAttnThreads, kDirect> sk, sv;
    const T* const kp = static_cast<const T*>(keys.k);
    const T* const vp = static_cast<const T*>(keys.v);
    clear_tiles<kDirect>(tid, kAttnThreads, lds[0][0], sizeof lds, a.d == D);
    if (tiles > 0) {
        sk.fetch(tid, kp, keys.ldk, 0, keys.count - 1, a.d, lds[0][0]);
        sv.fetch(tid, vp, keys.ldv, 0, keys.count - 1, a.d, lds[0][1]);
        sk.commit(tid, lds[0][0]);
        sv.commit(tid, lds[0][1]);
    }
    __syncthreads();
    for (int t = 0; t < tiles; ++t) {
        const bool more = t + 1 < tiles;
        if (more) {
            sk.fetch(tid, kp, keys.ldk, (t + 1) * BN, keys.count - 1, a.d, lds[(t + 1) & 1][0]);
            sv.fetch(tid, vp, keys.ldv, (t + 1) * BN, keys.count - 1, a.d, lds[(t + 1) & 1][1]);
        }
        const int key0 = t * BN;
        if (key0 < wave_keys) {
            const uint32_t kt = Tl::rows_at(lds_at(lds[t & 1][0])), kc = Tl::columns_at(lds_at(lds[t & 1][0]));
            const uint32_t vt = Tl::rows_at(lds_at(lds[t & 1][1]));
            // the weights of 32 keys and their gradients
            const auto weights = [&](int n, f32x16& s, f32x16& dp) {
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
#pragma unroll
                for (int i = 0; i < Tl::kSteps; ++i) {
                    s = mma<T>(Tl::rows(kt, 32 * n, i), q[i], s);
                    dp = mma<T>(Tl::rows(vt, 32 * n, i), g[i], dp);
                }
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], a.scale_log2, -lse2));
                if (key0 + BN > wave_all) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (key0 + 32 * n + result_row(r) >= my_keys) s[r] = dp[r] = 0.0f;
                }
            };
            if (wave_keys <= BN) {
                delta = 0.0f;
#pragma unroll 1
                for (int n = 0; n < BN / 32; ++n) {
                    f32x16 s, dp;
                    weights(n, s, dp);
#pragma unroll
                    for (int r = 0; r < 16; ++r) delta = __builtin_fmaf(s[r], dp[r], delta);
                }
                delta = both_sum(delta);
            }
#pragma unroll
            for (int n = 0; n < BN / 32; ++n) {
                f32x16 s, dp;
                weights(n, s, dp);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] *= dp[r] - delta;
                if (my_keys < 2) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = 0.0f;
                }
                const Factor<T> ds(s);
#pragma unroll
                for (int b = 0; b < D / 32; ++b) dq[b] = Tl::columns(kc, 32 * n, b, ds.p, dq[b]);
            }
        }
        if (more) {
            sk.commit(tid, lds[(t + 1) & 1][0]);
            sv.commit(tid, lds[(t + 1) & 1][1]);
        }
        __syncthreads();
    }
    if (mine) {
        st_result<T, D>(static_cast<T*>(a.dq) + at * a.lddq + col, dq, a.scale, a.d);
        if (lane < 32) a.delta[stat] = delta;
    }
}

// Two waves a SIMD have 256 registers each.  Heads of 128 bf16 elements leave no
// room there for both keys and values beside the gradients': the values stay in
// LDS, and tiles are half as long so that two workgroups still share a CU (held in
// registers they spilled, and every reload waited for the tile on its way: 301 us
// where this takes 190, 8 x 1024 rows, 18 heads, 6 of keys).
template <typename T, int D>
constexpr bool kValuesInLds = kIsBf16<T> && D == 128;
template <typename T, int D>
constexpr int kRowsAtOnce = kValuesInLds<T, D> ? 32 : kTileRows<T>;

template <typename T, int D, bool kDirect>
__global__ __launch_bounds__(kAttnThreads, kIsBf16<T> ? 2 : 1) void attn_dkv_kernel(const AttnK a) {
    using Tl = Tile<T, D>;
    constexpr int BM = kRowsAtOnce<T, D>;
    constexpr bool kHeld = !kValuesInLds<T, D>;  // values in registers
    __shared__ __attribute__((aligned(16))) char lds[2][2][BM * Tl::kRow];
    __shared__ __attribute__((aligned(16))) char values[kHeld ? 16 : kAttnRows * Tl::kRow];
    __shared__ __attribute__((aligned(16))) float stats[2][2][BM];
    const AttnItem w = find_item(a.kv, a.kv_heads, false, kAttnShift);
    if (w.c.seq < 0 || w.c.r0 >= w.c.r1) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int begin = seq_begin(a.seq, w.c.seq);
    const int rows = seq_end(a.seq, w.c.seq, begin) - begin;
    const int count = w.c.end - w.c.begin;
    const int off = count - rows;

    const int key0 = w.c.r0 - w.c.begin;
    const int wave0 = key0 + __builtin_amdgcn_readfirstlane(tid >> 6) * 32;
    const int key = wave0 + (lane & 31);
    const bool mine = key < count;
    const int64_t at = static_cast<int64_t>(w.c.begin) + (mine ? key : 0);
    const int64_t col = static_cast<int64_t>(w.head) * a.d;

    Quad k[Tl::kSteps], v[kHeld ? Tl::kSteps : 1];
    ld_rows<T, D>(static_cast<const T*>(a.k) + at * a.ldk + col, mine, a.d, a.flip, k);
    if constexpr (kHeld) {
        ld_rows<T, D>(static_cast<const T*>(a.v) + at * a.ldv + col, mine, a.d, false, v);
    } else {
        Stage<T, D, kAttnRows, kAttnThreads, false> sv;
        sv.fetch(tid, static_cast<const T*>(a.v) + w.c.begin * a.ldv + col, a.ldv, key0, count - 1, a.d, values);
        sv.commit(tid, values);
    }
    const uint32_t vt = Tl::rows_at(lds_at(values)) + (wave0 - key0) * Tl::kRow;

    // tiles of rows from the first that sees a key of the workgroup
    const int row0 = !a.causal || key0 - off < 0 ? 0 : key0 - off;
    const int t0 = row0 / BM;
    const int each = row0 < rows ? (rows + BM - 1) / BM - t0 : 0;
    const int tiles = each * a.group;

    f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) dk[b][r] = dv[b][r] = 0.0f;

    Stage<T, D, BM, kAttnThreads, kDirect> sq, sg;
    float stat = 0.0f;
    const auto fetch = [&](int head, int tile, int buf) {
        const int64_t c = static_cast<int64_t>(w.head * a.group + head) * a.d;
        sq.fetch(tid, static_cast<const T*>(a.q) + begin * a.ldq + c, a.ldq, tile * BM, rows - 1, a.d, lds[buf][0]);
        sg.fetch(tid, static_cast<const T*>(a.gout) + begin * a.ldgo + c, a.ldgo, tile * BM, rows - 1, a.d, lds[buf][1]);
        if (tid < 2 * BM) {
            const int r = tile * BM + tid % BM;
            const int64_t i = static_cast<int64_t>(w.head * a.group + head) * a.seq.rows + begin + (r < rows ? r : rows - 1);
            stat = tid < BM ? log2_sum(a.lse[i]) : a.delta[i];
        }
    };
    const auto commit = [&](int buf) {
        sq.commit(tid, lds[buf][0]);
        sg.commit(tid, lds[buf][1]);
        if (tid < 2 * BM) stats[buf][tid / BM][tid % BM] = stat;
    };
    clear_tiles<kDirect>(tid, kAttnThreads, lds[0][0], sizeof lds, a.d == D);
    const int lo = a.causal ? key - off : 0;   // rows lo .. rows - 1 see this lane's key
    const int alone = count == 1 ? 0 : -off;   // the row that sees one key (with one key, every row)
    if (tiles > 0) {
        fetch(0, t0, 0);
        commit(0);
    }
    __syncthreads();
    int head = 0, tile = t0;
    for (int t = 0; t < tiles; ++t) {
        const bool more = t + 1 < tiles;
        const int r0 = tile * BM;
        if (++tile == t0 + each) {
            tile = t0;
            ++head;
        }
        if (more) fetch(head, tile, (t + 1) & 1);
        if (wave0 < count && (!a.causal || wave0 <= r0 + BM - 1 + off)) {
            const uint32_t qt = Tl::rows_at(lds_at(lds[t & 1][0])), qc = Tl::columns_at(lds_at(lds[t & 1][0]));
            const uint32_t gt = Tl::rows_at(lds_at(lds[t & 1][1])), gc = Tl::columns_at(lds_at(lds[t & 1][1]));
            const bool hides = r0 + BM > rows || (a.causal && wave0 + 31 > r0 + off);
            const bool lone = count == 1 || (a.causal && alone >= r0 && alone < r0 + BM);
            // (the barriers keep the compiler from fetching fragments of the next
            // product early: their registers would not be there)
#pragma unroll
            for (int n = 0; n < BM / 32; ++n) {
                f32x16 s, dp;
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
#pragma unroll
                for (int i = 0; i < Tl::kSteps; ++i) s = mma<T>(Tl::rows(qt, 32 * n, i), k[i], s);
                if (hides) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int i = r0 + 32 * n + result_row(r);
                        s[r] = i >= lo && i < rows ? s[r] : -INFINITY;
                    }
                }
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 lse2 = *reinterpret_cast<const f32x4*>(&stats[t & 1][0][32 * n + result_row(4 * g)]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[4 * g + j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[4 * g + j], a.scale_log2, -lse2[j]));
                }
                __builtin_amdgcn_sched_barrier(0);
                {
                    const Factor<T> p(s);
#pragma unroll
                    for (int b = 0; b < D / 32; ++b) dv[b] = Tl::columns(gc, 32 * n, b, p.p, dv[b]);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < Tl::kSteps; ++i) dp = mma<T>(Tl::rows(gt, 32 * n, i), kHeld ? v[kHeld ? i : 0] : Tl::rows(vt, 0, i), dp);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 delta = *reinterpret_cast<const f32x4*>(&stats[t & 1][1][32 * n + result_row(4 * g)]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[4 * g + j] *= dp[4 * g + j] - delta[j];
                }
                if (lone) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (count == 1 || r0 + 32 * n + result_row(r) == alone) s[r] = 0.0f;
                }
                __builtin_amdgcn_sched_barrier(0);
                {
                    const Factor<T> ds(s);
#pragma unroll
                    for (int b = 0; b < D / 32; ++b) dk[b] = Tl::columns(qc, 32 * n, b, ds.p, dk[b]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (more) commit((t + 1) & 1);
        __syncthreads();
    }
    if (mine) {
        st_result<T, D>(static_cast<T*>(a.dk) + at * a.lddk + col, dk, a.scale, a.d);
        st_result<T, D>(static_cast<T*>(a.dv) + at * a.lddv + col, dv, 1.0f, a.d);
    }
}

// Zeros in the rows outside the sequences of s (all: in every row).
hipError_t clear_rows(const SeqK& s, bool all, int es, std::initializer_list<std::array<int64_t, 3>> tensors,
                      hipStream_t stream) {
    if (s.rows == 0 || (!s.cu && !all)) return hipSuccess;
    OutsideK o = {};
    o.seq = s;
    o.es = es;
    o.all = all;
    int i = 0;
    for (const auto& t : tensors) {
        o.t[i].p = reinterpret_cast<void*>(t[0]);
        o.t[i].ld = t[1];
        o.t[i++].c = t[2];
    }
    ReduceK none = {};
    none.c = 1;
    return launch_reduce_parts(none, o, stream);
}

}  // namespace

hipError_t launch_attn_bwd(const gspn_attn_args& a, int dtype, hipStream_t stream) {
    AttnK k = make_attn(a);
    k.delta = static_cast<float*>(a.workspace);
    const int es = dtype == GSPN_F32 ? 4 : 2;
    const bool all = a.seq.nseq == 0;
    const int64_t cq = a.heads * a.d, ck = a.kv_heads * a.d;
    const auto address = [](void* p) { return static_cast<int64_t>(reinterpret_cast<intptr_t>(p)); };
    hipError_t e = clear_rows(k.seq, all, es, {{address(a.dq), a.lddq, cq}}, stream);
    if (e != hipSuccess) return e;
    e = clear_rows(k.kv, all, es, {{address(a.dk), a.lddk, ck}, {address(a.dv), a.lddv, ck}}, stream);
    if (e != hipSuccess || all) return e;
    const auto replay = [&](const char* kn) {
        (void)kn;
        GSPN_REPLAY_ROWS(kn, "q", a.q, a.seq.rows, a.ldq, cq, es);
        GSPN_REPLAY_ROWS(kn, "gout", a.gout, a.seq.rows, a.ldgo, cq, es);
        GSPN_REPLAY_ROWS(kn, "k", a.k, a.kv_rows, a.ldk, ck, es);
        GSPN_REPLAY_ROWS(kn, "v", a.v, a.kv_rows, a.ldv, ck, es);
        GSPN_REPLAY_ROWS(kn, "lse", a.lse, a.heads, a.seq.rows, a.seq.rows, 4);
        GSPN_REPLAY_ROWS(kn, "row sums", a.workspace, a.heads, a.seq.rows, a.seq.rows, 4);
    };
    if (a.seq.rows > 0) {
        const dim3 grid(static_cast<unsigned>(
            chunk_ids(a.seq.cu != nullptr, a.seq.rows, a.seq.nseq, kAttnShift) * a.heads));
        const bool direct = attn_direct(a.k, a.ldk, a.d, es) && attn_direct(a.v, a.ldv, a.d, es);
        replay("attn_dq_kernel");
        GSPN_REPLAY_ROWS("attn_dq_kernel", "out", a.out, a.seq.rows, a.ldo, cq, es);
        GSPN_REPLAY_ROWS("attn_dq_kernel", "dq", a.dq, a.seq.rows, a.lddq, cq, es);
        attn_dispatch(dtype, a.d, direct, [&](auto t, auto width, auto straight) {
            using T = decltype(t);
            constexpr int D = decltype(width)::value;
            constexpr bool kDirect = decltype(straight)::value;
            GSPN_REPLAYED("attn_dq_kernel", kAttnThreads, 4 * kTileRows<T> * D * static_cast<int64_t>(sizeof(T)));
            hipLaunchKernelGGL((attn_dq_kernel<T, D, kDirect>), grid, dim3(kAttnThreads), 0, stream, k);
        });
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.kv_rows > 0) {
        const dim3 grid(static_cast<unsigned>(chunk_ids(k.kv.cu != nullptr, a.kv_rows, a.seq.nseq, kAttnShift) *
                                              a.kv_heads));
        const bool direct = attn_direct(a.q, a.ldq, a.d, es) && attn_direct(a.gout, a.ldgo, a.d, es);
        replay("attn_dkv_kernel");
        GSPN_REPLAY_ROWS("attn_dkv_kernel", "dk", a.dk, a.kv_rows, a.lddk, ck, es);
        GSPN_REPLAY_ROWS("attn_dkv_kernel", "dv", a.dv, a.kv_rows, a.lddv, ck, es);
        attn_dispatch(dtype, a.d, direct, [&](auto t, auto width, auto straight) {
            using T = decltype(t);
            constexpr int D = decltype(width)::value;
            constexpr bool kDirect = decltype(straight)::value;
            GSPN_REPLAYED("attn_dkv_kernel", kAttnThreads,
                          kRowsAtOnce<T, D> * (4 * D * static_cast<int64_t>(sizeof(T)) + 16) +
                              (kValuesInLds<T, D> ? kAttnRows * D * static_cast<int64_t>(sizeof(T)) : 16));
            hipLaunchKernelGGL((attn_dkv_kernel<T, D, kDirect>), grid, dim3(kAttnThreads), 0, stream, k);
        });
        e = hipGetLastError();
    }
    return e;
}

}  // namespace gspn
