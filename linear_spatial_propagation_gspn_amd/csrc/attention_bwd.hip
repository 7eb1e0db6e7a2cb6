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
// root of the keys: rows that see one tile of keys or less (64; fp32: 32) get theirs
// from the weights, sum_j p_ij <gout_i, v_j>, whatever the others of their wave see.
// A row that sees one key has p = 1 whatever the score: its ds is 0, not the rounding
// that is left of the difference.  For bf16, p and ds are rounded to bf16 as factors,
// for the forward's reason: a second factor each would take three more products.
#include "attention.hpp"

#include <array>
#include <initializer_list>

namespace gspn {
namespace {

// lse in powers of two; +Inf where there is none, so that every weight is 0.
__device__ __forceinline__ float log2_sum(float lse) {
    return lse == -INFINITY ? INFINITY : lse * 1.44269504088896340736f;
}

// Queries at rest, keys and values in tiles as in the forward.  8 x 1024 rows, 18
// heads, 6 of keys, of 128: 101 us; four maps of 3136 tokens, 16 heads of 72: 360,
// the matrix unit busy in 55% of the cycles.  Products one after the other, as
// the compiler orders them: interleaved by hand as in the forward they took 16%
// longer.
template <typename T, int D, bool kDirect>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_dq_kernel(const AttnK a) {
    using Tl = Tile<T, D>;
    constexpr int BN = kTileRows<T>;
    __shared__ __attribute__((aligned(kTileAlign))) char lds[2][2][BN * Tl::kRow];
    const AttnItem w = find_item(a.seq, a.heads, a.causal != 0, kAttnShift, blockIdx.x);
    if (w.c.seq < 0 || w.c.r0 >= w.c.r1) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int rows = w.c.end - w.c.begin;
    const Keys<T> keys = find_keys<T>(a, w.c.seq, w.c.begin, rows, w.head / a.group);
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

    f32x16 dq[kBlocks<D>];
#pragma unroll
    for (int b = 0; b < kBlocks<D>; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) dq[b][r] = 0.0f;
    Stage<T, D, BN, kAttnThreads, kDirect> sk, sv;
    const T* const kp = keys.k.fresh;
    const T* const vp = keys.v.fresh;
    clear_tiles<kDirect>(tid, kAttnThreads, lds[0][0], sizeof lds, a.d == D);
    if (tiles > 0) {
        sk.fetch(tid, kp, a.ldk, 0, keys.count - 1, a.d, lds[0][0]);
        sv.fetch(tid, vp, a.ldv, 0, keys.count - 1, a.d, lds[0][1]);
        sk.commit(tid, lds[0][0]);
        sv.commit(tid, lds[0][1]);
    }
    __syncthreads();
    // the weights of 32 keys of tile t and their gradients
    const auto weights = [&](int t, int n, f32x16& s, f32x16& dp) {
        const uint32_t kt = Tl::rows_at(lds_at(lds[t & 1][0])), vt = Tl::rows_at(lds_at(lds[t & 1][1]));
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < Tl::kSteps; ++i) {
            if (!Tl::holds(i, a.d)) continue;
            s = mma<T>(Tl::rows(kt, 32 * n, i), q[i], s);
            dp = mma<T>(Tl::rows(vt, 32 * n, i), g[i], dp);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], a.scale_log2, -lse2));
        if ((t + 1) * BN > wave_all) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (t * BN + 32 * n + result_row(r) >= my_keys) s[r] = dp[r] = 0.0f;
        }
    };
    if (wave_keys > 0 && wave_all <= BN) {  // some row's keys are all in the first tile
        float sum = 0.0f;
#pragma unroll 1
        for (int n = 0; n < BN / 32; ++n) {
            f32x16 s, dp;
            weights(0, n, s, dp);
#pragma unroll
            for (int r = 0; r < 16; ++r) sum = __builtin_fmaf(s[r], dp[r], sum);
        }
        sum = both_sum(sum);
        delta = my_keys <= BN ? sum : delta;
    }
    for (int t = 0; t < tiles; ++t) {
        const bool more = t + 1 < tiles;
        if (more) {
            sk.fetch(tid, kp, a.ldk, (t + 1) * BN, keys.count - 1, a.d, lds[(t + 1) & 1][0]);
            sv.fetch(tid, vp, a.ldv, (t + 1) * BN, keys.count - 1, a.d, lds[(t + 1) & 1][1]);
        }
        if (t * BN < wave_keys) {
            const uint32_t kc = Tl::columns_at(lds_at(lds[t & 1][0]));
#pragma unroll
            for (int n = 0; n < BN / 32; ++n) {
                f32x16 s, dp;
                weights(t, n, s, dp);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] *= dp[r] - delta;
                if (my_keys < 2) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = 0.0f;
                }
                const Factor<T> ds(s);
#pragma unroll
                for (int b = 0; b < kBlocks<D>; ++b) dq[b] = Tl::columns(kc, 32 * n, b, ds.p, dq[b]);
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

// Values of a workgroup's keys for the keys' gradients.  Two waves a SIMD have
// 256 registers each: heads of 128 bf16 elements leave no room there for both
// keys and values beside the gradients' sums, and spilled every reload waits for
// the tiles on their way (8 x 1024 rows, 18 heads, 6 of keys, when it was chosen:
// 301 us, 211 with values in LDS).  All but the last
// of the products' steps lie in LDS then, the last in registers, so that two
// workgroups share a CU.  Rows of 240 bytes need no swizzle.
template <typename T, int D>
constexpr bool kValuesInLds = kIsBf16<T> && D == 128;
constexpr int kValueRow = 240;
constexpr int kValueSteps = 7;

// Rows of queries in a tile: 32 for each half of the waves.
constexpr int kBwdRows = 64;

// Keys at rest: two waves of 32 of them, twice, each pair for one half of every
// tile of rows (joined in LDS at the end).  Long walks are half as long so, which
// counts where later rows see more keys: 8 x 1024 rows, 18 heads, 6 of keys, 211
// us with 128 keys a workgroup, 118 so.  Four maps of 3136 tokens,
// 16 heads of 72: 584 us; what bounds both is the matrix unit (busy in 37 and 41%
// of the cycles) behind LDS, which gives two fragments a product.
template <typename T, int D, bool kDirect>
__global__ __launch_bounds__(kAttnThreads, kIsBf16<T> ? 2 : 1) void attn_dkv_kernel(const AttnK a) {
    using Tl = Tile<T, D>;
    constexpr int BM = kBwdRows;
    constexpr bool kInLds = kValuesInLds<T, D>;
    __shared__ __attribute__((aligned(kTileAlign))) char lds[2][2][BM * Tl::kRow];
    __shared__ __attribute__((aligned(16))) char values[kInLds ? kKeyRows * kValueRow : 16];
    __shared__ __attribute__((aligned(16))) float stats[2][2][BM];
    const int part = static_cast<int>(blockIdx.x % a.splits);
    const AttnItem w = find_item(a.kv, a.kv_heads, false, kKeyShift, blockIdx.x / a.splits);
    if (w.c.seq < 0 || w.c.r0 >= w.c.r1) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = wave >> 1;
    const int begin = seq_begin(a.seq, w.c.seq);
    const int rows = seq_end(a.seq, w.c.seq, begin) - begin;
    const int count = w.c.end - w.c.begin;
    const int off = count - rows;

    const int key0 = w.c.r0 - w.c.begin;
    const int wave0 = key0 + (wave & 1) * 32;
    const int key = wave0 + (lane & 31);
    const bool mine = key < count;
    const int64_t at = static_cast<int64_t>(w.c.begin) + (mine ? key : 0);
    const int64_t col = static_cast<int64_t>(w.head) * a.d;

    Quad k[Tl::kSteps], v[kInLds ? 1 : Tl::kSteps];
    ld_rows<T, D>(static_cast<const T*>(a.k) + at * a.ldk + col, mine, a.d, a.flip, k);
    const T* const value = static_cast<const T*>(a.v) + at * a.ldv + col;
    const uint32_t vt = lds_at(values) + ((wave & 1) * 32 + (lane & 31)) * kValueRow + (lane >> 5) * 16;
    if constexpr (kInLds) {
        const int c = (lane >> 5) * Tl::kE;
        v[0] = ld16(value + kValueSteps * 2 * Tl::kE + c, mine ? a.d - kValueSteps * 2 * Tl::kE - c : 0);
        if (half == 0) {
#pragma unroll
            for (int i = 0; i < kValueSteps; ++i)
                *(lds_quad*)(vt + 32 * i) = ld16(value + 2 * i * Tl::kE + c, mine ? a.d - 2 * i * Tl::kE - c : 0);
        }
    } else {
        ld_rows<T, D>(value, mine, a.d, false, v);
    }

    // tiles of rows from the first that sees a key of the workgroup, for each head; this part's of them
    const int row0 = !a.causal || key0 - off < 0 ? 0 : key0 - off;
    const int t0 = row0 / BM;
    const int each = row0 < rows ? (rows + BM - 1) / BM - t0 : 0;
    const int64_t all = static_cast<int64_t>(each) * a.group;
    const int first = static_cast<int>(all * part / a.splits);
    const int tiles = static_cast<int>(all * (part + 1) / a.splits);

    f32x16 dk[kBlocks<D>], dv[kBlocks<D>];
#pragma unroll
    for (int b = 0; b < kBlocks<D>; ++b)
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
            stat = (tid < BM ? a.lse : a.delta)[i];  // (not used before commit: that would wait for the tiles)
        }
    };
    const auto commit = [&](int buf) {
        sq.commit(tid, lds[buf][0]);
        sg.commit(tid, lds[buf][1]);
        if (tid < 2 * BM) stats[buf][tid / BM][tid % BM] = tid < BM ? log2_sum(stat) : stat;
    };
    clear_tiles<kDirect>(tid, kAttnThreads, lds[0][0], sizeof lds, a.d == D);
    const int lo = a.causal ? key - off : 0;   // rows lo .. rows - 1 see this lane's key
    const int alone = count == 1 ? 0 : -off;   // the row that sees one key (with one key, every row)
    int head = each > 0 ? first / each : 0, tile = t0 + (each > 0 ? first % each : 0);
    if (first < tiles) {
        fetch(head, tile, 0);
        commit(0);
    }
    __syncthreads();
    for (int t = first; t < tiles; ++t) {
        const bool more = t + 1 < tiles;
        const int buf = (t - first) & 1;
        const int r0 = tile * BM + half * 32;
        if (++tile == t0 + each) {
            tile = t0;
            ++head;
        }
        if (more) fetch(head, tile, buf ^ 1);
        if (wave0 < count && r0 < rows && (!a.causal || wave0 <= r0 + 31 + off)) {
            const uint32_t half_at = half * 32 * Tl::kRow;
            const uint32_t qt = Tl::rows_at(lds_at(lds[buf][0]) + half_at), qc = Tl::columns_at(lds_at(lds[buf][0]) + half_at);
            const uint32_t gt = Tl::rows_at(lds_at(lds[buf][1]) + half_at), gc = Tl::columns_at(lds_at(lds[buf][1]) + half_at);
            const bool hides = r0 + 32 > rows || (a.causal && wave0 + 31 > r0 + off);
            const bool lone = count == 1 || (a.causal && alone >= r0 && alone < r0 + 32);
            // (the barriers keep the compiler from fetching fragments of the next
            // product early: their registers would not be there)
            f32x16 s, dp;
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < Tl::kSteps; ++i)
                if (Tl::holds(i, a.d)) s = mma<T>(Tl::rows(qt, 0, i), k[i], s);
            if (hides) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int i = r0 + result_row(r);
                    s[r] = i >= lo && i < rows ? s[r] : -INFINITY;
                }
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 lse2 = *reinterpret_cast<const f32x4*>(&stats[buf][0][half * 32 + result_row(4 * g)]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[4 * g + j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[4 * g + j], a.scale_log2, -lse2[j]));
            }
            if constexpr (kInLds) __builtin_amdgcn_sched_barrier(0);
            {
                const Factor<T> p(s);
#pragma unroll
                for (int b = 0; b < kBlocks<D>; ++b) dv[b] = Tl::columns(gc, 0, b, p.p, dv[b]);
            }
            if constexpr (kInLds) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < Tl::kSteps; ++i) {
                if (!Tl::holds(i, a.d)) continue;
                if constexpr (kInLds)
                    dp = mma<T>(Tl::rows(gt, 0, i), i < kValueSteps ? *(const lds_quad*)(vt + 32 * i) : v[0], dp);
                else
                    dp = mma<T>(Tl::rows(gt, 0, i), v[i], dp);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 delta = *reinterpret_cast<const f32x4*>(&stats[buf][1][half * 32 + result_row(4 * g)]);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[4 * g + j] *= dp[4 * g + j] - delta[j];
            }
            if (lone) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (count == 1 || r0 + result_row(r) == alone) s[r] = 0.0f;
            }
            if constexpr (kInLds) __builtin_amdgcn_sched_barrier(0);
            {
                const Factor<T> ds(s);
#pragma unroll
                for (int b = 0; b < kBlocks<D>; ++b) dk[b] = Tl::columns(qc, 0, b, ds.p, dk[b]);
            }
            if constexpr (kInLds) __builtin_amdgcn_sched_barrier(0);
        }
        if (more) commit(buf ^ 1);
        // (used here whatever happened: a load that may be under way still would be waited
        // for wherever its register is next written, among the fetches, and they with it:
        // four maps of 3136 tokens, 16 heads of 72, 750 us, 626 so)
        asm volatile("" ::"v"(stat));
        __syncthreads();
    }

    // the second half of the waves hands its sums to the first
    constexpr int kJoin = 8 * kBlocks<D>;  // f32x4 of a lane
    f32x4* const join = reinterpret_cast<f32x4*>(lds[0][0]) + (wave & 1) * kJoin * 64 + lane;
    static_assert(sizeof lds >= 2 * kJoin * 64 * 16);
    if (half == 1) {
#pragma unroll
        for (int b = 0; b < kBlocks<D>; ++b)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                join[(8 * b + g) * 64] = f32x4{dk[b][4 * g], dk[b][4 * g + 1], dk[b][4 * g + 2], dk[b][4 * g + 3]};
                join[(8 * b + 4 + g) * 64] = f32x4{dv[b][4 * g], dv[b][4 * g + 1], dv[b][4 * g + 2], dv[b][4 * g + 3]};
            }
    }
    __syncthreads();
    if (half == 1 || !mine) return;
#pragma unroll
    for (int b = 0; b < kBlocks<D>; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x4 x = join[(8 * b + g) * 64], y = join[(8 * b + 4 + g) * 64];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dk[b][4 * g + j] += x[j];
                dv[b][4 * g + j] += y[j];
            }
        }
    if (a.splits > 1) {
        const int64_t size = static_cast<int64_t>(a.kv.rows) * a.kv_heads * a.d;
        float* const to = a.part + part * 2 * size + at * a.kv_heads * a.d + col;
        st_result<float, D>(to, dk, a.scale, a.d);
        st_result<float, D>(to + size, dv, 1.0f, a.d);
    } else {
        st_result<T, D>(static_cast<T*>(a.dk) + at * a.lddk + col, dk, a.scale, a.d);
        st_result<T, D>(static_cast<T*>(a.dv) + at * a.lddv + col, dv, 1.0f, a.d);
    }
}

// The parts' sums, in order, of the rows inside the sequences.
template <typename T>
__global__ __launch_bounds__(kAttnThreads) void attn_parts_kernel(const AttnK a) {
    const int width = a.kv_heads * a.d;
    const int64_t size = static_cast<int64_t>(a.kv.rows) * width;
    const int last = a.kv.nseq - 1;
    const int lo = a.kv.cu ? seq_begin(a.kv, 0) : 0;
    const int hi = a.kv.cu ? seq_end(a.kv, last, seq_begin(a.kv, last)) : a.kv.rows;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAttnThreads + threadIdx.x; i < 2 * size;
         i += static_cast<int64_t>(gridDim.x) * kAttnThreads) {
        const int64_t e = i < size ? i : i - size;
        const int64_t row = e / width;
        if (row < lo || row >= hi) continue;
        float s = 0.0f;
        for (int p = 0; p < a.splits; ++p) s += a.part[p * 2 * size + i];
        T* const to = static_cast<T*>(i < size ? a.dk : a.dv) + row * (i < size ? a.lddk : a.lddv) + (e - row * width);
        Store<T>::st(to, s);
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

// Parts that the rows which a workgroup of keys walks are cut into: as many as
// fill two workgroups a CU, none of fewer than two tiles on average.  Their sums
// pass through memory in fp32, little where there are few keys (the sum of the
// parts takes 4 us of the 27 + 4 for 2003 rows over 539 keys, 6 heads of 40).
int attn_bwd_parts(int64_t rows, int64_t nseq, int64_t heads, int64_t kv_rows, int64_t kv_heads) {
    const int64_t groups = chunk_ids(true, kv_rows, nseq, kKeyShift) * kv_heads;
    const int64_t tiles = (rows / nseq + kBwdRows - 1) / kBwdRows * (heads / kv_heads);
    int64_t n = 512 / groups;
    if (n > tiles / 2) n = tiles / 2;
    if (n > kAttnMaxParts) n = kAttnMaxParts;
    return n < 1 ? 1 : static_cast<int>(n);
}

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
            GSPN_REPLAYED("attn_dq_kernel", kAttnThreads, int64_t{4} * kTileRows<T> * Tile<T, D>::kRow);
            hipLaunchKernelGGL((attn_dq_kernel<T, D, kDirect>), grid, dim3(kAttnThreads), 0, stream, k);
        });
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.kv_rows > 0) {
        k.splits = attn_bwd_parts(a.seq.rows, a.seq.nseq, a.heads, a.kv_rows, a.kv_heads);
        k.part = k.delta + (a.heads * a.seq.rows + 3) / 4 * 4;
        const dim3 grid(static_cast<unsigned>(chunk_ids(k.kv.cu != nullptr, a.kv_rows, a.seq.nseq, kKeyShift) *
                                              a.kv_heads * k.splits));
        const bool direct = attn_direct(a.q, a.ldq, a.d, es) && attn_direct(a.gout, a.ldgo, a.d, es);
        replay("attn_dkv_kernel");
        GSPN_REPLAY_ROWS("attn_dkv_kernel", "dk", a.dk, a.kv_rows, a.lddk, ck, es);
        GSPN_REPLAY_ROWS("attn_dkv_kernel", "dv", a.dv, a.kv_rows, a.lddv, ck, es);
        if (k.splits > 1) GSPN_REPLAY_ROWS("attn_dkv_kernel", "parts", k.part, 2 * k.splits * a.kv_rows, ck, ck, 4);
        attn_dispatch(dtype, a.d, direct, [&](auto t, auto width, auto straight) {
            using T = decltype(t);
            constexpr int D = decltype(width)::value;
            constexpr bool kDirect = decltype(straight)::value;
            GSPN_REPLAYED("attn_dkv_kernel", kAttnThreads,
                          kBwdRows * (int64_t{4} * Tile<T, D>::kRow + 16) +
                              (kValuesInLds<T, D> ? kKeyRows * kValueRow : 16));
            hipLaunchKernelGGL((attn_dkv_kernel<T, D, kDirect>), grid, dim3(kAttnThreads), 0, stream, k);
        });
        e = hipGetLastError();
        if (e != hipSuccess || k.splits == 1) return e;
        const int64_t blocks = (2 * a.kv_rows * ck + kAttnThreads - 1) / kAttnThreads;
        GSPN_REPLAY_ROWS("attn_parts_kernel", "parts", k.part, 2 * k.splits * a.kv_rows, ck, ck, 4);
        GSPN_REPLAY_ROWS("attn_parts_kernel", "dk", a.dk, a.kv_rows, a.lddk, ck, es);
        GSPN_REPLAY_ROWS("attn_parts_kernel", "dv", a.dv, a.kv_rows, a.lddv, ck, es);
        GSPN_REPLAYED("attn_parts_kernel", kAttnThreads, 0);
        const dim3 sums(static_cast<unsigned>(blocks < 2048 ? blocks : 2048));
        if (dtype == GSPN_F32)
            hipLaunchKernelGGL((attn_parts_kernel<float>), sums, dim3(kAttnThreads), 0, stream, k);
        else
            hipLaunchKernelGGL((attn_parts_kernel<bf16_t>), sums, dim3(kAttnThreads), 0, stream, k);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace gspn
