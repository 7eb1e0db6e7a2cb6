// attention.hip -- softmax attention over whole prompts, with grouped heads,
// packed sequences and prompts that continue a cache entry.
#include "attention.hpp"

namespace gspn {
namespace {

// Eight new rows of keys and values into their entries, four loads a lane on their
// way before the first store.
template <typename T>
__device__ __forceinline__ void append_rows(const AttnK& a, uint32_t id) {
    const Chunk c = find_chunk(a.seq, id, kAppendShift);
    if (c.seq < 0 || c.r0 >= c.r1) return;
    const Keys<T> keys = find_keys<T>(a, c.seq, c.begin, c.end - c.begin, 0);
    if (keys.state != 0) return;
    constexpr int kE = 16 / sizeof(T);
    const int width = a.kv_heads * a.d;
    const int64_t at = keys.k.held + (c.r0 - c.begin);
    const uint32_t chunks = width / kE;  // whole ones of a row; keys' and values' rows in turn
    const uint32_t all = 2 * (c.r1 - c.r0) * chunks;
    const auto place = [&](uint32_t row, int e, const T** from, T** to) {
        const int r = row >> 1, value = row & 1;
        *from = static_cast<const T*>(value ? a.v : a.k) + (c.r0 + r) * (value ? a.ldv : a.ldk) + e;
        *to = const_cast<T*>((value ? keys.v : keys.k).entry) + (at + r) * width + e;
    };
    constexpr int kAhead = 4;
    for (uint32_t i0 = threadIdx.x; i0 < all; i0 += kAhead * kAttnThreads) {
        Quad x[kAhead];
        T* to[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint32_t i = i0 + j * kAttnThreads < all ? i0 + j * kAttnThreads : i0;
            const T* from;
            place(i / chunks, i % chunks * kE, &from, &to[j]);
            __builtin_memcpy(&x[j], from, 16);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) asm volatile("" : "+v"(x[j]));  // all on their way before the first store
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i0 + j * kAttnThreads < all) __builtin_memcpy(to[j], &x[j], 16);
    }
    const int rest = width - chunks * kE;
    for (int i = threadIdx.x; i < 2 * (c.r1 - c.r0) * rest; i += kAttnThreads) {
        const T* from;
        T* to;
        place(i / rest, chunks * kE + i % rest, &from, &to);
        *to = *from;
    }
}

// Attention of 128 rows, 32 a wave, over their keys in tiles of 64 (fp32: 32) that
// the waves share: one pass with a running maximum and sum (Softmax), keys and
// values twice in LDS.  Bound by the matrix unit, and by the power that it takes:
// a prompt of 16384 rows, 32 heads of 128, takes 2070 us, 1060 TFLOP/s, with
// the unit busy in 59% of the cycles at a clock of 1.6 GHz; a large plain product
// reaches 1160 to 1220.  Short walks pay for their start, which takes as long as
// two to four tiles: 16 ragged prompts of 8192 rows in all 140 us, 595 TFLOP/s.
// bf16 numerators are rounded to bf16 for their product: what that loses, as a
// second factor, would bring the results from 0.0020 of their size (root mean
// square) to 0.0018 of the exact ones, for 2810 us and 168 in place of those.
// A walk is never cut along its keys: eight rows behind 32768 held ones, 32 heads on
// 8 of keys, take 660 us where the entry's bytes take 26.
// kCache: the rows that an entry holds are read there, the new ones where they
// are (any other way the copies would have to be done first: 12 us of 147), and
// workgroups behind the others copy them over while the last walks end (before
// the others they cost 9 us more).
template <typename T, int D, bool kDirect, bool kCache>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_fwd_kernel(const AttnK a) {
    using Tl = Tile<T, D>;
    constexpr int BN = kTileRows<T>;
    __shared__ __attribute__((aligned(kTileAlign))) char lds[2][2][BN * Tl::kRow];
    if constexpr (kCache) {
        if (blockIdx.x >= static_cast<uint32_t>(a.walks)) {
            append_rows<T>(a, blockIdx.x - a.walks);
            return;
        }
    }
    const AttnItem w = find_item(a.seq, a.heads, a.causal != 0, kAttnShift, blockIdx.x);
    if (w.c.seq < 0 || w.c.r0 >= w.c.r1) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int rows = w.c.end - w.c.begin;
    const Keys<T> keys = find_keys<T>(a, w.c.seq, w.c.begin, rows, w.head / a.group);
    const int off = keys.count - rows;  // row i sees i + off + 1 keys where later ones are hidden

    const int wave0 = w.c.r0 - w.c.begin + __builtin_amdgcn_readfirstlane(tid >> 6) * 32;  // the wave's first row
    const int row = wave0 + (lane & 31);
    const bool mine = row < rows;
    const int64_t at = static_cast<int64_t>(w.c.begin) + (mine ? row : 0);
    T* const out = static_cast<T*>(a.out) + at * a.ldo + static_cast<int64_t>(w.head) * a.d;
    float* const lse = a.lse ? a.lse + static_cast<int64_t>(w.head) * a.seq.rows + at : nullptr;
    if (keys.state == kBadSlot) {
        f32x16 o[kBlocks<D>];
        for (int b = 0; b < kBlocks<D>; ++b)
            for (int r = 0; r < 16; ++r) o[b][r] = NAN;
        if (mine) {
            st_result<T, D>(out, o, 1.0f, a.d);
            if (lse && lane < 32) *lse = NAN;
        }
        return;
    }

    Quad q[Tl::kSteps];
    ld_rows<T, D>(static_cast<const T*>(a.q) + at * a.ldq + static_cast<int64_t>(w.head) * a.d, mine, a.d, a.flip, q);
    const auto seen = [&](int r) {  // keys that row r sees
        const int n = a.causal ? r + off + 1 : keys.count;
        return n < 0 ? 0 : n < keys.count ? n : keys.count;
    };
    const int last = (w.c.r1 < w.c.end ? w.c.r1 : w.c.end) - 1 - w.c.begin;
    const int tiles = (seen(last) + BN - 1) / BN;
    const int wave_last = wave0 + 31 < rows ? wave0 + 31 : rows - 1;
    const int wave_keys = wave0 < rows ? seen(wave_last) : 0;  // no row of the wave sees more
    const int wave_all = wave0 < rows ? seen(wave0) : 0;       // every one sees these
    const int my_keys = mine ? seen(row) : 0;

    Softmax<D> sm;
    Stage<T, D, BN, kAttnThreads, kDirect> sk, sv;
    clear_tiles<kDirect>(tid, kAttnThreads, lds[0][0], sizeof lds, a.d == D);
    const int wave_tiles = (wave_keys + BN - 1) / BN;
    const auto fetch = [&](auto& stage, const Rows<T>& from, int t, char* tile) {
        if constexpr (kCache)
            stage.fetch(tid, from, t * BN, keys.count - 1, a.d, tile);
        else
            stage.fetch(tid, from.fresh, from.ld, t * BN, keys.count - 1, a.d, tile);
    };
    const auto fetch_k = [&](int t) { fetch(sk, keys.k, t, lds[t & 1][0]); };
    const auto fetch_v = [&](int t) { fetch(sv, keys.v, t, lds[t & 1][1]); };
    const auto scores = [&](int buf, f32x16(&s)[BN / 32]) {
        const uint32_t kt = Tl::rows_at(lds_at(lds[buf][0]));
#pragma unroll
        for (int n = 0; n < BN / 32; ++n) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[n][r] = 0.0f;
#pragma unroll
            for (int i = 0; i < Tl::kSteps; ++i)
                if (Tl::holds(i, a.d)) s[n] = mma<T>(Tl::rows(kt, 32 * n, i), q[i], s[n]);
        }
    };
    const auto hide = [&](int t, f32x16(&s)[BN / 32]) {
        if ((t + 1) * BN > wave_all) {
            int most = my_keys;
            asm volatile("" : "+v"(most));  // (or the comparisons would be made in every tile)
#pragma unroll
            for (int n = 0; n < BN / 32; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (t * BN + 32 * n + result_row(r) >= most) s[n][r] = -INFINITY;
        }
    };
    const auto values = [&](int buf, const f32x16(&s)[BN / 32]) {
        const uint32_t vt = Tl::columns_at(lds_at(lds[buf][1]));
#pragma unroll
        for (int n = 0; n < BN / 32; ++n) {
            const Factor<T> p(s[n]);
#pragma unroll
            for (int b = 0; b < kBlocks<D>; ++b) sm.o[b] = Tl::columns(vt, 32 * n, b, p.p, sm.o[b]);
        }
    };
    if constexpr (!kIsBf16<T>) {
        // fp32 products take so long that nothing else counts
        if (tiles > 0) {
            fetch_k(0);
            fetch_v(0);
            sk.commit(tid, lds[0][0]);
            sv.commit(tid, lds[0][1]);
        }
        __syncthreads();
        for (int t = 0; t < tiles; ++t) {
            if (t + 1 < tiles) {
                fetch_k(t + 1);
                fetch_v(t + 1);
            }
            if (t < wave_tiles) {
                f32x16 s[BN / 32];
                scores(t & 1, s);
                hide(t, s);
                sm.meet(s, a.scale_log2);
                sm.weigh(s, a.scale_log2);
                values(t & 1, s);
                sm.add(s);
            }
            if (t + 1 < tiles) {
                sk.commit(tid, lds[(t + 1) & 1][0]);
                sv.commit(tid, lds[(t + 1) & 1][1]);
            }
            __syncthreads();
        }
    } else {
        // A tile's scores are formed while those before it become weights, and its
        // maximum while those weigh their values: keys run two tiles ahead of the
        // walk, values one.  Each product is followed by its share of the softmax,
        // which the vector unit does meanwhile; the compiler, left to itself, does the
        // one after the other.
        f32x16 even[BN / 32], odd[BN / 32];
        if (tiles > 0) {
            fetch_k(0);
            fetch_v(0);
            if (kDirect && tiles > 1) fetch_k(1);
            sk.commit(tid, lds[0][0]);
            sv.commit(tid, lds[0][1]);
            if (!kDirect && tiles > 1) {
                fetch_k(1);
                sk.commit(tid, lds[1][0]);
            }
        }
        __syncthreads();
        if (wave_tiles > 0) {
            scores(0, even);
            hide(0, even);
            sm.meet(even, a.scale_log2);
        }
        __syncthreads();
        const auto step = [&](int t, auto buffer, f32x16(&s)[BN / 32], f32x16(&next)[BN / 32]) {
            constexpr int buf = decltype(buffer)::value;
            constexpr int kElems = BN / 2;  // of a lane's scores
            if (t + 2 < tiles) fetch_k(t + 2);
            if (t + 1 < tiles) fetch_v(t + 1);
            {
                uint32_t kt = Tl::rows_at(lds_at(lds[buf ^ 1][0]));
                uint32_t vt = Tl::columns_at(lds_at(lds[buf][1]));
                asm volatile("" : "+v"(kt), "+v"(vt));  // (every address held over the loop would be spilled)
                const float base = sm.m == -INFINITY ? 0.0f : sm.m * a.scale_log2;
                constexpr int kScores = BN / 32 * Tl::kSteps, kAhead = 3;
                Quad kf[kAhead + 1];
                Quad p[kElems / 8];
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int n = 0; n < BN / 32; ++n)
#pragma unroll
                    for (int r = 0; r < 16; ++r) next[n][r] = 0.0f;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) kf[i] = Tl::rows(kt, i % (BN / 32) * 32, i / (BN / 32));
#pragma unroll
                for (int i = 0; i < kScores; ++i) {
                    const int j = i + kAhead;
                    if (j < kScores) kf[j % (kAhead + 1)] = Tl::rows(kt, j % (BN / 32) * 32, j / (BN / 32));
                    next[i % (BN / 32)] = mma<T>(kf[i % (kAhead + 1)], q[i / (BN / 32)], next[i % (BN / 32)]);
#pragma unroll
                    for (int e = kElems * i / kScores; e < kElems * (i + 1) / kScores; ++e) {
                        s[e / 16][e % 16] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e / 16][e % 16], a.scale_log2, -base));
                        sum[e % 2] += s[e / 16][e % 16];
                        if (e % 2) p[e / 8][e / 2 % 4] = pack_bf16x2(s[e / 16][e % 16 - 1], s[e / 16][e % 16]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                sm.l += sum[0] + sum[1];
                asm volatile("" : "+v"(sm.l));  // (here, not after the next products)
                constexpr int kN = kBlocks<D>, kValues = BN / 16 * kN;
                const auto vf_at = [&](int i) { return Tl::column(vt, i / (2 * kN) * 32, i % kN, i / kN % 2); };
                Quad vf[kAhead + 1];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) vf[i] = vf_at(i);
                float top = next[0][0];
#pragma unroll
                for (int i = 0; i < kValues; ++i) {
                    const int j = i + kAhead;
                    if (j < kValues) vf[j % (kAhead + 1)] = vf_at(j);
                    sm.o[i % kN] = mma<T>(vf[i % (kAhead + 1)], p[i / kN], sm.o[i % kN]);
#pragma unroll
                    for (int e = kElems * i / kValues; e < kElems * (i + 1) / kValues; ++e)
                        top = __builtin_fmaxf(top, next[e / 16][e % 16]);
                    __builtin_amdgcn_sched_barrier(0);
                }
                asm volatile("" : "+v"(top));
                if ((t + 2) * BN > wave_all) {
                    hide(t + 1, next);
                    top = sm.most(next);
                }
                sm.meet(top, a.scale_log2);
            }
            if (t + 2 < tiles) sk.commit(tid, lds[buf][0]);
            if (t + 1 < tiles) sv.commit(tid, lds[buf ^ 1][1]);
            __syncthreads();
        };
        int t = 0;
        for (; t + 2 < wave_tiles; t += 2) {
            step(t, std::integral_constant<int, 0>{}, even, odd);
            step(t + 1, std::integral_constant<int, 1>{}, odd, even);
        }
        if (t + 1 < wave_tiles) {
            step(t, std::integral_constant<int, 0>{}, even, odd);
            ++t;
#pragma unroll
            for (int n = 0; n < BN / 32; ++n) even[n] = odd[n];
        }
        // the wave's last tile, and those that only other waves walk
        for (; t < tiles; ++t) {
            if (t + 2 < tiles) fetch_k(t + 2);
            if (t + 1 < tiles) fetch_v(t + 1);
            if (t < wave_tiles) {
                sm.weigh(even, a.scale_log2);
                values(t & 1, even);
                sm.add(even);
            }
            if (t + 2 < tiles) sk.commit(tid, lds[t & 1][0]);
            if (t + 1 < tiles) sv.commit(tid, lds[(t + 1) & 1][1]);
            __syncthreads();
        }
    }
    const float l = both_sum(sm.l);
    if (mine) {
        st_result<T, D>(out, sm.o, my_keys > 0 ? 1.0f / l : 0.0f, a.d);
        if (lse && lane < 32)
            *lse = my_keys > 0 ? (sm.m * a.scale_log2 + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f : -INFINITY;
    }
}

void replay_fwd(const char* kn, const gspn_attn_args& a, int64_t es) {
    (void)kn;
    (void)a;
    (void)es;
    GSPN_REPLAY_ROWS(kn, "q", a.q, a.seq.rows, a.ldq, a.heads * a.d, es);
    GSPN_REPLAY_ROWS(kn, "k", a.k, a.kv_rows, a.ldk, a.kv_heads * a.d, es);
    GSPN_REPLAY_ROWS(kn, "v", a.v, a.kv_rows, a.ldv, a.kv_heads * a.d, es);
    GSPN_REPLAY_ROWS(kn, "out", a.out, a.seq.rows, a.ldo, a.heads * a.d, es);
    GSPN_REPLAY_ROWS(kn, "lse", a.lse, a.heads, a.seq.rows, a.seq.rows, 4);
    if (a.k_pool) {
        GSPN_REPLAY_ROWS(kn, "k_pool", a.k_pool, a.seq.nslots * a.capacity, a.kv_heads * a.d, a.kv_heads * a.d, es);
        GSPN_REPLAY_ROWS(kn, "v_pool", a.v_pool, a.seq.nslots * a.capacity, a.kv_heads * a.d, a.kv_heads * a.d, es);
        GSPN_REPLAY_ROWS(kn, "held", a.held, 1, a.seq.nseq, a.seq.nseq, 4);
    }
}

}  // namespace

AttnK make_attn(const gspn_attn_args& a) {
    AttnK k = {};
    k.seq = make_seq(a.seq);
    gspn_sequences kv = a.seq;
    kv.rows = a.kv_rows;
    if (a.kv_cu) kv.cu = a.kv_cu;
    kv.slots = nullptr;
    k.kv = make_seq(kv);
    k.heads = static_cast<int32_t>(a.heads);
    k.kv_heads = static_cast<int32_t>(a.kv_heads);
    k.group = static_cast<int32_t>(a.heads / a.kv_heads);
    k.d = static_cast<int32_t>(a.d);
    k.causal = a.causal != 0;
    k.flip = a.scale < 0.0;
    k.scale = static_cast<float>(a.scale);
    k.scale_log2 = scale_log2(a.scale);
    // (so that a hidden score, -Inf, stays one when it is scaled; the largest other becomes 2^-21)
    if (k.scale_log2 == 0.0f) k.scale_log2 = 0x1p-149f;
    k.q = a.q;
    k.k = a.k;
    k.v = a.v;
    k.out = a.out;
    k.lse = a.lse;
    k.k_pool = a.k_pool;
    k.v_pool = a.v_pool;
    k.capacity = a.capacity;
    k.held = a.held;
    k.gout = a.gout;
    k.dq = a.dq;
    k.dk = a.dk;
    k.dv = a.dv;
    k.ldq = a.ldq;
    k.ldk = a.ldk;
    k.ldv = a.ldv;
    k.ldo = a.ldo;
    k.ldgo = a.ldgo;
    k.lddq = a.lddq;
    k.lddk = a.lddk;
    k.lddv = a.lddv;
    return k;
}

hipError_t launch_attn_fwd(const gspn_attn_args& a, int dtype, hipStream_t stream) {
    AttnK k = make_attn(a);
    const int64_t es = dtype == GSPN_F32 ? 4 : 2;
    const bool ragged = a.seq.cu != nullptr;
    k.walks = static_cast<int32_t>(chunk_ids(ragged, a.seq.rows, a.seq.nseq, kAttnShift) * a.heads);
    const int64_t copies = a.k_pool ? chunk_ids(ragged, a.seq.rows, a.seq.nseq, kAppendShift) : 0;
    const dim3 grid(static_cast<unsigned>(k.walks + copies));
    replay_fwd("attn_fwd_kernel", a, es);
    const int64_t ck = a.kv_heads * a.d;
    const bool direct = attn_direct(a.k, a.ldk, a.d, es) && attn_direct(a.v, a.ldv, a.d, es) &&
                        (!a.k_pool || (attn_direct(a.k_pool, ck, a.d, es) && attn_direct(a.v_pool, ck, a.d, es)));
    attn_dispatch(dtype, a.d, direct, [&](auto t, auto width, auto straight) {
        using T = decltype(t);
        constexpr int D = decltype(width)::value;
        constexpr bool kDirect = decltype(straight)::value;
        GSPN_REPLAYED("attn_fwd_kernel", kAttnThreads, int64_t{4} * kTileRows<T> * Tile<T, D>::kRow);
        if (a.k_pool)
            hipLaunchKernelGGL((attn_fwd_kernel<T, D, kDirect, true>), grid, dim3(kAttnThreads), 0, stream, k);
        else
            hipLaunchKernelGGL((attn_fwd_kernel<T, D, kDirect, false>), grid, dim3(kAttnThreads), 0, stream, k);
    });
    return hipGetLastError();
}

}  // namespace gspn
