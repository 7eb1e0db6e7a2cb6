// attention_step.hip -- attention of single tokens over cache entries.
//
// One query row for each sequence and head: bound by the entries' bytes, each
// read once for all the query heads that share it.  The heads of a group are
// the 32 columns of the products.  A sequence's keys are cut into `splits` runs,
// a workgroup each; its four waves walk every fourth tile of 32 keys through LDS
// of their own, without a barrier, and are joined at the end, as the runs are
// by a second launch.  64 tokens over entries of 2048 to 4096 rows, 8 heads of keys
// of 128: 162 us, 4870 GB/s, 94% of what a copy reaches.  Two entries of 46000
// rows, 2 heads of keys: 64 runs each, 23 us and 4.3 to join them.
// bf16 numerators go into their product as two factors, themselves rounded and
// what that lost: one factor alone took 160 us, and the results lay 0.0023 (root
// mean square, of their size) from the exact ones, 0.0017 so, their own rounding.
#include "attention.hpp"

namespace gspn {
namespace {

constexpr int kStepKeys = 32;                // of a wave's tile
constexpr int kStepWaves = kAttnThreads / 64;
constexpr int kStepRound = kStepKeys * kStepWaves;

template <typename T, int D>
__global__ __launch_bounds__(kAttnThreads, 1) void attn_step_kernel(const AttnK a) {
    using Tl = Tile<T, D>;
    // the waves' tiles, and where they are joined afterwards
    constexpr int kTiles = 2 * kStepKeys * Tl::kRow;
    constexpr int kJoin = 32 * (32 * kBlocks<D> + 2) * 4;
    constexpr int kSum = 32 * 32 * kBlocks<D>, kMost = kSum + 32;
    constexpr int kWave = kTiles > kJoin ? kTiles : kJoin;
    static_assert(kWave % Tl::kAlign == 0);  // each wave's tiles lie as the first one's do
    __shared__ __attribute__((aligned(kTileAlign))) char lds[kStepWaves][kWave];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int blocks = (a.group + 31) / 32;  // of 32 heads of a group
    int64_t id = blockIdx.x;
    const int split = static_cast<int>(id % a.splits);
    id /= a.splits;
    const int block = static_cast<int>(id % blocks);
    id /= blocks;
    const int kv_head = static_cast<int>(id % a.kv_heads);
    const int seq = static_cast<int>(id / a.kv_heads);

    const int column = block * 32 + (lane & 31);
    const int head = kv_head * a.group + column;
    const bool mine = column < a.group;
    const Keys<T> keys = find_keys<T>(a, seq, seq, 1, kv_head);
    T* const out = static_cast<T*>(a.out) + seq * a.ldo + static_cast<int64_t>(head) * a.d;
    // a split's results: numerators' sum and maximum behind the d values
    float* const part = a.splits > 1
        ? a.part + ((static_cast<int64_t>(seq) * a.heads + head) * a.splits + split) * (a.d + 2) : nullptr;
    if (keys.state != 0) {
        if (wave != 0 || split != 0 || lane >= 32 || !mine) return;
        if (part) {
            part[a.d] = keys.state == kBadSlot ? NAN : -1.0f;  // read by the join before anything else
        } else if (keys.state == kBadSlot) {
            for (int i = 0; i < a.d; ++i) Store<T>::st(out + i, NAN);
        }
        return;
    }

    Quad q[Tl::kSteps];
    ld_rows<T, D>(static_cast<const T*>(a.q) + seq * a.ldq + static_cast<int64_t>(mine ? head : 0) * a.d, mine, a.d,
                  a.flip, q);
    const int held = keys.count - 1;  // the new row's place
    const int rounds = (keys.count + kStepRound - 1) / kStepRound;
    const int each = (rounds + a.splits - 1) / a.splits;
    const int begin = split * each * kStepRound;
    const int64_t most = static_cast<int64_t>(begin) + static_cast<int64_t>(each) * kStepRound;
    const int end = most < keys.count ? static_cast<int>(most) : keys.count;

    const T* const kp = keys.k.entry;
    const T* const vp = keys.v.entry;
    const T* const knew = keys.k.fresh;
    const T* const vnew = keys.v.fresh;
    if (begin <= held && held < end && block == 0 && wave == 0) {  // nobody reads this row of the pool
        for (int i = lane; i < a.d; i += 64) {
            const_cast<T*>(kp)[held * keys.k.ld_held + i] = knew[i];
            const_cast<T*>(vp)[held * keys.v.ld_held + i] = vnew[i];
        }
    }

    constexpr int kN = kStepKeys * Tl::kChunks / 64;
    Quad sk[kN], sv[kN];
    const auto load = [&](int key0) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int at = i * 64 + lane;
            const int r = key0 + at / Tl::kChunks, c = at % Tl::kChunks * Tl::kE;
            sk[i] = ld16((r < held ? kp + r * keys.k.ld_held : knew) + c, a.d - c);
            sv[i] = ld16((r < held ? vp + r * keys.v.ld_held : vnew) + c, a.d - c);
        }
    };
    char* const kt = lds[wave];
    char* const vt = lds[wave] + kStepKeys * Tl::kRow;
    const uint32_t kr = Tl::rows_at(lds_at(kt)), vc = Tl::columns_at(lds_at(vt));
    Softmax<D> sm;
    int key0 = begin + wave * kStepKeys;
    if (key0 < end) load(key0);
    for (; key0 < end; key0 += kStepRound) {
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int at = i * 64 + lane;
            const int r = at / Tl::kChunks, c = at % Tl::kChunks;
            *reinterpret_cast<Quad*>(kt + r * Tl::kRow + Tl::swizzle(r, c) * 16) = sk[i];
            *reinterpret_cast<Quad*>(vt + r * Tl::kRow + Tl::swizzle(r, c) * 16) = sv[i];
        }
        __builtin_amdgcn_wave_barrier();
        if (key0 + kStepRound < end) load(key0 + kStepRound);
        f32x16 s[1];
#pragma unroll
        for (int r = 0; r < 16; ++r) s[0][r] = 0.0f;
#pragma unroll
        for (int i = 0; i < Tl::kSteps; ++i)
            if (Tl::holds(i, a.d)) s[0] = mma<T>(Tl::rows(kr, 0, i), q[i], s[0]);
        if (key0 + kStepKeys > end) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (key0 + result_row(r) >= end) s[0][r] = -INFINITY;
        }
        sm.meet(s, a.scale_log2);
        sm.weigh(s, a.scale_log2);
        sm.add(s);
        const Factor<T> p(s[0]);
#pragma unroll
        for (int b = 0; b < kBlocks<D>; ++b) sm.o[b] = Tl::columns(vc, 0, b, p.p, sm.o[b]);
        if constexpr (kIsBf16<T>) {
            const Factor<T> rest = p.left_of(s[0]);
#pragma unroll
            for (int b = 0; b < kBlocks<D>; ++b) sm.o[b] = Tl::columns(vc, 0, b, rest.p, sm.o[b]);
        }
    }

    // the waves' results: [32][d values, sum, maximum], each on the others' scale
    __syncthreads();
    float* const join = reinterpret_cast<float*>(lds[wave]);
    const float l = both_sum(sm.l);
#pragma unroll
    for (int b = 0; b < kBlocks<D>; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) join[(32 * b + result_row(r)) * 32 + (lane & 31)] = sm.o[b][r];
    if (lane < 32) {
        join[kSum + lane] = l;
        join[kMost + lane] = sm.m;
    }
    __syncthreads();
    float f[kStepWaves], top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kStepWaves; ++j) {
        f[j] = reinterpret_cast<const float*>(lds[j])[kMost + (lane & 31)];
        top = __builtin_fmaxf(top, f[j]);
    }
    if (top == -INFINITY) top = 0.0f;  // no key, or every score -Inf
#pragma unroll
    for (int j = 0; j < kStepWaves; ++j) {
        f[j] = __builtin_amdgcn_exp2f((f[j] - top) * a.scale_log2);
        sum = __builtin_fmaf(f[j], reinterpret_cast<const float*>(lds[j])[kSum + (lane & 31)], sum);
    }
    if (!mine) return;
    const float inv = part ? 1.0f : 1.0f / sum;
    for (int e = wave * 2 + (lane >> 5); e < a.d; e += 2 * kStepWaves) {
        float o = 0.0f;
#pragma unroll
        for (int j = 0; j < kStepWaves; ++j)
            o = __builtin_fmaf(f[j], reinterpret_cast<const float*>(lds[j])[e * 32 + (lane & 31)], o);
        if (part)
            part[e] = o;
        else
            Store<T>::st(out + e, o * inv);
    }
    if (part && tid < 32) {
        part[a.d] = sum;
        part[a.d + 1] = top;
    }
}

// The splits of one row and head, a workgroup each: every wave sums a fourth of
// them (a wave alone took 34 us for 64 splits of 32 rows, as long as the keys).
template <typename T>
__global__ __launch_bounds__(kAttnThreads) void attn_step_join_kernel(const AttnK a) {
    __shared__ float sums[kStepWaves][GSPN_ATTENTION_MAX_HEAD];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = blockIdx.x;
    const int width = a.d + 2;
    const float* const part = a.part + id * a.splits * width;
    const int64_t seq = id / a.heads;
    T* const out = static_cast<T*>(a.out) + seq * a.ldo + (id - seq * a.heads) * a.d;
    const bool in = lane < a.splits;
    const float l = in ? part[lane * width + a.d] : 0.0f;
    const float m = in ? part[lane * width + a.d + 1] : -INFINITY;  // (what it is where l is 0 does not count)
    const float first = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(l)));
    if (first < 0.0f) return;  // padding
    if (first != first) {      // an error, or NaN among the values
        for (int e = threadIdx.x; e < a.d; e += kAttnThreads) Store<T>::st(out + e, NAN);
        return;
    }
    float top = l == 0.0f ? -INFINITY : m;
#pragma unroll
    for (int i = 32; i > 0; i /= 2) top = __builtin_fmaxf(top, __shfl_xor(top, i));
    const float f = l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f((m - top) * a.scale_log2);
    const float inv = 1.0f / wave_sum(f * l);
    const int e0 = lane < a.d ? lane : 0, e1 = lane + 64 < a.d ? lane + 64 : 0;
    float o0 = 0.0f, o1 = 0.0f;
    constexpr int kAhead = 8;
    for (int j0 = wave; j0 < a.splits; j0 += kAhead * kStepWaves) {
        float v0[kAhead], v1[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int j = j0 + i * kStepWaves < a.splits ? j0 + i * kStepWaves : j0;
            v0[i] = part[j * width + e0];
            v1[i] = part[j * width + e1];
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int j = j0 + i * kStepWaves;
            if (j < a.splits) {
                const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), j));
                o0 = __builtin_fmaf(w, v0[i], o0);
                o1 = __builtin_fmaf(w, v1[i], o1);
            }
        }
    }
    sums[wave][lane] = o0;
    sums[wave][lane + 64] = o1;
    __syncthreads();
    const int e = threadIdx.x;
    if (e < a.d) {
        float o = 0.0f;
#pragma unroll
        for (int w = 0; w < kStepWaves; ++w) o += sums[w][e];
        Store<T>::st(out + e, o * inv);
    }
}

}  // namespace

// Runs of a sequence's keys: 512 workgroups or more, none shorter than four rounds
// of its waves over a full entry, which take about as long as the join's launch.
// (Two share a CU, but for heads past 96 bf16 or 64 fp32 elements, whose waves hold
// more than 256 registers.)  The host knows the entries' capacity, not what they
// hold: with 512 groups or more an entry is one run, and a long one among short ones
// is waited for (one of 32768 rows among 63 of 512, 8 heads of keys: 486 us, 52 of bytes).
int attn_splits(int64_t nseq, int64_t heads, int64_t kv_heads, int64_t capacity) {
    const int64_t groups = nseq * kv_heads * ((heads / kv_heads + 31) / 32);
    if (groups < 1) return 1;
    const int64_t fill = (512 + groups - 1) / groups;
    const int64_t most = capacity / (4 * kStepRound);
    int64_t n = fill < most ? fill : most;
    if (n > kAttnMaxSplits) n = kAttnMaxSplits;
    return n < 1 ? 1 : static_cast<int>(n);
}

hipError_t launch_attn_step(const gspn_attn_args& a, int dtype, hipStream_t stream) {
    AttnK k = make_attn(a);
    k.splits = attn_splits(a.seq.nseq, a.heads, a.kv_heads, a.capacity);
    k.part = static_cast<float*>(a.workspace);
    const int64_t es = dtype == GSPN_F32 ? 4 : 2;
    const int64_t cq = a.heads * a.d, ck = a.kv_heads * a.d, parts = a.seq.nseq * a.heads * k.splits;
    const int64_t blocks = a.seq.nseq * a.kv_heads * ((k.group + 31) / 32) * k.splits;
    (void)es;
    (void)cq;
    (void)ck;
    GSPN_REPLAY_ROWS("attn_step_kernel", "q", a.q, a.seq.rows, a.ldq, cq, es);
    GSPN_REPLAY_ROWS("attn_step_kernel", "k", a.k, a.seq.rows, a.ldk, ck, es);
    GSPN_REPLAY_ROWS("attn_step_kernel", "v", a.v, a.seq.rows, a.ldv, ck, es);
    GSPN_REPLAY_ROWS("attn_step_kernel", "out", a.out, a.seq.rows, a.ldo, cq, es);
    GSPN_REPLAY_ROWS("attn_step_kernel", "k_pool", a.k_pool, a.seq.nslots * a.capacity, ck, ck, es);
    GSPN_REPLAY_ROWS("attn_step_kernel", "v_pool", a.v_pool, a.seq.nslots * a.capacity, ck, ck, es);
    GSPN_REPLAY_ROWS("attn_step_kernel", "held", a.held, 1, a.seq.nseq, a.seq.nseq, 4);
    if (k.splits > 1) GSPN_REPLAY_ROWS("attn_step_kernel", "runs", a.workspace, parts, a.d + 2, a.d + 2, 4);
    attn_dispatch(dtype, a.d, false, [&](auto t, auto width, auto) {
        using T = decltype(t);
        constexpr int D = decltype(width)::value;
        GSPN_REPLAYED("attn_step_kernel", kAttnThreads,
                      4 * kStepKeys * (2 * Tile<T, D>::kRow > (32 * kBlocks<D> + 2) * 4 ? 2 * Tile<T, D>::kRow
                                                                                    : (32 * kBlocks<D> + 2) * 4));
        hipLaunchKernelGGL((attn_step_kernel<T, D>), dim3(static_cast<unsigned>(blocks)), dim3(kAttnThreads), 0, stream,
                           k);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || k.splits == 1) return e;
    const dim3 grid(static_cast<unsigned>(a.seq.nseq * a.heads));
    GSPN_REPLAY_ROWS("attn_step_join_kernel", "runs", a.workspace, parts, a.d + 2, a.d + 2, 4);
    GSPN_REPLAY_ROWS("attn_step_join_kernel", "out", a.out, a.seq.rows, a.ldo, cq, es);
    GSPN_REPLAYED("attn_step_join_kernel", kAttnThreads, kStepWaves * GSPN_ATTENTION_MAX_HEAD * 4);
    if (dtype == GSPN_F32)
        hipLaunchKernelGGL((attn_step_join_kernel<float>), grid, dim3(kAttnThreads), 0, stream, k);
    else
        hipLaunchKernelGGL((attn_step_join_kernel<bf16_t>), grid, dim3(kAttnThreads), 0, stream, k);
    return hipGetLastError();
}

}  // namespace gspn
