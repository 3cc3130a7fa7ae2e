// Beam search next to the recurrence: the choice of the continuations and the reordering of the
// fixed-size states (include/kda.h, kda_beam_select and kda_beam_reorder).
//
// Choice.  With x the logits of a beam, c[k, v] = score_k + x_v - log sum_u exp(x_u).  Within a beam
// the order of c is that of x, so every beam needs only its n_out best logits, and one pass over the
// logits gives them together with the running maximum and sum of the log-sum: the bytes of the
// logits bound it.  A row is split over workgroups; a second launch joins the parts of a group's rows
// and orders the remaining candidates by c in fp64.
//
// The best logits are found with a threshold: the maxima of n_out disjoint groups of threads are
// n_out different logits, so the least of them is no larger than the n_out-th best, and whatever
// lies below it is out.  What is left (about n_out log n_out logits of each round for unordered ones) is
// collected and ranked by a key of value and token, so ties go to the lower token whatever the order of
// collection.
//
// Where more are left than a wave's list holds, the choice is made by repeated maxima over the keys
// instead, n_out more passes over that part of the row: right, but slow.  It happens
//  * where a thread group sees nothing but equal logits for a whole round: a flat row, or a mask of a finite
//    value over a long stretch of the vocabulary or over almost all of it.  128 beams of 131 072 bf16 logits,
//    n_out = 8: 17 us; 60 with the upper half at -1e4 or at the type's lowest value, 91 with all but 100
//    tokens there; 14 to 18 with the same masks at -inf, and with half of the tokens masked at random.
//  * for many rows and a large n_out, since every round's threshold is its own: the same vocabulary, n_out = 16, 24
//    and 32: 23, 44 and 43 us for 128 beams, 75, 701 and 921 for 512, 134, 1663 and 2191 for 1024.
#include <math.h>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxOut = 64;     // n_out and K at most
constexpr int kThreads = 256;
constexpr int kPer = 16;        // logits of a thread per round
constexpr int kRound = kThreads * kPer;
constexpr int kWaves = kThreads / 64;
constexpr int kList = 256;      // collected keys of a wave's share of a part of a row

// Keys order like (value descending, token ascending) when compared as larger first.  No key of a
// token is 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t key_of(float x, int token) {
    return ((uint64_t)ordered(x + 0.f) << 32) | (0xFFFFFFFFu - (uint32_t)token);
}
// NaN counts as -inf (the maximum's result is its other operand); -0 becomes +0 where a key is made
__device__ __forceinline__ float clean(float x) { return fmaxf(x, -INFINITY); }

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t x, int off) {
    const uint32_t lo = __shfl_xor((uint32_t)x, off, 64), hi = __shfl_xor((uint32_t)(x >> 32), off, 64);
    return ((uint64_t)hi << 32) | lo;
}

// Parts of a row in the workspace: keys [rows, parts, n_out], then (maximum, sum) [rows, parts].
struct SelectPlan {
    int parts;
    int per_part;  // tokens of a part, a multiple of kRound
};

__host__ __device__ inline int64_t div_up(int64_t x, int64_t m) { return (x + m - 1) / m; }

inline SelectPlan select_plan(int64_t rows, int V) {
    // about eight workgroups per CU, and at least one round each; rounds begin at 16-byte boundaries,
    // up to 7 tokens before the row
    const int64_t rounds = div_up((int64_t)V + 7, kRound);
    int64_t parts = div_up(2048, rows < 1 ? 1 : rows);
    parts = parts > rounds ? rounds : parts;
    const int64_t per = div_up(rounds, parts);
    return SelectPlan{(int)div_up(rounds, per), (int)(per * kRound)};
}

// The logits of a thread's kPer tokens of the round at `base` (row + base is 16-byte aligned).  A
// whole round is read in 16-byte vectors; one that the row's ends cut, value by value with the
// tokens strided over the threads, so that short ones fill every thread.
template <typename T>
struct Round {
    static constexpr int W = 16 / sizeof(T);  // logits per vector
    static __device__ __forceinline__ int token(int base, int i, bool whole) {
        return whole ? base + (i / W) * kThreads * W + (int)threadIdx.x * W + i % W
                     : base + i * kThreads + (int)threadIdx.x;
    }
    static constexpr int NV = kPer / W;
    static __device__ __forceinline__ void fetch(const T* row, int base, u32x4 (&raw)[NV]) {
#pragma unroll
        for (int v = 0; v < NV; ++v) raw[v] = *reinterpret_cast<const u32x4*>(row + token(base, v * W, true));
    }
    // as they are: NaN stays NaN, which no comparison below lets through
    static __device__ __forceinline__ void values(const u32x4 (&raw)[NV], float (&x)[kPer]) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t word = raw[i / W][(i % W) * sizeof(T) / 4];
            if (sizeof(T) == 4) x[i] = __uint_as_float(word);
            else x[i] = __uint_as_float((i & 1) ? word & 0xFFFF0000u : word << 16);
        }
    }
    // (each load is waited for before the next one, because of its guard: 16 latencies in a row's last round)
    static __device__ __forceinline__ void singles(const T* row, int base, int first, int last, float (&x)[kPer]) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int t = token(base, i, false);
            x[i] = t >= first && t < last ? clean(ld_in(row, t)) : -INFINITY;
        }
    }
    static __device__ __forceinline__ void load(const T* row, int base, int first, int last, bool whole,
                                                float (&x)[kPer]) {
        if (whole) {
            u32x4 raw[NV];
            fetch(row, base, raw);
            values(raw, x);
#pragma unroll
            for (int i = 0; i < kPer; ++i) x[i] = clean(x[i]);
        } else {
            singles(row, base, first, last, x);
        }
    }
};

// sum of exp(x - m), m the maximum (-inf: nothing is above it).  One product and sum per logit: with r =
// fl(m log2 e), exp(x - m) = 2^(x log2 e - r) 2^(r - m log2 e), the last factor once for all.  That needs a small
// r - m log2 e, which is half a unit in the last place of r and grows with m: up to |m| = 2^24 it is 1 at most.
// Beyond (at 2.1e9 it reaches 128, where the hardware's exponential is 0 for one factor and finite for the
// other) the wave takes the difference first.  m infinite goes there too, and inf - inf makes the sum NaN.
__device__ __forceinline__ float exp_sum(const float (&x)[kPer], float m) {
    constexpr float kLog2e = 1.4426950408889634f;
    const float ref = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
    if (__any(fabsf(ref) > 16777216.f)) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum += fast_exp(x[i] - ref);
        return sum;
    }
    const float r = ref * kLog2e, rest = -__builtin_fmaf(ref, kLog2e, -r);
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], kLog2e, -r));
    return sum * __builtin_amdgcn_exp2f(rest);
}

// x of lane ^ 1, ^ 2, then mirrored in 8 and in 16 lanes, then of lane ^ 16 and ^ 32: six steps after
// which a maximum or minimum covers the wave
template <int LEVEL>
__device__ __forceinline__ float other_lane(float x) {
    if constexpr (LEVEL < 4) {
        constexpr int ctrl = LEVEL == 0 ? 0xB1 : LEVEL == 1 ? 0x4E : LEVEL == 2 ? 0x141 : 0x140;
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), ctrl, 0xF, 0xF, true));
    } else {
        return __shfl_xor(x, LEVEL == 4 ? 16 : 32, 64);
    }
}
template <int LEVEL>
__device__ __forceinline__ float max_min_step(float x, int shift) {
    const float y = other_lane<LEVEL>(x);
    return LEVEL < shift ? fmaxf(x, y) : fminf(x, y);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void beam_scan_kernel(BeamSelectArgs a, SelectPlan plan, int group_shift,
                                                             uint64_t* keys, float2* sums) {
    __shared__ uint64_t s_list[kWaves][kList + 8];
    __shared__ uint64_t s_key[kWaves];
    __shared__ float s_m[kWaves], s_l[kWaves], s_g[2][kWaves];
    __shared__ int s_count[kWaves];
    using R = Round<T>;
    static_assert(kThreads == 256, "the groups' reduction below is written for four waves");
    const int64_t row = blockIdx.x / plan.parts;
    const int part = blockIdx.x % plan.parts, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint64_t* out = keys + (row * plan.parts + part) * a.n_out;
    const T* x0 = static_cast<const T*>(a.logits) + row * a.row_stride;
    // tokens of the part, from `begin` (aligned, before the row for part 0 of a row that is not)
    const int begin = part * plan.per_part - (int)((reinterpret_cast<uintptr_t>(x0) & 15) / sizeof(T));
    const int first = begin < 0 ? 0 : begin, last = begin + plan.per_part < a.V ? begin + plan.per_part : a.V;
    u32x4 next[R::NV];
    bool ready = begin >= 0 && begin + kRound <= last;
    if (ready) R::fetch(x0, begin, next);  // not behind the look at `finished`, whose latency it would add
    if (a.finished && a.finished[row]) {
        // the end token at log-probability 0, then the others in order at -inf
        if (tid < a.n_out) {
            uint64_t k = 0;
            if (part == 0) {
                const int t = tid - 1 < a.eos ? tid - 1 : tid;
                k = tid == 0 ? key_of(0.f, a.eos) : t < a.V ? key_of(-INFINITY, t) : 0;
            }
            out[tid] = k;
        }
        if (tid == 0) sums[row * plan.parts + part] = part == 0 ? make_float2(0.f, 1.f) : make_float2(-INFINITY, 0.f);
        return;
    }
    int mine = 0;  // keys this wave has collected
    float m = -INFINITY, l = 0.f, bar = -INFINITY;  // running maximum and sum of this thread, threshold
    for (int base = begin, turn = 0; base < last; base += kRound, turn ^= 1) {
        const bool whole = ready;
        float x[kPer];
        if (whole) R::values(next, x);
        else R::singles(x0, base, first, last, x);
        // the next round's logits are on their way while this one is worked on
        ready = base + kRound >= 0 && base + 2 * kRound <= last;
        if (ready) R::fetch(x0, base + kRound, next);
        float four[kPer / 4], top = -INFINITY;  // maxima of four logits each, and of all
#pragma unroll
        for (int i = 0; i < kPer / 4; ++i) {
            four[i] = fmaxf(fmaxf(fmaxf(-INFINITY, x[4 * i]), x[4 * i + 1]), fmaxf(x[4 * i + 2], x[4 * i + 3]));
            top = fmaxf(top, four[i]);
        }
        const float now = fmaxf(m, top);
        l = l * fast_exp(m - (now == -INFINITY ? 0.f : now)) + exp_sum(x, now);
        m = now;
        // the least of the maxima of groups of 2^group_shift threads
        float g = top;
        g = max_min_step<0>(g, group_shift);
        g = max_min_step<1>(g, group_shift);
        g = max_min_step<2>(g, group_shift);
        g = max_min_step<3>(g, group_shift);
        g = max_min_step<4>(g, group_shift);
        g = max_min_step<5>(g, group_shift);
        if (lane == 0) s_g[turn][wave] = g;
        __syncthreads();
        g = s_g[turn][0];
        float h = s_g[turn][2];
        g = group_shift > 6 ? fmaxf(g, s_g[turn][1]) : fminf(g, s_g[turn][1]);
        h = group_shift > 6 ? fmaxf(h, s_g[turn][3]) : fminf(h, s_g[turn][3]);
        bar = fmaxf(bar, group_shift > 7 ? fmaxf(g, h) : fminf(g, h));
        // every wave appends to a list of its own, in step, which needs no atomics (-inf is not collected)
        const float least = bar == -INFINITY ? -3.402823466e38f : bar;
#pragma unroll
        for (int q = 0; q < kPer / 4; ++q) {
            if (!__any(four[q] >= least)) continue;
#pragma unroll
            for (int i = 4 * q; i < 4 * q + 4; ++i) {
                const bool in = x[i] >= least;
                const uint64_t mask = __ballot(in);
                if (mask) {
                    const int at = mine + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                                    __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
                    if (in && at < kList) s_list[wave][at] = key_of(x[i], R::token(base, i, whole));
                    mine += __popcll(mask);
                }
            }
        }
    }
    if (__syncthreads_or(l != l)) {  // a NaN (which counts as -inf) or a logit of +inf: the sum once more
        m = -INFINITY;
        l = 0.f;
        for (int base = begin; base < last; base += kRound) {
            float x[kPer], now = m;
            R::load(x0, base, first, last, base >= 0 && base + kRound <= last, x);
#pragma unroll
            for (int i = 0; i < kPer; ++i) now = fmaxf(now, x[i]);
            const float ref = now == -INFINITY ? 0.f : now;
            l *= fast_exp(m - ref);
#pragma unroll
            for (int i = 0; i < kPer; ++i) l += fast_exp(x[i] - ref);
            m = now;
        }
    }
    // log-sum of the part
    float M = m;
    M = max_min_step<0>(M, 6);
    M = max_min_step<1>(M, 6);
    M = max_min_step<2>(M, 6);
    M = max_min_step<3>(M, 6);
    M = max_min_step<4>(M, 6);
    M = max_min_step<5>(M, 6);
    float sum = l * fast_exp(m - (M == -INFINITY ? 0.f : M));
    sum += other_lane<0>(sum);
    sum += other_lane<1>(sum);
    sum += other_lane<2>(sum);
    sum += other_lane<3>(sum);
    sum += other_lane<4>(sum);
    sum += other_lane<5>(sum);
    if (lane == 0) {
        s_m[wave] = M;
        s_l[wave] = sum;
    }
    if (lane == 0) s_count[wave] = mine;
    if (mine < kList && lane < 8) s_list[wave][mine + lane] = 0;  // for the ranks' unrolled loop
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWaves; ++w) M = fmaxf(M, s_m[w]);
        sum = 0.f;
        for (int w = 0; w < kWaves; ++w) sum += s_l[w] * fast_exp(s_m[w] - (M == -INFINITY ? 0.f : M));
        sums[row * plan.parts + part] = make_float2(M, sum);
    }
    int count = 0, most = 0;
    for (int w = 0; w < kWaves; ++w) {
        count += s_count[w];
        most = most > s_count[w] ? most : s_count[w];
    }
    if (most <= kList) {
        if (count < a.n_out && wave == 0) {
            // fewer logits than places are above -inf, and all of those are in the lists: the first of
            // the part's other tokens follow at -inf
            int filled = count;
            for (int t0 = first; t0 < last && filled < a.n_out; t0 += 64) {
                bool other = t0 + lane < last;
                for (int w = 0; w < kWaves; ++w)
                    for (int j = 0; j < s_count[w]; ++j)
                        other = other && 0xFFFFFFFFu - (uint32_t)s_list[w][j] != (uint32_t)(t0 + lane);
                const uint64_t mask = __ballot(other);
                const int at = filled + __popcll(mask & ((1ull << lane) - 1));
                if (other && at < a.n_out) out[at] = key_of(-INFINITY, t0 + lane);
                filled += __popcll(mask);
            }
            if (lane >= filled && lane < a.n_out) out[lane] = 0;
        }
        // the lists' keys one after another over the threads, so that few waves do it
        for (int i = tid; i < count; i += kThreads) {
            int j = i, in = 0;
            while (j >= s_count[in]) j -= s_count[in++];
            const uint64_t k = s_list[in][j];
            int rank = 0;
            for (int w = 0; w < kWaves; ++w)
                for (int j0 = 0; j0 < s_count[w]; j0 += 8) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) rank += s_list[w][j0 + j] > k;
                }
            if (rank < a.n_out) out[rank] = k;
        }
        return;
    }
    // too many at or above the threshold: one maximum of the keys below the last one after another
    uint64_t limit = ~0ull;
    for (int o = 0; o < a.n_out; ++o) {
        uint64_t best = 0;
        for (int base = begin; base < last; base += kRound) {
            const bool whole = base >= 0 && base + kRound <= last;
            float x[kPer];
            R::load(x0, base, first, last, whole, x);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int t = R::token(base, i, whole);
                const uint64_t k = t >= first && t < last ? key_of(x[i], t) : 0;
                if (k < limit && k > best) best = k;
            }
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            const uint64_t y = shfl_xor64(best, off);
            best = y > best ? y : best;
        }
        __syncthreads();
        if (lane == 0) s_key[wave] = best;
        __syncthreads();
        for (int w = 0; w < kWaves; ++w) best = s_key[w] > best ? s_key[w] : best;
        if (tid == 0) out[o] = best;
        limit = best;
    }
}

// A candidate of the join: c, the beam and the key inside the beam.
struct Cand {
    double c;
    uint64_t key;
    int beam;
};
// whether a comes before b
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
    if (a.c != b.c) return a.c > b.c;
    if (a.beam != b.beam) return a.beam < b.beam;
    return a.key > b.key;
}

constexpr int kJoinThreads = 256;  // >= kMaxOut
constexpr int kJoinList = 1024;
constexpr int kPassing = 64;       // lists followed one by one

__global__ __launch_bounds__(kJoinThreads) void beam_join_kernel(BeamSelectArgs a, SelectPlan plan,
                                                                 const uint64_t* keys, const float2* sums) {
    __shared__ double s_lse[kMaxOut], s_score[kMaxOut], s_top[kJoinThreads];
    __shared__ double s_c[kJoinList];
    __shared__ uint64_t s_key[kJoinList];
    __shared__ int s_beam[kJoinList];
    __shared__ Cand s_best[kJoinThreads / 64];
    __shared__ double s_m[kJoinThreads / 64];
    __shared__ int s_count, s_lists, s_pass[kPassing];
    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid == 0) s_count = s_lists = 0;
    // the beams' log-sums: 16 lanes per beam over its parts
    for (int k = tid >> 4; k < a.K; k += kJoinThreads / 16) {
        const float2* y = sums + (b * a.K + k) * plan.parts;
        float M = -INFINITY;
        double sum = 0.;
        for (int p = tid & 15; p < plan.parts; p += 16) M = fmaxf(M, y[p].x);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
        for (int p = tid & 15; p < plan.parts; p += 16)
            if (y[p].y != 0.f) sum += (double)fast_exp(y[p].x - M) * (double)y[p].y;
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
        if ((tid & 15) == 0) {
            s_lse[k] = sum == 0. ? -INFINITY : (double)M + log(sum);
            s_score[k] = (double)a.scores[b * a.K + k];
        }
    }
    __syncthreads();
    const int per_beam = plan.parts * a.n_out, n = a.K * per_beam;
    const uint64_t* ks = keys + b * n;
    auto cand = [&](int i) {
        Cand x;
        x.beam = i / per_beam;
        x.key = ks[i];
        const double c = s_score[x.beam] + (double)unordered((uint32_t)(x.key >> 32)) - s_lse[x.beam];
        x.c = c != c ? -INFINITY : c;
        return x;
    };
    // Threshold: the n_out-th largest of at least n_out candidates.  These are the first `depth` of every
    // part's list, which are in descending order, or their maxima per thread where there are more than
    // threads.
    const int lists = a.K * plan.parts, depth = (a.n_out + lists - 1) / lists, probes = lists * depth;
    const int held = probes < kJoinThreads ? probes : kJoinThreads;
    auto probe = [&](int i) { return cand(depth == 1 ? i * a.n_out : i / depth * a.n_out + i % depth); };
    double top = -INFINITY;
    for (int i = tid; i < probes; i += kJoinThreads) {
        const Cand x = probe(i);
        if (x.key) top = fmax(top, x.c);
    }
    s_top[tid] = top;
    __syncthreads();
    int larger = 0;
    for (int i0 = 0; i0 < held; i0 += 8) {  // threads without a candidate hold -inf
#pragma unroll
        for (int i = 0; i < 8; ++i) larger += s_top[i0 + i] > top;
    }
    double bar = tid < held && larger < a.n_out ? top : INFINITY;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) bar = fmin(bar, __shfl_xor(bar, off, 64));
    if (lane == 0) s_m[wave] = bar;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinThreads / 64; ++w) bar = fmin(bar, s_m[w]);
    auto collect = [&](const Cand& x) {
        if (!x.key || !(x.c >= bar && x.c > -INFINITY)) return;
        const int at = atomicAdd(&s_count, 1);
        if (at < kJoinList) {
            s_c[at] = x.c;
            s_key[at] = x.key;
            s_beam[at] = x.beam;
        }
    };
    if (depth == 1) {
        // only the lists whose first candidate reaches the threshold can have others that do: about n_out
        for (int i = tid; i < lists; i += kJoinThreads) {
            const Cand x = lists <= kJoinThreads && top < bar ? Cand{-INFINITY, 0, 0} : probe(i);
            if (x.key && x.c >= bar && x.c > -INFINITY) {
                const int at = atomicAdd(&s_lists, 1);
                if (at < kPassing) s_pass[at] = i;
            }
        }
        __syncthreads();
        const int found = s_lists;
        if (found <= kPassing) {
            for (int i = tid; i < found * a.n_out; i += kJoinThreads)
                collect(cand(s_pass[i / a.n_out] * a.n_out + i % a.n_out));
        } else {
            for (int i = tid; i < n; i += kJoinThreads) collect(cand(i));
        }
    } else {
        for (int i = tid; i < n; i += kJoinThreads) collect(cand(i));
    }
    __syncthreads();
    auto emit = [&](int o, const Cand& x) {
        const int64_t at = b * a.n_out + o;
        const int token = (int)(0xFFFFFFFFu - (uint32_t)x.key);
        a.scores_out[at] = (float)x.c;
        a.parents[at] = x.beam;
        a.tokens[at] = token;
        if (a.finished) a.finished_out[at] = (a.finished[b * a.K + x.beam] != 0 || token == a.eos) ? 1 : 0;
    };
    const int count = s_count;
    if (count >= a.n_out && count <= kJoinList) {
        for (int i = tid; i < count; i += kJoinThreads) {
            const Cand x{s_c[i], s_key[i], s_beam[i]};
            int rank = 0;
            for (int j0 = 0; j0 < count; j0 += 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = j0 + j < count ? j0 + j : i;  // itself is not before itself
                    rank += before(Cand{s_c[at], s_key[at], s_beam[at]}, x);
                }
            }
            if (rank < a.n_out) emit(rank, x);
        }
        return;
    }
    Cand limit{INFINITY, ~0ull, -1};  // before every candidate
    for (int o = 0; o < a.n_out; ++o) {
        Cand best{-INFINITY, 0, 0x7FFFFFFF};  // behind every candidate
        for (int i = tid; i < n; i += kJoinThreads) {
            const Cand x = cand(i);
            if (x.key && before(limit, x) && before(x, best)) best = x;
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            Cand y;
            y.c = __shfl_xor(best.c, off, 64);
            y.key = shfl_xor64(best.key, off);
            y.beam = __shfl_xor(best.beam, off, 64);
            if (before(y, best)) best = y;
        }
        __syncthreads();
        if (lane == 0) s_best[wave] = best;
        __syncthreads();
        for (int w = 0; w < kJoinThreads / 64; ++w)
            if (before(s_best[w], best)) best = s_best[w];
        if (tid == 0) emit(o, best);
        limit = best;
    }
}

// ------------------------------------------------------------------------------------------
// reorder
// ------------------------------------------------------------------------------------------
// In place without scratch: a thread owns one 16-byte column of all K rows of a group, reads the
// rows it needs into registers and then writes the rows that change, so nobody reads what another
// one has written.  Rows that stay cost nothing, and a row with several children is read from
// memory once.
constexpr int kReorderThreads = 256;

template <int KM>
__global__ __launch_bounds__(kReorderThreads) void beam_reorder_kernel(PoolList pl, const int32_t* parents, int K,
                                                                       int64_t groups) {
    // column group, then state, then group of beams
    int64_t g = blockIdx.x;
    const int64_t cg = g % groups;
    g /= groups;
    const int st = (int)(g % pl.count);
    const int64_t b = g / pl.count;
    const int64_t bytes = pl.bytes[st], at = cg * kReorderThreads * 16;
    if (at >= bytes) return;
    const uint32_t left = bytes - at < kReorderThreads * 16 ? (uint32_t)(bytes - at) : kReorderThreads * 16;
    char* base = pl.base[st] + b * K * bytes + at;
    const int32_t* par = parents + b * K;
    // Every row is loaded and stored, but through a descriptor of no bytes where it stays: nothing is
    // read or written then, and there are no branches (the compiler made one path for each of the 2^K
    // combinations of conditions, 234 registers for K = 8: 77 against 65 us for 128 states of 2 MiB)
    u32x4 x[KM];
    bool moves[KM];
#pragma unroll
    for (int k = 0; k < KM; ++k) {
        int from = k < K ? __builtin_amdgcn_readfirstlane(par[k]) : k;
        moves[k] = from != k && from >= 0 && from < K;
        if (!moves[k]) from = 0;
        x[k] = __builtin_amdgcn_raw_buffer_load_b128(make_rsrc(base + from * bytes, moves[k] ? left : 0),
                                                     threadIdx.x * 16, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < KM; ++k)
        __builtin_amdgcn_raw_buffer_store_b128(x[k], make_rsrc(base + (moves[k] ? k : 0) * bytes, moves[k] ? left : 0),
                                               threadIdx.x * 16, 0, 0);
}

// log2 of the threads per group when 256 threads make at least n_out groups
int group_shift_of(int n_out) {
    int shift = 8;
    while ((1 << (8 - shift)) < n_out) --shift;
    return shift;
}

}  // namespace

int64_t beam_select_groups(int64_t B, int K, int V) { return B * K * select_plan(B * K, V).parts; }

size_t beam_select_workspace(int64_t B, int K, int V, int n_out) {
    const SelectPlan p = select_plan(B * K, V);
    return (size_t)div_up(B * K * p.parts * ((int64_t)n_out + 1) * 8, 256) * 256;
}

hipError_t launch_beam_select(const BeamSelectArgs& a, hipStream_t s) {
    const int64_t rows = (int64_t)a.B * a.K;
    if (rows == 0) return hipSuccess;
    const SelectPlan plan = select_plan(rows, a.V);
    uint64_t* keys = static_cast<uint64_t*>(a.ws);
    float2* sums = reinterpret_cast<float2*>(keys + rows * plan.parts * a.n_out);
    const int shift = group_shift_of(a.n_out);
    const bool timed = timing_on();
    if (timed) timed_begin(kKernelBeamScan, s);
    const dim3 grid((unsigned)(rows * plan.parts));
    if (a.bf16)
        hipLaunchKernelGGL(beam_scan_kernel<uint16_t>, grid, dim3(kThreads), 0, s, a, plan, shift, keys, sums);
    else
        hipLaunchKernelGGL(beam_scan_kernel<float>, grid, dim3(kThreads), 0, s, a, plan, shift, keys, sums);
    hipError_t e = hipGetLastError();
    if (timed) timed_end(s);
    if (e != hipSuccess) return e;
    if (timed) timed_begin(kKernelBeamJoin, s);
    hipLaunchKernelGGL(beam_join_kernel, dim3((unsigned)a.B), dim3(kJoinThreads), 0, s, a, plan, keys, sums);
    e = hipGetLastError();
    if (timed) timed_end(s);
    return e;
}

static hipError_t launch_reorder_slice(const PoolList& p, const int32_t* parents, int64_t B, int K, int64_t groups,
                                       hipStream_t s) {
    const dim3 grid((unsigned)(groups * p.count * B)), block(kReorderThreads);
    const bool timed = timing_on();
    if (timed) timed_begin(kKernelBeamReorder, s);
    if (K <= 4) hipLaunchKernelGGL(beam_reorder_kernel<4>, grid, block, 0, s, p, parents, K, groups);
    else if (K <= 8) hipLaunchKernelGGL(beam_reorder_kernel<8>, grid, block, 0, s, p, parents, K, groups);
    else if (K <= 16) hipLaunchKernelGGL(beam_reorder_kernel<16>, grid, block, 0, s, p, parents, K, groups);
    else if (K <= 32) hipLaunchKernelGGL(beam_reorder_kernel<32>, grid, block, 0, s, p, parents, K, groups);
    else hipLaunchKernelGGL(beam_reorder_kernel<64>, grid, block, 0, s, p, parents, K, groups);
    const hipError_t e = hipGetLastError();
    if (timed) timed_end(s);
    return e;
}

hipError_t launch_beam_reorder(const PoolList& p, const int32_t* parents, int B, int K, hipStream_t s) {
    int64_t most = 0;
    for (int i = 0; i < p.count; ++i) most = p.bytes[i] > most ? p.bytes[i] : most;
    if (B == 0 || K <= 1 || most == 0) return hipSuccess;
    // in slices of the states and of the groups of beams where a grid does not hold them
    const int64_t groups = div_up(most, kReorderThreads * 16), fit = max_groups(kReorderThreads) / groups;
    hipError_t e = hipSuccess;
    for (int i0 = 0; i0 < p.count && e == hipSuccess; i0 += (int)fit) {
        PoolList part = p;
        part.count = p.count - i0 < fit ? p.count - i0 : (int)fit;
        const int64_t step = fit / part.count;
        for (int64_t b0 = 0; b0 < B && e == hipSuccess; b0 += step) {
            for (int i = 0; i < part.count; ++i) {
                part.bytes[i] = p.bytes[i0 + i];
                part.base[i] = p.base[i0 + i] + b0 * K * part.bytes[i];
            }
            e = launch_reorder_slice(part, parents + b0 * K, B - b0 < step ? B - b0 : step, K, groups, s);
        }
    }
    return e;
}

}  // namespace kda
