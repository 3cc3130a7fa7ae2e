// Log-probabilities of given tokens with the row's log-sum, entropy and best alternatives, and their gradient with
// respect to the logits (include/kda.h, kda_token_logprobs and kda_token_logprobs_grad).
//
// With x a row of logits:  lse = log sum_u exp(x_u),   logprob = x_token - lse,
//     H = -sum_u p_u log p_u = lse - sum_u p_u x_u,   p_u = exp(x_u - lse).
// One pass gives everything: a running maximum m, the sum l of exp(x - m), and for the entropy s, the sum of
// exp(x - m) (x - m), from which H = log l - s / l.  The bytes of the logits bound it, with the vector units close
// behind: a bf16 logit has 12 instruction slots of a lane while it arrives at 6 TB/s, and its exponential
// takes four of them.  So everything else is kept to a few per logit:
//  * A thread keeps a reference m of its own, which moves only when a round's maximum is more than 1 above it (a
//    branch that a wave takes a few times per row).  With r = fl(m log2 e), exp(x - m) = 2^(x log2 e - r) 2^rest,
//    rest = r - m log2 e: one fused product and sum and one exponential per logit, the last factor once for all.
//    Beyond |m| = 2^24, where rest leaves [-1, 1], the difference x - m is taken first.
//  * Best alternatives: the n-th largest of the maxima so far of 64 disjoint groups of threads is a lower bound of the
//    n-th best logit; its upper 16 bits are found by 16 counts over a wave.  It is taken again in rounds 0, 1, 2, 4,
//    8, ..., since it moves less and less; the logits at or above it are collected into lists, those below the last
//    bound taken out, and the rest ranked by (value, token) at the end.  Lists that are too long to rank, or overflow,
//    are made again with the bound in all its bits, the latter from the row once more: a long stretch of equal logits
//    before better ones (a mask of a finite value), and fp32 logits whose offset is large against their spread (of 100 +-
//    0.1 half of a row is at or above the 100.0 of the upper bits; 2048 rows of 50257 of them, 20 best: 136 us, others
//    71, 1377 without those bits).  Where that overflows too (equal logits at the bound), the row is read once for each
//    place (all equal, 20 best: 1360 us).  (2048 rows of 50257 in bf16: 20 best with the entropy 58 us, 115 with the
//    least of the maxima of 32 groups as the bound, which lets five times as many logits pass; 5 best 53, none 43.)
//  * A row belongs to one wave where it is short, to a workgroup where it is not, and to several workgroups where
//    there are few rows; a second launch joins their parts.
//  * Logits and gradients of more than the 256 MB of the memory's own cache pass the caches by: 4096 rows of 131072 in
//    bf16, 184 to 195 us by the card, 5.5 to 5.8 TB/s (8 us more without); their gradient 341 to 344 us, 6.2 TB/s (373).
//    Less of them stays there from the product before: 2048 rows of 50257, 205 MB, 42 us, past the caches 44.
#include <math.h>

#include <type_traits>

#include "kda_device.h"
#include "kda_internal.h"
#include "kda_rows.h"

namespace kda {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxTop = 64;
constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPer = 16;       // logits of a thread per round
constexpr int kList = 512;     // collected keys of a wave (the best 64 of one round come with 270 on average, 6 rows of
                               // 3315 logits took 131 us with lists of 256, 68 now)
constexpr int kMaxParts = 64;
template <int N>
using Bits = std::integral_constant<int, N>;
constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.6931471805599453;

// 16 bytes; PASS: the caches are left to others
template <bool PASS>
__device__ __forceinline__ u32x4 load_16(const void* at) {
    const u32x4* p = static_cast<const u32x4*>(at);
    return PASS ? __builtin_nontemporal_load(p) : *p;
}

// The logits of a thread's round.  `wide`: the round lies inside the part and is read in 16-byte vectors; else the
// tokens are strided over the threads, and those outside of the part become -inf.
template <typename T, int TPR>
struct Rounds {
    static constexpr int W = 16 / sizeof(T), NV = kPer / W, SIZE = TPR * kPer;
    static __device__ __forceinline__ int token(int base, int i, bool wide, int t) {
        return wide ? base + (i / W) * TPR * W + t * W + i % W : base + i * TPR + t;
    }
    template <bool PASS>
    static __device__ __forceinline__ void fetch(const T* row, int base, int t, u32x4 (&raw)[NV]) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            raw[v] = load_16<PASS>(row + base + v * TPR * W + t * W);
    }
    static __device__ __forceinline__ void values(const u32x4 (&raw)[NV], float (&x)[kPer]) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t word = raw[i / W][(i % W) * sizeof(T) / 4];
            if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(word);
            else x[i] = __uint_as_float((i & 1) ? word & 0xFFFF0000u : word << 16);
        }
    }
    // first < last
    static __device__ __forceinline__ void cut(const T* row, int base, int first, int last, int t, float (&x)[kPer]) {
        T raw[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = token(base, i, false, t);
            raw[i] = row[at < first ? first : at >= last ? last - 1 : at];
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = token(base, i, false, t);
            x[i] = at >= first && at < last ? ld_in(raw, i) : -INFINITY;
        }
    }
};

// A thread's running sums: l and s are in units of 2^-rest, s in base 2.
template <bool ENT>
struct Sums {
    float m = -INFINITY, ref = 0.f, r = 0.f, rest = 0.f, l = 0.f, s = 0.f;

    __device__ __forceinline__ void to_true(float& L, float& S) const {
        const float f = exp2_hw(rest);
        L = l * f;
        S = ENT ? f * (s + rest * l) : 0.f;
    }
    __device__ __forceinline__ void move(float top) {
        float L, S;
        to_true(L, S);
        const float d = (ref - top) * kLog2e, f = l == 0.f ? 0.f : exp2_hw(d);
        S = f == 0.f ? 0.f : f * (S + L * d);
        L = L * f;
        m = ref = top;
        const bool far = fabsf(top) > 16777216.f;
        r = far ? 0.f : top * kLog2e;
        rest = far ? 0.f : -__builtin_fmaf(top, kLog2e, -r);
        const float g = exp2_hw(-rest);
        l = L * g;
        if (ENT) s = S * g - rest * l;
    }
    // CLEAN: NaN has been made -inf, and a reference of +inf adds nothing
    template <bool CLEAN>
    __device__ __forceinline__ void add(const float (&x)[kPer], float top) {
        const bool up = top > m + 1.f || (m == -INFINITY && top > m);
        if (__any(up)) {
            if (up) move(top);
        }
        if (CLEAN && m == INFINITY) {
            l = 1.f;
            s = 0.f;
            return;
        }
        float z[kPer];
        if (__any(fabsf(ref) > 16777216.f)) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) z[i] = __builtin_fmaf(x[i] - ref, kLog2e, -rest);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) z[i] = __builtin_fmaf(x[i], kLog2e, -r);
        }
        float p[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) p[i] = exp2_hw(z[i]);
        // four sums side by side
        float a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = (p[i] + p[i + 4]) + (p[i + 8] + p[i + 12]);
            if (ENT) {
                b[i] = 0.f;  // (a weight of 0 times its exponent of -inf is 0)
#pragma unroll
                for (int j = 0; j < kPer; j += 4) b[i] = __builtin_fmaf(p[i + j], fmaxf(z[i + j], -1e30f), b[i]);
            }
        }
        l += (a[0] + a[1]) + (a[2] + a[3]);
        if (ENT) s += (b[0] + b[1]) + (b[2] + b[3]);
    }
};

// (maximum, sum, base-2 entropy sum) of two parts
struct Part {
    float m, l, s;
};
__device__ __forceinline__ Part joined(Part a, Part b) {
    const float m = fmaxf(a.m, b.m);
    auto take = [&](const Part& p, float& l, float& s) {
        const float d = p.m == m ? 0.f : (p.m - m) * kLog2e, f = p.l == 0.f ? 0.f : exp2_hw(d);
        l += p.l * f;
        if (f != 0.f) s += f * (p.s + p.l * d);
    };
    Part c{m, 0.f, 0.f};
    take(a, c.l, c.s);
    take(b, c.l, c.s);
    return c;
}
__device__ __forceinline__ Part over_wave(Part p) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        Part q;
        q.m = __shfl_xor(p.m, off, 64);
        q.l = __shfl_xor(p.l, off, 64);
        q.s = __shfl_xor(p.s, off, 64);
        p = joined(p, q);
    }
    return p;
}

// What one thread writes for a row; returns the log-sum in fp64.
template <typename T>
__device__ __forceinline__ double finish(const LogprobArgs& a, int64_t row, const Part& p) {
    const double log_l = p.l > 0.f ? log((double)p.l) : 0.;
    const bool fine = p.l > 0.f && fabsf(p.m) != INFINITY;
    const double lse = fine ? (double)p.m + log_l : p.m == INFINITY ? INFINITY : -INFINITY;
    if (a.lse) a.lse[row] = (float)lse;
    if (a.entropy) {
        const double h = fine ? log_l - (double)p.s / (double)p.l * kLn2 : 0.;
        a.entropy[row] = h > 0. ? (float)h : 0.f;
    }
    if (a.logprobs) {
        const int t = a.tokens[row];
        float y = 0.f;
        if (t >= 0 && t < a.V) {
            const double d = (double)clean(ld_in(static_cast<const T*>(a.logits) + row * a.row_stride, t)) - lse;
            y = d == d ? (float)d : -INFINITY;
        }
        a.logprobs[row] = y;
    }
    return lse;
}
__device__ __forceinline__ void put_best(const LogprobArgs& a, int64_t row, int i, uint64_t key, double lse) {
    const double d = (double)unordered((uint32_t)(key >> 32)) - lse;
    a.top_logprobs[row * a.top + i] = d == d ? (float)d : -INFINITY;
    a.top_tokens[row * a.top + i] = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
}

struct LogprobPlan {
    int waves;     // of a row's part: 1 or 4
    int parts;     // of a row
    int per_part;  // tokens of a part, a multiple of a round
};

template <typename T, int WPR, bool TOP, bool ENT, bool PASS>
__global__ __launch_bounds__(kThreads) void logprob_scan_kernel(LogprobArgs a, LogprobPlan plan, uint64_t* keys,
                                                                float4* sums) {
    constexpr int TPR = 64 * WPR;
    using R = Rounds<T, TPR>;
    __shared__ uint64_t s_list[TOP ? kWaves : 1][TOP ? kList + 8 : 1], s_best[TOP ? kWaves : 1][TOP ? kMaxTop : 1];
    __shared__ float s_m[kWaves], s_l[kWaves], s_s[kWaves], s_g[2][64];
    __shared__ double s_lse;
    __shared__ int s_count[kWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = WPR == 1 ? lane : (int)threadIdx.x;         // thread of the row
    const int w0 = WPR == 1 ? wave : 0;                       // first wave of the row
    const int64_t item = WPR == 1 ? (int64_t)blockIdx.x * kWaves + wave : (int64_t)blockIdx.x;
    const int64_t row = item / plan.parts;
    const int part = (int)(item - row * plan.parts);
    if (row >= a.R) return;  // (a wave of its own: no barrier below)
    auto sync = [] {
        if constexpr (WPR == 1) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        } else {
            __syncthreads();
        }
    };
    const T* x0 = static_cast<const T*>(a.logits) + row * a.row_stride;
    // tokens of the part, from `begin` (aligned, before the row for part 0 of a row that is not)
    const int begin = part * plan.per_part - (int)((reinterpret_cast<uintptr_t>(x0) & 15) / sizeof(T));
    const int first = begin < 0 ? 0 : begin, last = begin + plan.per_part < a.V ? begin + plan.per_part : a.V;

    Sums<ENT> sum;
    float most = -INFINITY, bar = -INFINITY;  // this thread's maximum, the row's bound
    int mine = 0, turns = 0;                  // keys this wave has collected
    auto raise = [&](auto bits) {  // the n-th largest of the maxima of 64 groups of threads, by its upper bits
        constexpr int BITS = decltype(bits)::value, LOW = 32 - BITS;
        float g = most;
        if constexpr (WPR == 4) {
            g = max_min_step<0>(g, 2);
            g = max_min_step<1>(g, 2);
            const int turn = turns++ & 1;
            if ((lane & 3) == 0) s_g[turn][wave * 16 + lane / 4] = g;
            __syncthreads();
            g = s_g[turn][lane];
        }
        const uint32_t u = ordered(g) >> LOW;
        uint32_t least = 0;
#pragma unroll
        for (int bit = BITS - 1; bit >= 0; --bit) {
            const uint32_t more = least | 1u << bit;
            least = __popcll(__ballot(u >= more)) >= a.top ? more : least;
        }
        bar = least << LOW > ordered(-INFINITY) ? unordered(least << LOW) : -INFINITY;
    };
    auto collect = [&](const float (&x)[kPer], float top, int base, bool wide) {
        const float least = bar == -INFINITY ? -3.402823466e38f : bar;  // -inf is not collected
        if (!__any(top >= least)) return;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const bool in = x[i] >= least;
            const uint64_t mask = __ballot(in);
            if (mask) {
                const int at = mine + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                                __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
                if (in && at < kList) s_list[wave][at] = key_of(x[i], R::token(base, i, wide, t));
                mine += __popcll(mask);
            }
        }
    };
    auto filter = [&] {  // this wave's keys below the bound leave its list
        if (bar == -INFINITY || mine > kList) return;
        const uint32_t least = ordered(bar + 0.f);
        int kept = 0;
        for (int i0 = 0; i0 < mine; i0 += 64) {
            const uint64_t k = s_list[wave][i0 + lane < mine ? i0 + lane : 0];
            const uint64_t mask = __ballot(i0 + lane < mine && (uint32_t)(k >> 32) >= least);
            const int at = kept + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                            __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
            if (mask >> lane & 1) s_list[wave][at] = k;  // (not behind what has been read)
            kept += __popcll(mask);
        }
        mine = kept;
    };
    // (the maxima leave out NaN)
    auto top_of = [](const float (&x)[kPer]) {
        float y = -INFINITY;
#pragma unroll
        for (int i = 0; i < kPer; i += 2) y = fmaxf(fmaxf(y, x[i]), x[i + 1]);
        return y;
    };

    u32x4 next[R::NV];
    bool ready = begin >= 0 && begin + R::SIZE <= last;
    if (ready) R::template fetch<PASS>(x0, begin, t, next);
    int round = 0;
    for (int base = begin; base < last; base += R::SIZE, ++round) {
        const bool wide = ready;
        float x[kPer];
        if (wide) R::values(next, x);
        else R::cut(x0, base, first, last, t, x);
        ready = base + R::SIZE >= 0 && base + 2 * R::SIZE <= last;
        if (ready) R::template fetch<PASS>(x0, base + R::SIZE, t, next);  // on its way while this one is worked on
        const float top = top_of(x);
        sum.template add<false>(x, top);
        if constexpr (TOP) {
            most = fmaxf(most, top);
            if ((round & (round - 1)) == 0) {
                raise(Bits<16>());
                if (mine > kList / 2) filter();
            }
            collect(x, top, base, wide);
        }
    }
    bool odd = sum.l != sum.l;
    if (WPR == 1 ? __any(odd) : __syncthreads_or(odd)) {  // a NaN (which counts as -inf) or +inf: the sums once more
        sum = Sums<ENT>();
        for (int base = begin; base < last; base += R::SIZE) {
            float x[kPer];
            R::cut(x0, base, first, last, t, x);
#pragma unroll
            for (int i = 0; i < kPer; ++i) x[i] = clean(x[i]);
            sum.template add<true>(x, top_of(x));
        }
    }
    Part p{sum.m, 0.f, 0.f};
    sum.to_true(p.l, p.s);
    p = over_wave(p);
    if constexpr (WPR == 4) {
        if (lane == 0) {
            s_m[wave] = p.m;
            s_l[wave] = p.l;
            s_s[wave] = p.s;
        }
        __syncthreads();
        p = Part{s_m[0], s_l[0], s_s[0]};
#pragma unroll
        for (int w = 1; w < kWaves; ++w) p = joined(p, Part{s_m[w], s_l[w], s_s[w]});
    }
    double lse = 0.;
    if (plan.parts > 1) {
        if (t == 0) sums[row * plan.parts + part] = make_float4(p.m, p.l, p.s, 0.f);
    } else if (t == 0) {
        lse = finish<T>(a, row, p);
    }
    if constexpr (!TOP) return;
    raise(Bits<16>());
    filter();

    // the row's best, in order
    auto counts = [&](int& total) {  // of the row's waves; whether a list has overflowed
        if (mine < kList && lane < 8) s_list[wave][mine + lane] = 0;  // for the ranks' unrolled loop
        if (WPR == 1) {
            total = mine;
            return mine > kList;
        }
        __syncthreads();
        if (lane == 0) s_count[wave] = mine;
        __syncthreads();
        total = 0;
        int full = 0;
        for (int w = 0; w < kWaves; ++w) {
            total += s_count[w];
            full |= s_count[w] > kList;
        }
        return full != 0;
    };
    int total;
    bool full = counts(total);
    // Too many: those at or above the bound in all its bits (bf16 has no others), of the lists or of the row once more.
    if (full || (sizeof(T) == 4 && total > kList)) {
        raise(Bits<8 * sizeof(T)>());
        if (full) {
            mine = 0;
            for (int base = begin; base < last; base += R::SIZE) {
                float x[kPer];
                R::cut(x0, base, first, last, t, x);
                collect(x, top_of(x), base, false);
            }
        } else {
            filter();
        }
        full = counts(total);
    }
    uint64_t* best = s_best[w0];
    if (!full) {
        sync();
        if (total < a.top && (WPR == 1 || wave == 0)) {
            // fewer logits than places are above -inf, and all of those are in the lists: the first of the part's
            // other tokens follow at -inf
            int filled = total;
            for (int at0 = first; at0 < last && filled < a.top; at0 += 64) {
                bool other = at0 + lane < last;
                for (int w = w0; w < w0 + WPR; ++w) {
                    const int n = WPR == 1 ? mine : s_count[w];
                    for (int j = 0; j < n; ++j)
                        other = other && 0xFFFFFFFFu - (uint32_t)s_list[w][j] != (uint32_t)(at0 + lane);
                }
                const uint64_t mask = __ballot(other);
                const int at = filled + __popcll(mask & ((1ull << lane) - 1));
                if (other && at < a.top) best[at] = key_of(-INFINITY, at0 + lane);
                filled += __popcll(mask);
            }
            if (lane >= filled && lane < a.top) best[lane] = 0;
        }
        for (int i = t; i < total; i += TPR) {
            int j = i, in = w0;
            if constexpr (WPR == 4)
                while (j >= s_count[in]) j -= s_count[in++];
            const uint64_t k = s_list[in][j];
            int rank = 0;
            for (int w = w0; w < w0 + WPR; ++w) {
                const int n = WPR == 1 ? mine : s_count[w];
                for (int j0 = 0; j0 < n; j0 += 8) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) rank += s_list[w][j0 + e] > k;
                }
            }
            if (rank < a.top) best[rank] = k;
        }
    } else {  // too many at the bound: one maximum of the keys below the last one after another
        uint64_t limit = ~0ull;
        for (int o = 0; o < a.top; ++o) {
            uint64_t top = 0;
            for (int base = begin; base < last; base += R::SIZE) {
                float x[kPer];
                R::cut(x0, base, first, last, t, x);
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int at = R::token(base, i, false, t);
                    const uint64_t k = at >= first && at < last ? key_of(clean(x[i]), at) : 0;
                    if (k < limit && k > top) top = k;
                }
            }
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) {
                const uint64_t y = shfl_xor64(top, off);
                top = y > top ? y : top;
            }
            if constexpr (WPR == 4) {
                __syncthreads();
                if (lane == 0) s_list[wave][0] = top;
                __syncthreads();
                for (int w = 0; w < kWaves; ++w) top = s_list[w][0] > top ? s_list[w][0] : top;
            }
            if (t == 0) best[o] = top;
            limit = top;
        }
    }
    if constexpr (WPR == 4) {
        if (t == 0) s_lse = lse;
    } else {
        lse = __shfl(lse, 0, 64);
    }
    sync();
    if constexpr (WPR == 4) lse = s_lse;
    if (t < a.top) {
        if (plan.parts > 1) keys[(row * plan.parts + part) * a.top + t] = best[t];
        else put_best(a, row, t, best[t], lse);
    }
}

// Join of a row's parts: a wave for a row, its lanes over the parts, whose lists are in order.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprob_join_kernel(LogprobArgs a, LogprobPlan plan, const uint64_t* keys,
                                                                const float4* sums) {
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (row >= a.R) return;
    const bool on = lane < plan.parts;
    const float4 y = sums[row * plan.parts + (on ? lane : 0)];
    const uint64_t* mine = keys + (row * plan.parts + (on ? lane : 0)) * a.top;
    uint64_t head = on && a.top ? mine[0] : 0, next = on && a.top > 1 ? mine[1] : 0;
    const Part p = over_wave(on ? Part{y.x, y.y, y.z} : Part{-INFINITY, 0.f, 0.f});
    double lse = 0.;
    if (lane == 0) lse = finish<T>(a, row, p);
    lse = __shfl(lse, 0, 64);
    int at = 0;
    uint64_t got = 0;  // lane o: the o-th best
    for (int o = 0; o < a.top; ++o) {
        // the first lane with the largest value: the parts' tokens ascend
        const float value = head ? unordered((uint32_t)(head >> 32)) : -INFINITY;
        float top = value;
        top = max_min_step<0>(top, 6);
        top = max_min_step<1>(top, 6);
        top = max_min_step<2>(top, 6);
        top = max_min_step<3>(top, 6);
        top = max_min_step<4>(top, 6);
        top = max_min_step<5>(top, 6);
        const uint64_t among = __ballot(head != 0 && value == top);
        if (among == 0) break;
        const int from = __builtin_ctzll(among);
        const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)head, from);
        const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(head >> 32), from);
        if (lane == o) got = (uint64_t)hi << 32 | lo;
        if (lane == from) {
            head = next;
            next = ++at + 1 < a.top ? mine[at + 1] : 0;
        }
    }
    if (lane < a.top) put_best(a, row, lane, got, lse);
}

// ------------------------------------------------------------------------------------------
// gradient
// ------------------------------------------------------------------------------------------
// dx_v = p_v (d_lse - d_logprob - d_H (log p_v + H)) + d_logprob [v = token].  Pure traffic in small pieces: a wave
// takes 64 x 16 logits of a row.
template <typename T, bool ENT, bool PASS>
__global__ __launch_bounds__(kThreads) void logprob_grad_kernel(LogprobGradArgs a, int chunks) {
    constexpr int W = 16 / sizeof(T), NV = kPer / W, SPAN = 64 * kPer;
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = item / chunks;
    if (row >= a.R) return;
    const T* x0 = static_cast<const T*>(a.logits) + row * a.row_stride;
    T* y0 = static_cast<T*>(a.d_logits) + row * a.out_stride;
    const int phase = (int)((reinterpret_cast<uintptr_t>(x0) & 15) / sizeof(T));
    const bool alike = (reinterpret_cast<uintptr_t>(y0) & 15) == (reinterpret_cast<uintptr_t>(x0) & 15);
    const int base = (int)(item - row * chunks) * SPAN - phase;
    if (base >= a.V) return;
    const bool wide = alike && base >= 0 && base + SPAN <= a.V;
    u32x4 raw[NV];
    T one[kPer];
    if (wide) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            raw[v] = load_16<PASS>(x0 + base + v * 64 * W + lane * W);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = base + i * 64 + lane;
            one[i] = x0[at < 0 ? 0 : at >= a.V ? a.V - 1 : at];
        }
    }
    const float lse = a.lse[row];
    const int token = a.tokens ? a.tokens[row] : -1;
    const bool fine = fabsf(lse) < INFINITY;
    const float d = fine && token >= 0 && token < a.V && a.d_logprobs ? a.d_logprobs[row] : 0.f;
    const float flat = (a.d_lse ? a.d_lse[row] : 0.f) - d;
    const float dh = ENT ? a.d_entropy[row] : 0.f, h = ENT ? a.entropy[row] : 0.f;
    auto grad = [&](float x) {
        const float lp = x - lse, p = exp2_hw(lp * kLog2e);
        const float y = p * (ENT ? __builtin_fmaf(-dh, lp + h, flat) : flat);
        return p > 0.f && fine ? y : 0.f;  // weights of 0 and NaN
    };
    if (wide) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = base + v * 64 * W + lane * W;
            float g[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const uint32_t word = raw[v][i * sizeof(T) / 4];
                g[i] = grad(sizeof(T) == 4 ? __uint_as_float(word)
                                           : __uint_as_float((i & 1) ? word & 0xFFFF0000u : word << 16));
            }
            if ((unsigned)(token - c0) < (unsigned)W) {
#pragma unroll
                for (int i = 0; i < W; ++i) g[i] += token - c0 == i ? d : 0.f;
            }
            u32x4 out;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 4) {
                    out[i] = __float_as_uint(g[i]);
                } else {
                    out[i] = pack_bf16(g[2 * i], g[2 * i + 1]);
                }
            }
            if constexpr (PASS) __builtin_nontemporal_store(out, reinterpret_cast<u32x4*>(y0 + c0));
            else *reinterpret_cast<u32x4*>(y0 + c0) = out;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = base + i * 64 + lane;
            if (at < 0 || at >= a.V) continue;
            const float g = grad(ld_in(one, i)) + (at == token ? d : 0.f);
            if constexpr (sizeof(T) == 4) y0[at] = g;
            else y0[at] = __builtin_bit_cast(uint16_t, (__bf16)g);
        }
    }
}

// Whether so many bytes pass the caches by.
bool pass_by(int64_t bytes) { return bytes > (int64_t)256 << 20; }

LogprobPlan plan_of(int64_t R, int V) {
    LogprobPlan p;
    // a wave per row up to two of a workgroup's rounds
    p.waves = V <= 2 * kThreads * kPer ? 1 : kWaves;
    const int64_t size = 64 * p.waves * kPer, rounds = div_up((int64_t)V + 7, size);
    // with few rows, parts for about four waves per SIMD
    int64_t parts = div_up(1024, R < 1 ? 1 : R);
    parts = parts > kMaxParts ? kMaxParts : parts;
    parts = parts > rounds ? rounds : parts;
    const int64_t per = div_up(rounds, parts);
    p.parts = (int)div_up(rounds, per);
    p.per_part = (int)(per * size);
    return p;
}

template <typename T, int WPR, bool TOP>
void launch_scan(const LogprobArgs& a, const LogprobPlan& p, uint64_t* keys, float4* sums, hipStream_t s) {
    const int64_t items = a.R * p.parts;
    const dim3 grid((unsigned)(WPR == 1 ? div_up(items, kWaves) : items)), block(kThreads);
    const bool past = WPR == kWaves && pass_by(a.R * a.V * (int64_t)sizeof(T));
    if (past) {
        if (a.entropy) hipLaunchKernelGGL((logprob_scan_kernel<T, WPR, TOP, true, WPR == kWaves>), grid, block, 0, s, a, p, keys, sums);
        else hipLaunchKernelGGL((logprob_scan_kernel<T, WPR, TOP, false, WPR == kWaves>), grid, block, 0, s, a, p, keys, sums);
    } else {
        if (a.entropy) hipLaunchKernelGGL((logprob_scan_kernel<T, WPR, TOP, true, false>), grid, block, 0, s, a, p, keys, sums);
        else hipLaunchKernelGGL((logprob_scan_kernel<T, WPR, TOP, false, false>), grid, block, 0, s, a, p, keys, sums);
    }
}
template <typename T>
void launch_scan(const LogprobArgs& a, const LogprobPlan& p, uint64_t* keys, float4* sums, hipStream_t s) {
    if (p.waves == 1) {
        if (a.top) launch_scan<T, 1, true>(a, p, keys, sums, s);
        else launch_scan<T, 1, false>(a, p, keys, sums, s);
    } else {
        if (a.top) launch_scan<T, kWaves, true>(a, p, keys, sums, s);
        else launch_scan<T, kWaves, false>(a, p, keys, sums, s);
    }
}

int64_t sums_bytes(int64_t R, const LogprobPlan& p) { return div_up(R * p.parts * (int64_t)sizeof(float4), 256) * 256; }

int64_t grad_chunks(int V) { return div_up((int64_t)V + 7, 64 * kPer); }

template <typename T, bool ENT>
void launch_grad(const LogprobGradArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)logprob_grad_groups(a.R, a.V)), block(kThreads);
    const int chunks = (int)grad_chunks(a.V);
    if (pass_by(2 * a.R * a.V * (int64_t)sizeof(T)))
        hipLaunchKernelGGL((logprob_grad_kernel<T, ENT, true>), grid, block, 0, s, a, chunks);
    else hipLaunchKernelGGL((logprob_grad_kernel<T, ENT, false>), grid, block, 0, s, a, chunks);
}
template <typename T>
void launch_grad(const LogprobGradArgs& a, hipStream_t s) {
    if (a.d_entropy) launch_grad<T, true>(a, s);
    else launch_grad<T, false>(a, s);
}

}  // namespace

int64_t logprob_groups(int64_t R, int V) { return R * plan_of(R, V).parts; }

size_t logprob_workspace(int64_t R, int V, int top) {
    const LogprobPlan p = plan_of(R, V);
    if (p.parts == 1 || R == 0) return 0;
    return (size_t)(sums_bytes(R, p) + R * p.parts * top * (int64_t)sizeof(uint64_t));
}

hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t s) {
    if (a.R == 0) return hipSuccess;
    const LogprobPlan p = plan_of(a.R, a.V);
    float4* sums = static_cast<float4*>(a.ws);
    uint64_t* keys = p.parts > 1 ? reinterpret_cast<uint64_t*>(static_cast<char*>(a.ws) + sums_bytes(a.R, p)) : nullptr;
    const bool timed = timing_on();
    if (timed) timed_begin(kKernelLogprobScan, s);
    if (a.bf16) launch_scan<uint16_t>(a, p, keys, sums, s);
    else launch_scan<float>(a, p, keys, sums, s);
    hipError_t e = hipGetLastError();
    if (timed) timed_end(s);
    if (e != hipSuccess || p.parts == 1) return e;
    if (timed) timed_begin(kKernelLogprobJoin, s);
    const dim3 grid((unsigned)div_up(a.R, kWaves)), block(kThreads);
    if (a.bf16) hipLaunchKernelGGL(logprob_join_kernel<uint16_t>, grid, block, 0, s, a, p, keys, sums);
    else hipLaunchKernelGGL(logprob_join_kernel<float>, grid, block, 0, s, a, p, keys, sums);
    e = hipGetLastError();
    if (timed) timed_end(s);
    return e;
}

int64_t logprob_grad_groups(int64_t R, int V) { return div_up(R * grad_chunks(V), kWaves); }

hipError_t launch_logprob_grad(const LogprobGradArgs& a, hipStream_t s) {
    if (a.R == 0) return hipSuccess;
    const bool timed = timing_on();
    if (timed) timed_begin(kKernelLogprobGrad, s);
    if (a.bf16) launch_grad<uint16_t>(a, s);
    else launch_grad<float>(a, s);
    const hipError_t e = hipGetLastError();
    if (timed) timed_end(s);
    return e;
}

}  // namespace kda
