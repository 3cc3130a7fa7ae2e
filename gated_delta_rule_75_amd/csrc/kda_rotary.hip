// Rotary positions of queries and keys, to tensors or straight into a cache's pages (include/kda.h,
// kda_rotary and kda_rotary_append).
//
// Pair i < r / 2 of a token at position p is turned by the angle a = p f_i:
//     (x, y) -> amplitude (x cos a - y sin a, x sin a + y cos a)
// with x, y the channels i, i + r / 2 (halves) or 2 i, 2 i + 1 (interleaved); channels from r on are copied.
//
// Pure traffic: every value is read once and written once.  The angles must not add to it.
//  * A workgroup takes one token, or as many of few heads as its threads have two steps for.  It forms the cosines
//    and sines of each pair once, in LDS, for all heads of its tokens; p f is an fp64 product and is reduced by
//    multiples of 2 pi there (a position of 2^17 in fp32 would be off by 2^-7 rad), the rest is fp32.
//  * The first values are asked for before the angles are formed, so that these hide behind the loads.  Many small
//    workgroups keep the chip's loads and stores apart in time better than few large ones, and neither is kept in the
//    caches (non-temporal).  65536 tokens of 32 + 32 heads of 128, bf16: 361 to 375 us by the card, 5.7 to 5.9 TB/s (on
//    the faster one 16 tokens a workgroup: 438, 8: 417, 4: 402, without the hint for stores 382; a copy of that size: 420).
//    Into pages, segments of 1K to 16K tokens, 8 in all: 196 to 200 us, 6.0 TB/s, where the hint for stores saves 24 us and
//    the attention behind it takes as long as before.
//  * A thread always has the same place in a row.  Halves that start at 16-byte boundaries: a vector of the first
//    half and its partner.  Interleaved: pairs lie inside one vector.  Halves that do not (r / 2 no multiple of a
//    vector): the rows of a step are laid into LDS, from where each thread takes its partners (5.9 TB/s too).
// One query head and one key head of 64 share their angles with no other: 3.3 TB/s, bound by the angles.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kMaxTokens = 16;
constexpr int kTurns = 2048;  // angles of a workgroup at most

enum Mode { kHalves, kInterleaved, kStaged };

// 16 bytes to their values, and rounded back (bf16: nearest even)
template <typename T>
struct Vec {
    static constexpr int W = 16 / sizeof(T);
    static __device__ __forceinline__ void widen(u32x4 raw, float (&x)[W]) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(raw[i]);
            else x[i] = __uint_as_float((i & 1) ? raw[i / 2] & 0xFFFF0000u : raw[i / 2] << 16);
        }
    }
    static __device__ __forceinline__ u32x4 narrow(const float (&x)[W]) {
        u32x4 raw;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) raw[i] = __float_as_uint(x[i]);
            else raw[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        }
        return raw;
    }
};

// (x, y) turned by (cos, sin)
__device__ __forceinline__ float first_of(float x, float y, float2 t) { return __builtin_fmaf(x, t.x, -(y * t.y)); }
__device__ __forceinline__ float second_of(float x, float y, float2 t) { return __builtin_fmaf(x, t.y, y * t.x); }

// cos and sin of the angle position * freq, times the amplitude
__device__ __forceinline__ float2 turn_of(int64_t position, double freq, float amplitude, bool inverse) {
    constexpr double kTwoPiHi = 6.283185307179586, kTwoPiLo = 2.4492935982947064e-16;
    const double a = (double)position * freq, n = rint(a * 0.15915494309189535);
    const double rest = __builtin_fma(-n, kTwoPiLo, __builtin_fma(-n, kTwoPiHi, a));
    float sin, cos;
    sincospif((float)(rest * 0.3183098861837907), &sin, &cos);
    return make_float2(cos * amplitude, (inverse ? -sin : sin) * amplitude);
}

struct RotaryPlan {
    int tokens;       // of a workgroup
    int rows;         // rows (heads) of a token: queries, keys, values
    int units;        // threads of a row
    uint32_t rows_magic, units_magic;  // 2^32 / . + 1: exact below 2^32 / . (1 is left out)
};

template <typename T, int MODE, bool PLACE>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, RotaryPlan plan) {
    using V = Vec<T>;
    constexpr int W = V::W, NV = MODE == kHalves ? 2 : 1;  // vectors of a thread's step
    constexpr int kUnroll = 4 / NV;
    __shared__ float2 s_turn[kTurns];
    __shared__ int64_t s_k[kMaxTokens], s_v[kMaxTokens];
    __shared__ int s_on[kMaxTokens];
    __shared__ __attribute__((aligned(16))) T s_row[MODE == kStaged ? kThreads * W : 8];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t t0 = (int64_t)blockIdx.x * plan.tokens;
    const int nt = (int)(a.T - t0 < plan.tokens ? a.T - t0 : plan.tokens), pairs = a.r / 2;

    // this thread's place: row `my_row` of every step's rows, unit `u` of it
    const int step_rows = kThreads / plan.units;
    const int my_row = plan.units == 1 ? tid : (int)__umulhi((uint32_t)tid, plan.units_magic);
    const int u = tid - my_row * plan.units;
    const bool used = my_row < step_rows;
    const int total = nt * plan.rows;
    // channels of its vectors, and its first pair (kHalves, kInterleaved)
    int c0 = u * W, c1 = 0, pair = u * (W / 2);
    bool turned = c0 < a.r;
    if constexpr (MODE == kHalves) {
        turned = c0 < pairs;
        pair = c0;
        // behind the rotated channels, two neighbours
        c1 = turned ? c0 + pairs : 2 * c0 + W;
        c0 = turned ? c0 : 2 * c0;
    }
    u32x4 raw[kUnroll][NV];
    int tok[kUnroll], row[kUnroll];
    auto fetch = [&](int x0) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int x = x0 + i * step_rows + my_row;
            tok[i] = plan.rows == 1 ? x : (int)__umulhi((uint32_t)x, plan.rows_magic);
            row[i] = x - tok[i] * plan.rows;
            if (!used || x >= total) continue;
            const bool is_q = row[i] < a.Hq, is_k = !PLACE || row[i] < a.Hq + a.Hk;
            const T* base = static_cast<const T*>(is_q ? a.q : is_k ? a.k : a.v);
            const int64_t stride = is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride;
            const int h = is_q ? row[i] : is_k ? row[i] - a.Hq : row[i] - a.Hq - a.Hk;
            const T* p = base + (t0 + tok[i]) * stride + (int64_t)h * a.d;
            raw[i][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + c0));
            if constexpr (NV == 2) raw[i][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + c1));
        }
    };
    fetch(0);

    for (int j = wave; j < nt; j += kWaves) {
        const int64_t t = t0 + j;
        int64_t pos, ko = -1, vo = -1;
        bool on = true;
        if constexpr (PLACE) {
            int64_t n = t, i = 0;
            if (a.cu) {
                n = segment_of(a.cu, a.N, t);
                i = t - a.cu[n];
                on = i >= 0 && t < a.cu[n + 1];
            }
            pos = (int64_t)a.start[n] + i;
            const uint32_t col = (uint32_t)pos / (uint32_t)a.page_size;  // 0 <= pos < 2^32 where it counts
            if (on && pos >= 0 && col < (uint32_t)a.pt.width) {
                const int32_t p = a.pt.table[n * a.pt.stride + col];
                if (p >= 0 && p < a.pt.n_pages) {
                    const int64_t slot = (pos - (int64_t)col * a.page_size) * a.d;
                    ko = p * a.kp_stride + slot;
                    vo = p * a.vp_stride + slot;
                }
            }
        } else {
            pos = a.positions[t];
        }
        if (lane == 0) {
            s_on[j] = on;
            s_k[j] = ko;
            s_v[j] = vo;
        }
        for (int i = lane; i < pairs; i += 64) s_turn[j * pairs + i] = turn_of(pos, a.freqs[i], a.amplitude, a.inverse);
    }
    __syncthreads();

    for (int x0 = 0; x0 < total; x0 += kUnroll * step_rows) {
        if (x0 > 0) fetch(x0);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const bool here = used && x0 + i * step_rows + my_row < total;
            const int j = here ? tok[i] : 0;
            const bool is_q = row[i] < a.Hq, is_v = PLACE && row[i] >= a.Hq + a.Hk;
            const float2* turn = s_turn + j * pairs;
            u32x4 got[NV];
#pragma unroll
            for (int e = 0; e < NV; ++e) got[e] = raw[i][e];
            if constexpr (MODE == kStaged) {
                __syncthreads();  // the step before has been read
                if (here) *reinterpret_cast<u32x4*>(s_row + my_row * a.d + c0) = got[0];
                __syncthreads();
                if (here && !is_v && turned) {
                    float x[W], y[W];
                    V::widen(got[0], x);
                    const T* other = s_row + my_row * a.d;
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        const int c = c0 + e;
                        const bool low = c < pairs;
                        const float z = c < a.r ? ld_in(other, low ? c + pairs : c - pairs) : 0.f;
                        const float2 w = turn[c < a.r ? (low ? c : c - pairs) : 0];
                        y[e] = c < a.r ? (low ? first_of(x[e], z, w) : second_of(z, x[e], w)) : x[e];
                    }
                    got[0] = V::narrow(y);
                }
            } else if (turned && !is_v) {
                float x[W], y[W];
                V::widen(got[0], x);
                if constexpr (MODE == kHalves) {
                    V::widen(got[1], y);
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        const float2 w = turn[pair + e];
                        const float z = first_of(x[e], y[e], w);
                        y[e] = second_of(x[e], y[e], w);
                        x[e] = z;
                    }
                    got[1] = V::narrow(y);
                } else {
#pragma unroll
                    for (int e = 0; e < W; e += 2) {
                        if (c0 + e >= a.r) continue;
                        const float2 w = turn[pair + e / 2];
                        const float z = first_of(x[e], x[e + 1], w);
                        x[e + 1] = second_of(x[e], x[e + 1], w);
                        x[e] = z;
                    }
                }
                got[0] = V::narrow(x);
            }
            if (!here) continue;
            T* to;
            if (is_q) {
                if (PLACE && !s_on[j]) continue;
                to = static_cast<T*>(a.q_out) + (t0 + j) * a.q_out_stride + (int64_t)row[i] * a.d;
            } else if constexpr (PLACE) {
                const int64_t at = is_v ? s_v[j] : s_k[j];
                if (at < 0) continue;
                const int h = row[i] - a.Hq - (is_v ? a.Hk : 0);
                to = static_cast<T*>(is_v ? a.vp : a.kp) + at + (int64_t)h * a.page_size * a.d;
            } else {
                to = static_cast<T*>(a.k_out) + (t0 + j) * a.k_out_stride + (int64_t)(row[i] - a.Hq) * a.d;
            }
            __builtin_nontemporal_store(got[0], reinterpret_cast<u32x4*>(to + c0));
            if constexpr (NV == 2) __builtin_nontemporal_store(got[1], reinterpret_cast<u32x4*>(to + c1));
        }
    }
}

int rows_of(const RotaryArgs& a) { return a.Hq + a.Hk * (a.kp ? 2 : 1); }
// Halves whose vectors start at 16-byte boundaries: a thread has a vector of each.
bool whole_halves(const RotaryArgs& a) {
    const int W = a.bf16 ? 8 : 4;
    return !a.interleaved && a.r / 2 % W == 0 && a.d % (2 * W) == 0;
}
int units_of(const RotaryArgs& a) { return a.d / ((a.bf16 ? 8 : 4) * (whole_halves(a) ? 2 : 1)); }
// Tokens of a workgroup: as many as its threads have two steps for (7 + 1 heads of 64, bf16: 50 us against 61 with one
// step, 47 with four, which cost 40 heads of 128 a tenth), and whose angles have a place in LDS.  Where that gives more
// workgroups than a launch has, more of them, while the division by the rows is exact.
int tokens_of(const RotaryArgs& a) {
    const int64_t units = units_of(a), rows = rows_of(a), pairs = a.r / 2;
    int64_t t = 2 * kThreads / (units * rows);
    t = t < 1 ? 1 : t > kMaxTokens ? kMaxTokens : t;
    t = t * pairs > kTurns ? kTurns / pairs : t;
    while ((a.T + t - 1) / t > max_groups(kThreads) && 2 * t <= kMaxTokens && 2 * t * pairs <= kTurns &&
           2 * t * rows * rows < ((int64_t)1 << 32))
        t *= 2;
    return (int)t;
}

template <typename T, bool PLACE>
void launch_typed(const RotaryArgs& a, hipStream_t s) {
    RotaryPlan p;
    p.rows = rows_of(a);
    p.tokens = tokens_of(a);
    p.units = units_of(a);
    p.rows_magic = (uint32_t)(0xFFFFFFFFu / (uint32_t)p.rows + 1u);
    p.units_magic = (uint32_t)(0xFFFFFFFFu / (uint32_t)p.units + 1u);
    const dim3 grid((unsigned)((a.T + p.tokens - 1) / p.tokens)), block(kThreads);
    if (a.interleaved) hipLaunchKernelGGL((rotary_kernel<T, kInterleaved, PLACE>), grid, block, 0, s, a, p);
    else if (whole_halves(a)) hipLaunchKernelGGL((rotary_kernel<T, kHalves, PLACE>), grid, block, 0, s, a, p);
    else hipLaunchKernelGGL((rotary_kernel<T, kStaged, PLACE>), grid, block, 0, s, a, p);
}

}  // namespace

int64_t rotary_groups(const RotaryArgs& a) {
    const int64_t t = tokens_of(a);
    return (a.T + t - 1) / t;
}

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    const bool timed = timing_on();
    if (timed) timed_begin(kKernelRotary, s);
    if (a.bf16) {
        if (a.kp) launch_typed<uint16_t, true>(a, s);
        else launch_typed<uint16_t, false>(a, s);
    } else {
        if (a.kp) launch_typed<float, true>(a, s);
        else launch_typed<float, false>(a, s);
    }
    const hipError_t e = hipGetLastError();
    if (timed) timed_end(s);
    return e;
}

}  // namespace kda
