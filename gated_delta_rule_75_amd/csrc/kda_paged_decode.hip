// Softmax attention of one new token per sequence over a paged key-value cache (include/kda.h,
// kda_paged_decode):
//     s_t = scale q . k_t,   out = sum_t exp(s_t - m) v_t / l,   l = sum_t exp(s_t - m),
//     lse = m + log l,       m = max_t s_t
// over the visible tokens: all of them, or with a window the last ones and the first `sinks`.
//
// The visible keys and values are read once and little is done with each, so the traffic bounds it:
// everything else has to stay out of its way.
//  * Tiles of 16 tokens; a page holds a whole number of them, so a tile has one address.  Sinks and
//    window give one list of tiles, cut into parts of at most 128 tiles; a workgroup of four waves
//    takes one part of one key-value head for 16 or 32 of its query heads, each wave every fourth
//    step of it.  With few sequences the parts get short, so that the chip is filled; their partial
//    results (m, l, unnormalised out) are joined by a second launch.
//  * A wave reads the page numbers of all its tiles with one load at the start; its tiles go straight to
//    registers, and nothing goes through LDS before the end.  bf16 with D <= 128 has the next step's tiles
//    in flight while it works on this one.  fp32 does not: the compiler moves their loads behind the
//    score products and the softmax, so that only the second product covers them.  With long sequences the
//    other waves of the SIMD make up for it (64 sequences of 8192 tokens, 8 key heads: bf16 5.8 TB/s, fp32 6.0 at
//    D = 128 and 5.8 at 64), with short parts they do not (48 sequences with a window of 1024, 4 key heads,
//    D = 64, fp32: 4.1).  D = 256 loads a step and then works on it: bf16 with all 24 loads out first (6.1
//    TB/s), fp32 with two or three between the products at a time (5.5).
//  * Scores are K Q^T on the matrix cores, tokens as rows and query heads as columns.  The result
//    leaves four consecutive tokens of one head in each lane, which is how the next product wants
//    them: out^T = V^T P^T sums over tokens in any order, so a lane's own tokens serve as its
//    slice of the sum.  V arrives as rows of D / 16 channels per lane; a channel's tokens are
//    paired by byte permutes (bf16; fp32 needs none).  Rows of V^T are channels in the order
//    (D / 16) lane + c, which the write of the result undoes.  Maxima, sums and rescaling are per
//    head, which is per lane.
//  * bf16: the weights go into the second product as the sum of three bf16 (each what the ones before
//    left).  The first leaves 2^-8 of a weight at most, the second 2^-17, the third nothing: its 8 bits
//    hold what is left of 24 (from 2^-103 up, where the last bit is still a normal number).  One would show
//    in the fp32 result, and two still doubled its error (7 to 9e-7 against 4 to 5e-7 relative for the
//    output; the time is the same, the matrix cores wait for memory).
//  * Loads are bounded by descriptors that end with the tile's last visible token (none for a tile
//    without a page), and rows before the first visible one are replaced by it, so no slot that is
//    not visible is ever used, whatever it holds.
#include <math.h>

#include <type_traits>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kTile = 16;          // tokens
// Tiles of a part at most, up to 64 per wave (one page number per lane).  Long parts have fewer starts
// and partial results, short ones even out sequences of different lengths: 128 against 256 tiles took 261
// against 279 us for 64 sequences of 1K to 16K tokens, and 371 against 365 us for 64 of 8K.
constexpr int kMaxPartTiles = 128;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Visible tiles of a sequence: sink tiles 0 .. head_tiles-1, then the tiles from near / 16 on.
struct Visible {
    int head, near, len;  // tokens 0 .. head-1 and near .. len-1 are visible, head <= near
    int head_tiles, first, tiles;
};
__device__ __forceinline__ Visible visible(const PagedDecodeArgs& a, int64_t n) {
    Visible v;
    int len = a.lengths[n];
    len = len < 0 ? 0 : len > a.max_length ? (int)a.max_length : len;
    v.len = len;
    v.near = a.window > 0 && len > a.window ? len - a.window : 0;
    v.head = a.sinks < v.near ? a.sinks : v.near;
    v.head_tiles = (v.head + kTile - 1) / kTile;
    v.first = v.near / kTile;
    v.tiles = v.head_tiles + (len + kTile - 1) / kTile - v.first;
    return v;
}

// partial results in the workspace: (m, l) [N * Hq, parts], then out [N * Hq, parts, D]
struct PartPlan {
    int part_tiles, parts, heads;  // heads: query heads of a workgroup
};

// One step's tiles in registers.  bf16: two tiles, K as the rows of the first product's left operand
// (lane lr, lg: token lr, channels 32 ks + 8 lg ..), V as rows (tokens 4 lg + j, channels of lane lr).
// fp32: one tile.
template <typename T, int D>
struct Step;

template <int D>
struct Step<uint16_t, D> {
    static constexpr int NT = 2, KS = D / 32, VEC = D / 16;
    u32x4 k[NT][KS];
    uint32_t v[NT][4][VEC / 2];
    int lo[NT], hi[NT];  // visible rows of each tile
};
template <int D>
struct Step<float, D> {
    static constexpr int NT = 1, KS = D / 16, VEC = D / 16;
    u32x4 k[NT][KS];
    uint32_t v[NT][4][VEC];
    int lo[NT], hi[NT];
};

template <int W>
__device__ __forceinline__ void load_words(__amdgpu_buffer_rsrc_t r, int voff, uint32_t (&x)[W]) {
    if constexpr (W == 2) {
        const u32x2 y = __builtin_amdgcn_raw_buffer_load_b64(r, voff, 0, 0);
        x[0] = y.x; x[1] = y.y;
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const u32x4 y = __builtin_amdgcn_raw_buffer_load_b128(r, voff + 4 * i, 0, 0);
            x[i] = y.x; x[i + 1] = y.y; x[i + 2] = y.z; x[i + 3] = y.w;
        }
    }
}

__device__ __forceinline__ floatx4 mfma_bf16(u32x4 a, u32x4 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// two fp32 weights to packed bf16 (nearest even), and what is left of them
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 y = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, y);
}
__device__ __forceinline__ float low_of(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high_of(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

template <typename T, int D, int HT>
__global__ __launch_bounds__(kThreads, HT == 2 && D == 128 ? 1 : 2) void paged_decode_kernel(PagedDecodeArgs a, PartPlan plan, float2* part_ml,
                                                                   float* part_o) {
    using S = Step<T, D>;
    constexpr bool kBf16 = std::is_same<T, uint16_t>::value;
    constexpr int NT = S::NT, KS = S::KS, VEC = S::VEC, ES = sizeof(T);
    constexpr bool kAhead = D <= 128;  // D = 256: a step is 32 KB a wave, twice that has no registers (229 of 256 used)
    constexpr int kRow = D + 4;        // LDS row of a head, shifted by one 16-byte bank group per head
    __shared__ __attribute__((aligned(16))) float s_o[2][16][kRow];
    __shared__ float s_m[kWaves][16 * HT], s_l[kWaves][16 * HT];

    const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // parts slowest: consecutive workgroups go to different XCDs, and the parts behind a short
    // sequence's end, which return at once, must not all fall to the same ones (with the parts fastest
    // and eight of them, XCD 0 got every sequence's first part and XCD 7 only the longest ones' last:
    // 370 against 276 us for 64 sequences of 1K to 16K tokens)
    const int G = a.Hq / a.Hkv, head_groups = (G + 16 * HT - 1) / (16 * HT);
    const int64_t groups = a.N * a.Hkv * head_groups;
    int64_t g = blockIdx.x % groups;
    const int part = (int)(blockIdx.x / groups);
    const int g0 = (int)(g % head_groups) * 16 * HT;  // first query head of this workgroup in its group
    g /= head_groups;
    const int h = (int)(g % a.Hkv);
    const int64_t n = g / a.Hkv;

    // The loads that need nothing but the indexes go first: the queries (columns of the first product),
    // and without a window the page numbers of this wave's tiles, whose places do not depend on the
    // length (with one, the length's latency comes before theirs).
    u32x4 q[HT][KS];
#pragma unroll
    for (int t = 0; t < HT; ++t) {
        const int hq = g0 + 16 * t + lr;
        const T* row = static_cast<const T*>(a.q) + n * a.q_stride + (int64_t)(h * G + (hq < G ? hq : 0)) * D;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            q[t][ks] = *reinterpret_cast<const u32x4*>(row + ks * (D / KS) + lg * (16 / ES));
    }
    // one tile per lane: NT * (w + 4 * (lane / NT)) + lane % NT of the part
    const int t0 = part * plan.part_tiles, my_tile = t0 + NT * (w + kWaves * (lane / NT)) + lane % NT;
    const int tiles_per_page = a.page_size / kTile;
    const int32_t* row = a.pt.table + n * a.pt.stride;
    int32_t my_page = -1;
    if (a.window == 0 && my_tile / tiles_per_page < a.pt.width) my_page = row[my_tile / tiles_per_page];
    const Visible vis = visible(a, n);
    if (t0 >= vis.tiles && part > 0) return;  // the join does not look at it
    const int t1 = t0 + plan.part_tiles < vis.tiles ? t0 + plan.part_tiles : vis.tiles;

    int my_slot = 0, my_lo = 0, my_hi = 0;
    if (my_tile < t1) {
        const bool sink = my_tile < vis.head_tiles;
        const int tile = sink ? my_tile : vis.first + my_tile - vis.head_tiles;
        const int col = tile / tiles_per_page;
        if (a.window != 0) my_page = row[col];
        const int lo = (sink ? 0 : vis.near) - tile * kTile, hi = (sink ? vis.head : vis.len) - tile * kTile;
        my_slot = (tile - col * tiles_per_page) * kTile;
        my_lo = lo > 0 ? lo : 0;
        my_hi = hi < kTile ? hi : kTile;
        if (my_page >= a.pt.n_pages) my_page = -1;
    } else {
        my_page = -1;
    }
    const int steps = (t1 - t0 + NT * kWaves - 1) / (NT * kWaves);  // of the workgroup; some waves' last are empty
#pragma unroll
    for (int t = 0; t < HT; ++t)
        if (g0 + 16 * t + lr >= G) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) q[t][ks] = u32x4{0, 0, 0, 0};
        }

    auto load = [&](S& s, int step) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int at = (NT * step + t) & 63;
            const int page = __builtin_amdgcn_readlane(my_page, at), slot = __builtin_amdgcn_readlane(my_slot, at);
            const bool on = page >= 0 && step < steps;
            s.lo[t] = __builtin_amdgcn_readlane(my_lo, at);
            s.hi[t] = on ? __builtin_amdgcn_readlane(my_hi, at) : 0;
            const int64_t inner = ((int64_t)h * a.page_size + slot) * D, p = on ? page : 0;
            const __amdgpu_buffer_rsrc_t kr =
                make_rsrc(static_cast<const T*>(a.kp) + p * a.kp_stride + inner, (uint32_t)(s.hi[t] * D * ES));
            const __amdgpu_buffer_rsrc_t vr =
                make_rsrc(static_cast<const T*>(a.vp) + p * a.vp_stride + inner, (uint32_t)(s.hi[t] * D * ES));
            const int krow = lr > s.lo[t] ? lr : s.lo[t];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                s.k[t][ks] = __builtin_amdgcn_raw_buffer_load_b128(kr, krow * D * ES + lg * 16, ks * (D / KS) * ES, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int vrow = 4 * lg + j > s.lo[t] ? 4 * lg + j : s.lo[t];
                load_words(vr, vrow * D * ES + lr * VEC * ES, s.v[t][j]);
            }
        }
    };

    floatx4 o[HT][VEC];
    float m[HT], l[HT];
#pragma unroll
    for (int t = 0; t < HT; ++t) {
        m[t] = -INFINITY;
        l[t] = 0.f;
#pragma unroll
        for (int c = 0; c < VEC; ++c) o[t][c] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
    const float scale2 = a.scale * kLog2e;  // scores in base-2 units

    auto work = [&](const S& s) {
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
            float p[NT][4];
            float top = -INFINITY;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                floatx4 x = {0.f, 0.f, 0.f, 0.f};
                if constexpr (kBf16) {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) x = mfma_bf16(s.k[t][ks], q[ht][ks], x);
                } else {
                    // four sums side by side: a quarter of the chain of dependent steps, and of its rounding
                    floatx4 y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            y[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(s.k[t][ks][i]),
                                                                        __uint_as_float(q[ht][ks][i]), y[i], 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = (y[0][i] + y[1][i]) + (y[2][i] + y[3][i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * lg + i;
                    p[t][i] = r >= s.lo[t] && r < s.hi[t] ? x[i] * scale2 : -INFINITY;
                    top = fmaxf(top, p[t][i]);
                }
            }
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float now = fmaxf(m[ht], top), base = now == -INFINITY ? 0.f : now;
            const float keep = exp2_hw(m[ht] - base);
            m[ht] = now;
            float sum = 0.f;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[t][i] = exp2_hw(p[t][i] - base);
                    sum += p[t][i];
                }
            l[ht] = l[ht] * keep + sum;
            // the step's share is summed by itself and added with one fp32 rounding: a running sum inside
            // the matrix cores loses twice as much over a long part (measured: 1.2e-6 against 7e-7)
            if constexpr (kBf16) {
                u32x4 hi, lo, rest;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const uint32_t y = pack_bf16(p[t][i], p[t][i + 1]);
                        hi[2 * t + i / 2] = y;
                        const float e0 = p[t][i] - low_of(y), e1 = p[t][i + 1] - high_of(y);
                        const uint32_t z = pack_bf16(e0, e1);
                        lo[2 * t + i / 2] = z;
                        rest[2 * t + i / 2] = pack_bf16(e0 - low_of(z), e1 - high_of(z));
                    }
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    const uint32_t sel = (c & 1) ? 0x07060302u : 0x05040100u;
                    u32x4 v;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; i += 2)
                            v[2 * t + i / 2] = __builtin_amdgcn_perm(s.v[t][i + 1][c / 2], s.v[t][i][c / 2], sel);
                    const floatx4 share = mfma_bf16(
                        v, hi, mfma_bf16(v, lo, mfma_bf16(v, rest, floatx4{0.f, 0.f, 0.f, 0.f})));
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[ht][c][i] = o[ht][c][i] * keep + share[i];
                }
            } else {
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    floatx4 share = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        share = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(s.v[0][i][c]), p[0][i], share, 0,
                                                                     0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[ht][c][i] = o[ht][c][i] * keep + share[i];
                }
            }
        }
    };

    if constexpr (kAhead) {
        S x, y;
        load(x, 0);
        for (int i = 0; i < steps; i += 2) {
            load(y, i + 1);
            work(x);
            load(x, i + 2);
            work(y);
        }
    } else {
        S x;
        for (int i = 0; i < steps; ++i) {
            load(x, i);
            work(x);
        }
    }

    // join the four waves
#pragma unroll
    for (int t = 0; t < HT; ++t) {
        l[t] += __shfl_xor(l[t], 16, 64);
        l[t] += __shfl_xor(l[t], 32, 64);
        if (lg == 0) {
            s_m[w][16 * t + lr] = m[t];
            s_l[w][16 * t + lr] = l[t];
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < HT; ++t) {
        float M = s_m[0][16 * t + lr];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) M = fmaxf(M, s_m[i][16 * t + lr]);
        const float base = M == -INFINITY ? 0.f : M, keep = exp2_hw(m[t] - base);
        float L = 0.f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) L += s_l[i][16 * t + lr] * exp2_hw(s_m[i][16 * t + lr] - base);
        // this lane's channels of head lr: 4 VEC lg + VEC i + c
#pragma unroll
        for (int c = 0; c < VEC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[t][c][i] *= keep;
        auto put = [&](int slot) {
            float* d = &s_o[slot][lr][4 * VEC * lg];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < VEC; c += 4)
                    *reinterpret_cast<floatx4*>(d + VEC * i + c) =
                        floatx4{o[t][c][i], o[t][c + 1][i], o[t][c + 2][i], o[t][c + 3][i]};
        };
        auto add = [&](int slot) {
            const float* d = &s_o[slot][lr][4 * VEC * lg];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < VEC; c += 4) {
                    const floatx4 y = *reinterpret_cast<const floatx4*>(d + VEC * i + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[t][c + e][i] += y[e];
                }
        };
        if (w >= 2) put(w - 2);
        __syncthreads();
        if (w < 2) add(w);
        __syncthreads();
        if (w == 1) put(0);
        __syncthreads();
        const int hq = g0 + 16 * t + lr;
        if (w == 0) {
            add(0);
            if (hq < G) {
                const int64_t row = n * a.Hq + h * G + hq;
                float* d;
                float f;
                if (plan.parts == 1) {
                    d = a.o + row * D;
                    f = L == 0.f ? 0.f : 1.f / L;
                    if (a.lse && lg == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
                } else {
                    d = part_o + (row * plan.parts + part) * D;
                    f = 1.f;
                    if (lg == 0) part_ml[row * plan.parts + part] = make_float2(M, L);
                }
                d += 4 * VEC * lg;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < VEC; c += 4)
                        *reinterpret_cast<floatx4*>(d + VEC * i + c) =
                            floatx4{o[t][c][i] * f, o[t][c + 1][i] * f, o[t][c + 2][i] * f, o[t][c + 3][i] * f};
            }
        }
        if (t + 1 < HT) __syncthreads();
    }
}

// Join of the parts: one workgroup per query head.  Every wave forms the joint maximum; wave w takes
// parts w, w + 4, ... with its lanes over the channels.  (One wave per head took 15.5 us for 128 parts
// of 128 heads.)
template <int D>
__global__ __launch_bounds__(kThreads) void paged_join_kernel(PagedDecodeArgs a, PartPlan plan, const float2* part_ml,
                                                              const float* part_o) {
    constexpr int CH = D / 64;
    __shared__ float s_o[kWaves][D], s_l[kWaves];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = blockIdx.x;
    const float2* ml = part_ml + row * plan.parts;
    const float* po = part_o + row * plan.parts * D + lane * CH;
    // The first loads do not wait for the number of parts: they stay inside the row's share of the
    // workspace, and what was not written for this call is replaced by 0 below.
    constexpr int kFirst = 8;
    float2 y0 = ml[lane < plan.parts ? lane : plan.parts - 1];
    float x0[kFirst][CH];
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
        const int p = w + kWaves * i < plan.parts ? w + kWaves * i : plan.parts - 1;
#pragma unroll
        for (int c = 0; c < CH; ++c) x0[i][c] = po[(int64_t)p * D + c];
    }
    const Visible vis = visible(a, row / a.Hq);
    const int parts = vis.tiles > 0 ? (vis.tiles + plan.part_tiles - 1) / plan.part_tiles : 1;
    if (lane >= parts) y0 = make_float2(-INFINITY, 0.f);
    float M = y0.x;
    for (int p = 64 + lane; p < parts; p += 64) M = fmaxf(M, ml[p].x);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f, acc[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) acc[c] = 0.f;
    // weights of the first 64 parts in the lanes; part w + 4 i is wave w's
    float wgt = exp2_hw(y0.x - base);
    if ((lane & (kWaves - 1)) == w) L = y0.y * wgt;
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
        const int p = w + kWaves * i;
        const float f = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wgt), p));
#pragma unroll
        for (int c = 0; c < CH; ++c) acc[c] += p < parts ? f * x0[i][c] : 0.f;
    }
    for (int p0 = w + kWaves * kFirst; p0 < parts; p0 += 64 * kWaves) {  // lane i: part p0 + 4 i
        wgt = 0.f;
        if (p0 + kWaves * lane < parts) {
            const float2 y = ml[p0 + kWaves * lane];
            wgt = exp2_hw(y.x - base);
            if (p0 + kWaves * lane >= 64) L += y.y * wgt;  // the first 64 are in already
        }
        const int left = (parts - p0 + kWaves - 1) / kWaves, count = left < 64 ? left : 64;
        for (int i0 = 0; i0 < count; i0 += 8) {  // eight loads in flight; parts behind the last have weight 0
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wgt), i0 + i));
                const int at = i0 + i < count ? i0 + i : count - 1;
#pragma unroll
                for (int c = 0; c < CH; ++c) acc[c] += f * po[(int64_t)(p0 + kWaves * at) * D + c];
            }
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) L += __shfl_xor(L, off, 64);
#pragma unroll
    for (int c = 0; c < CH; ++c) s_o[w][lane * CH + c] = acc[c];
    if (lane == 0) s_l[w] = L;
    __syncthreads();
    if (threadIdx.x >= D) return;
    L = 0.f;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        L += s_l[i];
        x += s_o[i][threadIdx.x];
    }
    a.o[row * D + threadIdx.x] = L == 0.f ? 0.f : x / L;
    if (a.lse && threadIdx.x == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

int64_t div_up(int64_t x, int64_t m) { return (x + m - 1) / m; }

// 32 query heads a workgroup where a key-value head has more than 16 (fp32 and D = 256 have no
// registers for that)
int head_tiles_of(int G, int d, int bf16) { return bf16 && d <= 128 && G > 16 ? 2 : 1; }

// workgroups of a part
int64_t part_groups(int64_t N, int Hq, int Hkv, int d, int bf16) {
    return N * Hkv * div_up(Hq / Hkv, 16 * head_tiles_of(Hq / Hkv, d, bf16));
}

PartPlan part_plan(int64_t N, int Hq, int Hkv, int d, int bf16, int64_t max_length, int window, int sinks) {
    const int step_tiles = kWaves * (bf16 ? 2 : 1);
    int64_t tiles = div_up(max_length, kTile);
    if (window > 0 && max_length > window) {
        const int64_t most = div_up(sinks, kTile) + div_up(window, kTile) + 1;
        tiles = most < tiles + 1 ? most : tiles + 1;
    }
    PartPlan p;
    p.heads = 16 * head_tiles_of(Hq / Hkv, d, bf16);
    const int64_t groups = part_groups(N, Hq, Hkv, d, bf16);
    int64_t per = 0;
    if ((window > 0 && max_length > window) || N <= 2) {
        // Sequences behind their window all have the same tiles, and so has a lone one: the part length with
        // the fewest rounds of resident workgroups times steps, where a workgroup's start and end count as
        // three steps and the join as four.  Against the rule below, whole calls: 13.4 and 21.3 us for 100
        // sequences with a window of 512, 14.1 and 17.7 for a lone one of 9000 tokens, 20.6 and 33.9 for one
        // of 30000 in fp32; at worst 25.9 and 24.4, for 48 with a window of 1024 in fp32.
        // Two sequences may differ, but half of the launch at least follows the longer one, and the rule below
        // aims at workgroups for many: 11.9 and 12.3 us for two of 3000 tokens (fp32 16.0 and 23.9), 16.3 and
        // 16.9 for 9000 and 300 (fp32 23.5 and 27.8), 26.8 and 29.4 for 30 000 and 1000 (fp32 48.1 and 52.2),
        // 40.7 and 41.4 for two of 30 000; equal from there on.
        // Resident workgroups: 256 CUs times the waves of a SIMD, which are what 512 registers hold of 134 (D = 64),
        // 371 (D = 128 with 32 heads) or 196 to 236 (the others) each.
        const int64_t slots = 256 * (d == 64 && p.heads == 16 ? 3 : d == 128 && p.heads == 32 ? 1 : 2);
        int64_t best = 0;
        for (int64_t steps = 1; steps * step_tiles <= kMaxPartTiles; ++steps) {
            const int64_t parts = div_up(tiles, steps * step_tiles), rounds = div_up(groups * parts, slots);
            const int64_t cost = rounds * (steps + 3) + (parts > 1 ? 4 : 0);
            if (per == 0 || cost < best) {
                best = cost;
                per = steps * step_tiles;
            }
        }
    } else {
        // Lengths differ, nobody knows how: workgroups enough for about four per CU if all were of the
        // bound.  512 to 2048 of them were within 10% of one another over lengths and shapes, none ahead in
        // all.
        per = div_up(tiles * (groups > 0 ? groups : 1), 1024);
        per = div_up(per > 0 ? per : 1, step_tiles) * step_tiles;
        if (tiles <= 4 * step_tiles) per = 4 * step_tiles;  // four steps take no longer than a join
    }
    p.part_tiles = (int)(per > kMaxPartTiles ? kMaxPartTiles : per);
    p.parts = (int)(tiles > 0 ? div_up(tiles, p.part_tiles) : 1);
    return p;
}

}  // namespace

bool paged_decode_supported(int d) { return d == 64 || d == 128 || d == 256; }

int64_t paged_decode_groups(int64_t N, int Hq, int Hkv, int d, int bf16, int64_t max_length, int window, int sinks,
                            size_t* workspace) {
    *workspace = 0;
    int64_t groups = part_groups(N, Hq, Hkv, d, bf16);
    if (groups > max_groups(kThreads)) return groups;  // (the plan's products stay within 64 bits below that)
    const int parts = part_plan(N, Hq, Hkv, d, bf16, max_length, window, sinks).parts;
    groups *= parts;
    if (parts == 1) return groups;
    if (N * Hq > groups) groups = N * Hq;  // the join's
    if (groups <= max_groups(kThreads))
        *workspace = (size_t)(div_up(N * Hq * parts * 8, 256) * 256 + N * Hq * parts * (int64_t)d * 4);
    return groups;
}

template <typename T, int D>
static void launch_typed(const PagedDecodeArgs& a, const PartPlan& p, float2* ml, float* po, hipStream_t s) {
    const unsigned grid = (unsigned)(part_groups(a.N, a.Hq, a.Hkv, a.d, a.bf16) * p.parts);
    if constexpr (std::is_same<T, uint16_t>::value && D <= 128) {
        if (p.heads == 32) {
            hipLaunchKernelGGL((paged_decode_kernel<T, D, 2>), dim3(grid), dim3(kThreads), 0, s, a, p, ml, po);
            return;
        }
    }
    hipLaunchKernelGGL((paged_decode_kernel<T, D, 1>), dim3(grid), dim3(kThreads), 0, s, a, p, ml, po);
}

hipError_t launch_paged_decode(const PagedDecodeArgs& a, hipStream_t s) {
    if (a.N == 0) return hipSuccess;
    const PartPlan p = part_plan(a.N, a.Hq, a.Hkv, a.d, a.bf16, a.max_length, a.window, a.sinks);
    float2* ml = static_cast<float2*>(a.ws);
    float* po = reinterpret_cast<float*>(static_cast<char*>(a.ws) + div_up(a.N * a.Hq * p.parts * 8, 256) * 256);
    const bool timed = timing_on();
    if (timed) timed_begin(kKernelPagedDecode, s);
    if (a.bf16) {
        if (a.d == 64) launch_typed<uint16_t, 64>(a, p, ml, po, s);
        else if (a.d == 128) launch_typed<uint16_t, 128>(a, p, ml, po, s);
        else launch_typed<uint16_t, 256>(a, p, ml, po, s);
    } else {
        if (a.d == 64) launch_typed<float, 64>(a, p, ml, po, s);
        else if (a.d == 128) launch_typed<float, 128>(a, p, ml, po, s);
        else launch_typed<float, 256>(a, p, ml, po, s);
    }
    hipError_t e = hipGetLastError();
    if (timed) timed_end(s);
    if (e != hipSuccess || p.parts == 1) return e;
    if (timed) timed_begin(kKernelPagedJoin, s);
    const dim3 grid((unsigned)(a.N * a.Hq)), block(kThreads);
    if (a.d == 64) hipLaunchKernelGGL(paged_join_kernel<64>, grid, block, 0, s, a, p, ml, po);
    else if (a.d == 128) hipLaunchKernelGGL(paged_join_kernel<128>, grid, block, 0, s, a, p, ml, po);
    else hipLaunchKernelGGL(paged_join_kernel<256>, grid, block, 0, s, a, p, ml, po);
    e = hipGetLastError();
    if (timed) timed_end(s);
    return e;
}

}  // namespace kda
