// Softmax attention of a chunk of new tokens per sequence over a paged key-value cache (include/kda.h,
// kda_paged_prefill):
//     s_t = scale q . k_t,   out = sum_t exp(s_t - m) v_t / l,   l = sum_t exp(s_t - m),   lse = m + log l
// for the query at position p, over t <= p, with a window over p - window < t <= p and t < sinks.
//
// Rows are (token, query head of the group) pairs of one key-value head, so that the heads that share keys share
// their loads.  Scores are K Q^T and outputs V^T P^T on 32 x 32 matrix instructions: rows of queries are columns of
// both results, so a lane holds values of one query only.  The softmax needs one exchange between the two halves
// of a wave, and the scores that a lane holds are, rounded, its share of the second product's right operand.
#include <math.h>

#include <type_traits>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 16 bytes per lane from a buffer to LDS: lane i's go to to + 16 i; those behind the descriptor's end become 0.  Written
// out, since the compiler would let every read of LDS wait for all such loads, also of those for the next tile.
// (The clobber keeps the compiler's own uses of m0 whole, each of which sets it right before.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t from, int offset, uint32_t more, const char* to) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)to);
    // (a descriptor that vector instructions have written needs five wait states before a load)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(at), "v"(offset), "s"(from), "s"(more)
                 : "m0", "memory");
}
#pragma clang diagnostic pop
// Everything that this wave's loads bring into LDS is there (a barrier alone does not wait for it), and it has read what
// it asked LDS for, so that the next loads may go there.
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kPage = 16;  // tokens that surely share a page

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 y = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, y);
}
__device__ __forceinline__ f32x16 zeros() {
    f32x16 z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
    return z;
}

// LDS tiles are blocks of 128 bytes of each row, [ROW / 128][BN][128], in 16-byte pieces: piece c of a block's row r is
// at place c ^ swizzle(r).  Then 16 successive rows of one piece of the keys, and 64 bytes of 4 successive rows of the
// values, lie in different banks, and all reads of a lane differ by constants from a few addresses.
__device__ __forceinline__ int swizzle_k(int r) { return ((r >> 1) & 1) << 2 | ((r >> 2) & 3); }
template <int ES>
__device__ __forceinline__ int swizzle_v(int r) { return ES == 2 ? ((r >> 1) & 1) << 2 : 0; }

// How a kernel instance splits its work.  ROWS: four waves with 32 rows each share a tile of keys.  Otherwise the
// waves share 32 rows and each has tiles of its own.
template <typename T, int D, bool ROWS>
struct Shape {
    static constexpr int ES = sizeof(T), ROW = D * ES;
    static constexpr int BN = ROWS && ROW <= 256 && ES == 2 ? 64 : 32;  // keys of a tile
    static constexpr int WAVES = ROWS ? 4 : ROW <= 256 ? 4 : ROW == 512 ? 2 : 1;
    static constexpr int THREADS = 64 * WAVES;
    static constexpr int RT = ROWS ? 128 : 32;               // rows of a workgroup
    static constexpr int TILE = BN * ROW;                    // bytes of a tile's keys
    static constexpr int BUFS = ROWS ? 1 : WAVES;            // tiles at a time
    static constexpr int GROUPS = ROWS && ROW <= 512 ? 2 : 1;  // workgroups a CU should hold
};

// Row tiles of all sequences: tile k of sequence n has slot floor(cu[n] G / RT) + n + k, which leaves every sequence
// enough slots.  The sequence of a slot (wave-uniform), by 64 probes at a time.
__device__ __forceinline__ int64_t slot_begin(const int32_t* cu, int64_t n, int G, int RT) {
    return (int64_t)cu[n] * G / RT + n;
}
__device__ __forceinline__ int64_t sequence_of(const int32_t* cu, int64_t N, int64_t slot, int G, int RT) {
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, left = N - 1;
    while (left > 0) {
        const int64_t step = (left + 63) / 64, at = (lane + 1) * step;
        const bool in = at <= left;
        const int hits = __popcll(__ballot(in && slot_begin(cu, lo + (in ? at : left), G, RT) <= slot));
        lo += hits * step;
        left -= hits * step;
        left = left < step - 1 ? left : step - 1;
    }
    return lo;
}

struct PrefillPlan {
    int64_t slots;
    int parts, part_tiles;
};

template <typename T, int D, bool ROWS>
__global__ __launch_bounds__((Shape<T, D, ROWS>::THREADS), (Shape<T, D, ROWS>::GROUPS)) void paged_prefill_kernel(
    PagedPrefillArgs a, PrefillPlan plan, float2* part_ml, float* part_o) {
    using S = Shape<T, D, ROWS>;
    constexpr bool kBf16 = std::is_same<T, uint16_t>::value;
    constexpr int ES = S::ES, ROW = S::ROW, BN = S::BN, WAVES = S::WAVES, RT = S::RT, KG = BN / 32, CT = D / 32;
    constexpr int LOADS = kPage * ROW / 1024;      // 1 KiB loads of 16 rows
    constexpr int QW = ROW / 32;                   // 16-byte pieces of a lane's query row
    __shared__ __attribute__((aligned(1024))) char s_kv[S::BUFS][2][2 * S::TILE];  // keys and values, twice
    __shared__ int s_on[2][BN / kPage];
    __shared__ float s_m[WAVES][32], s_l[WAVES][32];

    const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, hl = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = a.Hq / a.Hkv;
    // heads fastest: workgroups of one head go to the same XCDs where the heads divide the eight, whose L2 then
    // holds that head's keys; late tiles first: they have the most keys
    int64_t b = blockIdx.x;
    const int h = (int)(b % a.Hkv);
    b /= a.Hkv;
    const int64_t slot = plan.slots - 1 - b % plan.slots;
    const int part = (int)(b / plan.slots);
    const int64_t n = sequence_of(a.cu, a.N, slot, G, RT);
    const int64_t cu0 = a.cu[n] < 0 ? 0 : a.cu[n], cu1 = a.cu[n + 1] < a.T ? a.cu[n + 1] : a.T;
    const int64_t fresh = cu1 - cu0, row0 = (slot - slot_begin(a.cu, n, G, RT)) * RT;
    if (row0 < 0 || row0 >= fresh * G) return;
    const int rows = (int)(fresh * G - row0 < RT ? fresh * G - row0 : RT);
    const int64_t i0 = row0 / G;
    const int g0 = (int)(row0 - i0 * G);
    const int length = a.lengths[n] > 0 ? a.lengths[n] : 0;
    const int cap = length < a.max_length ? length : (int)a.max_length;
    // positions (64 bits: a contract that is broken gives any)
    auto position = [&](int r) {
        const int64_t p = (int64_t)length - fresh + i0 + (g0 + r) / G;
        return (int)(p < -1 ? -1 : p);
    };
    const int p_first = position(0), p_last = position(rows - 1);
    const int end = p_last + 1 < cap ? p_last + 1 : cap;
    // visible to some row: 0 .. head-1 and near .. end-1
    int near = a.window > 0 && p_first >= a.window ? p_first - a.window + 1 : 0;
    near = near < end ? near : end;
    const int head = a.sinks < near ? a.sinks : near;
    const int head_tiles = (head + BN - 1) / BN, first = near / BN;
    const int tiles = head_tiles + (end + BN - 1) / BN - first;
    const int t0 = part * plan.part_tiles, t1 = t0 + plan.part_tiles < tiles ? t0 + plan.part_tiles : tiles;

    // this lane's row
    const int my = ROWS ? w * 32 + lr : lr;
    const bool mine = my < rows;
    const int my_i = (g0 + (mine ? my : 0)) / G, my_g = g0 + (mine ? my : 0) - my_i * G;
    const int64_t token = cu0 + i0 + my_i;
    const int wave_first = ROWS ? w * 32 : 0, wave_rows = rows - wave_first < 32 ? rows - wave_first : 32;
    const int pw_first = position(wave_rows > 0 ? wave_first : 0), pw_last = position(wave_rows > 0 ? wave_first + wave_rows - 1 : 0);
    const int p = mine ? position(my) : pw_last;
    const int p_near = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
    const bool active = wave_rows > 0;

    // The scores' sign goes to the queries, so that the factor is positive; a scale of 0 makes them 0.
    const float scale2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
    u32x4 q[QW];
    {
        const T* qr = static_cast<const T*>(a.q) + token * a.q_stride + (int64_t)(h * G + my_g) * D;
        const uint32_t flip = a.scale < 0.f ? (kBf16 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
        for (int s = 0; s < QW; ++s) {
            u32x4 x = {0, 0, 0, 0};
            if (mine && a.scale != 0.f) {
                x = *reinterpret_cast<const u32x4*>(qr + (2 * s + hl) * (16 / ES));
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] ^= flip;
            }
            q[s] = x;
        }
    }

    // loads of tiles: the page numbers of the next 64 of this wave's 16-token pieces are in its lanes
    constexpr int SUBS = BN / kPage;                          // pieces of a tile
    constexpr int STEP = ROWS ? 1 : WAVES;                    // tiles between a wave's
    constexpr int PER = ROWS ? 64 : 64 / SUBS;                // tiles that the lanes cover
    const int my_sub = ROWS ? w % SUBS : lane % SUBS;
    const int w0 = ROWS ? 0 : w;
    const int32_t* table = a.pt.table + n * a.pt.stride;
    int lane_page = -1;
    auto base_of = [&](int t) { return t < head_tiles ? t * BN : (first + t - head_tiles) * BN; };
    auto look_up = [&](int i) {  // for the wave's tiles i ..
        const int t = t0 + w0 + STEP * (i + (ROWS ? lane : lane / SUBS));
        lane_page = -1;
        if (t < t1) {
            const uint32_t col = (uint32_t)(base_of(t) + my_sub * kPage) / (uint32_t)a.page_size;
            if (col < (uint32_t)a.pt.width) lane_page = table[col];
            if (lane_page >= a.pt.n_pages) lane_page = -1;
        }
    };
    // byte offsets of this lane's 16 bytes inside rows 0 .. 7 and 8 .. 15 of a piece
    int k_at[2], v_at[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = 8 * e + lane / 8;
        k_at[e] = r * ROW + ((lane % 8) ^ swizzle_k(r)) * 16;
        v_at[e] = r * ROW + ((lane % 8) ^ swizzle_v<ES>(r)) * 16;
    }
    // piece `sub` of tile t: keys or values, from the page to its place in LDS; rows behind the last visible one, or
    // without a page, become 0
    auto load_piece = [&](const void* pages, int64_t stride, int page, int t, int sub, const int (&at)[2], char* to) {
        const int pos = base_of(t) + sub * kPage, limit = t < head_tiles ? head : end;
        const int left = page >= 0 ? limit - pos : 0, on = left < 0 ? 0 : left > kPage ? kPage : left;
        const int slot16 = (int)((uint32_t)pos % (uint32_t)a.page_size);
        const T* from = static_cast<const T*>(pages) + (page >= 0 ? page : 0) * stride +
                        ((int64_t)h * a.page_size + slot16) * D;
        const __amdgpu_buffer_rsrc_t r = make_rsrc(from, (uint32_t)(on * ROW));
#pragma unroll
        for (int e = 0; e < LOADS; ++e)
            load_lds(r, at[e & 1], (e >> 1) * 128, to + (e >> 1) * BN * 128 + sub * kPage * 128 + (e & 1) * 1024);
    };
    auto load = [&](int i, char* to, int* on) {  // the wave's tile i
        const int t = t0 + w0 + STEP * i;
        if (i % PER == 0) look_up(i);
        if (t >= t1) return;
        if constexpr (ROWS) {
            const int page = __builtin_amdgcn_readlane(lane_page, i & 63), sub = w % SUBS;
            if (SUBS == WAVES || w < SUBS) load_piece(a.kp, a.kp_stride, page, t, sub, k_at, to);
            if (SUBS == WAVES || w >= SUBS) load_piece(a.vp, a.vp_stride, page, t, sub, v_at, to + S::TILE);
            if (lane == 0 && w < SUBS) on[sub] = page >= 0;
        } else {
#pragma unroll
            for (int sub = 0; sub < SUBS; ++sub) {
                const int page = __builtin_amdgcn_readlane(lane_page, (i % PER) * SUBS + sub);
                load_piece(a.kp, a.kp_stride, page, t, sub, k_at, to);
                load_piece(a.vp, a.vp_stride, page, t, sub, v_at, to + S::TILE);
            }
        }
    };

    f32x16 o[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) o[c] = zeros();
    float m = -INFINITY, ref = 0.f, l = 0.f;  // running maximum (of the unscaled scores), its product with scale2

    int k_lane[4], v_lane[2];  // this lane's places in a tile's blocks
#pragma unroll
    for (int s = 0; s < 4; ++s) k_lane[s] = lr * 128 + ((2 * s + hl) ^ swizzle_k(lr)) * 16;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if constexpr (kBf16) {
            const int row = 4 * hl + ((lane & 15) >> 2), piece = 4 * c + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
            v_lane[c] = row * 128 + (piece ^ swizzle_v<ES>(row)) * 16 + (lane & 1) * 8;
        } else {
            v_lane[c] = 4 * hl * 128 + lr * 4;
        }
    }
    // Words of the values of channels 32 c + lane of the tile vt: the left operand of the second product.
    auto value = [&](const char* vt, int c, int kg, int st) {  // bf16: 16 keys
        // four keys of one channel per transposing read
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = kg * 32 + 16 * st + 8 * e;
            const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(
                vt + (c >> 1) * BN * 128 + row * 128 + v_lane[c & 1]));
            const u32x2 z = __builtin_bit_cast(u32x2, y);
            v[2 * e] = z.x;
            v[2 * e + 1] = z.y;
        }
        return v;
    };
    auto value32 = [&](const char* vt, int c, int kg, int i) {  // fp32: two keys
        return *reinterpret_cast<const float*>(vt + c * BN * 128 + (kg * 32 + 8 * (i >> 2) + (i & 3)) * 128 + v_lane[0]);
    };
    // bits of the bf16 of a word that are not finite
    auto odd_bits = [](uint32_t v) {
        return ((v & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((v & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
    };

    // One tile of the wave's rows.  EDGE: some key of it is not visible to some row.
    auto work = [&](const char* kt, int base, int lo, int hi, int absent, auto edge) {
        constexpr bool EDGE = decltype(edge)::value;
        const char* vt = kt + S::TILE;
        f32x16 x[KG];
#pragma unroll
        for (int kg = 0; kg < KG; ++kg) {
            x[kg] = zeros();
#pragma unroll
            for (int s = 0; s < QW; ++s) {
                const u32x4 k = *reinterpret_cast<const u32x4*>(kt + (s / 4) * BN * 128 + kg * 32 * 128 + k_lane[s & 3]);
                if constexpr (kBf16) {
                    x[kg] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, k),
                                                                    __builtin_bit_cast(bf16x8, q[s]), x[kg], 0, 0, 0);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[kg] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(k[i]), __uint_as_float(q[s][i]),
                                                                     x[kg], 0, 0, 0);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        float top = -INFINITY;
#pragma unroll
        for (int kg = 0; kg < KG; ++kg)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if constexpr (EDGE) {
                    const int at = kg * 32 + 8 * (i >> 2) + 4 * hl + (i & 3), t = base + at;
                    const bool on = (t >= lo) & (t < hi) & (t <= p) & ((t >= p_near) | (t < a.sinks)) &
                                    !((absent >> (at / kPage)) & 1);
                    x[kg][i] = on ? x[kg][i] : -INFINITY;
                }
                top = fmaxf(top, x[kg][i]);
            }
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        // The maximum is followed where it has grown by more than 2^8: weights stay below 2^8 otherwise, which
        // neither their rounding nor the sums mind
        const bool up = (top - m) * scale2 > 8.f;
        if (__any(up)) {
            const float now = up ? top : m, r = now == -INFINITY ? 0.f : now * scale2;
            const float keep = exp2_hw(m == -INFINITY ? -INFINITY : ref - r);
            l *= keep;
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[c][i] *= keep;
            m = now;
            ref = r;
        }
        uint32_t pf[KG][8];
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kg = 0; kg < KG; ++kg)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[kg][i] = exp2_hw(__builtin_fmaf(x[kg][i], scale2, -ref));
                sum[i & 3] += x[kg][i];
            }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        // bf16: the weights are rounded to 8 bits for the product, as the output is; the sum l has them unrounded
        if constexpr (kBf16) {
#pragma unroll
            for (int kg = 0; kg < KG; ++kg)
#pragma unroll
                for (int i = 0; i < 16; i += 2) pf[kg][i / 2] = pack_bf16(x[kg][i], x[kg][i + 1]);
        }
        // In a tile with hidden keys, values that are not finite count as 0: a hidden one's weight of 0 would make
        // them NaN.  Their sight makes the sums NaN below.
        uint32_t odd = 0;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
#pragma unroll
            for (int kg = 0; kg < KG; ++kg) {
                if constexpr (kBf16) {
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        u32x4 v = value(vt, c, kg, st);
                        if constexpr (EDGE) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t y = odd_bits(v[i]);
                                odd |= y;
                                v[i] &= ~y;
                            }
                        }
                        const u32x4 y = {pf[kg][4 * st], pf[kg][4 * st + 1], pf[kg][4 * st + 2], pf[kg][4 * st + 3]};
                        o[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v),
                                                                       __builtin_bit_cast(bf16x8, y), o[c], 0, 0, 0);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float v = value32(vt, c, kg, i);
                        if constexpr (EDGE) {
                            const bool y = !(fabsf(v) < INFINITY);
                            odd |= y;
                            v = y ? 0.f : v;
                        }
                        o[c] = __builtin_amdgcn_mfma_f32_32x32x2f32(v, x[kg][i], o[c], 0, 0, 0);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (EDGE) {
            if (__any(odd != 0)) {  // how many such values each sum has a weight for
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    f32x16 count = zeros();
#pragma unroll
                    for (int kg = 0; kg < KG; ++kg) {
                        if constexpr (kBf16) {
#pragma unroll
                            for (int st = 0; st < 2; ++st) {
                                u32x4 v = value(vt, c, kg, st), y;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint32_t z = pf[kg][4 * st + i];
                                    v[i] = odd_bits(v[i]) & 0x3F803F80u;
                                    y[i] = ((z & 0x7FFFu) ? 0x3F80u : 0u) | ((z & 0x7FFF0000u) ? 0x3F800000u : 0u);
                                }
                                count = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                    __builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, y), count, 0, 0, 0);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                count = __builtin_amdgcn_mfma_f32_32x32x2f32(
                                    fabsf(value32(vt, c, kg, i)) < INFINITY ? 0.f : 1.f, x[kg][i] != 0.f ? 1.f : 0.f, count,
                                    0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[c][i] = count[i] > 0.f ? NAN : o[c][i];
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    };
    auto tile = [&](int t, const char* kt, int absent) {
        const bool sink = t < head_tiles;
        const int base = base_of(t), lo = sink ? 0 : near, hi = sink ? head : end;
        if (!active || base > pw_last) return;
        const bool whole = absent == 0 && base >= lo && base + BN <= hi && base + BN - 1 <= pw_first &&
                           (a.window == 0 || base > pw_last - a.window || base + BN <= a.sinks);
        if (whole) work(kt, base, lo, hi, 0, std::false_type{});
        else work(kt, base, lo, hi, absent, std::true_type{});
    };

    if constexpr (ROWS) {
        const int steps = t1 - t0;
        auto absent_of = [&](const int* on) {
            int x = 0;
#pragma unroll
            for (int s = 0; s < SUBS; ++s) x |= (on[s] ? 0 : 1) << s;
            return __builtin_amdgcn_readfirstlane(x);
        };
        if (steps > 0) load(0, s_kv[0][0], s_on[0]);
        for (int i = 0; i < steps; ++i) {
            wait_loads();
            __syncthreads();  // tile i is there, and the other buffer has been read
            load(i + 1, s_kv[0][(i + 1) & 1], s_on[(i + 1) & 1]);
            tile(t0 + i, s_kv[0][i & 1], absent_of(s_on[i & 1]));
        }
    } else {
        const int steps = t1 - t0 - w > 0 ? (t1 - t0 - w + WAVES - 1) / WAVES : 0;
        auto absent_of = [&](int i) {
            int x = 0;
#pragma unroll
            for (int s = 0; s < SUBS; ++s) x |= (__builtin_amdgcn_readlane(lane_page, (i % PER) * SUBS + s) < 0 ? 1 : 0) << s;
            return x;
        };
        int on = 0;
        if (steps > 0) {
            load(0, s_kv[w][0], nullptr);
            on = absent_of(0);
        }
        for (int i = 0; i < steps; ++i) {
            int then = 0;
            wait_loads();
            if (i + 1 < steps) {
                load(i + 1, s_kv[w][(i + 1) & 1], nullptr);
                then = absent_of(i + 1);
            }
            tile(t0 + w + WAVES * i, s_kv[w][i & 1], on);
            on = then;
        }
    }

    l += __shfl_xor(l, 32, 64);
    const int64_t out_row = token * a.Hq + h * G + my_g;
    auto finish = [&](float M, float L, int64_t row) {  // log-sum of a row
        if (a.lse) a.lse[row] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
    };
    if constexpr (ROWS) {
        if (!mine) return;
        const float base = m == -INFINITY ? -INFINITY : ref;
        if (plan.parts > 1) {
            if (hl == 0) part_ml[out_row * plan.parts + part] = make_float2(base, l);
            if (l == 0.f) return;
            float* to = part_o + (out_row * plan.parts + part) * D;
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<f32x4*>(to + c * 32 + 8 * e + 4 * hl) =
                        f32x4{o[c][4 * e], o[c][4 * e + 1], o[c][4 * e + 2], o[c][4 * e + 3]};
            return;
        }
        if (hl == 0) finish(base, l, out_row);
        const float f = l == 0.f ? 0.f : 1.f / l;
        T* to = static_cast<T*>(a.o) + out_row * D;
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x4 y = {o[c][4 * e] * f, o[c][4 * e + 1] * f, o[c][4 * e + 2] * f, o[c][4 * e + 3] * f};
                T* at = to + c * 32 + 8 * e + 4 * hl;
                if constexpr (kBf16) *reinterpret_cast<u32x2*>(at) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
                else *reinterpret_cast<f32x4*>(at) = y;
            }
    } else {
        // join the waves: their sums go where the tiles were, half of the channels into each buffer
        constexpr int HALF = D / 2, PITCH = HALF + 4;
        static_assert(32 * PITCH * 4 <= 2 * S::TILE, "half of a wave's outputs fits a buffer");
        const float base = m == -INFINITY ? -INFINITY : ref;
        if (hl == 0) {
            s_m[w][lr] = base;
            s_l[w][lr] = l;
        }
        __syncthreads();
        auto joint = [&](int r) {
            float M = s_m[0][r];
#pragma unroll
            for (int i = 1; i < WAVES; ++i) M = fmaxf(M, s_m[i][r]);
            return M;
        };
        const float M = joint(lr), keep = base == -INFINITY ? 0.f : exp2_hw(base - M);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            float* to = reinterpret_cast<float*>(s_kv[w][c / (CT / 2)]) + lr * PITCH + c % (CT / 2) * 32 + 4 * hl;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<f32x4*>(to + 8 * e) = f32x4{o[c][4 * e] * keep, o[c][4 * e + 1] * keep,
                                                              o[c][4 * e + 2] * keep, o[c][4 * e + 3] * keep};
        }
        __syncthreads();
        for (int x = tid; x < rows * (D / 4); x += S::THREADS) {
            const int r = x / (D / 4), c = x % (D / 4) * 4;
            const float top = joint(r);
            float L = 0.f;
            f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < WAVES; ++i) {
                L += top == -INFINITY ? 0.f : s_l[i][r] * exp2_hw(s_m[i][r] - top);
                const float* from = reinterpret_cast<const float*>(s_kv[i][c / HALF]) + r * PITCH + c % HALF;
                y += *reinterpret_cast<const f32x4*>(from);
            }
            const int ri = (g0 + r) / G;
            const int64_t row = (cu0 + i0 + ri) * a.Hq + h * G + (g0 + r - ri * G);
            if (plan.parts > 1) {
                if (c == 0) part_ml[row * plan.parts + part] = make_float2(top, L);
                *reinterpret_cast<f32x4*>(part_o + (row * plan.parts + part) * D + c) = y;
                continue;
            }
            if (c == 0) finish(top, L, row);
            const float f = L == 0.f ? 0.f : 1.f / L;
            T* at = static_cast<T*>(a.o) + row * D + c;
            if constexpr (kBf16)
                *reinterpret_cast<u32x2*>(at) = u32x2{pack_bf16(y[0] * f, y[1] * f), pack_bf16(y[2] * f, y[3] * f)};
            else *reinterpret_cast<f32x4*>(at) = y * f;
        }
    }
}

// Join of the parts: a wave for a row, its lanes over the channels.
template <typename T, int D>
__global__ __launch_bounds__(256) void prefill_join_kernel(PagedPrefillArgs a, PrefillPlan plan, const float2* part_ml,
                                                           const float* part_o) {
    constexpr int CH = D / 64;
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t token = row / a.Hq;
    // rows of no sequence have no parts and keep what they hold
    if (token >= a.T || token < a.cu[0] || token >= a.cu[a.N]) return;
    const float2 y = lane < plan.parts ? part_ml[row * plan.parts + lane] : make_float2(-INFINITY, 0.f);
    float M = y.x;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
    // (a NaN sum stays: its part takes part)
    const float f = y.y == 0.f ? 0.f : exp2_hw(y.x - M);
    float L = y.y * f;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) L += __shfl_xor(L, off, 64);
    float acc[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) acc[c] = 0.f;
    const float* po = part_o + row * plan.parts * D + lane * CH;
    for (int i = 0; i < plan.parts; ++i) {
        const float part = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(y.y), i));
        const float g = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), i));
        if (part == 0.f) continue;  // its outputs have not been written
#pragma unroll
        for (int c = 0; c < CH; ++c) acc[c] += g * po[(int64_t)i * D + c];
    }
    const float r = L == 0.f ? 0.f : 1.f / L;
    T* to = static_cast<T*>(a.o) + row * D + lane * CH;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int c = 0; c < CH; ++c) to[c] = acc[c] * r;
    } else if constexpr (CH == 1) {
        to[0] = (uint16_t)pack_bf16(acc[0] * r, 0.f);
    } else {
#pragma unroll
        for (int c = 0; c < CH; c += 2) *reinterpret_cast<uint32_t*>(to + c) = pack_bf16(acc[c] * r, acc[c + 1] * r);
    }
    if (a.lse && lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

int64_t div_up(int64_t x, int64_t m) { return (x + m - 1) / m; }

constexpr int kMaxParts = 64;

// Few rows for each sequence: the waves share the rows and split the keys.
bool many_rows(int64_t N, int64_t T, int G) { return T * G > 32 * N; }

PrefillPlan plan_of(int64_t N, int64_t T, int Hq, int Hkv, int d, int es, int64_t max_length, int window, int sinks) {
    const int G = Hq / Hkv, row = d * es;
    const bool rows = many_rows(N, T, G);
    const int rt = rows ? 128 : 32, bn = rows && row <= 256 && es == 2 ? 64 : 32;
    const int waves = rows ? 1 : row <= 256 ? 4 : row == 512 ? 2 : 1;
    PrefillPlan p;
    p.slots = T * G / rt + N;
    int64_t tiles = div_up(max_length, bn);
    if (window > 0 && max_length > window) {
        const int64_t most = div_up(sinks, bn) + div_up((int64_t)window + div_up(rt, G) + 1, bn) + 1;
        tiles = most < tiles + 1 ? most : tiles + 1;
    }
    // parts for two workgroups per CU, of at least four steps each
    const int64_t base = p.slots * Hkv, steps = div_up(tiles, waves);
    int64_t parts = base > 0 ? 512 / base : 1;
    parts = parts < steps / 4 ? parts : steps / 4;
    parts = parts < 1 ? 1 : parts > kMaxParts ? kMaxParts : parts;
    p.part_tiles = (int)(div_up(steps > 0 ? steps : 1, parts) * waves);
    p.parts = (int)(tiles > 0 ? div_up(tiles, p.part_tiles) : 1);
    return p;
}
PrefillPlan plan_of(const PagedPrefillArgs& a) {
    return plan_of(a.N, a.T, a.Hq, a.Hkv, a.d, a.bf16 ? 2 : 4, a.max_length, a.window, a.sinks);
}

template <typename T, int D>
void launch_typed(const PagedPrefillArgs& a, const PrefillPlan& p, float2* ml, float* po, hipStream_t s) {
    const dim3 grid((unsigned)(p.slots * a.Hkv * p.parts));
    if (many_rows(a.N, a.T, a.Hq / a.Hkv))
        hipLaunchKernelGGL((paged_prefill_kernel<T, D, true>), grid, dim3(Shape<T, D, true>::THREADS), 0, s, a, p, ml, po);
    else
        hipLaunchKernelGGL((paged_prefill_kernel<T, D, false>), grid, dim3(Shape<T, D, false>::THREADS), 0, s, a, p, ml, po);
}
template <typename T>
void launch_typed(const PagedPrefillArgs& a, const PrefillPlan& p, float2* ml, float* po, hipStream_t s) {
    if (a.d == 64) launch_typed<T, 64>(a, p, ml, po, s);
    else if (a.d == 128) launch_typed<T, 128>(a, p, ml, po, s);
    else launch_typed<T, 256>(a, p, ml, po, s);
}
template <typename T>
void launch_join(const PagedPrefillArgs& a, const PrefillPlan& p, const float2* ml, const float* po, hipStream_t s) {
    const dim3 grid((unsigned)div_up(a.T * a.Hq, 4)), block(256);
    if (a.d == 64) hipLaunchKernelGGL((prefill_join_kernel<T, 64>), grid, block, 0, s, a, p, ml, po);
    else if (a.d == 128) hipLaunchKernelGGL((prefill_join_kernel<T, 128>), grid, block, 0, s, a, p, ml, po);
    else hipLaunchKernelGGL((prefill_join_kernel<T, 256>), grid, block, 0, s, a, p, ml, po);
}

int64_t ml_bytes(const PagedPrefillArgs& a, const PrefillPlan& p) { return div_up(a.T * a.Hq * p.parts * 8, 256) * 256; }

}  // namespace

int64_t paged_prefill_groups(const PagedPrefillArgs& a, size_t* workspace) {
    *workspace = 0;
    const int64_t slots = a.T * (a.Hq / a.Hkv) / 32 + a.N;  // at most
    if (slots * a.Hkv > max_groups(256)) return slots * a.Hkv;
    const PrefillPlan p = plan_of(a);
    const int64_t groups = p.slots * a.Hkv * p.parts;
    if (p.parts > 1) *workspace = (size_t)(ml_bytes(a, p) + a.T * a.Hq * p.parts * (int64_t)a.d * 4);
    return groups;
}

hipError_t launch_paged_prefill(const PagedPrefillArgs& a, hipStream_t s) {
    if (a.T == 0 || a.N == 0) return hipSuccess;
    const PrefillPlan p = plan_of(a);
    float2* ml = static_cast<float2*>(a.ws);
    float* po = p.parts > 1 ? reinterpret_cast<float*>(static_cast<char*>(a.ws) + ml_bytes(a, p)) : nullptr;
    const bool timed = timing_on();
    if (timed) timed_begin(kKernelPagedPrefill, s);
    if (a.bf16) launch_typed<uint16_t>(a, p, ml, po, s);
    else launch_typed<float>(a, p, ml, po, s);
    hipError_t e = hipGetLastError();
    if (timed) timed_end(s);
    if (e != hipSuccess || p.parts == 1) return e;
    if (timed) timed_begin(kKernelPrefillJoin, s);
    if (a.bf16) launch_join<uint16_t>(a, p, ml, po, s);
    else launch_join<float>(a, p, ml, po, s);
    e = hipGetLastError();
    if (timed) timed_end(s);
    return e;
}

}  // namespace kda
