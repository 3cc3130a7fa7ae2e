// Softmax attention of a chunk of new tokens per sequence over a paged key-value cache (include/kda.h,
// kda_paged_prefill):
//     s_t = scale q . k_t,   out = sum_t exp(s_t - m) v_t / l,   l = sum_t exp(s_t - m),   lse = m + log l
// for the query at position p, over t <= p, with a window over p - window < t <= p and t < sinks.
//
// Rows are (token, query head of the group) pairs of one key-value head, so that the heads that share keys share
// their loads.  Scores are K Q^T and outputs V^T P^T on 32 x 32 matrix instructions: rows of queries are columns of
// both results, so a lane holds values of one query only.  The softmax needs one exchange between the two halves
// of a wave, and the scores that a lane holds are, rounded, its share of the second product's right operand.
//
// With many rows bf16 weights are rounded once for their product with the values, as its operand is; their sum is of the
// weights themselves.  Outputs are then off by 0.0022 of their size instead of 0.0017, the rounding of the outputs alone.
// A second product with what the rounding left, as with few rows, would cost 4.8 ms instead of 3.4 for the long prompt
// below, 138 us instead of 111 for 8 prompts of 48 to 2048 tokens after 1 to 8000, 336 instead of 238 for 4096 tokens after
// 4096 with d = 64.
//
// Many rows are bound by the matrix cores: 8192 tokens after 24576, 32 heads of 128 over 8, bf16, 3.4 to 3.6 ms by the card,
// 1060 to 1140 TFLOP/s (these are busy 64% of the time at the 1.7 GHz that the power then allows; a library's product of
// 8192^3 reaches 1250).  4096 tokens after 4096 with d = 64: 233 to 240 us, 860 to 890 TFLOP/s.
// fp32 with a window of 1024 and d = 64: 300 us, 94 TFLOP/s of visible pairs (busy 77%, of 154 that fp32 products reach).
// Few rows are bound by HBM: 64 sequences of 8192 tokens with 5 new ones each, 374 us, 5.8 TB/s (fp32 5.8).  Short calls
// are bound by latency: 64 tokens alone 12 us, in a chain of segment, length, page and keys.
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
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 16 bytes per lane from a buffer to LDS: lane i's go to at + 16 i; those behind the descriptor's end become 0.  Written
// out, since the compiler would let every read of LDS wait for all such loads, also of those for the next tile.
// (The clobber keeps the compiler's own uses of m0 whole, each of which sets it right before.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds(u32x4 from, int offset, uint32_t more, uint32_t at) {
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
// The same for all but the last N loads (loads of the compiler's that come between make it wait for more).
template <int N>
__device__ __forceinline__ void wait_loads_but() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kPage = 16;  // tokens that surely share a page

// the larger of lane and lane ^ 32
__device__ __forceinline__ float other_half_max(float x) {
    const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
}
// what the rounding of a and b to y has left of them, rounded
__device__ __forceinline__ uint32_t rest_of(float a, float b, uint32_t y) {
    return pack_bf16(a - __uint_as_float(y << 16), b - __uint_as_float(y & 0xFFFF0000u));
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

// How a kernel instance splits its work.
// ROWS (many rows): four waves with 32 rows each share a tile of keys and values, and load the next into a second buffer.
// Otherwise (few rows) the waves share 32 rows and each has tiles of its own, in one buffer: the next keys are asked for
// when the scores are there, the next values behind the outputs, so that twice as many waves' loads are under way.
template <typename T, int D, bool ROWS>
struct Shape {
    static constexpr int ES = sizeof(T), ROW = D * ES;
    static constexpr int BN = ROWS && ROW <= 256 && ES == 2 ? 64 : 32;  // keys of a tile
    static constexpr int WAVES = ROWS ? 4 : ROW <= 256 ? 4 : ROW == 512 ? 2 : 1;
    static constexpr int THREADS = 64 * WAVES;
    static constexpr int RT = ROWS ? 128 : 32;               // rows of a workgroup
    static constexpr int TILE = BN * ROW;                    // bytes of a tile's keys
    static constexpr int BUFS = ROWS ? 2 : WAVES;            // tiles in LDS
    // waves that share a SIMD's registers (bf16, d = 256: with two, 100 registers spill, and their loads wait for the next
    // tile's; 8192 tokens after 8192, 16 heads over 4, 1.53 to 1.58 ms, with two 1.66)
    static constexpr int PER_SIMD = ROW <= (ROWS && ES == 4 ? 512 : 256) ? 2 : 1;
};

// Row tiles of all sequences, not split: tile k of sequence n has slot floor(cu[n] G / RT) + n + k, which leaves every
// sequence enough slots.  The sequence of a slot (wave-uniform), by 64 probes at a time.
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

// The host does not know the lengths, so the work is split on the device: with up to 64 sequences every workgroup looks at
// all of them and comes to the same shares.  A sequence's row tiles are split into parts of at most P steps, P the total
// over kGroups workgroups (a little more where that gives no more parts than those), and the parts are numbered.  With
// more sequences the parts' length goes by the bound of the lengths.  16 sequences with 5 new tokens each, 32 heads over
// 8, after 1000 to 16379 tokens: 84 us, 135 us with parts by the bound; kGroups of 384 and 1024: 89 and 92 us.  Parts of
// 8 steps at least: one such sequence after 8000 tokens takes 24 us instead of 19 with 4; fp32 steps are longer, 14 tokens
// after 471 of 6 heads of 128 over 3: 21 us, with 4 steps at least 42.
constexpr int kMaxParts = 64;
constexpr int kGroups = 512;  // two workgroups per CU (one with many rows and d = 256)
struct PrefillPlan {
    int64_t slots;  // row tiles of a key-value head at most
    int groups;     // workgroups of a head that the chip holds; 0: nothing is split
    int parts, steps;  // parts of a row tile and their steps by the bound; 0: by the lengths
    int least;         // steps of a part at least
};
// A workgroup's share.
struct Item {
    int64_t n, tile;         // the row tile, of sequence n (-1: none)
    int part, parts, steps;  // steps of a part
    int64_t split;           // the row tile's first among the split parts
    int places;              // split parts in all
};

// What the workspace holds: the number of split parts; of each its sequence, row tile, the parts of that and its place
// among them; of the split parts of every head (reference, sum) of the rows, then their outputs [RT, D].
struct Partials {
    int* count;
    int4* part;
    float2* ml;
    float* out;
};
__host__ __device__ __forceinline__ int64_t places_of(int groups) { return 2 * (int64_t)groups; }

// Steps of a row tile that ends at `length`, at most.
__host__ __device__ __forceinline__ int steps_to(const PagedPrefillArgs& a, int64_t length, int RT, int BN, int STEP) {
    const int64_t end = length < 0 ? 0 : length < a.max_length ? length : a.max_length;
    int64_t tiles = (end + BN - 1) / BN;
    if (a.window > 0) {
        const int64_t most = ((int64_t)a.sinks + BN - 1) / BN + ((int64_t)a.window + RT + BN - 1) / BN + 1;
        tiles = tiles + 1 < most ? tiles + 1 : most;
    }
    const int64_t s = (tiles + STEP - 1) / STEP;
    return (int)(s < 1 ? 1 : s);
}

template <int RT, int BN, int STEP>
__device__ __forceinline__ Item item_of(const PagedPrefillArgs& a, const PrefillPlan& plan, int64_t j) {
    const int G = a.Hq / a.Hkv;
    Item x{-1, 0, 0, 1, 0x7FFFFFFF, 0, 0};
    if (plan.groups == 0 || plan.parts > 0) {
        if (plan.parts > 0) {
            x.parts = plan.parts;
            x.steps = plan.steps;
            x.part = (int)(j / plan.slots);
            j %= plan.slots;
            x.split = j * plan.parts;
            x.places = (int)plan.slots * plan.parts;
        }
        j = plan.slots - 1 - j;  // late tiles first: they have the most keys
        x.n = sequence_of(a.cu, a.N, j, G, RT);
        x.tile = j - slot_begin(a.cu, x.n, G, RT);
        return x;
    }
    // a sequence in each lane
    const int lane = threadIdx.x & 63;
    int tiles = 0, steps = 1;
    float work = 0.f;  // twice the steps of all
    if (lane < a.N) {
        const int64_t c0 = a.cu[lane] < 0 ? 0 : a.cu[lane], c1 = a.cu[lane + 1] < a.T ? a.cu[lane + 1] : a.T;
        const int64_t fresh = c1 > c0 ? c1 - c0 : 0, length = a.lengths[lane];
        tiles = (int)((fresh * G + RT - 1) / RT);
        steps = steps_to(a, length, RT, BN, STEP);
        work = (float)tiles * (float)(steps + steps_to(a, length - fresh + RT, RT, BN, STEP));
    }
    float total = work;
    int all = tiles;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        total += __shfl_xor(total, off, 64);
        all += __shfl_xor(all, off, 64);
    }
    all = __builtin_amdgcn_readfirstlane(all);
    // The shares to choose from, one in each lane: P, 1.09 P and so on.  Those from 2 P on split into few enough parts,
    // since a split row tile's parts are at most twice its steps / P.
    const float share = ceilf(total * 1.0001f / (2 * plan.groups));
    const float P = ceilf(fmaxf(fminf(share, 1e7f), (float)plan.least) * exp2_hw(0.125f * lane)), per = 1.f / P;
    auto parts_of = [&](float steps, float P, float per) { return fminf(floorf((steps + P - 1.f) * per), (float)kMaxParts); };
    float parts = 0.f, split = 0.f;
    for (int n = 0; n < a.N; ++n) {
        const float t = (float)__builtin_amdgcn_readlane(tiles, n), s = (float)__builtin_amdgcn_readlane(steps, n);
        const float y = t * fmaxf(parts_of(s, P, per), 1.f);
        parts += y;
        split += y > t ? y : 0.f;
    }
    // (few row tiles: no more parts than groups, if a share below 2 P gives that)
    uint64_t good = __ballot(2 * all > plan.groups || parts <= (float)plan.groups) & 0xFF;
    const uint64_t fits = __ballot(split <= (float)places_of(plan.groups));
    if ((good & fits) == 0) good = ~0ull;
    const int at_lane = __builtin_ctzll(good & fits);
    const float chosen = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(P), at_lane));
    const float chosen_per = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(per), at_lane));
    // the item among the parts of all, late tiles first: they have the most keys
    const int k = (int)fmaxf(parts_of((float)steps, chosen, chosen_per), 1.f), mine = tiles * k, mine_split = k > 1 ? mine : 0;
    int before = mine, split_before = mine_split;  // of this sequence and those behind it
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_down(before, off, 64), z = __shfl_down(split_before, off, 64);
        if (lane + off < 64) before += y, split_before += z;
    }
    const int items = __builtin_amdgcn_readfirstlane(before);
    x.places = __builtin_amdgcn_readfirstlane(split_before);
    before -= mine;
    split_before -= mine_split;
    if (j >= items) return x;
    const int in = __builtin_ctzll(__ballot(before <= (int)j && (int)j < before + mine));
    const int inside = __builtin_amdgcn_readlane(before + mine, in) - 1 - (int)j;
    x.n = in;
    x.parts = __builtin_amdgcn_readlane(k, in);
    x.tile = inside / x.parts;
    x.part = inside - (int)x.tile * x.parts;
    x.steps = (__builtin_amdgcn_readlane(steps, in) + x.parts - 1) / x.parts;
    x.split = x.parts > 1 ? __builtin_amdgcn_readlane(split_before, in) + x.tile * x.parts : 0;
    return x;
}

// A row tile and what its rows see.
struct RowTile {
    int64_t cu0, i0;  // the sequence's first packed token, the tile's first token in it
    int g0, rows;     // the first row's head in the group, rows
    int64_t shift;    // position of the sequence's first new token
    int near, end, head, head_tiles, first, tiles;  // visible: 0 .. head-1 and near .. end-1
    // (64 bits: a contract that is broken gives any)
    __device__ __forceinline__ int position(int r, int G) const {
        const int64_t p = shift + i0 + (g0 + r) / G;
        return (int)(p < -1 ? -1 : p);
    }
};
template <int RT, int BN>
__device__ __forceinline__ bool row_tile_of(const PagedPrefillArgs& a, const Item& x, RowTile& t) {
    if (x.n < 0 || x.tile < 0) return false;
    const int G = a.Hq / a.Hkv;
    t.cu0 = a.cu[x.n] < 0 ? 0 : a.cu[x.n];
    const int64_t cu1 = a.cu[x.n + 1] < a.T ? a.cu[x.n + 1] : a.T, fresh = cu1 - t.cu0, row0 = x.tile * RT;
    if (row0 >= fresh * G) return false;
    t.rows = (int)(fresh * G - row0 < RT ? fresh * G - row0 : RT);
    t.i0 = row0 / G;
    t.g0 = (int)(row0 - t.i0 * G);
    const int length = a.lengths[x.n] > 0 ? a.lengths[x.n] : 0;
    const int cap = length < a.max_length ? length : (int)a.max_length;
    t.shift = length - fresh;
    const int p_first = t.position(0, G), p_last = t.position(t.rows - 1, G);
    t.end = p_last + 1 < cap ? p_last + 1 : cap;
    const int near = a.window > 0 && p_first >= a.window ? p_first - a.window + 1 : 0;
    t.near = near < t.end ? near : t.end;
    t.head = a.sinks < t.near ? a.sinks : t.near;
    t.head_tiles = (t.head + BN - 1) / BN;
    t.first = t.near / BN;
    t.tiles = t.head_tiles + (t.end + BN - 1) / BN - t.first;
    return true;
}
// Parts that a row tile has in fact (the steps that decide on them are an upper bound).
__device__ __forceinline__ int parts_in_fact(const Item& x, const RowTile& t, int STEP) {
    if (x.parts == 1) return 1;
    const int per = x.steps * STEP, y = (t.tiles + per - 1) / per;
    return y < 1 ? 1 : y;
}


template <typename T, int D, bool ROWS>
__global__ __launch_bounds__((Shape<T, D, ROWS>::THREADS), (Shape<T, D, ROWS>::PER_SIMD)) void paged_prefill_kernel(
    PagedPrefillArgs a, PrefillPlan plan, Partials ws) {
    using S = Shape<T, D, ROWS>;
    constexpr bool kBf16 = std::is_same<T, uint16_t>::value;
    constexpr int ES = S::ES, ROW = S::ROW, BN = S::BN, WAVES = S::WAVES, RT = S::RT, KG = BN / 32, CT = D / 32;
    constexpr int LOADS = kPage * ROW / 1024;      // 1 KiB loads of 16 rows
    constexpr int QW = ROW / 32;                   // 16-byte pieces of a lane's query row
    __shared__ __attribute__((aligned(1024))) char s_kv[S::BUFS][2 * S::TILE];  // keys, values
    __shared__ float s_m[WAVES][32], s_l[WAVES][32];

    const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, hl = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = a.Hq / a.Hkv;
    // heads fastest: workgroups of one head go to the same XCDs where the heads divide the eight, whose L2 then
    // holds that head's keys
    const int h = (int)(blockIdx.x % a.Hkv);
    const Item item = item_of<RT, BN, ROWS ? 1 : WAVES>(a, plan, blockIdx.x / a.Hkv);
    RowTile tile;
    const bool any = row_tile_of<RT, BN>(a, item, tile);
    const int parts = any ? parts_in_fact(item, tile, ROWS ? 1 : WAVES) : 0;
    if (plan.groups && h == 0 && tid == 0) {  // for the join
        const int64_t place = item.split + item.part;
        if (blockIdx.x == 0) *ws.count = item.places;
        if (item.parts > 1 && place < places_of(plan.groups))
            ws.part[place] = make_int4((int)item.n, (int)item.tile, parts, item.part);
    }
    if (item.part >= parts || (parts > 1 && item.split + item.part >= places_of(plan.groups))) return;
    const int64_t cu0 = tile.cu0, i0 = tile.i0;
    const int g0 = tile.g0, rows = tile.rows, near = tile.near, end = tile.end, head = tile.head;
    const int head_tiles = tile.head_tiles, first = tile.first, tiles = tile.tiles;
    const int part_tiles = parts > 1 ? item.steps * (ROWS ? 1 : WAVES) : tiles;
    const int t0 = item.part * part_tiles, t1 = t0 + part_tiles < tiles ? t0 + part_tiles : tiles;
    auto position = [&](int r) { return tile.position(r, G); };

    // this lane's row, and its row of q and out (formed again behind the loop, where registers are free)
    const int my = ROWS ? w * 32 + lr : lr;
    const bool mine = my < rows;
    auto token_of = [&](int r) { return cu0 + i0 + (g0 + r) / G; };
    auto head_of = [&](int r) { return h * G + (g0 + r) % G; };
    const int wave_first = ROWS ? w * 32 : 0, wave_rows = rows - wave_first < 32 ? rows - wave_first : 32;
    const int pw_first = position(wave_rows > 0 ? wave_first : 0), pw_last = position(wave_rows > 0 ? wave_first + wave_rows - 1 : 0);
    const int p = mine ? position(my) : pw_last;
    const int p_near = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
    const int p_near_last = a.window > 0 && pw_last >= a.window ? pw_last - a.window + 1 : 0;
    const bool active = wave_rows > 0;

    // The scores' sign goes to the queries, so that the factor is positive; a scale of 0 makes them 0.
    const float scale2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
    u32x4 q[QW];
    {
        const T* qr = static_cast<const T*>(a.q) + token_of(mine ? my : 0) * a.q_stride + (int64_t)head_of(mine ? my : 0) * D;
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

    // Loads of tiles.  The lanes hold the pages of the wave's next tiles, a lane for each 16-token piece, and those of
    // the tiles behind these are on their way.
    constexpr int SUBS = BN / kPage;            // pieces of a tile
    constexpr int STEP = ROWS ? 1 : WAVES;      // tiles between a wave's
    constexpr int PER = 64 / SUBS;              // tiles that the lanes cover
    const int w0 = ROWS ? 0 : w;
    const int near_shift = (first - head_tiles) * BN;
    auto base_of = [&](int t) { return t * BN + (t < head_tiles ? 0 : near_shift); };
    uint64_t lane_k = 0, lane_v = 0;  // byte offsets of the pieces in the pools
    uint64_t absent = ~0ull;          // lanes without a page
    int next_page = -1, next_slot = 0;
    auto look_up = [&](int i) {  // for the wave's tiles i .. i + PER - 1
        const int t = t0 + w0 + STEP * (i + lane / SUBS);
        next_page = -1;
        if (t < t1) {
            const uint32_t pos = base_of(t) + lane % SUBS * kPage, col = pos / (uint32_t)a.page_size;
            next_slot = (int)(pos - col * (uint32_t)a.page_size);
            if (col < (uint32_t)a.pt.width) next_page = a.pt.table[item.n * a.pt.stride + col];
        }
    };
    auto advance = [&](int i) {
        const bool on = next_page >= 0 && next_page < a.pt.n_pages;
        const int64_t page = on ? next_page : 0, inner = ((int64_t)h * a.page_size + (on ? next_slot : 0)) * D;
        lane_k = (uint64_t)(page * a.kp_stride + inner) * ES;
        lane_v = (uint64_t)(page * a.vp_stride + inner) * ES;
        absent = __ballot(!on);
        look_up(i + PER);
    };
    // byte offsets of this lane's 16 bytes inside rows 0 .. 7 and 8 .. 15 of a piece
    int k_at[2], v_at[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = 8 * e + lane / 8;
        k_at[e] = r * ROW + ((lane % 8) ^ swizzle_k(r)) * 16;
        v_at[e] = r * ROW + ((lane % 8) ^ swizzle_v<ES>(r)) * 16;
    }
    const uint32_t lds = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)s_kv[ROWS ? 0 : w]);
    // A wave's loads of a tile: PIECES pieces (keys or values of 16 tokens) of LOADS loads each, from the page to their
    // place in LDS.  Rows behind the last visible one, without a page or behind the last tile become 0.
    constexpr int PIECES = ROWS ? 2 * SUBS / WAVES : 2 * SUBS, ALL_LOADS = PIECES * LOADS;
    u32x4 from;
    struct Next {
        int i, base, limit;  // the wave's tile, its first token, the end of what is visible
    };
    auto next_of = [&](int i) {
        const int t = t0 + w0 + STEP * i, sink = t < head_tiles;
        const int base = t * BN + (sink ? 0 : near_shift), limit = sink ? head : end;
        return Next{i, base, t < t1 ? limit : 0};
    };
    auto load = [&](const Next& x, int n) {  // load n of a tile
        const int i = x.i, u = n / LOADS, e = n % LOADS;
        // rows: piece w of the keys, then of the values (or one of these); else all of the keys, then of the values
        const int sub = ROWS ? w % SUBS : u % SUBS;
        const bool keys = ROWS ? (PIECES == 2 ? u == 0 : w < SUBS) : u < SUBS;
        if (e == 0) {
            const int lane_of = i % PER * SUBS + sub;
            const uint64_t at = keys ? lane_k : lane_v;
            const uint64_t y = reinterpret_cast<uint64_t>(keys ? a.kp : a.vp) +
                               ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(at >> 32), lane_of) << 32 |
                                (uint32_t)__builtin_amdgcn_readlane((uint32_t)at, lane_of));
            const int left = min(max(x.limit - x.base - sub * kPage, 0), kPage);
            const int on = (absent >> lane_of) & 1 ? 0 : left;
            from = u32x4{(uint32_t)y, (uint32_t)(y >> 32) & 0xFFFFu, (uint32_t)(on * ROW), 0x00020000u};
#pragma unroll
            for (int c = 0; c < 3; ++c) from[c] = __builtin_amdgcn_readfirstlane(from[c]);  // says that it is uniform
        }
        load_lds(from, (keys ? k_at : v_at)[e & 1], (e >> 1) * 128,
                 lds + (ROWS ? (i & 1) * 2 * S::TILE : 0) + (keys ? 0 : S::TILE) + (e >> 1) * BN * 128 + sub * kPage * 128 + (e & 1) * 1024);
    };
    auto load_some = [&](const Next& x, int from, int to) {
#pragma unroll
        for (int n = from; n < to; ++n) load(x, n);
    };
    auto absent_of = [&](int i) { return (int)(absent >> (i % PER * SUBS)) & ((1 << SUBS) - 1); };

    f32x16 o[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) o[c] = zeros();
    // The reference of a row's weights is the largest (unscaled) score of the first tile in which it sees a key, and
    // stays: larger scores later give weights above 1, with the same relative precision, and nothing has to be
    // rescaled or compared.  Only where sums have left the range of fp32 in the end (a score beyond the reference by
    // some 80), the largest score of all is looked for in another pass and the row's sums are formed again.
    float m = -INFINITY, ref = 0.f;  // reference, its product with scale2 (0 while there is none)
    int pass = 0;
    bool left = false;  // this row's sums have left the range
    uint32_t spoiled[CT / 2];  // outputs that a value which is not finite enters, a bit for each
#pragma unroll
    for (int c = 0; c < CT / 2; ++c) spoiled[c] = 0;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};

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
    // The bits of the bf16 of a word that are not finite: an exponent of ones carries into the sign's place.
    auto odd_bits = [](uint32_t v) {
        const uint32_t s = ((v & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
        return (s << 1) - (s >> 15);
    };

    // One tile that every row of the wave sees whole.  What is read from LDS is a stream of 16-byte pieces per lane:
    // the keys' in order, then the values'.  Six of them are on their way, each is used by the products of one step
    // and replaced by the next; the softmax of the first 32 keys goes under the score products of the second, that of the
    // second under the outputs of the first, and what it takes to ask for the next tile under the scores.  The order is
    // written out, since the compiler's own asks LDS for each
    // piece right before its use.
    constexpr int NK = QW, NV = kBf16 ? 2 * CT : 4 * CT;  // pieces of 32 keys, and of their values
    constexpr int AHEAD = ROWS && ROW == 512 && !kBf16 ? 4 : 6;
    constexpr int EACH = (ALL_LOADS + KG * NK - 1) / (KG * NK);  // loads of the next tile under each of the first steps
    auto work = [&](const char* kt, const Next& next) {
        const char* vt = kt + S::TILE;
        auto piece = [&](int j) {
            u32x4 y;
            if (j < KG * NK) {
                y = *reinterpret_cast<const u32x4*>(kt + (j % NK / 4) * BN * 128 + (j / NK) * 32 * 128 + k_lane[j % NK & 3]);
            } else {
                const int kg = (j - KG * NK) / NV, at = (j - KG * NK) % NV, c = at % CT;
                if constexpr (kBf16) {
                    y = value(vt, c, kg, at / CT);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = __float_as_uint(value32(vt, c, kg, at / CT * 4 + i));
                }
            }
            return y;
        };
        f32x16 x[KG];
        float e[KG][16];      // weights
        u32x4 rounded[KG][2];
        auto weights = [&](int kg, int from, int to) {
#pragma unroll
            for (int i = from; i < to; ++i) {
                e[kg][i] = exp2_hw(__builtin_fmaf(x[kg][i], scale2, -ref));
                sum[i & 3] += e[kg][i];
                if (kBf16 && (i & 1)) rounded[kg][i / 8][i % 8 / 2] = pack_bf16(e[kg][i - 1], e[kg][i]);
            }
        };
        u32x4 ring[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) ring[j] = piece(j);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < KG * (NK + NV); ++j) {
            const u32x4 y = ring[j % AHEAD];
            if (j < KG * NK) {
                const int kg = j / NK, s = j % NK;
                if (s == 0) x[kg] = zeros();
                if constexpr (kBf16) {
                    x[kg] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, y),
                                                                    __builtin_bit_cast(bf16x8, q[s]), x[kg], 0, 0, 0);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[kg] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(y[i]), __uint_as_float(q[s][i]),
                                                                     x[kg], 0, 0, 0);
                }
                // (not in the first step: the last product of the scores takes a while)
                if (kg > 0 && s > 0) weights(kg - 1, 16 * (s - 1) / (NK - 1), 16 * s / (NK - 1));
            } else {
                const int kg = (j - KG * NK) / NV, at = (j - KG * NK) % NV, c = at % CT, part = at / CT;
                if (kg == 0 && at == 0 && KG == 1) weights(0, 0, 16);
                if constexpr (kBf16) {
                    o[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8, y), __builtin_bit_cast(bf16x8, rounded[kg][part]), o[c], 0, 0, 0);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[c] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(y[i]), e[kg][4 * part + i], o[c], 0, 0, 0);
                }
                if (kg + 1 < KG && at > 0) weights(kg + 1, 16 * (at - 1) / (NV - 1), 16 * at / (NV - 1));
            }
            if (j + AHEAD < KG * (NK + NV)) ring[j % AHEAD] = piece(j + AHEAD);
            if (j < (ALL_LOADS + EACH - 1) / EACH) {
#pragma unroll
                for (int n = j * EACH; n < (j + 1) * EACH && n < ALL_LOADS; ++n) load(next, n);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // What this lane's row sees of a tile that begins at token `base`: places first .. first + many - 1, and the sinks' 0 ..
    // more - 1, for this lane's half, but for the pieces that are gone.
    struct Seen {
        int top, first, many, less, more, gone;  // no place from `top` on
        __device__ __forceinline__ bool operator()(int kg, int i) const {
            const int at = kg * 32 + 8 * (i >> 2) + (i & 3);
            return (((uint32_t)(first + at) < (uint32_t)many) | ((uint32_t)(less + at) < (uint32_t)more)) &
                   !((gone >> (at / kPage)) & 1);
        }
    };
    auto seen_from = [&](int base, int lo, int hi, int gone) {
        const int top = (hi - 1 < p ? hi - 1 : p) - base + 1;
        const int from = (lo > p_near ? lo : p_near) - base, many = top > from ? top - from : 0;
        const int sink = (a.sinks < base + top ? a.sinks : base + top) - lo, more = sink > 0 ? sink : 0;
        return Seen{top, 4 * hl - from, many, 4 * hl - (lo - base), more, gone};
    };

    // One tile of which some key is not visible to some row (`hidden`), or where some row has no reference yet.
    auto work_edge = [&](const char* kt, int base, int lo, int hi, int gone, bool hidden, const Next& next) {
        const char* vt = kt + S::TILE;
        if constexpr (!ROWS) wait_loads_but<ALL_LOADS / 2>();
        f32x16 x[KG];
        u32x4 ring[AHEAD];
        auto key = [&](int j) {
            return *reinterpret_cast<const u32x4*>(kt + (j % NK / 4) * BN * 128 + (j / NK) * 32 * 128 + k_lane[j % NK & 3]);
        };
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) ring[j] = key(j);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < KG * NK; ++j) {
            const u32x4 k = ring[j % AHEAD];
            const int kg = j / NK, s = j % NK;
            if (s == 0) x[kg] = zeros();
            if constexpr (kBf16) {
                x[kg] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, k),
                                                                __builtin_bit_cast(bf16x8, q[s]), x[kg], 0, 0, 0);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[kg] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(k[i]), __uint_as_float(q[s][i]), x[kg], 0, 0, 0);
            }
            if (j + AHEAD < KG * NK) ring[j % AHEAD] = key(j + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!ROWS) {
            wait_loads_but<ALL_LOADS / 2>();
            load_some(next, 0, ALL_LOADS / 2);
        }
        if (hidden) {
            const auto seen = seen_from(base, lo, hi, gone);
            if (a.window == 0 && gone == 0) {  // (from and lo are 0 or before the tile)
#pragma unroll
                for (int kg = 0; kg < KG; ++kg)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        x[kg][i] = kg * 32 + 8 * (i >> 2) + (i & 3) < seen.top - 4 * hl ? x[kg][i] : -INFINITY;
            } else {
#pragma unroll
                for (int kg = 0; kg < KG; ++kg)
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[kg][i] = seen(kg, i) ? x[kg][i] : -INFINITY;
            }
        }
        if (pass == 1 || __any(m == -INFINITY)) {
            float top = -INFINITY;
#pragma unroll
            for (int kg = 0; kg < KG; ++kg)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, x[kg][i]);
            top = other_half_max(top);
            m = pass == 1 && left ? fmaxf(m, top) : m == -INFINITY ? top : m;
            ref = m == -INFINITY ? 0.f : m * scale2;
        }
        uint32_t pf[KG][8], pr[KG][8];
#pragma unroll
        for (int kg = 0; kg < KG; ++kg)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[kg][i] = exp2_hw(__builtin_fmaf(x[kg][i], scale2, -ref));
                sum[i & 3] += x[kg][i];
            }
        if constexpr (kBf16) {
#pragma unroll
            for (int kg = 0; kg < KG; ++kg)
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    pf[kg][i / 2] = pack_bf16(x[kg][i], x[kg][i + 1]);
                    if (!ROWS) pr[kg][i / 2] = rest_of(x[kg][i], x[kg][i + 1], pf[kg][i / 2]);
                }
        }
        // In a tile with hidden keys, values that are not finite count as 0: a hidden one's weight of 0 would make them
        // NaN.  The outputs that see them are noted below.
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!ROWS) wait_loads_but<ALL_LOADS / 2>();
        auto val = [&](int j) {
            const int kg = j / NV, c = j % NV % CT, part = j % NV / CT;
            u32x4 y;
            if constexpr (kBf16) {
                y = value(vt, c, kg, part);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = __float_as_uint(value32(vt, c, kg, part * 4 + i));
            }
            return y;
        };
        bool odd = false;
        if (hidden) {
            // the largest as unsigned and as signed numbers: a NaN or infinity of either sign is above the finite ones there
            if constexpr (kBf16) {
                s16x2 most = {0, 0};
                u16x2 least = {0, 0};
#pragma unroll
                for (int j = 0; j < KG * NV; ++j) {
                    const u32x4 y = val(j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        most = __builtin_elementwise_max(most, __builtin_bit_cast(s16x2, (uint32_t)y[i]));
                        least = __builtin_elementwise_max(least, __builtin_bit_cast(u16x2, (uint32_t)y[i]));
                    }
                }
                odd = max(most[0], most[1]) >= 0x7F80 || max(least[0], least[1]) >= 0xFF80;
            } else {
                int most = 0;
                uint32_t least = 0;
#pragma unroll
                for (int j = 0; j < KG * NV; ++j) {
                    const u32x4 y = val(j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        most = max(most, (int)y[i]);
                        least = max(least, (uint32_t)y[i]);
                    }
                }
                odd = most >= 0x7F800000 || least >= 0xFF800000u;
            }
            odd = __any(odd);
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) ring[j] = val(j);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < KG * NV; ++j) {
            u32x4 v = ring[j % AHEAD];
            const int kg = j / NV, c = j % NV % CT, part = j % NV / CT;
            if (odd) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (kBf16) v[i] &= ~odd_bits(v[i]);
                    else v[i] = fabsf(__uint_as_float(v[i])) < INFINITY ? v[i] : 0u;
                }
            }
            if constexpr (kBf16) {
                const u32x4 y = {pf[kg][4 * part], pf[kg][4 * part + 1], pf[kg][4 * part + 2], pf[kg][4 * part + 3]};
                o[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v),
                                                               __builtin_bit_cast(bf16x8, y), o[c], 0, 0, 0);
                if constexpr (!ROWS) {
                    const u32x4 z = {pr[kg][4 * part], pr[kg][4 * part + 1], pr[kg][4 * part + 2], pr[kg][4 * part + 3]};
                    o[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v),
                                                                   __builtin_bit_cast(bf16x8, z), o[c], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[c] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(v[i]), x[kg][4 * part + i], o[c], 0, 0, 0);
            }
            if (j + AHEAD < KG * NV) ring[j % AHEAD] = val(j + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (odd) {  // how many such values each row sees: a weight of 0 makes NaN of them too, as it does in other tiles
            const auto seen = seen_from(base, lo, hi, gone);
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
                                v[i] = odd_bits(v[i]) & 0x3F803F80u;
                                y[i] = (seen(kg, 8 * st + 2 * i) ? 0x3F80u : 0u) | (seen(kg, 8 * st + 2 * i + 1) ? 0x3F800000u : 0u);
                            }
                            count = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                __builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, y), count, 0, 0, 0);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            count = __builtin_amdgcn_mfma_f32_32x32x2f32(
                                fabsf(value32(vt, c, kg, i)) < INFINITY ? 0.f : 1.f, seen(kg, i) ? 1.f : 0.f, count,
                                0, 0, 0);
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) spoiled[c / 2] |= (count[i] > 0.f ? 1u : 0u) << (c % 2 * 16 + i);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (!ROWS) {
            wait_loads_but<ALL_LOADS / 2>();
            load_some(next, ALL_LOADS / 2, ALL_LOADS);
        }
    };
    // The same for few rows: keys and values wait for their own loads, and ask for the next ones behind their last use.
    auto work_keys = [&](const char* kt, const Next& next) {
        const char* vt = kt + S::TILE;
        f32x16 x = zeros();
        u32x4 ring[AHEAD];
        wait_loads_but<ALL_LOADS / 2>();
        auto key = [&](int s) {
            return *reinterpret_cast<const u32x4*>(kt + (s / 4) * BN * 128 + k_lane[s & 3]);
        };
#pragma unroll
        for (int s = 0; s < AHEAD && s < NK; ++s) ring[s] = key(s);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < NK; ++s) {
            const u32x4 y = ring[s % AHEAD];
            if constexpr (kBf16) {
                x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, y),
                                                            __builtin_bit_cast(bf16x8, q[s]), x, 0, 0, 0);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(y[i]), __uint_as_float(q[s][i]), x, 0, 0, 0);
            }
            if (s + AHEAD < NK) ring[s % AHEAD] = key(s + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_loads_but<ALL_LOADS / 2>();  // (the keys have been read)
        load_some(next, 0, ALL_LOADS / 2);
        float e[16];
        u32x4 high[2], rest[2];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            e[i] = exp2_hw(__builtin_fmaf(x[i], scale2, -ref));
            sum[i & 3] += e[i];
            if (kBf16 && (i & 1)) {
                high[i / 8][i % 8 / 2] = pack_bf16(e[i - 1], e[i]);
                rest[i / 8][i % 8 / 2] = rest_of(e[i - 1], e[i], high[i / 8][i % 8 / 2]);
            }
        }
        wait_loads_but<ALL_LOADS / 2>();
        auto val = [&](int j) {
            u32x4 y;
            if constexpr (kBf16) {
                y = value(vt, j % CT, 0, j / CT);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = __float_as_uint(value32(vt, j % CT, 0, j / CT * 4 + i));
            }
            return y;
        };
#pragma unroll
        for (int j = 0; j < AHEAD && j < NV; ++j) ring[j] = val(j);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const u32x4 y = ring[j % AHEAD];
            const int c = j % CT, part = j / CT;
            if constexpr (kBf16) {
                o[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, y),
                                                               __builtin_bit_cast(bf16x8, high[part]), o[c], 0, 0, 0);
                o[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, y),
                                                               __builtin_bit_cast(bf16x8, rest[part]), o[c], 0, 0, 0);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[c] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(y[i]), e[4 * part + i], o[c], 0, 0, 0);
            }
            if (j + AHEAD < NV) ring[j % AHEAD] = val(j + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_loads_but<ALL_LOADS / 2>();  // (the values have been read)
        load_some(next, ALL_LOADS / 2, ALL_LOADS);
    };

    // tiles that every row of the wave sees whole: from the last row's window on, up to the first row's position
    bool ready = false;  // all rows of the wave have a reference
    const int whole_lo = p_near_last > near ? p_near_last : near, whole_hi = pw_first + 1 < end ? pw_first + 1 : end;
    const int whole_t0 = head_tiles - first + (whole_lo + BN - 1) / BN, whole_t1 = head_tiles - first + whole_hi / BN;
    auto hides = [&](int i) {
        const int t = t0 + w0 + STEP * i;
        return absent_of(i) != 0 || t < whole_t0 || t >= whole_t1;
    };
    auto whole = [&](int i) { return ready && !hides(i); };
    auto begin = [&](int i) {
        if ((i + 1) % PER == 0) advance(i + 1);
        if constexpr (ROWS) {  // tile i is there, and the other buffer has been read
            wait_loads();
            __syncthreads();
        }
    };

    const int steps = t1 - t0 - w0 > 0 ? (t1 - t0 - w0 + STEP - 1) / STEP : 0;
    float l;
    for (;; ++pass) {
        ready = pass == 2;
        look_up(0);
        advance(0);
        load_some(next_of(0), 0, ALL_LOADS);
        // (two loops, since the compiler would copy the outputs for every tile where two paths of one loop change them)
        for (int i = 0; i < steps;) {
            for (; i < steps && !whole(i); ++i) {
                const int t = t0 + w0 + STEP * i, base = base_of(t), gone = absent_of(i);
                const bool hidden = hides(i);
                begin(i);
                if constexpr (ROWS) {
                    load_some(next_of(i + 1), 0, ALL_LOADS);
                    if (!active || base > pw_last) continue;
                }
                work_edge(s_kv[ROWS ? i & 1 : w], base, t < head_tiles ? 0 : near, t < head_tiles ? head : end, gone,
                          hidden, next_of(i + 1));
                ready = pass != 1 && !__any(m == -INFINITY);
            }
            for (; i < steps && whole(i); ++i) {
                begin(i);
                if constexpr (ROWS) work(s_kv[i & 1], next_of(i + 1));
                else work_keys(s_kv[w], next_of(i + 1));
            }
        }
        wait_loads();
        l = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (pass == 2) break;
        bool again = pass == 1;
        if (pass == 0) {
            float odd = l * 0.f;
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) odd = __builtin_fmaf(o[c][i], 0.f, odd);
            left = odd != odd;
            left = left | (__shfl_xor((int)left, 32, 64) != 0);
            again = __any(left);
        }
        if (ROWS ? !__syncthreads_or(again) : !again) break;
#pragma unroll
        for (int c = 0; c < CT; ++c) o[c] = zeros();
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = 0.f;
    }

    l += __shfl_xor(l, 32, 64);
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[c][i] = (spoiled[c / 2] >> (c % 2 * 16 + i)) & 1 ? NAN : o[c][i];
    // Sums that are joined with others are brought near 1 first, by a power of two.
    float base = m == -INFINITY ? -INFINITY : ref;
    if (!ROWS || parts > 1) {
        const int e = l > 0.f && l < INFINITY ? __builtin_amdgcn_frexp_expf(l) : 0;
        l = __builtin_amdgcn_ldexpf(l, -e);
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[c][i] = __builtin_amdgcn_ldexpf(o[c][i], -e);
        if (m != -INFINITY) base = ref + (float)e;
    }
    int mine_again = mine ? my : 0;
    asm volatile("" : "+v"(mine_again));
    const int64_t out_row = token_of(mine_again) * a.Hq + head_of(mine_again);
    auto finish = [&](float M, float L, int64_t row) {  // log-sum of a row
        if (a.lse) a.lse[row] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
    };
    if constexpr (ROWS) {
        // A lane's outputs are four channels of its row at a time: stored like that, every request would carry 16 bytes of
        // a row.  They go through LDS (each wave has a quarter of it), where 16 bytes are at piece ^ row of theirs.  (7
        // sequences of 2048 tokens, 40 heads of 128 over 8, window 19: 139 to 149 us, 164 straight from the registers.)
        __syncthreads();  // the tiles have been read
        if (!active) return;
        auto store = [&](auto type, float f, auto row_of) {  // outputs times f, as `type`, row r of the wave to row_of(r)
            using E = decltype(type);
            constexpr int EB = sizeof(E), CC = D * EB * 32 <= S::TILE ? D : S::TILE / (32 * EB), PIECES = CC * EB / 16;
            constexpr int MASK = PIECES < 16 ? PIECES - 1 : 15;
            char* at = s_kv[0] + w * S::TILE;
#pragma unroll
            for (int k = 0; k < D / CC; ++k) {
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int x = 0; x < CC / 8; ++x) {
                    const int c = (k * CC + 8 * x) / 32, e = x % 4, byte = (8 * x + 4 * hl) * EB;
                    char* to = at + lr * CC * EB + (((byte >> 4) ^ (lr & MASK)) << 4) + (byte & 15);
                    const f32x4 y = {o[c][4 * e] * f, o[c][4 * e + 1] * f, o[c][4 * e + 2] * f, o[c][4 * e + 3] * f};
                    if constexpr (EB == 2) *reinterpret_cast<u32x2*>(to) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
                    else *reinterpret_cast<f32x4*>(to) = y;
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int x = 0; x < PIECES / 2; ++x) {
                    const int r = (x * 64 + lane) / PIECES, piece = (x * 64 + lane) % PIECES;
                    E* to = row_of(r);
                    if (r < wave_rows)
                        *reinterpret_cast<u32x4*>(to + k * CC + piece * (16 / EB)) =
                            *reinterpret_cast<const u32x4*>(at + r * CC * EB + ((piece ^ (r & MASK)) << 4));
                }
            }
        };
        if (parts > 1) {
            const int64_t at = (h * places_of(plan.groups) + item.split + item.part) * RT;
            if (mine && hl == 0) ws.ml[at + my] = make_float2(base, l);
            store(0.f, 1.f, [&](int r) { return ws.out + (at + wave_first + r) * D; });
            return;
        }
        if (mine && hl == 0) finish(base, l, out_row);
        store(T(), l == 0.f ? 0.f : 1.f / l, [&](int r) {
            const uint32_t lo = __shfl((uint32_t)out_row, r, 64), hi = __shfl((uint32_t)(out_row >> 32), r, 64);
            return static_cast<T*>(a.o) + (int64_t)((uint64_t)hi << 32 | lo) * D;
        });
    } else {
        // join the waves: their sums go where the tiles were, four channels c of row r at place c / 4 ^ r % 8 of its row
        static_assert(32 * D * 4 <= 2 * S::TILE, "a wave's outputs fit its buffer");
        auto place = [&](int i, int r, int c) { return reinterpret_cast<f32x4*>(s_kv[i]) + r * (D / 4) + (c / 4 ^ (r & 7)); };
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
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *place(w, lr, c * 32 + 8 * e + 4 * hl) =
                    f32x4{o[c][4 * e] * keep, o[c][4 * e + 1] * keep, o[c][4 * e + 2] * keep, o[c][4 * e + 3] * keep};
        }
        __syncthreads();
        for (int x = tid; x < rows * (D / 4); x += S::THREADS) {
            const int r = x / (D / 4), c = x % (D / 4) * 4;
            const float top = joint(r);
            float L = 0.f;
            f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < WAVES; ++i) {
                L += s_l[i][r] * (s_m[i][r] == -INFINITY ? 0.f : exp2_hw(s_m[i][r] - top));  // (NaN without a reference stays)
                y += *place(i, r, c);
            }
            if (parts > 1) {
                const int64_t at = (h * places_of(plan.groups) + item.split + item.part) * RT + r;
                if (c == 0) ws.ml[at] = make_float2(top, L);
                *reinterpret_cast<f32x4*>(ws.out + at * D + c) = y;
                continue;
            }
            const int64_t row = token_of(r) * a.Hq + head_of(r);
            if (c == 0) finish(top, L, row);
            const float f = L == 0.f ? 0.f : 1.f / L;
            T* at = static_cast<T*>(a.o) + row * D + c;
            if constexpr (kBf16)
                *reinterpret_cast<u32x2*>(at) = u32x2{pack_bf16(y[0] * f, y[1] * f), pack_bf16(y[2] * f, y[3] * f)};
            else *reinterpret_cast<f32x4*>(at) = y * f;
        }
    }
}

// Join of the parts of the row tiles that are split: 4 channels of a row for each thread.  A row tile's blocks of rows go
// round its parts and kJoin workgroups of each.
constexpr int kJoin = 4;
template <typename T, int D, bool ROWS>
__global__ __launch_bounds__(256) void prefill_join_kernel(PagedPrefillArgs a, PrefillPlan plan, Partials ws) {
    using S = Shape<T, D, ROWS>;
    constexpr int RT = S::RT, AHEAD = 8, COLS = D / 4, RG = 256 / COLS;  // rows of a block
    __shared__ float2 s_ml[kMaxParts][RG];
    const int tid = threadIdx.x, G = a.Hq / a.Hkv, h = (int)(blockIdx.x % a.Hkv);
    const int b = (int)(blockIdx.x / a.Hkv), place = b / kJoin, r = tid / COLS, c = tid % COLS * 4;
    const int places = (int)places_of(plan.groups);
    if (place >= *ws.count) return;
    const int4 info = ws.part[place];
    const int parts = info.z, first = place - info.w;
    if (parts < 2 || parts > kMaxParts || info.w < 0 || info.w >= parts || first < 0 || first + parts > places) return;
    if (info.x < 0 || info.x >= a.N) return;
    Item item{};
    item.n = info.x;
    item.tile = info.y;
    RowTile tile;
    if (!row_tile_of<RT, S::BN>(a, item, tile)) return;
    for (int r0 = (info.w + b % kJoin * parts) * RG; r0 < tile.rows; r0 += kJoin * parts * RG) {
        const int64_t at = (h * places_of(plan.groups) + first) * RT + r0;
        // (rows behind the tile's last have places too)
        const float* from = ws.out + (at + r) * D + c;
        f32x4 z[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) z[i] = *reinterpret_cast<const f32x4*>(from + (int64_t)(i < parts ? i : 0) * RT * D);
        for (int x = tid; x < parts * RG; x += 256) s_ml[x / RG][x % RG] = ws.ml[at + x / RG * RT + x % RG];
        __syncthreads();
        float M = -INFINITY, L = 0.f;
        for (int i = 0; i < parts; ++i) M = fmaxf(M, s_ml[i][r].x);
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
        for (int i0 = 0; i0 < parts; i0 += AHEAD) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (i0 + i >= parts) break;
                const float2 x = s_ml[i0 + i][r];
                const float f = x.x == -INFINITY ? 0.f : exp2_hw(x.x - M);
                L += x.y * f;
                y += z[i] * f;
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (i0 + AHEAD + i < parts) z[i] = *reinterpret_cast<const f32x4*>(from + (int64_t)(i0 + AHEAD + i) * RT * D);
        }
        __syncthreads();  // the next block's references go there
        if (r0 + r >= tile.rows) continue;
        const float f = L == 0.f ? 0.f : 1.f / L;
        const int64_t row = (tile.cu0 + tile.i0 + (tile.g0 + r0 + r) / G) * a.Hq + h * G + (tile.g0 + r0 + r) % G;
        T* to = static_cast<T*>(a.o) + row * D + c;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<u32x2*>(to) = u32x2{pack_bf16(y[0] * f, y[1] * f), pack_bf16(y[2] * f, y[3] * f)};
        else *reinterpret_cast<f32x4*>(to) = y * f;
        if (c == 0 && a.lse) a.lse[row] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
    }
}

// Few rows for each sequence, on average (the host knows no more): the waves share the rows and split the keys.  A prompt
// next to single tokens makes them many, and the others' row tiles mostly empty: 2048 tokens next to 4 single ones after
// 65536 take 1.07 ms, next to 31 after 10000 240 us, alone 54.
bool many_rows(const PagedPrefillArgs& a) { return a.T * (a.Hq / a.Hkv) > 32 * a.N; }

// A variant's sizes, as in Shape.
struct Sizes {
    int rt, bn, step;
    bool rows;
};
Sizes sizes_of(const PagedPrefillArgs& a) {
    const int row = a.d * (a.bf16 ? 2 : 4);
    if (many_rows(a)) return {128, row <= 256 && a.bf16 ? 64 : 32, 1, true};
    return {32, 32, row <= 256 ? 4 : row == 512 ? 2 : 1, false};
}

// us of a workgroup's step alone on its CU, about.
float step_time(const PagedPrefillArgs& a) {
    return a.bf16 ? (many_rows(a) ? (a.d == 64 ? 0.7f : 1.1f) : a.d == 256 ? 0.9f : 0.4f) : a.d * (1.9f / 64);
}

// What is split.  Few rows: two shortest parts and more, and no more than several rounds of workgroups.  Many rows: where
// the longest row tile takes longer than its share, which runs next to another, and than the parts' results and the join
// (5 us) together.  32 heads of 128 over 8, in bf16, us split and not: 33 tokens after 1000 (16 tiles, 17 steps) 19 and 28;
// 300 after 1500 (80, 29) 32 and 39; 512 after 1500 (136, 32) 39 and 43; 600 after 600 (152, 19) 38 and 32; 900 after 1500
// (232, 38) 56 and 50; 2048 (520, 33) 78 and 55.  fp32 steps take so long that uneven lengths are worth it up to a round of
// workgroups: 40 sequences of 8 to 344 tokens after 1326 to 3978, 4 heads of 128 (284, 136), 316 and 721.
PrefillPlan plan_of(const PagedPrefillArgs& a) {
    PrefillPlan p{};
    const Sizes z = sizes_of(a);
    p.slots = a.T * (a.Hq / a.Hkv) / z.rt + a.N;
    const int64_t steps = steps_to(a, a.max_length, z.rt, z.bn, z.step), tiles = p.slots * a.Hkv;
    const float t = step_time(a), out = 1.6e-6f * z.rt * a.d;  // us of a part's outputs, written and read at 5 TB/s
    p.least = t < 1.5f ? 4 : t < 2.5f ? 2 : 1;
    if (z.rows) {
        const float parts = fminf((float)kGroups, (float)tiles * steps / p.least);
        float saved = tiles <= 256 ? t * steps * (1.f - 0.85f / 256 * tiles) : 0.f;
        if (!a.bf16 && tiles > 256 && tiles <= kGroups) saved = 0.2f * t * steps;
        if (saved < 5.f + parts * out) return p;
    } else if (tiles > 2048 || steps < 2 * p.least) {
        return p;
    }
    p.groups = (int)div_up(z.rows && a.d == 256 ? kGroups / 2 : kGroups, a.Hkv);
    if (a.N > 64) {
        int64_t parts = p.groups / p.slots;
        parts = parts < steps / p.least ? parts : steps / p.least;
        p.parts = (int)(parts < kMaxParts ? parts : kMaxParts);
        if (p.parts < 2) p.parts = p.groups = 0;
        else p.steps = (int)div_up(steps, p.parts);
    }
    return p;
}
int64_t items_of(const PrefillPlan& p) {
    return p.parts ? p.slots * p.parts : p.slots + (p.groups ? places_of(p.groups) : 0);
}
int64_t part_rows(const PagedPrefillArgs& a, const PrefillPlan& p) { return a.Hkv * places_of(p.groups) * sizes_of(a).rt; }
size_t part_bytes(const PrefillPlan& p) { return (size_t)(places_of(p.groups) * 16 + 256); }

template <typename T, int D, bool ROWS>
hipError_t launch_shape(const PagedPrefillArgs& a, const PrefillPlan& p, const Partials& y, hipStream_t s) {
    using S = Shape<T, D, ROWS>;
    const bool timed = timing_on();
    if (timed) timed_begin(kKernelPagedPrefill, s);
    hipLaunchKernelGGL((paged_prefill_kernel<T, D, ROWS>), dim3((unsigned)(items_of(p) * a.Hkv)), dim3(S::THREADS), 0, s, a, p, y);
    hipError_t e = hipGetLastError();
    if (timed) timed_end(s);
    if (e != hipSuccess || !p.groups) return e;
    const unsigned join = (unsigned)(places_of(p.groups) * a.Hkv * kJoin);
    if (timed) timed_begin(kKernelPrefillJoin, s);
    hipLaunchKernelGGL((prefill_join_kernel<T, D, ROWS>), dim3(join), dim3(256), 0, s, a, p, y);
    e = hipGetLastError();
    if (timed) timed_end(s);
    return e;
}
template <typename T, int D>
hipError_t launch_typed(const PagedPrefillArgs& a, const PrefillPlan& p, const Partials& y, hipStream_t s) {
    return many_rows(a) ? launch_shape<T, D, true>(a, p, y, s) : launch_shape<T, D, false>(a, p, y, s);
}
template <typename T>
hipError_t launch_typed(const PagedPrefillArgs& a, const PrefillPlan& p, const Partials& y, hipStream_t s) {
    return a.d == 64 ? launch_typed<T, 64>(a, p, y, s) : a.d == 128 ? launch_typed<T, 128>(a, p, y, s) : launch_typed<T, 256>(a, p, y, s);
}

}  // namespace

int64_t paged_prefill_groups(const PagedPrefillArgs& a, size_t* workspace) {
    *workspace = 0;
    const int64_t slots = a.T * (a.Hq / a.Hkv) / 32 + a.N;  // at most
    if (slots * a.Hkv > max_groups(256)) return slots * a.Hkv;
    const PrefillPlan p = plan_of(a);
    if (p.groups && a.T > 0 && a.N > 0) *workspace = part_bytes(p) + (size_t)(part_rows(a, p) * (8 + (int64_t)a.d * 4));
    return items_of(p) * a.Hkv;
}

hipError_t launch_paged_prefill(const PagedPrefillArgs& a, hipStream_t s) {
    if (a.T == 0 || a.N == 0) return hipSuccess;
    const PrefillPlan p = plan_of(a);
    Partials y{};
    if (p.groups) {
        y.count = static_cast<int*>(a.ws);
        y.part = reinterpret_cast<int4*>(static_cast<char*>(a.ws) + 256);
        y.ml = reinterpret_cast<float2*>(static_cast<char*>(a.ws) + part_bytes(p));
        y.out = reinterpret_cast<float*>(y.ml + part_rows(a, p));
    }
    return a.bf16 ? launch_typed<uint16_t>(a, p, y, s) : launch_typed<float>(a, p, y, s);
}

}  // namespace kda
