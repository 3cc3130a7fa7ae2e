// Pages of a key-value cache: writing new tokens, sharing, reserving, freeing, compacting and
// copying pages (include/kda.h, "Serving next to the recurrence").
//
// The only state besides the tables is one reference count per page.  Free pages are found from
// the counts: a scan turns them into one bit per page with a running count per 64-bit word and per
// block, after which the r-th free page is two binary searches and a select inside one word, and
// the number of used pages before a page one look-up.  Nothing keeps a list whose order could
// depend on the order in which workgroups ran, so the pages handed out are always the lowest free
// ones and every integer result is the same from run to run.  The atomics are integer additions and
// exchanges whose results do not depend on their order.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kBlockPages = 4096;              // pages per block of the scan
constexpr int kBlockWords = kBlockPages / 64;  // 64-bit words per block

// ------------------------------------------------------------------------------------------
// append: keys and values of new tokens into their pages
// ------------------------------------------------------------------------------------------
// Pure traffic: each value is read once and written once.  A workgroup takes `tb` tokens; its first
// threads find the page slot of each (a table look-up, and a binary search over cu_seqlens for
// packed segments), then all of them move 16-byte vectors of keys and values, a token's head at a
// time (128 .. 1024 contiguous bytes of a page).
constexpr int kAppendThreads = 256;
constexpr int kAppendMaxTokens = 16;

constexpr int kAppendUnroll = 4;

template <bool PACKED>
__global__ __launch_bounds__(kAppendThreads) void append_kernel(CacheAppendArgs a, int tb, int vpt, int vph_shift,
                                                                uint32_t vpt_magic) {
    __shared__ int64_t s_k[kAppendMaxTokens], s_v[kAppendMaxTokens];  // slot offsets in bytes, -1: dropped
    const int64_t t0 = (int64_t)blockIdx.x * tb;
    const int nt = (int)(a.T_total - t0 < tb ? a.T_total - t0 : tb);
    const int row_bytes = a.d * a.esz, total = nt * vpt;
    const char* ks = static_cast<const char*>(a.k) + t0 * a.k_stride * a.esz;
    const char* vs = static_cast<const char*>(a.v) + t0 * a.v_stride * a.esz;
    const int64_t kst = a.k_stride * a.esz, vst = a.v_stride * a.esz;
    u32x4 kv[kAppendUnroll], vv[kAppendUnroll];
    int tok[kAppendUnroll];
    auto fetch = [&](int x0) {
#pragma unroll
        for (int i = 0; i < kAppendUnroll; ++i) {
            const int x = x0 + i * kAppendThreads + threadIdx.x;
            tok[i] = (int)__umulhi((uint32_t)x, vpt_magic);  // x / vpt (exact: x * vpt < 2^32)
            if (x < total) {
                const int64_t r = x - tok[i] * vpt;
                kv[i] = *reinterpret_cast<const u32x4*>(ks + tok[i] * kst + r * 16);
                vv[i] = *reinterpret_cast<const u32x4*>(vs + tok[i] * vst + r * 16);
            }
        }
    };
    fetch(0);  // on their way while the slots are looked up
    if ((int)threadIdx.x < nt || (PACKED && a.N <= 64 && threadIdx.x < 64)) {
        const int64_t t = t0 + threadIdx.x;
        int64_t n = t, i = 0;
        bool in = (int)threadIdx.x < nt;
        if (PACKED && a.N <= 64) {
            // the segment ends in the lanes of one wave: the tokens' segments are counts of the ends at or
            // before them, one load instead of a binary search's chain
            const int lane = threadIdx.x;
            const int64_t end = lane < a.N ? a.cu[lane + 1] : INT64_MAX;
            n = 0;
            for (int j = 0; j < nt; ++j) {
                const int c = __popcll(__ballot(end <= t0 + j));
                if (j == lane) n = c;
            }
            if (n >= a.N) n = a.N - 1;
            if (in) {
                i = t - a.cu[n];
                in = i >= 0 && t < a.cu[n + 1];
            }
        } else if (PACKED) {  // the last segment that begins at or before t (empty ones begin where the next does)
            int64_t lo = 0, hi = a.N - 1;
            while (lo < hi) {
                const int64_t mid = (lo + hi + 1) >> 1;
                if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
            }
            n = lo;
            i = t - a.cu[n];
            in = in && i >= 0 && t < a.cu[n + 1];
        }
        int64_t ko = -1, vo = -1;
        if (in) {
            const int64_t pos = (int64_t)a.start[n] + i, col = pos / a.page_size;
            if (pos >= 0 && col < a.pt.width) {
                const int32_t p = a.pt.table[n * a.pt.stride + col];
                if (p >= 0 && p < a.pt.n_pages) {
                    const int64_t slot = (pos - col * a.page_size) * row_bytes;
                    ko = p * a.kp_stride * a.esz + slot;
                    vo = p * a.vp_stride * a.esz + slot;
                }
            }
        }
        if ((int)threadIdx.x < nt) {
            s_k[threadIdx.x] = ko;
            s_v[threadIdx.x] = vo;
        }
    }
    __syncthreads();
    const int64_t head_bytes = (int64_t)a.page_size * row_bytes;
    const int vmask = (1 << vph_shift) - 1;
    for (int x0 = 0; x0 < total; x0 += kAppendUnroll * kAppendThreads) {
        if (x0 > 0) fetch(x0);
#pragma unroll
        for (int i = 0; i < kAppendUnroll; ++i) {
            const int x = x0 + i * kAppendThreads + threadIdx.x;
            if (x >= total) continue;
            const int64_t ko = s_k[tok[i]], vo = s_v[tok[i]];
            if (ko < 0) continue;
            const int r = x - tok[i] * vpt;
            const int64_t at = (int64_t)(r >> vph_shift) * head_bytes + (r & vmask) * 16;
            // stores past the caches: 6% faster for 131072 tokens of 8 heads, now 5.6 TB/s (loads past them
            // gain 3% there and cost 12% for a call that fits the caches)
            __builtin_nontemporal_store(kv[i], reinterpret_cast<u32x4*>(static_cast<char*>(a.kp) + ko + at));
            __builtin_nontemporal_store(vv[i], reinterpret_cast<u32x4*>(static_cast<char*>(a.vp) + vo + at));
        }
    }
}

// ------------------------------------------------------------------------------------------
// fork and free: table rows and counts
// ------------------------------------------------------------------------------------------
constexpr int kTableThreads = 256;

__device__ __forceinline__ bool is_page(int32_t e, int n_pages) { return e >= 0 && e < n_pages; }

// One thread per entry of the wider of the two sets.  An entry that stays what it was touches no
// count; otherwise the new page gains a reference and the old one loses it.
__global__ __launch_bounds__(kTableThreads) void fork_kernel(CacheForkArgs a, uint32_t cols) {
    const int64_t row = blockIdx.x / cols;
    const int j = (blockIdx.x % cols) * kTableThreads + threadIdx.x;
    const bool was = row < a.N, is = row < a.N_out;
    const int32_t parent = is ? a.parents[row] : -1;
    const bool live = parent >= 0 && parent < a.N;
    if (j < a.pt.width) {
        const int32_t old = was ? a.pt.table[row * a.pt.stride + j] : -1;
        const int32_t now = live ? a.pt.table[parent * a.pt.stride + j] : -1;
        if (is) a.table_out[row * a.out_stride + j] = now;
        if (old != now) {
            if (is_page(now, a.pt.n_pages)) atomicAdd(a.refs + now, 1);
            if (is_page(old, a.pt.n_pages)) atomicSub(a.refs + old, 1);
        }
    }
    if (j == 0 && is) a.lengths_out[row] = live ? a.lengths[parent] : 0;
}

// The exchange makes the first of several workgroups that were given the same row the only one that
// sees its pages.
__global__ __launch_bounds__(kTableThreads) void free_kernel(CacheFreeArgs a, uint32_t cols) {
    const int32_t row = a.rows[blockIdx.x / cols];
    if (row < 0 || row >= a.N) return;
    const int j = (blockIdx.x % cols) * kTableThreads + threadIdx.x;
    if (j < a.width) {
        const int32_t old = atomicExch(a.table + row * a.stride + j, -1);
        if (is_page(old, a.n_pages)) atomicSub(a.refs + old, 1);
    }
    if (j == 0) a.lengths[row] = 0;
}

// ------------------------------------------------------------------------------------------
// scan of the counts
// ------------------------------------------------------------------------------------------
// Workspace of reserve and compact.  `bits`: one bit per page (free pages for reserve, used ones
// for compact); `shared`: one bit per page with more than one reference when the call began (reserve);
// `before`: set bits of the word's block before the word; `block`: set bits of the block; `aux`: per
// sequence the number of pages needed (reserve), or the counts of the moved pages (compact); `sums`: the
// pages needed before each group of sequences (reserve, many sequences).
struct CacheWs {
    uint64_t* bits;
    uint64_t* shared;
    uint32_t* before;
    int32_t* block;
    int32_t* aux;
    int32_t* sums;
    int words, blocks;
};

__host__ __device__ inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

__host__ __device__ inline int64_t aux_entries(int64_t N, int64_t n_pages) { return N > n_pages / 2 ? N : n_pages / 2; }

__host__ __device__ inline CacheWs cache_ws(void* ws, int64_t N, int64_t n_pages) {
    CacheWs w;
    const int64_t blocks = up(n_pages, kBlockPages) / kBlockPages, words = blocks * kBlockWords;
    char* p = static_cast<char*>(ws);
    w.bits = reinterpret_cast<uint64_t*>(p);
    w.shared = reinterpret_cast<uint64_t*>(p + words * 8);
    w.before = reinterpret_cast<uint32_t*>(p + words * 16);
    w.block = reinterpret_cast<int32_t*>(p + words * 20);
    // (no rounding up in between: the compiler took it apart into an address that is no multiple of 4 and an
    // offset of 15, whose low bits a scalar load drops, each for itself)
    w.aux = w.block + blocks;
    w.sums = w.aux + aux_entries(N, n_pages);
    w.words = (int)words;
    w.blocks = (int)blocks;
    return w;
}

constexpr int kScanThreads = 256;

// One block of 4096 pages per workgroup: wave w takes words w, w + 4, ...; pages behind the pool
// count as not set.  (For compact the guarded loads wait for one another, 9.0 us for 24 576 pages; for
// reserve they go out together, 3.7.)
template <bool FREE>
__device__ __forceinline__ void scan_block(const int32_t* refs, int n_pages, const CacheWs& w, int b) {
    __shared__ uint32_t s_pop[kBlockWords];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    int32_t r[kBlockWords / 4];
#pragma unroll
    for (int i = 0; i < kBlockWords / 4; ++i) {
        const int p = b * kBlockPages + (i * 4 + wave) * 64 + lane;
        r[i] = p < n_pages ? refs[p] : (FREE ? 1 : 0);
    }
#pragma unroll
    for (int i = 0; i < kBlockWords / 4; ++i) {
        const uint64_t m = __ballot(FREE ? r[i] <= 0 : r[i] > 0), more = FREE ? __ballot(r[i] > 1) : 0;
        if (lane == 0) {
            w.bits[b * kBlockWords + i * 4 + wave] = m;
            if (FREE) w.shared[b * kBlockWords + i * 4 + wave] = more;
            s_pop[i * 4 + wave] = __popcll(m);
        }
    }
    __syncthreads();
    if (threadIdx.x < kBlockWords) {  // one wave: running counts of the block's 64 words
        const uint32_t own = s_pop[lane];
        uint32_t x = own;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t y = __shfl_up(x, off, 64);
            if (lane >= off) x += y;
        }
        w.before[b * kBlockWords + lane] = x - own;
        if (lane == 63) w.block[b] = (int32_t)x;
    }
}

// Exclusive running sums of the blocks' counts into LDS; the total is s_prefix[blocks].
constexpr int kMaxBlocks = (1 << 24) / kBlockPages;

__device__ __forceinline__ void block_prefix(const CacheWs& w, int32_t* s_prefix) {
    // wave 0: 64 blocks at a time
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int32_t carry = 0;
        for (int b0 = 0; b0 < w.blocks; b0 += 64) {
            const int32_t own = b0 + lane < w.blocks ? w.block[b0 + lane] : 0;
            int32_t x = own;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int32_t y = __shfl_up(x, off, 64);
                if (lane >= off) x += y;
            }
            if (b0 + lane < w.blocks) s_prefix[b0 + lane] = carry + x - own;
            carry += __shfl(x, 63, 64);
        }
        if (lane == 0) s_prefix[w.blocks] = carry;
    }
    __syncthreads();
}

// the page of the r-th set bit, 0 <= r < total
__device__ __forceinline__ int32_t select_page(const CacheWs& w, const int32_t* s_prefix, int32_t r) {
    int lo = 0, hi = w.blocks - 1;
    while (lo < hi) {  // the last block that begins at or before rank r
        const int mid = (lo + hi + 1) >> 1;
        if (s_prefix[mid] <= r) lo = mid; else hi = mid - 1;
    }
    const int b = lo;
    uint32_t k = (uint32_t)(r - s_prefix[b]);
    lo = 0;
    hi = kBlockWords - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (w.before[b * kBlockWords + mid] <= k) lo = mid; else hi = mid - 1;
    }
    const uint64_t m = w.bits[b * kBlockWords + lo];
    k -= w.before[b * kBlockWords + lo];
    int at = 0;
#pragma unroll
    for (int half = 32; half > 0; half >>= 1) {
        const uint32_t c = __popcll((m >> at) & ((1ull << half) - 1));
        if (k >= c) {
            k -= c;
            at += half;
        }
    }
    return b * kBlockPages + lo * 64 + at;
}

// set bits before page p, 0 <= p <= n_pages rounded up to a block
__device__ __forceinline__ int32_t bits_before(const CacheWs& w, const int32_t* s_prefix, int32_t p) {
    const int b = p / kBlockPages;
    if (b >= w.blocks) return s_prefix[w.blocks];
    const int word = p >> 6;
    return s_prefix[b] + (int32_t)w.before[word] + __popcll(w.bits[word] & ((1ull << (p & 63)) - 1));
}

__device__ __forceinline__ bool bit_of(const uint64_t* bits, int32_t p) { return (bits[p >> 6] >> (p & 63)) & 1; }

// The scan of a small pool by one workgroup, in LDS.
constexpr int kSmallThreads = 1024;
constexpr int kSmallBlocks = 2, kSmallPages = kSmallBlocks * kBlockPages;
constexpr int kSmallRows = 32;        // sequences of a small reserve: two per wave
constexpr int kSmallEntries = 16384;  // table entries of a small compaction: sixteen per thread
struct SmallScan {
    uint64_t bits[kSmallBlocks * kBlockWords];
    uint64_t shared[kSmallBlocks * kBlockWords];
    uint32_t before[kSmallBlocks * kBlockWords];
    int32_t block[kSmallBlocks];
    int32_t prefix[kSmallBlocks + 1];
    int32_t aux[kSmallPages / 2];
};

// Every thread of the workgroup; a barrier has to follow before anything but `bits` of its own wave is
// read.
template <bool FREE>
__device__ __forceinline__ CacheWs small_scan(const int32_t* refs, int n_pages, SmallScan& s) {
    constexpr int kWords = kSmallBlocks * kBlockWords, kPer = kWords / (kSmallThreads / 64);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    CacheWs w{s.bits, s.shared, s.before, s.block, s.aux, nullptr, kWords, kSmallBlocks};
    int32_t r[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int p = (i * (kSmallThreads / 64) + wave) * 64 + lane;
        r[i] = p < n_pages ? refs[p] : (FREE ? 1 : 0);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint64_t m = __ballot(FREE ? r[i] <= 0 : r[i] > 0), more = FREE ? __ballot(r[i] > 1) : 0;
        if (lane == 0) {
            s.bits[i * (kSmallThreads / 64) + wave] = m;
            if (FREE) s.shared[i * (kSmallThreads / 64) + wave] = more;
        }
    }
    __syncthreads();
    if (wave == 0) {
        int32_t carry = 0;
        for (int b = 0; b < kSmallBlocks; ++b) {
            const uint32_t own = __popcll(s.bits[b * kBlockWords + lane]);
            uint32_t x = own;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const uint32_t y = __shfl_up(x, off, 64);
                if (lane >= off) x += y;
            }
            s.before[b * kBlockWords + lane] = x - own;
            const int32_t total = __shfl((int32_t)x, 63, 64);
            if (lane == 0) {
                s.block[b] = total;
                s.prefix[b] = carry;
                s.prefix[b + 1] = carry + total;
            }
            carry += total;
        }
    }
    return w;
}

// ------------------------------------------------------------------------------------------
// reserve
// ------------------------------------------------------------------------------------------
// First launch: the blocks' scans, and one wave per sequence that counts the pages it needs.  The scan
// also keeps a bit for every shared page, which carries the verdict on the counts as they were when
// the call began over to the last launch, which changes them.  Nothing of a table is written before it
// is known whether its sequence is served, so one that is not keeps every entry, whatever it holds.
constexpr int kRowsPerGroup = kScanThreads / 64;
// Sequences up to which every group of the second launch adds up the needs before it, which grows with
// their square; for more a launch between the two does it once (reserve_sums_kernel).  Kernel time of the
// call without and with that launch: 21.6 and 24.0 us for 8192 sequences, 29.1 and 29.4 for 12 288, 36.2 and 34.0
// for 16 384, 2.07 and 0.35 ms for 262 144.
constexpr int64_t kDirectRows = 12288;

// columns that hold the new tokens' positions; none where nothing is to be reserved, bad where the
// row is too narrow
struct Span64 {
    int64_t first, last;
    bool none, bad;
};
__device__ __forceinline__ Span64 new_columns(int32_t len, int32_t add, int page_size, int width) {
    Span64 s{0, -1, true, false};
    if (add <= 0) return s;
    if (len < 0) {
        s.bad = true;
        return s;
    }
    s.first = len / page_size;
    s.last = ((int64_t)len + add - 1) / page_size;
    s.bad = s.last >= width || (int64_t)len + add > INT32_MAX;
    s.none = s.bad;
    return s;
}

// pages that sequence n needs from column first + skip on, by the counts before any has changed (one wave)
__device__ __forceinline__ int32_t count_need(const CacheReserveArgs& a, int64_t n, const Span64& s, int skip) {
    const int lane = threadIdx.x & 63;
    int32_t need = 0;
    for (int64_t j0 = s.first + skip; j0 <= s.last; j0 += 64) {
        const int64_t j = j0 + lane;
        bool want = false;
        if (j <= s.last) {
            const int32_t p = a.table[n * a.stride + j];
            want = !is_page(p, a.n_pages) || a.refs[p] > 1;
        }
        need += __popcll(__ballot(want));
    }
    return need;
}

// hands out the pages to the columns from first + skip on that need one; the first has rank `base` among the
// free pages (one wave).  Returns the pair of the first column in lane 0: the page it had and the one it
// has got, or -1.
__device__ __forceinline__ int2 take_pages(const CacheReserveArgs& a, const CacheWs& w, const int32_t* s_prefix,
                                           int64_t n, const Span64& s, int skip, int64_t base) {
    const int lane = threadIdx.x & 63;
    int2 pair = make_int2(-1, -1);
    for (int64_t j0 = s.first + skip; j0 <= s.last; j0 += 64) {
        const int64_t j = j0 + lane;
        int32_t* e = a.table + n * a.stride + j;
        const int32_t old = j <= s.last ? *e : -1;
        const bool page = is_page(old, a.n_pages), want = j <= s.last && (!page || bit_of(w.shared, old));
        const uint64_t m = __ballot(want);
        if (want) {
            const int32_t p = select_page(w, s_prefix, (int32_t)(base + __popcll(m & ((1ull << lane) - 1))));
            *e = p;
            a.refs[p] = 1;
            if (page) {
                atomicSub(a.refs + old, 1);
                if (j == s.first) pair = make_int2(old, p);
            }
        }
        base += __popcll(m);
    }
    return pair;
}

__global__ __launch_bounds__(kScanThreads) void reserve_scan_kernel(CacheReserveArgs a) {
    const CacheWs w = cache_ws(a.ws, a.N, a.n_pages);
    if ((int)blockIdx.x < w.blocks) {
        scan_block<true>(a.refs, a.n_pages, w, blockIdx.x);
        return;
    }
    const int64_t n = (int64_t)(blockIdx.x - w.blocks) * kRowsPerGroup + (threadIdx.x >> 6);
    if (n >= a.N) return;
    const Span64 s = new_columns(a.lengths[n], a.new_tokens[n], a.page_size, a.width);
    const int32_t need = s.none ? 0 : count_need(a, n, s, 0);
    if ((threadIdx.x & 63) == 0) w.aux[n] = s.bad ? -1 : need;
}

// Pages needed before each group of sequences, by one workgroup that keeps the running sum.  A sum stops at
// kNoPages, more than a pool has, so that it fits 32 bits however much is asked for.
constexpr int kSumThreads = 1024;
constexpr int32_t kNoPages = 1 << 30;

__global__ __launch_bounds__(kSumThreads) void reserve_sums_kernel(CacheReserveArgs a) {
    __shared__ int64_t s_wave[2][kSumThreads / 64];
    const CacheWs w = cache_ws(a.ws, a.N, a.n_pages);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t groups = (a.N + kRowsPerGroup - 1) / kRowsPerGroup;
    int64_t carry = 0;
    for (int64_t g0 = 0, turn = 0; g0 < groups; g0 += kSumThreads, turn ^= 1) {
        const int64_t g = g0 + threadIdx.x;
        int64_t own = 0;
#pragma unroll
        for (int i = 0; i < kRowsPerGroup; ++i) {
            const int64_t n = g * kRowsPerGroup + i;
            const int32_t need = w.aux[n < a.N ? n : a.N - 1];
            own += n < a.N && need > 0 ? need : 0;
        }
        int64_t x = own;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int64_t y = __shfl_up(x, off, 64);
            if (lane >= off) x += y;
        }
        if (lane == 63) s_wave[turn][wave] = x;
        __syncthreads();  // (the other half of s_wave is written next, so one barrier a turn is enough)
        int64_t before = carry, all = carry;
        for (int i = 0; i < kSumThreads / 64; ++i) {
            before += i < wave ? s_wave[turn][i] : 0;
            all += s_wave[turn][i];
        }
        before += x - own;
        if (g < groups) w.sums[g] = before < kNoPages ? (int32_t)before : kNoPages;
        carry = all < kNoPages ? all : kNoPages;
    }
}

// Second launch: one wave per sequence.  Its first page is the free one whose rank is the sum of the
// needs before it.
__global__ __launch_bounds__(kScanThreads) void reserve_kernel(CacheReserveArgs a) {
    __shared__ int32_t s_prefix[kMaxBlocks + 1];
    __shared__ int64_t s_sum[kRowsPerGroup];
    const CacheWs w = cache_ws(a.ws, a.N, a.n_pages);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n0 = (int64_t)blockIdx.x * kRowsPerGroup, n = n0 + wave;
    // pages needed by the sequences before this group
    int64_t sum = 0;
    if (a.N <= kDirectRows) {
        for (int64_t i = threadIdx.x; i < n0; i += kScanThreads) sum += w.aux[i] > 0 ? w.aux[i] : 0;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    } else if (wave == 0) {
        sum = w.sums[blockIdx.x];
    }
    if (lane == 0) s_sum[wave] = sum;
    block_prefix(w, s_prefix);  // ends with a barrier
    if (n >= a.N) return;
    int64_t base = 0;
    for (int i = 0; i < kRowsPerGroup; ++i) base += s_sum[i];
    for (int i = 0; i < wave; ++i) base += w.aux[n0 + i] > 0 ? w.aux[n0 + i] : 0;
    const int32_t len = a.lengths[n], add = a.new_tokens[n], need = w.aux[n];
    const Span64 s = new_columns(len, add, a.page_size, a.width);
    const bool served = add > 0 && need >= 0 && base + need <= s_prefix[w.blocks];
    int2 pair = make_int2(-1, -1);
    if (served) pair = take_pages(a, w, s_prefix, n, s, 0, base);
    if (lane == 0) {  // the first column's page is the only one that can be partly filled
        const bool part = pair.x >= 0 && len % a.page_size;
        a.copies[2 * n] = part ? pair.x : -1;
        a.copies[2 * n + 1] = part ? pair.y : -1;
        a.granted[n] = served ? add : 0;
        if (served) a.lengths[n] = len + add;
    }
}

// Small pools and few sequences: both steps in one workgroup, with the scan in LDS and the first 64
// columns of each sequence in registers in between (further ones are read again).  The second launch
// costs the caller 2.5 us, which is what bounds a small call.
__global__ __launch_bounds__(kSmallThreads) void reserve_small_kernel(CacheReserveArgs a) {
    constexpr int R = kSmallRows / (kSmallThreads / 64);
    __shared__ SmallScan s;
    __shared__ int32_t s_need[kSmallRows];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    int32_t len[R], add[R], e[R], need[R];
    Span64 span[R];
    bool want[R];
    // The scan's loads go out together, but behind the chain of the sequences' own (length, entry, count), of
    // which each waits for the one before.
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int n = wave + i * (kSmallThreads / 64);
        len[i] = n < a.N ? a.lengths[n] : 0;
        add[i] = n < a.N ? a.new_tokens[n] : 0;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int n = wave + i * (kSmallThreads / 64);
        span[i] = new_columns(len[i], add[i], a.page_size, a.width);
        e[i] = -1;
        want[i] = !span[i].none && span[i].first + lane <= span[i].last;
        if (want[i]) e[i] = a.table[n * a.stride + span[i].first + lane];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (!is_page(e[i], a.n_pages)) e[i] = -1;
        if (e[i] >= 0 && a.refs[e[i]] <= 1) want[i] = false;
    }
    const CacheWs w = small_scan<true>(a.refs, a.n_pages, s);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int n = wave + i * (kSmallThreads / 64);
        need[i] = __popcll(__ballot(want[i]));
        if (!span[i].none && span[i].last >= span[i].first + 64) need[i] += count_need(a, n, span[i], 64);
        if (lane == 0 && n < a.N) s_need[n] = span[i].bad ? -1 : need[i];
    }
    __syncthreads();  // the scan too, and every look at a count before the first change
    // running sums of the needs, in the lanes of every wave
    int64_t before = lane < a.N && s_need[lane < kSmallRows ? lane : 0] > 0 ? s_need[lane] : 0;
    const int64_t own = before;
#pragma unroll
    for (int off = 1; off < kSmallRows; off <<= 1) {
        const int64_t y = __shfl_up(before, off, 64);
        if (lane >= off) before += y;
    }
    before -= own;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int n = wave + i * (kSmallThreads / 64);
        if (n >= a.N) continue;
        const int64_t base = __shfl(before, n, 64);
        const bool served = add[i] > 0 && !span[i].bad && base + need[i] <= s.prefix[w.blocks];
        const uint64_t m = __ballot(want[i]);
        int32_t p = -1;
        if (served && want[i]) {
            p = select_page(w, s.prefix, (int32_t)(base + __popcll(m & ((1ull << lane) - 1))));
            a.table[n * a.stride + span[i].first + lane] = p;
            a.refs[p] = 1;
            if (e[i] >= 0) atomicSub(a.refs + e[i], 1);
        }
        if (served && span[i].last >= span[i].first + 64)
            take_pages(a, w, s.prefix, n, span[i], 64, base + __popcll(m));
        if (lane == 0) {  // the first column's page is the only one that can be partly filled
            const bool part = p >= 0 && e[i] >= 0 && len[i] % a.page_size;
            a.copies[2 * n] = part ? e[i] : -1;
            a.copies[2 * n + 1] = part ? p : -1;
            a.granted[n] = served ? add[i] : 0;
            if (served) a.lengths[n] = len[i] + add[i];
        }
    }
}

// ------------------------------------------------------------------------------------------
// compact
// ------------------------------------------------------------------------------------------
// With L used pages, the holes are the free pages before L and the movers the used ones at or
// behind it; there are as many of one as of the other, and sources and targets are disjoint, so the
// copies can run in any order.
__global__ __launch_bounds__(kScanThreads) void compact_scan_kernel(CacheCompactArgs a) {
    scan_block<false>(a.refs, a.pt.n_pages, cache_ws(a.ws, a.N, a.pt.n_pages), blockIdx.x);
}

// page p's part in the moves (pages before p, and before the number L of used pages: `front`)
__device__ __forceinline__ void plan_page(const CacheCompactArgs& a, const CacheWs& w, const int32_t* s_prefix, int p,
                                          int32_t L, int32_t front) {
    const bool used = bit_of(w.bits, p);
    if (used != (p < L)) {
        const int32_t before = bits_before(w, s_prefix, p);
        if (!used) {
            a.moves[2 * (int64_t)(p - before) + 1] = p;
        } else {
            a.moves[2 * (int64_t)(before - front)] = p;
            w.aux[before - front] = a.refs[p];
        }
    }
    if (p < a.pt.n_pages / 2 && p >= L - front) {
        a.moves[2 * (int64_t)p] = -1;
        a.moves[2 * (int64_t)p + 1] = -1;
    }
}

__device__ __forceinline__ void remap_count(const CacheCompactArgs& a, const CacheWs& w, const int32_t* s_prefix, int p,
                                            int32_t L) {
    int32_t r = 0;
    if (p < L) r = bit_of(w.bits, p) ? a.refs[p] : w.aux[p - bits_before(w, s_prefix, p)];
    a.refs_out[p] = r;
}

__device__ __forceinline__ void remap_entry(const CacheCompactArgs& a, const CacheWs& w, const int32_t* s_prefix,
                                            int64_t row, int j, int32_t L, int32_t front) {
    int32_t e = a.pt.table[row * a.pt.stride + j];
    if (e >= L && e < a.pt.n_pages && bit_of(w.bits, e))
        e = a.moves[2 * (int64_t)(bits_before(w, s_prefix, e) - front) + 1];
    a.table_out[row * a.out_stride + j] = e;
}

__global__ __launch_bounds__(kScanThreads) void compact_plan_kernel(CacheCompactArgs a) {
    __shared__ int32_t s_prefix[kMaxBlocks + 1];
    const CacheWs w = cache_ws(a.ws, a.N, a.pt.n_pages);
    block_prefix(w, s_prefix);
    const int32_t L = s_prefix[w.blocks], front = bits_before(w, s_prefix, L);
    const int p = blockIdx.x * kScanThreads + threadIdx.x;
    if (p < a.pt.n_pages) plan_page(a, w, s_prefix, p, L, front);
}

__global__ __launch_bounds__(kScanThreads) void compact_remap_kernel(CacheCompactArgs a, int count_groups,
                                                                     int col_groups) {
    __shared__ int32_t s_prefix[kMaxBlocks + 1];
    const CacheWs w = cache_ws(a.ws, a.N, a.pt.n_pages);
    block_prefix(w, s_prefix);
    const int32_t L = s_prefix[w.blocks];
    if ((int)blockIdx.x < count_groups) {
        const int p = blockIdx.x * kScanThreads + threadIdx.x;
        if (p < a.pt.n_pages) remap_count(a, w, s_prefix, p, L);
        return;
    }
    const int g = blockIdx.x - count_groups;
    const int j = (g % col_groups) * kScanThreads + threadIdx.x;
    if (j < a.pt.width) remap_entry(a, w, s_prefix, g / col_groups, j, L, bits_before(w, s_prefix, L));
}

// Small pools and tables: the three steps in one workgroup, with the scan in LDS.
__global__ __launch_bounds__(kSmallThreads) void compact_small_kernel(CacheCompactArgs a) {
    __shared__ SmallScan s;
    const CacheWs w = small_scan<false>(a.refs, a.pt.n_pages, s);
    __syncthreads();
    const int32_t L = s.prefix[w.blocks], front = bits_before(w, s.prefix, L);
    for (int p = threadIdx.x; p < a.pt.n_pages; p += kSmallThreads) plan_page(a, w, s.prefix, p, L, front);
    __syncthreads();  // `aux`, and the moves, which no thread has read before
    for (int p = threadIdx.x; p < a.pt.n_pages; p += kSmallThreads) remap_count(a, w, s.prefix, p, L);
    const int entries = (int)a.N * a.pt.width;
    for (int i = threadIdx.x; i < entries; i += kSmallThreads)
        remap_entry(a, w, s.prefix, i / a.pt.width, i % a.pt.width, L, front);
}

// ------------------------------------------------------------------------------------------
// copies of pages
// ------------------------------------------------------------------------------------------
// Traffic only.  A workgroup of one wave copies 4 KiB and is done: workgroups start in order, so that
// the chip works through the pages as one stream.  Larger pieces and loops over them spread it over more
// of the memory and are slower (a plain copy of 2 GiB: 6.3 to 6.7 TB/s with 1 to 4 KiB a workgroup, 5.8
// to 6.0 with 16, 5.2 to 5.8 with 32, 4.5 to 5.8 in loops of 512 to 16384 workgroups).  The guards of a
// page's last piece make the compiler wait for each of a thread's four loads before the next: it is the
// other workgroups that keep the memory busy.
//
// A long list may be mostly empty (a compaction's has room for every second page).  There a workgroup
// takes one piece of kFar pairs, which stand a kFar-th of the list apart, so that an empty
// stretch costs few workgroups of its own.  10 300 of 24 576 pages of 128 KiB moved: 447 us against 534 with
// looping workgroups (441 with four pairs); 730 moved, in the same list: 53 against 34 us (68 with four).
constexpr int kCopyThreads = 64, kCopyUnroll = 4;
constexpr int kCopyPiece = kCopyThreads * kCopyUnroll * 16;
constexpr int kFar = 8;
constexpr int64_t kManyPieces = 1 << 13;

template <int K>
__global__ __launch_bounds__(kCopyThreads) void pages_copy_kernel(PoolList pl, int n_pages, const int32_t* pairs,
                                                                  int64_t n_pairs, int64_t apart, uint32_t pieces) {
    const uint32_t per_pair = pl.count * pieces;
    const int64_t first = blockIdx.x / per_pair;
    const uint32_t rest = blockIdx.x % per_pair;
    const int pool = rest / pieces;
    const int64_t off = (int64_t)(rest % pieces) * kCopyPiece + threadIdx.x * 16;
    char* base = pl.base[pool] + off;
    const int64_t stride = pl.stride[pool];
    const int64_t left = (pl.bytes[pool] - off) >> 4;  // vectors from this thread's on
    int32_t src[K], dst[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int64_t p = first + i * apart;
        src[i] = dst[i] = -1;
        if (p < n_pairs) {
            src[i] = pairs[2 * p];
            dst[i] = pairs[2 * p + 1];
        }
    }
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (is_page(src[i], n_pages) && is_page(dst[i], n_pages) && src[i] != dst[i]) {
            const u32x4* from = reinterpret_cast<const u32x4*>(base + src[i] * stride);
            u32x4* to = reinterpret_cast<u32x4*>(base + dst[i] * stride);
            u32x4 x[kCopyUnroll];
#pragma unroll
            for (int u = 0; u < kCopyUnroll; ++u)
                if (u * kCopyThreads < left) x[u] = from[u * kCopyThreads];
#pragma unroll
            for (int u = 0; u < kCopyUnroll; ++u)
                if (u * kCopyThreads < left) __builtin_nontemporal_store(x[u], to + u * kCopyThreads);
        }
}

template <typename F>
hipError_t timed_launch(int id, hipStream_t s, F launch) {
    const bool timed = timing_on();
    if (timed) timed_begin(id, s);
    launch();
    const hipError_t e = hipGetLastError();
    if (timed) timed_end(s);
    return e;
}

int64_t div_up(int64_t x, int64_t m) { return (x + m - 1) / m; }

}  // namespace

static int append_tokens(int64_t T_total, int vpt) {
    int tb = (4 * kAppendThreads) / vpt;  // about four vectors of keys per thread
    if (tb > T_total / 512) tb = (int)(T_total / 512);  // few tokens: spread over the chip
    return tb < 1 ? 1 : tb > kAppendMaxTokens ? kAppendMaxTokens : tb;
}

int64_t cache_append_groups(int64_t T_total, int H, int d, int esz) {
    return div_up(T_total, append_tokens(T_total, H * (d * esz / 16)));
}

hipError_t launch_cache_append(const CacheAppendArgs& a, hipStream_t s) {
    if (a.T_total == 0) return hipSuccess;
    const int vph = a.d * a.esz / 16, vpt = a.H * vph, tb = append_tokens(a.T_total, vpt);
    const uint32_t magic = (uint32_t)(((1ull << 32) + vpt - 1) / vpt);
    const unsigned grid = (unsigned)div_up(a.T_total, tb);
    return timed_launch(kKernelCacheAppend, s, [&] {
        if (a.cu)
            hipLaunchKernelGGL(append_kernel<true>, dim3(grid), dim3(kAppendThreads), 0, s, a, tb, vpt,
                               __builtin_ctz(vph), magic);
        else
            hipLaunchKernelGGL(append_kernel<false>, dim3(grid), dim3(kAppendThreads), 0, s, a, tb, vpt,
                               __builtin_ctz(vph), magic);
    });
}

int64_t cache_rows_groups(int64_t rows, int width) { return rows * (width ? div_up(width, kTableThreads) : 1); }

int64_t cache_reserve_groups(int64_t N, int64_t n_pages) {
    return div_up(n_pages, kBlockPages) + div_up(N, kRowsPerGroup);
}

int64_t cache_compact_groups(int64_t N, int width, int64_t n_pages) {
    return div_up(n_pages, kScanThreads) + N * div_up(width, kScanThreads);
}

hipError_t launch_cache_fork(const CacheForkArgs& a, hipStream_t s) {
    const int64_t rows = a.N > a.N_out ? a.N : a.N_out;
    if (rows == 0) return hipSuccess;
    const int64_t cols = cache_rows_groups(1, a.pt.width);
    return timed_launch(kKernelCacheFork, s, [&] {
        hipLaunchKernelGGL(fork_kernel, dim3((unsigned)(cols * rows)), dim3(kTableThreads), 0, s, a,
                           (uint32_t)cols);
    });
}

hipError_t launch_cache_free(const CacheFreeArgs& a, hipStream_t s) {
    if (a.n_rows == 0) return hipSuccess;
    const int64_t cols = cache_rows_groups(1, a.width);
    return timed_launch(kKernelCacheFree, s, [&] {
        hipLaunchKernelGGL(free_kernel, dim3((unsigned)(cols * a.n_rows)), dim3(kTableThreads), 0, s, a,
                           (uint32_t)cols);
    });
}

size_t cache_workspace(int64_t N, int64_t n_pages) {
    const int64_t blocks = div_up(n_pages, kBlockPages), sums = div_up(N, kRowsPerGroup);
    return (size_t)up(blocks * kBlockWords * 20 + (blocks + aux_entries(N, n_pages) + sums) * 4, 256);
}

hipError_t launch_cache_reserve(const CacheReserveArgs& a, hipStream_t s) {
    if (a.N == 0) return hipSuccess;
    if (a.n_pages <= kSmallPages && a.N <= kSmallRows)
        return timed_launch(kKernelCacheReserve, s, [&] {
            hipLaunchKernelGGL(reserve_small_kernel, dim3(1), dim3(kSmallThreads), 0, s, a);
        });
    const int64_t blocks = div_up(a.n_pages, kBlockPages), groups = div_up(a.N, kRowsPerGroup);
    hipError_t e = timed_launch(kKernelCacheScan, s, [&] {
        hipLaunchKernelGGL(reserve_scan_kernel, dim3((unsigned)(blocks + groups)), dim3(kScanThreads), 0, s, a);
    });
    if (e == hipSuccess && a.N > kDirectRows)
        e = timed_launch(kKernelCacheScan, s, [&] {
            hipLaunchKernelGGL(reserve_sums_kernel, dim3(1), dim3(kSumThreads), 0, s, a);
        });
    if (e != hipSuccess) return e;
    return timed_launch(kKernelCacheReserve, s, [&] {
        hipLaunchKernelGGL(reserve_kernel, dim3((unsigned)groups), dim3(kScanThreads), 0, s, a);
    });
}

hipError_t launch_cache_compact(const CacheCompactArgs& a, hipStream_t s) {
    const int64_t blocks = div_up(a.pt.n_pages, kBlockPages), groups = div_up(a.pt.n_pages, kScanThreads);
    const int64_t cols = div_up(a.pt.width, kScanThreads);
    if (a.pt.n_pages <= kSmallPages && a.N * a.pt.width <= kSmallEntries)
        return timed_launch(kKernelCachePlan, s, [&] {
            hipLaunchKernelGGL(compact_small_kernel, dim3(1), dim3(kSmallThreads), 0, s, a);
        });
    hipError_t e = timed_launch(kKernelCacheScan, s, [&] {
        hipLaunchKernelGGL(compact_scan_kernel, dim3((unsigned)blocks), dim3(kScanThreads), 0, s, a);
    });
    if (e == hipSuccess)
        e = timed_launch(kKernelCachePlan, s, [&] {
            hipLaunchKernelGGL(compact_plan_kernel, dim3((unsigned)groups), dim3(kScanThreads), 0, s, a);
        });
    if (e != hipSuccess) return e;
    return timed_launch(kKernelCacheRemap, s, [&] {
        hipLaunchKernelGGL(compact_remap_kernel, dim3((unsigned)(groups + a.N * cols)), dim3(kScanThreads), 0, s, a,
                           (int)groups, cols ? (int)cols : 1);
    });
}

hipError_t launch_pages_copy(const PoolList& p, int n_pages, const int32_t* pairs, int64_t n_pairs, hipStream_t s) {
    int64_t most = 0;
    for (int i = 0; i < p.count; ++i) most = p.bytes[i] > most ? p.bytes[i] : most;
    if (n_pairs == 0 || most == 0) return hipSuccess;
    const int64_t pieces = div_up(most, kCopyPiece), per_pair = pieces * p.count;
    const bool many = n_pairs * per_pair > kManyPieces && n_pairs >= 4 * kFar;
    const int64_t apart = many ? div_up(n_pairs, kFar) : n_pairs;
    // in slices of the list where a grid does not hold it
    const int64_t most_pairs = max_groups(kCopyThreads) / per_pair;
    hipError_t e = hipSuccess;
    for (int64_t p0 = 0; p0 < apart && e == hipSuccess; p0 += most_pairs) {
        const int64_t groups = apart - p0 < most_pairs ? apart - p0 : most_pairs;
        e = timed_launch(kKernelPagesCopy, s, [&] {
            const dim3 grid((unsigned)(groups * per_pair)), block(kCopyThreads);
            const int32_t* at = pairs + 2 * p0;
            if (many)
                hipLaunchKernelGGL(pages_copy_kernel<kFar>, grid, block, 0, s, p, n_pages, at, n_pairs - p0, apart,
                                   (uint32_t)pieces);
            else
                hipLaunchKernelGGL(pages_copy_kernel<1>, grid, block, 0, s, p, n_pages, at, n_pairs - p0, apart,
                                   (uint32_t)pieces);
        });
    }
    return e;
}

}  // namespace kda
