// Internal interface between the C-ABI layer (kda_api.cpp) and the kernel
// translation units.  Not installed; not part of the ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// Per-kernel event timing (diagnostics).  When timing is on for the calling
// thread, launchers bracket each kernel with timed_begin/timed_end.
enum KernelId {
    kKernelPrep = 1,
    kKernelState = 2,
    kKernelChunkF32 = 3,
    kKernelDecode = 4,
    kKernelBwdFactors = 5,
    kKernelBwdFwdChain = 6,
    kKernelBwdRevChain = 7,
    kKernelBwdGradState = 8,
    kKernelBwdGradChunk = 9,
    kKernelCacheAppend = 10,
    kKernelPagedDecode = 11,
    kKernelPagedJoin = 12,
    kKernelCacheFork = 13,
    kKernelCacheFree = 14,
    kKernelCacheScan = 15,
    kKernelCacheReserve = 16,
    kKernelCachePlan = 17,
    kKernelCacheRemap = 18,
    kKernelPagesCopy = 19,
    kKernelBeamScan = 20,
    kKernelBeamJoin = 21,
    kKernelBeamReorder = 22
};
bool timing_on();
void timed_begin(int kernel_id, hipStream_t s);
void timed_end(hipStream_t s);

// Sequences of a prefill/append call.  Either `cu` (device int32 [N+1]) is set,
// or every sequence has `T_fixed` tokens and sequence n starts at n * T_fixed.
struct PrefillArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const void* beta;
    const float* s0;  // [N, H, dk, dv] or nullptr
    float* o;         // [T_total, H, dv]
    float* sT;        // [N, H, dk, dv] or nullptr
    const int32_t* cu;
    int64_t N;
    int64_t T_fixed;
    int64_t T_total;
    int H, dk, dv, chunk;
    int bf16;  // storage type of q, k, v, beta
    void* ws;
    size_t ws_bytes;
    int gate_head;          // g is [T_total, H] (one decay per token and head) instead of [T_total, H, dk]
    float* snap;            // state snapshots, or nullptr
    int snap_every;         // chunks between snapshots
    const int32_t* snap_cu; // varlen: first snapshot row of each sequence (device)
    int64_t snap_per_seq;   // fixed length: snapshots per sequence
    int prologue;           // raw inputs: normalise q, k; beta = sigmoid(beta); g = -gate_scale * softplus(g)
    float gate_scale;
};

struct DecodeArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const void* beta;
    const float* s_in;
    float* s_out;
    float* o;
    int64_t N;
    int H, dk, dv;
    int bf16;
    int gate_head;  // g is [N, H] (one decay per sequence and head) instead of [N, H, dk]
    int prologue;   // raw inputs, as in PrefillArgs
    float gate_scale;
};

// Chunked backward.  Sequences are packed (device cu_seqlens [N+1]); outputs are fp32.
struct BwdArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const void* beta;
    const int32_t* cu;
    int64_t N;
    int64_t T_total;
    int H, dk, dv, chunk;
    int bf16;       // storage type of q, k, v, beta
    int gate_head;  // g is [T_total, H]; gg is then [T_total, H] too
    const float* s0;   // [N, H, dk, dv] or nullptr
    const float* dO;   // [T_total, H, dv]
    const float* dsT;  // [N, H, dk, dv] or nullptr
    float* gq;         // [T_total, H, dk]
    float* gk;         // [T_total, H, dk]
    float* gv;         // [T_total, H, dv]
    float* gg;         // [T_total, H, dk] or [T_total, H]
    float* gbeta;      // [T_total, H]
    float* gs0;        // [N, H, dk, dv] or nullptr
    float* ws;
    float* s_fin;      // windowed passes: the forward chain's state after the window [N, H, dk, dv], or nullptr
};

bool chunk_bwd_supported(int dk, int dv, int chunk);
size_t chunk_bwd_workspace(int64_t N, int64_t T_total, int H, int dk, int dv, int chunk);
hipError_t launch_chunk_bwd(const BwdArgs& a, hipStream_t s);

// generic fp32-arithmetic chunked kernel (any supported shape, either storage type)
bool chunk_f32_supported(int dk, int dv, int chunk);
hipError_t launch_chunk_f32(const PrefillArgs& a, hipStream_t s);

// matrix-core chunked path (bfloat16 storage, dk = dv = 128, chunk = 64)
bool chunk_mfma_supported(int bf16, int dk, int dv, int chunk);
size_t chunk_mfma_workspace(int64_t N, int64_t T_fixed, int64_t T_total, bool fixed, int H, int chunk);
hipError_t launch_chunk_mfma(const PrefillArgs& a, hipStream_t s);
// the fixed device scratch of the entry point that allocates nothing: its size, and its address
// on the device of stream s (resolved once per device)
size_t noalloc_scratch_bytes();
hipError_t noalloc_scratch(hipStream_t s, void** out);

// decode step
bool decode_supported(int dk, int dv);
hipError_t launch_decode(const DecodeArgs& a, hipStream_t s);

// ---------------------------------------------------------------------------------------
// paged key-value cache and beam search
// ---------------------------------------------------------------------------------------
// A launch holds fewer than 2^32 threads along an axis of its grid: the workgroups of `threads` it may have.
// The `*_groups` functions below give the most workgroups (of 256 threads) of a call's launches.
constexpr int64_t max_groups(int threads) { return 0xFFFFFFFFll / threads; }

// Pages [n_pages, H_kv, page_size, d] and the table that names them (include/kda.h).
struct PageTable {
    const int32_t* table;
    int64_t stride;  // elements between rows
    int width;       // entries of a row
    int n_pages;
};

struct CacheAppendArgs {
    const void* k;
    const void* v;
    int64_t k_stride, v_stride;  // elements between tokens
    const int32_t* cu;           // [N + 1] or nullptr (one token per sequence)
    const int32_t* start;        // [N]
    int64_t N, T_total;
    void* kp;
    void* vp;
    int64_t kp_stride, vp_stride;  // elements between pages
    PageTable pt;
    int page_size, H, d, esz;
};
int64_t cache_append_groups(int64_t T_total, int H, int d, int esz);
hipError_t launch_cache_append(const CacheAppendArgs& a, hipStream_t s);

struct PagedDecodeArgs {
    const void* q;
    int64_t q_stride;
    const void* kp;
    const void* vp;
    int64_t kp_stride, vp_stride;
    PageTable pt;
    const int32_t* lengths;
    int64_t N;
    int page_size, Hq, Hkv, d, bf16;
    float scale;
    int window, sinks;
    int64_t max_length;  // > 0, at most width * page_size
    float* o;
    float* lse;  // or nullptr
    void* ws;
};
bool paged_decode_supported(int d);
// the same, and in `workspace` (0 where they do not fit a launch) the bytes of the partial results
int64_t paged_decode_groups(int64_t N, int Hq, int Hkv, int d, int bf16, int64_t max_length, int window, int sinks,
                            size_t* workspace);
hipError_t launch_paged_decode(const PagedDecodeArgs& a, hipStream_t s);

struct CacheForkArgs {
    PageTable pt;
    const int32_t* lengths;
    int64_t N;
    int32_t* refs;
    const int32_t* parents;
    int64_t N_out;
    int32_t* table_out;
    int64_t out_stride;
    int32_t* lengths_out;
};
int64_t cache_rows_groups(int64_t rows, int width);  // fork and free
hipError_t launch_cache_fork(const CacheForkArgs& a, hipStream_t s);

struct CacheFreeArgs {
    int32_t* table;
    int64_t stride;
    int width, n_pages;
    int32_t* lengths;
    int64_t N;
    int32_t* refs;
    const int32_t* rows;
    int64_t n_rows;
};
hipError_t launch_cache_free(const CacheFreeArgs& a, hipStream_t s);

struct CacheReserveArgs {
    int32_t* table;
    int64_t stride;
    int width, n_pages, page_size;
    int32_t* lengths;
    int64_t N;
    int32_t* refs;
    const int32_t* new_tokens;
    int32_t* copies;
    int32_t* granted;
    void* ws;
};
int64_t cache_reserve_groups(int64_t N, int64_t n_pages);
hipError_t launch_cache_reserve(const CacheReserveArgs& a, hipStream_t s);

struct CacheCompactArgs {
    PageTable pt;
    int64_t N;
    const int32_t* refs;
    int32_t* table_out;
    int64_t out_stride;
    int32_t* refs_out;
    int32_t* moves;
    void* ws;
};
int64_t cache_compact_groups(int64_t N, int width, int64_t n_pages);
hipError_t launch_cache_compact(const CacheCompactArgs& a, hipStream_t s);
size_t cache_workspace(int64_t N, int64_t n_pages);

// Buffers of one launch that copies pages or reorders rows.
constexpr int kMaxPools = 32;
struct PoolList {
    char* base[kMaxPools];
    int64_t stride[kMaxPools];  // bytes between pages
    int64_t bytes[kMaxPools];   // bytes of a page
    int count;
};
hipError_t launch_pages_copy(const PoolList& p, int n_pages, const int32_t* pairs, int64_t n_pairs, hipStream_t s);
hipError_t launch_beam_reorder(const PoolList& p, const int32_t* parents, int B, int K, hipStream_t s);

struct BeamSelectArgs {
    const void* logits;
    int64_t row_stride;
    const float* scores;
    const uint8_t* finished;
    int B, K, V, n_out, eos, bf16;
    float* scores_out;
    int32_t* parents;
    int32_t* tokens;
    uint8_t* finished_out;
    void* ws;
};
int64_t beam_select_groups(int64_t B, int K, int V);
size_t beam_select_workspace(int64_t B, int K, int V, int n_out);
hipError_t launch_beam_select(const BeamSelectArgs& a, hipStream_t s);

}  // namespace kda
