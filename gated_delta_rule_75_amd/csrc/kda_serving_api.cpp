// C ABI of the paged key-value cache and of beam search: argument validation and launch.
// Declarations and contracts: include/kda.h.
#include "kda.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <vector>

#include "kda_serving_check.h"

namespace {

using namespace kda::api;

int read_pools(const char* name, void* const* base, const int64_t* strides, const int64_t* bytes, int32_t count,
               int64_t rows) {
    if (count < 0) return fail(KDA_ERR_INVALID_ARG, "%s: the number of buffers must be >= 0", name);
    if (count > 0 && (!base || !bytes)) return fail(KDA_ERR_INVALID_ARG, "%s: the buffers' arrays are required", name);
    for (int32_t i = 0; i < count; ++i) {
        const int64_t st = strides ? strides[i] : bytes[i];
        if (bytes[i] < 0 || bytes[i] >= ((int64_t)1 << 32) || st < bytes[i] || !sane_stride(st))
            return fail(KDA_ERR_INVALID_ARG, "%s: buffer %d: bad row size or stride", name, i);
        if (rows > 0 && bytes[i] > 0 && !base[i]) return fail(KDA_ERR_INVALID_ARG, "%s: buffer %d is NULL", name, i);
        if (!aligned16(base[i]) || bytes[i] % 16 || st % 16)
            return fail(KDA_ERR_MISALIGNED, "%s: buffer %d: address, row size and stride must be multiples of 16", name, i);
    }
    for (int32_t i = 0; i < count; ++i)
        for (int32_t j = i + 1; j < count; ++j) {
            const Pool a{base[i], strides ? strides[i] : bytes[i], bytes[i], rows};
            const Pool b{base[j], strides ? strides[j] : bytes[j], bytes[j], rows};
            if (a.page > 0 && b.page > 0 && overlap(a, b))
                return fail(KDA_ERR_ALIAS, "%s: buffers %d and %d overlap", name, i, j);
        }
    return KDA_OK;
}

kda::PoolList take_pools(void* const* base, const int64_t* strides, const int64_t* bytes, int32_t first,
                         int32_t count) {
    kda::PoolList p{};
    p.count = count - first < kda::kMaxPools ? count - first : kda::kMaxPools;
    for (int i = 0; i < p.count; ++i) {
        p.base[i] = static_cast<char*>(base[first + i]);
        p.bytes[i] = bytes[first + i];
        p.stride[i] = strides ? strides[first + i] : bytes[first + i];
    }
    return p;
}

}  // namespace

extern "C" {

int kda_validate_page_table(const int32_t* page_table, int64_t table_stride, const int32_t* lengths, int32_t N,
                            int32_t table_pages, int32_t page_size, int32_t n_pages, int64_t max_length) {
    if (N < 0 || table_pages < 0 || page_size <= 0 || (N > 0 && (!lengths || (table_pages > 0 && !page_table))))
        return fail(KDA_ERR_INVALID_ARG, "kda_validate_page_table: bad arguments");
    int64_t most = (int64_t)table_pages * page_size;
    if (max_length > 0 && max_length < most) most = max_length;
    for (int32_t n = 0; n < N; ++n) {
        if (lengths[n] < 0 || lengths[n] > most)
            return fail(KDA_ERR_INVALID_ARG, "lengths[%d] = %d, expected 0 .. %lld", n, lengths[n], (long long)most);
        for (int32_t j = 0; j < table_pages; ++j) {
            const int32_t e = page_table[n * table_stride + j];
            if (e < -1 || e >= n_pages)
                return fail(KDA_ERR_INVALID_ARG, "page_table[%d, %d] = %d, expected -1 .. %d", n, j, e, n_pages - 1);
        }
    }
    return ok();
}

int kda_cache_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens,
                     const int32_t* start, int32_t N, int64_t T_total, void* k_pages, void* v_pages,
                     int64_t k_page_stride, int64_t v_page_stride, int32_t n_pages, int32_t page_size,
                     const int32_t* page_table, int64_t table_stride, int32_t table_pages, int32_t H_kv, int32_t d,
                     int32_t dtype, void* hip_stream) {
    static const char* name = "kda_cache_append";
    if (int rc = check_table(name, page_table, table_stride, N, table_pages, n_pages)) return rc;
    const int64_t es = dtype == KDA_BF16 ? 2 : 4;
    if (!sane_stride(k_page_stride) || !sane_stride(v_page_stride) || !sane_stride(k_stride) || !sane_stride(v_stride))
        return fail(KDA_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40)", name);
    const int64_t page = page_bytes_of(H_kv, page_size, d, es), row = (int64_t)H_kv * d * es;
    const Pool kp = pool_of(k_pages, k_page_stride * es, page, n_pages);
    const Pool vp = pool_of(v_pages, v_page_stride * es, page, n_pages);
    if (int rc = check_pages(name, kp, vp, page_size, H_kv, d, dtype, true)) return rc;
    if (T_total < 0 || T_total > kMaxCount) return fail(KDA_ERR_INVALID_ARG, "%s: T_total must be in [0, 2^31)", name);
    if (int rc = check_groups(name, kda::cache_append_groups(T_total, H_kv, d, (int)es))) return rc;
    if (!cu_seqlens && T_total != N)
        return fail(KDA_ERR_INVALID_ARG, "%s: without cu_seqlens T_total must be N", name);
    if (T_total > 0 && (N < 1 || !k || !v || !start))
        return fail(KDA_ERR_INVALID_ARG, "%s: k, v, start and at least one sequence are required", name);
    if (T_total > 1 && (k_stride * es < row || v_stride * es < row))
        return fail(KDA_ERR_INVALID_ARG, "%s: tokens overlap (stride below H_kv * d)", name);
    if (!aligned16(k) || !aligned16(v) || (T_total > 1 && (k_stride * es % 16 || v_stride * es % 16)))
        return fail(KDA_ERR_MISALIGNED, "%s: the tokens of k and v must be 16-byte aligned", name);
    if (!aligned_to(cu_seqlens, 4) || !aligned_to(start, 4))
        return fail(KDA_ERR_MISALIGNED, "%s: cu_seqlens and start must be 4-byte aligned", name);
    const Span ins[] = {{k, extent(T_total, k_stride * es, row)},
                        {v, extent(T_total, v_stride * es, row)},
                        {cu_seqlens, cu_seqlens ? ((size_t)N + 1) * 4 : 0},
                        {start, (size_t)N * 4},
                        table_span(page_table, table_stride, N, table_pages)};
    for (const Span& in : ins)
        if (overlap(kp.span(), in) || overlap(vp.span(), in))
            return fail(KDA_ERR_ALIAS, "%s: the pages overlap an input", name);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (debug_check()) {
        std::vector<int32_t> cu;
        if (cu_seqlens) {
            if (int rc = fetch(cu_seqlens, (size_t)N + 1, s, cu, name)) return rc;
            if (int rc = kda_validate_cu_seqlens(cu.data(), N, T_total)) return rc;
        }
    }
    if (injected_launch_failure()) return injected(name);
    kda::CacheAppendArgs a{};
    a.k = k; a.v = v; a.k_stride = k_stride; a.v_stride = v_stride;
    a.cu = cu_seqlens; a.start = start; a.N = N; a.T_total = T_total;
    a.kp = k_pages; a.vp = v_pages; a.kp_stride = k_page_stride; a.vp_stride = v_page_stride;
    a.pt = kda::PageTable{page_table, table_stride, table_pages, n_pages};
    a.page_size = page_size; a.H = H_kv; a.d = d; a.esz = (int)es;
    return check_hip(kda::launch_cache_append(a, s), s, name);
}

size_t kda_paged_decode_workspace(int32_t N, int32_t H_q, int32_t H_kv, int32_t d, int32_t dtype, int64_t max_length,
                                  int32_t window, int32_t sinks) {
    if (N < 0 || H_kv <= 0 || H_kv > 1024 || H_q <= 0 || H_q % H_kv || H_q > 16384 || !valid_dtype(dtype) ||
        !kda::paged_decode_supported(d) || max_length < 0 || window < 0 || sinks < 0)
        return (size_t)-1;
    size_t need;
    const int64_t groups =
        kda::paged_decode_groups(N, H_q, H_kv, d, dtype == KDA_BF16, max_length, window, sinks, &need);
    return groups > kda::max_groups(256) ? (size_t)-1 : need;
}

int kda_paged_decode(const void* q, int64_t q_stride, const void* k_pages, const void* v_pages, int64_t k_page_stride,
                     int64_t v_page_stride, int32_t n_pages, int32_t page_size, const int32_t* page_table,
                     int64_t table_stride, int32_t table_pages, const int32_t* lengths, int32_t N, int32_t H_q,
                     int32_t H_kv, int32_t d, int32_t dtype, float scale, int32_t window, int32_t sinks,
                     int64_t max_length, float* out, float* lse, void* workspace, size_t workspace_bytes,
                     void* hip_stream) {
    static const char* name = "kda_paged_decode";
    if (int rc = check_table(name, page_table, table_stride, N, table_pages, n_pages)) return rc;
    const int64_t es = dtype == KDA_BF16 ? 2 : 4;
    if (!sane_stride(k_page_stride) || !sane_stride(v_page_stride) || !sane_stride(q_stride))
        return fail(KDA_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40)", name);
    const int64_t page = page_bytes_of(H_kv, page_size, d, es), row = (int64_t)H_q * d * es;
    const Pool kp = pool_of(k_pages, k_page_stride * es, page, n_pages);
    const Pool vp = pool_of(v_pages, v_page_stride * es, page, n_pages);
    if (int rc = check_pages(name, kp, vp, page_size, H_kv, d, dtype, false)) return rc;
    if (H_q <= 0 || H_q % H_kv || H_q > 16384)
        return fail(KDA_ERR_INVALID_ARG, "%s: H_q must be a multiple of H_kv up to 16384", name);
    if (!std::isfinite(scale)) return fail(KDA_ERR_INVALID_ARG, "%s: scale must be finite", name);
    if (window < 0 || sinks < 0 || (sinks > 0 && window == 0))
        return fail(KDA_ERR_INVALID_ARG, "%s: window and sinks must be >= 0, and sinks 0 without a window", name);
    if (max_length < 0) return fail(KDA_ERR_INVALID_ARG, "%s: max_length must be >= 0", name);
    const int64_t room = (int64_t)table_pages * page_size;
    const int64_t most = max_length > 0 && max_length < room ? max_length : room;
    if (room > 0x7FFFFFFF - 4096)
        return fail(KDA_ERR_INVALID_ARG, "%s: table_pages * page_size must be below 2^31 - 4096", name);
    size_t need;
    const int64_t groups =
        kda::paged_decode_groups(N, H_q, H_kv, d, dtype == KDA_BF16, most, window, sinks, &need);
    if (int rc = check_groups(name, groups)) return rc;
    if (N > 0 && (!q || !lengths || !out)) return fail(KDA_ERR_INVALID_ARG, "%s: q, lengths and out are required", name);
    if (N > 1 && q_stride * es < row) return fail(KDA_ERR_INVALID_ARG, "%s: queries overlap (stride below H_q * d)", name);
    if (!aligned16(q) || (N > 1 && q_stride * es % 16))
        return fail(KDA_ERR_MISALIGNED, "%s: the rows of q must be 16-byte aligned", name);
    if (!aligned16(out) || !aligned_to(lse, 4) || !aligned_to(lengths, 4))
        return fail(KDA_ERR_MISALIGNED, "%s: out must be 16-byte, lse and lengths 4-byte aligned", name);
    if (int rc = check_workspace(name, workspace, workspace_bytes, need)) return rc;
    const Span ins[] = {{q, extent(N, q_stride * es, row)}, kp.span(), vp.span(),
                        table_span(page_table, table_stride, N, table_pages), {lengths, (size_t)N * 4}};
    const Span outs[] = {{out, (size_t)N * H_q * d * 4}, {lse, lse ? (size_t)N * H_q * 4 : 0}, {workspace, need}};
    if (int rc = check_alias(name, outs, ins)) return rc;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (debug_check())
        if (int rc = debug_check_table(name, page_table, table_stride, lengths, N, table_pages, page_size, n_pages, most, s))
            return rc;
    if (injected_launch_failure()) return injected(name);
    kda::PagedDecodeArgs a{};
    a.q = q; a.q_stride = q_stride; a.kp = k_pages; a.vp = v_pages;
    a.kp_stride = k_page_stride; a.vp_stride = v_page_stride;
    a.pt = kda::PageTable{page_table, table_stride, table_pages, n_pages};
    a.lengths = lengths; a.N = N; a.page_size = page_size; a.Hq = H_q; a.Hkv = H_kv; a.d = d;
    a.bf16 = dtype == KDA_BF16; a.scale = scale; a.window = window; a.sinks = sinks; a.max_length = most;
    a.o = out; a.lse = lse; a.ws = workspace;
    return check_hip(kda::launch_paged_decode(a, s), s, name);
}

int kda_cache_fork(const int32_t* page_table, int64_t table_stride, const int32_t* lengths, int32_t N,
                   int32_t table_pages, int32_t* refcount, int32_t n_pages, const int32_t* parents, int32_t N_out,
                   int32_t* table_out, int64_t table_out_stride, int32_t* lengths_out, void* hip_stream) {
    static const char* name = "kda_cache_fork";
    if (int rc = check_table(name, page_table, table_stride, N, table_pages, n_pages)) return rc;
    if (int rc = check_table(name, table_out, table_out_stride, N_out, table_pages, n_pages)) return rc;
    if (!sane_stride(table_stride) || !sane_stride(table_out_stride))
        return fail(KDA_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40)", name);
    if (!refcount || (N > 0 && !lengths) || (N_out > 0 && (!parents || !lengths_out)))
        return fail(KDA_ERR_INVALID_ARG, "%s: refcount, lengths, parents and lengths_out are required", name);
    if (int rc = check_groups(name, kda::cache_rows_groups(N > N_out ? N : N_out, table_pages))) return rc;
    const void* words[] = {lengths, refcount, parents, lengths_out};
    for (const void* p : words)
        if (!aligned_to(p, 4)) return fail(KDA_ERR_MISALIGNED, "%s: int32 buffers must be 4-byte aligned", name);
    const Span ins[] = {table_span(page_table, table_stride, N, table_pages), {lengths, (size_t)N * 4},
                        {parents, (size_t)N_out * 4}};
    const Span outs[] = {table_span(table_out, table_out_stride, N_out, table_pages), {lengths_out, (size_t)N_out * 4},
                         {refcount, (size_t)n_pages * 4}};
    if (int rc = check_alias(name, outs, ins)) return rc;
    if (injected_launch_failure()) return injected(name);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    kda::CacheForkArgs a{};
    a.pt = kda::PageTable{page_table, table_stride, table_pages, n_pages};
    a.lengths = lengths; a.N = N; a.refs = refcount; a.parents = parents; a.N_out = N_out;
    a.table_out = table_out; a.out_stride = table_out_stride; a.lengths_out = lengths_out;
    return check_hip(kda::launch_cache_fork(a, s), s, name);
}

int kda_cache_free(int32_t* page_table, int64_t table_stride, int32_t* lengths, int32_t N, int32_t table_pages,
                   int32_t* refcount, int32_t n_pages, const int32_t* rows, int32_t n_rows, void* hip_stream) {
    static const char* name = "kda_cache_free";
    if (int rc = check_table(name, page_table, table_stride, N, table_pages, n_pages)) return rc;
    if (!sane_stride(table_stride)) return fail(KDA_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40)", name);
    if (n_rows < 0) return fail(KDA_ERR_INVALID_ARG, "%s: the number of rows must be >= 0", name);
    if (int rc = check_groups(name, kda::cache_rows_groups(n_rows, table_pages))) return rc;
    if (!refcount || (N > 0 && !lengths) || (n_rows > 0 && !rows))
        return fail(KDA_ERR_INVALID_ARG, "%s: refcount, lengths and rows are required", name);
    if (!aligned_to(lengths, 4) || !aligned_to(refcount, 4) || !aligned_to(rows, 4))
        return fail(KDA_ERR_MISALIGNED, "%s: int32 buffers must be 4-byte aligned", name);
    const Span ins[] = {{rows, (size_t)n_rows * 4}};
    const Span outs[] = {table_span(page_table, table_stride, N, table_pages), {lengths, (size_t)N * 4},
                         {refcount, (size_t)n_pages * 4}};
    if (int rc = check_alias(name, outs, ins)) return rc;
    if (injected_launch_failure()) return injected(name);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    kda::CacheFreeArgs a{};
    a.table = page_table; a.stride = table_stride; a.width = table_pages; a.n_pages = n_pages; a.lengths = lengths;
    a.N = N; a.refs = refcount; a.rows = rows; a.n_rows = n_rows;
    return check_hip(kda::launch_cache_free(a, s), s, name);
}

size_t kda_cache_workspace_size(int32_t N, int32_t n_pages) {
    if (N < 0 || n_pages < 0 || n_pages >= kMaxPages) return (size_t)-1;
    return kda::cache_workspace(N, n_pages);
}

int kda_cache_reserve(int32_t* page_table, int64_t table_stride, int32_t* lengths, int32_t N, int32_t table_pages,
                      int32_t* refcount, int32_t n_pages, int32_t page_size, const int32_t* new_tokens,
                      int32_t* copies, int32_t* granted, void* workspace, size_t workspace_bytes, void* hip_stream) {
    static const char* name = "kda_cache_reserve";
    if (int rc = check_table(name, page_table, table_stride, N, table_pages, n_pages)) return rc;
    if (!sane_stride(table_stride)) return fail(KDA_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40)", name);
    if (page_size < 1) return fail(KDA_ERR_INVALID_ARG, "%s: page_size must be positive", name);
    if (int rc = check_groups(name, kda::cache_reserve_groups(N, n_pages))) return rc;
    if (!refcount || (N > 0 && (!lengths || !new_tokens || !copies || !granted)))
        return fail(KDA_ERR_INVALID_ARG, "%s: refcount, lengths, new_tokens, copies and granted are required", name);
    const void* words[] = {lengths, refcount, new_tokens, copies, granted};
    for (const void* p : words)
        if (!aligned_to(p, 4)) return fail(KDA_ERR_MISALIGNED, "%s: int32 buffers must be 4-byte aligned", name);
    const size_t need = kda::cache_workspace(N, n_pages);
    if (int rc = check_workspace(name, workspace, workspace_bytes, need)) return rc;
    const Span ins[] = {{new_tokens, (size_t)N * 4}};
    const Span outs[] = {table_span(page_table, table_stride, N, table_pages), {lengths, (size_t)N * 4},
                         {refcount, (size_t)n_pages * 4}, {copies, (size_t)N * 8}, {granted, (size_t)N * 4},
                         {workspace, need}};
    if (int rc = check_alias(name, outs, ins)) return rc;
    if (injected_launch_failure()) return injected(name);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    kda::CacheReserveArgs a{};
    a.table = page_table; a.stride = table_stride; a.width = table_pages; a.n_pages = n_pages;
    a.page_size = page_size; a.lengths = lengths; a.N = N; a.refs = refcount; a.new_tokens = new_tokens;
    a.copies = copies; a.granted = granted; a.ws = workspace;
    return check_hip(kda::launch_cache_reserve(a, s), s, name);
}

int kda_cache_compact(const int32_t* page_table, int64_t table_stride, int32_t N, int32_t table_pages,
                      const int32_t* refcount, int32_t n_pages, int32_t* table_out, int64_t table_out_stride,
                      int32_t* refcount_out, int32_t* moves, void* workspace, size_t workspace_bytes,
                      void* hip_stream) {
    static const char* name = "kda_cache_compact";
    if (int rc = check_table(name, page_table, table_stride, N, table_pages, n_pages)) return rc;
    if (int rc = check_table(name, table_out, table_out_stride, N, table_pages, n_pages)) return rc;
    if (!sane_stride(table_stride) || !sane_stride(table_out_stride))
        return fail(KDA_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40)", name);
    if (!refcount || !refcount_out || (n_pages > 1 && !moves))
        return fail(KDA_ERR_INVALID_ARG, "%s: refcount, refcount_out and moves are required", name);
    if (int rc = check_groups(name, kda::cache_compact_groups(N, table_pages, n_pages))) return rc;
    const void* words[] = {refcount, refcount_out, moves};
    for (const void* p : words)
        if (!aligned_to(p, 4)) return fail(KDA_ERR_MISALIGNED, "%s: int32 buffers must be 4-byte aligned", name);
    const size_t need = kda::cache_workspace(N, n_pages);
    if (int rc = check_workspace(name, workspace, workspace_bytes, need)) return rc;
    const Span tin = table_span(page_table, table_stride, N, table_pages);
    const Span tout = table_span(table_out, table_out_stride, N, table_pages);
    const Span rin{refcount, (size_t)n_pages * 4}, rout{refcount_out, (size_t)n_pages * 4};
    const bool table_place = table_out == page_table && table_out_stride == table_stride;
    if ((!table_place && overlap(tin, tout)) || (refcount_out != refcount && overlap(rin, rout)))
        return fail(KDA_ERR_ALIAS, "%s: an output partially overlaps its input", name);
    if (overlap(tin, rout) || overlap(rin, tout)) return fail(KDA_ERR_ALIAS, "%s: an output overlaps an input", name);
    const Span ins[] = {tin, rin};
    const Span outs[] = {{moves, (size_t)(n_pages / 2) * 8}, {workspace, need}};
    if (int rc = check_alias(name, outs, ins)) return rc;
    const Span rest[] = {tout, rout};
    if (int rc = check_alias(name, outs, rest)) return rc;
    if (overlap(tout, rout)) return fail(KDA_ERR_ALIAS, "%s: outputs overlap", name);
    if (injected_launch_failure()) return injected(name);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    kda::CacheCompactArgs a{};
    a.pt = kda::PageTable{page_table, table_stride, table_pages, n_pages};
    a.N = N; a.refs = refcount; a.table_out = table_out; a.out_stride = table_out_stride;
    a.refs_out = refcount_out; a.moves = moves; a.ws = workspace;
    return check_hip(kda::launch_cache_compact(a, s), s, name);
}

int kda_pages_copy(void* const* pools, const int64_t* page_strides, const int64_t* page_bytes, int32_t n_pools,
                   int32_t n_pages, const int32_t* pairs, int64_t n_pairs, void* hip_stream) {
    static const char* name = "kda_pages_copy";
    if (n_pages < 0 || n_pairs < 0 || n_pairs > kMaxCount)
        return fail(KDA_ERR_INVALID_ARG, "%s: n_pages and n_pairs must be in [0, 2^31)", name);
    if (n_pools > 0 && !page_strides) return fail(KDA_ERR_INVALID_ARG, "%s: page_strides is required", name);
    if (int rc = read_pools(name, pools, page_strides, page_bytes, n_pools, n_pages)) return rc;
    if (n_pairs > 0 && !pairs) return fail(KDA_ERR_INVALID_ARG, "%s: pairs is required", name);
    if (!aligned_to(pairs, 4)) return fail(KDA_ERR_MISALIGNED, "%s: pairs must be 4-byte aligned", name);
    for (int32_t i = 0; i < n_pools; ++i)
        if (overlap(Pool{pools[i], page_strides[i], page_bytes[i], n_pages}.span(), Span{pairs, (size_t)n_pairs * 8}))
            return fail(KDA_ERR_ALIAS, "%s: pool %d overlaps pairs", name, i);
    if (injected_launch_failure()) return injected(name);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    hipError_t e = hipSuccess;
    for (int32_t i = 0; i < n_pools && e == hipSuccess; i += kda::kMaxPools)
        e = kda::launch_pages_copy(take_pools(pools, page_strides, page_bytes, i, n_pools), n_pages, pairs, n_pairs, s);
    return check_hip(e, s, name);
}

size_t kda_beam_select_workspace(int32_t B, int32_t K, int32_t V, int32_t n_out) {
    if (B < 0 || K < 1 || K > 64 || n_out < 1 || n_out > 64 || V < 1 || V >= (1 << 24) || (int64_t)K * V < n_out)
        return (size_t)-1;
    return kda::beam_select_workspace(B, K, V, n_out);
}

int kda_beam_select(const void* logits, int64_t row_stride, const float* scores, const uint8_t* finished, int32_t B,
                    int32_t K, int32_t V, int32_t n_out, int32_t eos, int32_t dtype, float* scores_out,
                    int32_t* parents, int32_t* tokens, uint8_t* finished_out, void* workspace, size_t workspace_bytes,
                    void* hip_stream) {
    static const char* name = "kda_beam_select";
    if (!valid_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "%s: dtype must be KDA_F32 or KDA_BF16", name);
    const size_t need = kda_beam_select_workspace(B, K, V, n_out);
    if (need == (size_t)-1)
        return fail(KDA_ERR_INVALID_ARG, "%s: B=%d K=%d V=%d n_out=%d: expected B >= 0, 1 <= K, n_out <= 64, "
                    "1 <= V < 2^24, n_out <= K * V", name, B, K, V, n_out);
    if (finished && (eos < 0 || eos >= V)) return fail(KDA_ERR_INVALID_ARG, "%s: eos must be in [0, V)", name);
    if ((finished != nullptr) != (finished_out != nullptr) && B > 0)
        return fail(KDA_ERR_INVALID_ARG, "%s: finished and finished_out go together", name);
    if (B > 0 && (!logits || !scores || !scores_out || !parents || !tokens))
        return fail(KDA_ERR_INVALID_ARG, "%s: logits, scores and the outputs are required", name);
    const int64_t rows = (int64_t)B * K, es = dtype == KDA_BF16 ? 2 : 4;
    if (!sane_stride(row_stride) || (rows > 1 && row_stride < V))
        return fail(KDA_ERR_INVALID_ARG, "%s: row_stride must be in [V, 2^40)", name);
    if (int rc = check_groups(name, kda::beam_select_groups(B, K, V))) return rc;
    if (!aligned_to(logits, es)) return fail(KDA_ERR_MISALIGNED, "%s: logits must be aligned to their element", name);
    const void* words[] = {scores, scores_out, parents, tokens};
    for (const void* p : words)
        if (!aligned_to(p, 4)) return fail(KDA_ERR_MISALIGNED, "%s: 32-bit buffers must be 4-byte aligned", name);
    if (int rc = check_workspace(name, workspace, workspace_bytes, need)) return rc;
    const size_t no = (size_t)B * n_out;
    const Span ins[] = {{logits, extent(rows, row_stride * es, (int64_t)V * es)}, {scores, (size_t)rows * 4},
                        {finished, finished ? (size_t)rows : 0}};
    const Span outs[] = {{scores_out, no * 4}, {parents, no * 4}, {tokens, no * 4},
                         {finished_out, finished_out ? no : 0}, {workspace, need}};
    if (int rc = check_alias(name, outs, ins)) return rc;
    if (injected_launch_failure()) return injected(name);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    kda::BeamSelectArgs a{};
    a.logits = logits; a.row_stride = row_stride; a.scores = scores; a.finished = finished;
    a.B = B; a.K = K; a.V = V; a.n_out = n_out; a.eos = eos; a.bf16 = dtype == KDA_BF16;
    a.scores_out = scores_out; a.parents = parents; a.tokens = tokens; a.finished_out = finished_out;
    a.ws = workspace;
    return check_hip(kda::launch_beam_select(a, s), s, name);
}

int kda_beam_reorder(void* const* states, const int64_t* row_bytes, int32_t n_states, const int32_t* parents,
                     int32_t B, int32_t K, void* hip_stream) {
    static const char* name = "kda_beam_reorder";
    if (B < 0 || K < 1 || K > 64) return fail(KDA_ERR_INVALID_ARG, "%s: expected B >= 0 and 1 <= K <= 64", name);
    const int64_t rows = (int64_t)B * K;
    if (int rc = read_pools(name, states, nullptr, row_bytes, n_states, rows)) return rc;
    if (rows > 0 && !parents) return fail(KDA_ERR_INVALID_ARG, "%s: parents is required", name);
    if (!aligned_to(parents, 4)) return fail(KDA_ERR_MISALIGNED, "%s: parents must be 4-byte aligned", name);
    for (int32_t i = 0; i < n_states; ++i) {
        if (overlap(Span{states[i], (size_t)(rows * row_bytes[i])}, Span{parents, (size_t)rows * 4}))
            return fail(KDA_ERR_ALIAS, "%s: state %d overlaps parents", name, i);
    }
    if (injected_launch_failure()) return injected(name);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    hipError_t e = hipSuccess;
    for (int32_t i = 0; i < n_states && e == hipSuccess; i += kda::kMaxPools)
        e = kda::launch_beam_reorder(take_pools(states, nullptr, row_bytes, i, n_states), parents, B, K, s);
    return check_hip(e, s, name);
}

}  // extern "C"
