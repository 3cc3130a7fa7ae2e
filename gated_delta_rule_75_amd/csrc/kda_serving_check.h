// Argument checks that the serving calls share (kda_serving_api.cpp, kda_prompt_api.cpp): strided pools of
// pages, page tables, workspaces and overlaps.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <vector>

#include "kda_api_util.h"
#include "kda_internal.h"

namespace kda {
namespace api {

constexpr int64_t kMaxCount = 0x7FFFFFFF;
constexpr int32_t kMaxPages = 1 << 24;

// Bytes from the first to the end of the last of n rows of `row` bytes, `stride` apart (at most 2^62).
inline size_t extent(int64_t n, int64_t stride, int64_t row) {
    constexpr int64_t most = (int64_t)1 << 61;
    if (n <= 0) return 0;
    if (row > most || (n > 1 && stride > most / (n - 1))) return (size_t)1 << 62;
    return (size_t)((n - 1) * stride + row);
}

// Bytes of a page; 0 where the sizes are out of range (check_pages refuses them).
inline int64_t page_bytes_of(int32_t H, int32_t page_size, int32_t d, int64_t es) {
    if (H <= 0 || H > 1024 || page_size <= 0 || page_size > 4096 || d <= 0 || d > 1024) return 0;
    return (int64_t)H * page_size * d * es;
}

// A strided pool of pages.
struct Pool {
    const void* p;
    int64_t stride, page;  // bytes
    int64_t n;
    Span span() const { return Span{p, p ? extent(n, stride, page) : 0}; }
};

// (a single page has no stride)
inline Pool pool_of(const void* p, int64_t stride, int64_t page, int64_t n) { return Pool{p, n > 1 ? stride : page, page, n}; }

// Whether two pools share bytes.  Pools that interleave in one buffer (equal strides) do not when
// the pages of one lie between those of the other.
inline bool overlap(const Pool& a, const Pool& b) {
    if (!overlap(a.span(), b.span())) return false;
    if (a.stride != b.stride) return true;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(a.p), hi = reinterpret_cast<uintptr_t>(b.p);
    const int64_t fwd = hi >= lo ? (int64_t)((hi - lo) % (uintptr_t)a.stride)
                                 : (a.stride - (int64_t)((lo - hi) % (uintptr_t)a.stride)) % a.stride;
    return fwd < a.page || a.stride - fwd < b.page;
}

// strides and sizes small enough that no byte offset leaves 63 bits
inline bool sane_stride(int64_t elements) { return elements >= 0 && elements < ((int64_t)1 << 40); }

inline int check_table(const char* name, const int32_t* table, int64_t stride, int64_t N, int32_t width, int32_t n_pages) {
    if (N < 0 || width < 0) return fail(KDA_ERR_INVALID_ARG, "%s: sizes must be >= 0", name);
    if (n_pages < 1 || n_pages >= kMaxPages)
        return fail(KDA_ERR_INVALID_ARG, "%s: n_pages must be in [1, 2^24)", name);
    if (N > 0 && width > 0 && !table) return fail(KDA_ERR_INVALID_ARG, "%s: a page table is required", name);
    if (N > 1 && stride < width) return fail(KDA_ERR_INVALID_ARG, "%s: table rows overlap (stride below the width)", name);
    if (N > 1 && !sane_stride(stride)) return fail(KDA_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40)", name);
    if (!aligned_to(table, 4)) return fail(KDA_ERR_MISALIGNED, "%s: the page table must be 4-byte aligned", name);
    return KDA_OK;
}

inline Span table_span(const int32_t* t, int64_t stride, int64_t N, int32_t width) {
    return Span{t, width > 0 ? extent(N, N > 1 ? stride * 4 : 0, (int64_t)width * 4) : 0};
}

inline int check_pages(const char* name, const Pool& k, const Pool& v, int32_t page_size, int32_t H, int32_t d,
                int32_t dtype, bool written) {
    if (!valid_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "%s: dtype must be KDA_F32 or KDA_BF16", name);
    if (H <= 0 || H > 1024) return fail(KDA_ERR_INVALID_ARG, "%s: H_kv must be in [1, 1024]", name);
    if (!kda::paged_decode_supported(d)) return fail(KDA_ERR_UNSUPPORTED, "%s: d=%d not implemented", name, d);
    if (page_size < 16 || page_size > 4096 || page_size % 16)
        return fail(KDA_ERR_UNSUPPORTED, "%s: page_size=%d, expected a multiple of 16 up to 4096", name, page_size);
    if (!k.p || !v.p) return fail(KDA_ERR_INVALID_ARG, "%s: k_pages and v_pages are required", name);
    if (k.stride < k.page || v.stride < v.page)
        return fail(KDA_ERR_INVALID_ARG, "%s: pages overlap (stride below the page)", name);
    if (!aligned16(k.p) || !aligned16(v.p) || k.stride % 16 || v.stride % 16)
        return fail(KDA_ERR_MISALIGNED, "%s: pages must be 16-byte aligned", name);
    if (written && overlap(k, v)) return fail(KDA_ERR_ALIAS, "%s: k_pages and v_pages overlap", name);
    return KDA_OK;
}

// A launch of the call would not fit a grid.
inline int check_groups(const char* name, int64_t groups) {
    if (groups <= kda::max_groups(256)) return KDA_OK;
    return fail(KDA_ERR_INVALID_ARG, "%s: the call is too large (%lld workgroups of 256 threads; a launch holds fewer "
                "than 2^32 threads)", name, (long long)groups);
}

inline int check_workspace(const char* name, void* ws, size_t bytes, size_t need) {
    if (!aligned_to(ws, 256)) return fail(KDA_ERR_MISALIGNED, "%s: workspace must be 256-byte aligned", name);
    if (need && (!ws || bytes < need))
        return fail(KDA_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", name, need, ws ? bytes : (size_t)0);
    return KDA_OK;
}

// Outputs (and the workspace) may overlap neither an input nor one another.
template <size_t NO, size_t NI>
int check_alias(const char* name, const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (size_t i = 0; i < NO; ++i) {
        for (const Span& in : ins)
            if (overlap(outs[i], in)) return fail(KDA_ERR_ALIAS, "%s: an output overlaps an input", name);
        for (size_t j = i + 1; j < NO; ++j)
            if (overlap(outs[i], outs[j])) return fail(KDA_ERR_ALIAS, "%s: outputs or the workspace overlap", name);
    }
    return KDA_OK;
}

// Lengths and table entries on the device (KDA_DEBUG_CHECK=1).
inline int debug_check_table(const char* name, const int32_t* table, int64_t stride, const int32_t* lengths, int32_t N,
                      int32_t width, int32_t page_size, int32_t n_pages, int64_t max_length, hipStream_t s) {
    std::vector<int32_t> t, len;
    if (int rc = fetch(lengths, (size_t)N, s, len, name)) return rc;
    if (int rc = fetch(table, table_span(table, stride, N, width).bytes / 4, s, t, name)) return rc;
    return kda_validate_page_table(t.data(), stride, len.data(), N, width, page_size, n_pages, max_length);
}

inline int injected(const char* name) {
    return fail(KDA_ERR_HIP, "%s: injected launch failure (KDA_TEST_FAIL_LAUNCH)", name);
}

}  // namespace api
}  // namespace kda
