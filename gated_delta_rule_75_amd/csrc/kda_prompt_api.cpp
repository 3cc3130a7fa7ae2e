// C ABI of the prompt chunks' calls: argument validation and launch.  Declarations and contracts: include/kda.h.
#include "kda.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <vector>

#include "kda_serving_check.h"

namespace {

using namespace kda::api;

// Token rows of a strided tensor (a single row has no stride).
Pool rows_of(const void* p, int64_t stride, int64_t row, int64_t n) { return n > 0 ? pool_of(p, stride, row, n) : Pool{p, row, row, 0}; }

bool same(const Pool& a, const Pool& b) { return a.p == b.p && a.stride == b.stride; }

int check_rows(const char* name, const char* what, const Pool& x) {
    if (x.n > 0 && !x.p) return fail(KDA_ERR_INVALID_ARG, "%s: %s is required", name, what);
    if (x.stride < x.page) return fail(KDA_ERR_INVALID_ARG, "%s: tokens of %s overlap (stride below its heads)", name, what);
    if (!aligned16(x.p) || x.stride % 16)
        return fail(KDA_ERR_MISALIGNED, "%s: the tokens of %s must be 16-byte aligned", name, what);
    return KDA_OK;
}

int check_turn(const char* name, const double* freqs, int32_t H_q, int32_t d, int32_t rotary_dim, int32_t layout,
               float amplitude) {
    if (H_q <= 0 || H_q > 16384) return fail(KDA_ERR_INVALID_ARG, "%s: H_q must be in [1, 16384]", name);
    if (rotary_dim < 2 || rotary_dim > d || rotary_dim % 2)
        return fail(KDA_ERR_INVALID_ARG, "%s: rotary_dim must be even, 2 .. d", name);
    if (layout != KDA_ROTARY_HALVES && layout != KDA_ROTARY_INTERLEAVED)
        return fail(KDA_ERR_INVALID_ARG, "%s: layout must be KDA_ROTARY_HALVES or KDA_ROTARY_INTERLEAVED", name);
    if (!std::isfinite(amplitude)) return fail(KDA_ERR_INVALID_ARG, "%s: amplitude must be finite", name);
    if (!freqs) return fail(KDA_ERR_INVALID_ARG, "%s: freqs are required", name);
    if (!aligned_to(freqs, 8)) return fail(KDA_ERR_MISALIGNED, "%s: freqs must be 8-byte aligned", name);
    return KDA_OK;
}

int check_logits(const char* name, const void* x, int64_t stride, int64_t R, int32_t V, int32_t dtype) {
    if (!valid_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "%s: dtype must be KDA_F32 or KDA_BF16", name);
    if (R < 0 || R > kMaxCount) return fail(KDA_ERR_INVALID_ARG, "%s: R must be in [0, 2^31)", name);
    if (V < 1 || V >= (1 << 24)) return fail(KDA_ERR_INVALID_ARG, "%s: V=%d, expected 1 .. 2^24 - 1", name, V);
    if (!sane_stride(stride)) return fail(KDA_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40)", name);
    if (R > 1 && stride < V) return fail(KDA_ERR_INVALID_ARG, "%s: rows overlap (stride below V)", name);
    if (R > 0 && !x) return fail(KDA_ERR_INVALID_ARG, "%s: logits and d_logits are required", name);
    if (!aligned_to(x, dtype == KDA_BF16 ? 2 : 4))
        return fail(KDA_ERR_MISALIGNED, "%s: logits must be aligned to their type", name);
    return KDA_OK;
}

Span logit_span(const void* x, int64_t stride, int64_t R, int32_t V, int64_t es) {
    return Span{x, extent(R, R > 1 ? stride * es : 0, V * es)};
}

}  // namespace

extern "C" {

int kda_rotary(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const int32_t* positions,
               const double* freqs, int64_t T, int32_t H_q, int32_t H_k, int32_t d, int32_t rotary_dim,
               int32_t layout, float amplitude, int32_t inverse, int32_t dtype, void* q_out, int64_t q_out_stride,
               void* k_out, int64_t k_out_stride, void* hip_stream) {
    static const char* name = "kda_rotary";
    if (!valid_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "%s: dtype must be KDA_F32 or KDA_BF16", name);
    if (T < 0 || T > kMaxCount) return fail(KDA_ERR_INVALID_ARG, "%s: T must be in [0, 2^31)", name);
    if (d < 8 || d > 512 || d % 8) return fail(KDA_ERR_UNSUPPORTED, "%s: d=%d, expected a multiple of 8 up to 512", name, d);
    if (H_k < 0 || H_k > 1024) return fail(KDA_ERR_INVALID_ARG, "%s: H_k must be in [0, 1024]", name);
    if (int rc = check_turn(name, freqs, H_q, d, rotary_dim, layout, amplitude)) return rc;
    if (H_k == 0 && (k || k_out))
        return fail(KDA_ERR_INVALID_ARG, "%s: k, k_out and H_k go together", name);
    if (!sane_stride(q_stride) || !sane_stride(k_stride) || !sane_stride(q_out_stride) || !sane_stride(k_out_stride))
        return fail(KDA_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40)", name);
    const int64_t es = dtype == KDA_BF16 ? 2 : 4, qrow = (int64_t)H_q * d * es, krow = (int64_t)H_k * d * es;
    const Pool qi = rows_of(q, q_stride * es, qrow, T), qo = rows_of(q_out, q_out_stride * es, qrow, T);
    const int64_t kn = H_k ? T : 0;
    const Pool ki = rows_of(k, k_stride * es, krow, kn), ko = rows_of(k_out, k_out_stride * es, krow, kn);
    if (int rc = check_rows(name, "q", qi)) return rc;
    if (int rc = check_rows(name, "q_out", qo)) return rc;
    if (int rc = check_rows(name, "k", ki)) return rc;
    if (int rc = check_rows(name, "k_out", ko)) return rc;
    if (T > 0 && !positions) return fail(KDA_ERR_INVALID_ARG, "%s: positions are required", name);
    if (!aligned_to(positions, 4)) return fail(KDA_ERR_MISALIGNED, "%s: positions must be 4-byte aligned", name);
    const Span ps{positions, (size_t)T * 4}, fs{freqs, (size_t)rotary_dim * 4};
    if ((!same(qi, qo) && overlap(qi, qo)) || (!same(ki, ko) && overlap(ki, ko)) || overlap(qo, ki) || overlap(ko, qi))
        return fail(KDA_ERR_ALIAS, "%s: an output overlaps an input that it is not", name);
    if (overlap(qo, ko)) return fail(KDA_ERR_ALIAS, "%s: q_out and k_out overlap", name);
    for (const Pool& o : {qo, ko})
        if (overlap(o.span(), ps) || overlap(o.span(), fs))
            return fail(KDA_ERR_ALIAS, "%s: an output overlaps positions or freqs", name);
    kda::RotaryArgs a{};
    a.q = q; a.k = k; a.q_stride = q_stride; a.k_stride = k_stride;
    a.q_out = q_out; a.k_out = k_out; a.q_out_stride = q_out_stride; a.k_out_stride = k_out_stride;
    a.positions = positions; a.T = T; a.freqs = freqs;
    a.Hq = H_q; a.Hk = H_k; a.d = d; a.r = rotary_dim; a.interleaved = layout == KDA_ROTARY_INTERLEAVED;
    a.inverse = inverse != 0; a.bf16 = dtype == KDA_BF16; a.amplitude = amplitude;
    if (int rc = check_groups(name, kda::rotary_groups(a))) return rc;
    if (injected_launch_failure()) return injected(name);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    return check_hip(kda::launch_rotary(a, s), s, name);
}

int kda_rotary_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                      int64_t v_stride, const int32_t* cu_seqlens, const int32_t* start, int32_t N, int64_t T_total,
                      const double* freqs, int32_t rotary_dim, int32_t layout, float amplitude, void* q_out,
                      int64_t q_out_stride, void* k_pages, void* v_pages, int64_t k_page_stride,
                      int64_t v_page_stride, int32_t n_pages, int32_t page_size, const int32_t* page_table,
                      int64_t table_stride, int32_t table_pages, int32_t H_q, int32_t H_kv, int32_t d, int32_t dtype,
                      void* hip_stream) {
    static const char* name = "kda_rotary_append";
    if (int rc = check_table(name, page_table, table_stride, N, table_pages, n_pages)) return rc;
    const int64_t es = dtype == KDA_BF16 ? 2 : 4;
    if (!sane_stride(k_page_stride) || !sane_stride(v_page_stride) || !sane_stride(q_stride) ||
        !sane_stride(k_stride) || !sane_stride(v_stride) || !sane_stride(q_out_stride))
        return fail(KDA_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40)", name);
    const int64_t page = page_bytes_of(H_kv, page_size, d, es);
    const Pool kp = pool_of(k_pages, k_page_stride * es, page, n_pages);
    const Pool vp = pool_of(v_pages, v_page_stride * es, page, n_pages);
    if (int rc = check_pages(name, kp, vp, page_size, H_kv, d, dtype, true)) return rc;
    if (T_total < 0 || T_total > kMaxCount) return fail(KDA_ERR_INVALID_ARG, "%s: T_total must be in [0, 2^31)", name);
    if (int rc = check_turn(name, freqs, H_q, d, rotary_dim, layout, amplitude)) return rc;
    if (!cu_seqlens && T_total != N)
        return fail(KDA_ERR_INVALID_ARG, "%s: without cu_seqlens T_total must be N", name);
    if (T_total > 0 && (N < 1 || !start))
        return fail(KDA_ERR_INVALID_ARG, "%s: start and at least one sequence are required", name);
    const int64_t qrow = (int64_t)H_q * d * es, row = (int64_t)H_kv * d * es;
    const Pool qi = rows_of(q, q_stride * es, qrow, T_total), qo = rows_of(q_out, q_out_stride * es, qrow, T_total);
    const Pool ki = rows_of(k, k_stride * es, row, T_total), vi = rows_of(v, v_stride * es, row, T_total);
    if (int rc = check_rows(name, "q", qi)) return rc;
    if (int rc = check_rows(name, "q_out", qo)) return rc;
    if (int rc = check_rows(name, "k", ki)) return rc;
    if (int rc = check_rows(name, "v", vi)) return rc;
    if (!aligned_to(cu_seqlens, 4) || !aligned_to(start, 4))
        return fail(KDA_ERR_MISALIGNED, "%s: cu_seqlens and start must be 4-byte aligned", name);
    if ((!same(qi, qo) && overlap(qi, qo)) || overlap(qo, ki) || overlap(qo, vi))
        return fail(KDA_ERR_ALIAS, "%s: q_out overlaps an input that it is not", name);
    const Span ins[] = {qi.span(), ki.span(), vi.span(), qo.span(),
                        {cu_seqlens, cu_seqlens ? ((size_t)N + 1) * 4 : 0}, {start, (size_t)N * 4},
                        {freqs, (size_t)rotary_dim * 4}, table_span(page_table, table_stride, N, table_pages)};
    for (const Span& in : ins)
        if (overlap(kp.span(), in) || overlap(vp.span(), in))
            return fail(KDA_ERR_ALIAS, "%s: the pages overlap another argument", name);
    for (int i = 4; i < 8; ++i)
        if (overlap(qo.span(), ins[i])) return fail(KDA_ERR_ALIAS, "%s: q_out overlaps an input that it is not", name);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    kda::RotaryArgs a{};
    a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.q_out = q_out; a.q_out_stride = q_out_stride;
    a.cu = cu_seqlens; a.start = start; a.N = N; a.T = T_total; a.freqs = freqs;
    a.Hq = H_q; a.Hk = H_kv; a.d = d; a.r = rotary_dim; a.interleaved = layout == KDA_ROTARY_INTERLEAVED;
    a.bf16 = dtype == KDA_BF16; a.amplitude = amplitude;
    a.kp = k_pages; a.vp = v_pages; a.kp_stride = k_page_stride; a.vp_stride = v_page_stride;
    a.pt = kda::PageTable{page_table, table_stride, table_pages, n_pages};
    a.page_size = page_size;
    if (int rc = check_groups(name, kda::rotary_groups(a))) return rc;
    if (debug_check() && cu_seqlens) {
        std::vector<int32_t> cu;
        if (int rc = fetch(cu_seqlens, (size_t)N + 1, s, cu, name)) return rc;
        if (int rc = kda_validate_cu_seqlens(cu.data(), N, T_total)) return rc;
    }
    if (injected_launch_failure()) return injected(name);
    return check_hip(kda::launch_rotary(a, s), s, name);
}

size_t kda_paged_prefill_workspace(int32_t N, int64_t T_total, int32_t H_q, int32_t H_kv, int32_t d, int32_t dtype,
                                   int64_t max_length, int32_t window, int32_t sinks) {
    if (N < 0 || T_total < 0 || T_total > kMaxCount || H_kv <= 0 || H_kv > 1024 || H_q <= 0 || H_q % H_kv ||
        H_q > 16384 || !valid_dtype(dtype) || !kda::paged_decode_supported(d) || max_length < 0 ||
        max_length > kMaxCount - 4096 || window < 0 || sinks < 0)
        return (size_t)-1;
    kda::PagedPrefillArgs a{};
    a.N = N; a.T = T_total; a.Hq = H_q; a.Hkv = H_kv; a.d = d; a.bf16 = dtype == KDA_BF16;
    a.window = window; a.sinks = sinks;
    // (0 is no bound, as in the call: what splits a short table's rows, a longer one's splits too, in as many bytes)
    a.max_length = max_length > 0 ? max_length : kMaxCount - 4096;
    size_t need;
    return kda::paged_prefill_groups(a, &need) > kda::max_groups(256) ? (size_t)-1 : need;
}

int kda_paged_prefill(const void* q, int64_t q_stride, const void* k_pages, const void* v_pages, int64_t k_page_stride,
                      int64_t v_page_stride, int32_t n_pages, int32_t page_size, const int32_t* page_table,
                      int64_t table_stride, int32_t table_pages, const int32_t* lengths, const int32_t* cu_seqlens,
                      int32_t N, int64_t T_total, int32_t H_q, int32_t H_kv, int32_t d, int32_t dtype, float scale,
                      int32_t window, int32_t sinks, int64_t max_length, void* out, float* lse, void* workspace,
                      size_t workspace_bytes, void* hip_stream) {
    static const char* name = "kda_paged_prefill";
    if (int rc = check_table(name, page_table, table_stride, N, table_pages, n_pages)) return rc;
    const int64_t es = dtype == KDA_BF16 ? 2 : 4;
    if (!sane_stride(k_page_stride) || !sane_stride(v_page_stride) || !sane_stride(q_stride))
        return fail(KDA_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40)", name);
    const int64_t page = page_bytes_of(H_kv, page_size, d, es);
    const Pool kp = pool_of(k_pages, k_page_stride * es, page, n_pages);
    const Pool vp = pool_of(v_pages, v_page_stride * es, page, n_pages);
    if (int rc = check_pages(name, kp, vp, page_size, H_kv, d, dtype, false)) return rc;
    if (T_total < 0 || T_total > kMaxCount) return fail(KDA_ERR_INVALID_ARG, "%s: T_total must be in [0, 2^31)", name);
    if (H_q <= 0 || H_q % H_kv || H_q > 16384)
        return fail(KDA_ERR_INVALID_ARG, "%s: H_q must be a multiple of H_kv up to 16384", name);
    if (!std::isfinite(scale)) return fail(KDA_ERR_INVALID_ARG, "%s: scale must be finite", name);
    if (window < 0 || sinks < 0 || (sinks > 0 && window == 0))
        return fail(KDA_ERR_INVALID_ARG, "%s: window and sinks must be >= 0, and sinks 0 without a window", name);
    if (max_length < 0) return fail(KDA_ERR_INVALID_ARG, "%s: max_length must be >= 0", name);
    const int64_t room = (int64_t)table_pages * page_size;
    const int64_t most = max_length > 0 && max_length < room ? max_length : room;
    if (room > kMaxCount - 4096)
        return fail(KDA_ERR_INVALID_ARG, "%s: table_pages * page_size must be below 2^31 - 4096", name);
    if (T_total > 0 && (N < 1 || !lengths || !cu_seqlens || !out))
        return fail(KDA_ERR_INVALID_ARG, "%s: lengths, cu_seqlens, out and at least one sequence are required", name);
    const Pool qi = rows_of(q, q_stride * es, (int64_t)H_q * d * es, T_total);
    if (int rc = check_rows(name, "q", qi)) return rc;
    if (!aligned16(out) || !aligned_to(lse, 4) || !aligned_to(lengths, 4) || !aligned_to(cu_seqlens, 4))
        return fail(KDA_ERR_MISALIGNED, "%s: out must be 16-byte, lse, lengths and cu_seqlens 4-byte aligned", name);
    kda::PagedPrefillArgs a{};
    a.q = q; a.q_stride = q_stride; a.kp = k_pages; a.vp = v_pages;
    a.kp_stride = k_page_stride; a.vp_stride = v_page_stride;
    a.pt = kda::PageTable{page_table, table_stride, table_pages, n_pages};
    a.lengths = lengths; a.cu = cu_seqlens; a.N = N; a.T = T_total; a.page_size = page_size;
    a.Hq = H_q; a.Hkv = H_kv; a.d = d; a.bf16 = dtype == KDA_BF16; a.scale = scale;
    a.window = window; a.sinks = sinks; a.max_length = most;
    a.o = out; a.lse = lse; a.ws = workspace;
    size_t need;
    if (int rc = check_groups(name, kda::paged_prefill_groups(a, &need))) return rc;
    if (int rc = check_workspace(name, workspace, workspace_bytes, need)) return rc;
    const Span ins[] = {qi.span(), kp.span(), vp.span(), table_span(page_table, table_stride, N, table_pages),
                        {lengths, (size_t)N * 4}, {cu_seqlens, ((size_t)N + 1) * 4}};
    const Span outs[] = {{out, (size_t)T_total * H_q * d * es}, {lse, lse ? (size_t)T_total * H_q * 4 : 0},
                         {workspace, need}};
    if (int rc = check_alias(name, outs, ins)) return rc;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (debug_check() && T_total > 0) {
        std::vector<int32_t> cu;
        if (int rc = fetch(cu_seqlens, (size_t)N + 1, s, cu, name)) return rc;
        if (int rc = kda_validate_cu_seqlens(cu.data(), N, T_total)) return rc;
        if (int rc = debug_check_table(name, page_table, table_stride, lengths, N, table_pages, page_size, n_pages, most, s))
            return rc;
    }
    if (injected_launch_failure()) return injected(name);
    return check_hip(kda::launch_paged_prefill(a, s), s, name);
}

size_t kda_token_logprobs_workspace(int64_t R, int32_t V, int32_t top) {
    if (R < 0 || R > kMaxCount || V < 1 || V >= (1 << 24) || top < 0 || top > 64 || top > V ||
        kda::logprob_groups(R, V) > kda::max_groups(256))
        return (size_t)-1;
    return kda::logprob_workspace(R, V, top);
}

int kda_token_logprobs(const void* logits, int64_t row_stride, const int32_t* tokens, int64_t R, int32_t V,
                       int32_t top, int32_t dtype, float* logprobs, float* lse, float* entropy, float* top_logprobs,
                       int32_t* top_tokens, void* workspace, size_t workspace_bytes, void* hip_stream) {
    static const char* name = "kda_token_logprobs";
    if (int rc = check_logits(name, logits, row_stride, R, V, dtype)) return rc;
    if (top < 0 || top > 64 || top > V) return fail(KDA_ERR_INVALID_ARG, "%s: top=%d, expected 0 .. 64 and at most V", name, top);
    if (int rc = check_groups(name, kda::logprob_groups(R, V))) return rc;
    if (R > 0 && (!logprobs != !tokens)) return fail(KDA_ERR_INVALID_ARG, "%s: tokens and logprobs go together", name);
    if (R > 0 && ((top == 0) != !top_logprobs || (top == 0) != !top_tokens))
        return fail(KDA_ERR_INVALID_ARG, "%s: top, top_logprobs and top_tokens go together", name);
    if (!aligned_to(tokens, 4) || !aligned_to(logprobs, 4) || !aligned_to(lse, 4) || !aligned_to(entropy, 4) ||
        !aligned_to(top_logprobs, 4) || !aligned_to(top_tokens, 4))
        return fail(KDA_ERR_MISALIGNED, "%s: tokens and outputs must be 4-byte aligned", name);
    const size_t need = kda::logprob_workspace(R, V, top);
    if (int rc = check_workspace(name, workspace, workspace_bytes, need)) return rc;
    const int64_t es = dtype == KDA_BF16 ? 2 : 4;
    const size_t n = (size_t)R * 4;
    const Span ins[] = {logit_span(logits, row_stride, R, V, es), {tokens, n}};
    const Span outs[] = {{logprobs, n}, {lse, n}, {entropy, n}, {top_logprobs, n * top}, {top_tokens, n * top},
                         {workspace, need}};
    if (int rc = check_alias(name, outs, ins)) return rc;
    if (injected_launch_failure()) return injected(name);
    kda::LogprobArgs a{};
    a.logits = logits; a.row_stride = row_stride; a.tokens = tokens; a.R = R; a.V = V; a.top = top;
    a.bf16 = dtype == KDA_BF16;
    a.logprobs = logprobs; a.lse = lse; a.entropy = entropy; a.top_logprobs = top_logprobs; a.top_tokens = top_tokens;
    a.ws = workspace;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    return check_hip(kda::launch_logprobs(a, s), s, name);
}

int kda_token_logprobs_grad(const void* logits, int64_t row_stride, const int32_t* tokens, const float* lse,
                            const float* entropy, const float* d_logprobs, const float* d_lse, const float* d_entropy,
                            int64_t R, int32_t V, int32_t dtype, void* d_logits, int64_t out_stride,
                            void* hip_stream) {
    static const char* name = "kda_token_logprobs_grad";
    if (int rc = check_logits(name, logits, row_stride, R, V, dtype)) return rc;
    if (int rc = check_logits(name, d_logits, out_stride, R, V, dtype)) return rc;
    if (int rc = check_groups(name, kda::logprob_grad_groups(R, V))) return rc;
    if (R > 0 && !lse) return fail(KDA_ERR_INVALID_ARG, "%s: lse is required", name);
    if (R > 0 && d_logprobs && !tokens) return fail(KDA_ERR_INVALID_ARG, "%s: d_logprobs needs tokens", name);
    if (R > 0 && d_entropy && !entropy) return fail(KDA_ERR_INVALID_ARG, "%s: d_entropy needs entropy", name);
    if (!aligned_to(tokens, 4) || !aligned_to(lse, 4) || !aligned_to(entropy, 4) || !aligned_to(d_logprobs, 4) ||
        !aligned_to(d_lse, 4) || !aligned_to(d_entropy, 4))
        return fail(KDA_ERR_MISALIGNED, "%s: the rows' values must be 4-byte aligned", name);
    const int64_t es = dtype == KDA_BF16 ? 2 : 4;
    const Pool x = rows_of(logits, row_stride * es, V * es, R), y = rows_of(d_logits, out_stride * es, V * es, R);
    const size_t n = (size_t)R * 4;
    const Span ins[] = {{tokens, n}, {lse, n}, {entropy, n}, {d_logprobs, n}, {d_lse, n}, {d_entropy, n}};
    if (!same(x, y) && overlap(x, y))
        return fail(KDA_ERR_ALIAS, "%s: d_logits overlaps logits and is not the same", name);
    for (const Span& in : ins)
        if (overlap(y.span(), in)) return fail(KDA_ERR_ALIAS, "%s: d_logits overlaps an input", name);
    if (injected_launch_failure()) return injected(name);
    kda::LogprobGradArgs a{};
    a.logits = logits; a.row_stride = row_stride; a.tokens = tokens; a.lse = lse; a.entropy = entropy;
    a.d_logprobs = d_logprobs; a.d_lse = d_lse; a.d_entropy = d_entropy; a.R = R; a.V = V;
    a.bf16 = dtype == KDA_BF16; a.d_logits = d_logits; a.out_stride = out_stride;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    return check_hip(kda::launch_logprob_grad(a, s), s, name);
}

}  // extern "C"
