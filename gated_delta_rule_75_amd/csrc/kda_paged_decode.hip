// Softmax attention of one new token per sequence over a paged key-value cache (include/kda.h,
// kda_paged_decode):
//     s_t = scale q . k_t,   out = sum_t exp(s_t - m) v_t / l,   l = sum_t exp(s_t - m),
//     lse = m + log l,       m = max_t s_t
// over the visible tokens: all of them, or with a window the last ones and the first `sinks`.
#include <math.h>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

// Visible tokens of a sequence of `len` tokens: 0 .. head-1 and near .. len-1 (head <= near).
struct Visible {
    int64_t head, near, len;
};
__device__ __forceinline__ Visible visible(const PagedDecodeArgs& a, int64_t n) {
    Visible v;
    int64_t len = a.lengths[n];
    len = len < 0 ? 0 : len > a.max_length ? a.max_length : len;
    v.len = len;
    v.near = a.window > 0 && len > a.window ? len - a.window : 0;
    v.head = a.sinks < v.near ? a.sinks : v.near;
    return v;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void paged_decode_kernel(PagedDecodeArgs a) {
    __shared__ float s_q[256], s_p[kThreads], s_red[kThreads / 64];
    __shared__ int64_t s_v[kThreads];
    const int64_t n = blockIdx.x / a.Hq;
    const int hq = blockIdx.x % a.Hq, h = hq / (a.Hq / a.Hkv);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid < a.d) s_q[tid] = ld_in(static_cast<const T*>(a.q), n * a.q_stride + (int64_t)hq * a.d + tid);
    const Visible vis = visible(a, n);
    const int64_t count = vis.head + vis.len - vis.near;
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int64_t i0 = 0; i0 < count; i0 += kThreads) {
        __syncthreads();
        float s = -INFINITY;
        int64_t vo = -1;
        if (i0 + tid < count) {
            const int64_t i = i0 + tid, t = i < vis.head ? i : vis.near + i - vis.head, col = t / a.page_size;
            const int32_t p = a.pt.table[n * a.pt.stride + col];
            if (p >= 0 && p < a.pt.n_pages) {
                const int64_t slot = ((int64_t)h * a.page_size + (t - col * a.page_size)) * a.d;
                const T* k = static_cast<const T*>(a.kp) + p * a.kp_stride + slot;
                vo = p * a.vp_stride + slot;
                s = 0.f;
                for (int c = 0; c < a.d; ++c) s += s_q[c] * ld_in(k, c);
                s *= a.scale;
            }
        }
        float top = s;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
        if (lane == 0) s_red[wave] = top;
        __syncthreads();
        float now = m;
        for (int w = 0; w < kThreads / 64; ++w) now = fmaxf(now, s_red[w]);
        const float base = now == -INFINITY ? 0.f : now, keep = expf(m - base);
        s_p[tid] = vo < 0 ? 0.f : expf(s - base);
        s_v[tid] = vo;
        __syncthreads();
        l *= keep;
        acc *= keep;
        m = now;
        for (int j = 0; j < kThreads; ++j) {
            if (s_v[j] < 0) continue;
            l += s_p[j];
            if (tid < a.d) acc += s_p[j] * ld_in(static_cast<const T*>(a.vp), s_v[j] + tid);
        }
    }
    if (tid < a.d) a.o[(n * a.Hq + hq) * a.d + tid] = l == 0.f ? 0.f : acc / l;
    if (a.lse && tid == 0) a.lse[n * a.Hq + hq] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

bool paged_decode_supported(int d) { return d == 64 || d == 128 || d == 256; }

size_t paged_decode_workspace(int64_t N, int Hq, int Hkv, int d, int bf16, int64_t max_length, int window, int sinks) {
    return 0;
}

hipError_t launch_paged_decode(const PagedDecodeArgs& a, hipStream_t s) {
    if (a.N == 0) return hipSuccess;
    const bool timed = timing_on();
    if (timed) timed_begin(kKernelPagedDecode, s);
    const dim3 grid((unsigned)(a.N * a.Hq));
    if (a.bf16) hipLaunchKernelGGL(paged_decode_kernel<uint16_t>, grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL(paged_decode_kernel<float>, grid, dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (timed) timed_end(s);
    return e;
}

}  // namespace kda
