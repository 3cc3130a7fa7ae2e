// Helpers shared by the C-ABI translation units (kda_api.cpp, kda_serving_api.cpp): the calling
// thread's error message, argument checks and the debug copies of device-resident data.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <vector>

#include "kda.h"

namespace kda {
namespace api {

// Sets the calling thread's message and returns `status`.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the message; KDA_OK.
int ok();
bool env_flag(const char* name);

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned_to(p, 16); }

struct Span {
    const void* p;
    size_t bytes;
};

inline bool overlap(Span a, Span b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Status of a launch (KDA_DEBUG_SYNC=1 also waits for the stream).
int check_hip(hipError_t e, hipStream_t s, const char* what);
// Host-side stand-in for a launch failure, for tests of the error path only.
inline bool injected_launch_failure() { return env_flag("KDA_TEST_FAIL_LAUNCH"); }
inline bool debug_check() { return env_flag("KDA_DEBUG_CHECK"); }

// Copies `count` values of device memory to the host once the stream has drained (debug check).
template <typename T>
int fetch(const void* dev, size_t count, hipStream_t s, std::vector<T>& out, const char* name) {
    try {
        out.resize(count);
    } catch (...) {  // no exception may leave a C entry point
        return fail(KDA_ERR_HIP, "%s (debug check): no host memory for %zu values", name, count);
    }
    if (!count) return KDA_OK;
    hipError_t e = hipStreamSynchronize(s);
    if (e == hipSuccess) e = hipMemcpy(out.data(), dev, count * sizeof(T), hipMemcpyDeviceToHost);
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "%s (debug check): %s", name, hipGetErrorString(e));
    return KDA_OK;
}

inline bool valid_dtype(int32_t d) { return d == KDA_F32 || d == KDA_BF16; }

}  // namespace api
}  // namespace kda
