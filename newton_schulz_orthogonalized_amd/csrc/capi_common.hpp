// Host helpers shared by the sources of the C ABI (defined in capi.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <exception>
#include <functional>
#include <vector>

namespace mu {

// Set the calling thread's error text and return the status.
int fail(int code, const char* fmt, ...);
int hip_fail(hipError_t e, const char* what);
void clear_error();

constexpr size_t ALIGN = 256;   // of workspaces
inline size_t align_up(size_t x, size_t a = ALIGN) { return (x + a - 1) / a * a; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Buffer overlap check over all device ranges of one call.
struct Range {
    uintptr_t lo, hi;
    int owner;
};
bool ranges_overlap(std::vector<Range>& r);

// fn() enqueues one launch on s; with profiling on (and s not capturing) it is
// timed under kernel class `kernel`.
int timed_launch(int kernel, double flops, double bytes, hipStream_t s, const std::function<hipError_t()>& fn,
                 const char* what);

// Compute units of the current device (asked once per device).
int cu_count(int* out);

// The body of a C entry point: no C++ exception (an allocation that failed)
// leaves it.
template <typename F>
int guarded(F&& body) {
    try {
        clear_error();
        return body();
    } catch (const std::exception& e) {
        return fail(5, "host allocation failed: %s", e.what());
    } catch (...) {
        return fail(5, "unknown host error");
    }
}

}  // namespace mu
