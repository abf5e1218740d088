// Host-side helpers every entry point uses: the thread's error message, the
// overlap check of a call's buffers, and launches under the profiling hook.
// Defined in api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <vector>

namespace muon {

// Sets the message of muon_last_error() on this thread and returns `code`.
int fail(int code, const char* fmt, ...);

// Byte span of one buffer of a call; `tensor` names it in messages.
struct Span {
    uintptr_t lo, hi;
    int tensor;
};
int check_overlaps(std::vector<Span>& spans, const char* what);

// Streaming tensors (EMA, AdamW): at most 2^30 workgroups per launch, so a
// single tensor may hold at most this many elements (4 Ti elements; far above
// any device memory).
constexpr int64_t kMaxStreamElems = ((int64_t)1 << 30) * 1024;

// Profiling hook: whether launches are timed; an event pair for one launch
// (hipErrorOutOfMemory if none could be made); the pair handed back after both
// events were recorded.
bool profiling();
hipError_t profile_events(hipEvent_t& start, hipEvent_t& stop);
void profile_done(const char* name, hipEvent_t start, hipEvent_t stop);

// Runs `launch` (which returns the launch's hipError_t) bracketed by events
// when profiling is on.
template <typename F>
hipError_t timed_launch(const char* name, hipStream_t s, F launch) {
    if (!profiling()) return launch();
    hipEvent_t e0, e1;
    hipError_t err = profile_events(e0, e1);
    if (err == hipSuccess) err = hipEventRecord(e0, s);
    if (err == hipSuccess) err = launch();
    if (err == hipSuccess) err = hipEventRecord(e1, s);
    if (err == hipSuccess) profile_done(name, e0, e1);
    return err;
}

}  // namespace muon
