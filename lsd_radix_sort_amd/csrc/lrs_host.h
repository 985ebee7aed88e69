// lrs_host.h -- what every C entry point shares on the host (internal header):
// the caller's timer, the per-call context made from lrs_options, the pointer
// checks and the timed launch.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <vector>

#include "../../include/lsd_radix_sort.h"
#include "lrs_dispatch.h"

// A caller's kernel timer: start/stop event pairs and the kind of each launch.
struct lrs_timer {
    std::vector<hipEvent_t> pool;  // pairs: start, stop
    std::vector<int> kind;
    size_t used = 0;
    // tile phase records (builds with LRS_TILE_TRACE): the caller's device
    // buffer, its size and the words handed out so far
    uint64_t *trace = nullptr;
    uint64_t trace_words = 0;
    uint64_t trace_used = 0;
};

namespace lrs {

// Calls over at most this many elements are paced by the host: their timed
// launches are bracketed by recorded events (see TimedLaunch).
#ifndef LRS_HOST_PACED_MAX
#define LRS_HOST_PACED_MAX 65536
#endif
constexpr uint64_t kHostPacedMax = LRS_HOST_PACED_MAX;
constexpr size_t kMaxTimed = 65536;

// Polls of an unpublished look-back word before a tile counts its prefix from
// the keys (about 1 us each, so the default is tens of milliseconds: far beyond
// any wait of a running sort, and only a guarantee against waiting forever).
constexpr uint32_t kDefaultSpinLimit = LRS_DEFAULT_SPIN_LIMIT;

// Everything one call needs besides its arguments: the stream and the
// caller's options.  Nothing is kept between calls.
struct Ctx {
    hipStream_t s = nullptr;
    lrs_timer *timer = nullptr;
    uint32_t spin_limit = kDefaultSpinLimit;  // 0: every tile counts its prefix from the keys
    int scan = LRS_SCAN_LOOKBACK;
    uint64_t wide_from = 0;
    uint64_t elems = ~uint64_t(0);  // elements the call handles (sets how a timer times it)
};

// False for an invalid option.
inline bool make_ctx(void *stream, const lrs_options *o, Ctx &c) {
    c.s = static_cast<hipStream_t>(stream);
    if (o == nullptr) return true;
    if (o->scan_strategy != LRS_SCAN_LOOKBACK && o->scan_strategy != LRS_SCAN_REDUCE_THEN_SCAN) return false;
    c.scan = o->scan_strategy;
    c.timer = o->timer;
    // Timer events are for calls run eagerly: a timed call on a stream being
    // captured into a graph is refused before anything is enqueued.
    if (c.timer != nullptr && c.s != nullptr) {
        hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
        if (hipStreamIsCapturing(c.s, &st) != hipSuccess || st != hipStreamCaptureStatusNone) return false;
    }
    if (o->spin_limit != 0) c.spin_limit = o->spin_limit;
    if (o->prefix_from_keys) c.spin_limit = 0;
    c.wide_from = o->wide_from;
    return true;
}

inline uint64_t wide_from_of(const lrs_options *o) { return o ? o->wide_from : 0; }
inline bool options_ok(const lrs_options *o) {
    Ctx c;
    return make_ctx(nullptr, o, c);
}

inline bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

inline bool overlaps(const void *a, uint64_t na, const void *b, uint64_t nb) {
    if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// The row operators' matrices: element types, strides in elements (0: every
// row the same), and the bytes from the first element to past the last.
inline bool row_type_ok(int dtype) {
    return dtype == LRS_DTYPE_FP16 || dtype == LRS_DTYPE_BF16 || dtype == LRS_DTYPE_FP32;
}
inline uint64_t row_type_size(int dtype) { return dtype == LRS_DTYPE_FP32 ? 4 : 2; }
inline bool stride_ok(int64_t stride, int64_t rows) {
    return stride >= 0 &&
           (stride == 0 || static_cast<uint64_t>(rows) < (uint64_t(1) << 48) / static_cast<uint64_t>(stride));
}
inline uint64_t span(uint64_t rows, uint64_t stride, uint64_t n, uint64_t size) {
    return rows == 0 || n == 0 ? 0 : ((rows - 1) * stride + n) * size;
}

// One launch, timed into a timer slot when the call has a timer.  For calls
// over many elements the dispatch itself stamps the slot's events, so nothing
// is enqueued between dependent kernels.  Calls over at most kHostPacedMax
// elements, whose launches the host rather than the GPU paces, bracket each
// launch with recorded events instead, which cost the host less per launch;
// the closing event is recorded when the TimedLaunch goes out of scope, so
// its scope must end right after the launch.
struct TimedLaunch {
    Launch L;  // the stream, and the slot's events when the dispatch stamps them
    hipEvent_t after = nullptr;  // bracketing: recorded by done() or on scope exit
    TimedLaunch(const TimedLaunch &) = delete;
    TimedLaunch &operator=(const TimedLaunch &) = delete;
    explicit TimedLaunch(int kind, const Ctx &c) {
        L.s = c.s;
        lrs_timer *t = c.timer;
        if (t == nullptr || t->used >= kMaxTimed) return;
        const bool bracket = c.elems <= kHostPacedMax;
        const size_t i = t->used;
        if (t->pool.size() < 2 * (i + 1)) {
            // The events only time: without the system-scope fence a recorded
            // event would otherwise add (a cache write-back and invalidation).
            hipEvent_t a, b;
            if (hipEventCreateWithFlags(&a, hipEventDisableSystemFence) != hipSuccess) return;
            if (hipEventCreateWithFlags(&b, hipEventDisableSystemFence) != hipSuccess) {
                (void)hipEventDestroy(a);
                return;
            }
            t->pool.push_back(a);
            t->pool.push_back(b);
        }
        if (bracket) {
            if (hipEventRecord(t->pool[2 * i], c.s) != hipSuccess) return;
            after = t->pool[2 * i + 1];
        } else {
            L.start = t->pool[2 * i];
            L.stop = t->pool[2 * i + 1];
        }
        t->kind.resize(i + 1);
        t->kind[i] = kind;
        t->used = i + 1;
    }
    void done() {
        if (after != nullptr) (void)hipEventRecord(after, L.s);
        after = nullptr;
    }
    ~TimedLaunch() { done(); }
};

}  // namespace lrs
