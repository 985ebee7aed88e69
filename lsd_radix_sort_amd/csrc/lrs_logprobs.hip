// lrs_logprobs.hip -- log probabilities of given tokens, with the rows'
// entropy, the tokens' ranks, top alternatives and the gradient (gfx950).
//
// With d_j = (x_j - m) log2(e) / T for a row of logits x and its largest m,
// Z = sum 2^d_j and D = (sum 2^d_j d_j) / Z:
//   log p_j = ln2 (d_j - log2 Z),   entropy = ln2 (log2 Z - D),
//   grad_j = (a [j = t] - 2^d_j / Z (a + b ln2 (d_j - D))) / T.
// One pass gives m, Z and the sum behind D: each thread's sums are relative to
// the largest logit that it has met, and are scaled when it meets a larger one.
// A difference x - m is exact or rounded by its own last bit, so however large
// the logits are, exponents near 0 are right.
//
// A thread's terms are summed in 32 bits within one batch of loads.  Its batches
// are added in 64 bits where a row may have any number of them (forward, ranks
// alone), in 32 where it has at most 16 (a row whose alternatives are selected, a
// row that the step holds); what there is once a row, from the threads' sums on,
// is in 64 bits: an entropy is the difference of two numbers that nearly cancel.
// So the calls can differ in their last bits over the same row.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>

#include "../../include/lsd_radix_sort.h"
#include "lrs_host.h"
#include "lrs_rows.h"
#include "lrs_select.h"

namespace lrs {
namespace {

constexpr int kLogBlock = 256;
constexpr int kLoads = 4;              // of a batch
constexpr int kKept = 16;              // batches whose largest elements are kept
constexpr uint32_t kPickWords = 512;   // candidates in LDS, by fewer threads than that
constexpr uint32_t kJoinWords = 1024;  // of a row's pieces
constexpr double kLog2e = 1.44269504088896340736;
constexpr double kLn2 = 0.693147180559945309417;
constexpr uint32_t kLogStats = 3;
constexpr float kLowest = std::numeric_limits<float>::lowest();

// Of a piece of a row: its largest logit, the sums of 2^d and of 2^d d relative
// to that, and how many of its elements come before the token in the row sort.
struct Sums {
    double z, w;
    float m;
    uint32_t before;
};

struct LogArgs {
    const void *logits;
    uint64_t stride;
    uint64_t rows;
    uint32_t n;
    const void *tokens;
    uint64_t token_stride;
    int token_bytes;
    const uint8_t *mask;
    float c;              // log2(e) / T
    double factor;        // the same in 64 bits
    // 1 / T in two factors, of derivatives and of shares: either of them alone can leave the range of 32 bits
    float soft;           // at most 1, times a power of two
    int soft_power;
    float sharp;          // at least 1
    uint32_t splits, split_len;
    Sums *sums;           // [rows][splits]
    float *logprobs, *entropy, *stats;
    int32_t *ranks;
    const float *up, *up_entropy;
    void *grad;
    uint64_t grad_stride;
    uint32_t k;
    const void *top_values;  // patterns of the top k
    float *top_logprobs;
    double *lows;         // [rows]: log2 Z
    int64_t *top_indices;
    uint64_t *words;      // [rows][splits][k]
    uint64_t first_task;  // of this launch
};

__device__ inline int64_t token_of(const LogArgs &a, uint64_t row) {
    const uint64_t at = row * a.token_stride;
    return a.token_bytes == 8 ? static_cast<const int64_t *>(a.tokens)[at] : static_cast<const int32_t *>(a.tokens)[at];
}
__device__ inline float softened(const LogArgs &a, float derivative) { return __builtin_amdgcn_ldexpf(derivative * a.soft, a.soft_power); }
__device__ inline bool counted(const LogArgs &a, uint64_t row) { return a.mask == nullptr || a.mask[row] != 0; }

// The larger of two, NaN if either is.
__device__ inline float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Exponents below this give 2^d = 0 in 32 bits; cut off there, 2^d d is 0 for
// d = -inf too.
constexpr float kZeroBelow = -150.f;

// Sums relative to m, moved to a larger one.
__device__ inline void rebase(double &z, double &w, float m, float to, float c) {
    const float d = fmaxf((m - to) * c, kZeroBelow);
    const float s = __builtin_amdgcn_exp2f(d);
    w = s * fma(z, static_cast<double>(d), w);
    z = s * z;
}

// log2 of a positive number: the hardware's of 32 bits, and the rest from
// log(1 + e) = e - e^2 / 2 at e = v 2^-that - 1, below 2^-20.
__device__ inline double log2_64(double v) {
    int power;
    const double f = frexp(v, &power);
    const double y = __builtin_amdgcn_logf(static_cast<float>(f));
    const double e = f * exp2(-y) - 1.0;
    return v > 0 && v < INFINITY ? power + (y + fma(e * e, -0.5, e) * (1.0 / kLn2)) : log2(v);
}

// The row order of a 32-bit pattern as a signed number.
__device__ inline int image_of_bits(uint32_t bits) {
    const int v = static_cast<int>(bits);
    return v ^ ((v >> 31) & 0x7FFFFFFF);
}
// The pattern of an element, in the high bits where it has 16.
template <int T> __device__ inline uint32_t high_bits(typename Row<T>::Stored v) {
    return T == kRowF32 ? v : static_cast<uint32_t>(v) << 16;
}

// What a row's sums say, by one thread: its numbers, and log2 Z for the top k.
struct RowEnd {
    double mean;   // D
    double share;  // 1 / Z, 0 where the row counts for nothing
};
// log2 Z, infinity where the row is all -inf: log p is -inf there
__device__ inline double low_of(double z) { return z == 0 ? INFINITY : log2_64(z); }
__device__ inline RowEnd finish_row(const LogArgs &a, uint64_t row, bool on, bool given, float x, double z, double w, float m,
                                    uint32_t before) {
    const bool empty = z == 0;
    const double low = low_of(z), mean = w / z;
    double logprob = 0, entropy = 0;
    if (on) {
        entropy = empty ? 0 : kLn2 * (low - mean);
        if (given) logprob = empty ? -INFINITY : kLn2 * ((static_cast<double>(x) - m) * a.factor - low);
    }
    a.logprobs[row] = static_cast<float>(logprob);
    a.entropy[row] = static_cast<float>(entropy);
    if (a.ranks) a.ranks[row] = given ? static_cast<int32_t>(before) : -1;
    const RowEnd end{!on || empty ? 0 : mean, !on || empty ? 0 : 1 / z};
    if (a.stats) {
        float *s = a.stats + row * kLogStats;
        s[0] = m;
        s[1] = static_cast<float>(end.share);
        s[2] = static_cast<float>(end.mean);
    }
    if (a.lows) a.lows[row] = low;
    return end;
}
// log p of a logit.
__device__ inline float logprob_of(const LogArgs &a, float x, float m, double low) {
    return static_cast<float>(kLn2 * ((static_cast<double>(x) - m) * a.factor - low));
}

template <int T> __device__ inline void put_top(const LogArgs &a, uint64_t word, uint64_t at, float m, double low) {
    const uint32_t p = pattern_of<T == kRowF32 ? 4 : 2>(image_of(word), 0);
    a.top_logprobs[at] = logprob_of(a, Row<T>::value(static_cast<typename Row<T>::Stored>(p)), m, low);
    a.top_indices[at] = column_of(word);
}

// A thread's sums of 2^(x c - r), r its largest logit times c, over batches of
// loads.  r is a number of 32 bits, and a product less r is rounded once, so that
// sums of different references join exactly, whatever the rounding of r.  Past
// 2^29 that rounding could be more than a power holds: rows with such a largest
// logit (masks of the type's lowest value that fill a row) are summed anew.
constexpr float kLeastReference = -0x1p30f;
constexpr float kHugeReference = 0x1p29f;
template <typename Acc> struct Running {
    Acc z = 0, w = 0;
    float top = -INFINITY, r = kLeastReference;
    __device__ void move(float to) {
        const float d = fmaxf(r - to, kZeroBelow), s = __builtin_amdgcn_exp2f(d);
        w = s * (w + z * static_cast<Acc>(d));
        z = s * z;
        r = to;
    }
    // elements of which `most` is the largest
    template <int N> __device__ void add(const float (&f)[N], float most, float c) {
        top = larger(top, most);
        move(fmaxf(top * c, kLeastReference));
        float part = 0, part_w = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float d = fmaf(f[e], c, -r), p = __builtin_amdgcn_exp2f(d);
            part += p;
            part_w = fmaf(p, fmaxf(d, kZeroBelow), part_w);
        }
        z += part;
        w += part_w;
    }
};
__device__ inline bool huge(float top, float c) { return fabsf(top) < INFINITY && !(fabsf(top * c) < kHugeReference); }

template <int N> __device__ inline float largest(const float (&f)[N]) {
    float m = f[0];
#pragma unroll
    for (int e = 1; e + 1 < N; e += 2) m = larger(larger(m, f[e]), f[e + 1]);
    return N % 2 == 0 ? larger(m, f[N - 1]) : m;
}

template <int B> struct JoinLds {
    double z[B / kLanes], w[B / kLanes];
    float top[B / kLanes];
    uint32_t before[B / kLanes];
};
// The workgroup's sums relative to its largest logit, in its first thread;
// anew(m) gives a thread's sums relative to a huge m.
template <int B, typename Acc, typename Anew>
__device__ inline Sums join_sums(JoinLds<B> &lds, Running<Acc> &mine, float &top, uint32_t before, float c, Anew anew) {
    constexpr int kWaves = B / kLanes;
    const int wave = threadIdx.x / kLanes;
    top = wave_join(mine.top, -INFINITY, [](float p, float q) { return larger(p, q); });
    if (kWaves > 1) {
        if (threadIdx.x % kLanes == 0) lds.top[wave] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWaves; ++i) top = larger(top, lds.top[i]);
    }
    Sums s{};
    s.m = top == -INFINITY ? kLowest : top;
    float shift = 0;
    if (huge(top, c)) {
        const double2 sum = anew(top);
        s.z = sum.x;
        s.w = sum.y;
    } else {
        const float r = fmaxf(top * c, kLeastReference);
        mine.move(r);
        s.z = mine.z;
        s.w = mine.w;
        shift = static_cast<float>(static_cast<double>(top) * c - r);  // of exponents, to be relative to top itself
    }
    s.z = wave_sum(s.z);
    s.w = wave_sum(s.w);
    s.before = wave_sum(before);
    if (kWaves > 1) {
        if (threadIdx.x % kLanes == 0) {
            lds.z[wave] = s.z;
            lds.w[wave] = s.w;
            lds.before[wave] = s.before;
        }
        __syncthreads();
        if (threadIdx.x == 0)
            for (int i = 1; i < kWaves; ++i) {
                s.z += lds.z[i];
                s.w += lds.w[i];
                s.before += lds.before[i];
            }
    }
    if (fabsf(shift) < INFINITY && shift != 0) {
        // Over the very power that the largest logit's own term is, to 2^-46 by one step of Newton's method from the
        // opposite power (that alone left log p of up to 9e-8 above 0).  The term itself is 1 and every exponent at
        // most 0: what rounding left beyond is cut off, so that log p <= 0 and the entropy >= 0.  NaN stays.
        const double p = __builtin_amdgcn_exp2f(shift), q = __builtin_amdgcn_exp2f(-shift), inverse = q * fma(-p, q, 2.0);
        s.w = (s.w - s.z * shift) * inverse;
        s.z = s.z * inverse;
        s.w = s.w > 0 ? 0 : s.w;
        s.z = s.z < 1 ? 1 : s.z;
    }
    return s;
}

// What a row, or a piece of one, holds of the row order around its token.
template <int T> struct Token {
    using Stored = typename Row<T>::Stored;
    int64_t at;
    bool given, exact;   // exact: its order takes the patterns
    float x, from, least;  // its logit; what later columns are above, and earlier ones
    Stored pattern;
    __device__ Token(const LogArgs &a, uint64_t row) {
        at = token_of(a, row);
        given = at >= 0 && at < a.n;
        pattern = given ? static_cast<const Stored *>(a.logits)[row * a.stride + at] : 0;
        x = Row<T>::value(pattern);
        // a number of 32 bits is at least x where it is above the one before x
        const uint32_t bits = __builtin_bit_cast(uint32_t, x);
        from = x;
        least = __builtin_bit_cast(float, x > 0 ? bits - 1 : bits + 1);
        exact = given && !(fabsf(x) > 0 && x > -INFINITY);
    }
    // Whether an element comes before it.
    __device__ bool after(Stored v, uint32_t column) const {
        const int i = image_of_bits(high_bits<T>(v)), mine = image_of_bits(high_bits<T>(pattern));
        return i > mine || (i == mine && column < at);
    }
};

// One workgroup of B threads a row, or a piece of one.  PICK: at most kKept
// batches of loads a thread, whose largest elements are kept in LDS; the
// alternatives are selected from them as segmented_row_topk does, and batches
// that reach the bound are read again.  Else a row may have any length.
// ONCE: the logits are read past the caches (see read_once).
// Bound by HBM where rows fill the GPU (4096 x 131072 bf16 170 us = 6.3 TB/s, ranks 188,
// 8 alternatives 206: the chain after a row's last load), by the chain of load, sums,
// bound and ranking where they do not (8 us of one row shared by 16).
template <int T, int B, bool RANK, bool PICK, bool ONCE>
__global__ __launch_bounds__(B, B == 1024 ? 4 : B == 64 && PICK ? 3 : T == kRowF32 && PICK ? 5 : 7) void logprob_kernel(LogArgs a) {
    constexpr int kVec = Row<T>::kVec, kWidth = T == kRowF32 ? 4 : 2;
    using Stored = typename Row<T>::Stored;
    __shared__ JoinLds<B> join;
    __shared__ SelectLds<B, PICK && B < kPickWords ? kPickWords : B> lds;
    __shared__ Stored kept[PICK ? kKept : 1][B];
    __shared__ double whole;
    const uint32_t tid = threadIdx.x;
    const uint64_t task = a.first_task + xcd_chunk(blockIdx.x, gridDim.x);
    const uint64_t row = task / a.splits;
    const uint32_t first = static_cast<uint32_t>(task % a.splits) * a.split_len;
    const bool on = counted(a, row);
    const uint32_t len = on ? min(a.n - first, a.split_len) : 0, vecs = len / kVec, rest = vecs * kVec + tid;
    const Stored *x = static_cast<const Stored *>(a.logits) + row * a.stride + first;
    const uint32_t none = T == kRowF16 ? 0xFC00FC00u : T == kRowBF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
    const auto load = [&](uint32_t v) {
        u32x4 t{none, none, none, none};
        if (v < vecs) t = ONCE ? load16_once(x + static_cast<uint64_t>(v) * kVec) : load16(x + static_cast<uint64_t>(v) * kVec);
        return t;
    };
    const Token<T> token(a, row);
    const bool ranked = RANK && token.given && !token.exact;
    const float c = a.c;
    uint32_t before = 0;  // of this thread
    Running<std::conditional_t<PICK, float, double>> mine;
    // N loads of a thread, from load `v` on
    const auto take = [&](auto loads, const u32x4 *t, uint32_t v) {
        constexpr int N = decltype(loads)::value;
        float f[N * kVec], top[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            float g[kVec];
            unpack16<T>(t[u], g);
            top[u] = largest(g);
#pragma unroll
            for (int e = 0; e < kVec; ++e) f[u * kVec + e] = g[e];
        }
        const float all = largest(top);
        if (RANK && ranked && __ballot(!(all < token.x))) {
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int64_t last = static_cast<int64_t>(first) + static_cast<int64_t>(v + u * B + 1) * kVec;
                const float bound = last <= token.at ? token.least : token.from;
#pragma unroll
                for (int e = 0; e < kVec; ++e) before += f[u * kVec + e] > bound;
            }
        }
        mine.add(f, all, c);
        return all;
    };
    // whole batches, the next one's loads on their way; then the loads that are left, one at a time
    const uint32_t whole_batches = vecs / (kLoads * B);
    u32x4 t[kLoads], next[kLoads];
    if (whole_batches > 0) {
#pragma unroll
        for (int u = 0; u < kLoads; ++u) next[u] = load(u * B + tid);
    }
#pragma unroll 1
    for (uint32_t b = 0; b < whole_batches; ++b) {
#pragma unroll
        for (int u = 0; u < kLoads; ++u) t[u] = next[u];
        if (b + 1 < whole_batches) {
#pragma unroll
            for (int u = 0; u < kLoads; ++u) next[u] = load(((b + 1) * kLoads + u) * B + tid);
        }
        const float all = take(std::integral_constant<int, kLoads>(), t, b * kLoads * B + tid);
        if (PICK) kept[b][tid] = Row<T>::pattern(all);
    }
    if (whole_batches * kLoads * B < vecs) {
        float all = -INFINITY;
#pragma unroll 1
        for (uint32_t v = whole_batches * kLoads * B + tid; v - tid < vecs; v += B) {
            t[0] = load(v);
            all = larger(all, take(std::integral_constant<int, 1>(), t, v));
        }
        if (PICK) kept[whole_batches][tid] = Row<T>::pattern(all);
    }
    const bool extra = rest < len;
    if (len > vecs * kVec) {  // the elements after the last whole load
        const Stored v = extra ? x[rest] : Stored(0);
        const float f[1] = {extra ? Row<T>::value(v) : -INFINITY};
        if (RANK && ranked) before += extra && token.after(v, first + rest);
        mine.add(f, f[0], c);
    }
    if (RANK && token.given) {
        const int64_t at = token.at - first;
        if (token.exact || __ballot(__builtin_isnan(mine.top))) {  // by their patterns, from a second read
            before = extra && token.after(x[rest], first + rest);
            for (uint32_t v = tid; v < vecs; v += B)
                for (int e = 0; e < kVec; ++e) before += token.after(x[static_cast<uint64_t>(v) * kVec + e], first + v * kVec + e);
        } else if (at >= 0 && at < static_cast<int64_t>(vecs) * kVec && at / kVec % B == tid) {
            // equal ones of the token's own load, before it: the thread that has that
            for (int64_t i = at - at % kVec; i < at; ++i) before += x[i] == token.pattern;
        }
    }
    float top;  // of the workgroup
    const Sums s = join_sums<B>(join, mine, top, before, c, [&](float m) {
        double z = 0, w = 0;
        const auto add = [&](float f) {
            const float d = (f - m) * c, p = __builtin_amdgcn_exp2f(d);
            z += p;
            w += p * fmaxf(d, kZeroBelow);
        };
        for (uint32_t v = tid; v < vecs; v += B) {
            float f[kVec];
            unpack16<T>(load(v), f);
            for (int e = 0; e < kVec; ++e) add(f[e]);
        }
        if (extra) add(Row<T>::value(x[rest]));
        return double2{z, w};
    });
    if constexpr (PICK) {
        __shared__ int tops[B / kLanes];
        const int over = extra ? image<kWidth>(x[rest], 0) : INT32_MIN;
        const bool some = extra || tid < vecs;
        const uint32_t batches = (vecs + kLoads * B - 1) / (kLoads * B);
        int own = image<kWidth>(Row<T>::pattern(mine.top), 0), top_image = image<kWidth>(Row<T>::pattern(top), 0);
        if (__builtin_isnan(top)) {  // NaNs have an order among themselves, by their patterns
            own = over;
            for (uint32_t b = 0; b < batches; ++b) {
                int m = kWidth == 2 ? -32768 : INT32_MIN;
                for (int u = 0; u < kLoads; ++u) {
                    const uint32_t v = (b * kLoads + u) * B + tid;
                    if (v < vecs) m = max(m, vec_max<kWidth>(load(v), 0));
                }
                kept[b][tid] = static_cast<Stored>(pattern_of<kWidth>(m, 0));
                if (b * kLoads * B + tid < vecs) own = max(own, m);
            }
            top_image = wave_max_int(own);
            if (tid % kLanes == 0) tops[tid / kLanes] = top_image;
            __syncthreads();
            for (int i = 0; i < B / kLanes; ++i) top_image = max(top_image, tops[i]);
        }
        if (tid == 0) whole = s.z;
        clear_bins<B>(lds.bins);
        if (tid == 0) lds.count = 0;
        __syncthreads();
        const auto fill = [&](uint32_t shift) {
            if (some) add_to_bins(lds.bins, own, top_image, shift);
        };
        const auto reach = [&](int bound, auto take) {
            if (own >= bound && some) {
                uint32_t hits = 0;  // batches that are read again: mostly one
                for (uint32_t b = 0; b < batches; ++b) hits |= static_cast<uint32_t>(image<kWidth>(kept[b][tid], 0) >= bound) << b;
                while (hits) {
                    const uint32_t v = __builtin_ctz(hits) * (kLoads * B) + tid;
                    hits &= hits - 1;
                    u32x4 t[kLoads];
#pragma unroll
                    for (int u = 0; u < kLoads; ++u)
                        if (v + u * B < vecs) t[u] = load16(x + static_cast<uint64_t>(v + u * B) * kVec);
#pragma unroll
                    for (int u = 0; u < kLoads; ++u)
                        if (v + u * B < vecs) each_image<kWidth>(t[u], 0, (v + u * B) * kVec, take);
                }
                if (extra) take(over, rest);
            }
        };
        const auto put = [&](uint64_t w, uint32_t place) {
            if (a.splits == 1) put_top<T>(a, w, row * a.k + place, s.m, low_of(whole));
            else a.words[task * a.k + place] = w;
        };
        select_largest<kWidth, B>(lds, x, len, first, 0, a.k, top_image, true, fill, reach, put);
    }
    if (tid == 0) {
        if (a.splits == 1) finish_row(a, row, on, token.given, token.x, s.z, s.w, s.m, s.before);
        else a.sums[task] = s;
    }
}

// The rows' pieces joined, a workgroup each: their sums, and of their words the
// first k: 4.5 us after a launch that left its sums in the caches.
template <int T, bool PICK>
__global__ __launch_bounds__(PICK ? kLogBlock : kLanes) void logprob_join_kernel(LogArgs a) {
    constexpr int B = PICK ? kLogBlock : kLanes, kWidth = T == kRowF32 ? 4 : 2;
    __shared__ SelectLds<B, PICK ? kJoinWords : B> lds;
    __shared__ int tops[B / kLanes];
    __shared__ double low;
    __shared__ float most;
    for (uint64_t row = a.first_task + blockIdx.x; row < a.rows; row += gridDim.x) {
        if (threadIdx.x < kLanes) {
            const Token<T> token(a, row);
            float m = kLowest;
            for (uint32_t s = threadIdx.x; s < a.splits; s += kLanes) m = larger(m, a.sums[row * a.splits + s].m);
            m = wave_join(m, kLowest, [](float p, float q) { return larger(p, q); });
            double z = 0, w = 0;
            uint32_t before = 0;
            for (uint32_t s = threadIdx.x; s < a.splits; s += kLanes) {
                Sums p = a.sums[row * a.splits + s];
                rebase(p.z, p.w, p.m, m, a.c);
                z += p.z;
                w += p.w;
                before += p.before;
            }
            z = wave_sum(z);
            w = wave_sum(w);
            before = wave_sum(before);
            if (threadIdx.x == 0) {
                finish_row(a, row, counted(a, row), token.given, token.x, z, w, m, before);
                low = low_of(z);
                most = m;
            }
        }
        if constexpr (PICK)
            merge_words<kWidth, B>(lds, tops, a.words + row * a.splits * a.k, a.splits * a.k, a.k,
                                   [&](uint64_t w, uint32_t place) { put_top<T>(a, w, row * a.k + place, most, low); });
        __syncthreads();
    }
}

// The first k of a row sort, as segmented_row_topk gave them, to log probabilities.
template <int T>
__global__ __launch_bounds__(kLogBlock) void logprob_top_kernel(LogArgs a) {
    const uint64_t all = a.rows * a.k;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kLogBlock + threadIdx.x; i < all;
         i += static_cast<uint64_t>(gridDim.x) * kLogBlock) {
        const float *s = a.stats + i / a.k * kLogStats;
        const float x = Row<T>::value(static_cast<const typename Row<T>::Stored *>(a.top_values)[i]);
        a.top_logprobs[i] = logprob_of(a, x, s[0], a.lows[i / a.k]);
    }
}

// One workgroup: the gradient of a piece of a row.  Bound by HBM: 4096 x 131072
// bf16 403 us = 5.3 TB/s.
template <int T, bool ONCE>
__global__ __launch_bounds__(kLogBlock) void logprob_grad_kernel(LogArgs a) {
    constexpr int kVec = Row<T>::kVec;
    using Stored = typename Row<T>::Stored;
    const float c = a.c;
    for (uint64_t task = blockIdx.x; task < a.rows * a.splits; task += gridDim.x) {
        const uint64_t row = task / a.splits;
        const uint32_t first = static_cast<uint32_t>(task % a.splits) * a.split_len;
        const uint32_t len = min(a.n - first, a.split_len), vecs = len / kVec, rest = vecs * kVec + threadIdx.x;
        const Stored *x = static_cast<const Stored *>(a.logits) + row * a.stride + first;
        Stored *g = static_cast<Stored *>(a.grad) + row * a.grad_stride + first;
        const int64_t token = token_of(a, row);
        const bool given = token >= 0 && token < a.n;
        const float asked = a.up && given ? a.up[row] : 0.f, asked_entropy = a.up_entropy ? a.up_entropy[row] : 0.f;
        const float *s = a.stats + row * kLogStats;
        if (!counted(a, row) || s[1] == 0.f || (asked == 0.f && asked_entropy == 0.f)) {  // whatever its logits hold
            for (uint32_t v = threadIdx.x; v < vecs; v += kLogBlock) store16(g + static_cast<uint64_t>(v) * kVec, u32x4{0, 0, 0, 0});
            if (rest < len) g[rest] = 0;
            continue;
        }
        const float m = s[0], share = -s[1] * a.sharp, mean = s[2];
        const float up = softened(a, asked), slope = softened(a, asked_entropy) * static_cast<float>(kLn2);
        // p (a + b ln2 (d - D)), and what the given token has besides
        const uint32_t own = given && token >= first && token < first + len ? static_cast<uint32_t>(token - first) : ~0u;
        const auto of = [&](float f, uint32_t at) {
            const float d = (f - m) * c;
            const float v = __builtin_amdgcn_exp2f(d) * share * fmaf(slope, fmaxf(d, kZeroBelow) - mean, up);
            return at == own ? fmaf(up, a.sharp, v) : v;
        };
        for (uint32_t base = threadIdx.x; base < vecs; base += kLoads * kLogBlock) {
            u32x4 t[kLoads];
#pragma unroll
            for (int u = 0; u < kLoads; ++u)
                if (base + u * kLogBlock < vecs) {
                    const Stored *from = x + static_cast<uint64_t>(base + u * kLogBlock) * kVec;
                    t[u] = ONCE ? load16_once(from) : load16(from);
                }
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const uint32_t v = base + u * kLogBlock;
                float e[kVec];
                unpack16<T>(t[u], e);
                for (int i = 0; i < kVec; ++i) e[i] = of(e[i], v * kVec + i);
                if (v < vecs) store16_once(g + static_cast<uint64_t>(v) * kVec, pack16<T>(e));
            }
        }
        if (rest < len) g[rest] = Row<T>::pattern(of(Row<T>::value(x[rest]), rest));
    }
}

// A row's numbers and its gradient by one workgroup of B threads that holds it,
// V loads a thread, from its one read to its one write.  Bound by HBM: 4096 x 131072
// bf16 425 us, as a copy of so many bytes (forward and gradient 575).
template <int T, int B, int V>
__global__ __launch_bounds__(B, 4) void logprob_step_kernel(LogArgs a) {
    constexpr int kVec = Row<T>::kVec;
    using Stored = typename Row<T>::Stored;
    __shared__ JoinLds<B> join;
    __shared__ float shared[2];
    const uint32_t tid = threadIdx.x, vecs = a.n / kVec, rest = vecs * kVec + tid;
    const uint64_t row = a.first_task + xcd_chunk(blockIdx.x, gridDim.x);
    const Stored *x = static_cast<const Stored *>(a.logits) + row * a.stride;
    Stored *g = static_cast<Stored *>(a.grad) + row * a.grad_stride;
    const uint32_t none = T == kRowF16 ? 0xFC00FC00u : T == kRowBF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
    const bool on = counted(a, row), extra = rest < a.n;
    const auto below = [&](int u) { return static_cast<int>(tid) < static_cast<int>(vecs) - u * B; };
    u32x4 v[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        v[u] = u32x4{none, none, none, none};
        if (on && below(u)) v[u] = load16(reinterpret_cast<const uint8_t *>(x + u * B * kVec) + tid * 16);
    }
    const float over = on && extra ? Row<T>::value(x[rest]) : -INFINITY;
    const Token<T> token(a, row);
    const float asked = a.up && token.given ? a.up[row] : 0.f, asked_entropy = a.up_entropy ? a.up_entropy[row] : 0.f;
    const float c = a.c;
    // each pass unpacks the held words anew: their floats would take twice the registers
    const auto anew = [&]() {
#pragma unroll
        for (int u = 0; u < V; ++u) asm volatile("" : "+v"(v[u]));
    };
    Running<float> mine;
    constexpr int kBatch = V < kLoads ? V : kLoads;
#pragma unroll
    for (int b = 0; b < V; b += kBatch) {
        float f[kBatch * kVec];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            float e[kVec];
            unpack16<T>(v[b + u], e);
#pragma unroll
            for (int i = 0; i < kVec; ++i) f[u * kVec + i] = e[i];
        }
        mine.add(f, largest(f), c);
    }
    if (a.n > vecs * kVec) {
        const float f[1] = {over};
        mine.add(f, over, c);
    }
    anew();
    float top;
    const Sums s = join_sums<B>(join, mine, top, 0, c, [&](float m) {
        double z = 0, w = 0;
        const auto add = [&](float f) {
            const float d = (f - m) * c, p = __builtin_amdgcn_exp2f(d);
            z += p;
            w += p * fmaxf(d, kZeroBelow);
        };
#pragma unroll
        for (int u = 0; u < V; ++u) {
            float f[kVec];
            unpack16<T>(v[u], f);
#pragma unroll
            for (int e = 0; e < kVec; ++e) add(f[e]);
        }
        add(over);
        return double2{z, w};
    });
    anew();
    if (tid == 0) {
        const RowEnd end = finish_row(a, row, on, token.given, token.x, s.z, s.w, s.m, 0);
        shared[0] = -static_cast<float>(end.share * a.sharp);
        shared[1] = static_cast<float>(end.mean);
    }
    __syncthreads();
    // p (a + b ln2 (d - D)): nothing where nothing is asked, whatever the logits hold.
    // Exponents are relative to r, which is not quite the largest logit's.
    const float m = s.m, r = fmaxf(top * c, kLeastReference);
    const float shift = huge(top, c) ? 0.f : static_cast<float>(static_cast<double>(top) * c - r);
    const float up = softened(a, asked), down = softened(a, asked_entropy);
    const float share = shared[0], scaled = share * __builtin_amdgcn_exp2f(-shift);
    const float flat = scaled * up, slope = scaled * down * static_cast<float>(kLn2), mean = shared[1] + shift;
    const bool none_asked = !on || share == 0.f || (asked == 0.f && asked_entropy == 0.f);
    const auto pass = [&](auto of) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            float e[kVec];
            unpack16<T>(v[u], e);
#pragma unroll
            for (int i = 0; i < kVec; ++i) e[i] = of(e[i]);
            if (below(u)) store16_once(reinterpret_cast<uint8_t *>(g + u * B * kVec) + tid * 16, pack16<T>(e));
        }
        if (extra) g[rest] = Row<T>::pattern(of(over));
    };
    if (none_asked) pass([&](float) { return 0.f; });
    else if (huge(top, c)) pass([&](float f) {
        const float d = (f - m) * c;
        return __builtin_amdgcn_exp2f(d) * fmaf(slope, fmaxf(d, kZeroBelow) - mean, flat);
    });
    else if (slope == 0.f) pass([&](float f) { return __builtin_amdgcn_exp2f(fmaf(f, c, -r)) * flat; });
    else pass([&](float f) {
        const float d = fmaf(f, c, -r);
        return __builtin_amdgcn_exp2f(d) * fmaf(slope, fmaxf(d, kZeroBelow) - mean, flat);
    });
    if (!none_asked && token.given) {
        // the token's column over what was written there
        __syncthreads();
        if (tid == 0) {
            const float d = huge(top, c) ? (token.x - m) * c : fmaf(token.x, c, -r), p = __builtin_amdgcn_exp2f(d);
            g[token.at] = Row<T>::pattern(fmaf(up, a.sharp, p * fmaf(slope, fmaxf(d, kZeroBelow) - mean, flat)));
        }
    }
}

// -------------------------------------------------------------------- host

constexpr uint64_t kMaxGrid = 1u << 20;

// How the rows are laid out on workgroups.  A row that several share costs a
// second launch, 3 to 4 us, so that most have one:
//  - a wave for up to 4 KB of many rows (2000 x 2048 bf16 top 5 10.4 us, by 256
//    threads 12.4; of 1000 rows 9.7 and 8.0, of 2000 x 2056 10.9 and 12.9: the border
//    lies between them), for up to 32 KB of very many (2048 x 16384 bf16 13.8 against
//    15.7, 8192 of them 47.4 and 44.2), with up to 16 alternatives 12 KB (8192 x 6144 bf16
//    top 5 44.1 against 46.0, 8192 x 8192 53.2 and 47.5);
//  - else 256 threads (300 x 16384 bf16 top 5 11.0 us, shared 13.6), and 1024 where there
//    are no more rows than CUs and a row is more than a load a thread: 256 x 65536 bf16
//    top 5 13.0 us, by 256 threads 15.4, shared 18.0; 300 of them 24.0, 19.6 and 21.8; up to
//    64 KB of under 128 rows (48 x 32768 10.4, shared 11.9; 48 x 65536 12.8 and 12.5), up to
//    512 KB of more (128 x 131072 18.0, shared 18.3; of 256 x 262152 31.4 and 37.0).
// Shared are long rows of too few to fill the GPU, down to a batch of loads a thread
// (1 x 131072 bf16 top 5 11.0 us, 17.0 by 1024 threads; 300 x 262144 43.2, alone 45.0;
// 512 of them 56.4 and 56.2, but 47.6 and 41.9 without alternatives).  With alternatives (k > 0) a workgroup holds at most kKept batches, k is at
// most half of its threads, and the pieces' words fit one workgroup; where that
// cannot be (fused false) segmented_row_topk selects them from a second read
// (4096 x 131072 bf16 top 128 242 us, top 129 377, top 500 420).
struct LogPlan {
    int block = kLogBlock;
    uint32_t splits = 1, len = 8;
    bool pick = false, fused = true;
};
LogPlan logprob_plan(uint64_t rows, uint64_t n, uint64_t k, uint64_t size) {
    LogPlan p;
    const uint64_t vec = 16 / size, vecs = n / vec;
    if (rows >= 512 && vecs <= 64 * kLoads) p.block = 64;
    if (rows >= 2048 && (k == 0 ? vecs <= 2048 : k <= 16 && vecs <= 768)) p.block = 64;
    const uint64_t bytes = n * size;
    if (rows <= 256 && vecs > 1024 && bytes <= (rows < 128 ? 64 : 512) * 1024) p.block = 1024;
    const bool alone = p.block == 1024 || rows >= 1024 || (rows > 256 && bytes <= 256 * 1024);
    const uint64_t batch = static_cast<uint64_t>(kLoads) * p.block;
    uint64_t s = alone ? 1 : std::min<uint64_t>((vecs + batch - 1) / batch, 1024 / std::max<uint64_t>(1, rows));
    if (k > 0) s = std::min<uint64_t>(s, kJoinWords / k);
    s = std::max<uint64_t>(s, k > 0 ? (vecs + kKept * batch - 1) / (kKept * batch) : n >> 20);
    s = std::max<uint64_t>(s, 1);
    p.len = static_cast<uint32_t>(std::max<uint64_t>(8, ((n + s - 1) / s + 7) / 8 * 8));
    p.splits = static_cast<uint32_t>(std::max<uint64_t>(1, (n + p.len - 1) / p.len));
    if (k > 0) {
        const uint64_t most = p.len / vec, least = (n - (p.splits - 1) * uint64_t(p.len)) / vec;
        p.pick = true;
        // short rows' alternatives are a wave's own work there
        const bool brief = n <= kLanes || (k <= kLanes && n <= 1024);
        p.fused = !brief && most <= kKept * batch && few_wanted(k, p.block, least) && (p.splits == 1 || p.splits * k <= kJoinWords);
    }
    return p;
}

// How many workgroups share a row of the gradient, whose elements are independent.
void gradient_split(uint64_t rows, uint64_t n, uint32_t &splits, uint32_t &len) {
    uint64_t s = 1;
    if (rows < 2048) s = std::min<uint64_t>((2048 + rows - 1) / std::max<uint64_t>(rows, 1), n / 8192);
    s = std::max<uint64_t>(1, s);
    const uint64_t l = std::max<uint64_t>(8, ((n + s - 1) / s + 7) / 8 * 8);
    len = static_cast<uint32_t>(l);
    splits = static_cast<uint32_t>(std::max<uint64_t>(1, (n + l - 1) / l));
}

int check_sizes(int64_t rows, int64_t n, int64_t k, int dtype) {
    if (!row_type_ok(dtype)) return LRS_ERR_DTYPE;
    if (rows < 0 || n < 0 || k < 0 || k > n || k > LRS_MAX_TOPK || static_cast<uint64_t>(n) > LRS_MAX_ROW_LEN) return LRS_ERR_SIZE;
    if (static_cast<uint64_t>(rows) >= (uint64_t(1) << 40) / std::max<uint64_t>(1, static_cast<uint64_t>(n))) return LRS_ERR_SIZE;
    return LRS_OK;
}
struct LogSpace {
    uint64_t sums = 0, stats = 0, lows = 0, words = 0, values = 0, sort = 0, sort_bytes = 0, total = 0;
};
LogSpace logprob_space(uint64_t rows, uint64_t n, uint64_t k, int dtype) {
    LogSpace w;
    if (rows == 0) return w;
    auto place = [&](uint64_t bytes) {
        const uint64_t at = w.total;
        w.total += (bytes + 255) / 256 * 256;
        return at;
    };
    const uint64_t size = row_type_size(dtype);
    const LogPlan p = logprob_plan(rows, n, k, size);
    if (p.fused) {
        if (p.splits > 1) w.sums = place(rows * p.splits * sizeof(Sums));
        if (p.splits > 1) w.words = place(rows * p.splits * k * sizeof(uint64_t));
    } else {
        const LogPlan q = logprob_plan(rows, n, 0, size);
        if (q.splits > 1) w.sums = place(rows * q.splits * sizeof(Sums));
        w.lows = place(rows * sizeof(double));
        w.values = place(rows * k * size);
        w.sort_bytes = segmented_row_topk_workspace_size(rows, n, k, dtype, nullptr);
        w.sort = place(w.sort_bytes);
    }
    if (k == 0 || !p.fused) w.stats = place(rows * kLogStats * sizeof(float));
    return w;
}

// Everything the calls check of the inputs; fills the arguments.
int logprob_inputs(const lrs_logprobs *d, int64_t k, LogArgs &a) {
    if (d == nullptr) return LRS_ERR_NULL_POINTER;
    const int st = check_sizes(d->rows, d->n, k, d->dtype);
    if (st != LRS_OK) return st;
    if (d->token_bytes != 4 && d->token_bytes != 8) return LRS_ERR_DTYPE;
    if (!stride_ok(d->row_stride, d->rows) || !stride_ok(d->token_stride, d->rows)) return LRS_ERR_SIZE;
    if (!(d->temperature > 0) || !std::isfinite(d->temperature) || !std::isfinite(static_cast<float>(kLog2e / d->temperature)))
        return LRS_ERR_OPTION;
    if (d->rows > 0 && ((d->n > 0 && !d->logits) || !d->tokens)) return LRS_ERR_NULL_POINTER;
    if (misaligned(d->logits, row_type_size(d->dtype)) || misaligned(d->tokens, d->token_bytes)) return LRS_ERR_ALIGNMENT;
    a.logits = d->logits;
    a.stride = d->row_stride;
    a.rows = d->rows;
    a.n = static_cast<uint32_t>(d->n);
    a.tokens = d->tokens;
    a.token_stride = d->token_stride;
    a.token_bytes = d->token_bytes;
    a.mask = d->row_mask;
    const double inv_t = 1.0 / d->temperature;
    a.soft = static_cast<float>(std::frexp(std::min(inv_t, 1.0), &a.soft_power));
    a.sharp = static_cast<float>(std::max(inv_t, 1.0));
    a.factor = kLog2e * inv_t;
    // above 0, so that -inf times it is -inf
    a.c = std::max(static_cast<float>(a.factor), std::numeric_limits<float>::denorm_min());
    a.k = static_cast<uint32_t>(k);
    return LRS_OK;
}

// Whether [p, p + bytes) touches any input.
bool hits_input(const lrs_logprobs *d, const void *p, uint64_t bytes) {
    const uint64_t r = d->rows;
    return overlaps(p, bytes, d->logits, span(r, d->row_stride, d->n, row_type_size(d->dtype))) ||
           overlaps(p, bytes, d->tokens, span(r, d->token_stride, 1, d->token_bytes)) ||
           overlaps(p, bytes, d->row_mask, d->row_mask ? r : 0);
}
// Whether any of the outputs touches an input or another output.
template <int N> bool aliased(const lrs_logprobs *d, const void *const (&out)[N], const uint64_t (&bytes)[N]) {
    for (int i = 0; i < N; ++i) {
        if (out[i] == nullptr || bytes[i] == 0) continue;
        if (hits_input(d, out[i], bytes[i])) return true;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], bytes[i], out[j], bytes[j])) return true;
    }
    return false;
}

template <typename F> void by_type(int type, F f) {
    if (type == LRS_DTYPE_FP16) f(std::integral_constant<int, kRowF16>());
    else if (type == LRS_DTYPE_BF16) f(std::integral_constant<int, kRowBF16>());
    else f(std::integral_constant<int, kRowF32>());
}
bool launched() { return hipGetLastError() == hipSuccess; }
dim3 grid_of(uint64_t tasks) { return dim3(static_cast<uint32_t>(std::min<uint64_t>(tasks, kMaxGrid))); }

// Logits that the 256 MB behind the L2s cannot hold are read past the caches:
// forward of 4096 x 131072 bf16 172 us against 191, gradient 403 against 413.
// Smaller ones may be there from the product that made them, and are for the
// gradient that follows: 1027 x 32768 fp32 24 us against 26, gradient 42 against 49.
bool read_once(uint64_t rows, uint64_t n, uint64_t size) { return rows * n * size > (uint64_t(256) << 20); }

template <int T, bool RANK, bool PICK> void launch_plan(const LogPlan &p, const LogArgs &a, uint32_t tasks, const Launch &L) {
    const auto go = [&](auto once) {
        constexpr bool kOnce = decltype(once)::value;
        if (p.block == 64) launch_on(logprob_kernel<T, 64, RANK, PICK, kOnce>, dim3(tasks), dim3(64), L, a);
        else if (p.block == 1024) launch_on(logprob_kernel<T, 1024, RANK, PICK, kOnce>, dim3(tasks), dim3(1024), L, a);
        else launch_on(logprob_kernel<T, kLogBlock, RANK, PICK, kOnce>, dim3(tasks), dim3(kLogBlock), L, a);
    };
    if constexpr (PICK) go(std::false_type());  // batches are read again
    else if (read_once(a.rows, a.n, row_type_size(T))) go(std::true_type());
    else go(std::false_type());
}

// The rows' numbers, and with a plan that has room for them the alternatives.
int logprob_values(LogArgs a, const LogPlan &p, int dtype, const Ctx &c) {
    a.splits = p.splits;
    a.split_len = p.len;
    const uint64_t tasks = a.rows * a.splits;
    for (a.first_task = 0; a.first_task < tasks; a.first_task += kMaxGrid) {
        TimedLaunch t(4, c);
        const uint32_t now = static_cast<uint32_t>(std::min<uint64_t>(tasks - a.first_task, kMaxGrid));
        by_type(dtype, [&](auto i) {
            if (p.pick) launch_plan<i.value, true, true>(p, a, now, t.L);
            else if (a.ranks) launch_plan<i.value, true, false>(p, a, now, t.L);
            else launch_plan<i.value, false, false>(p, a, now, t.L);
        });
        if (!launched()) return LRS_ERR_HIP;
    }
    if (a.splits == 1) return LRS_OK;
    a.first_task = 0;
    TimedLaunch t(4, c);
    by_type(dtype, [&](auto i) {
        if (p.pick) launch_on(logprob_join_kernel<i.value, true>, grid_of(a.rows), dim3(kLogBlock), t.L, a);
        else launch_on(logprob_join_kernel<i.value, false>, grid_of(a.rows), dim3(kLanes), t.L, a);
    });
    return launched() ? LRS_OK : LRS_ERR_HIP;
}
// Rows of at most 256 KB are held: by 1024 threads where there are no more rows
// than CUs, by the fewest that hold one where several workgroups share a CU.
constexpr uint64_t kHeldBytes = 1024 * 16 * 16;
bool logprob_held(uint64_t rows, uint64_t n, uint64_t size) {
    // of few long rows, forward and gradient by many workgroups (1 x 131072 bf16: 14 us, 19 us held)
    return n * size <= kHeldBytes && (rows > 32 || n * size <= kHeldBytes / 2);
}
template <int T> void launch_step(const LogArgs &a, uint32_t rows, const Launch &L) {
    const uint64_t vecs = a.n / Row<T>::kVec;
    const auto go = [&](auto kernel, int block) { launch_on(kernel, dim3(rows), dim3(block), L, a); };
    if (a.rows <= 256) {
        if (vecs <= 1024 * 2) return go(logprob_step_kernel<T, 1024, 2>, 1024);
        if (vecs <= 1024 * 4) return go(logprob_step_kernel<T, 1024, 4>, 1024);
        if (vecs <= 1024 * 8) return go(logprob_step_kernel<T, 1024, 8>, 1024);
        return go(logprob_step_kernel<T, 1024, 16>, 1024);
    }
    if (vecs <= 64 * 4) return go(logprob_step_kernel<T, 64, 4>, 64);
    if (vecs <= 64 * 8) return go(logprob_step_kernel<T, 64, 8>, 64);
    if (vecs <= 128 * 8) return go(logprob_step_kernel<T, 128, 8>, 128);
    if (vecs <= 256 * 8) return go(logprob_step_kernel<T, 256, 8>, 256);
    if (vecs <= 256 * 16) return go(logprob_step_kernel<T, 256, 16>, 256);
    if (vecs <= 512 * 16) return go(logprob_step_kernel<T, 512, 16>, 512);
    go(logprob_step_kernel<T, 1024, 16>, 1024);
}
int logprob_step(LogArgs a, int dtype, const Ctx &c) {
    for (a.first_task = 0; a.first_task < a.rows; a.first_task += kMaxGrid) {
        TimedLaunch t(4, c);
        const uint32_t now = static_cast<uint32_t>(std::min<uint64_t>(a.rows - a.first_task, kMaxGrid));
        by_type(dtype, [&](auto i) { launch_step<i.value>(a, now, t.L); });
        if (!launched()) return LRS_ERR_HIP;
    }
    return LRS_OK;
}
int logprob_gradient(LogArgs a, int dtype, const Ctx &c) {
    if (a.rows == 0 || a.n == 0) return LRS_OK;
    gradient_split(a.rows, a.n, a.splits, a.split_len);
    TimedLaunch t(4, c);
    const bool once = read_once(a.rows, a.n, row_type_size(dtype));
    by_type(dtype, [&](auto i) {
        launch_on(once ? logprob_grad_kernel<i.value, true> : logprob_grad_kernel<i.value, false>, grid_of(a.rows * a.splits),
                  dim3(kLogBlock), t.L, a);
    });
    return launched() ? LRS_OK : LRS_ERR_HIP;
}

}  // namespace
}  // namespace lrs

using namespace lrs;

extern "C" {

size_t token_logprobs_workspace_size(int64_t rows, int64_t n, int64_t k, int dtype, const lrs_options *opts) {
    if (!options_ok(opts) || check_sizes(rows, n, k, dtype) != LRS_OK) return 0;
    return static_cast<size_t>(logprob_space(rows, n, k, dtype).total);
}

int token_logprobs_forward(const lrs_logprobs *in, float *logprobs, float *entropy, float *row_stats, void *workspace,
                           size_t workspace_bytes, void *stream, const lrs_options *opts) try {
    Ctx c;
    if (!make_ctx(stream, opts, c)) return LRS_ERR_OPTION;
    LogArgs a{};
    const int st = logprob_inputs(in, 0, a);
    if (st != LRS_OK) return st;
    if (a.rows == 0) return LRS_OK;
    const LogSpace w = logprob_space(a.rows, a.n, 0, in->dtype);
    if (!logprobs || !entropy || !workspace) return LRS_ERR_NULL_POINTER;
    if (misaligned(logprobs, 4) || misaligned(entropy, 4) || misaligned(row_stats, 4) || misaligned(workspace, 256))
        return LRS_ERR_ALIGNMENT;
    if (workspace_bytes < w.total) return LRS_ERR_WORKSPACE_TOO_SMALL;
    const void *const out[] = {logprobs, entropy, row_stats, workspace};
    const uint64_t bytes[] = {4 * a.rows, 4 * a.rows, 4 * kLogStats * a.rows, w.total};
    if (aliased(in, out, bytes)) return LRS_ERR_ALIASING;
    a.sums = reinterpret_cast<Sums *>(static_cast<uint8_t *>(workspace) + w.sums);
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.stats = row_stats;
    c.elems = a.rows * a.n;
    return logprob_values(a, logprob_plan(a.rows, a.n, 0, row_type_size(in->dtype)), in->dtype, c);
} catch (...) {
    return LRS_ERR_HIP;
}

int token_logprobs_topk(const lrs_logprobs *in, int64_t k, float *logprobs, float *entropy, int32_t *ranks,
                        float *top_logprobs, int64_t *top_indices, void *workspace, size_t workspace_bytes, void *stream,
                        const lrs_options *opts) try {
    Ctx c;
    if (!make_ctx(stream, opts, c)) return LRS_ERR_OPTION;
    LogArgs a{};
    const int st = logprob_inputs(in, k, a);
    if (st != LRS_OK) return st;
    if (a.mask != nullptr) return LRS_ERR_OPTION;
    if (a.rows == 0) return LRS_OK;
    const LogSpace w = logprob_space(a.rows, a.n, a.k, in->dtype);
    if (!logprobs || !entropy || !ranks || (k > 0 && (!top_logprobs || !top_indices)) || (w.total && !workspace))
        return LRS_ERR_NULL_POINTER;
    if (misaligned(logprobs, 4) || misaligned(entropy, 4) || misaligned(ranks, 4) || misaligned(top_logprobs, 4) ||
        misaligned(top_indices, 8) || (w.total && misaligned(workspace, 256)))
        return LRS_ERR_ALIGNMENT;
    if (workspace_bytes < w.total) return LRS_ERR_WORKSPACE_TOO_SMALL;
    const void *const out[] = {logprobs, entropy, ranks, top_logprobs, top_indices, workspace};
    const uint64_t bytes[] = {4 * a.rows, 4 * a.rows, 4 * a.rows, 4 * a.rows * a.k, 8 * a.rows * a.k, w.total};
    if (aliased(in, out, bytes)) return LRS_ERR_ALIASING;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const uint64_t size = row_type_size(in->dtype);
    const LogPlan p = logprob_plan(a.rows, a.n, a.k, size);
    a.sums = reinterpret_cast<Sums *>(ws + w.sums);
    a.words = reinterpret_cast<uint64_t *>(ws + w.words);
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.ranks = ranks;
    a.top_logprobs = top_logprobs;
    a.top_indices = top_indices;
    c.elems = a.rows * a.n;
    if (p.fused) return logprob_values(a, p, in->dtype, c);
    a.stats = reinterpret_cast<float *>(ws + w.stats);
    a.lows = reinterpret_cast<double *>(ws + w.lows);
    int fs = logprob_values(a, logprob_plan(a.rows, a.n, 0, size), in->dtype, c);
    if (fs != LRS_OK) return fs;
    fs = segmented_row_topk(a.logits, in->row_stride, ws + w.values, top_indices, in->rows, in->n, k, in->dtype, 1, ws + w.sort,
                            w.sort_bytes, stream, opts);
    if (fs != LRS_OK) return fs;
    a.top_values = ws + w.values;
    TimedLaunch t(4, c);
    by_type(in->dtype, [&](auto i) {
        launch_on(logprob_top_kernel<i.value>, grid_of((a.rows * a.k + kLogBlock - 1) / kLogBlock), dim3(kLogBlock), t.L, a);
    });
    return launched() ? LRS_OK : LRS_ERR_HIP;
} catch (...) {
    return LRS_ERR_HIP;
}

int token_logprobs_backward(const lrs_logprobs *in, const float *row_stats, const float *logprob_grad,
                            const float *entropy_grad, void *grad, int64_t grad_stride, void *stream,
                            const lrs_options *opts) try {
    Ctx c;
    if (!make_ctx(stream, opts, c)) return LRS_ERR_OPTION;
    LogArgs a{};
    const int st = logprob_inputs(in, 0, a);
    if (st != LRS_OK) return st;
    if (!stride_ok(grad_stride, in->rows) || (in->rows > 1 && grad_stride < in->n)) return LRS_ERR_SIZE;
    if (a.rows == 0 || a.n == 0) return LRS_OK;
    if (!row_stats || !grad || (!logprob_grad && !entropy_grad)) return LRS_ERR_NULL_POINTER;
    const uint64_t size = row_type_size(in->dtype), gb = span(a.rows, grad_stride, a.n, size);
    if (misaligned(row_stats, 4) || misaligned(logprob_grad, 4) || misaligned(entropy_grad, 4) || misaligned(grad, size))
        return LRS_ERR_ALIGNMENT;
    if (hits_input(in, grad, gb) || overlaps(grad, gb, row_stats, 4 * kLogStats * a.rows) ||
        overlaps(grad, gb, logprob_grad, 4 * a.rows) || overlaps(grad, gb, entropy_grad, 4 * a.rows))
        return LRS_ERR_ALIASING;
    a.stats = const_cast<float *>(row_stats);
    a.up = logprob_grad;
    a.up_entropy = entropy_grad;
    a.grad = grad;
    a.grad_stride = grad_stride;
    c.elems = a.rows * a.n;
    return logprob_gradient(a, in->dtype, c);
} catch (...) {
    return LRS_ERR_HIP;
}

int token_logprobs_step(const lrs_logprobs *in, const float *logprob_grad, const float *entropy_grad, float *logprobs,
                        float *entropy, void *grad, int64_t grad_stride, void *workspace, size_t workspace_bytes,
                        void *stream, const lrs_options *opts) try {
    Ctx c;
    if (!make_ctx(stream, opts, c)) return LRS_ERR_OPTION;
    LogArgs a{};
    const int st = logprob_inputs(in, 0, a);
    if (st != LRS_OK) return st;
    if (!stride_ok(grad_stride, in->rows) || (in->rows > 1 && grad_stride < in->n)) return LRS_ERR_SIZE;
    if (a.rows == 0) return LRS_OK;
    const LogSpace w = logprob_space(a.rows, a.n, 0, in->dtype);
    if (!logprobs || !entropy || !workspace || (a.n > 0 && !grad) || (!logprob_grad && !entropy_grad)) return LRS_ERR_NULL_POINTER;
    const uint64_t size = row_type_size(in->dtype), gb = span(a.rows, grad_stride, a.n, size);
    if (misaligned(logprobs, 4) || misaligned(entropy, 4) || misaligned(logprob_grad, 4) || misaligned(entropy_grad, 4) ||
        misaligned(grad, size) || misaligned(workspace, 256))
        return LRS_ERR_ALIGNMENT;
    if (workspace_bytes < w.total) return LRS_ERR_WORKSPACE_TOO_SMALL;
    const void *const out[] = {logprobs, entropy, grad, workspace};
    const uint64_t bytes[] = {4 * a.rows, 4 * a.rows, gb, w.total};
    if (aliased(in, out, bytes)) return LRS_ERR_ALIASING;
    for (int i = 0; i < 4; ++i)
        if (bytes[i] && (overlaps(out[i], bytes[i], logprob_grad, 4 * a.rows) || overlaps(out[i], bytes[i], entropy_grad, 4 * a.rows)))
            return LRS_ERR_ALIASING;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.sums = reinterpret_cast<Sums *>(ws + w.sums);
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.up = logprob_grad;
    a.up_entropy = entropy_grad;
    a.grad = grad;
    a.grad_stride = grad_stride;
    c.elems = a.rows * a.n;
    if (logprob_held(a.rows, a.n, size)) return logprob_step(a, in->dtype, c);
    a.stats = reinterpret_cast<float *>(ws + w.stats);
    const int fs = logprob_values(a, logprob_plan(a.rows, a.n, 0, size), in->dtype, c);
    return fs != LRS_OK ? fs : logprob_gradient(a, in->dtype, c);
} catch (...) {
    return LRS_ERR_HIP;
}

}  // extern "C"
