// lrs_select.h -- device helpers that find the largest elements of a row
// (internal header): order images, words that no two elements share, the bound
// that a few elements reach, and the places of those.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lrs_rows.h"

namespace lrs {

// Order image of a pattern, the wanted elements largest (signed).
__device__ inline int image16(uint32_t pattern, uint32_t flip) {
    const int v = static_cast<int16_t>(pattern);
    return static_cast<int16_t>((v ^ ((v >> 15) & 0x7FFF)) ^ static_cast<int>(flip));
}
__device__ inline int image32(uint32_t pattern, uint32_t flip) {
    const int v = static_cast<int>(pattern);
    return (v ^ ((v >> 31) & 0x7FFFFFFF)) ^ static_cast<int>(flip);
}
template <int W> __device__ inline int image(uint32_t pattern, uint32_t flip) {
    return W == 2 ? image16(pattern, flip) : image32(pattern, flip);
}
// The map is its own inverse.
template <int W> __device__ inline uint32_t pattern_of(int img, uint32_t flip) {
    const int v = img ^ static_cast<int>(flip);
    if (W == 2) return static_cast<uint32_t>(v ^ ((v >> 15) & 0x7FFF)) & 0xFFFFu;
    return static_cast<uint32_t>(v ^ ((v >> 31) & 0x7FFFFFFF));
}
__device__ inline uint64_t word_of(int img, uint32_t column) {
    return (static_cast<uint64_t>(static_cast<uint32_t>(img) ^ 0x80000000u) << 32) | (0xFFFFFFFFu - column);
}
__device__ inline int image_of(uint64_t word) { return static_cast<int>(static_cast<uint32_t>(word >> 32) ^ 0x80000000u); }
__device__ inline uint32_t column_of(uint64_t word) { return 0xFFFFFFFFu - static_cast<uint32_t>(word); }

// The largest of the wave's values, in every lane.
__device__ inline int wave_max_int(int v) {
    v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x111, 0xF, 0xF, false));  // row_shr 1, 2, 4, 8
    v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x112, 0xF, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x114, 0xF, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x118, 0xF, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x142, 0xF, 0xF, false));  // row_bcast 15, 31
    v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x143, 0xF, 0xF, false));
    return __builtin_amdgcn_readlane(v, kLanes - 1);
}
// The sum over this lane and those below.
__device__ inline uint32_t lanes_sum(uint32_t v) {
    v += moved<0x111>(v, 0u);
    v += moved<0x112>(v, 0u);
    v += moved<0x114>(v, 0u);
    v += moved<0x118>(v, 0u);
    v += moved<0x142, 0xA>(v, 0u);
    v += moved<0x143, 0xC>(v, 0u);
    return v;
}

// Bins of images below the largest, 2^shift images a bin; whoever lies lower
// is not counted.
constexpr uint32_t kBins = 2048, kCoarse = 64, kFine = kBins / kCoarse;
constexpr uint32_t kRankWords = 128;   // so many are ranked by counting all the others

struct Bins {
    uint32_t coarse[kCoarse];
    uint32_t fine[kBins];
};
template <int B> __device__ inline void clear_bins(Bins &h) {
    if (threadIdx.x < kCoarse) h.coarse[threadIdx.x] = 0;
    for (uint32_t i = threadIdx.x; i < kBins; i += B) h.fine[i] = 0;
}
__device__ inline void add_to_bins(Bins &h, int img, int top, uint32_t shift) {
    const uint32_t bin = (static_cast<uint32_t>(top) - static_cast<uint32_t>(img)) >> shift;
    if (bin < kBins) {
        atomicAdd(&h.fine[bin], 1u);
        atomicAdd(&h.coarse[bin / kFine], 1u);
    }
}
// By a whole wave: the first bin up to which `want` were counted, kBins if fewer were.
__device__ inline uint32_t bin_of(const Bins &h, uint32_t want) {
    const uint32_t lane = threadIdx.x % kLanes;
    const uint32_t c = h.coarse[lane], upto = lanes_sum(c);
    const uint64_t enough = __ballot(upto >= want);
    if (enough == 0) return kBins;
    const int q = __builtin_ctzll(enough);
    const uint32_t before = __builtin_amdgcn_readlane(upto - c, q);
    const uint32_t f = lane < kFine ? h.fine[q * kFine + lane] : 0;
    return q * kFine + __builtin_ctzll(__ballot(before + lanes_sum(f) >= want));
}

// Two images of 16 bits at once, the wanted elements largest.
typedef short i16x2 __attribute__((ext_vector_type(2)));
__device__ inline i16x2 image_pair(uint32_t w, uint32_t flip) {
    const i16x2 v = __builtin_bit_cast(i16x2, w);
    const uint32_t sign = __builtin_bit_cast(uint32_t, static_cast<i16x2>(v >> 15));
    return __builtin_bit_cast(i16x2, w ^ (sign & 0x7FFF7FFFu) ^ flip);
}
template <int W> __device__ inline int vec_max(u32x4 v, uint32_t flip) {
    if constexpr (W == 2) {
        const i16x2 m = __builtin_elementwise_max(
            __builtin_elementwise_max(image_pair(v[0], flip), image_pair(v[1], flip)),
            __builtin_elementwise_max(image_pair(v[2], flip), image_pair(v[3], flip)));
        return max(static_cast<int>(m.x), static_cast<int>(m.y));
    } else {
        return max(max(image32(v[0], flip), image32(v[1], flip)), max(image32(v[2], flip), image32(v[3], flip)));
    }
}

// The sum over the workgroup of a count (two barriers).
template <int B> __device__ inline uint32_t block_sum(uint32_t c, uint32_t *cells) {
    c = wave_sum(c);
    __syncthreads();
    if (threadIdx.x % kLanes == 0) cells[threadIdx.x / kLanes] = c;
    __syncthreads();
    c = 0;
    for (int w = 0; w < B / kLanes; ++w) c += cells[w];
    return c;
}

// f(image, column) for every element of a load.
template <int W, typename F> __device__ inline void each_image(u32x4 w, uint32_t flip, uint32_t at, F f) {
    constexpr int kVec = 16 / W;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        const uint32_t pat = W == 2 ? (w[e / 2] >> (16 * (e & 1))) & 0xFFFFu : w[e % 4];
        f(image<W>(pat, flip), at + e);
    }
}

// What a workgroup of B threads needs to select; bins and count are cleared before.
template <int B, uint32_t CAP> struct SelectLds {
    uint64_t buf[CAP];
    Bins bins;
    uint32_t cells[B / kLanes];
    uint32_t count;
};

// put(word, place) for the `want` largest of lds.buf[0, c) (c <= CAP), no image above
// `top` or below `low`.  Few count the words above
// theirs; more are dealt to bins in order first and count within their bin
// (300 of 512 threads: 3 us by counting all).
template <int B, uint32_t CAP, typename Put>
__device__ void write_ranked(SelectLds<B, CAP> &lds, uint32_t c, uint32_t want, int top, int64_t low, Put put) {
    uint64_t *const buf = lds.buf;
    Bins &bins = lds.bins;
    uint32_t *const cells = lds.cells;
    const uint32_t tid = threadIdx.x;
    if (c <= kRankWords) {
        for (uint32_t i = tid; i < c; i += B) {
            const uint64_t w = buf[i];
            uint32_t place = 0;
#pragma unroll 8
            for (uint32_t j = 0; j < c; ++j) place += buf[j] > w;
            if (place < want) put(w, place);
        }
    } else {
        constexpr int kOwn = CAP / B, kShare = kBins / B;
        clear_bins<B>(bins);
        const uint32_t range = static_cast<uint32_t>(static_cast<int64_t>(top) - low);
        const uint32_t shift = range < kBins ? 0 : 21 - __builtin_clz(range);
        uint64_t w[kOwn];
        uint32_t at[kOwn];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            w[i] = i * B + tid < c ? buf[i * B + tid] : 0;
            if (w[i]) at[i] = atomicAdd(&bins.fine[(static_cast<uint32_t>(top) - static_cast<uint32_t>(image_of(w[i]))) >> shift], 1u);
        }
        __syncthreads();
        uint32_t held[kShare], sum = 0;
#pragma unroll
        for (int i = 0; i < kShare; ++i) sum += held[i] = bins.fine[tid * kShare + i];
        const uint32_t upto = lanes_sum(sum);
        if (tid % kLanes == kLanes - 1) cells[tid / kLanes] = upto;
        __syncthreads();
        uint32_t start = upto - sum;
        for (uint32_t v = 0; v < tid / kLanes; ++v) start += cells[v];
#pragma unroll
        for (int i = 0; i < kShare; ++i) {
            bins.fine[tid * kShare + i] = start;
            start += held[i];
        }
        __syncthreads();
        const auto bin_at = [&](uint64_t word) { return (static_cast<uint32_t>(top) - static_cast<uint32_t>(image_of(word))) >> shift; };
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            if (w[i]) buf[bins.fine[bin_at(w[i])] + at[i]] = w[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            if (w[i]) {
                const uint32_t bin = bin_at(w[i]), from = bins.fine[bin], to = bin + 1 < kBins ? bins.fine[bin + 1] : c;
                uint32_t place = from;
                if (from < want)
                    for (uint32_t j = from; j < to; ++j) place += buf[j] > w[i];
                if (place < want) put(w[i], place);
            }
    }
}

// Whether the threads' largest elements give the bound: k of them at most half.
constexpr int kBatch = 4;
__host__ __device__ inline bool few_wanted(uint64_t want, uint64_t threads, uint64_t vecs) {
    return 2 * want <= (threads < vecs ? threads : vecs);
}

// put(word, place) for the `want` largest of the `len` elements at x (a row's from
// column `first` on), by a workgroup.  `top` is the largest image; fill(shift) adds
// images to the bins, of all elements or (by_thread) of each thread's largest one;
// reach(bound, take) calls take(image, place) for every element that reaches the
// bound, and may for others.  Where ties leave too many, the image of the last
// wanted one is found exactly and the first of its columns fill up.
template <int W, int B, uint32_t CAP, typename Stored, typename Fill, typename Reach, typename Put>
__device__ inline void select_largest(SelectLds<B, CAP> &lds, const Stored *x, uint32_t len, uint32_t first, uint32_t flip,
                                      uint32_t want, int top, bool by_thread, Fill fill, Reach reach, Put put) {
    constexpr int kVec = 16 / W;
    const uint32_t tid = threadIdx.x, vecs = len / kVec, rest = vecs * kVec + tid;
    const bool extra = rest < len;
    uint32_t shift = W == 2 ? 0 : 13, bin;
    for (;; shift += W == 2 ? 5 : 8) {  // at the second shift every image has a bin
        fill(shift);
        __syncthreads();
        bin = bin_of(lds.bins, want);
        if (bin < kBins) break;
        __syncthreads();
        clear_bins<B>(lds.bins);
        __syncthreads();
    }
    const int64_t low = static_cast<int64_t>(top) - ((static_cast<int64_t>(bin + 1) << shift) - 1);
    int bound = static_cast<int>(max(low, static_cast<int64_t>(W == 2 ? -32768 : INT32_MIN)));

    const auto take = [&](int img, uint32_t at) {
        if (img >= bound) {
            const uint32_t slot = atomicAdd(&lds.count, 1u);
            if (slot < CAP) lds.buf[slot] = word_of(img, first + at);
        }
    };
    reach(bound, take);
    __syncthreads();
    uint32_t c = lds.count;
    // The row is read again, some 16 to 33 times: ties of the last wanted one, and rows of which fewer threads than
    // `want` hold anything but the lowest image, which the bound then is (all but one in 10000 of 4096 x 131072 bf16
    // logits at -inf, with ranks: 20 alternatives 3333 us, 5 of them 646; one in 1000 left 379 and 372).
    if (c > CAP) {
        const auto again = [&](auto f) {
            for (uint32_t i = tid; i < vecs; i += B) each_image<W>(load16(x + i * kVec), flip, i * kVec, f);
            if (extra) f(image<W>(x[rest], flip), rest);
        };
        // the k-th image: at least `want` reach lo, fewer pass hi
        int lo = bound, hi = by_thread ? top : min(static_cast<int64_t>(top), low + (int64_t(1) << shift) - 1);
        while (lo < hi) {
            const int mid = (lo | hi) - ((lo ^ hi) >> 1);
            uint32_t n = 0;
            again([&](int img, uint32_t) { n += img >= mid; });
            if (block_sum<B>(n, lds.cells) >= want) lo = mid;
            else hi = mid - 1;
        }
        __syncthreads();
        if (tid == 0) lds.count = 0;
        __syncthreads();
        if (lo < INT32_MAX) {
            bound = lo + 1;
            again(take);
        }
        bound = lo;
        __syncthreads();
        c = lds.count;  // below `want`
        // the first columns of image lo: stripe by stripe, in the order of threads
        for (uint32_t base = 0; base <= vecs && c < want; base += B) {
            const uint32_t i = base + tid;
            // the elements after the last whole load are a stripe of their own threads' order
            const bool in = i < vecs, last = base + B > vecs;
            const u32x4 w = in ? load16(x + i * kVec) : u32x4{0, 0, 0, 0};
            const auto stripe = [&](bool on, auto elements) {
                uint32_t here = 0;
                if (on) elements([&](int img, uint32_t) { here += img == lo; });
                const uint32_t upto = lanes_sum(here);
                __syncthreads();
                if (tid % kLanes == kLanes - 1) lds.cells[tid / kLanes] = upto;
                __syncthreads();
                uint32_t at = c + upto - here, all = 0;
                for (uint32_t w = 0; w < B / kLanes; ++w) {
                    if (w < tid / kLanes) at += lds.cells[w];
                    all += lds.cells[w];
                }
                if (on) elements([&](int img, uint32_t column) {
                    if (img == lo) {
                        if (at < want) lds.buf[at] = word_of(lo, first + column);
                        ++at;
                    }
                });
                c = min(c + all, want);
            };
            stripe(in, [&](auto f) { each_image<W>(w, flip, i * kVec, f); });
            if (last) stripe(extra, [&](auto f) { f(image<W>(x[rest], flip), rest); });
        }
        __syncthreads();
    }
    write_ranked<B, CAP>(lds, c, want, top, bound, put);
}

// put(word, place) for the k largest of `total` words (at most CAP, zeros are none; k of
// them at least are), by the same bound: 1 x 131072 fp32 in 16 splits takes 9 us
// with it, 37 us of sorting the words before.
template <int W, int B, uint32_t CAP, typename Put>
__device__ inline void merge_words(SelectLds<B, CAP> &lds, int (&tops)[B / kLanes], const uint64_t *in, uint32_t total, uint32_t k,
                                   Put put) {
    constexpr int V = CAP / B;
    const uint32_t tid = threadIdx.x;
    uint64_t w[V];
    int top = INT32_MIN;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        w[u] = u * B + tid < total ? in[u * B + tid] : 0;
        if (w[u]) top = max(top, image_of(w[u]));
    }
    clear_bins<B>(lds.bins);
    if (tid == 0) lds.count = 0;
    top = wave_max_int(top);
    if (tid % kLanes == 0) tops[tid / kLanes] = top;
    __syncthreads();
    for (int i = 0; i < B / kLanes; ++i) top = max(top, tops[i]);
    uint32_t shift = W == 2 ? 0 : 13, bin;
    for (;; shift += W == 2 ? 5 : 8) {
#pragma unroll
        for (int u = 0; u < V; ++u)
            if (w[u]) add_to_bins(lds.bins, image_of(w[u]), top, shift);
        __syncthreads();
        bin = bin_of(lds.bins, k);
        if (bin < kBins) break;
        __syncthreads();
        clear_bins<B>(lds.bins);
        __syncthreads();
    }
    const int64_t low = static_cast<int64_t>(top) - ((static_cast<int64_t>(bin + 1) << shift) - 1);
#pragma unroll
    for (int u = 0; u < V; ++u)
        if (w[u] && image_of(w[u]) >= low) lds.buf[atomicAdd(&lds.count, 1u)] = w[u];
    __syncthreads();
    write_ranked<B, CAP>(lds, lds.count, k, top, low, put);
}

}  // namespace lrs
