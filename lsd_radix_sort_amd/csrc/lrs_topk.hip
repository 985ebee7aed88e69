// lrs_topk.hip -- the first k columns of a row sort without the sort (gfx950).
//
// Each element becomes one 64-bit word, order image above, complemented column
// below, so the wanted elements are the k largest words, no two words are
// alike, and ties go to the lowest column whatever order the words arrive in.
// One workgroup reads its row once, 16 bytes a lane.  The k-th largest of the
// first chunk's per-load maxima bounds the row's k-th largest from below; only
// elements at or above the bound enter a buffer in LDS, and when the buffer is
// nearly full its k largest stay and the least of them becomes the bound.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/lsd_radix_sort.h"
#include "lrs_host.h"
#include "lrs_rows.h"

namespace lrs {
namespace {

constexpr int kTopBlock = 256;
constexpr int kTopVecs = 8;       // 16-byte loads a thread has in flight
constexpr int kTopBuffer = 4096;  // words in LDS: k at most 1024 and one load of every thread, twice over

struct TopArgs {
    const void *x;
    uint64_t stride;      // elements from one row to the next
    uint64_t rows;
    uint32_t n;           // elements in a row
    uint32_t k;
    uint32_t splits;      // workgroups that share one row
    uint32_t split_len;   // elements each of them reads
    uint32_t flip;        // 0, or all ones for the smallest first
    void *values;         // patterns
    int64_t *indices;
    uint64_t *words;      // splits > 1: [rows][splits][k], 0 where a split has fewer
};

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

// Sorts buf[0, count) descending; the words from count to the next power of
// two are cleared (a real word is never 0).  Barriers before and after.
__device__ void sort_words(uint64_t *buf, uint32_t count) {
    uint32_t m = 2;
    while (m < count) m <<= 1;
    __syncthreads();
    for (uint32_t i = count + threadIdx.x; i < m; i += kTopBlock) buf[i] = 0;
    __syncthreads();
    for (uint32_t size = 2; size <= m; size <<= 1)
        for (uint32_t d = size >> 1; d > 0; d >>= 1) {
            for (uint32_t t = threadIdx.x; t < m / 2; t += kTopBlock) {
                const uint32_t i = 2 * t - (t & (d - 1)), j = i + d;
                const uint64_t a = buf[i], b = buf[j];
                const bool down = (i & size) == 0;
                if ((a < b) == down) {
                    buf[i] = b;
                    buf[j] = a;
                }
            }
            __syncthreads();
        }
}

template <int W> __device__ void write_row(const TopArgs &a, const uint64_t *buf, uint64_t row, uint32_t k) {
    for (uint32_t j = threadIdx.x; j < k; j += kTopBlock) {
        const uint64_t w = buf[j];
        const uint64_t at = row * a.k + j;
        if (W == 2)
            static_cast<uint16_t *>(a.values)[at] = static_cast<uint16_t>(pattern_of<2>(image_of(w), a.flip));
        else
            static_cast<uint32_t *>(a.values)[at] = pattern_of<4>(image_of(w), a.flip);
        a.indices[at] = column_of(w);
    }
}

template <int W>
__global__ __launch_bounds__(kTopBlock) void topk_kernel(TopArgs a) {
    constexpr int kVec = 16 / W;
    constexpr uint32_t kStep = kTopBlock * kVec;        // elements of one load of every thread
    constexpr uint32_t kChunk = kStep * kTopVecs;
    __shared__ uint64_t buf[kTopBuffer];
    __shared__ uint32_t count;
    __shared__ uint32_t sums[2][kTopBlock / kLanes];
    using Stored = typename Row<W == 2 ? kRowF16 : kRowF32>::Stored;

    for (uint64_t task = blockIdx.x; task < a.rows * a.splits; task += gridDim.x) {
        const uint64_t row = task / a.splits;
        const uint32_t split = static_cast<uint32_t>(task % a.splits);
        const uint32_t first = split * a.split_len;
        const uint32_t len = min(a.split_len, a.n - first);
        const Stored *x = static_cast<const Stored *>(a.x) + row * a.stride + first;
        const uint32_t vecs = len / kVec;
        const uint32_t want = min(a.k, len);
        // elements whose image is below `bound` cannot be among the k
        int bound = INT32_MIN;
        bool closed = false;  // nothing that comes later can be among the k either
        __syncthreads();      // the last task's readers of buf are done
        if (threadIdx.x == 0) count = 0;
        __syncthreads();

        // keep the k largest words; later elements with the k-th one's image
        // come after it, so from now on only larger images enter
        auto shrink = [&]() {
            sort_words(buf, count);
            const int img = image_of(buf[want - 1]);
            __syncthreads();
            if (threadIdx.x == 0) count = want;
            closed = img == INT32_MAX;
            bound = closed ? img : img + 1;
            __syncthreads();
        };
        auto add = [&](int img, uint32_t at) {
            if (img >= bound && !closed) {
                const uint32_t slot = atomicAdd(&count, 1u);
                if (slot < kTopBuffer) buf[slot] = word_of(img, first + at);
            }
        };
        auto add_vec = [&](u32x4 v, uint32_t vec) {
            for (int e = 0; e < kVec; ++e) {
                const uint32_t pat = W == 2 ? (v[e / 2] >> (16 * (e & 1))) & 0xFFFFu : v[e % 4];
                add(image<W>(pat, a.flip), vec * kVec + e);
            }
        };

        for (uint32_t base = 0; base < vecs; base += kChunk / kVec) {
            u32x4 v[kTopVecs];
            int top[kTopVecs];
            for (int u = 0; u < kTopVecs; ++u) {
                const uint32_t vec = base + u * kTopBlock + threadIdx.x;
                if (vec < vecs) v[u] = load16(x + static_cast<uint64_t>(vec) * kVec);
            }
            for (int u = 0; u < kTopVecs; ++u) {
                const uint32_t vec = base + u * kTopBlock + threadIdx.x;
                int m = INT32_MIN;
                for (int e = 0; e < kVec; ++e) {
                    const uint32_t pat = W == 2 ? (v[u][e / 2] >> (16 * (e & 1))) & 0xFFFFu : v[u][e % 4];
                    m = max(m, image<W>(pat, a.flip));
                }
                top[u] = vec < vecs ? m : INT32_MIN;
            }
            if (base == 0 && min(vecs, kChunk / kVec) >= want) {
                // the largest image that at least `want` loads reach, to within
                // the search's early end
                int lo = INT32_MIN, hi = INT32_MAX;
                if (W == 2) lo = -32768, hi = 32767;
                uint32_t round = 0;
                while (lo < hi) {
                    const int mid = static_cast<int>((static_cast<int64_t>(lo) + hi + 1) >> 1);
                    uint32_t c = 0;
                    for (int u = 0; u < kTopVecs; ++u) {
                        const bool in = base + u * kTopBlock + threadIdx.x < vecs;
                        c += __popcll(__ballot(in && top[u] >= mid));
                    }
                    uint32_t *s = sums[round++ & 1];
                    if (threadIdx.x % kLanes == 0) s[threadIdx.x / kLanes] = c;
                    __syncthreads();
                    c = 0;
                    for (int w = 0; w < kTopBlock / kLanes; ++w) c += s[w];
                    if (c >= want) {
                        lo = mid;
                        if (c <= want + want / 4) break;
                    } else {
                        hi = mid - 1;
                    }
                }
                bound = lo;
            }
            const uint32_t before = count;
            __syncthreads();
            for (int u = 0; u < kTopVecs; ++u) {
                const uint32_t vec = base + u * kTopBlock + threadIdx.x;
                if (vec < vecs && top[u] >= bound) add_vec(v[u], vec);
            }
            __syncthreads();
            if (count > kTopBuffer) {
                // too many at once: one load of every thread at a time
                __syncthreads();
                if (threadIdx.x == 0) count = before;
                __syncthreads();
                for (int u = 0; u < kTopVecs; ++u) {
                    const uint32_t held = count;
                    __syncthreads();  // every thread has read it before one adds
                    if (held + kStep > kTopBuffer) shrink();
                    const uint32_t vec = base + u * kTopBlock + threadIdx.x;
                    if (vec < vecs && top[u] >= bound) add_vec(v[u], vec);
                    __syncthreads();
                }
            }
            if (count > kTopBuffer / 2) shrink();
        }
        __syncthreads();
        // the elements after the last whole load
        const uint32_t tail = vecs * kVec + threadIdx.x;
        if (tail < len) add(image<W>(x[tail], a.flip), tail);
        __syncthreads();
        const uint32_t c = count;
        sort_words(buf, c);
        if (a.splits == 1) {
            write_row<W>(a, buf, row, a.k);
        } else {
            uint64_t *out = a.words + task * a.k;
            for (uint32_t j = threadIdx.x; j < a.k; j += kTopBlock) out[j] = j < want ? buf[j] : 0;
        }
    }
}

// ---- short rows -----------------------------------------------------------
//
// Rows of at most 64 elements: an element a lane, 64 / P rows a wave (P the
// power of two at or above n), sorted by a bitonic network across the P lanes.
// A 16-bit image and the column fit one 32-bit word.
template <int W> struct ShortWord;
template <> struct ShortWord<2> {
    using T = uint32_t;
    __device__ static T make(int img, uint32_t column) {
        return (static_cast<uint32_t>(img + 32768) << 16) | (0xFFFFu - column);
    }
    __device__ static int img(T w) { return static_cast<int>(w >> 16) - 32768; }
    __device__ static uint32_t column(T w) { return 0xFFFFu - (w & 0xFFFFu); }
    __device__ static T lane(T w, int l) { return __builtin_amdgcn_readlane(w, l); }
};
template <> struct ShortWord<4> {
    using T = uint64_t;
    __device__ static T make(int img, uint32_t column) { return word_of(img, column); }
    __device__ static int img(T w) { return image_of(w); }
    __device__ static uint32_t column(T w) { return column_of(w); }
    __device__ static T lane(T w, int l) {
        const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(w >> 32), l);
        const uint32_t low = __builtin_amdgcn_readlane(static_cast<uint32_t>(w), l);
        return (static_cast<uint64_t>(hi) << 32) | low;
    }
};

// The word of lane ^ D.
template <int D> __device__ inline uint32_t swap_lanes(uint32_t v) {
    if constexpr (D < 32) return __builtin_amdgcn_ds_swizzle(v, (D << 10) | 0x1F);
    else return __shfl_xor(v, D);
}
template <int D> __device__ inline uint64_t swap_lanes(uint64_t v) {
    return (static_cast<uint64_t>(swap_lanes<D>(static_cast<uint32_t>(v >> 32))) << 32) |
           swap_lanes<D>(static_cast<uint32_t>(v));
}
template <int SIZE, int D, typename T> __device__ inline void lane_merge(T &w, int lane) {
    if constexpr (D > 0) {
        const T o = swap_lanes<D>(w);
        const bool keep_larger = ((lane & SIZE) == 0) == ((lane & D) == 0);
        w = keep_larger == (w < o) ? o : w;
        lane_merge<SIZE, D / 2>(w, lane);
    }
}
// Sorts the words of every P lanes, the largest in the lowest lane.
template <int P, int SIZE = 2, typename T> __device__ inline void lane_sort(T &w, int lane) {
    if constexpr (SIZE <= P) {
        lane_merge<SIZE, SIZE / 2>(w, SIZE == P ? lane & (P - 1) : lane);
        lane_sort<P, 2 * SIZE>(w, lane);
    }
}

template <int W> __device__ inline void write_short(const TopArgs &a, typename ShortWord<W>::T w, uint64_t at) {
    using Word = ShortWord<W>;
    if (W == 2)
        static_cast<uint16_t *>(a.values)[at] = static_cast<uint16_t>(pattern_of<2>(Word::img(w), a.flip));
    else
        static_cast<uint32_t *>(a.values)[at] = pattern_of<4>(Word::img(w), a.flip);
    a.indices[at] = Word::column(w);
}

template <int W, int P>
__global__ __launch_bounds__(kTopBlock) void topk_lanes_kernel(TopArgs a) {
    using Word = ShortWord<W>;
    using Stored = typename Row<W == 2 ? kRowF16 : kRowF32>::Stored;
    const int lane = threadIdx.x % kLanes, j = lane % P;
    constexpr uint64_t kRows = kTopBlock / P;
    for (uint64_t base = blockIdx.x * kRows; base < a.rows; base += gridDim.x * kRows) {
        const uint64_t row = base + threadIdx.x / P;
        typename Word::T w = 0;  // below every element's
        if (row < a.rows && j < static_cast<int>(a.n))
            w = Word::make(image<W>(static_cast<const Stored *>(a.x)[row * a.stride + j], a.flip), j);
        lane_sort<P>(w, lane);
        if (row < a.rows && j < static_cast<int>(a.k)) write_short<W>(a, w, row * a.k + j);
    }
}

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
// The largest of each 16 lanes' values, in all of them.
__device__ inline int row16_max(int v) {
    v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x128, 0xF, 0xF, false));  // row_ror 8, 4, 2, 1
    v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x124, 0xF, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x122, 0xF, 0xF, false));
    return max(v, __builtin_amdgcn_update_dpp(INT32_MIN, v, 0x121, 0xF, 0xF, false));
}
__device__ inline uint32_t lanes_below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                     __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
}

// E consecutive elements of a row as images, INT32_MIN past its end.
template <int W, int E> __device__ inline void load_images(const typename Row<W == 2 ? kRowF16 : kRowF32>::Stored *x,
                                                           uint32_t at, uint32_t n, uint32_t flip, int (&img)[E]) {
    constexpr int kVec = 16 / W;
#pragma unroll
    for (int q = 0; q < E / kVec; ++q) {
        const uint32_t first = at + q * kVec;
        u32x4 v{};
        if (first + kVec <= n) {
            v = load16(x + first);
        } else if (first < n) {
            for (int e = 0; e < kVec; ++e) {
                const uint32_t pat = first + e < n ? x[first + e] : 0;
                if (W == 2) v[e / 2] |= pat << (16 * (e & 1));
                else v[e % 4] = pat;
            }
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const uint32_t pat = W == 2 ? (v[e / 2] >> (16 * (e & 1))) & 0xFFFFu : v[e % 4];
            img[q * kVec + e] = first + e < n ? image<W>(pat, flip) : INT32_MIN;
        }
    }
}

// Rows of at most 16 * E elements and small k: 16 lanes a row, E consecutive
// elements a lane, sorted within the lane.  k times the 16 lanes' heads give
// the next largest, the lowest lane's where they are equal, and that lane
// moves on.
template <int W, int E>
__global__ __launch_bounds__(kTopBlock) void topk_heads_kernel(TopArgs a) {
    using Stored = typename Row<W == 2 ? kRowF16 : kRowF32>::Stored;
    const int j = threadIdx.x % 16;
    constexpr uint64_t kRows = kTopBlock / 16;
    const uint32_t n = a.n, at = j * E;
    for (uint64_t base = blockIdx.x * kRows; base < a.rows; base += gridDim.x * kRows) {
        const uint64_t row = base + threadIdx.x / 16;
        int img[E];
        uint32_t order = 0;  // the places of the sorted elements within the lane, 4 bits each
        load_images<W, E>(static_cast<const Stored *>(a.x) + min(row, a.rows - 1) * a.stride, at, n, a.flip, img);
        int pos[E];
#pragma unroll
        for (int e = 0; e < E; ++e) pos[e] = e;
        // neighbours change places until none is out of order, so equal ones keep theirs
#pragma unroll
        for (int r = 0; r < E; ++r)
#pragma unroll
            for (int e = r & 1; e + 1 < E; e += 2) {
                const bool up = img[e] < img[e + 1];
                const int x = img[e], p = pos[e];
                img[e] = up ? img[e + 1] : x;
                img[e + 1] = up ? x : img[e + 1];
                pos[e] = up ? pos[e + 1] : p;
                pos[e + 1] = up ? p : pos[e + 1];
            }
#pragma unroll
        for (int e = 0; e < E; ++e) order |= static_cast<uint32_t>(pos[e]) << (4 * e);
        uint32_t left = at >= n ? 0 : min(n - at, static_cast<uint32_t>(E));
        int mine = 0, column = 0;
        for (uint32_t r = 0; r < a.k; ++r) {
            const int top = row16_max(img[0]);
            // an element past the row's end has the lowest image; a real one of that image is still left
            const int first = ~row16_max(img[0] == top && left > 0 ? ~j : INT32_MIN);
            const bool here = first == j;
            // the column from the lane that holds it, to the lane that writes it
            const int c = row16_max(here ? static_cast<int>(at + (order & 15u)) : -1);
            if (j == static_cast<int>(r)) {
                mine = top;
                column = c;
            }
            if (here) {
#pragma unroll
                for (int e = 0; e + 1 < E; ++e) img[e] = img[e + 1];
                img[E - 1] = INT32_MIN;
                order >>= 4;
                --left;
            }
        }
        if (row < a.rows && j < static_cast<int>(a.k)) {
            const uint64_t out = row * a.k + j;
            if (W == 2)
                static_cast<uint16_t *>(a.values)[out] = static_cast<uint16_t>(pattern_of<2>(mine, a.flip));
            else
                static_cast<uint32_t *>(a.values)[out] = pattern_of<4>(mine, a.flip);
            a.indices[out] = column;
        }
    }
}

// Rows of at most 64 * V loads and k <= 64: a wave a row, held in registers.
// A bisection over the lanes' largest images, and over all where that leaves
// too many, finds a bound that at least k and at most 64 elements reach; those
// move to a lane each and count the words above theirs, which is their place.
template <int W, int V>
__global__ __launch_bounds__(kTopBlock) void topk_wave_kernel(TopArgs a) {
    constexpr int kVec = 16 / W;
    constexpr int kLowest = W == 2 ? -32768 : INT32_MIN;
    using Word = ShortWord<W>;
    using Stored = typename Row<W == 2 ? kRowF16 : kRowF32>::Stored;
    __shared__ typename Word::T held[kTopBlock / kLanes][kLanes];
    const int lane = threadIdx.x % kLanes, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    constexpr uint64_t kRows = kTopBlock / kLanes;
    const uint32_t n = a.n, k = a.k;
    const uint32_t lanes = min(static_cast<uint32_t>(kLanes), (n + kVec - 1) / kVec);  // that hold elements
    const uint32_t enough = min(max(16u, 2 * k), static_cast<uint32_t>(kLanes));
    for (uint64_t row = blockIdx.x * kRows + wave; row < a.rows; row += gridDim.x * kRows) {
        const Stored *x = static_cast<const Stored *>(a.x) + row * a.stride;
        int img[V][kVec];
        int most = INT32_MIN;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            load_images<W, kVec>(x, (u * kLanes + lane) * kVec, n, a.flip, img[u]);
#pragma unroll
            for (int e = 0; e < kVec; ++e) most = max(most, img[u][e]);
        }
        auto reach = [&](int bound) {
            uint32_t c = 0;
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int e = 0; e < kVec; ++e) c += __popcll(__ballot(img[u][e] >= bound));
            return bound == INT32_MIN ? n : c;
        };
        // at least k elements reach lo, and fewer than k anything above hi
        int hi = wave_max_int(most), lo = kLowest;
        uint32_t c = n;
        if (lanes >= k) {
            lo = ~wave_max_int(lane < static_cast<int>(lanes) ? ~most : INT32_MIN);
            uint32_t reached = lanes;
            int top = hi;
            while (reached > k + k / 4 && lo < top) {
                const int mid = (lo | top) - ((lo ^ top) >> 1);
                const uint32_t m = __popcll(__ballot(most >= mid));
                reached = m >= k ? m : reached;
                lo = m >= k ? mid : lo;
                top = m >= k ? top : mid - 1;
            }
            c = reach(lo);
        }
        while (c > enough && lo < hi) {
            const int mid = (lo | hi) - ((lo ^ hi) >> 1);
            const uint32_t m = reach(mid);
            c = m >= k ? m : c;
            lo = m >= k ? mid : lo;
            hi = m >= k ? hi : mid - 1;
        }
        // more than 64 left: their images are equal but for fewer than k above
        const bool ties = c > kLanes;
        uint32_t count = 0;
        if (!ties || lo < INT32_MAX) {
            const int bound = ties ? lo + 1 : lo;
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const uint32_t at = (u * kLanes + lane) * kVec + e;
                    const bool in = at < n && img[u][e] >= bound;
                    const uint64_t mask = __ballot(in);
                    if (mask == 0) continue;
                    if (in) held[wave][count + lanes_below(mask)] = Word::make(img[u][e], at);
                    count += __popcll(mask);
                }
        }
        if (ties) {  // the first of the equal ones, one after the other
            int next = -1;
            while (count < k) {
                int first = INT32_MIN;  // the complement of the lowest column after `next`
#pragma unroll
                for (int u = 0; u < V; ++u)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        const int at = (u * kLanes + lane) * kVec + e;
                        if (at < static_cast<int>(n) && at > next && img[u][e] == lo) first = max(first, ~at);
                    }
                next = ~wave_max_int(first);
                if (lane == 0) held[wave][count] = Word::make(lo, next);
                ++count;
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const typename Word::T w = lane < static_cast<int>(count) ? held[wave][lane] : 0;
        __builtin_amdgcn_wave_barrier();
        uint32_t place = 0;
        for (uint32_t j = 0; j < count; j += 4)  // the words of lanes past the last are 0
#pragma unroll
            for (int i = 0; i < 4; ++i) place += Word::lane(w, j + i) > w;
        if (lane < static_cast<int>(count) && place < k) write_short<W>(a, w, row * k + place);
    }
}

// The k largest of a row's splits * k words.
template <int W>
__global__ __launch_bounds__(kTopBlock) void topk_merge_kernel(TopArgs a) {
    __shared__ uint64_t buf[kTopBuffer];
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const uint32_t total = a.splits * a.k;  // at most kTopBuffer
        const uint64_t *in = a.words + row * total;
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < total; i += kTopBlock) buf[i] = in[i];
        sort_words(buf, total);
        write_row<W>(a, buf, row, a.k);
    }
}

// Rows that one wave, or part of one, sorts in registers.
constexpr uint64_t kWaveVecs = 8;  // 16-byte loads a lane at most
bool topk_short(uint64_t n, uint64_t k, uint64_t size) {
    return n <= kLanes || (k <= kLanes && n <= kLanes * kWaveVecs * 16 / size);
}

template <int W> void launch_short(const TopArgs &a, const Launch &L) {
    const auto grid = [&](uint64_t rows_each) {
        return dim3(static_cast<uint32_t>(std::min<uint64_t>((a.rows + rows_each - 1) / rows_each, 1u << 20)));
    };
    const dim3 block(kTopBlock);
    if (a.n <= 8) return launch_on(topk_lanes_kernel<W, 8>, grid(kTopBlock / 8), block, L, a);
    if (a.n <= 16) return launch_on(topk_lanes_kernel<W, 16>, grid(kTopBlock / 16), block, L, a);
    if (a.n <= 128 && a.k <= 16) {
        if (W == 4 && a.n <= 64) return launch_on(topk_heads_kernel<W, 16 / W>, grid(kTopBlock / 16), block, L, a);
        return launch_on(topk_heads_kernel<W, 8>, grid(kTopBlock / 16), block, L, a);
    }
    if (a.n <= 32) return launch_on(topk_lanes_kernel<W, 32>, grid(kTopBlock / 32), block, L, a);
    if (a.n <= 64) return launch_on(topk_lanes_kernel<W, 64>, grid(kTopBlock / 64), block, L, a);
    const uint64_t vecs = (a.n + kLanes * 16 / W - 1) / (kLanes * 16 / W);
    const dim3 waves = grid(kTopBlock / kLanes);
    if (vecs <= 1) return launch_on(topk_wave_kernel<W, 1>, waves, block, L, a);
    if (vecs <= 2) return launch_on(topk_wave_kernel<W, 2>, waves, block, L, a);
    if (vecs <= 4) return launch_on(topk_wave_kernel<W, 4>, waves, block, L, a);
    launch_on(topk_wave_kernel<W, 8>, waves, block, L, a);
}

// How many workgroups share a row: enough that few rows still occupy the GPU,
// each with a piece worth a workgroup, and no more words than one merges.
uint32_t topk_splits(uint64_t rows, uint64_t n, uint64_t k) {
    if (rows == 0 || rows >= 256) return 1;
    const uint64_t piece = std::max<uint64_t>(4096, 8 * k);
    uint64_t s = std::min<uint64_t>((512 + rows - 1) / rows, n / piece);
    s = std::min<uint64_t>(s, kTopBuffer / k);
    return static_cast<uint32_t>(std::max<uint64_t>(1, s));
}

int check_topk(int64_t rows, int64_t n, int64_t k, int64_t stride, int dtype) {
    if (!row_type_ok(dtype)) return LRS_ERR_DTYPE;
    if (rows < 0 || n < 0 || k < 0 || !stride_ok(stride, rows)) return LRS_ERR_SIZE;
    if (static_cast<uint64_t>(n) > LRS_MAX_ROW_LEN || k > n || k > LRS_MAX_TOPK) return LRS_ERR_SIZE;
    if (n > 0 && static_cast<uint64_t>(rows) >= (uint64_t(1) << 40) / static_cast<uint64_t>(n)) return LRS_ERR_SIZE;
    return LRS_OK;
}

uint64_t topk_bytes(uint64_t rows, uint64_t n, uint64_t k, uint64_t size) {
    if (rows == 0 || k == 0 || topk_short(n, k, size)) return 0;
    const uint64_t s = topk_splits(rows, n, k);
    return s > 1 ? rows * s * k * sizeof(uint64_t) : 0;
}

}  // namespace
}  // namespace lrs

using namespace lrs;

extern "C" {

size_t segmented_row_topk_workspace_size(int64_t rows, int64_t n, int64_t k, int dtype, const lrs_options *opts) {
    if (!options_ok(opts) || check_topk(rows, n, k, n, dtype) != LRS_OK) return 0;
    return static_cast<size_t>(topk_bytes(rows, n, k, row_type_size(dtype)));
}

int segmented_row_topk(const void *x, int64_t row_stride, void *vals_out, int64_t *idx_out, int64_t rows, int64_t n,
                       int64_t k, int dtype, int descending, void *workspace, size_t workspace_bytes, void *stream,
                       const lrs_options *opts) try {
    Ctx c;
    if (!make_ctx(stream, opts, c)) return LRS_ERR_OPTION;
    const int st = check_topk(rows, n, k, row_stride, dtype);
    if (st != LRS_OK) return st;
    if (rows == 0 || k == 0) return LRS_OK;
    const uint64_t R = rows, N = n, K = k, size = row_type_size(dtype);
    const uint64_t need = topk_bytes(R, N, K, size);
    if (!x || !vals_out || !idx_out || (need && !workspace)) return LRS_ERR_NULL_POINTER;
    if (misaligned(x, size) || misaligned(vals_out, size) || misaligned(idx_out, 8) ||
        (need && misaligned(workspace, 256)))
        return LRS_ERR_ALIGNMENT;
    if (workspace_bytes < need) return LRS_ERR_WORKSPACE_TOO_SMALL;
    const uint64_t xb = span(R, row_stride, N, size), vb = R * K * size, ib = R * K * 8;
    if (overlaps(vals_out, vb, x, xb) || overlaps(idx_out, ib, x, xb) || overlaps(vals_out, vb, idx_out, ib) ||
        overlaps(workspace, need, x, xb) || overlaps(workspace, need, vals_out, vb) ||
        overlaps(workspace, need, idx_out, ib))
        return LRS_ERR_ALIASING;

    c.elems = R * N;
    TopArgs a{};
    a.x = x;
    a.stride = static_cast<uint64_t>(row_stride);
    a.rows = R;
    a.n = static_cast<uint32_t>(N);
    a.k = static_cast<uint32_t>(K);
    a.splits = topk_splits(R, N, K);
    // whole 16-byte loads to a split
    a.split_len = static_cast<uint32_t>(((N + a.splits - 1) / a.splits + 7) / 8 * 8);
    a.splits = static_cast<uint32_t>((N + a.split_len - 1) / a.split_len);
    a.flip = descending ? 0u : ~0u;
    a.values = vals_out;
    a.indices = idx_out;
    a.words = static_cast<uint64_t *>(workspace);
    if (topk_short(N, K, size)) {
        TimedLaunch t(4, c);
        if (size == 2)
            launch_short<2>(a, t.L);
        else
            launch_short<4>(a, t.L);
        return hipGetLastError() == hipSuccess ? LRS_OK : LRS_ERR_HIP;
    }
    const dim3 grid(static_cast<uint32_t>(std::min<uint64_t>(R * a.splits, 1u << 20)));
    {
        TimedLaunch t(4, c);
        if (size == 2)
            launch_on(topk_kernel<2>, grid, dim3(kTopBlock), t.L, a);
        else
            launch_on(topk_kernel<4>, grid, dim3(kTopBlock), t.L, a);
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
    }
    if (a.splits > 1) {
        TimedLaunch t(4, c);
        const dim3 merge(static_cast<uint32_t>(R));
        if (size == 2)
            launch_on(topk_merge_kernel<2>, merge, dim3(kTopBlock), t.L, a);
        else
            launch_on(topk_merge_kernel<4>, merge, dim3(kTopBlock), t.L, a);
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
    }
    return LRS_OK;
} catch (...) {
    return LRS_ERR_HIP;
}

}  // extern "C"
