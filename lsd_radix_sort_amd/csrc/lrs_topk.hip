// lrs_topk.hip -- the first k columns of a row sort without the sort (gfx950).
//
// Each element becomes one 64-bit word, order image above, complemented column
// below, so the wanted elements are the k largest words, no two words are
// alike, and ties go to the lowest column whatever order the words arrive in.
// Every form looks for a bound that at least k elements reach and few more,
// and ranks only those.  A row must be read once; what else a form costs is its
// chain of dependent steps, so each keeps as many rows on a CU as it can.  By
// length: a lane network (n <= 64), lanes' sorted heads (n <= 128, k <= 16), a
// wave (n <= 1024, k <= 64), a workgroup (up to 256 KB), several workgroups and
// a merge, and streaming where the merge would not fit.
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
    uint64_t first_task;  // of this launch
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
template <int B> __device__ void sort_words(uint64_t *buf, uint32_t count) {
    uint32_t m = 2;
    while (m < count) m <<= 1;
    __syncthreads();
    for (uint32_t i = count + threadIdx.x; i < m; i += B) buf[i] = 0;
    __syncthreads();
    for (uint32_t size = 2; size <= m; size <<= 1)
        for (uint32_t d = size >> 1; d > 0; d >>= 1) {
            for (uint32_t t = threadIdx.x; t < m / 2; t += B) {
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

// Streaming, for rows (or shares of one) over 256 KB.  The k-th largest of the
// first chunk's per-load maxima bounds the row's k-th largest from below; only
// elements at or above the bound enter a buffer in LDS, and when the buffer is
// nearly full its k largest stay and the least of them becomes the bound.  The
// sorts bound it: 1024 x 65536 fp16, k = 64 took 78 us so, 30 us in the form
// for shorter rows below.
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
            sort_words<kTopBlock>(buf, count);
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
        sort_words<kTopBlock>(buf, c);
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
// A 16-bit image and the column fit one 32-bit word.  65536 x 8 takes as long as
// an empty launch (3 us); 65536 x 64 fp32 takes 22 us, 21 steps of 64-bit words,
// so small k goes to the form after next.
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

// E consecutive elements of a row as images, INT32_MIN past its end.
template <int W, int E> __device__ inline void load_images(const typename Row<W == 2 ? kRowF16 : kRowF32>::Stored *x,
                                                           uint32_t at, uint32_t n, uint32_t flip, int (&img)[E]) {
    constexpr int kVec = 16 / W;
    u32x4 v[E / kVec];
#pragma unroll
    for (int q = 0; q < E / kVec; ++q) {
        const uint32_t first = at + q * kVec;
        v[q] = u32x4{0, 0, 0, 0};
        if (first + kVec <= n) v[q] = load16(x + first);
        if (n % kVec != 0 && first < n && first + kVec > n)
            for (int e = 0; e < kVec; ++e) {
                const uint32_t pat = first + e < n ? x[first + e] : 0;
                if (W == 2) v[q][e / 2] |= pat << (16 * (e & 1));
                else v[q][e % 4] = pat;
            }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int q = i / kVec, e = i % kVec;
        const uint32_t pat = W == 2 ? (v[q][e / 2] >> (16 * (e & 1))) & 0xFFFFu : v[q][e % 4];
        img[i] = at + i < n ? image<W>(pat, flip) : INT32_MIN;
    }
}

// Rows of at most 16 * E elements and small k: 16 lanes a row, E consecutive
// elements a lane, sorted within the lane.  k times the 16 lanes' heads give
// the next largest, the lowest lane's where they are equal, and that lane
// moves on.  Bound by issue: the network within a lane once for four rows, some
// 25 instructions a head; 65536 x 64 fp32, k = 6 in 10 us (floor 4 us).
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
// Lanes' largest images are tried as a bound until one is reached by k to 2 k
// lanes; the elements that reach it, at most 64, move to a lane each and count
// the words above theirs, which is their place.  Where that leaves more than
// 64, a bisection over the images of all finds the bound.  Bound by issue, not
// memory: scalar steps count as much as vector ones, so the bound is looked
// for among the lanes (9 scalar instructions a try) and places are summed by
// lanes.  32768 x 256 fp32, k = 8: 13.8 us, 172 vector and 140 scalar
// instructions a row (a bisection in their place: 315 scalar, 21.5 us).
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
        const auto column = [&](int u, int e) { return static_cast<uint32_t>((u * kLanes + lane) * kVec + e); };
        int bound = kLowest;
        if (lanes >= k) {
            uint64_t left = ~uint64_t(0) >> (kLanes - lanes);
            while (left) {
                const int pivot = __builtin_amdgcn_readlane(most, __builtin_ctzll(left));
                const uint64_t reach = __ballot(most >= pivot);
                const uint32_t c = __popcll(reach);
                if (c < k) {
                    left &= ~reach;
                } else {
                    bound = pivot;
                    left &= c <= 2 * k ? 0 : __ballot(most > pivot);
                }
            }
        }
        // the elements that reach the bound: this lane's, and those of lanes below
        uint32_t own, upto, count;
        const auto add_up = [&]() {
            own = 0;
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int e = 0; e < kVec; ++e) own += img[u][e] >= bound;
            if (bound == INT32_MIN) {  // nor do the places past the row's end
                own = 0;
#pragma unroll
                for (int u = 0; u < V; ++u) own += min(max(static_cast<int>(n - column(u, 0)), 0), kVec);
            }
            upto = lanes_sum(own);
            count = __builtin_amdgcn_readlane(upto, kLanes - 1);
        };
        add_up();
        bool ties = false;
        int tied = 0;  // their image
        if (count > kLanes) {
            int lo = bound, hi = wave_max_int(most);  // fewer than k are above hi
            while (count > kLanes && lo < hi) {
                bound = (lo | hi) - ((lo ^ hi) >> 1);
                add_up();
                if (count >= k) lo = bound;
                else hi = bound - 1;
                if (count < k) count = kLanes + 1;
            }
            bound = lo;
            add_up();
            // more than 64 still: their images are equal but for fewer than k above
            ties = count > kLanes;
            if (ties) {
                tied = lo;
                count = 0;
                if (lo < INT32_MAX) {
                    bound = lo + 1;
                    add_up();
                }
            }
        }
        if (own && count) {
            uint32_t slot = upto - own;
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (img[u][e] >= bound && (bound != INT32_MIN || column(u, e) < n))
                        held[wave][slot++] = Word::make(img[u][e], column(u, e));
        }
        if (ties) {  // the first of the equal ones, one after the other
            int next = -1;
            while (count < k) {
                int first = INT32_MIN;  // the complement of the lowest column after `next`
#pragma unroll
                for (int u = 0; u < V; ++u)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        const int at = column(u, e);
                        if (at < static_cast<int>(n) && at > next && img[u][e] == tied) first = max(first, ~at);
                    }
                next = ~wave_max_int(first);
                if (lane == 0) held[wave][count] = Word::make(tied, next);
                ++count;
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const typename Word::T w = lane < static_cast<int>(count) ? held[wave][lane] : 0;
        __builtin_amdgcn_wave_barrier();
        // 32 bits order the words unless images are equal, which the sum of the
        // places would show; the words of lanes past the last are 0
        const uint32_t high = W == 2 ? static_cast<uint32_t>(w) : static_cast<uint32_t>(static_cast<uint64_t>(w) >> 32);
        const bool on = lane < static_cast<int>(count);
        uint32_t place = 0;
        for (uint32_t j = 0; j < count; j += 4)
#pragma unroll
            for (int i = 0; i < 4; ++i) place += static_cast<uint32_t>(__builtin_amdgcn_readlane(high, j + i)) > high;
        if (W == 4 && wave_sum(on ? place : 0) != count * (count - 1) / 2) {
            place = 0;
            for (uint32_t j = 0; j < count; ++j) place += Word::lane(w, j) > w;
        }
        if (on && place < k) write_short<W>(a, w, row * k + place);
    }
}

// ---- a row, or a piece of one, by one workgroup -------------------------------

// Bins of images below the largest, 2^shift images a bin; whoever lies lower
// is not counted.
constexpr uint32_t kBins = 2048, kCoarse = 64, kFine = kBins / kCoarse;
constexpr uint32_t kHeldWords = 2048;  // candidates in LDS; half of them where k is at most 512
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

// The candidates' places and their output, from buf[0, c), `want` of them wanted
// (c <= CAP), no image above `top` or below `low`.  Few count the words above
// theirs; more are dealt to bins in order first and count within their bin
// (300 of 512 threads: 3 us by counting all).
template <int W, int B, int CAP>
__device__ void write_ranked(const TopArgs &a, uint64_t *buf, Bins &bins, uint32_t *cells, uint32_t c, uint32_t want, int top,
                             int64_t low, uint64_t task, uint64_t row) {
    const auto put = [&](uint64_t w, uint32_t place) {
        if (a.splits == 1) {
            const uint64_t at = row * a.k + place;
            if (W == 2)
                static_cast<uint16_t *>(a.values)[at] = static_cast<uint16_t>(pattern_of<2>(image_of(w), a.flip));
            else
                static_cast<uint32_t *>(a.values)[at] = pattern_of<4>(image_of(w), a.flip);
            a.indices[at] = column_of(w);
        } else {
            a.words[task * a.k + place] = w;
        }
    };
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
    if (a.splits > 1)
        for (uint32_t j = want + tid; j < a.k; j += B) a.words[task * a.k + j] = 0;
}

// Whether the threads' largest elements give the bound: k of them at most half.
constexpr int kBatch = 4;
__host__ __device__ inline bool few_wanted(uint64_t want, uint64_t threads, uint64_t vecs) {
    return 2 * want <= (threads < vecs ? threads : vecs);
}

// One workgroup of B threads a row (or a split of one), V loads of 16 bytes a
// thread.  A histogram below the largest image, of the threads' largest images
// where k is at most half of them and of all elements otherwise (HOLD), gives a
// bound that at least k elements reach; they go to LDS as words.  Where ties
// leave too many, the k-th image is found exactly and the first of its columns
// fill up.  With HOLD the row stays in registers.  Without, only the largest
// image of each load does, and the few loads that reach the bound are read
// again: half the registers, so twice the rows on a CU, whose chains of barriers
// hide behind each other's loads (333 x 50021 fp32, k = 129: 16.4 us, 24.6 us
// held; 1024 x 65536 fp16, k = 64: 30.5 us = 4.4 TB/s, 33.4 us held; 512 x 131072
// fp32: 5.4 TB/s; 1 x 131072 bf16: 9 us, held 10.4 us).
template <int W, int B, int V, bool HOLD>
__global__ __launch_bounds__(B, HOLD ? 4 : 8) void topk_held_kernel(TopArgs a) {
    constexpr int kVec = 16 / W;
    using Stored = typename Row<W == 2 ? kRowF16 : kRowF32>::Stored;
    constexpr uint32_t kWords = HOLD ? kHeldWords : kHeldWords / 2;
    __shared__ uint64_t buf[kWords];
    __shared__ Bins bins;
    __shared__ int tops[B / kLanes];
    __shared__ uint32_t cells[B / kLanes];
    __shared__ uint32_t count;
    const uint32_t tid = threadIdx.x;
    const uint64_t task = a.first_task + xcd_chunk(blockIdx.x, gridDim.x);
    const uint64_t row = task / a.splits;
    const uint32_t first = static_cast<uint32_t>(task % a.splits) * a.split_len;
    const uint32_t len = min(a.split_len, a.n - first), want = min(a.k, len);
    const uint32_t vecs = len / kVec, rest = vecs * kVec + tid;
    const Stored *x = static_cast<const Stored *>(a.x) + row * a.stride + first;

    u32x4 v[HOLD ? V : 1];
    const auto below = [&](int u) { return static_cast<int>(tid) < static_cast<int>(vecs) - u * B; };
    const auto source = [&](int u) { return reinterpret_cast<const uint8_t *>(x + u * B * kVec) + tid * 16; };
    if constexpr (HOLD) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            v[u] = u32x4{0, 0, 0, 0};
            if (below(u)) v[u] = load16_once(source(u));
        }
    }
    const bool extra = rest < len;
    const int over = extra ? image<W>(x[rest], a.flip) : INT32_MIN;
    clear_bins<B>(bins);
    if (tid == 0) count = 0;

    // the largest of each load (not held: two 16-bit images to a word), of all
    int most[HOLD || W == 4 ? V : V / 2], top = over;
    if constexpr (HOLD) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            most[u] = below(u) ? vec_max<W>(v[u], a.flip) : INT32_MIN;
            top = max(top, most[u]);
        }
    } else {
#pragma unroll
        for (int b = 0; b < V; b += kBatch) {
            u32x4 t[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (below(b + u)) t[u] = load16(source(b + u));
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int m = below(b + u) ? vec_max<W>(t[u], a.flip) : W == 2 ? -32768 : INT32_MIN;
                top = max(top, below(b + u) ? m : top);
                if (W == 4) most[b + u] = m;
                else if (u % 2 == 0) most[(b + u) / 2] = m & 0xFFFF;
                else most[(b + u) / 2] |= m << 16;
            }
        }
    }
    const int mine = top;
    const bool some = extra || below(0);
    top = wave_max_int(top);
    if (tid % kLanes == 0) tops[tid / kLanes] = top;
    __syncthreads();
    for (int w = 0; w < B / kLanes; ++w) top = max(top, tops[w]);

    // f for every element of a load
    const auto each = [&](u32x4 w, uint32_t at, auto f) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const uint32_t pat = W == 2 ? (w[e / 2] >> (16 * (e & 1))) & 0xFFFFu : w[e % 4];
            f(image<W>(pat, a.flip), at + e);
        }
    };
    const auto place_of = [&](int u) { return (u * B + tid) * kVec; };
    // each pass makes the images anew: kept, they would take twice the registers
    const auto anew = [&]() {
#pragma unroll
        for (int u = 0; u < (HOLD ? V : 0); ++u) asm volatile("" : "+v"(v[u]));
    };
    anew();
    const bool by_thread = !HOLD || few_wanted(want, B, vecs);
    uint32_t shift = W == 2 ? 0 : 13, bin;
    for (;; shift += W == 2 ? 5 : 8) {  // at the second shift every image has a bin
        if (by_thread) {
            if (some) add_to_bins(bins, mine, top, shift);
        } else {
#pragma unroll
            for (int u = 0; u < (HOLD ? V : 0); ++u)
                if (below(u)) each(v[u], 0, [&](int img, uint32_t) { add_to_bins(bins, img, top, shift); });
            if (extra) add_to_bins(bins, over, top, shift);
        }
        anew();
        __syncthreads();
        bin = bin_of(bins, want);
        if (bin < kBins) break;
        __syncthreads();
        clear_bins<B>(bins);
        __syncthreads();
    }
    const int64_t low = static_cast<int64_t>(top) - ((static_cast<int64_t>(bin + 1) << shift) - 1);
    int bound = static_cast<int>(max(low, static_cast<int64_t>(W == 2 ? -32768 : INT32_MIN)));

    const auto take = [&](int img, uint32_t at) {
        if (img >= bound) {
            const uint32_t slot = atomicAdd(&count, 1u);
            if (slot < kWords) buf[slot] = word_of(img, first + at);
        }
    };
    if (mine >= bound && some) {
        if constexpr (HOLD) {
#pragma unroll
            for (int u = 0; u < V; ++u)
                if (most[u] >= bound && below(u)) each(v[u], place_of(u), take);
        } else {
            uint32_t hits = 0;  // loads that are read again: mostly one
#pragma unroll
            for (int u = 0; u < V; ++u) {
                const int m = W == 4 ? most[u] : u % 2 ? most[u / 2] >> 16 : static_cast<int16_t>(most[u / 2]);
                hits |= static_cast<uint32_t>(m >= bound && below(u)) << u;
            }
            while (hits) {
                const uint32_t at = (__builtin_ctz(hits) * B + tid) * kVec;
                hits &= hits - 1;
                each(load16(x + at), at, take);
            }
        }
        if (extra) take(over, rest);
    }
    __syncthreads();
    uint32_t c = count;
    if (c > kWords) {  // rare: the row is read again
        const auto again = [&](auto f) {
            for (uint32_t i = tid; i < vecs; i += B) each(load16(x + i * kVec), i * kVec, f);
            if (extra) f(over, rest);
        };
        // the k-th image: at least `want` reach lo, fewer pass hi
        int lo = bound, hi = by_thread ? top : min(static_cast<int64_t>(top), low + (int64_t(1) << shift) - 1);
        while (lo < hi) {
            const int mid = (lo | hi) - ((lo ^ hi) >> 1);
            uint32_t n = 0;
            again([&](int img, uint32_t) { n += img >= mid; });
            if (block_sum<B>(n, cells) >= want) lo = mid;
            else hi = mid - 1;
        }
        __syncthreads();
        if (tid == 0) count = 0;
        __syncthreads();
        if (lo < INT32_MAX) {
            bound = lo + 1;
            again(take);
        }
        bound = lo;
        __syncthreads();
        c = count;  // below `want`
        // the first columns of image lo: stripe by stripe, in the order of threads
        for (uint32_t base = 0; base <= vecs && c < want; base += B) {
            const uint32_t i = base + tid;
            // the elements after the last whole load are a stripe of their own threads' order
            const bool in = i < vecs, last = base + B > vecs;
            const u32x4 w = in ? load16(x + i * kVec) : u32x4{0, 0, 0, 0};
            const auto fill = [&](bool on, auto elements) {
                uint32_t here = 0;
                if (on) elements([&](int img, uint32_t) { here += img == lo; });
                const uint32_t upto = lanes_sum(here);
                __syncthreads();
                if (tid % kLanes == kLanes - 1) cells[tid / kLanes] = upto;
                __syncthreads();
                uint32_t at = c + upto - here, all = 0;
                for (uint32_t w = 0; w < B / kLanes; ++w) {
                    if (w < tid / kLanes) at += cells[w];
                    all += cells[w];
                }
                if (on) elements([&](int img, uint32_t column) {
                    if (img == lo) {
                        if (at < want) buf[at] = word_of(lo, first + column);
                        ++at;
                    }
                });
                c = min(c + all, want);
            };
            fill(in, [&](auto f) { each(w, i * kVec, f); });
            if (last) fill(extra, [&](auto f) { f(over, rest); });
        }
        __syncthreads();
    }
    write_ranked<W, B, kWords>(a, buf, bins, cells, c, want, top, bound, task, row);
}

// The k largest of a row's splits * k words, by the same bound: 1 x 131072 fp32
// in 16 splits takes 9 us with it, 37 us of sorting the words before.
constexpr int kMergeBlock = 1024;
template <int W>
__global__ __launch_bounds__(kMergeBlock) void topk_merge_kernel(TopArgs a) {
    constexpr int B = kMergeBlock, V = kTopBuffer / B;
    __shared__ uint64_t buf[kTopBuffer];
    __shared__ Bins bins;
    __shared__ int tops[B / kLanes];
    __shared__ uint32_t cells[B / kLanes];
    __shared__ uint32_t count;
    const uint64_t row = a.first_task + blockIdx.x;
    const uint32_t tid = threadIdx.x, total = a.splits * a.k;  // at most kTopBuffer
    const uint64_t *in = a.words + row * total;
    uint64_t w[V];
    int top = INT32_MIN;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        w[u] = u * B + tid < total ? in[u * B + tid] : 0;
        if (w[u]) top = max(top, image_of(w[u]));
    }
    clear_bins<B>(bins);
    if (tid == 0) count = 0;
    top = wave_max_int(top);
    if (tid % kLanes == 0) tops[tid / kLanes] = top;
    __syncthreads();
    for (int i = 0; i < B / kLanes; ++i) top = max(top, tops[i]);
    uint32_t shift = W == 2 ? 0 : 13, bin;
    for (;; shift += W == 2 ? 5 : 8) {
#pragma unroll
        for (int u = 0; u < V; ++u)
            if (w[u]) add_to_bins(bins, image_of(w[u]), top, shift);
        __syncthreads();
        bin = bin_of(bins, a.k);
        if (bin < kBins) break;
        __syncthreads();
        clear_bins<B>(bins);
        __syncthreads();
    }
    const int64_t low = static_cast<int64_t>(top) - ((static_cast<int64_t>(bin + 1) << shift) - 1);
#pragma unroll
    for (int u = 0; u < V; ++u)
        if (w[u] && image_of(w[u]) >= low) buf[atomicAdd(&count, 1u)] = w[u];
    __syncthreads();
    a.splits = 1;  // what is written is the row
    write_ranked<W, B, kTopBuffer>(a, buf, bins, cells, count, a.k, top, low, row, row);
}

// Rows that one wave, or part of one, sorts in registers.
constexpr uint64_t kWaveElems = 1024;
bool topk_short(uint64_t n, uint64_t k) {
    return n <= kLanes || (k <= kLanes && n <= kWaveElems);
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
    if constexpr (W == 4) launch_on(topk_wave_kernel<W, 4>, waves, block, L, a);
}

// Rows, or splits of rows, of at most 256 KB go to one workgroup.
constexpr uint64_t kHeldBytes = 1024 * 16 * 16;

// How many workgroups share a row: one where one can take it (1 x 131072 bf16:
// 9 us; in pieces of 32 KB 9.8 us and a second launch); else as many as leave each 256 KB, or, of few rows, 32 KB
// (1 x 131072 fp32: 9.3 us, 12.9 us in two pieces).  Their words have to fit the
// merge; rows too long for that are streamed.
uint32_t topk_splits(uint64_t rows, uint64_t n, uint64_t k, uint64_t size) {
    if (rows == 0 || n * size <= kHeldBytes) return 1;
    const uint64_t most = kTopBuffer / k, least = (n * size + kHeldBytes - 1) / kHeldBytes;
    const uint64_t few = rows <= 64 ? std::min<uint64_t>(256 / rows, n * size / 32768) : 1;
    return static_cast<uint32_t>(std::min<uint64_t>(most, std::max<uint64_t>(least, few)));
}

// Threads by the rows there are: workgroups of 1024 where there are no more
// than CUs, the fewest threads that take a row at 16 loads each where several
// share a CU.
template <int W> void launch_held(const TopArgs &a, uint32_t tasks, const Launch &L) {
    const uint64_t vecs = a.split_len / (16 / W);
    const uint64_t least = std::min<uint64_t>(a.split_len, a.n - (a.splits - 1) * uint64_t(a.split_len)) / (16 / W);
    const auto go = [&](auto held, auto again, int block) {
        launch_on(few_wanted(a.k, block, least) ? again : held, dim3(tasks), dim3(block), L, a);
    };
    if (a.rows * a.splits <= 256) {
        if (vecs <= 1024 * 4) return go(topk_held_kernel<W, 1024, 4, true>, topk_held_kernel<W, 1024, 4, false>, 1024);
        if (vecs <= 1024 * 8) return go(topk_held_kernel<W, 1024, 8, true>, topk_held_kernel<W, 1024, 8, false>, 1024);
        return go(topk_held_kernel<W, 1024, 16, true>, topk_held_kernel<W, 1024, 16, false>, 1024);
    }
    if (vecs <= 256 * 2) return go(topk_held_kernel<W, 256, 2, true>, topk_held_kernel<W, 256, 4, false>, 256);
    if (vecs <= 256 * 4) return go(topk_held_kernel<W, 256, 4, true>, topk_held_kernel<W, 256, 4, false>, 256);
    if (vecs <= 256 * 8) return go(topk_held_kernel<W, 256, 8, true>, topk_held_kernel<W, 256, 8, false>, 256);
    if (vecs <= 256 * 16) return go(topk_held_kernel<W, 256, 16, true>, topk_held_kernel<W, 256, 16, false>, 256);
    if (vecs <= 512 * 16) return go(topk_held_kernel<W, 512, 16, true>, topk_held_kernel<W, 512, 16, false>, 512);
    go(topk_held_kernel<W, 1024, 16, true>, topk_held_kernel<W, 1024, 16, false>, 1024);
}

int check_topk(int64_t rows, int64_t n, int64_t k, int64_t stride, int dtype) {
    if (!row_type_ok(dtype)) return LRS_ERR_DTYPE;
    if (rows < 0 || n < 0 || k < 0 || !stride_ok(stride, rows)) return LRS_ERR_SIZE;
    if (static_cast<uint64_t>(n) > LRS_MAX_ROW_LEN || k > n || k > LRS_MAX_TOPK) return LRS_ERR_SIZE;
    if (n > 0 && static_cast<uint64_t>(rows) >= (uint64_t(1) << 40) / static_cast<uint64_t>(n)) return LRS_ERR_SIZE;
    return LRS_OK;
}

uint64_t topk_bytes(uint64_t rows, uint64_t n, uint64_t k, uint64_t size) {
    if (rows == 0 || k == 0 || topk_short(n, k)) return 0;
    const uint64_t s = topk_splits(rows, n, k, size);
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
    a.splits = topk_splits(R, N, K, size);
    // whole 16-byte loads to a split
    a.split_len = static_cast<uint32_t>(((N + a.splits - 1) / a.splits + 7) / 8 * 8);
    a.splits = static_cast<uint32_t>((N + a.split_len - 1) / a.split_len);
    a.flip = descending ? 0u : ~0u;
    a.values = vals_out;
    a.indices = idx_out;
    a.words = static_cast<uint64_t *>(workspace);
    if (topk_short(N, K)) {
        TimedLaunch t(4, c);
        if (size == 2)
            launch_short<2>(a, t.L);
        else
            launch_short<4>(a, t.L);
        return hipGetLastError() == hipSuccess ? LRS_OK : LRS_ERR_HIP;
    }
    constexpr uint64_t kMaxGrid = 1u << 20;
    const uint64_t tasks = R * a.splits;
    if (a.split_len * size <= kHeldBytes) {
        for (; a.first_task < tasks; a.first_task += kMaxGrid) {
            TimedLaunch t(4, c);
            const uint32_t now = static_cast<uint32_t>(std::min<uint64_t>(tasks - a.first_task, kMaxGrid));
            if (size == 2)
                launch_held<2>(a, now, t.L);
            else
                launch_held<4>(a, now, t.L);
            if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
        }
    } else {
        TimedLaunch t(4, c);
        const dim3 grid(static_cast<uint32_t>(std::min<uint64_t>(tasks, kMaxGrid)));
        if (size == 2)
            launch_on(topk_kernel<2>, grid, dim3(kTopBlock), t.L, a);
        else
            launch_on(topk_kernel<4>, grid, dim3(kTopBlock), t.L, a);
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
    }
    // a launch of 2^32 threads or more would wrap without an error
    for (a.first_task = 0; a.splits > 1 && a.first_task < R; a.first_task += kMaxGrid) {
        TimedLaunch t(4, c);
        const dim3 merge(static_cast<uint32_t>(std::min<uint64_t>(R - a.first_task, kMaxGrid)));
        if (size == 2)
            launch_on(topk_merge_kernel<2>, merge, dim3(kMergeBlock), t.L, a);
        else
            launch_on(topk_merge_kernel<4>, merge, dim3(kMergeBlock), t.L, a);
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
    }
    return LRS_OK;
} catch (...) {
    return LRS_ERR_HIP;
}

}  // extern "C"
