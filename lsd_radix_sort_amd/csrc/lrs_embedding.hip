// lrs_embedding.hip -- embedding lookup, and the gradient of its table by
// sorted tokens (gfx950).
//
// out[t] = scale W[id_t]; dW[v] = scale * sum of g[t] over the tokens with id_t =
// v.  The sum over the tokens of one id is a segmented sum once the pairs (id,
// place) are sorted, which the library's stable sort does; within an id the
// places then stand in order, so the sum has one order however the GPU runs it.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/lsd_radix_sort.h"
#include "lrs_host.h"
#include "lrs_rows.h"

namespace lrs {
namespace {

constexpr int kEmbBlock = 256;

struct Ids {
    const void *at;
    uint64_t stride;
    uint32_t length;
    int bytes;
    __device__ int64_t operator[](uint32_t t) const {
        const uint64_t i = t / length * stride + t % length;
        return bytes == 8 ? static_cast<const int64_t *>(at)[i] : static_cast<const int32_t *>(at)[i];
    }
};

// Eight elements as floats, and back, at any element alignment.
template <int T> __device__ inline void load8(const void *rows, uint64_t at, float (&f)[8]) {
    const auto *p = static_cast<const typename Row<T>::Stored *>(rows) + at;
    if constexpr (T == kRowF32) {
        const u32x4 a = load16(p), b = load16(p + 4);
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = a[i], v = b[i];
            f[i] = __builtin_bit_cast(float, u);
            f[4 + i] = __builtin_bit_cast(float, v);
        }
    } else {
        unpack16<T>(load16(p), f);
    }
}
template <int T> __device__ inline void store8(void *rows, uint64_t at, const float (&f)[8]) {
    auto *p = static_cast<typename Row<T>::Stored *>(rows) + at;
    if constexpr (T == kRowF32) {
        const float a[4] = {f[0], f[1], f[2], f[3]}, b[4] = {f[4], f[5], f[6], f[7]};
        store16(p, pack16<kRowF32>(a));
        store16(p + 4, pack16<kRowF32>(b));
    } else {
        store16(p, pack16<T>(f));
    }
}

// ------------------------------------------------------------------ lookup

struct LookupArgs {
    const void *weight;
    uint64_t weight_stride;
    Ids ids;
    void *out;
    uint64_t out_stride;
    uint32_t tokens, vocab, width;
    float scale;
};

template <int T, int O>
__global__ __launch_bounds__(kEmbBlock) void lookup_kernel(LookupArgs a) {
    const uint32_t pieces = (a.width + 7) / 8;
    const uint64_t all = static_cast<uint64_t>(a.tokens) * pieces;
    for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * kEmbBlock + threadIdx.x; u < all;
         u += static_cast<uint64_t>(gridDim.x) * kEmbBlock) {
        const uint32_t t = static_cast<uint32_t>(u / pieces), first = static_cast<uint32_t>(u % pieces) * 8;
        const int64_t id = a.ids[t];
        const bool inside = id >= 0 && id < a.vocab;
        const uint64_t from = inside ? id * a.weight_stride + first : 0, to = t * a.out_stride + first;
        if (first + 8 <= a.width) {
            float f[8] = {};
            if (inside) load8<T>(a.weight, from, f);
            for (int i = 0; i < 8; ++i) f[i] = inside ? f[i] * a.scale : 0.f;
            store8<O>(a.out, to, f);
        } else {
            for (uint32_t i = 0; first + i < a.width; ++i) {
                float f = 0.f;
                if (inside) f = Row<T>::value(static_cast<const typename Row<T>::Stored *>(a.weight)[from + i]) * a.scale;
                static_cast<typename Row<O>::Stored *>(a.out)[to + i] = Row<O>::pattern(f);
            }
        }
    }
}

// ---------------------------------------------------------------- gradient
//
// After the sort the tokens of an id are neighbours, so the gradient is three
// kinds of work, one launch for all: the sums of ids with few tokens, the sums
// of those with many, and the rows of ids with none, which are cleared.  Text
// has a few ids that make up a large share of it, so no wave sums more than
// some 2 kRun rows: an id with a whole aligned run of kRun places is `long`, its
// whole runs are summed by a wave each beforehand (in 32 bits, by place), and a
// workgroup adds those and what is left at both ends.

constexpr uint32_t kRun = 32;
constexpr uint32_t kNoKey = ~0u;

struct GradArgs {
    const void *grad;
    uint64_t grad_stride;
    Ids ids;
    void *out;
    uint64_t out_stride;
    uint32_t tokens, vocab, width;
    float scale;
    int64_t padding;
    int accumulate;
    uint32_t *keys, *places;              // unsorted
    const uint32_t *sorted, *order;       // the sorted keys and their places
    uint32_t *present;                    // a bit for every id, set where a token names it
    uint32_t *longs;                      // how many ids are long, then the first whole run of each
    float *runs;                          // [tokens / kRun][width]: sums of whole runs
    uint32_t pieces;                      // of a row, a group of lanes each
    uint32_t chunk;                       // sorted places whose ids one group sums
    uint32_t long_blocks, few_blocks;     // of the sums' launch; the others clear rows
};

// The keys of the sort: ids, those that count for nothing behind the last.
__global__ __launch_bounds__(kEmbBlock) void embed_keys_kernel(GradArgs a) {
    const uint32_t t = blockIdx.x * kEmbBlock + threadIdx.x;
    if (t == 0) a.longs[0] = 0;
    if (!a.accumulate)
        for (uint32_t w = t; w < (a.vocab + 31) / 32; w += gridDim.x * kEmbBlock) a.present[w] = 0;
    if (t >= a.tokens) return;
    const int64_t id = a.ids[t];
    a.keys[t] = id >= 0 && id < a.vocab && id != a.padding ? static_cast<uint32_t>(id) : a.vocab;
    a.places[t] = t;
}

// What a lane holds of a row: eight columns, fewer at the row's end.
struct Columns {
    uint32_t first, count;
    __device__ Columns(uint32_t piece, uint32_t lanes, uint32_t lane, uint32_t width) {
        first = (piece * lanes + lane) * 8;
        count = first < width ? min(width - first, 8u) : 0;
    }
};
template <int T> __device__ inline void load_columns(const void *rows, uint64_t row, Columns c, float (&f)[8]) {
    if (c.count == 8) {
        load8<T>(rows, row + c.first, f);
    } else {
        const auto *p = static_cast<const typename Row<T>::Stored *>(rows) + row + c.first;
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e) f[e] = e < c.count ? Row<T>::value(p[e]) : 0.f;
    }
}
// A finished sum to the table's gradient.
template <int O> __device__ inline void put_row(const GradArgs &a, uint32_t id, Columns c, const float (&sum)[8]) {
    const uint64_t row = id * a.out_stride;
    float f[8] = {};
    if (a.accumulate) load_columns<O>(a.out, row, c, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = a.accumulate ? fmaf(sum[e], a.scale, f[e]) : sum[e] * a.scale;
    if (c.count == 8) {
        store8<O>(a.out, row + c.first, f);
    } else {
        auto *p = static_cast<typename Row<O>::Stored *>(a.out) + row + c.first;
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e)
            if (e < c.count) p[e] = Row<O>::pattern(f[e]);
    }
}
template <int LANES> __device__ inline uint32_t uniform(uint32_t v) {
    return LANES == kLanes ? __builtin_amdgcn_readfirstlane(v) : v;
}

// Marks the ids that tokens name, lists the long ones and sums their whole runs.
template <int T, int LANES>
__global__ __launch_bounds__(kEmbBlock) void embed_runs_kernel(GradArgs a) {
    constexpr uint32_t kGroups = kEmbBlock / LANES;
    const uint32_t marking = (a.tokens + kEmbBlock - 1) / kEmbBlock, runs = a.tokens / kRun;
    if (blockIdx.x < marking) {
        const uint32_t i = blockIdx.x * kEmbBlock + threadIdx.x;
        if (i >= a.tokens) return;
        const uint32_t key = a.sorted[i];
        if (key >= a.vocab) return;
        if (!a.accumulate && (i == 0 || a.sorted[i - 1] != key)) atomicOr(&a.present[key / 32], 1u << (key % 32));
        if (i % kRun == 0 && i + kRun <= a.tokens && a.sorted[i + kRun - 1] == key && (i == 0 || a.sorted[i - kRun] != key))
            a.longs[1 + atomicAdd(&a.longs[0], 1u)] = i / kRun;
        return;
    }
    const uint64_t tasks = static_cast<uint64_t>(runs) * a.pieces, groups = static_cast<uint64_t>(gridDim.x - marking) * kGroups;
    for (uint64_t task = static_cast<uint64_t>(blockIdx.x - marking) * kGroups + threadIdx.x / LANES; task < tasks; task += groups) {
        const uint32_t run = uniform<LANES>(static_cast<uint32_t>(task / a.pieces)), piece = uniform<LANES>(static_cast<uint32_t>(task % a.pieces));
        const uint32_t *key = a.sorted + static_cast<uint64_t>(run) * kRun, *order = a.order + static_cast<uint64_t>(run) * kRun;
        if (key[0] != key[kRun - 1] || key[0] >= a.vocab) continue;
        const Columns c(piece, LANES, threadIdx.x % LANES, a.width);
        constexpr uint32_t kAtOnce = T == kRowF32 ? 8 : 16;
        float sum[8] = {};
#pragma unroll 1
        for (uint32_t i = 0; i < kRun; i += kAtOnce) {
            float f[kAtOnce][8];
#pragma unroll
            for (uint32_t j = 0; j < kAtOnce; ++j) load_columns<T>(a.grad, order[i + j] * a.grad_stride, c, f[j]);
#pragma unroll
            for (uint32_t j = 0; j < kAtOnce; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += f[j][e];
        }
        float *out = a.runs + static_cast<uint64_t>(run) * a.width + c.first;
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e)
            if (e < c.count) out[e] = sum[e];
    }
}

// The long id `which`: a workgroup, whose groups take the whole runs in equal
// shares, the first one also the places before them, the last one those after.
template <int T, int O, int LANES> __device__ void sum_long(const GradArgs &a, uint32_t which, uint32_t piece) {
    constexpr uint32_t kGroups = kEmbBlock / LANES;
    __shared__ float parts[kGroups][LANES * 8];
    const uint32_t lane = threadIdx.x % kLanes, group = threadIdx.x / LANES;
    const uint32_t first = __builtin_amdgcn_readfirstlane(a.longs[1 + which]), key = a.sorted[first * kRun];
    const Columns c(piece, LANES, threadIdx.x % LANES, a.width);
    uint32_t runs = 1;  // whole ones
    for (;;) {
        const uint64_t end = (static_cast<uint64_t>(first) + runs + lane + 1) * kRun;
        const uint64_t same = __ballot(end <= a.tokens && a.sorted[end - 1] == key);
        const uint32_t more = same == ~uint64_t(0) ? kLanes : __builtin_ctzll(~same);
        runs += more;
        if (more < kLanes) break;
    }
    const uint32_t from = first * kRun, to = from + runs * kRun;
    const uint32_t before = __popcll(__ballot(lane < kRun && from > lane && a.sorted[from - 1 - lane] == key));
    const uint32_t after = __popcll(__ballot(lane < kRun && a.tokens - to > lane && a.sorted[to + lane] == key));
    float sum[8] = {};
    const auto add_rows = [&](uint32_t i, uint32_t end) {
        for (; i < end; i += 4) {
            float f[4][8];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
                if (i + j < end) load_columns<T>(a.grad, a.order[i + j] * a.grad_stride, c, f[j]);
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
                if (i + j < end)
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[e] += f[j][e];
        }
    };
    if (group == 0) add_rows(from - before, from);
    const uint32_t share = (runs + kGroups - 1) / kGroups, mine = min(group * share, runs), next = min(mine + share, runs);
    for (uint32_t r = mine; r < next; r += 4) {
        float f[4][8];
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
            if (r + j < next) load_columns<kRowF32>(a.runs, static_cast<uint64_t>(first + r + j) * a.width, c, f[j]);
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
            if (r + j < next)
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += f[j][e];
    }
    if (group == kGroups - 1) add_rows(to, to + after);
    __syncthreads();  // the last task's readers are done
#pragma unroll
    for (int e = 0; e < 8; ++e) parts[group][e * LANES + threadIdx.x % LANES] = sum[e];
    __syncthreads();
    if (group == 0) {
        for (uint32_t g = 1; g < kGroups; ++g)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += parts[g][e * LANES + threadIdx.x % LANES];
        put_row<O>(a, key, c, sum);
    }
}

// The ids whose first place is among `chunk` sorted ones from `begin` on, but
// for the long ones: a group of lanes, four rows on their way at a time.
template <int T, int O, int LANES> __device__ void sum_few(const GradArgs &a, uint32_t begin, uint32_t piece) {
    const Columns c(piece, LANES, threadIdx.x % LANES, a.width);
    const uint32_t last = a.tokens - 1, end = min(begin + a.chunk, a.tokens);
    uint32_t previous = begin == 0 ? kNoKey : a.sorted[begin - 1], id = kNoKey;  // id: of the sum under way
    float sum[8] = {};
    for (uint32_t i = begin; i < end || id != kNoKey; i += 4) {
        // keys at the end of the run that would make an id starting here long
        const uint32_t next = (i / kRun + 1) * kRun + kRun - 1;
        const uint32_t far = next <= last ? uniform<LANES>(a.sorted[next]) : kNoKey;
        const uint32_t near = i % kRun == 0 && i + kRun - 1 <= last ? uniform<LANES>(a.sorted[i + kRun - 1]) : kNoKey;
        uint32_t owner[4], at[4];
        bool head[4], done = false;
        uint32_t now = id;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t key = i + j <= last ? uniform<LANES>(a.sorted[i + j]) : kNoKey;
            at[j] = i + j <= last ? uniform<LANES>(a.order[i + j]) : 0;
            head[j] = key != previous;
            previous = key;
            done |= head[j] && i + j >= end;
            if (head[j]) now = done || key >= a.vocab || key == (j == 0 && i % kRun == 0 ? near : far) ? kNoKey : key;
            owner[j] = now;
        }
        float f[4][8];
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
            if (owner[j] != kNoKey) load_columns<T>(a.grad, at[j] * a.grad_stride, c, f[j]);
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            if (head[j]) {
                if (id != kNoKey) put_row<O>(a, id, c, sum);
                id = owner[j];
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] = 0.f;
            }
            if (id != kNoKey)
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += f[j][e];
        }
    }
}

// Clears the rows of 32 ids that no token names.
template <int O> __device__ void clear_rows(const GradArgs &a, uint32_t word, uint32_t piece) {
    constexpr uint32_t kPiece = kEmbBlock;  // eights of columns
    const uint32_t all = (a.width + 7) / 8, first = piece * kPiece, eights = min(kPiece, all - first);
    const uint32_t present = a.tokens ? a.present[word] : 0;
    for (uint32_t u = threadIdx.x; u < 32 * eights; u += kEmbBlock) {
        const uint32_t r = u / eights, id = word * 32 + r, col = (first + u % eights) * 8;
        if (id >= a.vocab || ((present >> r) & 1)) continue;
        auto *p = static_cast<typename Row<O>::Stored *>(a.out) + id * a.out_stride + col;
        if (col + 8 <= a.width) {
            store16_once(p, u32x4{0, 0, 0, 0});
            if (O == kRowF32) store16_once(p + 4, u32x4{0, 0, 0, 0});
        } else {
            for (uint32_t e = 0; col + e < a.width; ++e) p[e] = 0;
        }
    }
}

template <int T, int O, int LANES>
__global__ __launch_bounds__(kEmbBlock) void embed_sum_kernel(GradArgs a) {
    constexpr uint32_t kGroups = kEmbBlock / LANES;
    uint32_t block = blockIdx.x;
    if (block < a.long_blocks) {
        const uint64_t tasks = static_cast<uint64_t>(a.longs[0]) * a.pieces;
        for (uint64_t t = block; t < tasks; t += a.long_blocks)
            sum_long<T, O, LANES>(a, static_cast<uint32_t>(t / a.pieces), static_cast<uint32_t>(t % a.pieces));
        return;
    }
    block -= a.long_blocks;
    if (block < a.few_blocks) {
        const uint64_t chunks = (a.tokens + a.chunk - 1) / a.chunk, tasks = chunks * a.pieces;
        for (uint64_t t = static_cast<uint64_t>(block) * kGroups + threadIdx.x / LANES; t < tasks; t += static_cast<uint64_t>(a.few_blocks) * kGroups)
            sum_few<T, O, LANES>(a, uniform<LANES>(static_cast<uint32_t>(t / a.pieces)) * a.chunk, uniform<LANES>(static_cast<uint32_t>(t % a.pieces)));
        return;
    }
    block -= a.few_blocks;
    const uint32_t pieces = ((a.width + 7) / 8 + kEmbBlock - 1) / kEmbBlock, words = (a.vocab + 31) / 32;
    const uint64_t tasks = static_cast<uint64_t>(words) * pieces, blocks = gridDim.x - a.long_blocks - a.few_blocks;
    for (uint64_t t = block; t < tasks; t += blocks) clear_rows<O>(a, static_cast<uint32_t>(t / pieces), static_cast<uint32_t>(t % pieces));
}

// -------------------------------------------------------------------- host

constexpr uint64_t kMaxGrid = 1u << 20;

int check_sizes(int64_t tokens, int64_t vocab, int64_t width) {
    if (tokens < 0 || vocab < 0 || width < 0 || tokens > INT32_MAX || vocab >= INT32_MAX ||
        static_cast<uint64_t>(width) > LRS_MAX_ROW_LEN)
        return LRS_ERR_SIZE;
    const uint64_t rows = static_cast<uint64_t>(std::max(tokens, vocab));
    if (width > 0 && rows >= (uint64_t(1) << 40) / static_cast<uint64_t>(width)) return LRS_ERR_SIZE;
    return LRS_OK;
}

// Checks the ids; gives their number.
int check_ids(const lrs_token_ids *t, Ids &ids, int64_t &tokens) {
    if (t == nullptr) return LRS_ERR_NULL_POINTER;
    if (t->id_bytes != 4 && t->id_bytes != 8) return LRS_ERR_DTYPE;
    if (t->lines < 0 || t->length < 0 || (t->length > 0 && t->lines > INT32_MAX / t->length) || t->length > INT32_MAX ||
        !stride_ok(t->stride, t->lines))
        return LRS_ERR_SIZE;
    tokens = t->lines * t->length;
    if (tokens > 0 && t->ids == nullptr) return LRS_ERR_NULL_POINTER;
    if (misaligned(t->ids, t->id_bytes)) return LRS_ERR_ALIGNMENT;
    ids = Ids{t->ids, static_cast<uint64_t>(t->stride), static_cast<uint32_t>(t->length), t->id_bytes};
    return LRS_OK;
}
uint64_t id_span(const lrs_token_ids *t) { return span(t->lines, t->stride, t->length, t->id_bytes); }

// f for the two types, as template arguments.
template <typename F> void by_type(int type, F f) {
    if (type == LRS_DTYPE_FP16) f(std::integral_constant<int, kRowF16>());
    else if (type == LRS_DTYPE_BF16) f(std::integral_constant<int, kRowBF16>());
    else f(std::integral_constant<int, kRowF32>());
}
template <typename F> void by_types(int in, int out, F f) {
    by_type(in, [&](auto t) { by_type(out, [&](auto o) { f(t, o); }); });
}

struct GradSpace {
    uint64_t keys = 0, places = 0, sorted = 0, order = 0, sort = 0, sort_bytes = 0, present = 0, longs = 0, runs = 0, total = 0;
};
int key_bits(uint64_t vocab) {
    int b = 1;
    while ((vocab >> b) != 0) ++b;  // keys are at most vocab
    return b;
}
GradSpace grad_space(uint64_t tokens, uint64_t vocab, uint64_t width, const lrs_options *opts) {
    GradSpace w;
    if (tokens == 0) return w;
    auto place = [&](uint64_t bytes) {
        const uint64_t at = w.total;
        w.total += (bytes + 255) / 256 * 256;
        return at;
    };
    w.keys = place(4 * tokens);
    w.places = place(4 * tokens);
    w.sorted = place(4 * tokens);
    w.order = place(4 * tokens);
    w.sort_bytes = radix_sort_workspace_size(tokens, 0, key_bits(vocab), 8, 1, opts);
    w.sort = place(w.sort_bytes);
    w.present = place((vocab + 31) / 32 * 4);
    w.longs = place(4 * (1 + tokens / kRun));
    w.runs = place(tokens / kRun * width * 4);
    return w;
}

// Rows of at most 128 columns take a quarter of a wave.
template <int T, int O, int LANES> void launch_sums(GradArgs a, const Ctx &c) {
    constexpr uint64_t kGroups = kEmbBlock / LANES;
    const auto blocks = [](uint64_t tasks, uint64_t each) { return (tasks + each - 1) / each; };
    a.pieces = static_cast<uint32_t>(blocks(a.width, LANES * 8));
    // few tokens: more groups, with fewer places each
    a.chunk = static_cast<uint64_t>(a.tokens) * a.pieces < 16384 ? 4 : 16;
    const uint64_t runs = a.tokens / kRun;
    if (a.tokens > 0 && (runs > 0 || !a.accumulate)) {
        TimedLaunch t(4, c);
        const uint64_t grid = blocks(a.tokens, kEmbBlock) + std::min(blocks(runs * a.pieces, kGroups), kMaxGrid);
        launch_on(embed_runs_kernel<T, LANES>, dim3(static_cast<uint32_t>(grid)), dim3(kEmbBlock), t.L, a);
        if (hipPeekAtLastError() != hipSuccess) return;
    }
    a.long_blocks = static_cast<uint32_t>(std::min<uint64_t>(runs * a.pieces, 512));
    a.few_blocks = static_cast<uint32_t>(std::min(blocks(blocks(a.tokens, a.chunk) * a.pieces, kGroups), kMaxGrid));
    uint64_t grid = a.long_blocks + a.few_blocks;
    if (!a.accumulate) grid += std::min(blocks(a.vocab, 32) * blocks(a.width, 8 * kEmbBlock), kMaxGrid);
    if (grid == 0) return;
    TimedLaunch t(4, c);
    launch_on(embed_sum_kernel<T, O, LANES>, dim3(static_cast<uint32_t>(grid)), dim3(kEmbBlock), t.L, a);
}

}  // namespace
}  // namespace lrs

using namespace lrs;

extern "C" {

int embedding_forward(const void *weight, int64_t weight_stride, const lrs_token_ids *tokens, void *out,
                      int64_t out_stride, int64_t vocab, int64_t width, int dtype, int out_dtype, float scale,
                      void *stream, const lrs_options *opts) try {
    Ctx c;
    if (!make_ctx(stream, opts, c) || !std::isfinite(scale)) return LRS_ERR_OPTION;
    if (!row_type_ok(dtype) || !row_type_ok(out_dtype)) return LRS_ERR_DTYPE;
    LookupArgs a{};
    int64_t count = 0;
    int st = check_ids(tokens, a.ids, count);
    if (st == LRS_OK) st = check_sizes(count, vocab, width);
    if (st != LRS_OK) return st;
    if (!stride_ok(weight_stride, vocab) || !stride_ok(out_stride, count) || (count > 1 && out_stride < width))
        return LRS_ERR_SIZE;
    if (count == 0 || width == 0) return LRS_OK;
    if (!out || (vocab > 0 && !weight)) return LRS_ERR_NULL_POINTER;
    const uint64_t size = row_type_size(dtype), out_size = row_type_size(out_dtype);
    if (misaligned(weight, size) || misaligned(out, out_size)) return LRS_ERR_ALIGNMENT;
    const uint64_t ob = span(count, out_stride, width, out_size);
    if (overlaps(out, ob, weight, span(vocab, weight_stride, width, size)) || overlaps(out, ob, tokens->ids, id_span(tokens)))
        return LRS_ERR_ALIASING;
    a.weight = weight;
    a.weight_stride = weight_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.tokens = static_cast<uint32_t>(count);
    a.vocab = static_cast<uint32_t>(vocab);
    a.width = static_cast<uint32_t>(width);
    a.scale = scale;
    c.elems = static_cast<uint64_t>(count) * width;
    const uint64_t pieces = static_cast<uint64_t>(count) * ((width + 7) / 8);
    const dim3 grid(static_cast<uint32_t>(std::min<uint64_t>((pieces + kEmbBlock - 1) / kEmbBlock, kMaxGrid)));
    TimedLaunch t(4, c);
    by_types(dtype, out_dtype, [&](auto i, auto o) { launch_on(lookup_kernel<i.value, o.value>, grid, dim3(kEmbBlock), t.L, a); });
    return hipGetLastError() == hipSuccess ? LRS_OK : LRS_ERR_HIP;
} catch (...) {
    return LRS_ERR_HIP;
}

size_t embedding_backward_workspace_size(int64_t tokens, int64_t vocab, int64_t width, const lrs_options *opts) {
    if (!options_ok(opts) || check_sizes(tokens, vocab, width) != LRS_OK) return 0;
    return static_cast<size_t>(grad_space(tokens, vocab, width, opts).total);
}

int embedding_backward(const void *grad, int64_t grad_stride, const lrs_token_ids *tokens, void *grad_weight,
                       int64_t weight_stride, int64_t vocab, int64_t width, int dtype, int out_dtype, float scale,
                       int64_t padding_index, int accumulate, void *workspace, size_t workspace_bytes, void *stream,
                       const lrs_options *opts) try {
    Ctx c;
    if (!make_ctx(stream, opts, c) || !std::isfinite(scale)) return LRS_ERR_OPTION;
    if (!row_type_ok(dtype) || !row_type_ok(out_dtype)) return LRS_ERR_DTYPE;
    GradArgs a{};
    int64_t count = 0;
    int st = check_ids(tokens, a.ids, count);
    if (st == LRS_OK) st = check_sizes(count, vocab, width);
    if (st != LRS_OK) return st;
    if (!stride_ok(grad_stride, count) || !stride_ok(weight_stride, vocab) || (vocab > 1 && weight_stride < width))
        return LRS_ERR_SIZE;
    if (vocab == 0 || width == 0) return LRS_OK;
    const GradSpace w = grad_space(count, vocab, width, opts);
    if (!grad_weight || (count > 0 && (!grad || !workspace))) return LRS_ERR_NULL_POINTER;
    const uint64_t size = row_type_size(dtype), out_size = row_type_size(out_dtype);
    if (misaligned(grad, size) || misaligned(grad_weight, out_size) || (w.total && misaligned(workspace, 256)))
        return LRS_ERR_ALIGNMENT;
    if (workspace_bytes < w.total) return LRS_ERR_WORKSPACE_TOO_SMALL;
    const uint64_t wb = span(vocab, weight_stride, width, out_size), gb = span(count, grad_stride, width, size);
    if (overlaps(grad_weight, wb, grad, gb) || overlaps(grad_weight, wb, tokens->ids, id_span(tokens)) ||
        overlaps(grad_weight, wb, workspace, w.total) || overlaps(workspace, w.total, grad, gb) ||
        overlaps(workspace, w.total, tokens->ids, id_span(tokens)))
        return LRS_ERR_ALIASING;
    a.grad = grad;
    a.grad_stride = grad_stride;
    a.out = grad_weight;
    a.out_stride = weight_stride;
    a.tokens = static_cast<uint32_t>(count);
    a.vocab = static_cast<uint32_t>(vocab);
    a.width = static_cast<uint32_t>(width);
    a.scale = scale;
    a.padding = padding_index;
    a.accumulate = accumulate != 0;
    c.elems = static_cast<uint64_t>(count) * width;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (count > 0) {
        a.keys = reinterpret_cast<uint32_t *>(ws + w.keys);
        a.places = reinterpret_cast<uint32_t *>(ws + w.places);
        uint32_t *sorted = reinterpret_cast<uint32_t *>(ws + w.sorted), *order = reinterpret_cast<uint32_t *>(ws + w.order);
        a.sorted = sorted;
        a.order = order;
        a.present = reinterpret_cast<uint32_t *>(ws + w.present);
        a.longs = reinterpret_cast<uint32_t *>(ws + w.longs);
        a.runs = reinterpret_cast<float *>(ws + w.runs);
        {
            TimedLaunch t(4, c);
            launch_on(embed_keys_kernel, dim3((a.tokens + kEmbBlock - 1) / kEmbBlock), dim3(kEmbBlock), t.L, a);
        }
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
        st = radix_sort_pairs(a.keys, a.places, sorted, order, a.tokens, 0, key_bits(vocab), 8, ws + w.sort, w.sort_bytes,
                              stream, opts);
        if (st != LRS_OK) return st;
    }
    by_types(dtype, out_dtype, [&](auto i, auto o) {
        if (width <= 16 * 8) launch_sums<i.value, o.value, 16>(a, c);
        else launch_sums<i.value, o.value, kLanes>(a, c);
    });
    return hipGetLastError() == hipSuccess ? LRS_OK : LRS_ERR_HIP;
} catch (...) {
    return LRS_ERR_HIP;
}

}  // extern "C"
