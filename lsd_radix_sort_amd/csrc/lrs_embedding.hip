// lrs_embedding.hip -- embedding lookup, and the gradient of its table by
// sorted tokens (gfx950).
//
// out[t] = scale W[id_t]; dW[v] = scale * sum of g[t] over the tokens with id_t =
// v.  The sum over the tokens of one id is a segmented sum once the pairs (id,
// place) are sorted, by the library's stable sort or, for fewer tokens, by a
// counting sort of the ids in one launch; within an id the places then stand in
// order, so the sum has one order however the GPU runs it.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/lsd_radix_sort.h"
#include "lrs_host.h"
#include "lrs_rows.h"
#include "lrs_select.h"

namespace lrs {
namespace {

constexpr int kEmbBlock = 256;

struct Ids {
    const void *at;
    uint64_t stride;
    uint32_t length;
    int bytes;
    __device__ int64_t operator[](uint32_t t) const {
        const uint64_t i = t < length ? t : t / length * stride + t % length;
        return bytes == 8 ? static_cast<const int64_t *>(at)[i] : static_cast<const int32_t *>(at)[i];
    }
};

// What a lane holds of a piece of a row: eight neighbouring columns, or, where
// one of the types has 32 bits, two fours that lie apart, so that the lanes of a
// store lie side by side in each type (32-byte steps cost 2.8 times as much).
template <int LANES, bool FOURS> struct Columns {
    static constexpr int kParts = FOURS ? 2 : 1, kSize = 8 / kParts;
    uint32_t first[kParts], count[kParts];
    __device__ Columns(uint32_t piece, uint32_t width) : Columns(piece, width, threadIdx.x % LANES) {}
    __device__ Columns(uint32_t piece, uint32_t width, uint32_t lane) {
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            first[p] = piece * LANES * 8 + p * LANES * kSize + lane * kSize;
            count[p] = first[p] < width ? min(width - first[p], static_cast<uint32_t>(kSize)) : 0;
        }
    }
};
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_align2 __attribute__((aligned(2)));

// Those columns of one row as they are stored.
template <int T, int LANES, bool FOURS> struct Eight {
    using At = Columns<LANES, FOURS>;
    static constexpr int kWords = T == kRowF32 ? 8 : 4, kEach = kWords / At::kParts;
    uint32_t w[kWords];
    // ONCE: not kept in the caches (a template argument: of two branches alike but for that, one is made)
    template <bool ONCE> __device__ void load(const void *rows, uint64_t row, const At &c) {
#pragma unroll
        for (int p = 0; p < At::kParts; ++p) {
            const auto *x = static_cast<const typename Row<T>::Stored *>(rows) + row + c.first[p];
            uint32_t *v = w + p * kEach;
            if (c.count[p] == At::kSize) {
                if constexpr (kEach == 4) {
                    const u32x4 q = ONCE ? load16_once(x) : load16(x);
                    for (int i = 0; i < 4; ++i) v[i] = q[i];
                } else {
                    static_assert(kEach == 2);
                    const auto *y = reinterpret_cast<const u32x2_align2 *>(x);
                    const u32x2 q = ONCE ? __builtin_nontemporal_load(y) : *y;
                    v[0] = q.x;
                    v[1] = q.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kEach; ++i) v[i] = 0;
#pragma unroll
                for (uint32_t e = 0; e < At::kSize; ++e) {
                    const uint32_t q = e < c.count[p] ? x[e] : 0;
                    if constexpr (T == kRowF32) v[e] = q;
                    else v[e / 2] |= q << (16 * (e & 1));
                }
            }
        }
    }
    __device__ void values(float (&f)[8]) const {
        if constexpr (T == kRowF32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __builtin_bit_cast(float, w[e]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) Row<T>::unpack(w[i], f[2 * i], f[2 * i + 1]);
        }
    }
    __device__ void add_to(float (&sum)[8]) const {
        float f[8];
        values(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += f[e];
    }
    template <bool ONCE> __device__ static void store(void *rows, uint64_t row, const At &c, const float (&f)[8]) {
        const auto put = [&](void *x, u32x4 v) { ONCE ? store16_once(x, v) : store16(x, v); };
#pragma unroll
        for (int p = 0; p < At::kParts; ++p) {
            auto *x = static_cast<typename Row<T>::Stored *>(rows) + row + c.first[p];
            const float *g = f + p * At::kSize;
            if (c.count[p] == At::kSize) {
                if constexpr (T == kRowF32) {
                    put(x, u32x4{__builtin_bit_cast(uint32_t, g[0]), __builtin_bit_cast(uint32_t, g[1]),
                                 __builtin_bit_cast(uint32_t, g[2]), __builtin_bit_cast(uint32_t, g[3])});
                } else if constexpr (FOURS) {
                    const u32x2 v{Row<T>::pack(g[0], g[1]), Row<T>::pack(g[2], g[3])};
                    auto *y = reinterpret_cast<u32x2_align2 *>(x);
                    if constexpr (ONCE) __builtin_nontemporal_store(v, y);
                    else *y = v;
                } else {
                    put(x, u32x4{Row<T>::pack(g[0], g[1]), Row<T>::pack(g[2], g[3]), Row<T>::pack(g[4], g[5]),
                                 Row<T>::pack(g[6], g[7])});
                }
            } else {
#pragma unroll
                for (uint32_t e = 0; e < At::kSize; ++e)
                    if (e < c.count[p]) x[e] = Row<T>::pattern(g[e]);
            }
        }
    }
};

// ------------------------------------------------------------------ lookup

struct LookupArgs {
    const void *weight;
    uint64_t weight_stride;
    Ids ids;
    void *out;
    uint64_t out_stride;
    uint32_t tokens, vocab, width;
    uint32_t tasks;  // of a token
    float scale;
};

template <int LANES> __device__ inline uint32_t uniform(uint32_t v) {
    return LANES == kLanes ? __builtin_amdgcn_readfirstlane(v) : v;
}

// A group of lanes has up to kSlots loads on their way: pieces of one token's row,
// or, where a piece is a row, tokens.  (Pieces past a row's end are idle slots: two
// of four at 1024 columns, one at 1031, which has another for 7 columns.)  Always
// written past the caches: 32768 x 4096 bf16 of text, calls in a row, whose 97 MB of
// table rows stay behind the L2s, 63 us, 81 us through the caches, which the rows'
// repeated reads need more; of a table that is not there 84 us = 4.4 TB/s.
constexpr uint32_t kSlots = 4;
template <int T, int O, int LANES>
__global__ __launch_bounds__(kEmbBlock) void lookup_kernel(LookupArgs a) {
    constexpr bool kFours = T == kRowF32 || O == kRowF32, kNarrow = LANES < kLanes;
    constexpr uint32_t kGroups = kEmbBlock / LANES;
    const uint64_t tasks = kNarrow ? (static_cast<uint64_t>(a.tokens) + kSlots - 1) / kSlots : static_cast<uint64_t>(a.tokens) * a.tasks;
    for (uint64_t task = static_cast<uint64_t>(blockIdx.x) * kGroups + threadIdx.x / LANES; task < tasks;
         task += static_cast<uint64_t>(gridDim.x) * kGroups) {
        // a.tasks is 1 unless rows are long
        const uint64_t first = kNarrow ? task * kSlots : a.tasks == 1 ? task : task / a.tasks;
        const uint32_t piece = kNarrow ? 0 : uniform<LANES>(static_cast<uint32_t>(task - first * a.tasks)) * kSlots;
        uint32_t token[kSlots];
        int64_t id[kSlots];
        bool on[kSlots], inside[kSlots];
#pragma unroll
        for (uint32_t j = 0; j < kSlots; ++j) {
            token[j] = uniform<LANES>(static_cast<uint32_t>(kNarrow ? first + j : first));
            on[j] = kNarrow ? first + j < a.tokens : (piece + j) * LANES * 8 < a.width;
            id[j] = kNarrow ? (on[j] ? a.ids[token[j]] : -1) : j == 0 ? a.ids[token[0]] : id[0];
            inside[j] = id[j] >= 0 && id[j] < a.vocab;
        }
        Eight<T, LANES, kFours> row[kSlots];
#pragma unroll
        for (uint32_t j = 0; j < kSlots; ++j)
            if (on[j] && inside[j])
                row[j].template load<false>(a.weight, id[j] * a.weight_stride, Columns<LANES, kFours>(kNarrow ? 0 : piece + j, a.width));
#pragma unroll
        for (uint32_t j = 0; j < kSlots; ++j) {
            if (!on[j]) continue;
            float f[8];
            row[j].values(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = inside[j] ? f[e] * a.scale : 0.f;
            Eight<O, LANES, kFours>::template store<true>(a.out, token[j] * a.out_stride,
                                                          Columns<LANES, kFours>(kNarrow ? 0 : piece + j, a.width), f);
        }
    }
}

// ---------------------------------------------------------------- gradient
//
// After the sort the tokens of an id are neighbours.  Text has a few ids that
// make up a large share of it, and most ids in none, so the work is cut into
// even pieces: a wave takes a run of sorted places, and of each id that begins
// there all places, less than two runs, unless the id has an aligned run to
// itself.  Such an id is long: every wave adds up what its own run holds of it,
// and a second launch joins those sums.  The rows of ids without tokens are
// cleared in the first launch, too.  Bound by HBM: 32768 tokens of text, 131072 x
// 4096 bf16 206 to 217 us = 6.2 TB/s and more.

constexpr uint32_t kMaxRun = 16;

// What the sums do with the gradient: write it, the sums past the caches or the
// cleared rows past them (see launch_sums), or add to it.
enum Mode : int { kSumsOnce, kClearOnce, kAdd };

constexpr int kJoinBlock = 1024;
constexpr uint32_t kShort = 8;  // runs of a long id that a group of lanes joins alone

// A long id: the first of its whole runs, how many there are, and whether the
// runs before and after them hold places of it.
struct Long {
    uint32_t run, runs, key;
    uint16_t before, after;
};

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
    uint32_t *long_count;                 // of more than kShort runs, of fewer
    Long *longs;                          // [runs]: the former from the front, the latter from the back
    float *parts;                         // [2][runs][pieces][lanes * 8]: see part_of
    uint32_t run;                         // places in a run: 4, 8 or 16
    uint32_t runs;                        // the last one maybe shorter
    uint32_t pieces;                      // of a row, a group of lanes each
    uint32_t sum_blocks;                  // blocks that sum; the others clear
    uint32_t *present;                    // a bit for every id that a token names
    uint32_t range;                       // ids whose places one workgroup orders, a multiple of 32
    uint32_t line_factor;                 // 2^32 over the ids' length, rounded up
};

// The keys of the sort: ids, those that count for nothing behind the last.
__global__ __launch_bounds__(kEmbBlock) void embed_keys_kernel(GradArgs a) {
    const uint32_t t = blockIdx.x * kEmbBlock + threadIdx.x;
    if (t < 2) a.long_count[t] = 0;
    if (!a.accumulate)
        for (uint32_t w = t; w < (a.vocab + 31) / 32; w += gridDim.x * kEmbBlock) a.present[w] = 0;
    if (t >= a.tokens) return;
    const int64_t id = a.ids[t];
    a.keys[t] = id >= 0 && id < a.vocab && id != a.padding ? static_cast<uint32_t>(id) : a.vocab;
    a.places[t] = t;
}

// The bits of the ids that tokens name.
__global__ __launch_bounds__(kEmbBlock) void embed_present_kernel(GradArgs a) {
    const uint32_t i = blockIdx.x * kEmbBlock + threadIdx.x;
    if (i >= a.tokens) return;
    const uint32_t key = a.sorted[i];
    if (key < a.vocab && (i == 0 || a.sorted[i - 1] != key)) atomicOr(&a.present[key / 32], 1u << (key % 32));
}

// For few tokens a workgroup finds the places of a range of ids by itself,
// from a read of all of them: what a sort needs several launches for, one after
// the other.  A wave takes a share of the tokens, N for each lane, and counts the
// range's ids among them; the counts, added up by id and then by wave, say where
// each wave's first token of an id goes, and the wave deals its tokens out in
// order.  Bound by the instructions for an id that is not in the range, which are
// 255 of 256: masks of whole waves and scalar counts.  8192 tokens 7 us, 32768 18 us
// (the sort takes 35 to 45); twice as many a lane spill.
constexpr int kOrderBlock = 1024;
constexpr uint32_t kMaxRange = 1024;
template <int N, typename Id>
__global__ __launch_bounds__(kOrderBlock) void embed_order_kernel(GradArgs a, uint32_t *sorted, uint32_t *order) {
    constexpr uint32_t kWaves = kOrderBlock / kLanes;
    __shared__ uint32_t counter[kWaves][kMaxRange];
    __shared__ uint32_t cells[2][kWaves];
    const uint32_t lane = threadIdx.x % kLanes, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    const uint32_t first = blockIdx.x * a.range, ids = min(a.range, a.vocab - first);
    const uint32_t from = wave * (N * kLanes) + lane;
    Id id[N];
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
        const uint32_t t = from + i * kLanes, line = a.ids.length == 1 ? t : __umulhi(t, a.line_factor);
        id[i] = t < a.tokens ? static_cast<const Id *>(a.ids.at)[static_cast<uint64_t>(line) * a.ids.stride + (t - line * a.ids.length)] : -1;
    }
    if (blockIdx.x == 0 && threadIdx.x < 2) a.long_count[threadIdx.x] = 0;
    for (uint32_t i = lane; i < ids; i += kLanes) counter[wave][i] = 0;
    // within the range: the id's place there
    uint32_t of[N], below = 0;
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
        const bool counts = id[i] >= 0 && static_cast<int64_t>(id[i]) != a.padding;
        below += __popcll(__ballot(counts && id[i] < static_cast<Id>(first)));
        of[i] = counts && id[i] < static_cast<Id>(a.vocab) ? static_cast<uint32_t>(id[i]) - first : ~0u;
        if (of[i] < ids) atomicAdd(&counter[wave][of[i]], 1u);
    }
    if (lane == 0) cells[0][wave] = below;
    __syncthreads();
    // a thread an id: its tokens, and where they begin
    uint32_t mine = 0;
    if (threadIdx.x < ids)
        for (uint32_t w = 0; w < kWaves; ++w) mine += counter[w][threadIdx.x];
    const uint64_t named = __ballot(mine > 0);
    if (lane % 32 == 0 && threadIdx.x < ids) a.present[(first + threadIdx.x) / 32] = static_cast<uint32_t>(named >> lane);
    const uint32_t upto = lanes_sum(mine);
    if (lane == kLanes - 1) cells[1][wave] = upto;
    __syncthreads();
    uint32_t start = upto - mine, all = 0;
    for (uint32_t w = 0; w < kWaves; ++w) {
        all += cells[0][w] + cells[1][w];
        start += cells[0][w] + (w < wave ? cells[1][w] : 0);
    }
    if (threadIdx.x < ids)
        for (uint32_t w = 0; w < kWaves; ++w) {
            const uint32_t c = counter[w][threadIdx.x];
            counter[w][threadIdx.x] = start;
            start += c;
        }
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
        for (uint64_t left = __ballot(of[i] < ids); left;) {  // an id at a time
            const uint32_t one = __builtin_amdgcn_readlane(of[i], __builtin_ctzll(left));
            const uint64_t same = __ballot(of[i] == one);
            const uint32_t at = counter[wave][one];
            if (of[i] == one) {
                const uint32_t p = at + __builtin_amdgcn_mbcnt_hi(same >> 32, __builtin_amdgcn_mbcnt_lo(same, 0));
                sorted[p] = first + one;
                order[p] = from + i * kLanes;
            }
            counter[wave][one] = at + __popcll(same);
            left &= ~same;
        }
    }
    // behind the last id: what counts for nothing
    if (blockIdx.x == gridDim.x - 1)
        for (uint32_t i = all + threadIdx.x; i < a.tokens; i += kOrderBlock) sorted[i] = a.vocab;
}

// A finished sum to the table's gradient, on top of what that holds or not.
template <int O, int LANES, bool FOURS, int MODE>
__device__ inline void put_row(const GradArgs &a, uint32_t id, const Columns<LANES, FOURS> &c, const float (&sum)[8],
                               const Eight<O, LANES, FOURS> &old) {
    float f[8] = {};
    if (MODE == kAdd) old.values(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = MODE == kAdd ? fmaf(sum[e], a.scale, f[e]) : sum[e] * a.scale;
    Eight<O, LANES, FOURS>::template store<MODE == kSumsOnce>(a.out, id * a.out_stride, c, f);
}

// Where a run's sum of a long id is kept: one place for the id that begins in
// an earlier run or has the whole one, one for the id that begins within.
template <int LANES> __device__ inline float *part_of(const GradArgs &a, uint32_t begins, uint32_t run, uint32_t piece, uint32_t lane) {
    return a.parts + ((static_cast<uint64_t>(begins) * a.runs + run) * a.pieces + piece) * (LANES * 8) + lane * 4;
}

// How many keys are below `id`, as `from` are at least: by a whole wave, 64
// places tried at a time.
__device__ inline uint32_t keys_below(const uint32_t *keys, uint32_t from, uint32_t count, uint32_t id) {
    const uint32_t lane = threadIdx.x % kLanes;
    uint32_t lo = from, hi = count;
    while (hi - lo > kLanes) {
        const uint32_t step = (hi - lo + kLanes - 1) / kLanes;
        const uint64_t at = static_cast<uint64_t>(lo) + (lane + 1) * static_cast<uint64_t>(step) - 1;
        lo += __popcll(__ballot(at < hi && keys[at] < id)) * step;
        hi = lo > hi ? lo : min(hi, lo + step - 1);
    }
    return lo + __popcll(__ballot(lo + lane < hi && keys[lo + lane] < id));
}

// The ids of a run.  A wave looks at 64 places at once, from the one before the
// run on; its groups of lanes take an equal share of the beginnings each, the
// first one also the id that continues.  Rows are on their way several at a
// time, whatever ids they are of.
template <int T, int O, int LANES, int MODE> __device__ void sum_run(const GradArgs &a, uint32_t run, uint32_t piece) {
    constexpr bool kFours = T == kRowF32 || O == kRowF32, ADD = MODE == kAdd;
    constexpr uint32_t kGroups = kLanes / LANES;
    static_assert(3 * kMaxRun - 1 < kLanes, "an id that is not long ends among the places looked at");
    const uint32_t len = a.run, last_lane = len, share = len / kGroups;  // last_lane: of the run's last place
    const uint32_t lane = threadIdx.x % kLanes, begin = run * len;
    const uint64_t place = static_cast<uint64_t>(begin) + lane - 1;  // of this lane
    const bool real = place < a.tokens;                            // not before the first either
    const uint32_t key = real ? a.sorted[place] : a.vocab, order = real ? a.order[place] : 0;
    const uint32_t back = run > 0 ? a.sorted[begin - len] : a.vocab;
    const uint32_t left = __builtin_amdgcn_update_dpp(~0u, key, 0x138, 0xF, 0xF, false);  // wave_shr:1
    // bit l: the place of lane l begins an id; past the last token, and where ids count for nothing, every place does
    const uint64_t heads = __ballot(lane > 0 && (key != left || key >= a.vocab || (lane == 1 && run == 0)));
    const uint64_t counts = __ballot(real && key < a.vocab);
    const auto bits = [](uint32_t from, uint32_t to) { return ((uint64_t(1) << to) - 1) & ~((uint64_t(1) << from) - 1); };  // to < 64
    const auto end_of = [&](uint32_t l) {  // the place after the id that has lane l's
        const uint64_t later = heads & ~((uint64_t(2) << l) - 1);
        return later ? static_cast<uint32_t>(__builtin_ctzll(later)) : static_cast<uint32_t>(kLanes);
    };
    // the places that this group sums, and those of them that are of long ids
    const uint32_t group = LANES == kLanes ? 0 : lane / LANES, from = 1 + group * share;
    uint64_t todo = 0, of_long = 0;
    for (uint64_t h = heads & counts & bits(from, from + share); h; h &= h - 1) {
        const uint32_t l = __builtin_ctzll(h), end = end_of(l), whole = l == 1 ? 1 : last_lane + 1;  // its first aligned run, if it has one
        if (end < whole + len) todo |= bits(l, end);
        else of_long |= bits(l, last_lane + 1);
    }
    const uint32_t key1 = __builtin_amdgcn_readlane(key, 1);
    const uint32_t end1 = end_of(1);
    const bool full = (counts & 2) && end1 > last_lane;  // one id has the whole run
    if (group == 0 && (counts & 2) && !(heads & 2) && (full || back == key1)) of_long |= bits(1, min(end1, last_lane + 1));
    todo |= of_long;
    if (full && back != key1 && piece == 0) {  // the id's first whole run
        const uint32_t end = keys_below(a.sorted, begin + len, a.tokens, key1 + 1), runs = end / len - run;
        if (lane == 0) {
            const bool few = runs <= kShort;
            const uint32_t at = atomicAdd(&a.long_count[few], 1u);
            a.longs[few ? a.runs - 1 - at : at] = Long{run, runs, key1, static_cast<uint16_t>(!(heads & 2)),
                                                       static_cast<uint16_t>(end % len != 0)};
        }
    }
    const Columns<LANES, kFours> c(piece, a.width);
    constexpr int kAtOnce = T == kRowF32 || ADD ? 4 : MODE == kClearOnce ? 16 : 8;
    float sum[8] = {};
    while (__ballot(todo != 0)) {  // until all groups are done: each reads places that others' lanes hold
        Eight<T, LANES, kFours> row[kAtOnce];
        Eight<O, LANES, kFours> old[ADD ? kAtOnce : 1];
        uint32_t id[kAtOnce];
        uint32_t on = 0, last = 0, part = 0, begins = 0;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            uint32_t l = 0;
            if (todo) {
                l = __builtin_ctzll(todo);
                todo &= todo - 1;
                on |= 1u << j;
                const uint32_t of = static_cast<uint32_t>(of_long >> l) & 1;
                part |= of << j;
                last |= (static_cast<uint32_t>((heads >> (l + 1)) & 1) | (of & (l == last_lane))) << j;
                begins |= static_cast<uint32_t>((heads & bits(2, l + 1)) != 0) << j;
            }
            const uint32_t at = LANES == kLanes ? __builtin_amdgcn_readlane(order, l) : __shfl(order, l);
            id[j] = LANES == kLanes ? __builtin_amdgcn_readlane(key, l) : __shfl(key, l);
            if ((on >> j) & 1) row[j].template load<true>(a.grad, at * a.grad_stride, c);
            if (ADD && ((last & ~part) >> j) & 1) old[ADD ? j : 0].template load<false>(a.out, id[j] * a.out_stride, c);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if ((on >> j) & 1) row[j].add_to(sum);
            if ((last >> j) & 1) {
                if ((part >> j) & 1) {
                    float *p = part_of<LANES>(a, (begins >> j) & 1, run, piece, threadIdx.x % LANES);
                    *reinterpret_cast<float4 *>(p) = float4{sum[0], sum[1], sum[2], sum[3]};
                    *reinterpret_cast<float4 *>(p + LANES * 4) = float4{sum[4], sum[5], sum[6], sum[7]};
                } else {
                    put_row<O, LANES, kFours, MODE>(a, id[j], c, sum, old[ADD ? j : 0]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] = 0.f;
            }
        }
    }
}

// Clears the rows of 32 ids that no token names, or a piece of each: 32 KB, so
// that the last pieces do not leave most of the GPU idle.
constexpr uint32_t kClearPiece = 64;  // 16-byte stores
template <int O, bool ONCE> __device__ void clear_rows(const GradArgs &a, uint32_t word, uint32_t piece) {
    constexpr uint32_t kVec = Row<O>::kVec;
    const uint32_t id0 = word * 32, ids = min(32u, a.vocab - id0);
    const uint32_t named = a.tokens ? a.present[word] : 0;
    const uint32_t all = (a.width + kVec - 1) / kVec, first = piece * kClearPiece, stores = min(kClearPiece, all - first);
    // rows side by side: a piece of one takes at most a quarter of the threads
    const uint32_t shift = 32 - __builtin_clz((stores - 1) | 1), rows = kEmbBlock >> shift, u = threadIdx.x & ((1u << shift) - 1);
    if (u >= stores) return;
    const uint64_t col = static_cast<uint64_t>(first + u) * kVec;
    for (uint32_t r = threadIdx.x >> shift; r < ids; r += rows) {
        if ((named >> r) & 1) continue;
        auto *p = static_cast<typename Row<O>::Stored *>(a.out) + (id0 + r) * a.out_stride;
        if (col + kVec <= a.width) (ONCE ? store16_once : store16)(p + col, u32x4{0, 0, 0, 0});
        else
            for (uint32_t e = 0; col + e < a.width; ++e) p[col + e] = 0;
    }
}

template <int T, int O, int LANES, int MODE>
__global__ __launch_bounds__(kEmbBlock) void embed_sum_kernel(GradArgs a) {
    constexpr uint32_t kWaves = kEmbBlock / kLanes;
    if (blockIdx.x < a.sum_blocks) {
        const uint64_t tasks = static_cast<uint64_t>(a.runs) * a.pieces;
        for (uint64_t t = static_cast<uint64_t>(blockIdx.x) * kWaves + threadIdx.x / kLanes; t < tasks; t += static_cast<uint64_t>(a.sum_blocks) * kWaves)
            sum_run<T, O, LANES, MODE>(a, __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(t / a.pieces)),
                                      __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(t % a.pieces)));
        return;
    }
    if constexpr (MODE != kAdd) {
        const uint32_t pieces = ((a.width + Row<O>::kVec - 1) / Row<O>::kVec + kClearPiece - 1) / kClearPiece, words = (a.vocab + 31) / 32;
        const uint64_t tasks = static_cast<uint64_t>(words) * pieces;
        for (uint64_t t = blockIdx.x - a.sum_blocks; t < tasks; t += gridDim.x - a.sum_blocks)
            clear_rows<O, MODE == kClearOnce>(a, static_cast<uint32_t>(t / pieces), static_cast<uint32_t>(t % pieces));
    }
}

// The whole gradient of few tokens in one launch, where the launches are most of
// the time.  A workgroup takes a range of ids and a piece of their rows: it orders
// the range's places as above, in LDS, and clears the rows that none names.  Its
// groups of lanes then take even shares of the places; an id that has places in
// several shares is joined over LDS by the group of the first.  200 tokens of text,
// 5003 x 256 fp32: 5.6 us, 13 in three launches; the worst, 2048 of one id and 128
// columns: 18 us, 17 in three.
constexpr uint32_t kFewTokens = 2048, kFewRange = 512;
template <int T, int O, int LANES, int MODE>
__global__ __launch_bounds__(kOrderBlock) void embed_few_kernel(GradArgs a) {
    constexpr bool kFours = T == kRowF32 || O == kRowF32;
    constexpr uint32_t kWaves = kOrderBlock / kLanes, kGroups = kOrderBlock / LANES, N = kFewTokens / kOrderBlock;
    __shared__ uint32_t counter[kWaves][kFewRange], cells[kWaves], named[kFewRange / 32];
    __shared__ uint16_t place[kFewTokens], id_of[kFewTokens];
    __shared__ float4 parts[kGroups][2][2][LANES];  // of the id that continues, of the one that goes on
    const uint32_t lane = threadIdx.x % kLanes, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    const uint32_t first = blockIdx.x * a.range, ids = min(a.range, a.vocab - first);
    const uint32_t from = wave * (N * kLanes) + lane;
    int64_t id[N];
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
        const uint32_t t = from + i * kLanes, line = a.ids.length == 1 ? t : __umulhi(t, a.line_factor);
        const uint64_t at = static_cast<uint64_t>(line) * a.ids.stride + (t - line * a.ids.length);
        id[i] = t >= a.tokens ? -1 : a.ids.bytes == 8 ? static_cast<const int64_t *>(a.ids.at)[at] : static_cast<const int32_t *>(a.ids.at)[at];
    }
    for (uint32_t i = lane; i < ids; i += kLanes) counter[wave][i] = 0;
    uint32_t of[N];
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
        of[i] = id[i] >= first && id[i] - first < ids && id[i] != a.padding ? static_cast<uint32_t>(id[i]) - first : ~0u;
        if (of[i] < ids) atomicAdd(&counter[wave][of[i]], 1u);
    }
    __syncthreads();
    uint32_t mine = 0;
    if (threadIdx.x < ids)
        for (uint32_t w = 0; w < kWaves; ++w) mine += counter[w][threadIdx.x];
    const uint64_t some = __ballot(mine > 0);
    if (lane % 32 == 0 && threadIdx.x < kFewRange) named[threadIdx.x / 32] = static_cast<uint32_t>(some >> lane);
    const uint32_t upto = lanes_sum(mine);
    if (lane == kLanes - 1) cells[wave] = upto;
    __syncthreads();
    uint32_t start = upto - mine, all = 0;
    for (uint32_t w = 0; w < kWaves; ++w) {
        all += cells[w];
        start += w < wave ? cells[w] : 0;
    }
    if (threadIdx.x < ids)
        for (uint32_t w = 0; w < kWaves; ++w) {
            const uint32_t c = counter[w][threadIdx.x];
            counter[w][threadIdx.x] = start;
            start += c;
        }
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
        for (uint64_t left = __ballot(of[i] < ids); left;) {  // an id at a time
            const uint32_t one = __builtin_amdgcn_readlane(of[i], __builtin_ctzll(left));
            const uint64_t same = __ballot(of[i] == one);
            const uint32_t at = counter[wave][one];
            if (of[i] == one) {
                const uint32_t p = at + __builtin_amdgcn_mbcnt_hi(same >> 32, __builtin_amdgcn_mbcnt_lo(same, 0));
                place[p] = static_cast<uint16_t>(from + i * kLanes);
                id_of[p] = static_cast<uint16_t>(one);
            }
            counter[wave][one] = at + __popcll(same);
            left &= ~same;
        }
    }
    const uint32_t piece = blockIdx.y;
    const Columns<LANES, kFours> c(piece, a.width);
    if constexpr (MODE != kAdd) {
        constexpr uint32_t kVec = Row<O>::kVec, kStores = LANES * 8 / kVec;  // a thread each, rows side by side
        const uint32_t col = piece * LANES * 8 + threadIdx.x % kStores * kVec;
        for (uint32_t r = threadIdx.x / kStores; r < ids; r += kOrderBlock / kStores) {
            if ((named[r / 32] >> (r % 32)) & 1) continue;
            auto *p = static_cast<typename Row<O>::Stored *>(a.out) + (first + r) * a.out_stride;
            if (col + kVec <= a.width) store16(p + col, u32x4{0, 0, 0, 0});
            else
                for (uint32_t e = col; e < a.width; ++e) p[e] = 0;
        }
    }
    __syncthreads();
    const uint32_t group = threadIdx.x / LANES, here = threadIdx.x % LANES, share = (all + kGroups - 1) / kGroups;
    const uint32_t begin = min(group * share, all), end = min(begin + share, all);
    const uint32_t continued = begin > 0 && begin < end ? id_of[begin - 1] : ~0u;  // the id before this share
    constexpr uint32_t kAtOnce = MODE == kAdd ? (kFours ? 4 : 8) : T == kRowF32 ? 8 : 16;
    Eight<O, LANES, kFours> old[MODE == kAdd ? kAtOnce : 1];
    float sum[8] = {};
    for (uint32_t p = begin; p < end; p += kAtOnce) {
        Eight<T, LANES, kFours> row[kAtOnce];
        uint32_t done = 0, own = 0;  // bits: the last place of an id, of one that begins in this share
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; ++j) {
            if (p + j >= end) continue;
            const uint32_t key = id_of[p + j], next = p + j + 1 < all ? id_of[p + j + 1] : ~0u;
            done |= static_cast<uint32_t>(key != next) << j;
            own |= static_cast<uint32_t>(key != continued) << j;
            row[j].template load<false>(a.grad, place[p + j] * a.grad_stride, c);
            if (MODE == kAdd && key != next && key != continued)
                old[MODE == kAdd ? j : 0].template load<false>(a.out, (first + key) * a.out_stride, c);
        }
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; ++j) {
            if (p + j >= end) continue;
            row[j].add_to(sum);
            if (((done >> j) & 1) == 0 && p + j + 1 < end) continue;
            if ((done >> j) & (own >> j) & 1) {
                put_row<O, LANES, kFours, MODE>(a, first + id_of[p + j], c, sum, old[MODE == kAdd ? j : 0]);
            } else {
                auto &part = parts[group][(own >> j) & 1];
                part[0][here] = float4{sum[0], sum[1], sum[2], sum[3]};
                part[1][here] = float4{sum[4], sum[5], sum[6], sum[7]};
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = 0.f;
        }
    }
    __syncthreads();
    const uint32_t last = begin < end ? id_of[end - 1] : ~0u;
    if (begin < end && end < all && id_of[end] == last && last != continued) {
        if (MODE == kAdd) old[0].template load<false>(a.out, (first + last) * a.out_stride, c);
        const auto add = [&](const float4 (&part)[2][LANES]) {
            const float4 p = part[0][here], q = part[1][here];
            const float f[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += f[e];
        };
        add(parts[group][1]);
        const uint32_t stop = (counter[kWaves - 1][last] + share - 1) / share;  // after the groups that have places of it
#pragma unroll 4
        for (uint32_t g = group + 1; g < stop; ++g) add(parts[g][0]);
        put_row<O, LANES, kFours, MODE>(a, first + last, c, sum, old[0]);
    }
}

// The long ids.  Those of few runs take a group of lanes each and piece (65536
// tokens, each id 13 times, 64 columns: 83 us in all, 126 by a workgroup each);
// those of many a workgroup for 16 lanes of a piece, whose groups of 16 take the
// runs in equal shares, joined in an order of their own (32768 tokens of one id,
// 4096 columns: 107 us in all, 134 by a workgroup for the piece, and 102 by 8 lanes,
// which cost text 3 us).
template <int O, int LANES, bool FOURS>
__global__ __launch_bounds__(kJoinBlock) void embed_join_kernel(GradArgs a) {
    constexpr uint32_t kAtOnce = 4, kNarrow = 16, kShares = kJoinBlock / kNarrow, kSubs = LANES / kNarrow;
    __shared__ float4 shared[kJoinBlock / kLanes][2][kNarrow];
    float sum[8] = {};
    const auto add = [&](float4 p, float4 q) {
        const float f[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += f[e];
    };
    // the sum of runs [from, to), from the part of the run before them on if that is wanted
    const auto sum_runs = [&](const Long &of, uint32_t piece, uint32_t lane, bool before, uint32_t from, uint32_t to) {
        const auto halves = [&](uint32_t begins, uint32_t run, float4 &p, float4 &q) {
            const float *at = part_of<LANES>(a, begins, run, piece, lane);
            p = *reinterpret_cast<const float4 *>(at);
            q = *reinterpret_cast<const float4 *>(at + LANES * 4);
        };
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = 0.f;
        if (before) {
            float4 p, q;
            halves(1, of.run - 1, p, q);
            add(p, q);
        }
        for (uint32_t r = from; r < to; r += kAtOnce) {
            float4 p[kAtOnce], q[kAtOnce];
#pragma unroll
            for (uint32_t j = 0; j < kAtOnce; ++j)
                if (r + j < to) halves(0, of.run + r + j, p[j], q[j]);
#pragma unroll
            for (uint32_t j = 0; j < kAtOnce; ++j)
                if (r + j < to) add(p[j], q[j]);
        }
    };
    const auto put = [&](uint32_t key, uint32_t piece, uint32_t lane) {
        const Columns<LANES, FOURS> c(piece, a.width, lane);
        Eight<O, LANES, FOURS> old;
        if (a.accumulate) {
            old.template load<false>(a.out, key * a.out_stride, c);
            put_row<O, LANES, FOURS, kAdd>(a, key, c, sum, old);
        } else {
            put_row<O, LANES, FOURS, kClearOnce>(a, key, c, sum, old);
        }
    };
    const uint32_t here = threadIdx.x % kNarrow, slot = threadIdx.x / kNarrow;
    const uint64_t many = static_cast<uint64_t>(a.long_count[0]) * a.pieces * kSubs;
    for (uint64_t task = blockIdx.x; task < many; task += gridDim.x) {
        const Long of = a.longs[task / (a.pieces * kSubs)];
        const uint32_t sub = static_cast<uint32_t>(task % (a.pieces * kSubs)), piece = sub / kSubs, lane = sub % kSubs * kNarrow + here;
        const uint32_t all = of.runs + of.after, share = (all + kShares - 1) / kShares, from = min(slot * share, all);
        sum_runs(of, piece, lane, slot == 0 && of.before, from, min(from + share, all));
        // over a wave's groups, then over the waves
#pragma unroll
        for (uint32_t d = kNarrow; d < kLanes; d *= 2)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor(sum[e], d);
        __syncthreads();  // the last task's readers are done
        if (threadIdx.x % kLanes < kNarrow) {
            shared[threadIdx.x / kLanes][0][here] = float4{sum[0], sum[1], sum[2], sum[3]};
            shared[threadIdx.x / kLanes][1][here] = float4{sum[4], sum[5], sum[6], sum[7]};
        }
        __syncthreads();
        if (threadIdx.x < kNarrow) {
            for (uint32_t w = 1; w < kJoinBlock / kLanes; ++w) add(shared[w][0][here], shared[w][1][here]);
            put(of.key, piece, lane);
        }
    }
    constexpr uint32_t kGroups = kJoinBlock / LANES;
    const uint32_t group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const uint64_t few = static_cast<uint64_t>(a.long_count[1]) * a.pieces;
    for (uint64_t task = static_cast<uint64_t>(gridDim.x - 1 - blockIdx.x) * kGroups + group; task < few;
         task += static_cast<uint64_t>(gridDim.x) * kGroups) {
        const Long of = a.longs[a.runs - 1 - task / a.pieces];
        const uint32_t piece = static_cast<uint32_t>(task % a.pieces);
        sum_runs(of, piece, lane, of.before, 0, of.runs + of.after);
        put(of.key, piece, lane);
    }
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

// Rows of at most 128 columns take a quarter of a wave.
uint64_t lanes_of(uint64_t width) { return width <= 16 * 8 ? 16 : kLanes; }
uint64_t over(uint64_t tasks, uint64_t each) { return (tasks + each - 1) / each; }

// Places in a run: as many as leave enough waves.
uint64_t run_of(uint64_t tokens, uint64_t width) {
    const uint64_t groups = tokens * over(width, lanes_of(width) * 8);
    return groups >= 16 * 8192 ? 16 : groups >= 8 * 2048 ? 8 : 4;
}
// Ids a workgroup orders: as few as make a workgroup a CU.
uint64_t range_of(uint64_t vocab) { return std::min<uint64_t>(over(vocab, 256 * 32) * 32, kMaxRange); }
bool ordered_directly(uint64_t tokens, uint64_t vocab) {
    return tokens <= 32 * kOrderBlock && over(vocab, range_of(vocab)) <= 1024;
}

// One launch for so few tokens that any workgroup can sum all of their rows (a
// CU reads some 40 GB/s: 1024 x 256 bf16 of one id 14 us, 17 in three launches), and a table that a
// workgroup a CU, as far as kFewRange goes, clears as fast as many would.
constexpr uint64_t kFewElements = 1 << 18, kFewCleared = 1 << 24;
uint64_t few_lanes(uint64_t width) { return width <= 16 * 8 ? 16 : width <= 32 * 8 ? 32 : kLanes; }
uint64_t few_range(uint64_t vocab, uint64_t width) {
    return std::min<uint64_t>(over(vocab * over(width, few_lanes(width) * 8), 256 * 32) * 32, kFewRange);
}
bool few(uint64_t tokens, uint64_t vocab, uint64_t width, bool accumulate) {
    return tokens <= kFewTokens && tokens * width <= kFewElements &&
           over(vocab, few_range(vocab, width)) * over(width, few_lanes(width) * 8) <= 1024 &&
           (accumulate || vocab * width <= kFewCleared);
}

struct GradSpace {
    uint64_t keys = 0, places = 0, sorted = 0, order = 0, sort = 0, sort_bytes = 0, present = 0, long_count = 0, longs = 0, parts = 0, total = 0;
};
int key_bits(uint64_t vocab) {
    int b = 1;
    while ((vocab >> b) != 0) ++b;  // keys are at most vocab
    return b;
}
GradSpace grad_space(uint64_t tokens, uint64_t vocab, uint64_t width, const lrs_options *opts) {
    GradSpace w;
    if (tokens == 0 || vocab == 0 || width == 0) return w;
    auto place = [&](uint64_t bytes) {
        const uint64_t at = w.total;
        w.total += (bytes + 255) / 256 * 256;
        return at;
    };
    w.sorted = place(4 * tokens);
    w.order = place(4 * tokens);
    w.present = place(over(vocab, 32) * 4);
    if (!ordered_directly(tokens, vocab)) {
        w.keys = place(4 * tokens);
        w.places = place(4 * tokens);
        w.sort_bytes = radix_sort_workspace_size(tokens, 0, key_bits(vocab), 8, 1, opts);
        w.sort = place(w.sort_bytes);
    }
    const uint64_t runs = over(tokens, run_of(tokens, width)), lanes = lanes_of(width);
    w.long_count = place(8);
    w.longs = place(runs * sizeof(Long));
    w.parts = place(2 * runs * over(width, lanes * 8) * lanes * 8 * sizeof(float));
    return w;
}

template <int T, int O, int LANES, int MODE> void launch_sums(GradArgs a, const Ctx &c) {
    a.pieces = static_cast<uint32_t>(over(a.width, LANES * 8));
    a.run = static_cast<uint32_t>(run_of(a.tokens, a.width));
    a.runs = static_cast<uint32_t>(over(a.tokens, a.run));
    const uint64_t tasks = static_cast<uint64_t>(a.runs) * a.pieces;
    const uint64_t clears = MODE == kAdd ? 0 : std::min(over(a.vocab, 32) * over(over(a.width, Row<O>::kVec), kClearPiece), kMaxGrid);
    a.sum_blocks = static_cast<uint32_t>(std::min(over(tasks, kEmbBlock / kLanes), kMaxGrid));
    if (a.sum_blocks + clears == 0) return;
    {
        TimedLaunch t(4, c);
        launch_on(embed_sum_kernel<T, O, LANES, MODE>, dim3(static_cast<uint32_t>(a.sum_blocks + clears)), dim3(kEmbBlock), t.L, a);
    }
    if (a.tokens < a.run || hipPeekAtLastError() != hipSuccess) return;
    TimedLaunch t(4, c);
    launch_on(embed_join_kernel<O, LANES, T == kRowF32 || O == kRowF32>, dim3(static_cast<uint32_t>(std::min<uint64_t>(tasks * (LANES / 16), 512))),
              dim3(kJoinBlock), t.L, a);
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
    const uint64_t lanes = width <= 16 * 8 ? 16 : width <= 32 * 8 ? 32 : kLanes;
    a.tasks = static_cast<uint32_t>(over(width, lanes * 8 * kSlots));
    const uint64_t tasks = lanes < kLanes ? over(count, kSlots) : static_cast<uint64_t>(count) * a.tasks;
    const dim3 grid(static_cast<uint32_t>(std::min(over(tasks, kEmbBlock / lanes), kMaxGrid)));
    TimedLaunch t(4, c);
    by_types(dtype, out_dtype, [&](auto i, auto o) {
        const auto go = [&](auto kernel) { launch_on(kernel, grid, dim3(kEmbBlock), t.L, a); };
        if (lanes == 16) go(lookup_kernel<i.value, o.value, 16>);
        else if (lanes == 32) go(lookup_kernel<i.value, o.value, 32>);
        else go(lookup_kernel<i.value, o.value, kLanes>);
    });
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
    // exact for tokens below 2^16, and lengths up to there
    a.line_factor = static_cast<uint32_t>(over(uint64_t(1) << 32, std::max<uint32_t>(2, a.ids.length)));
    if (count > 0 && few(count, vocab, width, a.accumulate)) {
        a.range = static_cast<uint32_t>(few_range(vocab, width));
        TimedLaunch t(4, c);
        by_types(dtype, out_dtype, [&](auto i, auto o) {
            const uint64_t lanes = few_lanes(width);
            const dim3 grid(static_cast<uint32_t>(over(vocab, a.range)), static_cast<uint32_t>(over(width, lanes * 8)));
            const auto go = [&](auto adds, auto sets) { launch_on(a.accumulate ? adds : sets, grid, dim3(kOrderBlock), t.L, a); };
            if (lanes == 16) go(embed_few_kernel<i.value, o.value, 16, kAdd>, embed_few_kernel<i.value, o.value, 16, kSumsOnce>);
            else if (lanes == 32) go(embed_few_kernel<i.value, o.value, 32, kAdd>, embed_few_kernel<i.value, o.value, 32, kSumsOnce>);
            else go(embed_few_kernel<i.value, o.value, kLanes, kAdd>, embed_few_kernel<i.value, o.value, kLanes, kSumsOnce>);
        });
        return hipGetLastError() == hipSuccess ? LRS_OK : LRS_ERR_HIP;
    }
    if (count > 0) {
        uint32_t *sorted = reinterpret_cast<uint32_t *>(ws + w.sorted), *order = reinterpret_cast<uint32_t *>(ws + w.order);
        a.sorted = sorted;
        a.order = order;
        a.long_count = reinterpret_cast<uint32_t *>(ws + w.long_count);
        a.longs = reinterpret_cast<Long *>(ws + w.longs);
        a.present = reinterpret_cast<uint32_t *>(ws + w.present);
        a.parts = reinterpret_cast<float *>(ws + w.parts);
        const bool direct = ordered_directly(count, vocab);
        {
            TimedLaunch t(4, c);
            if (direct) {
                a.range = static_cast<uint32_t>(range_of(vocab));
                const dim3 grid(static_cast<uint32_t>(over(vocab, a.range)));
                const auto go = [&](auto wide, auto narrow) {
                    a.ids.bytes == 8 ? launch_on(wide, grid, dim3(kOrderBlock), t.L, a, sorted, order)
                                     : launch_on(narrow, grid, dim3(kOrderBlock), t.L, a, sorted, order);
                };
                if (count <= 2 * kOrderBlock) go(embed_order_kernel<2, int64_t>, embed_order_kernel<2, int32_t>);
                else if (count <= 8 * kOrderBlock) go(embed_order_kernel<8, int64_t>, embed_order_kernel<8, int32_t>);
                else if (count <= 16 * kOrderBlock) go(embed_order_kernel<16, int64_t>, embed_order_kernel<16, int32_t>);
                else go(embed_order_kernel<32, int64_t>, embed_order_kernel<32, int32_t>);
            } else {
                a.keys = reinterpret_cast<uint32_t *>(ws + w.keys);
                a.places = reinterpret_cast<uint32_t *>(ws + w.places);
                launch_on(embed_keys_kernel, dim3((a.tokens + kEmbBlock - 1) / kEmbBlock), dim3(kEmbBlock), t.L, a);
            }
        }
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
        if (!direct) {
            st = radix_sort_pairs(a.keys, a.places, sorted, order, a.tokens, 0, key_bits(vocab), 8, ws + w.sort, w.sort_bytes,
                                  stream, opts);
            if (st != LRS_OK) return st;
            if (!a.accumulate) {
                TimedLaunch t(4, c);
                launch_on(embed_present_kernel, dim3((a.tokens + kEmbBlock - 1) / kEmbBlock), dim3(kEmbBlock), t.L, a);
                if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
            }
        }
    }
    by_types(dtype, out_dtype, [&](auto i, auto o) {
        const auto go = [&](auto mode) {
            constexpr int kMode = decltype(mode)::value;
            lanes_of(width) == 16 ? launch_sums<i.value, o.value, 16, kMode>(a, c) : launch_sums<i.value, o.value, kLanes, kMode>(a, c);
        };
        // Beside reads past the caches: a gradient far larger than the 256 MB
        // behind the L2s is cleared past them, and its sums are not (1.07 GB from
        // 32768 tokens: 228 us, 252 with both and 269 with neither); of a smaller one the
        // sums are (320 MB from 8188 tokens: 63 us, 76 with both, 71 with neither).
        if (a.accumulate) go(std::integral_constant<int, kAdd>());
        else if (wb > (uint64_t(512) << 20)) go(std::integral_constant<int, kClearOnce>());
        else go(std::integral_constant<int, kSumsOnce>());
    });
    return hipGetLastError() == hipSuccess ? LRS_OK : LRS_ERR_HIP;
} catch (...) {
    return LRS_ERR_HIP;
}

}  // extern "C"
