// lrs_balance.hip -- per-expert counts and the load balance loss (gfx950).
//
// c_e counts the chosen slots of expert e, f_e = E c_e / sum c.  With p the
// softmax (or normalised sigmoid) of a row of router logits, b = sum_e f_e p_e
// and z = log sum exp, the loss is the mean over the n counted rows of
// alpha b + beta z^2; its gradient is p_e (alpha (f_e - b) + 2 beta z) / n for the
// softmax and alpha p_e (1 - sigmoid_e)(f_e - b) / n for the sigmoid.  The counts
// are the digit histogram of the expert ids; they carry no gradient.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/lsd_radix_sort.h"
#include "lrs_host.h"
#include "lrs_rows.h"

namespace lrs {
namespace {

constexpr int kBalBlock = 256;
constexpr int kBalWaves = kBalBlock / kLanes;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

struct CountArgs {
    const void *idx;
    int idx_bytes;
    uint64_t stride;
    const uint8_t *mask;
    int32_t *counts;
    int32_t *kept;
    uint64_t rows;
    uint32_t k, experts;
};

// The counts alone, for a program that adds them up over ranks: a clearing
// launch, then histograms in LDS that go out by atomics.  524288 ids of 256
// experts 10.2 us (floor 0.7), 128 ids of 64 3.6 us: bound by the two launches
// and a load, a division and an LDS add one after the other for each id.
__global__ __launch_bounds__(kBalBlock) void count_clear_kernel(CountArgs a) {
    for (uint32_t e = threadIdx.x; e < a.experts; e += kBalBlock) a.counts[e] = 0;
    if (threadIdx.x == 0 && a.kept) *a.kept = 0;
}

__global__ __launch_bounds__(kBalBlock) void count_kernel(CountArgs a) {
    __shared__ int32_t hist[LRS_MAX_EXPERTS];
    __shared__ int32_t kept;
    for (uint32_t e = threadIdx.x; e < a.experts; e += kBalBlock) hist[e] = 0;
    if (threadIdx.x == 0) kept = 0;
    __syncthreads();
    // rows * k and rows are below 2^31, and 32-bit divisions cost a fifth of 64-bit ones
    const uint32_t total = static_cast<uint32_t>(a.rows * a.k), step = gridDim.x * kBalBlock;
    const uint32_t rows = static_cast<uint32_t>(a.rows);
    for (uint32_t i = blockIdx.x * kBalBlock + threadIdx.x; i < total; i += step) {
        const uint32_t row = i / a.k;
        const uint64_t at = row * a.stride + (i - row * a.k);
        if (a.mask && !a.mask[row]) continue;
        const int64_t e = a.idx_bytes == 8 ? static_cast<const int64_t *>(a.idx)[at] : static_cast<const int32_t *>(a.idx)[at];
        if (e >= 0 && e < a.experts) atomicAdd(&hist[e], 1);
    }
    if (a.kept && a.mask) {
        int32_t mine = 0;
        for (uint32_t r = blockIdx.x * kBalBlock + threadIdx.x; r < rows; r += step)
            mine += a.mask[r] != 0;
        mine = wave_sum(mine);
        if (threadIdx.x % kLanes == 0) atomicAdd(&kept, mine);
    }
    __syncthreads();
    // whole numbers: the order of these adds does not show
    for (uint32_t e = threadIdx.x; e < a.experts; e += kBalBlock)
        if (hist[e]) atomicAdd(&a.counts[e], hist[e]);
    if (threadIdx.x == 0 && a.kept) {
        if (a.mask) atomicAdd(a.kept, kept);
        else if (blockIdx.x == 0) *a.kept = static_cast<int32_t>(a.rows);
    }
}

// The counts of a whole call by several workgroups: each its own share of the
// ids, [blocks][experts + 1], the counted rows of its share last.  No order and
// no clearing is needed; whoever uses the counts adds the shares.  524288 ids in
// 64 shares: 4.2 us, two trips to memory and the LDS adds (32 shares: 6.3 us, 8
// shares 13.5 us; adding them up costs 1.7 us more for 64 than for 8).
constexpr int kShareBlock = 1024;
constexpr uint32_t kShareIds = 8;  // a thread has in flight

struct IdArgs {
    const void *idx;
    int idx_bytes;
    uint64_t stride;
    const uint8_t *mask;
    uint32_t rows, k, experts;
};
__device__ inline int64_t id_at(const IdArgs &a, uint64_t at) {
    return a.idx_bytes == 8 ? static_cast<const int64_t *>(a.idx)[at] : static_cast<const int32_t *>(a.idx)[at];
}
// Adds ids [first, last) of the rows x k matrix, and the rows [row0, row1) that
// count, to a histogram in LDS (experts + 1 cells, cleared by the caller).
template <int B> __device__ void count_ids(const IdArgs &a, uint32_t first, uint32_t last, uint32_t row0, uint32_t row1,
                                           int32_t *hist) {
    const bool dense = a.stride == a.k && !a.mask;
    for (uint32_t base = first + threadIdx.x; base < last; base += B * kShareIds) {
        int64_t id[kShareIds];
#pragma unroll
        for (uint32_t u = 0; u < kShareIds; ++u) {
            const uint32_t i = base + u * B;
            id[u] = -1;
            if (i < last && base <= 0xFFFFFFFFu - u * B) {
                const uint32_t row = dense ? 0 : i / a.k;
                if (dense || !a.mask || a.mask[row])
                    id[u] = id_at(a, dense ? i : static_cast<uint64_t>(row) * a.stride + (i - row * a.k));
            }
        }
#pragma unroll
        for (uint32_t u = 0; u < kShareIds; ++u)
            if (id[u] >= 0 && id[u] < a.experts) atomicAdd(&hist[id[u]], 1);
    }
    int32_t kept = 0;
    for (uint32_t r = row0 + threadIdx.x; r < row1; r += B) kept += !a.mask || a.mask[r];
    kept = wave_sum(kept);
    if (threadIdx.x % kLanes == 0 && kept) atomicAdd(&hist[a.experts], kept);
}

__global__ __launch_bounds__(kShareBlock) void count_share_kernel(IdArgs a, int32_t *shares, uint32_t *ticket) {
    __shared__ int32_t hist[LRS_MAX_EXPERTS + 1];
    for (uint32_t e = threadIdx.x; e <= a.experts; e += kShareBlock) hist[e] = 0;
    __syncthreads();
    const uint32_t total = a.rows * a.k, blocks = gridDim.x, b = blockIdx.x;
    const uint64_t t = total, r = a.rows;
    count_ids<kShareBlock>(a, static_cast<uint32_t>(t * b / blocks), static_cast<uint32_t>(t * (b + 1) / blocks),
                           static_cast<uint32_t>(r * b / blocks), static_cast<uint32_t>(r * (b + 1) / blocks), hist);
    __syncthreads();
    for (uint32_t e = threadIdx.x; e <= a.experts; e += kShareBlock)
        shares[static_cast<uint64_t>(b) * (a.experts + 1) + e] = hist[e];
    if (b == 0 && threadIdx.x == 0) *ticket = 0;
}

struct BalArgs {
    const void *x;
    uint64_t stride;
    uint64_t rows;
    uint32_t experts;
    uint32_t lanes;           // that share a row
    const uint8_t *mask;
    // the counts: given, or as shares, or (neither) counted from `ids` by the one workgroup there is
    const int32_t *counts;
    const int32_t *kept;
    const int32_t *shares;
    uint32_t share_count;
    IdArgs ids;
    int32_t *counts_out;      // with shares or ids
    int32_t *kept_out;
    float alpha, beta;
    double *partial;          // by workgroup
    uint32_t *ticket;         // workgroups that are done; null: another kernel adds the partial sums
    uint32_t blocks;
    float *loss;
    const float *loss_grad;
    void *grad;
    uint64_t grad_stride;
};

__device__ inline float mean_of(double sum, int32_t kept) { return kept > 0 ? static_cast<float>(sum / kept) : 0.f; }

// A row's elements in the registers of `lanes` neighbours, V loads of 16 bytes
// each, from its one read to the gradient; 64 / lanes rows a wave at a time.
// 65536 x 256 bf16: 18.5 us, 3.6 TB/s.  Some 200 vector instructions a turn of 16
// elements a lane and 500 around the turns take 12 us of it, adding up the counts
// and taking the ticket 4 us.
template <int T, bool SIG, int V, int B>
__global__ __launch_bounds__(B) void balance_kernel(BalArgs a) {
    constexpr int kVec = Row<T>::kVec;
    using Stored = typename Row<T>::Stored;
    __shared__ int32_t hist[LRS_MAX_EXPERTS + 1];
    __shared__ __align__(16) float shared_load[LRS_MAX_EXPERTS + 8];
    __shared__ double part[(B / kLanes)];
    __shared__ int64_t sums[(B / kLanes)];
    __shared__ uint32_t arrived;
    const uint32_t tid = threadIdx.x, E = a.experts;
    const int lane = tid % kLanes, wave = tid / kLanes;
    const uint32_t sub = lane % a.lanes;

    // the first rows are on their way while the counts are added up
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * (B / a.lanes);
    uint64_t row = static_cast<uint64_t>(blockIdx.x) * (B / a.lanes) + tid / a.lanes;
    const uint32_t none = T == kRowF16 ? 0xFC00FC00u : T == kRowBF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
    u32x4 v[V];
#pragma unroll
    for (int u = 0; u < V; ++u) v[u] = u32x4{none, none, none, none};
    bool counted = false;
    // a place past the row's end keeps -inf; a row that does not count keeps
    // what was there, and nothing comes of it
    const auto load_row = [&](uint64_t r) {
        counted = r < a.rows && (!a.mask || a.mask[r]);
        if (!counted) return;
        const Stored *x = static_cast<const Stored *>(a.x) + r * a.stride;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const uint32_t at = (u * a.lanes + sub) * kVec;
            if (at + kVec <= E) v[u] = load16_once(x + at);
            if (E % kVec != 0 && at < E && at + kVec > E) {
                float f[kVec];
                for (int e = 0; e < kVec; ++e) f[e] = at + e < E ? Row<T>::value(x[at + e]) : -INFINITY;
                v[u] = pack16<T>(f);
            }
        }
    };
    load_row(row);

    if (a.counts) {
        for (uint32_t e = tid; e < E; e += B) hist[e] = a.counts[e];
        if (tid == 0) hist[E] = a.kept ? *a.kept : static_cast<int32_t>(a.rows);
    } else if (a.shares) {
        // a thread a cell, or several where there are fewer cells
        const uint32_t team = max(1u, B / (E + 1));
        for (uint32_t e = tid; e <= E; e += B) hist[e] = 0;
        __syncthreads();
        for (uint32_t i = tid; i < team * (E + 1); i += B) {
            const uint32_t e = i % (E + 1);
            int32_t c = 0;
            for (uint32_t b = i / (E + 1); b < a.share_count; b += 8 * team) {
                int32_t part[8];
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const uint32_t s = b + j * team;
                    part[j] = s < a.share_count ? a.shares[s * (E + 1) + e] : 0;
                }
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) c += part[j];
            }
            atomicAdd(&hist[e], c);
        }
    } else {
        for (uint32_t e = tid; e <= E; e += B) hist[e] = 0;
        __syncthreads();
        count_ids<B>(a.ids, 0, a.ids.rows * a.ids.k, 0, a.ids.rows, hist);
    }
    __syncthreads();
    int64_t total = 0;
    for (uint32_t e = tid; e < E; e += B) total += hist[e];
    total = wave_sum(total);
    if (lane == 0) sums[wave] = total;
    if (!a.counts && blockIdx.x == 0) {
        for (uint32_t e = tid; e < E; e += B) a.counts_out[e] = hist[e];
        if (tid == 0 && a.kept_out) *a.kept_out = hist[E];
    }
    __syncthreads();
    total = 0;
    for (int w = 0; w < (B / kLanes); ++w) total += sums[w];
    const int32_t kept = hist[E];
    const double per = total > 0 ? static_cast<double>(E) / static_cast<double>(total) : 0;
    for (uint32_t e = tid; e < E + kVec; e += B) shared_load[e] = e < E ? static_cast<float>(hist[e] * per) : 0.f;
    __syncthreads();
    // this lane's columns stay the same from row to row
    float load[V][kVec];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const uint32_t at = min((u * a.lanes + sub) * kVec, E / kVec * kVec);  // places past the row hold -inf
#pragma unroll
        for (int e = 0; e < kVec; e += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(shared_load + at + e);
            load[u][e] = f.x;
            load[u][e + 1] = f.y;
            load[u][e + 2] = f.z;
            load[u][e + 3] = f.w;
        }
    }
    const float inv = kept > 0 ? 1.f / kept : 0.f;
    const float up = (a.loss_grad ? *a.loss_grad : 1.f) * inv;
    double loss = 0;
    // every group of a wave makes the same number of turns
    for (uint64_t base = row - tid / a.lanes; base < a.rows; base += step, row += step) {
        const bool mine = counted;
        float w[V][kVec];
#pragma unroll
        for (int u = 0; u < V; ++u) unpack16<T>(v[u], w[u]);
        if (base + step < a.rows) load_row(row + step);
        // exponents of 2 relative to `ref`: x log2(e) - ref, x taken from `from`,
        // the largest logit, in rows where that is so large that the rounding of
        // ref (2^-4 at 2^20, 2^7 at 2^32) would show as the largest's own exponent
        float ref = 0, from = 0, one = 1;
        const auto largest = [&]() {
            float m = w[0][0];
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int e = 0; e < kVec; e += 2) m = max3(m, w[u][e], w[u][e + 1]);
            m = group_max(m, a.lanes);
            return m == -INFINITY ? 0.f : m;
        };
        const auto take_from = [&](float logit) {
            from = logit;
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int e = 0; e < kVec; ++e) w[u][e] -= from;
        };
        if (SIG) {
            // Sigmoids below 2^-126 are 0, which would empty a row that lies far
            // below 0.  A row whose largest logit m is below -7 takes them times
            // e^-m, which p does not show: 1 / (e^m + e^(m - x)), and 1 - sigmoid
            // is e^(m - x) times that.  Such rows are few: m is looked for only
            // where a row's first logit in each of its lanes is that low.
            constexpr float kFar = -7.f;
            uint64_t low = __ballot(w[0][0] < kFar);
            for (uint32_t d = 1; d < a.lanes; d *= 2) low &= low >> d;
            if (low) {
                const float m = largest();
                take_from(m < kFar ? m : 0.f);
                one = __builtin_amdgcn_exp2f(from * kLog2e);
            }
        } else {
            const float m = largest();
            if (__any(fabsf(m) > 0x1p20f)) take_from(fabsf(m) > 0x1p20f ? m : 0.f);
            ref = (m - from) * kLog2e;
        }
        float s = 0, b = 0;
        float slope[SIG ? V : 1][kVec];  // sigmoid times 1 - sigmoid, without the cancellation
        const auto add = [&](int u, int e, float x) {
            w[u][e] = x;
            s += x;
            b = fmaf(x, load[u][e], b);
        };
        if (SIG) {
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float t = __builtin_amdgcn_exp2f(-w[u][e] * kLog2e), g = __builtin_amdgcn_rcpf(one + t);
                    slope[SIG ? u : 0][e] = g == 0.f ? 0.f : g * (g * t);
                    add(u, e, g);
                }
        } else {
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int e = 0; e < kVec; ++e) add(u, e, __builtin_amdgcn_exp2f(fmaf(w[u][e], kLog2e, -ref)));
        }
        const float2 sums = group_join(make_float2(s, b), a.lanes);
        s = sums.x;
        b = sums.y;
        const bool empty = s == 0.f;
        const float r = empty ? 0.f : __builtin_amdgcn_rcpf(s);
        b *= r;
        const float z = SIG || empty ? 0.f : fmaf(ref + __builtin_amdgcn_logf(s), kLn2, from);
        if (mine && sub == 0) loss += static_cast<double>(a.alpha * b + a.beta * z * z);
        if (a.grad && row < a.rows) {
            Stored *g = static_cast<Stored *>(a.grad) + row * a.grad_stride;
            const float p = a.alpha * r * up, q = fmaf(2.f * a.beta * z, r * up, -p * b);
#pragma unroll
            for (int u = 0; u < V; ++u) {
                const uint32_t at = (u * a.lanes + sub) * kVec;
                if (at >= E) continue;
                float d[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    d[e] = (SIG ? slope[SIG ? u : 0][e] : w[u][e]) * fmaf(p, load[u][e], q);
                const u32x4 out = mine ? pack16<T>(d) : u32x4{0, 0, 0, 0};
                if (at + kVec <= E) {
                    store16_once(g + at, out);
                } else {
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        if (at + e < E) g[at + e] = mine ? Row<T>::pattern(d[e]) : 0;
                }
            }
        }
    }
    if (!a.loss) return;
    loss = wave_sum(loss);
    if (lane == 0) part[wave] = loss;
    __syncthreads();
    if (tid == 0) {
        loss = 0;
        for (int w = 0; w < (B / kLanes); ++w) loss += part[w];
        if (gridDim.x == 1) {
            *a.loss = mean_of(loss, kept);
        } else if (!a.ticket) {
            a.partial[blockIdx.x] = loss;
        } else {
            // the exchange has come back before the ticket is taken, so the
            // last workgroup finds every sum at the memory all XCDs share
            unsigned long long was = __hip_atomic_exchange(reinterpret_cast<unsigned long long *>(a.partial + blockIdx.x),
                                                           __builtin_bit_cast(unsigned long long, loss), __ATOMIC_RELAXED,
                                                           __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("" : "+v"(was)::"memory");
            arrived = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    if (gridDim.x == 1 || !a.ticket) return;
    __syncthreads();
    if (arrived != gridDim.x - 1) return;
    loss = 0;
    for (uint32_t i = tid; i < gridDim.x; i += B)
        loss += __builtin_bit_cast(double, __hip_atomic_load(reinterpret_cast<unsigned long long *>(a.partial + i),
                                                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    loss = wave_sum(loss);
    if (lane == 0) part[wave] = loss;
    __syncthreads();
    if (tid == 0) {
        loss = 0;
        for (int w = 0; w < (B / kLanes); ++w) loss += part[w];
        *a.loss = mean_of(loss, kept);
    }
}

// The mean, from the workgroups' sums in a fixed order.
__global__ __launch_bounds__(kBalBlock) void balance_loss_kernel(BalArgs a) {
    __shared__ double part[kBalWaves];
    double s = 0;
    for (uint32_t i = threadIdx.x; i < a.blocks; i += kBalBlock) s += a.partial[i];
    s = wave_sum(s);
    if (threadIdx.x % kLanes == 0) part[threadIdx.x / kLanes] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0;
        for (int w = 0; w < kBalWaves; ++w) s += part[w];
        *a.loss = mean_of(s, a.kept ? *a.kept : static_cast<int32_t>(a.rows));
    }
}

// How a row is laid over lanes: the fewest places for its 16-byte words with at
// most 3 a lane (or as many as 64 lanes need), and of those the fewest lanes,
// whose sums take the fewest steps.
void balance_layout(uint64_t vecs, uint32_t &lanes, uint32_t &per_lane) {
    uint64_t best = ~uint64_t(0);
    lanes = 64;
    per_lane = 4;
    while (lanes * per_lane < vecs) per_lane *= 2;
    for (uint32_t l = 1; l <= 64; l *= 2)
        for (uint32_t p = 1; p <= 3; ++p)
            if (l * p >= vecs && l * p < best) {
                best = l * p;
                lanes = l;
                per_lane = p;
            }
}
// Workgroups of 1024 threads, one a CU, as every one of them adds up the counts
// first and takes the ticket last (65536 x 256 bf16: 25 us so, 29 us with 512
// of 256 threads, 33 us with 1024 of them); rows of more than 3 loads a lane
// need the registers of 256 threads.
constexpr uint32_t balance_block(uint32_t per_lane) { return per_lane <= 3 ? 1024 : kBalBlock; }
constexpr uint64_t kBalMaxBlocks = 1024;
uint32_t balance_blocks(uint64_t rows, uint64_t experts, uint64_t size) {
    uint32_t lanes, per_lane;
    balance_layout((experts * size + 15) / 16, lanes, per_lane);
    const uint64_t block = balance_block(per_lane), each = block / lanes;
    return static_cast<uint32_t>(std::min<uint64_t>(256 * 1024 / block, (rows + each - 1) / each));
}

template <int T, bool SIG> void balance_launch(const BalArgs &a, uint32_t per_lane, const Launch &L) {
    const auto go = [&](auto kernel) { launch_on(kernel, dim3(a.blocks), dim3(balance_block(per_lane)), L, a); };
    switch (per_lane) {
    case 1: return go(balance_kernel<T, SIG, 1, balance_block(1)>);
    case 2: return go(balance_kernel<T, SIG, 2, balance_block(2)>);
    case 3: return go(balance_kernel<T, SIG, 3, balance_block(3)>);
    case 4: return go(balance_kernel<T, SIG, 4, balance_block(4)>);
    case 8: return go(balance_kernel<T, SIG, 8, balance_block(8)>);
    default:
        if constexpr (T == kRowF32) go(balance_kernel<T, SIG, 16, balance_block(16)>);  // 16-bit rows need 8 at most
    }
}
int balance_launch(BalArgs a, int dtype, int score, const Ctx &c) {
    uint32_t per_lane;
    balance_layout((a.experts * row_type_size(dtype) + 15) / 16, a.lanes, per_lane);
    TimedLaunch t(4, c);
    const bool sig = score == LRS_SCORE_SIGMOID;
    if (dtype == LRS_DTYPE_FP16) sig ? balance_launch<kRowF16, true>(a, per_lane, t.L) : balance_launch<kRowF16, false>(a, per_lane, t.L);
    else if (dtype == LRS_DTYPE_BF16) sig ? balance_launch<kRowBF16, true>(a, per_lane, t.L) : balance_launch<kRowBF16, false>(a, per_lane, t.L);
    else sig ? balance_launch<kRowF32, true>(a, per_lane, t.L) : balance_launch<kRowF32, false>(a, per_lane, t.L);
    return hipGetLastError() == hipSuccess ? LRS_OK : LRS_ERR_HIP;
}

// One workgroup counts and takes the rows where both are little work.
constexpr uint64_t kAloneIds = 4096, kAloneElems = 32768;
uint32_t count_shares(uint64_t ids) {
    return static_cast<uint32_t>(std::min<uint64_t>(64, std::max<uint64_t>(1, ids / (kShareBlock * kShareIds))));
}
struct BalSpace {
    uint64_t partial = 0, ticket = 0, shares = 0, total = 0;
};
BalSpace balance_space(uint64_t rows, uint64_t k, uint64_t experts) {
    BalSpace w;
    w.ticket = kBalMaxBlocks * sizeof(double);
    w.shares = w.ticket + 256;
    w.total = w.shares + count_shares(rows * k) * (experts + 1) * sizeof(int32_t);
    return w;
}

int check_ids(int64_t index_stride, int index_bytes, int64_t rows, int64_t k, int64_t experts) {
    if (index_bytes != 4 && index_bytes != 8) return LRS_ERR_DTYPE;
    if (rows < 0 || k < 0 || experts < 1 || experts > LRS_MAX_EXPERTS || !stride_ok(index_stride, rows) ||
        rows > INT32_MAX || (k > 0 && rows > INT32_MAX / k))
        return LRS_ERR_SIZE;
    return LRS_OK;
}
int check_balance(int64_t row_stride, int64_t rows, int64_t experts, int dtype, int score, float balance_weight,
                  float z_weight, const void *grad, int64_t grad_stride) {
    if (!row_type_ok(dtype)) return LRS_ERR_DTYPE;
    if ((score != LRS_SCORE_SOFTMAX && score != LRS_SCORE_SIGMOID) || !std::isfinite(balance_weight) ||
        !std::isfinite(z_weight) || (score == LRS_SCORE_SIGMOID && z_weight != 0.f))
        return LRS_ERR_OPTION;
    if (rows < 0 || rows > INT32_MAX || experts < 1 || experts > LRS_MAX_EXPERTS || !stride_ok(row_stride, rows) ||
        (grad && (!stride_ok(grad_stride, rows) || (rows > 1 && grad_stride < experts))))
        return LRS_ERR_SIZE;
    return LRS_OK;
}

}  // namespace
}  // namespace lrs

using namespace lrs;

extern "C" {

int expert_counts(const void *indices, int64_t index_stride, int index_bytes, const uint8_t *row_mask,
                  int32_t *counts_out, int32_t *rows_counted, int64_t rows, int64_t k, int64_t experts, void *stream,
                  const lrs_options *opts) try {
    Ctx c;
    if (!make_ctx(stream, opts, c)) return LRS_ERR_OPTION;
    const int st = check_ids(index_stride, index_bytes, rows, k, experts);
    if (st != LRS_OK) return st;
    const bool some = rows > 0 && k > 0;
    if (!counts_out || (some && !indices)) return LRS_ERR_NULL_POINTER;
    if (misaligned(indices, index_bytes) || misaligned(counts_out, 4) || misaligned(rows_counted, 4)) return LRS_ERR_ALIGNMENT;
    const uint64_t ib = some ? span(rows, index_stride, k, index_bytes) : 0, mb = row_mask ? rows : 0;
    const uint64_t cb = 4 * experts, kb = rows_counted ? 4 : 0;
    if (overlaps(counts_out, cb, indices, ib) || overlaps(counts_out, cb, row_mask, mb) ||
        overlaps(rows_counted, kb, indices, ib) || overlaps(rows_counted, kb, row_mask, mb) ||
        overlaps(rows_counted, kb, counts_out, cb))
        return LRS_ERR_ALIASING;
    CountArgs a{indices, index_bytes, static_cast<uint64_t>(index_stride), row_mask, counts_out, rows_counted,
                static_cast<uint64_t>(rows), static_cast<uint32_t>(k), static_cast<uint32_t>(experts)};
    c.elems = a.rows * a.k;
    {
        TimedLaunch t(4, c);
        launch_on(count_clear_kernel, dim3(1), dim3(kBalBlock), t.L, a);
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
    }
    if (rows == 0) return LRS_OK;
    TimedLaunch t(4, c);
    const uint64_t work = std::max<uint64_t>(a.rows, a.rows * a.k);
    launch_on(count_kernel, dim3(static_cast<uint32_t>(std::min<uint64_t>(256, (work + 2047) / 2048))), dim3(kBalBlock), t.L, a);
    return hipGetLastError() == hipSuccess ? LRS_OK : LRS_ERR_HIP;
} catch (...) {
    return LRS_ERR_HIP;
}

size_t expert_balance_workspace_size(int64_t rows, int64_t experts, const lrs_options *opts) {
    if (!options_ok(opts) || rows < 1 || rows > INT32_MAX || experts < 1 || experts > LRS_MAX_EXPERTS) return 0;
    return kBalMaxBlocks * sizeof(double);
}

int expert_balance(const void *logits, int64_t row_stride, const int32_t *counts, const int32_t *rows_counted,
                   const uint8_t *row_mask, int64_t rows, int64_t experts, int dtype, int score, float balance_weight,
                   float z_weight, float *loss, const float *loss_grad, void *grad, int64_t grad_stride, void *workspace,
                   size_t workspace_bytes, void *stream, const lrs_options *opts) try {
    Ctx c;
    if (!make_ctx(stream, opts, c)) return LRS_ERR_OPTION;
    const int st = check_balance(row_stride, rows, experts, dtype, score, balance_weight, z_weight, grad, grad_stride);
    if (st != LRS_OK) return st;
    const uint64_t size = row_type_size(dtype);
    const uint64_t need = loss ? expert_balance_workspace_size(rows, experts, nullptr) : 0;
    if ((!loss && !grad && rows > 0) || !counts || (rows > 0 && !logits) || (need && !workspace) || (row_mask && !rows_counted))
        return LRS_ERR_NULL_POINTER;
    if (misaligned(logits, size) || misaligned(grad, size) || misaligned(counts, 4) || misaligned(rows_counted, 4) ||
        misaligned(loss, 4) || misaligned(loss_grad, 4) || (need && misaligned(workspace, 256)))
        return LRS_ERR_ALIGNMENT;
    if (workspace_bytes < need) return LRS_ERR_WORKSPACE_TOO_SMALL;
    const uint64_t gb = grad ? span(rows, grad_stride, experts, size) : 0, lb = loss ? 4 : 0;
    const void *in[] = {logits, counts, rows_counted, row_mask, loss_grad};
    const uint64_t inb[] = {span(rows, row_stride, experts, size), 4 * static_cast<uint64_t>(experts),
                            rows_counted ? 4u : 0u, row_mask ? static_cast<uint64_t>(rows) : 0, loss_grad ? 4u : 0u};
    for (int i = 0; i < 5; ++i)
        if (overlaps(grad, gb, in[i], inb[i]) || overlaps(loss, lb, in[i], inb[i]) || overlaps(workspace, need, in[i], inb[i]))
            return LRS_ERR_ALIASING;
    if (overlaps(grad, gb, loss, lb) || overlaps(workspace, need, grad, gb) || overlaps(workspace, need, loss, lb))
        return LRS_ERR_ALIASING;
    BalArgs a{};
    a.x = logits;
    a.stride = static_cast<uint64_t>(row_stride);
    a.rows = static_cast<uint64_t>(rows);
    a.experts = static_cast<uint32_t>(experts);
    a.mask = row_mask;
    a.counts = counts;
    a.kept = rows_counted;
    a.alpha = balance_weight;
    a.beta = z_weight;
    a.partial = static_cast<double *>(workspace);
    a.loss = loss;
    a.loss_grad = loss_grad;
    a.grad = grad;
    a.grad_stride = static_cast<uint64_t>(grad_stride);
    c.elems = a.rows * a.experts;
    if (rows > 0) {
        a.blocks = balance_blocks(a.rows, a.experts, size);
        const int launched = balance_launch(a, dtype, score, c);
        if (launched != LRS_OK) return launched;
    }
    if (loss && a.blocks != 1) {
        TimedLaunch t(4, c);
        launch_on(balance_loss_kernel, dim3(1), dim3(kBalBlock), t.L, a);
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
    }
    return LRS_OK;
} catch (...) {
    return LRS_ERR_HIP;
}

size_t expert_balance_step_workspace_size(int64_t rows, int64_t k, int64_t experts, const lrs_options *opts) {
    if (!options_ok(opts) || check_ids(0, 8, rows, k, experts) != LRS_OK) return 0;
    return static_cast<size_t>(balance_space(rows, k, experts).total);
}

int expert_balance_step(const void *logits, int64_t row_stride, const void *indices, int64_t index_stride, int index_bytes,
                        const uint8_t *row_mask, int64_t rows, int64_t k, int64_t experts, int dtype, int score,
                        float balance_weight, float z_weight, int32_t *counts_out, int32_t *rows_counted, float *loss,
                        void *grad, int64_t grad_stride, void *workspace, size_t workspace_bytes, void *stream,
                        const lrs_options *opts) try {
    Ctx c;
    if (!make_ctx(stream, opts, c)) return LRS_ERR_OPTION;
    int st = check_ids(index_stride, index_bytes, rows, k, experts);
    if (st != LRS_OK) return st;
    st = check_balance(row_stride, rows, experts, dtype, score, balance_weight, z_weight, grad, grad_stride);
    if (st != LRS_OK) return st;
    const uint64_t R = rows, K = k, E = experts, size = row_type_size(dtype);
    const bool some = R > 0 && K > 0;
    const BalSpace w = balance_space(R, K, E);
    if ((R > 0 && !logits) || (some && !indices) || !counts_out || !loss || !workspace) return LRS_ERR_NULL_POINTER;
    if (misaligned(logits, size) || misaligned(grad, size) || misaligned(indices, index_bytes) ||
        misaligned(counts_out, 4) || misaligned(rows_counted, 4) || misaligned(loss, 4) || misaligned(workspace, 256))
        return LRS_ERR_ALIGNMENT;
    if (workspace_bytes < w.total) return LRS_ERR_WORKSPACE_TOO_SMALL;
    const void *in[] = {logits, indices, row_mask};
    const uint64_t inb[] = {span(R, row_stride, E, size), some ? span(R, index_stride, K, index_bytes) : 0, row_mask ? R : 0};
    const void *out[] = {grad, loss, counts_out, rows_counted, workspace};
    const uint64_t outb[] = {grad ? span(R, grad_stride, E, size) : 0, 4, 4 * E, rows_counted ? 4u : 0u, w.total};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 3; ++j)
            if (overlaps(out[i], outb[i], in[j], inb[j])) return LRS_ERR_ALIASING;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], outb[i], out[j], outb[j])) return LRS_ERR_ALIASING;
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    BalArgs a{};
    a.x = logits;
    a.stride = static_cast<uint64_t>(row_stride);
    a.rows = R;
    a.experts = static_cast<uint32_t>(E);
    a.mask = row_mask;
    a.ids = IdArgs{indices, index_bytes, static_cast<uint64_t>(index_stride), row_mask, static_cast<uint32_t>(R),
                   static_cast<uint32_t>(K), static_cast<uint32_t>(E)};
    a.counts_out = counts_out;
    a.kept_out = rows_counted;
    a.alpha = balance_weight;
    a.beta = z_weight;
    a.partial = reinterpret_cast<double *>(ws);
    a.loss = loss;
    a.grad = grad;
    a.grad_stride = static_cast<uint64_t>(grad_stride);
    c.elems = R * E;
    if (R * K <= kAloneIds && R * E <= kAloneElems) {
        a.blocks = 1;
    } else {
        a.blocks = balance_blocks(R, E, size);
        a.ticket = reinterpret_cast<uint32_t *>(ws + w.ticket);
        a.shares = reinterpret_cast<int32_t *>(ws + w.shares);
        a.share_count = count_shares(R * K);
        TimedLaunch t(4, c);
        launch_on(count_share_kernel, dim3(a.share_count), dim3(kShareBlock), t.L, a.ids, const_cast<int32_t *>(a.shares),
                  a.ticket);
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
    }
    return balance_launch(a, dtype, score, c);
} catch (...) {
    return LRS_ERR_HIP;
}

}  // extern "C"
