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
    const uint64_t total = a.rows * a.k, step = static_cast<uint64_t>(gridDim.x) * kBalBlock;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kBalBlock + threadIdx.x; i < total; i += step) {
        const uint64_t row = i / a.k, at = row * a.stride + i % a.k;
        if (a.mask && !a.mask[row]) continue;
        const int64_t e = a.idx_bytes == 8 ? static_cast<const int64_t *>(a.idx)[at] : static_cast<const int32_t *>(a.idx)[at];
        if (e >= 0 && e < a.experts) atomicAdd(&hist[e], 1);
    }
    if (a.kept && a.mask) {
        int32_t mine = 0;
        for (uint64_t r = static_cast<uint64_t>(blockIdx.x) * kBalBlock + threadIdx.x; r < a.rows; r += step)
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

struct BalArgs {
    const void *x;
    uint64_t stride;
    uint64_t rows;
    uint32_t experts;
    const uint8_t *mask;
    const int32_t *counts;
    const int32_t *kept;
    float alpha, beta;
    double *partial;  // by workgroup
    uint32_t blocks;
    float *loss;
    const float *loss_grad;
    void *grad;
    uint64_t grad_stride;
};

// One wave a row.
template <int T, bool SIG, bool LOSS, bool GRAD>
__global__ __launch_bounds__(kBalBlock) void balance_kernel(BalArgs a) {
    using Stored = typename Row<T>::Stored;
    __shared__ float load[LRS_MAX_EXPERTS];
    __shared__ double part[kBalWaves];
    __shared__ int64_t total;
    const int lane = threadIdx.x % kLanes, wave = threadIdx.x / kLanes;
    if (wave == 0) {
        int64_t s = 0;
        for (uint32_t e = lane; e < a.experts; e += kLanes) s += a.counts[e];
        s = wave_sum(s);
        if (lane == 0) total = s;
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.experts; e += kBalBlock)
        load[e] = total > 0 ? static_cast<float>(static_cast<double>(a.counts[e]) * a.experts / total) : 0.f;
    __syncthreads();
    const int32_t kept = a.kept ? *a.kept : static_cast<int32_t>(a.rows);
    const float inv = kept > 0 ? 1.f / kept : 0.f;
    const float up = (GRAD && a.loss_grad ? *a.loss_grad : 1.f) * inv;
    double loss = 0;
    for (uint64_t row = static_cast<uint64_t>(blockIdx.x) * kBalWaves + wave; row < a.rows;
         row += static_cast<uint64_t>(gridDim.x) * kBalWaves) {
        const Stored *x = static_cast<const Stored *>(a.x) + row * a.stride;
        Stored *g = static_cast<Stored *>(a.grad) + row * a.grad_stride;
        const bool counted = !a.mask || a.mask[row];
        if (!counted) {
            if (GRAD)
                for (uint32_t e = lane; e < a.experts; e += kLanes) g[e] = 0;
            continue;
        }
        float m = 0;
        if (!SIG) {
            m = -INFINITY;
            for (uint32_t e = lane; e < a.experts; e += kLanes) m = fmaxf(m, Row<T>::value(x[e]));
            m = wave_max(m);
        }
        float s = 0, b = 0;
        for (uint32_t e = lane; e < a.experts; e += kLanes) {
            const float v = Row<T>::value(x[e]);
            const float w = SIG ? 1.f / (1.f + exp2f(-v * kLog2e)) : v == -INFINITY ? 0.f : exp2f((v - m) * kLog2e);
            s += w;
            b += w * load[e];
        }
        s = wave_sum(s);
        b = wave_sum(b);
        const bool empty = s == 0.f;
        const float r = empty ? 0.f : 1.f / s;
        b *= r;
        const float z = SIG || empty ? 0.f : m + log2f(s) * kLn2;
        if (LOSS) loss += static_cast<double>(a.alpha * b + a.beta * z * z);
        if (GRAD)
            for (uint32_t e = lane; e < a.experts; e += kLanes) {
                const float v = Row<T>::value(x[e]);
                float d;
                if (SIG) {
                    const float t = exp2f(-v * kLog2e), w = 1.f / (1.f + t);
                    // 1 - sigmoid(v) without the cancellation: sigmoid(-v)
                    d = w == 0.f ? 0.f : w * r * (1.f / (1.f + exp2f(v * kLog2e))) * a.alpha * (load[e] - b);
                } else {
                    const float p = v == -INFINITY ? 0.f : exp2f((v - m) * kLog2e) * r;
                    d = p * (a.alpha * (load[e] - b) + 2.f * a.beta * z);
                }
                g[e] = Row<T>::pattern(d * up);
            }
    }
    if (LOSS) {
        if (lane == 0) part[wave] = loss;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kBalWaves; ++w) loss += part[w];
            a.partial[blockIdx.x] = loss;
        }
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
        const int32_t kept = a.kept ? *a.kept : static_cast<int32_t>(a.rows);
        *a.loss = kept > 0 ? static_cast<float>(s / kept) : 0.f;
    }
}

constexpr uint64_t kBalMaxBlocks = 2048;
uint32_t balance_blocks(uint64_t rows) {
    return static_cast<uint32_t>(std::min<uint64_t>(kBalMaxBlocks, (rows + kBalWaves - 1) / kBalWaves));
}

template <int T, bool SIG> void balance_launch(const BalArgs &a, const Ctx &c) {
    TimedLaunch t(4, c);
    const dim3 grid(a.blocks), block(kBalBlock);
    if (a.loss && a.grad) launch_on(balance_kernel<T, SIG, true, true>, grid, block, t.L, a);
    else if (a.loss) launch_on(balance_kernel<T, SIG, true, false>, grid, block, t.L, a);
    else launch_on(balance_kernel<T, SIG, false, true>, grid, block, t.L, a);
}
template <int T> void balance_launch(const BalArgs &a, int score, const Ctx &c) {
    if (score == LRS_SCORE_SIGMOID) balance_launch<T, true>(a, c);
    else balance_launch<T, false>(a, c);
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
    if (index_bytes != 4 && index_bytes != 8) return LRS_ERR_DTYPE;
    if (rows < 0 || k < 0 || experts < 1 || experts > LRS_MAX_EXPERTS || !stride_ok(index_stride, rows) ||
        rows > INT32_MAX || (k > 0 && rows > INT32_MAX / k))
        return LRS_ERR_SIZE;
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
    return balance_blocks(rows) * sizeof(double);
}

int expert_balance(const void *logits, int64_t row_stride, const int32_t *counts, const int32_t *rows_counted,
                   const uint8_t *row_mask, int64_t rows, int64_t experts, int dtype, int score, float balance_weight,
                   float z_weight, float *loss, const float *loss_grad, void *grad, int64_t grad_stride, void *workspace,
                   size_t workspace_bytes, void *stream, const lrs_options *opts) try {
    Ctx c;
    if (!make_ctx(stream, opts, c)) return LRS_ERR_OPTION;
    if (!row_type_ok(dtype)) return LRS_ERR_DTYPE;
    if ((score != LRS_SCORE_SOFTMAX && score != LRS_SCORE_SIGMOID) || !std::isfinite(balance_weight) ||
        !std::isfinite(z_weight) || (score == LRS_SCORE_SIGMOID && z_weight != 0.f))
        return LRS_ERR_OPTION;
    if (rows < 0 || rows > INT32_MAX || experts < 1 || experts > LRS_MAX_EXPERTS || !stride_ok(row_stride, rows) ||
        (grad && (!stride_ok(grad_stride, rows) || (rows > 1 && grad_stride < experts))))
        return LRS_ERR_SIZE;
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
    a.blocks = balance_blocks(a.rows);
    a.loss = loss;
    a.loss_grad = loss_grad;
    a.grad = grad;
    a.grad_stride = static_cast<uint64_t>(grad_stride);
    c.elems = a.rows * a.experts;
    if (rows > 0) {
        if (dtype == LRS_DTYPE_FP16) balance_launch<kRowF16>(a, score, c);
        else if (dtype == LRS_DTYPE_BF16) balance_launch<kRowBF16>(a, score, c);
        else balance_launch<kRowF32>(a, score, c);
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
    }
    if (loss) {
        TimedLaunch t(4, c);
        launch_on(balance_loss_kernel, dim3(1), dim3(kBalBlock), t.L, a);
        if (hipGetLastError() != hipSuccess) return LRS_ERR_HIP;
    }
    return LRS_OK;
} catch (...) {
    return LRS_ERR_HIP;
}

}  // extern "C"
