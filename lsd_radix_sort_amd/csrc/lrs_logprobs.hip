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
// A thread's terms are summed in 32 bits within one batch of loads and in 64
// bits from there on, as is everything there is once a row: an entropy is the
// difference of two numbers that nearly cancel.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>

#include "../../include/lsd_radix_sort.h"
#include "lrs_host.h"
#include "lrs_rows.h"

namespace lrs {
namespace {

constexpr int kLogBlock = 256;
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
    double inv_t;
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
    double *row_log;      // [rows][2]: m and log2 Z, for the top k
};

__device__ inline int64_t token_of(const LogArgs &a, uint64_t row) {
    const uint64_t at = row * a.token_stride;
    return a.token_bytes == 8 ? static_cast<const int64_t *>(a.tokens)[at] : static_cast<const int32_t *>(a.tokens)[at];
}
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

// The row order of a 32-bit pattern as a signed number.
__device__ inline int image_of_bits(uint32_t bits) {
    const int v = static_cast<int>(bits);
    return v ^ ((v >> 31) & 0x7FFFFFFF);
}
// The pattern of an element, in the high bits where it has 16.
template <int T> __device__ inline uint32_t high_bits(typename Row<T>::Stored v) {
    return T == kRowF32 ? v : static_cast<uint32_t>(v) << 16;
}

// One workgroup: the sums over a piece of a row.
template <int T, bool RANK>
__global__ __launch_bounds__(kLogBlock) void logprob_sum_kernel(LogArgs a) {
    constexpr int kVec = Row<T>::kVec;
    constexpr int kBatch = 4;
    constexpr int kWaves = kLogBlock / kLanes;
    using Stored = typename Row<T>::Stored;
    __shared__ double wz[kWaves], ww[kWaves];
    __shared__ float wm[kWaves];
    __shared__ uint32_t wb[kWaves];
    const float c = a.c;
    for (uint64_t task = blockIdx.x; task < a.rows * a.splits; task += gridDim.x) {
        const uint64_t row = task / a.splits;
        const uint32_t first = static_cast<uint32_t>(task % a.splits) * a.split_len;
        const uint32_t len = min(a.n - first, a.split_len), vecs = len / kVec;
        const Stored *x = static_cast<const Stored *>(a.logits) + row * a.stride + first;
        float m = kLowest;
        double z = 0, w = 0;
        uint32_t before = 0;
        if (counted(a, row)) {
            const int64_t token = RANK ? token_of(a, row) : -1;
            const bool given = token >= 0 && token < a.n;
            int mine = 0;
            if (RANK && given) mine = image_of_bits(high_bits<T>((x - first)[token]));
            const auto count = [&](Stored v, uint32_t at) {
                const int img = image_of_bits(high_bits<T>(v));
                before += img > mine || (img == mine && first + at < token);
            };
            const auto sum = [&](const float *f, int n) {
                float top = m;
                for (int e = 0; e < n; ++e) top = larger(top, f[e]);
                rebase(z, w, m, top, c);
                m = top;
                float part = 0, part_w = 0;
                for (int e = 0; e < n; ++e) {
                    const float d = (f[e] - m) * c, p = __builtin_amdgcn_exp2f(d);
                    part += p;
                    part_w = fmaf(p, fmaxf(d, kZeroBelow), part_w);
                }
                z += part;
                w += part_w;
            };
            for (uint32_t v = threadIdx.x; v < vecs; v += kBatch * kLogBlock) {
                u32x4 t[kBatch];
                float f[kBatch * kVec];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const uint32_t at = min(v + u * kLogBlock, vecs - 1);
                    t[u] = load16(x + static_cast<uint64_t>(at) * kVec);
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const uint32_t at = v + u * kLogBlock;
                    float g[kVec];
                    unpack16<T>(t[u], g);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        f[u * kVec + e] = at < vecs ? g[e] : -INFINITY;
                        if (RANK && given && at < vecs)
                            count(T == kRowF32 ? t[u][e % 4] : static_cast<Stored>(t[u][e / 2] >> (16 * (e & 1))), at * kVec + e);
                    }
                }
                sum(f, kBatch * kVec);
            }
            const uint32_t rest = vecs * kVec + threadIdx.x;
            if (rest < len) {
                const float f = Row<T>::value(x[rest]);
                if (RANK && given) count(x[rest], rest);
                sum(&f, 1);
            }
        }
        // the threads' sums, relative to the largest logit of all
        const auto join = [](float p, float q) { return larger(p, q); };
        float top = wave_join(m, kLowest, join);
        __syncthreads();
        if (threadIdx.x % kLanes == 0) wm[threadIdx.x / kLanes] = top;
        __syncthreads();
        for (int i = 0; i < kWaves; ++i) top = larger(top, wm[i]);
        rebase(z, w, m, top, c);
        z = wave_sum(z);
        w = wave_sum(w);
        before = wave_sum(before);
        if (threadIdx.x % kLanes == 0) {
            wz[threadIdx.x / kLanes] = z;
            ww[threadIdx.x / kLanes] = w;
            wb[threadIdx.x / kLanes] = before;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kWaves; ++i) {
                z += wz[i];
                w += ww[i];
                before += wb[i];
            }
            a.sums[task] = Sums{z, w, top, before};
        }
    }
}

// What a row's sums say: a thread's whole work.
template <int T> __device__ inline void finish_row(const LogArgs &a, uint64_t row, double z, double w, float m, uint32_t before) {
    using Stored = typename Row<T>::Stored;
    const bool on = counted(a, row), empty = z == 0;
    const int64_t token = token_of(a, row);
    const bool given = token >= 0 && token < a.n;
    const double low = log2(z), mean = w / z;
    double logprob = 0, entropy = 0;
    if (on) {
        entropy = empty ? 0 : kLn2 * (low - mean);
        if (given) {
            const float x = Row<T>::value(static_cast<const Stored *>(a.logits)[row * a.stride + token]);
            logprob = empty ? -INFINITY : kLn2 * ((static_cast<double>(x) - m) * a.factor - low);
        }
    }
    a.logprobs[row] = static_cast<float>(logprob);
    a.entropy[row] = static_cast<float>(entropy);
    if (a.ranks) a.ranks[row] = given ? static_cast<int32_t>(before) : -1;
    if (a.stats) {
        float *s = a.stats + row * kLogStats;
        s[0] = m;
        s[1] = !on || empty ? 0.f : static_cast<float>(1 / z);
        s[2] = !on || empty ? 0.f : static_cast<float>(mean);
    }
    if (a.row_log) {
        a.row_log[2 * row] = m;
        a.row_log[2 * row + 1] = empty ? INFINITY : low;
    }
}

// One wave a row: the pieces' sums joined.
template <int T>
__global__ __launch_bounds__(kLanes) void logprob_row_kernel(LogArgs a) {
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
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
        if (threadIdx.x == 0) finish_row<T>(a, row, z, w, m, before);
    }
}

// Patterns of the top logits to log probabilities.
template <int T>
__global__ __launch_bounds__(kLogBlock) void logprob_top_kernel(LogArgs a) {
    const uint64_t all = a.rows * a.k;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kLogBlock + threadIdx.x; i < all;
         i += static_cast<uint64_t>(gridDim.x) * kLogBlock) {
        const double *of = a.row_log + 2 * (i / a.k);
        const double x = Row<T>::value(static_cast<const typename Row<T>::Stored *>(a.top_values)[i]);
        a.top_logprobs[i] = static_cast<float>(kLn2 * ((x - of[0]) * a.factor - of[1]));
    }
}

// One workgroup: the gradient of a piece of a row.
template <int T>
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
        const float up = a.up && given ? a.up[row] : 0.f, down = a.up_entropy ? a.up_entropy[row] : 0.f;
        const float *s = a.stats + row * kLogStats;
        if (!counted(a, row) || s[1] == 0.f || (up == 0.f && down == 0.f)) {  // whatever its logits hold
            for (uint32_t v = threadIdx.x; v < vecs; v += kLogBlock) store16(g + static_cast<uint64_t>(v) * kVec, u32x4{0, 0, 0, 0});
            if (rest < len) g[rest] = 0;
            continue;
        }
        const float inv_t = static_cast<float>(a.inv_t), m = s[0], share = -s[1] * inv_t, mean = s[2];
        const float slope = down * static_cast<float>(kLn2);
        // p (a + b ln2 (d - D)), and what the given token has besides
        const uint32_t own = given && token >= first && token < first + len ? static_cast<uint32_t>(token - first) : ~0u;
        const auto of = [&](float f, uint32_t at) {
            const float d = (f - m) * c;
            const float v = __builtin_amdgcn_exp2f(d) * share * fmaf(slope, fmaxf(d, kZeroBelow) - mean, up);
            return at == own ? fmaf(up, inv_t, v) : v;
        };
        for (uint32_t v = threadIdx.x; v < vecs; v += kLogBlock) {
            float e[kVec];
            unpack16<T>(load16(x + static_cast<uint64_t>(v) * kVec), e);
            for (int i = 0; i < kVec; ++i) e[i] = of(e[i], v * kVec + i);
            store16(g + static_cast<uint64_t>(v) * kVec, pack16<T>(e));
        }
        if (rest < len) g[rest] = Row<T>::pattern(of(Row<T>::value(x[rest]), rest));
    }
}

// -------------------------------------------------------------------- host

constexpr uint64_t kMaxGrid = 1u << 20;

// How many workgroups share a row: enough that few rows still fill the GPU,
// each with a piece worth a workgroup.
void logprob_split(uint64_t rows, uint64_t n, uint32_t &splits, uint32_t &len) {
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
    uint64_t sums = 0, stats = 0, row_log = 0, values = 0, sort = 0, sort_bytes = 0, total = 0;
};
LogSpace logprob_space(uint64_t rows, uint64_t n, uint64_t k, int dtype) {
    LogSpace w;
    if (rows == 0) return w;
    uint32_t splits, len;
    logprob_split(rows, n, splits, len);
    auto place = [&](uint64_t bytes) {
        const uint64_t at = w.total;
        w.total += (bytes + 255) / 256 * 256;
        return at;
    };
    w.sums = place(rows * splits * sizeof(Sums));
    w.stats = place(rows * kLogStats * sizeof(float));
    if (k > 0) {
        w.row_log = place(rows * 2 * sizeof(double));
        w.values = place(rows * k * row_type_size(dtype));
        w.sort_bytes = segmented_row_topk_workspace_size(rows, n, k, dtype, nullptr);
        w.sort = place(w.sort_bytes);
    }
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
    a.inv_t = 1.0 / d->temperature;
    a.factor = kLog2e * a.inv_t;
    // above 0, so that -inf times it is -inf
    a.c = std::max(static_cast<float>(a.factor), std::numeric_limits<float>::denorm_min());
    a.k = static_cast<uint32_t>(k);
    logprob_split(a.rows, a.n, a.splits, a.split_len);
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

int logprob_sums(const LogArgs &a, int dtype, const Ctx &c) {
    if (a.rows == 0) return LRS_OK;
    {
        TimedLaunch t(4, c);
        by_type(dtype, [&](auto i) {
            launch_on(a.ranks ? logprob_sum_kernel<i.value, true> : logprob_sum_kernel<i.value, false>, grid_of(a.rows * a.splits),
                      dim3(kLogBlock), t.L, a);
        });
    }
    if (!launched()) return LRS_ERR_HIP;
    TimedLaunch t(4, c);
    by_type(dtype, [&](auto i) { launch_on(logprob_row_kernel<i.value>, grid_of(a.rows), dim3(kLanes), t.L, a); });
    return launched() ? LRS_OK : LRS_ERR_HIP;
}
int logprob_gradient(const LogArgs &a, int dtype, const Ctx &c) {
    if (a.rows == 0 || a.n == 0) return LRS_OK;
    TimedLaunch t(4, c);
    by_type(dtype, [&](auto i) { launch_on(logprob_grad_kernel<i.value>, grid_of(a.rows * a.splits), dim3(kLogBlock), t.L, a); });
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
    return logprob_sums(a, in->dtype, c);
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
    if (!logprobs || !entropy || !ranks || (k > 0 && (!top_logprobs || !top_indices)) || !workspace) return LRS_ERR_NULL_POINTER;
    if (misaligned(logprobs, 4) || misaligned(entropy, 4) || misaligned(ranks, 4) || misaligned(top_logprobs, 4) ||
        misaligned(top_indices, 8) || misaligned(workspace, 256))
        return LRS_ERR_ALIGNMENT;
    if (workspace_bytes < w.total) return LRS_ERR_WORKSPACE_TOO_SMALL;
    const void *const out[] = {logprobs, entropy, ranks, top_logprobs, top_indices, workspace};
    const uint64_t bytes[] = {4 * a.rows, 4 * a.rows, 4 * a.rows, 4 * a.rows * a.k, 8 * a.rows * a.k, w.total};
    if (aliased(in, out, bytes)) return LRS_ERR_ALIASING;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.sums = reinterpret_cast<Sums *>(ws + w.sums);
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.ranks = ranks;
    a.row_log = k > 0 ? reinterpret_cast<double *>(ws + w.row_log) : nullptr;
    c.elems = a.rows * a.n;
    int fs = logprob_sums(a, in->dtype, c);
    if (fs != LRS_OK || k == 0) return fs;
    fs = segmented_row_topk(a.logits, in->row_stride, ws + w.values, top_indices, in->rows, in->n, k, in->dtype, 1, ws + w.sort,
                            w.sort_bytes, stream, opts);
    if (fs != LRS_OK) return fs;
    a.top_values = ws + w.values;
    a.top_logprobs = top_logprobs;
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
    a.stats = reinterpret_cast<float *>(ws + w.stats);
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.up = logprob_grad;
    a.up_entropy = entropy_grad;
    a.grad = grad;
    a.grad_stride = grad_stride;
    c.elems = a.rows * a.n;
    const int fs = logprob_sums(a, in->dtype, c);
    return fs != LRS_OK ? fs : logprob_gradient(a, in->dtype, c);
} catch (...) {
    return LRS_ERR_HIP;
}

}  // extern "C"
